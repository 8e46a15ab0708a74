"""4-bit group-scaled weights and 8-bit checkpoints at the edges of their formulas.  Formats, references and
bounds as in test_int4.py."""
import ctypes

import numpy as np
import pytest
import torch

from dit_weight_compression_tile_b200 import binding as B
from dit_weight_compression_tile_b200.linear import GroupedINT4Linear, int4_group_linear
from test_int4 import BF, HF, SHAPES, case, check, load, pack_ref, per_input, scale_grad_ref, store


def same_infinities(got, want):
    """NaN where the formula (in float64) is NaN, and its infinities; returns where it is finite"""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:8]
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    return np.isfinite(want)


# one CTA a tile, the contraction split over a cluster, pairs of CTAs; k ends inside a group, a word, a tile
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", [(3, 150, 129, 128), (20, 150, 33, 32), (40, 130, 200, 64), (100, 140, 100, 128),
                                         (600, 150, 70, 32), (1100, 40, 1, 64), (130, 2304, 1089, 64),
                                         (300, 2304, 1230, 128)])
def test_scale_grad_of_infinite_gradients(m, n, k, group, dtype):
    """infinite gradients meet the real inputs only, not the zeros behind the last"""
    q, _, _, x = case(n, k, group, dtype, 2, m)
    q[5:9] = np.abs(q[5:9]) + 1 - 9 * (q[5:9] == 8)
    q[5:9] = np.where(q[5:9] == 0, 1, np.minimum(np.abs(q[5:9]), 7))
    x = x.abs() + 0.5  # no code is 0
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(dtype)
    dy[0, 5] = dy[m - 1, 12] = float("inf")  # feature 12: codes of both signs and zeros
    dy[m // 2, 6] = float("-inf")
    dy[0, 7], dy[m - 1, 7] = float("inf"), float("-inf")
    dy[1, 8] = float("nan")
    c, a = pack_ref(x)
    assert (c[:, :k] > 0).all()
    ds = B.int4_scale_grad(dy.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(a).cuda(), store(q).cuda(), k,
                           group=group).cpu()
    with np.errstate(invalid="ignore"):
        ref, mag, sub = scale_grad_ref(dy, c, a, q, k, group)
    assert (ref[5] == np.inf).all() and (ref[6] == -np.inf).all() and np.isnan(ref[7:9]).all()
    fine = same_infinities(ds, ref)
    rows = fine.all(1)
    assert rows.sum() == n - 5
    check(ds[torch.from_numpy(rows)], ref[rows], mag[rows], sub[rows], m + group, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,k,group", [(150, 1, 32), (150, 200, 64), (130, 1027, 128), (5100, 330, 32), (40, 72, 64)])
@pytest.mark.parametrize("m", [1, 2, 9, 16, 17, 40, 300])
def test_infinite_scales(m, n, k, group, dtype):
    """an infinite scale spoils its feature as the formula does: inf where all of its products have one sign, NaN
    where one is 0 or two differ"""
    q, _, s, x = case(n, k, group, dtype, 4, m)
    x = x.abs() + 0.25
    q[:3] = np.where(q[:3] == 0, 1, np.minimum(np.abs(q[:3]), 7))
    q[3, :] = 2
    q[3, k - 1] = 0
    s[0, 0] = s[1, -1] = s[3, -1] = s[10, 0] = float("inf")
    s[2, 0] = float("-inf")
    if m > 1:
        x[1, 0] = 0
    with np.errstate(invalid="ignore"):
        w = q * per_input(s, group, k)
        xd = x.double().numpy()
        ref = np.stack([(xd * w[o]).sum(1) for o in (0, 1, 2, 3, 10)], 1)
    assert ref[0, 0] == np.inf and ref[0, 1] == np.inf and ref[0, 2] == -np.inf and np.isnan(ref[0, 3])
    y = B.int4_linear(x.cuda(), store(q).cuda(), s.cuda(), group=group).cpu()
    same_infinities(y[:, [0, 1, 2, 3, 10]], ref)
    rest = [o for o in range(n) if o not in (0, 1, 2, 3, 10)]
    y0, mag = xd @ w[rest].T, np.abs(xd) @ np.abs(w[rest]).T
    check(y[:, rest], y0, mag, np.abs(xd).sum(1, keepdims=True), k, dtype)
    dy = torch.from_numpy(np.random.default_rng(1).normal(size=(m, n))).to(dtype).abs() + 0.25
    with np.errstate(invalid="ignore"):
        want = (dy.double().numpy()[:, :, None] * w[None, :, :min(k, 64)]).sum(1) if n < 1000 else None
    if want is not None:
        dx = B.int4_linear_dx(dy.cuda(), store(q).cuda(), s.cuda(), k, group=group).cpu()
        same_infinities(dx[:, :min(k, 64)], want)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("k,group", [(512, 128), (300, 64), (131, 32)])
def test_large_activations_under_small_scales(m, k, group):
    """BF16 activations whose sums of x q pass fp32's range before the scale, and not after it"""
    n = 70
    q, codes, s, x = case(n, k, group, BF, 11, m)
    x = (x.double().clamp(-3, 3) * 1e38).to(BF)
    bias = torch.ones(n, dtype=BF)
    y = B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group, bias=bias.cuda())
    xd, w = x.double().numpy(), q * per_input(s, group, k)
    ref, mag = xd @ w.T + 1, np.abs(xd) @ np.abs(w).T + 1
    assert np.abs(ref).max() < 3e38  # the result is in range
    check(y, ref, mag, np.abs(xd).sum(1, keepdims=True), k + 1, BF)


def test_package_names_follow_their_modules(monkeypatch):
    """a function replaced in its module is what the package gives from then on, used before or not"""
    import dit_weight_compression_tile_b200 as ep
    from dit_weight_compression_tile_b200 import compressed, linear
    for module, name in ((B, "decompress"), (B, "lib"), (compressed, "TileANSConfig"), (linear, "CompressedLinear")):
        old = getattr(ep, name)
        assert old is getattr(module, name)
        monkeypatch.setattr(module, name, lambda: None)
        assert getattr(ep, name) is getattr(module, name) is not old
        monkeypatch.undo()
        assert getattr(ep, name) is old
    assert ep.int4_linear is B.int4_linear and ep.int4_group_linear is linear.int4_group_linear


def _host_forward(monkeypatch):
    """the layer's launch replaced by host arithmetic that writes through an address, as a kernel does"""
    def forward(x, codes, scales, group, bias, checkpoint, *status):
        w = torch.from_numpy(load(codes, x.shape[1]) * per_input(scales.detach(), group, x.shape[1]))
        y = x.new_empty((x.shape[0], codes.shape[0]))
        full = (x.detach().double() @ w.T).to(x.dtype)
        ctypes.memmove(y.data_ptr(), full.data_ptr(), 2 * int(y.numel()))
        return y, None
    monkeypatch.setattr(B, "int4_layer_forward", forward)


@pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning")
def test_a_trace_records_the_call(monkeypatch):
    _host_forward(monkeypatch)
    q, codes, s, x = case(9, 70, 32, BF, 0, 4)
    layer = GroupedINT4Linear(70, 9, bias=False, group=32)
    layer.codes.copy_(codes)
    layer.scales.data.copy_(s)
    other = x.flip(0)[:3].contiguous() * 2
    want, want_other = layer(x), layer(other)
    for grad in (False, True):  # of a frozen layer, without and with a gradient asked for
        with torch.set_grad_enabled(grad):
            traced = torch.jit.trace(layer, (x,), check_trace=False)
            assert torch.equal(traced(x), want) and torch.equal(traced(other), want_other)


@pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning")
def test_calls_without_a_function_refuse_a_trace():
    q, codes, s, x = case(8, 64, 32, BF, 0, 3)
    act, a = torch.zeros(3, 64, dtype=torch.int8), torch.ones(3, 1)
    for call in (lambda t: B.int4_linear(t, codes, s, group=32), lambda t: B.int4_linear_dx(t[:, :8], codes, s, 64, group=32),
                 lambda t: B.int4_quantize(t, 32)[0], lambda t: B.act8_pack(t)[0],
                 lambda t: B.int4_scale_grad(t[:, :8], act, a, codes, 64, group=32),
                 lambda t: B.act8_unpack(act, a, 64) + t, lambda t: B.int4_dequantize(codes, s, 64, 32) + t[:1]):
        with pytest.raises(B.EpError, match="traced"):
            torch.jit.trace(call, (x,), check_trace=False)


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning")
@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("m", [3, 40])
def test_a_traced_layer_computes(m, train):
    torch.manual_seed(0)
    layer = GroupedINT4Linear.from_linear(torch.nn.Linear(256, 96, dtype=BF, device="cuda"), group=64, train_scales=train)
    x, other = torch.randn(m, 256, device="cuda").to(BF), torch.randn(2, m + 1, 256, device="cuda").to(BF)
    for grad in (False, True):
        with torch.set_grad_enabled(grad):
            traced = torch.jit.trace(layer, (x,), check_trace=False)
            y = traced(x)
            assert torch.equal(y, layer(x)) and torch.equal(traced(other), layer(other))
            if grad and train:
                ds, want = (torch.autograd.grad(f(x), layer.scales, torch.ones_like(y))[0] for f in (traced, layer))
                assert torch.equal(ds, want)


# ---------------------------------------------------------------- waits that run out are reported
def test_status_is_no_part_of_a_checkpoint():
    layer = GroupedINT4Linear(70, 9, group=32)
    assert layer.status.dtype == torch.int32 and layer.status.tolist() == [0]
    assert set(layer.state_dict()) == {"codes", "scales", "bias"}
    layer.status.fill_(7)  # as after to_empty
    layer.load_state_dict(layer.state_dict())
    assert layer.status.tolist() == [0]
    del layer._buffers["status"]  # as unpickled from before it had one
    layer.load_state_dict(layer.state_dict())
    with pytest.raises(B.EpError):
        layer(torch.zeros(2, 70, dtype=BF))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40])
def test_every_product_of_a_layer_reports_its_waits(m, monkeypatch):
    """the layer's status word reaches each launch that waits, is left alone by those that end, and keeps its bits"""
    layer = GroupedINT4Linear.from_linear(torch.nn.Linear(96, 72, dtype=BF, device="cuda"), group=32, train_scales=True)
    own, given, real = layer.status.data_ptr(), {}, B.lib()

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                given.setdefault(name, []).append(args[-2])
                return getattr(real, name)(*args)
            return call if name in ("ep_int4_linear", "ep_int4_linear_dx", "ep_int4_scale_grad") else getattr(real, name)

    monkeypatch.setattr(B, "lib", Recorder)
    x = torch.randn(m, 96, device="cuda").to(BF).requires_grad_(True)
    layer(x).sum().backward()
    with torch.no_grad():
        layer(x)
    assert given == {"ep_int4_linear": [own, own], "ep_int4_linear_dx": [own], "ep_int4_scale_grad": [own]}
    assert layer.status.tolist() == [0]
    layer.status.fill_(32)
    layer(x).sum().backward()
    assert layer.status.tolist() == [32]
    given.clear()
    y = int4_group_linear(x, layer.codes, layer.scales, group=32)
    torch.autograd.grad(y, (x, layer.scales), torch.ones_like(y))
    assert given == {"ep_int4_linear": [None], "ep_int4_linear_dx": [None], "ep_int4_scale_grad": [None]}
    for bad in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32),
                torch.zeros(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(B.EpError):
            int4_group_linear(x, layer.codes, layer.scales, group=32, status=bad)


# ---------------------------------------------------------------- products of small integers: no tolerance
# Tokens and gradients of -1, 0, 1 and scales of the type's full length in [1/4, 1/2): every sum below is a multiple
# of 2^-9 (BF16) or 2^-12 (FP16) and below 2^10 (8192 terms of at most 4, whose random sum has a deviation of 2^7),
# 22 bits: fp32 holds each one exactly in any order, and the only roundings are the documented ones.  (The checkpoint's
# scales are powers of two: a c is exact.  Its sums are multiples of 1/2 below 2^15.)
EXACT = SHAPES + [(2048, 8192, 8192, 128), (17, 8192, 8192, 128), (48, 4096, 4096, 64), (1030, 4090, 4100, 32)]


def signs(rows, cols, seed):
    """-1, 0 or 1, and no zero in the last row and the last column, which a ragged tile would lose first"""
    v = torch.from_numpy(np.random.default_rng(seed).integers(-1, 2, (rows, cols)))
    v[-1] = torch.where(v[-1] == 0, 1 - 2 * (torch.arange(cols) % 2), v[-1])
    v[:, -1] = torch.where(v[:, -1] == 0, -1, v[:, -1])
    return v.cuda()


def exact_weight(n, k, group, dtype, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(-8, 8, (n, k))
    q[-1, :], q[:, -1] = np.where(q[-1] == 0, 3, q[-1]), np.where(q[:, -1] == 0, -5, q[:, -1])
    bits = 7 if dtype == BF else 10
    s = torch.from_numpy(rng.integers(2 ** bits, 2 ** (bits + 1), (n, -(-k // group))) * 2.0 ** -(bits + 2)).to(dtype)
    w = torch.from_numpy(q).cuda().double() * s.cuda().double().repeat_interleave(group, 1)[:, :k]
    return store(q).cuda(), s.cuda(), w, torch.from_numpy(q).cuda()


def assert_exact(call, want, dtype, mag=None, terms=0, limit=2 ** 11, times=3):
    """equal to the sum rounded once; a sum that fp32 cannot hold (FP16's multiples of 2^-12 from 2^12 on: 24 bits, one
    left for the sums on its way) is off by at most 2^-23 of the magnitudes' sum for each term.  (Weights and tokens of
    one seed, where n = k, agree in sign along the diagonal: 8192 terms of 1.3 on average make 11000 there.)"""
    exact = want.abs() < limit
    assert want.abs().max() < 2 ** 15 and exact.float().mean() > 0.99
    out = want.float().to(dtype)
    for _ in range(times):
        got = call()
        assert got.dtype == dtype and torch.equal(got[exact], out[exact]), int((got != out)[exact].sum())
        if not exact.all():
            u, err = torch.finfo(dtype).eps / 2, (got.double() - want).abs()
            assert (err <= u * want.abs() + (1 + u) * terms * 2.0 ** -23 * mag)[~exact].all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", EXACT)
def test_linear_of_integers(m, n, k, group, dtype):
    codes, s, w, _ = exact_weight(n, k, group, dtype, m + n)
    x = signs(m, k, m + k)
    bias = signs(1, n, n)[0].to(dtype) if n % 2 == 0 else None
    # up to 16 tokens the weight is exact, above its entries are rounded to the type
    want, mag = x.double() @ (w if m <= 16 else w.to(dtype).double()).T, x.double().abs() @ w.abs().T
    want = want if bias is None else want + bias.double()
    x = x.to(dtype)
    assert_exact(lambda: B.int4_linear(x, codes, s, group=group, bias=bias), want, dtype, mag + 1, k + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m", [1, 8, 9, 16])
@pytest.mark.parametrize("n,k,group", [(6001, 392, 32), (9000, 256, 128), (5100, 387, 32), (7000, 70, 64), (300, 672, 32),
                                       (1000, 257, 128), (1000, 384, 64), (64, 8200, 128)])
def test_few_tokens_of_integers(m, n, k, group, dtype):
    codes, s, w, _ = exact_weight(n, k, group, dtype, m + n)
    x = signs(m, k, m + k)
    assert_exact(lambda: B.int4_linear(x.to(dtype), codes, s, group=group), x.double() @ w.T, dtype,
                 x.double().abs() @ w.abs().T, k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", EXACT)
def test_input_grad_of_integers(m, n, k, group, dtype):
    codes, s, w, _ = exact_weight(n, k, group, dtype, m + n)
    dy = signs(m, n, m + n)
    want, mag = dy.double() @ w.to(dtype).double(), dy.double().abs() @ w.abs()
    dy = dy.to(dtype)
    assert_exact(lambda: B.int4_linear_dx(dy, codes, s, k, group=group), want, dtype, mag, n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", EXACT)
def test_scale_grad_of_integers(m, n, k, group, dtype):
    codes, _, _, q = exact_weight(n, k, group, dtype, m + n)
    dy, rng = signs(m, n, m + n), np.random.default_rng(k)
    c = np.zeros((m, -(-k // 16) * 16), np.int8)
    c[:, :k] = rng.integers(-3, 4, (m, k))
    c[-1, :k], c[:, k - 1] = np.where(c[-1, :k] == 0, 2, c[-1, :k]), np.where(c[:, k - 1] == 0, -1, c[:, k - 1])
    a = torch.from_numpy(2.0 ** rng.integers(-1, 1, (m, -(-k // 128)))).float().cuda()
    c = torch.from_numpy(c).cuda()
    p = (dy.double().T @ (c[:, :k].double() * a.double().repeat_interleave(128, 1)[:, :k])) * q
    want = torch.nn.functional.pad(p, (0, -k % group)).view(n, -1, group).sum(-1)
    dy = dy.to(dtype)
    assert_exact(lambda: B.int4_scale_grad(dy, c, a, codes, k, group=group), want, dtype, limit=2 ** 15)


@pytest.mark.gpu
def test_large_fp16_products():
    """the largest products in FP16 on real-valued inputs, against float64, the weight's rounding included"""
    m, n, k, group = 2048, 8192, 8192, 128
    torch.manual_seed(1)
    codes, s = B.int4_quantize(torch.randn(n, k, device="cuda") * 0.02, group, dtype=HF)
    x, dy = torch.randn(m, k, device="cuda").to(HF), (torch.randn(m, n, device="cuda") * 0.1).to(HF)
    w = B.int4_dequantize(codes, torch.ones_like(s), k, group).double() * s.double().repeat_interleave(group, 1)
    u, sub = 2.0 ** -11, 2.0 ** -25
    for got, t, v, terms in ((B.int4_linear(x, codes, s, group=group), x.double(), w.T, k),
                             (B.int4_linear_dx(dy, codes, s, k, group=group), dy.double(), w, n)):
        ref, mag, rms = t @ v, t.abs() @ v.abs(), (t.square() @ v.square()).sqrt()
        err, out = (got.double() - ref).abs(), u * ref.abs() * (1 + 2 * u) + sub
        assert (err <= (u + terms * 2.0 ** -23) * (1 + 2 * u) * mag + out + sub * t.abs().sum(1, keepdim=True)).all()
        # a weight's rounding is off by at most u |w|, one independent of the next: their sum's deviation is at most
        # u rms (uniform ones: u rms / sqrt 3), of which 8 are passed with odds below 1e-14 for each of 2^24 results; the
        # accumulator's steps, 2^-23 of at most 8 rms each, add their number's root
        assert (err <= 8 * u * rms + 8 * terms ** 0.5 * 2.0 ** -23 * 8 * rms + out).all()
    act = B.act8_pack(x)
    ds = B.int4_scale_grad(dy, *act, codes, k, group=group)
    q = B.int4_dequantize(codes, torch.ones_like(s), k, group).double()
    c, a = act[0].double(), act[1].double().repeat_interleave(128, 1)
    fold = lambda p: p.view(n, -1, group).sum(-1)  # noqa: E731
    ref = fold((dy.double().T @ (c * a)) * q)
    rms = fold((dy.double().T.square() @ (c * a).square()) * q.square()).sqrt()
    terms = m + group
    # as above; a c by u (1 + 2^-1) of itself (its low part's product is rounded too)
    tol = 8 * 1.5 * u * rms + 8 * terms ** 0.5 * 2.0 ** -23 * 8 * rms + u * ref.abs() * (1 + 2 * u) + sub
    assert ((ds.double() - ref).abs() <= tol).all()


# ---------------------------------------------------------------- FP16's range, as the header states it
@pytest.mark.gpu
def test_fp16_weights_beyond_the_range():
    """|s q| from 65520 on: exact up to 16 tokens, infinite where the weight is rounded to FP16"""
    k, group = 64, 32
    q = np.ones((3, k), np.int64)
    q[:, 5] = -8
    s = torch.tensor([[8184.0, 1.0], [8192.0, 1.0], [1.0, 0.5]], dtype=HF)
    w = q * per_input(s, group, k)
    for m in (4, 20):
        x = torch.full((m, k), 2.0 ** -7, dtype=HF)
        y = B.int4_linear(x.cuda(), store(q).cuda(), s.cuda(), group=group).cpu().double()
        want = torch.from_numpy(x.double().numpy() @ w.T)
        if m > 16:
            want[:, 1] = float("-inf")
        assert torch.equal(y, want.to(HF).double())
    dx = B.int4_linear_dx(torch.full((2, 3), 2.0 ** -7, dtype=HF).cuda(), store(q).cuda(), s.cuda(), k, group=group).cpu()
    assert (dx[:, 5] == float("-inf")).all() and torch.isfinite(dx[:, [i for i in range(k) if i != 5]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("src", [BF, torch.float32])
def test_fp16_scale_gradients_of_wider_activations(src):
    """activations from 65520 on spoil their group, others up to 2^-25 add nothing; BF16 gradients take both"""
    m, n, k, group = 8, 40, 384, 128
    q = np.ones((n, k), np.int64)
    x = torch.zeros(m, k)
    x[:, :128], x[3, 40], x[:, 128:256], x[:, 256:] = 1.0, 1.0e5, 2.0 ** -27, 2.0 ** -26
    x[:, 256] = 2.0 ** -10  # a group's largest; its others are far below it
    act = B.act8_pack(x.to(src).cuda())
    dy = torch.ones(m, n, device="cuda")
    wide = B.int4_scale_grad(dy.to(BF), *act, store(q).cuda(), k, group=group).cpu()
    c, a = act[0].cpu().double(), act[1].cpu().double().repeat_interleave(128, 1)
    want = (c * a).view(m, 3, 128).sum((0, 2))
    assert ((wide.double() - want).abs() <= 2 * 2.0 ** -8 * (1 + 2.0 ** -8) * want).all()  # a c and the result rounded
    half = B.int4_scale_grad(dy.to(HF), *act, store(q).cuda(), k, group=group).cpu()
    assert not torch.isfinite(half[:, 0]).any() and (half[:, 1] == 0).all()
    assert ((half[:, 2].double() - m * 2.0 ** -10).abs() <= 2.0 ** -11 * m * 2.0 ** -10 * 2).all()


# ---------------------------------------------------------------- the forms with pairs of CTAs and with steps of 128
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", [(1100, 5100, 330, 32), (1100, 5100, 263, 128), (40, 5100, 1999, 32), (20, 5100, 1930, 64)])
def test_infinite_scales_of_wide_forms(m, n, k, group, dtype):
    test_infinite_scales(m, n, k, group, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", [(40, 5100, 1999, 32), (20, 5100, 1930, 64), (17, 19000, 1025, 32), (48, 5100, 1537, 128)])
def test_ragged_steps_of_128(m, n, k, group, dtype):
    test_linear_of_integers(m, n, k, group, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 9, 17])
def test_infinite_scales_of_the_smallest_and_largest_activations(m):
    n, k, group = 20, 300, 64
    q, _, s, x = case(n, k, group, BF, 12, m)
    q[0] = 3
    s[0, 1] = float("inf")
    x[0] = 2.0 ** -126
    x[m - 1, 290:] = 1e38  # in another group than the infinite scale's, sums of x q beyond fp32
    s[:, 4] = 2.0 ** -30
    x[m - 1, :290] = 2.0 ** -126
    w = q * per_input(s, group, k)
    with np.errstate(invalid="ignore"):
        ref = (x.double().numpy()[:, None, :] * w[None]).sum(2)
    y = B.int4_linear(x.cuda(), store(q).cuda(), s.cuda(), group=group).cpu()
    assert ref[0, 0] == np.inf == ref[m - 1, 0]
    same_infinities(y, ref)
    xd = x.double().numpy()
    check(y[:, 1:], ref[:, 1:], np.abs(xd) @ np.abs(w[1:]).T, np.abs(xd).sum(1, keepdims=True), k, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m", [1, 7, 16])
@pytest.mark.parametrize("n,k,group,at", [(150, 700, 64, 699), (6001, 392, 32, 0), (5100, 300, 128, 299), (64, 8200, 128, 8000)])
def test_tokens_with_nan_and_infinity_beside_others(m, n, k, group, at, dtype):
    """each token's outputs are the formula's whatever the others hold, NaN and infinity at either end"""
    q, codes, s, x = case(n, k, group, dtype, 13, m)
    clean = B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group).cpu()
    bad = x.clone()
    bad[0, at] = float("nan")
    if m > 1:
        bad[m - 1, at], bad[m // 2, at] = float("inf"), float("-inf")
    y = B.int4_linear(bad.cuda(), codes.cuda(), s.cuda(), group=group).cpu()
    assert torch.isnan(y[0]).all()
    rest = [t for t in range(1, m) if t not in (m - 1, m // 2)]
    assert torch.equal(y[rest], clean[rest])
    column = torch.from_numpy(q[:, at])
    for t, sign in ((m - 1, 1), (m // 2, -1)) if m > 1 else ():
        same_infinities(y[t], np.where(q[:, at] == 0, np.nan, np.copysign(np.inf, sign * column.double().numpy())))


@pytest.mark.gpu
def test_a_layer_given_its_tensors_on_the_meta_device():
    layer = GroupedINT4Linear.from_linear(torch.nn.Linear(96, 72, dtype=BF, device="cuda"), group=32)
    x = torch.randn(20, 96, device="cuda").to(BF)
    fresh = GroupedINT4Linear(96, 72, group=32, device="meta")
    fresh.load_state_dict(layer.state_dict(), assign=True)
    assert torch.equal(fresh(x), layer(x)) and fresh.status.device == x.device and fresh.status.tolist() == [0]
    empty = GroupedINT4Linear(96, 72, group=32, device="meta").to_empty(device="cuda")
    empty.load_state_dict(layer.state_dict())
    assert torch.equal(empty(x), layer(x)) and empty.status.tolist() == [0]
