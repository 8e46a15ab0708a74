"""4-bit group-scaled weights and 8-bit activation checkpoints (include/eptile_int4.h): the operators
against plain float64 arithmetic, their refusals, and the layer that uses them together.

Bounds, with u = finfo.eps / 2 of the 16-bit type: a product's operands are exact in fp32 except the
weight s q (or the checkpoint's a c), which may be rounded once to the type (u relative, 2^-25 absolute
where fp16 is subnormal); a sum of c products in fp32 in any order, each addition off by at most 2^-23
relative (the tensor cores may truncate), errs by at most c 2^-23 times the sum of magnitudes; the
result is rounded once (u, or 2^-25 absolute)."""
import copy
import ctypes as C
import io
import os
import subprocess
import sys

import numpy as np
import pytest
import torch
import torch.nn as nn

from dit_weight_compression_tile_b200 import binding as B
from dit_weight_compression_tile_b200.linear import GroupedINT4Linear, int4_group_linear

BF, HF = torch.bfloat16, torch.float16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
SUB = {BF: 2.0 ** -133, HF: 2.0 ** -25}  # half the smallest subnormal


# ---------------------------------------------------------------- the formats and formulas, in numpy
def store(q):
    """codes (n, k) as stored: a loop over the eight places of a word"""
    n, k = q.shape
    words = -(-k // 32) * 4
    full = np.zeros((n, words * 8), np.int64)
    full[:, :k] = q
    out = np.zeros((n, words), np.uint32)
    for e in range(8):
        bit = 4 * (e // 2) + 16 * (e % 2)
        out |= ((full[:, e::8] + 8).astype(np.uint32) << np.uint32(bit))
    return torch.from_numpy(out.view(np.uint8).reshape(n, words * 4).copy())


def load(codes, k):
    w = codes.cpu().numpy().reshape(codes.shape[0], -1).view(np.uint32)
    out = np.zeros((w.shape[0], w.shape[1] * 8), np.int64)
    for e in range(8):
        out[:, e::8] = ((w >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & np.uint32(15)).astype(np.int64) - 8
    return out[:, :k]


def per_input(scales, group, k):
    return np.repeat(scales.double().cpu().numpy(), group, axis=1)[:, :k]


def case(n, k, group, dtype, seed, m=None):
    """random codes over all sixteen values, scales of different size, some rows of zeros"""
    rng = np.random.default_rng(seed)
    q = rng.integers(-8, 8, (n, k))
    s = torch.from_numpy(rng.lognormal(-5.5, 0.5, (n, -(-k // group)))).to(dtype)
    if n > 4:
        q[3] = 0
    x = None if m is None else torch.from_numpy(rng.normal(size=(m, k))).to(dtype)
    return q, store(q), s, x


def forward_ref(x, q, s, group, bias):
    xd, w = x.double().cpu().numpy(), q * per_input(s, group, q.shape[1])
    y, mag = xd @ w.T, np.abs(xd) @ np.abs(w).T
    sub = np.abs(xd).sum(1, keepdims=True)
    if bias is not None:
        y, mag = y + bias.double().cpu().numpy(), mag + np.abs(bias.double().cpu().numpy())
    return y, mag, sub


def check(got, ref, mag, sub, terms, dtype):
    u, tiny = U[dtype], SUB[dtype]
    tol = (u + terms * 2.0 ** -23) * (1 + 2 * u) * mag + u * np.abs(ref) + tiny * (sub + 1)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert got.dtype == dtype and np.isfinite(err).all()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))


def pack_ref(x):
    """codes and scales of the definition: fp32 scale, quotient rounded exactly (float64 decides)"""
    xd = x.double().cpu().numpy()
    m, k = xd.shape
    g = -(-k // 128)
    pad = np.zeros((m, g * 128))
    pad[:, :k] = xd
    a = (np.abs(pad.reshape(m, g, 128)).max(-1).astype(np.float32) / np.float32(127)).astype(np.float32)
    a[a == 0] = 1
    c = np.clip(np.rint(pad.reshape(m, g, 128) / a.astype(np.float64)[..., None]), -127, 127).reshape(m, -1)
    return c[:, :-(-k // 16) * 16].astype(np.int8), a


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 1 << 20  # never dereferenced: the calls return before a launch


def test_refused_before_any_launch():
    L = B.lib()

    def linear(codes=FAKE, scales=FAKE, n=64, k=64, group=32, dtype=B.BF16, x=FAKE, m=4, ldx=64, bias=None, y=FAKE):
        return L.ep_int4_linear(codes, scales, n, k, group, dtype, x, m, ldx, bias, y, None, None)

    for bad in (dict(codes=None), dict(scales=None), dict(x=None), dict(y=None), dict(codes=FAKE + 8), dict(x=FAKE + 1),
                dict(y=FAKE + 1), dict(bias=FAKE + 1), dict(scales=FAKE + 1), dict(n=0), dict(k=0), dict(n=2 ** 30 + 1),
                dict(k=2 ** 30 + 1, ldx=2 ** 31), dict(group=16), dict(group=256), dict(group=0), dict(dtype=B.FP32),
                dict(dtype=B.INT8), dict(m=-1), dict(ldx=63)):
        assert linear(**bad) == -1, bad
    assert linear(m=0) == 0 and linear(m=0, x=None, y=None) == 0

    def dx(codes=FAKE, scales=FAKE, n=64, k=64, group=32, dtype=B.BF16, dy=FAKE, m=4, ld=64, out=FAKE):
        return L.ep_int4_linear_dx(codes, scales, n, k, group, dtype, dy, m, ld, out, None, None)

    for bad in (dict(codes=None), dict(scales=None), dict(dy=None), dict(out=None), dict(codes=FAKE + 4), dict(ld=32),
                dict(group=48), dict(dtype=B.FP32), dict(m=-2), dict(out=FAKE + 1), dict(dy=FAKE + 1)):
        assert dx(**bad) == -1, bad
    assert dx(m=0) == 0

    def sg(dy=FAKE, ld=64, act=FAKE, a=FAKE, m=4, codes=FAKE, n=64, k=64, group=32, dtype=B.BF16, out=FAKE):
        return L.ep_int4_scale_grad(dy, ld, act, a, m, codes, n, k, group, dtype, out, None, None)

    for bad in (dict(dy=None), dict(act=None), dict(a=None), dict(codes=None), dict(out=None), dict(act=FAKE + 8),
                dict(a=FAKE + 2), dict(ld=63), dict(group=0), dict(dtype=B.FP32), dict(m=-1)):
        assert sg(**bad) == -1, bad

    def pack(x=FAKE, dtype=B.BF16, m=4, k=64, ld=64, codes=FAKE, a=FAKE):
        return L.ep_act8_pack(x, dtype, m, k, ld, codes, a, None)

    for bad in (dict(x=None), dict(codes=None), dict(a=None), dict(dtype=B.INT8), dict(k=0), dict(m=-1), dict(ld=60),
                dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=B.FP32), dict(codes=FAKE + 8), dict(a=FAKE + 2)):
        assert pack(**bad) == -1, bad
    assert pack(m=0, x=None, codes=None, a=None) == 0
    assert L.ep_act8_unpack(None, FAKE, 4, 64, FAKE, B.BF16, None) == -1
    assert L.ep_act8_unpack(FAKE, FAKE, 4, 64, FAKE, B.INT8, None) == -1
    assert L.ep_act8_unpack(FAKE, FAKE, 0, 64, FAKE, B.BF16, None) == 0
    assert L.ep_int4_quantize(FAKE, B.BF16, 4, 64, 64, 32, FAKE, FAKE, B.FP32, None) == -1
    assert L.ep_int4_quantize(FAKE, B.BF16, 4, 64, 63, 32, FAKE, FAKE, B.BF16, None) == -1
    assert L.ep_int4_quantize(FAKE, B.BF16, 4, 64, 64, 96, FAKE, FAKE, B.BF16, None) == -1
    assert L.ep_int4_dequantize(FAKE, FAKE, B.FP32, 4, 64, 32, FAKE, None) == -1
    assert L.ep_int4_dequantize(FAKE, None, B.BF16, 4, 64, 32, FAKE, None) == -1


def test_sizes_beyond_the_limit_are_refused():
    L, big = B.lib(), 2 ** 30 + 1
    for m in (big, 2 ** 40):
        assert L.ep_int4_linear(FAKE, FAKE, 1, 32, 32, B.BF16, FAKE, m, 32, None, FAKE, None, None) == -1
        assert L.ep_int4_linear_dx(FAKE, FAKE, 1, 32, 32, B.BF16, FAKE, m, 1, FAKE, None, None) == -1
        assert L.ep_int4_scale_grad(FAKE, 1, FAKE, FAKE, m, FAKE, 1, 32, 32, B.BF16, FAKE, None, None) == -1
        assert L.ep_act8_pack(FAKE, B.BF16, m, 32, 32, FAKE, FAKE, None) == -1
        assert L.ep_act8_unpack(FAKE, FAKE, m, 32, FAKE, B.BF16, None) == -1
    assert L.ep_act8_pack(FAKE, B.BF16, 1, big, big, FAKE, FAKE, None) == -1
    assert L.ep_int4_quantize(FAKE, B.BF16, big, 32, 32, 32, FAKE, FAKE, B.BF16, None) == -1
    assert L.ep_int4_dequantize(FAKE, FAKE, B.BF16, 1, big, 32, FAKE, None) == -1


def test_binding_and_layer_refuse():
    q, codes, s, x = case(8, 64, 32, BF, 0, 3)
    for call in (lambda: B.int4_linear(x, codes, s, group=32), lambda: B.int4_quantize(x, 32), lambda: B.act8_pack(x),
                 lambda: B.int4_linear_dx(x[:, :8], codes, s, 64, group=32),
                 lambda: B.int4_dequantize(codes, s, 64, 32), lambda: B.int4_linear(x, codes, s, group=48),
                 lambda: B.int4_quantize(x.double(), 32), lambda: B.int4_quantize(x, 16),
                 lambda: B.act8_pack(x.to(torch.int32)), lambda: B.int4_linear(x[0], codes, s, group=32),
                 lambda: B.act8_unpack(torch.zeros(2, 64, dtype=torch.int8), torch.ones(2, 1), 64),
                 lambda: int4_group_linear(torch.tensor(1.0), codes, s, group=32),
                 lambda: GroupedINT4Linear(64, 8, group=16), lambda: GroupedINT4Linear(64, 8, dtype=torch.float32),
                 lambda: GroupedINT4Linear(0, 8), lambda: GroupedINT4Linear.from_linear(nn.Linear(64, 8, dtype=BF)),
                 lambda: GroupedINT4Linear(64, 8)(x)):  # host tensors: there is no CPU form
        with pytest.raises(B.EpError):
            call()


def test_layer_state_on_the_host():
    layer = GroupedINT4Linear(70, 9, group=32)
    assert layer.codes.shape == (9, 48) and layer.scales.shape == (9, 3) and not layer.scales.requires_grad
    assert (load(layer.codes, 96) == 0).all()  # a zero weight, padding included
    assert layer.stored_nbytes == 9 * 48 + 2 * 27 and layer.compressed_bits == 8 * layer.stored_nbytes / 630
    q, codes, s, _ = case(9, 70, 32, BF, 1)
    layer.codes.copy_(codes)
    layer.scales.data.copy_(s)
    buf = io.BytesIO()
    torch.save(layer.state_dict(), buf)
    buf.seek(0)
    fresh = GroupedINT4Linear(70, 9, group=32, train_scales=True)
    res = fresh.load_state_dict(torch.load(buf, weights_only=True))
    assert not res.missing_keys and not res.unexpected_keys
    assert torch.equal(fresh.codes, codes) and torch.equal(fresh.scales, s) and fresh.scales.requires_grad
    with pytest.raises(RuntimeError):
        GroupedINT4Linear(70, 9, group=64).load_state_dict(layer.state_dict())


# ---------------------------------------------------------------- the quantizers
@pytest.mark.gpu
@pytest.mark.parametrize("n,k,group,src,dtype", [(1, 1, 32, BF, BF), (5, 70, 32, torch.float32, BF), (33, 1027, 64, HF, HF),
                                                 (16, 512, 128, BF, BF), (7, 130, 128, torch.float32, HF),
                                                 (300, 96, 32, HF, BF)])
def test_quantize_and_dequantize(n, k, group, src, dtype):
    rng = np.random.default_rng(n * k)
    w = torch.from_numpy(rng.normal(size=(n, k)) * 0.02).to(src)
    if n > 4:
        w[2, :] = 0
        w[3] = torch.from_numpy(rng.integers(-14, 15, k)).to(src) / 2  # quotients on the halves
        w[3, 0] = 7.0
    codes, s = B.int4_quantize(w.cuda(), group, dtype=dtype)
    g = -(-k // group)
    pad = np.zeros((n, g * group), np.float32)
    pad[:, :k] = w.float().numpy()
    pad = pad.reshape(n, g, group)
    want = torch.from_numpy(np.abs(pad).max(-1) / np.float32(7)).to(dtype)
    want[want == 0] = 1
    assert torch.equal(s.cpu(), want)
    q = np.clip(np.rint(pad.astype(np.float64) / want.double().numpy()[..., None]), -7, 7).reshape(n, -1)[:, :k]
    assert np.array_equal(load(codes, k), q.astype(np.int64))
    assert (load(codes, codes.shape[1] * 2)[:, k:] == 0).all()
    back = B.int4_dequantize(codes, s, k, group)
    assert torch.equal(back.cpu(), (torch.from_numpy(q * per_input(s, group, k))).to(dtype))
    # a strided source gives the same
    wide = torch.zeros(n, k + 3, dtype=src).cuda()
    wide[:, 1:k + 1] = w.cuda()
    codes2, s2 = B.int4_quantize(wide[:, 1:k + 1], group, dtype=dtype)
    assert torch.equal(codes, codes2) and torch.equal(s, s2)


@pytest.mark.gpu
def test_quantize_marks_groups_without_a_scale():
    w = torch.full((3, 128), 0.5)
    w[0, 5], w[1, 40], w[2, 100] = float("nan"), float("inf"), 1e6  # 1e6 / 7 is beyond fp16
    codes, s = B.int4_quantize(w.cuda(), 32, dtype=HF)
    nan = torch.isnan(s.cpu())
    assert nan.tolist() == [[True, False, False, False], [False, True, False, False], [False, False, False, True]]
    assert (load(codes, 128).reshape(3, 4, 32)[nan.numpy()] == 0).all()
    layer = GroupedINT4Linear(128, 3, group=32, dtype=HF, device="cuda")
    with pytest.raises(B.EpError) as e:
        layer.quantize_weight(w.cuda())
    assert e.value.status == -2 and (layer.scales == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,dtype", [(1, 1, BF), (3, 130, HF), (5, 1027, HF), (17, 256, torch.float32), (64, 4096, BF),
                                       (2, 100, torch.float32), (1, 16, HF)])
def test_pack_and_unpack(m, k, dtype):
    rng = np.random.default_rng(m + k)
    x = rng.normal(size=(m, k))
    x[:, ::50] *= 30
    if m > 2:
        x[1] = 0
        x[2] = np.rint(x[2] * 20) / 2  # quotients on the halves: amax 127 / 2 gives a = 1 / 2
        x[2, ::128] = 127.0
    x = torch.from_numpy(x).to(dtype)
    codes, a = B.act8_pack(x.cuda())
    want_c, want_a = pack_ref(x)
    assert np.array_equal(a.cpu().numpy(), want_a) and np.array_equal(codes.cpu().numpy(), want_c)
    for out in (BF, HF, torch.float32):
        back = B.act8_unpack(codes, a, k, out)
        v = (want_c[:, :k].astype(np.float32) * np.repeat(want_a, 128, 1)[:, :k]).astype(np.float32)
        assert torch.equal(back.cpu(), torch.from_numpy(v).to(out))
    wide = torch.zeros(m, k + 5, dtype=dtype).cuda()
    wide[:, 3:k + 3] = x.cuda()
    codes2, a2 = B.act8_pack(wide[:, 3:k + 3])
    assert torch.equal(codes, codes2) and torch.equal(a, a2)


@pytest.mark.gpu
def test_pack_extremes():
    x = torch.zeros(6, 256)
    x[0, 3], x[1, 200], x[2, 7] = float("nan"), float("-inf"), 3.0e38
    x[3, :128] = torch.arange(128) * 1e-44  # subnormal scales
    x[4, 0] = 1e-45  # the scale itself rounds to 0
    x[5, 1] = -127.0
    codes, a = B.act8_pack(x.cuda())
    a, codes = a.cpu(), codes.cpu()
    assert torch.isnan(a[0, 0]) and torch.isnan(a[1, 1]) and int(torch.isnan(a).sum()) == 2
    assert (codes[0] == 0).all() and (codes[1] == 0).all()
    keep = torch.tensor([2, 3, 4, 5])
    want_c, want_a = pack_ref(x[keep])
    assert np.array_equal(a[keep].numpy(), want_a) and np.array_equal(codes[keep].numpy(), want_c)
    assert codes[5, 1] == -127 and a[4, 0] == 1


# ---------------------------------------------------------------- the products
SHAPES = [(1, 1, 1, 32), (1, 64, 64, 32), (1, 1024, 1024, 128), (1, 130, 257, 64), (2, 16, 4096, 128), (3, 100, 96, 32),
          (5, 2050, 640, 64), (7, 129, 1000, 64), (8, 256, 2048, 128), (9, 96, 320, 32), (16, 128, 128, 128), (17, 300, 72, 32),
          (33, 200, 1027, 32), (48, 512, 1024, 128), (64, 1024, 96, 64), (100, 65, 130, 128), (128, 256, 512, 64),
          (129, 128, 256, 32), (200, 300, 400, 128), (256, 640, 64, 32), (257, 130, 70, 32), (512, 256, 1088, 64),
          (1000, 515, 130, 128),
          # many tiles, ragged in every direction: two CTAs to a tile, several tiles each
          (2040, 2104, 72, 32), (2040, 72, 2100, 64), (70, 2104, 1990, 32), (2300, 2048, 2304, 128), (700, 5000, 5100, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_linear(m, n, k, group, dtype):
    q, codes, s, x = case(n, k, group, dtype, m + n + k, m)
    bias = torch.from_numpy(np.random.default_rng(k).normal(size=n)).to(dtype) if (m + n) % 2 else None
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group, bias=cu(bias), status=status)
    ref, mag, sub = forward_ref(x, q, s, group, bias)
    check(y, ref, mag, sub, k + 1, dtype)
    assert int(status) == 0
    # the same bits again, and into the middle of a buffer whose other values stay
    buf = torch.full((m * n + 64,), 3.0, dtype=dtype, device="cuda")
    B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group, bias=cu(bias), out=buf[32:32 + m * n].view(m, n))
    assert torch.equal(buf[32:32 + m * n].view(m, n), y)
    assert (buf[:32] == 3).all() and (buf[32 + m * n:] == 3).all()


# few tokens against many features (a warp with several tiles of them, several waves of blocks), with rows of
# scales that can be read as one word and rows that cannot, and x on and off 16 bytes
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m", [1, 8, 9, 16])
@pytest.mark.parametrize("n,k,group", [(6001, 392, 32), (6001, 264, 64), (9000, 256, 128), (5100, 387, 32), (7000, 70, 64),
                                       (80001, 40, 32), (4800, 300, 128), (300, 672, 32), (1000, 300, 128), (1000, 257, 128),
                                       (1000, 384, 128), (1000, 384, 64)])
def test_linear_of_few_tokens(m, n, k, group, dtype):
    q, codes, s, x = case(n, k, group, dtype, m + n + k, m)
    y = B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group)
    check(y, *forward_ref(x, q, s, group, None), k + 1, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_input_grad(m, n, k, group, dtype):
    q, codes, s, _ = case(n, k, group, dtype, m + n + k)
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(dtype)
    dx = B.int4_linear_dx(dy.cuda(), codes.cuda(), s.cuda(), k, group=group)
    w, d = q * per_input(s, group, k), dy.double().numpy()
    check(dx, d @ w, np.abs(d) @ np.abs(w), np.abs(d).sum(1, keepdims=True), n, dtype)
    buf = torch.full((m * k + 64,), 3.0, dtype=dtype, device="cuda")
    B.int4_linear_dx(dy.cuda(), codes.cuda(), s.cuda(), k, group=group, out=buf[32:32 + m * k].view(m, k))
    assert torch.equal(buf[32:32 + m * k].view(m, k), dx)
    assert (buf[:32] == 3).all() and (buf[32 + m * k:] == 3).all()


def scale_grad_ref(dy, c, a, q, k, group):
    d, xh = dy.double().cpu().numpy(), c[:, :k].astype(np.float64) * np.repeat(a.astype(np.float64), 128, 1)[:, :k]
    starts = np.arange(0, k, group)
    fold = lambda p: np.add.reduceat(p, starts, axis=1)  # noqa: E731
    ref, mag = fold((d.T @ xh) * q), fold((np.abs(d).T @ np.abs(xh)) * np.abs(q))
    return ref, mag, fold(np.abs(d).sum(0)[:, None] * np.abs(q))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_scale_grad(m, n, k, group, dtype):
    q, codes, s, x = case(n, k, group, dtype, m + n + k, m)
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(dtype)
    c, a = pack_ref(x)
    act = torch.from_numpy(c).cuda(), torch.from_numpy(a).cuda()
    ds = B.int4_scale_grad(dy.cuda(), *act, codes.cuda(), k, group=group)
    ref, mag, sub = scale_grad_ref(dy, c, a, q, k, group)
    check(ds, ref, mag, sub, m + group, dtype)
    g = ds.shape[1]
    buf = torch.full((n * g + 64,), 3.0, dtype=dtype, device="cuda")
    B.int4_scale_grad(dy.cuda(), *act, codes.cuda(), k, group=group, out=buf[32:32 + n * g].view(n, g))
    assert torch.equal(buf[32:32 + n * g].view(n, g), ds)
    assert (buf[:32] == 3).all() and (buf[32 + n * g:] == 3).all()


@pytest.mark.gpu
def test_no_tokens():
    q, codes, s, _ = case(40, 70, 32, BF, 0)
    empty = torch.empty(0, 70, dtype=BF, device="cuda")
    assert B.int4_linear(empty, codes.cuda(), s.cuda(), group=32).shape == (0, 40)
    dy = torch.empty(0, 40, dtype=BF, device="cuda")
    assert B.int4_linear_dx(dy, codes.cuda(), s.cuda(), 70, group=32).shape == (0, 70)
    act = B.act8_pack(empty)
    ds = torch.full((40, 3), 5.0, dtype=BF, device="cuda")
    B.int4_scale_grad(dy, *act, codes.cuda(), 70, group=32, out=ds)
    assert (ds == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 6, 40, 300])
@pytest.mark.parametrize("layout", ["offset", "wide", "wide16", "transposed", "expanded"])
def test_strides(m, layout):
    """rows any distance apart, bases off 16 bytes, columns that are not contiguous"""
    n, k, group = 200, 264, 32
    q, codes, s, x = case(n, k, group, BF, m, m)
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(BF)

    def placed(t):
        r, c = t.shape
        if layout == "offset":
            b = torch.zeros(r * c + 1, dtype=BF, device="cuda")
            b[1:] = t.cuda().flatten()
            return b[1:].view(r, c)
        if layout == "wide":
            b = torch.full((r, c + 5), float("nan"), dtype=BF, device="cuda")
            b[:, :c] = t.cuda()
            return b[:, :c]
        if layout == "wide16":
            b = torch.full((r, c + 24), float("nan"), dtype=BF, device="cuda")
            b[:, 8:c + 8] = t.cuda()
            return b[:, 8:c + 8]
        if layout == "transposed":
            return t.t().contiguous().cuda().t()
        return t[:1].cuda().expand(r, c)

    xv, dv = placed(x), placed(dy)
    w = q * per_input(s, group, k)
    xd, dd = xv.double().cpu().numpy(), dv.double().cpu().numpy()
    ref, mag, sub = forward_ref(xv, q, s, group, None)
    check(B.int4_linear(xv, codes.cuda(), s.cuda(), group=group), ref, mag, sub, k, BF)
    check(B.int4_linear_dx(dv, codes.cuda(), s.cuda(), k, group=group), dd @ w, np.abs(dd) @ np.abs(w),
          np.abs(dd).sum(1, keepdims=True), n, BF)
    c, a = pack_ref(xv)
    act = B.act8_pack(xv)
    assert np.array_equal(act[0].cpu().numpy(), c) and np.array_equal(act[1].cpu().numpy(), a)
    check(B.int4_scale_grad(dv, *act, codes.cuda(), k, group=group), *scale_grad_ref(dv, c, a, q, k, group), m + group, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 20, 300])
def test_nan_and_infinity_propagate(m):
    """a bad input spoils what the formula says it spoils, and nothing else"""
    n, k, group = 150, 200, 64
    q, codes, s, x = case(n, k, group, BF, 5, m)
    q[:, 7] = np.where(q[:, 7] == 0, 1, q[:, 7])
    codes = store(q)
    x[1, 7] = float("nan")
    x[2, 199] = float("inf")
    y = B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group).cpu()
    assert torch.isnan(y[1]).all()
    want = torch.from_numpy(np.where(q[:, 199] == 0, np.nan, np.copysign(np.inf, q[:, 199])))
    assert torch.equal(torch.isnan(want), torch.isnan(y[2].double()))
    assert torch.equal(y[2].double().nan_to_num(0, 1, -1), want.nan_to_num(0, 1, -1))
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.isfinite(y[keep]).all()
    # a NaN scale spoils its output feature only; the last feature too, next to the padding
    s2 = s.clone()
    s2[n - 1, 0] = float("nan")
    y = B.int4_linear(x[keep].cuda(), codes.cuda(), s2.cuda(), group=group).cpu()
    assert torch.isnan(y[:, n - 1]).all() and torch.isfinite(y[:, :n - 1]).all()
    dy = torch.ones(m, n, dtype=BF)
    dy[0, 3] = float("nan")
    dx = B.int4_linear_dx(dy.cuda(), codes.cuda(), s.cuda(), k, group=group).cpu()
    assert torch.isnan(dx[0]).all() and torch.isfinite(dx[1:]).all()
    dx = B.int4_linear_dx(dy[1:].cuda(), codes.cuda(), s2.cuda(), k, group=group).cpu()
    assert torch.isnan(dx[:, :group]).all() and torch.isfinite(dx[:, group:]).all()
    act = B.act8_pack(x.cuda())  # token 1 is NaN in features 0..127, token 2 in 128..199
    ds = B.int4_scale_grad(torch.ones(m, n, dtype=BF, device="cuda"), *act, codes.cuda(), k, group=group).cpu()
    assert torch.isnan(ds).all()
    x[1, 7] = 0
    ds = B.int4_scale_grad(torch.ones(m, n, dtype=BF, device="cuda"), *B.act8_pack(x.cuda()), codes.cuda(), k,
                           group=group).cpu()
    assert torch.isfinite(ds[:, :2]).all() and torch.isnan(ds[:, 2:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 20, 300])
@pytest.mark.parametrize("k", [70, 96, 128])
def test_large_scales_do_not_spoil_the_padding(m, k):
    """fp16 scales whose -8 s would overflow, with codes that do not: the inputs beyond k add nothing"""
    n, group = 40, 32
    rng = np.random.default_rng(k)
    q = rng.integers(-7, 8, (n, k))
    s = torch.full((n, -(-k // group)), 9000.0, dtype=HF)
    x = torch.from_numpy(rng.normal(size=(m, k)) * 2.0 ** -8).to(HF)
    ref, mag, sub = forward_ref(x, q, s, group, None)
    check(B.int4_linear(x.cuda(), store(q).cuda(), s.cuda(), group=group), ref, mag, sub, k, HF)
    dy = torch.from_numpy(rng.normal(size=(m, n)) * 2.0 ** -8).to(HF)
    w, d = q * per_input(s, group, k), dy.double().numpy()
    check(B.int4_linear_dx(dy.cuda(), store(q).cuda(), s.cuda(), k, group=group), d @ w, np.abs(d) @ np.abs(w),
          np.abs(d).sum(1, keepdims=True), n, HF)


@pytest.mark.gpu
@pytest.mark.parametrize("amount", [1e-3, 1e-6, 3e4])
def test_scale_grad_of_small_and_large_activations(amount):
    """fp16 gradients on checkpoints whose scales an fp16 would not hold"""
    m, n, k, group = 100, 72, 264, 64
    q, codes, _, x = case(n, k, group, HF, 6, m)
    x = (x.double() / x.double().abs().max() * amount).float()
    c, a = B.act8_pack(x.cuda())
    dy = torch.from_numpy(np.random.default_rng(1).normal(size=(m, n)) * 2.0 ** -9).to(HF)
    ds = B.int4_scale_grad(dy.cuda(), c, a, codes.cuda(), k, group=group)
    check(ds, *scale_grad_ref(dy, c.cpu().numpy(), a.cpu().numpy(), q, k, group), m + group, HF)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,group", [(300, 2100, 1031, 32), (40, 4100, 4099, 64)])
def test_large_operands_off_16_bytes(m, n, k, group):
    q, codes, s, x = case(n, k, group, BF, 9, m)
    dy = torch.from_numpy(np.random.default_rng(3).normal(size=(m, n))).to(BF)
    ref, mag, sub = forward_ref(x, q, s, group, None)
    check(B.int4_linear(x.cuda(), codes.cuda(), s.cuda(), group=group), ref, mag, sub, k, BF)
    odd = torch.zeros(m * n + 1, dtype=BF, device="cuda")[1:].view(m, n)  # rows of n elements off by one
    odd.copy_(dy)
    w, d = q * per_input(s, group, k), dy.double().numpy()
    check(B.int4_linear_dx(odd, codes.cuda(), s.cuda(), k, group=group), d @ w, np.abs(d) @ np.abs(w),
          np.abs(d).sum(1, keepdims=True), n, BF)
    c, a = pack_ref(x)
    ds = B.int4_scale_grad(odd, torch.from_numpy(c).cuda(), torch.from_numpy(a).cuda(), codes.cuda(), k, group=group)
    check(ds, *scale_grad_ref(dy, c, a, q, k, group), m + group, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(17, 8192, 8192), (48, 4096, 16384), (40, 2048, 8192), (64, 2048, 2048), (100, 1536, 4000)])
def test_same_bits_of_few_tokens(m, n, k):
    """the same for contractions split over clusters of several sizes, and steps of 128"""
    torch.manual_seed(n)
    codes, s = B.int4_quantize(torch.randn(n, k, device="cuda") * 0.02, 64, dtype=BF)
    x, dy = torch.randn(m, k, device="cuda").to(BF), torch.randn(m, n, device="cuda").to(BF)
    act = B.act8_pack(x)
    wd = B.int4_dequantize(codes, s, k, 64).float()
    calls = [lambda: B.int4_linear(x, codes, s, group=64), lambda: B.int4_linear_dx(dy, codes, s, k, group=64),
             lambda: B.int4_scale_grad(dy, *act, codes, k, group=64)]
    first = [c() for c in calls]
    for _ in range(20):
        for f, c in zip(first, calls):
            assert torch.equal(f, c())
    for got, a, b, terms in ((first[0], x.float(), wd.T, k), (first[1], dy.float(), wd, n)):  # bounds as above
        ref, mag = a @ b, a.abs() @ b.abs()
        tol = (2 * U[BF] + terms * 2.0 ** -22) * mag + U[BF] * ref.abs() + 1e-6
        assert bool(((got.float() - ref).abs() <= tol).all())


@pytest.mark.gpu
def test_a_first_call_inside_a_capture():
    """a process whose first product is captured: what the launch asks about the device does not disturb it"""
    code = """
import torch
import dit_weight_compression_tile_b200 as ep
codes, s = ep.int4_quantize(torch.randn(2048, 2048, device="cuda").bfloat16())
for m in (5, 33, 600):
    x = torch.randn(m, 2048, device="cuda").bfloat16()
    y = torch.empty(m, 2048, device="cuda", dtype=torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.int4_linear(x, codes, s, out=y)
    g.replay()
    assert torch.equal(y, ep.int4_linear(x, codes, s)), m
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 11])
@pytest.mark.parametrize("n,k,at", [(8200, 8191, 0), (4096, 16384, 3)])
def test_large_weight_of_few_tokens_off_16_bytes(m, n, k, at):
    q, codes, s, x = case(n, k, 64, BF, m + k, m)
    flat = torch.zeros(m * k + at, dtype=BF, device="cuda")
    view = flat[at:].view(m, k)
    view.copy_(x)
    y = B.int4_linear(view, codes.cuda(), s.cuda(), group=64)
    assert torch.equal(flat[at:].view(m, k).cpu(), x)
    check(y, *forward_ref(x, q, s, 64, None), k + 1, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group", [(BF, 128), (HF, 32)])
@pytest.mark.parametrize("m,n,k", [(2048, 4096, 4096), (700, 5120, 5000), (512, 1024, 8192)])
def test_same_bits_on_every_call(m, n, k, dtype, group):
    """large products many times over, each the same to the last bit (a copy taken for the one before it
    shows here), and near the product of the reconstructed weight in fp32"""
    torch.manual_seed(m)
    w = torch.randn(n, k, device="cuda") * 0.02
    codes, s = B.int4_quantize(w, group, dtype=dtype)
    x, dy = torch.randn(m, k, device="cuda").to(dtype), (torch.randn(m, n, device="cuda") * 0.1).to(dtype)
    act = B.act8_pack(x)
    wd = B.int4_dequantize(codes, s, k, group).float()
    calls = [lambda: B.int4_linear(x, codes, s, group=group), lambda: B.int4_linear_dx(dy, codes, s, k, group=group),
             lambda: B.int4_scale_grad(dy, *act, codes, k, group=group)]
    first = [c() for c in calls]
    for _ in range(6):
        for f, c in zip(first, calls):
            assert torch.equal(f, c())
    # bounds: u for each operand rounded, k 2^-23 for sums (twice: the comparison sums in fp32 too), u for the result
    for got, a, b, terms in ((first[0], x.float(), wd.T, k), (first[1], dy.float(), wd, n)):
        ref, mag = a @ b, a.abs() @ b.abs()
        tol = (2 * U[dtype] + terms * 2.0 ** -22) * mag + U[dtype] * ref.abs() + 1e-6
        assert bool(((got.float() - ref).abs() <= tol).all())


@pytest.mark.gpu
def test_from_another_thread():
    """a thread that has made no CUDA call of its own"""
    import threading
    q, codes, s, x = case(96, 256, 64, BF, 4, 48)
    xc, cc, sc = x.cuda(), codes.cuda(), s.cuda()
    want, out, caught = B.int4_linear(xc, cc, sc, group=64), torch.zeros(48, 96, dtype=BF, device="cuda"), []
    torch.cuda.synchronize()

    def call():
        try:
            B.int4_linear(xc, cc, sc, group=64, out=out)
        except Exception as e:  # noqa: BLE001
            caught.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not caught and torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [5, 24])
def test_rows_beyond_32_bits(m):
    """rows so far apart that their offsets pass 2^31 elements"""
    n, k, group = 130, 96, 32
    q, codes, s, x = case(n, k, group, BF, 1, m)
    ld = (2 ** 31 // (m - 1) + 64) // 8 * 8
    base = torch.empty((m - 1) * ld + 256, dtype=BF, device="cuda")
    assert base.numel() > 2 ** 31
    xv = base.as_strided((m, k), (ld, 1))
    xv.copy_(x)
    ref, mag, sub = forward_ref(x, q, s, group, None)
    check(B.int4_linear(xv, codes.cuda(), s.cuda(), group=group), ref, mag, sub, k, BF)
    c, a = B.act8_pack(xv)
    want_c, want_a = pack_ref(x)
    assert np.array_equal(c.cpu().numpy(), want_c) and np.array_equal(a.cpu().numpy(), want_a)
    dv = base.as_strided((m, n), (ld, 1))
    dy = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n))).to(BF)
    dv.copy_(dy)
    w, d = q * per_input(s, group, k), dy.double().numpy()
    check(B.int4_linear_dx(dv, codes.cuda(), s.cuda(), k, group=group), d @ w, np.abs(d) @ np.abs(w),
          np.abs(d).sum(1, keepdims=True), n, BF)
    check(B.int4_scale_grad(dv, c, a, codes.cuda(), k, group=group), *scale_grad_ref(dy, want_c, want_a, q, k, group),
          m + group, BF)


@pytest.mark.gpu
def test_stream_argument_and_overlapping_calls():
    """calls on two streams at once, with outputs that belong to their stream"""
    n, k, group, m = 384, 512, 64, 64
    q, codes, s, x = case(n, k, group, BF, 3, m)
    xc, cc, sc = x.cuda(), codes.cuda(), s.cuda()
    want = B.int4_linear(xc, cc, sc, group=group)
    dwant = B.int4_linear_dx(want, cc, sc, k, group=group)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(8):
        st = streams[i % 2]
        y = B.int4_linear(xc, cc, sc, group=group, stream=st)
        outs.append((y, B.int4_linear_dx(y, cc, sc, k, group=group, stream=st)))
    torch.cuda.synchronize()
    for y, dx in outs:
        assert torch.equal(y, want) and torch.equal(dx, dwant)


# ---------------------------------------------------------------- the layer: a run of them together
def step_reference(x, q, s, bias, dy, group):
    """y, dx, ds, db of a training step in float64, the scales' gradient on the 8-bit checkpoint"""
    c, a = pack_ref(x)
    w, d = q * per_input(s, group, q.shape[1]), dy.double().cpu().numpy()
    return (forward_ref(x, q, s, group, bias), (d @ w, np.abs(d) @ np.abs(w), np.abs(d).sum(1, keepdims=True)),
            scale_grad_ref(dy, c, a, q, q.shape[1], group), d.sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tokens,n,k,group", [((1,), 64, 96, 32), ((2, 9), 200, 264, 64), ((4, 3, 11), 130, 1027, 128),
                                              ((300,), 256, 512, 64)])
def test_layer_step(tokens, n, k, group, dtype):
    torch.manual_seed(n)
    lin = nn.Linear(k, n, dtype=dtype, device="cuda")
    layer = GroupedINT4Linear.from_linear(lin, group=group, train_scales=True)
    assert torch.equal(layer.bias, lin.bias)
    layer.bias.requires_grad_(True)
    x = torch.randn(*tokens, k, device="cuda").to(dtype).requires_grad_(True)
    dy = torch.randn(*tokens, n, device="cuda").to(dtype)
    y = layer(x)
    assert y.shape == (*tokens, n)
    y.backward(dy)
    q, m = load(layer.codes, k), dy.numel() // n
    fwd, dx, ds, db = step_reference(x.detach().reshape(m, k), q, layer.scales.detach(), layer.bias.detach(),
                                     dy.reshape(m, n), group)
    check(y.detach().reshape(m, n), *fwd, k + 1, dtype)
    check(x.grad.reshape(m, k), *dx, n, dtype)
    check(layer.scales.grad, *ds, m + group, dtype)
    err = np.abs(layer.bias.grad.double().cpu().numpy() - db)
    assert (err <= U[dtype] * np.abs(db) + m * 2.0 ** -23 * np.abs(dy.reshape(m, n).double().cpu().numpy()).sum(0)).all()
    # the quantized weight is at most half a step off the source, plus the roundings of the scale and of s q
    wq, step = layer.dequantize().double(), layer.scales.detach().double().repeat_interleave(group, 1)[:, :k]
    assert ((wq - lin.weight.detach().double()).abs() <= step * (0.5 + 14 * U[dtype])).all()


@pytest.mark.gpu
def test_gradients_against_differences():
    """the forward is linear in the scales and in x, so differences of its own outputs are exact up to
    the outputs' roundings (u |y| each) and, for the scales, the checkpoint's half steps"""
    n, k, group, m = 96, 256, 64, 40
    q, codes, s, x = case(n, k, group, BF, 8, m)
    cc, sc, xc = codes.cuda(), s.cuda().requires_grad_(True), x.cuda().requires_grad_(True)
    dy = torch.from_numpy(np.random.default_rng(2).normal(size=(m, n))).to(BF).cuda()
    y = int4_group_linear(xc, cc, sc, group=group)
    dx, ds = torch.autograd.grad(y, (xc, sc), dy)
    y0, d = y.detach().double(), dy.double()
    a = np.repeat(pack_ref(x)[1].astype(np.float64), 128, 1)
    for g in range(k // group):  # double the scales of group g in every row: y changes by s ds' share
        s2 = s.clone()
        s2[:, g] *= 2
        y2 = B.int4_linear(xc.detach(), cc, s2.cuda(), group=group).double()
        change = (d * (y2 - y0)).sum(0)
        want = sc.detach()[:, g].double() * ds[:, g].double()
        # weights rounded to the type in both (u |x w| each), outputs rounded, checkpoint half a step off
        w = np.abs(q * per_input(s, group, k))
        w2 = np.abs(q * per_input(s2, group, k))
        gs = slice(g * group, (g + 1) * group)
        slack = 2.0 ** -8 * ((d.abs() * (y2.abs() + y0.abs())).sum(0) + want.abs()).cpu().numpy()
        slack = slack + (np.abs(d.cpu().numpy()) * (np.abs(x.double().numpy()) @ (w + w2).T)).sum(0) * (2.0 ** -8 + k * 2.0 ** -23)
        slack = slack + ((np.abs(d.cpu().numpy()).T @ (a[:, gs] / 2 + 2.0 ** -8 * np.abs(x.double().numpy()[:, gs]))) * w[:, gs]).sum(1)
        assert ((change - want).abs().cpu().numpy() <= slack).all()
    for j in (0, 100, 255):  # set column j of x to zero
        x2 = x.clone()
        x2[:, j] = 0
        y2 = B.int4_linear(x2.cuda(), cc, s.cuda(), group=group).double()
        change = (d * (y0 - y2)).sum(1)
        want = x[:, j].double().cuda() * dx[:, j].double()
        w = np.abs(q * per_input(s, group, k))
        slack = 2.0 ** -8 * ((d.abs() * (y2.abs() + y0.abs())).sum(1) + want.abs()).cpu().numpy()
        both = np.abs(x.double().numpy()) @ w.T * 2
        slack = slack + (np.abs(d.cpu().numpy()) * both).sum(1) * (2.0 ** -8 + k * 2.0 ** -23)
        slack = slack + np.abs(x[:, j].double().numpy()) * (np.abs(d.cpu().numpy()) @ w[:, j]) * (2.0 ** -8 + n * 2.0 ** -23)
        assert ((change - want).abs().cpu().numpy() <= slack).all()


@pytest.mark.gpu
def test_layer_keeps_only_what_the_backward_needs():
    layer = GroupedINT4Linear.from_linear(nn.Linear(256, 128, dtype=BF, device="cuda"), group=32)
    x = torch.randn(6, 256, device="cuda").to(BF)
    assert not layer(x).requires_grad  # frozen: nothing to differentiate
    x.requires_grad_(True)
    y = layer(x)
    kept = [t for t in y.grad_fn.saved_tensors if t is not None]
    assert all(t.dtype != torch.int8 for t in kept)  # no checkpoint without trained scales
    y.sum().backward()  # an expanded gradient
    assert x.grad is not None and layer.scales.grad is None
    layer.scales.requires_grad_(True)
    x2 = x.detach()
    y = layer(x2)
    kept = [t for t in y.grad_fn.saved_tensors if t is not None]
    assert any(t.dtype == torch.int8 for t in kept) and all(t.data_ptr() != x2.data_ptr() for t in kept)
    y.sum().backward()
    assert layer.scales.grad.shape == layer.scales.shape
    layer2 = copy.deepcopy(layer)
    assert torch.equal(layer2(x2), layer(x2))


@pytest.mark.gpu
def test_no_checkpoint_without_a_gradient(monkeypatch):
    kept = []
    forward = B.int4_layer_forward
    monkeypatch.setattr(B, "int4_layer_forward", lambda *a: kept.append(a[5]) or forward(*a))
    _, codes, s, x = case(40, 130, 64, BF, 3, 6)
    codes, s, x = codes.cuda(), s.cuda().requires_grad_(True), x.cuda()
    y = int4_group_linear(x, codes, s, group=64)
    with torch.no_grad():
        y0 = int4_group_linear(x.view(2, 3, 130), codes, s, group=64)
    with torch.inference_mode():
        y1 = int4_group_linear(x, codes, s, group=64)
    y2 = int4_group_linear(x.detach(), codes, s.detach(), group=64)
    assert y.requires_grad and not y0.requires_grad and not y2.requires_grad and y0.shape == (2, 3, 40)
    assert all(torch.equal(y, t.reshape(6, 40)) for t in (y0, y1, y2))
    assert kept == [True, False, False, False]
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises((RuntimeError, NotImplementedError)):
            int4_group_linear(dual, codes, s.detach(), group=64)


@pytest.mark.gpu
def test_training_the_scales_runs():
    torch.manual_seed(0)
    layers = nn.Sequential(*[GroupedINT4Linear.from_linear(nn.Linear(a, b, dtype=BF, device="cuda"), group=64,
                                                           train_scales=True) for a, b in ((192, 320), (320, 64))])
    opt = torch.optim.SGD([p for p in layers.parameters() if p.requires_grad], lr=1e-3)
    before = [layer.scales.detach().clone() for layer in layers]
    for _ in range(3):
        opt.zero_grad()
        loss = layers(torch.randn(50, 192, device="cuda").to(BF)).float().square().mean()
        loss.backward()
        assert all(torch.isfinite(layer.scales.grad).all() for layer in layers)
        opt.step()
    assert torch.isfinite(loss) and any(not torch.equal(b, layer.scales) for b, layer in zip(before, layers))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 12, 160])
def test_captured_step(m):
    """forward, checkpoint and backward of a layer captured into a graph and replayed on new inputs,
    beside a second captured graph and eager calls of the same layer"""
    n, k, group = 256, 320, 64
    layer = GroupedINT4Linear.from_linear(nn.Linear(k, n, dtype=BF, device="cuda"), group=group, train_scales=True)
    xs = [torch.randn(m, k, device="cuda").to(BF).requires_grad_(True) for _ in range(2)]
    dys = [torch.randn(m, n, device="cuda").to(BF) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, results = [], []
    with torch.cuda.stream(side):
        for x, dy in zip(xs, dys):  # warm-up
            torch.autograd.grad(layer(x), (x, layer.scales), dy)
        side.synchronize()
        for x, dy in zip(xs, dys):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                y = layer(x)
                results.append((y.detach(), *torch.autograd.grad(y, (x, layer.scales), dy)))
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(2):
        torch.manual_seed(seed)
        for x, dy in zip(xs, dys):
            x.data.copy_(torch.randn(m, k))
            dy.copy_(torch.randn(m, n))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for st, g in zip(streams, graphs):  # the two graphs at once
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for x, dy, got in zip(xs, dys, results):
            y = layer(x)
            want = (y.detach(), *torch.autograd.grad(y, (x, layer.scales), dy))
            assert all(torch.equal(a, b) for a, b in zip(got, want))
