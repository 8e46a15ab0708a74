"""Cases of the 4-bit group-scaled linear layer and of the 8-bit activation checkpoints that its
backward pass reads: sizes, inputs, the plain forms in elementary torch operations, the same results
in 64 bits and the bytes and products that each pass cannot do without.

The operators (weights (N, K): N output features, K input features; groups of `group` inputs share a
scale; q in -8 .. 7; T one 16-bit type for activations, scales, gradients and outputs):

  linear      y[t, o]  = sum_k x[t, k] s[o, k / group] q[o, k] (+ bias[o])
  input_grad  dx[t, k] = sum_o dy[t, o] s[o, k / group] q[o, k]
  pack        per token and 128 features: scale a = max |x| / 127 in 32 bits (1 where that is 0),
              code = x / a rounded to nearest even, in -127 .. 127
  scale_grad  ds[o, g] = sum_{k in g} q[o, k] sum_t dy[t, o] a[t, k / 128] code[t, k]
  step        y, dx and ds of one training step on the layer: forward, checkpoint, backward

Storage: eight codes to a 32-bit little-endian word, each q + 8 in four bits; inputs 0, 2, 4, 6 of the
eight in bits 0, 4, 8, 12, inputs 1, 3, 5, 7 in bits 16, 20, 24, 28; rows padded with q = 0 to a multiple
of 32 inputs.  Checkpoint codes: rows padded with 0 to a multiple of 16 features.
"""
import math

import torch

own = False

ACT_GROUP = 128  # features per scale of an activation checkpoint
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, m, n, k, group=128, dtype="bf16", bias=False):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "group": group, "dtype": dtype, "bias": bias}


def listed():
    return [
        # serving one token: a small projection, where the launch counts
        _case("linear_1tok_1024", "linear", 1, 1024, 1024),
        # serving one token through the largest weight of the framework's benchmark
        _case("linear_1tok_8192x28672", "linear", 1, 8192, 28672),
        # a small batch of sequences, ragged in both directions, with a bias
        _case("linear_7tok_ragged_fp16", "linear", 7, 4097, 4090, 64, "fp16", True),
        # a larger serving batch, one square projection
        _case("linear_48tok_4096", "linear", 48, 4096, 4096, 128, "bf16", True),
        # a prompt, or the forward pass of a training batch
        _case("linear_2048tok_8192", "linear", 2048, 8192, 8192),
        # the backward pass of that batch: the gradient that goes on to the layer before
        _case("input_grad_2048tok_8192", "input_grad", 2048, 8192, 8192),
        # the same for a short ragged batch with small groups
        _case("input_grad_33tok_ragged_fp16", "input_grad", 33, 1000, 1027, 32, "fp16"),
        # the activations of a training batch into 8 bits
        _case("pack_4096tok_8192", "pack", 4096, 1, 8192),
        # the activations of a few tokens, ragged
        _case("pack_5tok_ragged_fp16", "pack", 5, 1, 1027, 128, "fp16"),
        # the gradient of every group scale from the 8-bit checkpoint of a training batch
        _case("scale_grad_2048tok_8192", "scale_grad", 2048, 8192, 8192),
        # the same for a short ragged batch with small groups
        _case("scale_grad_77tok_ragged_fp16", "scale_grad", 77, 1000, 1027, 32, "fp16"),
        # one training step on a layer: forward, checkpoint and both gradients
        _case("step_1024tok_4096", "step", 1024, 4096, 4096, 64, "bf16", True),
    ]


def draw(rng):
    def size(lo, hi, ragged=0.4):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v if rng.random() < ragged or v < 64 else max(lo, v // 64 * 64)

    op = rng.choice(["linear", "linear", "linear", "input_grad", "pack", "scale_grad", "step"])
    group, dtype = rng.choice([32, 64, 128]), rng.choice(["bf16", "bf16", "fp16"])
    if op == "pack":
        return {"op": op, "m": size(1, 4096), "n": 1, "k": size(64, 8192), "group": 128, "dtype": dtype, "bias": False}
    bias = op in ("linear", "step") and rng.random() < 0.5
    if op == "linear" and rng.random() < 0.5:  # serving
        m, n, k = rng.randint(1, 16), size(256, 8192), size(256, 28672)
    else:
        m, n, k = size(1, 2048), size(128, 8192), size(128, 8192)
    return {"op": op, "m": m, "n": n, "k": k, "group": group, "dtype": dtype, "bias": bias}


# ---------------------------------------------------------------- inputs
def _pad(k, to):
    return (k + to - 1) // to * to


def _store(q):
    """codes q (N, K) in -8 .. 7 as the stored bytes (N, Kp / 2)"""
    n, k = q.shape
    u = torch.full((n, _pad(k, 32)), 8, dtype=torch.uint8, device=q.device)
    u[:, :k] = (q + 8).to(torch.uint8)
    u = u.view(n, -1, 8)
    order = torch.tensor([0, 4, 1, 5], device=q.device)  # byte b holds inputs order[b] and order[b] + 2
    return (u[:, :, order] | (u[:, :, order + 2] << 4)).reshape(n, -1)


def _weights(case, g):
    """a layer's weight as group scales and codes: rows of different size, normal within a row"""
    n, k, group, dt = case["n"], case["k"], case["group"], DTYPES[case["dtype"]]
    kp = _pad(k, group)
    w = torch.randn(n, kp, generator=g, device="cuda") * 0.02
    w *= torch.exp(torch.randn(n, 1, generator=g, device="cuda") * 0.3)
    w[:, k:] = 0
    wg = w.view(n, kp // group, group)
    scales = (wg.abs().amax(-1) / 7.0).to(dt)
    q = (wg / scales.float()[..., None]).round_().clamp_(-7, 7).view(n, kp)[:, :k]
    return _store(q), scales


def _activations(case, g):
    """tokens of unit size with a few features twenty times as large, as a transformer's are"""
    m, k = case["m"], case["k"]
    x = torch.randn(m, k, generator=g, device="cuda")
    x[:, torch.randint(0, k, (max(1, k // 256),), generator=g, device="cuda")] *= 20.0
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": case, "group": case["group"]}
    if op != "pack":
        s["codes"], s["scales"] = _weights(case, g)
    if op in ("linear", "pack", "step", "scale_grad"):
        x = _activations(case, g)
        if op == "scale_grad":
            s["act_codes"], s["act_scales"] = _plain_pack(x)
        else:
            s["x"] = x
    if op in ("input_grad", "scale_grad", "step"):
        s["dy"] = (torch.randn(case["m"], case["n"], generator=g, device="cuda") * 0.01).to(dt)
    if op in ("linear", "step"):
        s["bias"] = (torch.randn(case["n"], generator=g, device="cuda") * 0.1).to(dt) if case["bias"] else None
    if op == "step":
        s["x"].requires_grad_(True)
        s["scales"].requires_grad_(True)
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_codes(codes, k):
    """the stored bytes as float32 (N, K)"""
    n = codes.shape[0]
    b = codes.view(n, -1, 4)
    lo, hi = b & 15, b >> 4
    inputs = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]], -1)
    return inputs.view(n, -1)[:, :k].float() - 8.0


def _plain_weight(codes, scales, k, group):
    return _plain_codes(codes, k) * scales.float().repeat_interleave(group, 1)[:, :k]


def _plain_linear(x, codes, scales, group, bias):
    y = x.float() @ _plain_weight(codes, scales, x.shape[1], group).T
    return (y if bias is None else y + bias.float()).to(x.dtype)


def _plain_input_grad(dy, codes, scales, k, group):
    return (dy.float() @ _plain_weight(codes, scales, k, group)).to(dy.dtype)


def _plain_pack(x):
    m, k = x.shape
    groups = _pad(k, ACT_GROUP) // ACT_GROUP
    padded = torch.zeros(m, groups * ACT_GROUP, device=x.device)
    padded[:, :k] = x.float()
    xg = padded.view(m, groups, ACT_GROUP)
    a = xg.abs().amax(-1)
    a = a / torch.full_like(a, 127.0)
    a = torch.where(a == 0, torch.ones_like(a), a)
    q = (xg.double() / a.double()[..., None]).round().clamp(-127, 127)  # 64 bits: quotients next to a half
    return q.to(torch.int8).view(m, -1)[:, :_pad(k, 16)].contiguous(), a


def _plain_scale_grad(dy, act_codes, act_scales, codes, k, group):
    n = dy.shape[1]
    x = act_codes[:, :k].float() * act_scales.repeat_interleave(ACT_GROUP, 1)[:, :k]
    p = torch.zeros(n, _pad(k, group), device=dy.device)
    p[:, :k] = (dy.float().T @ x) * _plain_codes(codes, k)
    return p.view(n, -1, group).sum(-1).to(dy.dtype)


def run(state):
    op, group = state["op"], state["group"]
    k = state["case"]["k"]
    if own:
        import dit_weight_compression_tile_b200 as ep
        if op == "linear":
            return ep.int4_linear(state["x"], state["codes"], state["scales"], group=group, bias=state["bias"])
        if op == "input_grad":
            return ep.int4_linear_dx(state["dy"], state["codes"], state["scales"], k, group=group)
        if op == "pack":
            return ep.act8_pack(state["x"])
        if op == "scale_grad":
            return ep.int4_scale_grad(state["dy"], state["act_codes"], state["act_scales"], state["codes"], k, group=group)
        y = ep.int4_group_linear(state["x"], state["codes"], state["scales"], bias=state["bias"], group=group)
        dx, ds = torch.autograd.grad(y, (state["x"], state["scales"]), state["dy"])
        return y.detach(), dx, ds
    if op == "linear":
        return _plain_linear(state["x"], state["codes"], state["scales"], group, state["bias"])
    if op == "input_grad":
        return _plain_input_grad(state["dy"], state["codes"], state["scales"], k, group)
    if op == "pack":
        return _plain_pack(state["x"])
    if op == "scale_grad":
        return _plain_scale_grad(state["dy"], state["act_codes"], state["act_scales"], state["codes"], k, group)
    with torch.no_grad():
        y = _plain_linear(state["x"], state["codes"], state["scales"], group, state["bias"])
        act_codes, act_scales = _plain_pack(state["x"])
        dx = _plain_input_grad(state["dy"], state["codes"], state["scales"], k, group)
        ds = _plain_scale_grad(state["dy"], act_codes, act_scales, state["codes"], k, group)
    return y, dx, ds


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        op, k, group = case["op"], case["k"], case["group"]
        if "codes" in s:
            # bit position of each of a word's eight inputs
            words = s["codes"].contiguous().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
            shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda")
            q = (((words[:, :, None] >> shift) & 15) - 8).flatten(1)[:, :k].double()
            of = torch.arange(k, device="cuda") // group  # the group of each input
            w = q * s["scales"].double()[:, of]

        def packed(x):
            parts, scales = [], []
            for part in x.double().split(ACT_GROUP, dim=1):
                a = (part.abs().max(dim=1, keepdim=True).values.float() / torch.tensor(127.0, device="cuda")).double()
                a[a == 0] = 1.0
                parts.append(torch.round(part / a).clamp(-127.0, 127.0))
                scales.append(a)
            return torch.cat(parts, 1), torch.cat(scales, 1)

        def forward():
            y = torch.einsum("tk,ok->to", s["x"].double(), w)
            return y + s["bias"].double() if s["bias"] is not None else y

        def scale_grad(code, a):
            value = code * a[:, torch.arange(k, device="cuda") // ACT_GROUP]
            prod = torch.einsum("to,tk->ok", s["dy"].double(), value) * q
            out = torch.zeros(case["n"], s["scales"].shape[1], dtype=torch.float64, device="cuda")
            return out.index_add_(1, of, prod)

        if op == "linear":
            return forward()
        if op == "input_grad":
            return torch.einsum("to,ok->tk", s["dy"].double(), w)
        if op == "pack":
            code, a = packed(s["x"])
            whole = torch.zeros(case["m"], _pad(k, 16), dtype=torch.int8, device="cuda")
            whole[:, :k] = code.to(torch.int8)
            x = torch.nn.functional.pad(s["x"].double().abs(), (0, _pad(k, ACT_GROUP) - k))
            top = x.view(case["m"], -1, ACT_GROUP).max(-1).values
            return whole, torch.where(top == 0, 1.0, top / 127.0)
        if op == "scale_grad":
            return scale_grad(s["act_codes"][:, :k].double(), s["act_scales"].double())
        return forward(), torch.einsum("to,ok->tk", s["dy"].double(), w), scale_grad(*packed(s["x"]))


# ---------------------------------------------------------------- the least that a pass moves and computes
def work(case):
    op, m, n, k, group = case["op"], case["m"], case["n"], case["k"], case["group"]
    weight = n * _pad(k, 32) // 2
    scales = 2 * n * -(-k // group)
    ckpt = m * _pad(k, 16) + 4 * m * -(-k // ACT_GROUP)
    bias = 2 * n if case["bias"] else 0
    x, y, product = 2 * m * k, 2 * m * n, 2.0 * m * n * k
    if op in ("linear", "input_grad"):
        return {"bytes": weight + scales + x + y + bias, "flops": product}
    if op == "pack":
        return {"bytes": x + ckpt, "flops": 3.0 * m * k}
    if op == "scale_grad":
        return {"bytes": y + ckpt + weight + scales, "flops": product + 2.0 * n * k}
    # x, dy, the weight and its scales read; y, dx and ds written; the checkpoint written and read
    return {"bytes": 2 * (x + y) + weight + 2 * scales + 2 * ckpt + bias, "flops": 3 * product}
