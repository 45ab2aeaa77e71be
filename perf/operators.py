"""The gated feed-forward block (forward, backward, and served from MXFP4 weights), MXFP4 quantisation
and the MXFP4 product: what they compute in plain torch, at which sizes, and how the framework is called.

Shapes: x [m, H]; w1, w3 [I, H]; w2 [H, I], all (out, in).  MXFP4: e2m1 codes, two per byte (element 2j in
the low nibble), one e8m0 scale per 32 inputs of a row, the scales of 128 rows x 4 blocks packed as 512 bytes
[row % 32][row / 32][block]."""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MOST_VALUES = 5.0e7  # of a drawn quantisation


def listed():
    return [
        # one token through one expert-sized block: decode, latency counts
        {"name": "ffn_one_token", "op": "ffn", "m": 1, "H": 2048, "I": 768, "act": "silu"},
        # a decode batch through a wide block: the weights are what has to be read
        {"name": "ffn_decode_batch", "op": "ffn", "m": 48, "H": 7168, "I": 2048, "act": "silu"},
        # a prompt of odd length, sizes that no tile divides, the other activation
        {"name": "ffn_prompt_odd", "op": "ffn", "m": 1777, "H": 1016, "I": 2728, "act": "gelu"},
        # a long prefill: bound by the tensor cores
        {"name": "ffn_prefill", "op": "ffn", "m": 16384, "H": 7168, "I": 2048, "act": "silu"},
        # one training step of the block, forward and backward, at an ordinary batch
        {"name": "ffn_train", "op": "train", "m": 4096, "H": 2048, "I": 8192, "act": "silu"},
        # a small ragged microbatch, odd sizes, the other activation
        {"name": "ffn_train_odd", "op": "train", "m": 333, "H": 1032, "I": 2056, "act": "gelu"},
        # one token through one matrix of 4-bit weights
        {"name": "mx_linear_one_token", "op": "linear", "m": 1, "K": 7168, "N": 2048},
        # a prefill through a square projection of 4-bit weights
        {"name": "mx_linear_prefill", "op": "linear", "m": 8192, "K": 7168, "N": 7168},
        # one token through a block of 4-bit weights
        {"name": "mx_ffn_one_token", "op": "mxffn", "m": 1, "H": 7168, "I": 2048, "act": "silu"},
        # a prompt through the same block
        {"name": "mx_ffn_prompt", "op": "mxffn", "m": 4096, "H": 7168, "I": 2048, "act": "silu"},
        # weights to 4 bits and back, as when a trained block is made ready to serve
        {"name": "mx_quant_weights", "op": "quant", "rows": 14336, "n": 7168, "dtype": "bf16"},
        # a few fp32 rows of odd length
        {"name": "mx_quant_rows", "op": "quant", "rows": 37, "n": 4128, "dtype": "fp32"},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step))


def draw(rng):
    op = rng.choice(("ffn", "train", "linear", "mxffn", "quant"))
    if op == "quant":
        c = {"op": op, "rows": _log(rng, 1, 16384), "n": _log(rng, 32, 16384, 32), "dtype": rng.choice(("bf16", "fp32"))}
        c["rows"] = max(1, min(c["rows"], int(MOST_VALUES / c["n"])))
        return c
    if op == "linear":
        c = {"op": op, "m": _log(rng, 1, 16384), "K": _log(rng, 128, 8192, 32), "N": _log(rng, 128, 8192, 8)}
        c["m"] = max(1, min(c["m"], int(8.0e11 / (2.0 * c["K"] * c["N"]))))
        return c
    step = 32 if op == "mxffn" else 8
    c = {"op": op, "m": _log(rng, 1, 16384 if op == "ffn" else 8192), "H": _log(rng, 128, 7168, step),
         "I": _log(rng, 128, 8192, step), "act": rng.choice(("silu", "gelu"))}
    most = {"ffn": 1.4e12, "train": 1.2e12, "mxffn": 3.5e11}[op] / ((18.0 if op == "train" else 6.0) * c["H"] * c["I"])
    c["m"] = max(1, min(c["m"], int(most)))
    return c


def work(case):
    c = case
    if c["op"] == "quant":
        n = float(c["rows"]) * c["n"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + n * 17 / 32 + n * 2, "flops": 0.0}
    if c["op"] == "linear":
        m, K, N = float(c["m"]), c["K"], c["N"]
        return {"bytes": 2 * m * K + N * K * 17 / 32 + 2 * m * N, "flops": 2 * m * N * K}
    m, H, I = float(c["m"]), c["H"], c["I"]
    if c["op"] == "ffn":
        return {"bytes": 4 * m * H + 6.0 * H * I, "flops": 6 * m * H * I}
    if c["op"] == "mxffn":
        return {"bytes": 4 * m * H + 3.0 * H * I * 17 / 32, "flops": 6 * m * H * I}
    return {"bytes": 8 * m * H + 12.0 * H * I, "flops": 18 * m * H * I}  # forward and backward


# ---------------------------------------------------------------- MXFP4, plain

def _exponents(blocks):
    """blocks fp32 [..., 32] -> e = max(floor(log2 amax) - 2, -127), int32 [..., 1]."""
    _, e = torch.frexp(blocks.abs().amax(-1, keepdim=True))  # amax = f 2^e, f in [1/2, 1)
    return torch.where(blocks.abs().amax(-1, keepdim=True) > 0, (e - 3).clamp_min(-127), torch.full_like(e, -127))


def _round_e2m1(a):
    """|a| to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, ties to the even code, above 6 to 6."""
    a = a.clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _quantised(v):
    """fp32 [rows, n] -> the values that its MXFP4 codes and scales stand for, fp32."""
    b = v.reshape(v.shape[0], -1, 32)
    e = _exponents(b)
    half = torch.div(e, 2, rounding_mode="floor")  # 2^-e in two factors: 2^127 and beyond stay finite
    up = torch.ldexp(torch.ldexp(b, -half), half - e)
    q = torch.copysign(_round_e2m1(up.abs()), b)
    return torch.ldexp(torch.ldexp(q, half), e - half).reshape(v.shape)


def _pack(v):
    """fp32 [rows, n] -> (codes uint8 [rows, n/2], packed scales uint8), as a loader of 4-bit weights has them."""
    rows, n = v.shape
    b = v.reshape(rows, -1, 32)
    e = _exponents(b)
    q = _round_e2m1(torch.ldexp(b, -e).abs())
    table = torch.tensor(E2M1, device=v.device)
    code = torch.bucketize(q, table) + 8 * torch.signbit(b)
    code = code.reshape(rows, n).to(torch.uint8)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    nb = n // 32
    tall, wide = -(-rows // 128) * 128, -(-nb // 4) * 4
    s = torch.zeros(tall, wide, dtype=torch.uint8, device=v.device)
    s[:rows, :nb] = (e.reshape(rows, nb) + 127).to(torch.uint8)
    s = s.reshape(tall // 128, 4, 32, wide // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes, s


def _unpacked(codes, scales, dtype=torch.float32):
    """The matrix that packed codes and scales stand for."""
    rows, n = codes.shape[0], codes.shape[1] * 2
    table = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=codes.device, dtype=dtype)
    v = table[torch.stack((codes & 15, codes >> 4), -1).reshape(rows, n).int()]
    s = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:rows, : n // 32]
    return torch.ldexp(v.reshape(rows, -1, 32), s.int()[..., None] - 127).reshape(rows, n)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "quant":
        # rows of different sizes, a few channels that stand out, as weights and activations have them
        x = torch.randn(case["rows"], case["n"], generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-6, 4, (case["rows"], 1), generator=g, device="cuda").float())
        x[:, :: max(1, case["n"] // 7)] *= 20
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        return s
    if case["op"] == "linear":
        s["x"] = _normal(g, (case["m"], case["K"]), 1.0)
        s["w"] = _pack(_normal(g, (case["N"], case["K"]), case["K"] ** -0.5, torch.float32))
        return s
    m, H, I = case["m"], case["H"], case["I"]
    s["x"] = _normal(g, (m, H), 1.0)
    w = [_normal(g, (I, H), H ** -0.5), _normal(g, (I, H), H ** -0.5), _normal(g, (H, I), I ** -0.5)]
    if case["op"] == "mxffn":
        w = [_pack(t.float()) for t in w]
    s["w1"], s["w3"], s["w2"] = w
    if case["op"] == "train":
        s["dout"] = _normal(g, (m, H), 1.0)
    if own:  # the handle that a program keeps for a block's weights
        from mixture_experts_ffn_gemv_gb300 import binding
        s["block"] = binding.GatedFfn(s["w1"], s["w3"], s["w2"], act=case["act"])
    return s


# ---------------------------------------------------------------- one pass

def _logistic_arg(g, act):
    return g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)


def _act(g, act):
    return g / (1 + torch.exp(-_logistic_arg(g, act)))


def _act_and_slope(g, act):
    """act(g) = g s(t(g)) and its derivative s + g s (1 - s) t'."""
    s = 1 / (1 + torch.exp(-_logistic_arg(g, act)))
    dt = 1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    return g * s, s + g * s * (1 - s) * dt


def run(state):
    op = state["case"]["op"]
    if own:
        from mixture_experts_ffn_gemv_gb300 import binding
        if op == "quant":
            codes, scales = binding.moe_mxfp4_quant(state["x"])
            return binding.moe_mxfp4_dequant(codes, scales)
        if op == "linear":
            return binding.moe_mxfp4_linear(state["x"], *state["w"])
        if op == "train":
            out, saved = state["block"].forward(state["x"], save=True)
            dx, dw1, dw3, dw2 = state["block"].backward(state["dout"], state["x"], saved)
            return {"out": out, "dx": dx, "dw1": dw1, "dw3": dw3, "dw2": dw2}
        return state["block"].forward(state["x"])
    bf16 = torch.bfloat16
    if op == "quant":
        return _quantised(state["x"].float()).to(bf16)
    if op == "linear":
        return (_quantised(state["x"].float()) @ _unpacked(*state["w"]).T).to(bf16)
    act, x = state["case"]["act"], state["x"].float()
    if op == "mxffn":
        w1, w3, w2 = (_unpacked(*state[k]) for k in ("w1", "w3", "w2"))
        x = _quantised(x)
        h = _act(x @ w1.T, act) * (x @ w3.T)
        return (_quantised(h) @ w2.T).to(bf16)
    w1, w3, w2 = (state[k].float() for k in ("w1", "w3", "w2"))
    g, u = x @ w1.T, x @ w3.T
    if op == "ffn":
        return ((_act(g, act) * u) @ w2.T).to(bf16)
    a, slope = _act_and_slope(g, act)
    h = a * u
    out = h @ w2.T
    dout = state["dout"].float()
    dh = dout @ w2
    dg, du = dh * u * slope, dh * a
    dx = dg @ w1 + du @ w3
    grads = (out, dx, dg.T @ x, du.T @ x, dout.T @ h)
    return dict(zip(("out", "dx", "dw1", "dw3", "dw2"), (t.to(bf16) for t in grads)))


# ---------------------------------------------------------------- 64 bits

def _grid_values(v):
    """The MXFP4 reading of v [rows, n] in 64 bits: powers of two from logarithms of exact doubles, and each
    value's nearest of the grid found among all sixteen."""
    v = v.double()
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp_min(1e-300)))
    e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()  # where the logarithm was rounded
    scale = torch.exp2((e - 2).clamp_min(-127))
    r = (b / scale).abs()
    grid = torch.tensor(E2M1, device=v.device, dtype=torch.float64)
    mids = (grid[1:] + grid[:-1]) / 2
    up = torch.zeros_like(r, dtype=torch.int64)
    for k in range(7):  # a tie goes up only to an even code
        up += (r >= mids[k]) if k % 2 else (r > mids[k])
    return (torch.copysign(grid[up], b) * scale).reshape(v.shape)


def _matrix64(codes, scales):
    """The weights in 64 bits, read one nibble and one scale byte at a time by their own addresses."""
    rows, n = codes.shape[0], codes.shape[1] * 2
    c = torch.empty(rows, n, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes & 15).long(), (codes >> 4).long()
    mag = torch.tensor(E2M1, device=codes.device, dtype=torch.float64)[c & 7]
    r = torch.arange(rows, device=codes.device)[:, None]
    b = torch.arange(n // 32, device=codes.device)[None, :]
    at = ((r // 128 * scales.shape[1] + b // 4) * 32 + r % 32) * 16 + r % 128 // 32 * 4 + b % 4
    scale = torch.exp2(scales.reshape(-1)[at].double() - 127)
    return torch.where(c > 7, -mag, mag) * scale.repeat_interleave(32, 1)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "quant":
        return _grid_values(s["x"])
    if op == "linear":
        return torch.einsum("mk,nk->mn", _grid_values(s["x"]), _matrix64(*s["w"]))

    def sig(t):
        return torch.sigmoid(t)

    def pre(t):
        return t if case["act"] == "silu" else math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3)

    if op == "mxffn":
        x = _grid_values(s["x"])
        gate, up = (torch.einsum("mh,ih->mi", x, _matrix64(*s[k])) for k in ("w1", "w3"))
        return torch.einsum("mi,hi->mh", _grid_values(gate * sig(pre(gate)) * up), _matrix64(*s["w2"]))
    x = s["x"].double()
    w1, w3, w2 = (s[k].double() for k in ("w1", "w3", "w2"))
    if op == "ffn":
        gate = torch.einsum("mh,ih->mi", x, w1)
        return torch.einsum("mi,hi->mh", gate * sig(pre(gate)) * torch.einsum("mh,ih->mi", x, w3), w2)
    leaves = [t.requires_grad_() for t in (x, w1, w3, w2)]
    gate = x @ w1.T
    out = (gate * sig(pre(gate)) * (x @ w3.T)) @ w2.T
    dx, dw1, dw3, dw2 = torch.autograd.grad(out, leaves, s["dout"].double())
    return {"out": out.detach(), "dx": dx, "dw1": dw1, "dw3": dw3, "dw2": dw2}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
