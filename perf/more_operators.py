"""What stands around the layer and the block: the norm in front (with the residual's addition, to bf16 and to 8 bits) and
its backward pass, the router's balance and z losses with the gradient of its logits, and the low-rank adapters of many
requests beside a shared projection.  What they compute in plain torch, at which sizes, and how the framework is called.

Norm: r = bf16(x + residual), out = r / sqrt(mean r^2 + eps) * weight; 8 bits: e4m3 codes of out, one fp32 scale
amax / 448 per 128 columns (the last block of a row may be shorter).
Router: logits fp32 [m, E], ids int32 [m, k] (-1: a pair that was dropped), sequences of tokens given by their offsets
(tokens outside are padding).  For a sequence of T tokens, c[e] its pairs of expert e and p the normalised scores:
balance = E / (k T^2) sum_te c[e] p[t, e], z = 1 / T sum_t logsumexp(logits[t])^2.
Adapters: out[t] = y[t] + scale[i] B_i A_i x[t], i = ids[t] (-1: none), A [adapters, r, K], B [adapters, N, r]."""
import math
import random

import torch

own = False

EPS = 1e-6
MOST_VALUES = 1.1e8  # of a drawn norm
BLOCK = 128


def listed():
    return [
        # one token in front of an fp8 layer: bf16 for its router, codes for its experts
        {"name": "norm_one_token_fp8", "op": "norm", "m": 1, "H": 7168, "residual": True, "fp8": True},
        # a long prefill in front of the same layer
        {"name": "norm_prefill_fp8", "op": "norm", "m": 16384, "H": 7168, "residual": True, "fp8": True},
        # a prompt of odd length and width, the first norm of a model (nothing to add), bf16 alone
        {"name": "norm_prompt_odd", "op": "norm", "m": 1777, "H": 1016, "residual": False, "fp8": False},
        # a training step's norm, forward and backward, with the gradient that comes along the residual
        {"name": "norm_train", "op": "norm_train", "m": 16384, "H": 2048, "residual": True},
        # a small microbatch of odd width
        {"name": "norm_train_odd", "op": "norm_train", "m": 333, "H": 1032, "residual": True},
        # a small microbatch through a router of few experts: latency counts
        {"name": "router_train_small", "op": "router", "m": 333, "E": 8, "k": 2, "seqs": 1, "pad": 0, "scoring": "softmax"},
        # a training batch of four long sequences, many experts, sigmoid scores
        {"name": "router_train", "op": "router", "m": 16384, "E": 256, "k": 8, "seqs": 4, "pad": 0, "scoring": "sigmoid"},
        # many packed sequences of uneven length, some of them empty, padding behind the last
        {"name": "router_train_ragged", "op": "router", "m": 4099, "E": 128, "k": 8, "seqs": 37, "pad": 131, "scoring": "softmax"},
        # one token of one request
        {"name": "lora_one_token", "op": "lora", "m": 1, "K": 7168, "N": 2048, "r": 16, "adapters": 8, "requests": 1},
        # a decode batch, every token a request of its own, adapters shared by a few of them
        {"name": "lora_decode", "op": "lora", "m": 64, "K": 2048, "N": 7168, "r": 16, "adapters": 32, "requests": 64},
        # prompts of four requests in one batch
        {"name": "lora_prefill", "op": "lora", "m": 8192, "K": 7168, "N": 7168, "r": 64, "adapters": 4, "requests": 4},
        # prompts of odd lengths, odd sizes, a small rank
        {"name": "lora_prompts_odd", "op": "lora", "m": 1777, "K": 1016, "N": 2728, "r": 8, "adapters": 6, "requests": 9},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step))


def draw(rng):
    op = rng.choice(("norm", "norm_train", "router", "lora"))
    if op in ("norm", "norm_train"):
        c = {"op": op, "m": _log(rng, 1, 32768), "H": _log(rng, 8, 16384, 8), "residual": rng.random() < 0.7}
        c["m"] = max(1, min(c["m"], int(MOST_VALUES / (1 if op == "norm" else 3) / c["H"])))
        if op == "norm":
            c["fp8"] = rng.random() < 0.6
        return c
    if op == "router":
        c = {"op": op, "m": _log(rng, 1, 32768), "E": _log(rng, 2, 1024)}
        c["m"] = max(1, min(c["m"], int(8.0e6 / c["E"])))
        c["k"] = rng.randint(1, min(c["E"], 16))
        c["seqs"] = _log(rng, 1, 64)
        c["pad"] = rng.choice((0, rng.randint(0, c["m"] // 4)))
        c["scoring"] = rng.choice(("softmax", "sigmoid"))
        return c
    c = {"op": op, "m": _log(rng, 1, 8192), "K": _log(rng, 128, 8192, 8), "N": _log(rng, 128, 8192, 8),
         "r": rng.choice((8, 16, 24, 32, 64, 128)), "adapters": _log(rng, 1, 64)}
    c["requests"] = min(c["m"], _log(rng, 1, 256))
    c["adapters"] = max(1, min(c["adapters"], int(2.5e10 / (c["m"] * c["r"] * (c["K"] + c["N"])))))
    return c


def work(case):
    c = case
    m = float(c["m"])
    if c["op"] == "norm":
        per = 4 + (4 if c["residual"] else 0) + (1 + 4 / BLOCK if c["fp8"] else 0)
        return {"bytes": m * c["H"] * per + 4.0 * c["H"], "flops": 0.0}
    if c["op"] == "norm_train":  # x, residual, dout and its own gradient in; residual, out, dx, dweight out
        return {"bytes": m * c["H"] * (14 if c["residual"] else 10) + 8.0 * c["H"], "flops": 0.0}
    if c["op"] == "router":  # logits, ids and the weights' gradients in; the logits' gradients out
        return {"bytes": 8 * m * c["E"] + 8 * m * c["k"] + 4.0 * c["seqs"] * c["E"], "flops": 0.0}
    used = min(c["adapters"], c["requests"])
    return {"bytes": 2 * m * c["K"] + 4 * m * c["N"] + 2.0 * used * c["r"] * (c["K"] + c["N"]),
            "flops": 2 * m * c["r"] * (c["K"] + c["N"])}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _cuts(g, n, top):
    """n + 1 rising offsets from 0 to top, some of them equal."""
    inner = torch.sort(torch.randint(0, top + 1, (n - 1,), generator=g, device="cuda")).values
    ends = torch.tensor([0, top], device="cuda")
    return torch.cat((ends[:1], inner, ends[1:])).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    m = c["m"]
    if c["op"] in ("norm", "norm_train"):
        H = c["H"]
        # a residual stream: rows of different sizes, a few channels that stand out
        r = torch.randn(m, H, generator=g, device="cuda")
        r *= torch.exp2(torch.randint(-2, 4, (m, 1), generator=g, device="cuda").float())
        r[:, :: max(1, H // 5)] *= 12
        s["x"] = _normal(g, m, H) if c["residual"] else r.to(torch.bfloat16)
        s["residual"] = r.to(torch.bfloat16) if c["residual"] else None
        s["weight"] = 1 + _normal(g, H, std=0.2, dtype=torch.float32)
        if c["op"] == "norm_train":
            s["dout"] = _normal(g, m, H)
            s["dresidual"] = _normal(g, m, H) if c["residual"] else None
        return s
    if c["op"] == "router":
        E, k = c["E"], c["k"]
        liked = torch.randn(E, generator=g, device="cuda")  # some experts are asked for more than others
        s["logits"] = torch.randn(m, E, generator=g, device="cuda") * 1.5 + liked
        bias = torch.zeros(E, device="cuda") if c["scoring"] == "softmax" else -0.1 * liked
        score = s["logits"] if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-s["logits"])) + bias
        ids = torch.topk(score, k, dim=1).indices.to(torch.int32)
        s["offsets"] = _cuts(g, c["seqs"], m - c["pad"])
        ids[m - c["pad"]:] = -1
        s["ids"] = ids.contiguous()
        s["dtopk_w"] = _normal(g, m, k, std=0.05, dtype=torch.float32)
        s["dtopk_w"][m - c["pad"]:] = 0
        s["dbalance"] = torch.full((c["seqs"],), 0.01 * m / c["seqs"], device="cuda")
        s["dz"] = torch.full((c["seqs"],), 0.001 * m / c["seqs"], device="cuda")
        return s
    K, N, r, n = c["K"], c["N"], c["r"], c["adapters"]
    s["x"] = _normal(g, m, K)
    s["y"] = _normal(g, m, N)
    s["a"] = _normal(g, n, r, K, std=K ** -0.5)
    s["b"] = _normal(g, n, N, r, std=r ** -0.5)
    s["scale"] = 0.25 + 0.5 * torch.rand(n, generator=g, device="cuda")
    which = torch.randint(0, n, (c["requests"],), generator=g, device="cuda", dtype=torch.int32)
    if c["requests"] > 3:  # a request that uses no adapter
        which[c["requests"] // 2] = -1
    if c["requests"] == m:
        s["ids"] = which
    else:
        starts = _cuts(g, c["requests"], m)[1:].contiguous()
        at = torch.searchsorted(starts, torch.arange(m, device="cuda", dtype=torch.int32), right=True)
        s["ids"] = which[at.clamp_max(c["requests"] - 1)].contiguous()
    return s


# ---------------------------------------------------------------- one pass

def _norm(state, fp8):
    x, res = state["x"].float(), state["residual"]
    new = (x + res.float()).to(torch.bfloat16) if res is not None else None
    r = new.float() if new is not None else x
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * state["weight"]
    got = {"out": y.to(torch.bfloat16)}
    if new is not None:
        got["residual"] = new
    if fp8:
        m, H = y.shape
        nb = -(-H // BLOCK)
        b = torch.zeros(m, nb * BLOCK, device=y.device)
        b[:, :H] = y
        b = b.reshape(m, nb, BLOCK)
        amax = b.abs().amax(2, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        q = (b / scale).reshape(m, nb * BLOCK)[:, :H].contiguous()
        got["codes"] = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        got["scales"] = scale.reshape(m, nb)
    return got


def _norm_backward(r, weight, dout, dresidual):
    r, g = r.float(), dout.float() * weight
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r * rstd
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if dresidual is not None:
        dx = dx + dresidual.float()
    return dx.to(torch.bfloat16), (dout.double() * n.double()).sum(0).float()


def _router(state):
    c, logits, ids, off = state["case"], state["logits"], state["ids"].long(), state["offsets"]
    m, E, k, S = c["m"], c["E"], c["k"], c["seqs"]
    t = torch.arange(m, device=logits.device, dtype=torch.int32)
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)  # S: behind the last
    inside = seq < S
    at = seq.clamp_max(S - 1)
    T = (off[1:] - off[:-1]).float()
    valid = (ids >= 0) & inside[:, None]
    counts = torch.zeros(S * E, dtype=torch.int32, device=logits.device)
    counts.index_add_(0, (at[:, None] * E + ids.clamp_min(0)).reshape(-1), valid.reshape(-1).to(torch.int32))
    counts = counts.reshape(S, E)
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    soft = ex / total
    lse = (top + torch.log(total))[:, 0]
    sig = 1 / (1 + torch.exp(-logits))
    ssum = sig.sum(1, keepdim=True)
    p = soft if c["scoring"] == "softmax" else sig / ssum
    some = T.clamp_min(1)
    share = E * counts.float() / (k * some * some)[:, None]  # [S, E]
    w = share[at] * inside[:, None]
    each = torch.zeros(2, S, dtype=torch.float64, device=logits.device)
    each[0].index_add_(0, at, (p * w).sum(1).double())
    each[1].index_add_(0, at, (lse * lse * inside / some[at]).double())
    # gradients: of the losses, then of the weights of the selected
    G = w * state["dbalance"][at][:, None]
    d = p * (G - (G * p).sum(1, keepdim=True))
    if c["scoring"] == "sigmoid":
        d = d * (1 - sig)
    d = d + (state["dz"][at] * inside / some[at] * 2 * lse)[:, None] * soft
    picked = torch.gather(logits, 1, ids.clamp_min(0))
    dw, live = state["dtopk_w"], (ids >= 0)
    if c["scoring"] == "softmax":
        e = torch.exp(picked - picked.amax(1, keepdim=True)) * live
        wk = e / e.sum(1, keepdim=True).clamp_min(1e-30)
        dk = wk * (dw - (wk * dw).sum(1, keepdim=True))
    else:
        sk = 1 / (1 + torch.exp(-picked)) * live
        wk = sk / sk.sum(1, keepdim=True).clamp_min(1e-30)
        dk = wk * (1 - sk) * (dw - (wk * dw).sum(1, keepdim=True))
    d.scatter_add_(1, ids.clamp_min(0), dk * live)
    return {"balance": each[0].float(), "z": each[1].float(), "counts": counts, "dlogits": d}


def _lora(state):
    x, y, ids = state["x"].float(), state["y"].float(), state["ids"].long()
    n, r, K = state["a"].shape
    mine = torch.zeros(ids.numel(), n, device=x.device)
    mine.scatter_(1, ids.clamp_min(0)[:, None], (state["scale"][ids.clamp_min(0)] * (ids >= 0))[:, None])
    t = (x @ state["a"].float().reshape(n * r, K).T).reshape(-1, n, r) * mine[:, :, None]
    b = state["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    return (y + t.reshape(-1, n * r) @ b).to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from mixture_experts_ffn_gemv_gb300 import binding
        if op == "norm":
            n = binding.moe_add_rmsnorm(state["x"], state["weight"], EPS, residual=state["residual"], fp8=c["fp8"])
            got = {"out": n.out}
            if c["residual"]:
                got["residual"] = n.residual
            if c["fp8"]:
                got["codes"], got["scales"] = n.codes.view(torch.float8_e4m3fn), n.scales
            return got
        if op == "norm_train":
            n = binding.moe_add_rmsnorm(state["x"], state["weight"], EPS, residual=state["residual"])
            r = n.residual if c["residual"] else state["x"]
            dx, dweight = binding.moe_add_rmsnorm_backward(state["dout"], r, state["weight"], EPS,
                                                           dresidual=state["dresidual"])
            return {"out": n.out, "dx": dx, "dweight": dweight, **({"residual": r} if c["residual"] else {})}
        if op == "router":
            balance, z, counts = binding.moe_balance_loss(state["logits"], state["ids"], state["offsets"],
                                                          scoring=c["scoring"])
            d = binding.moe_route_backward(state["logits"], state["ids"], dtopk_w=state["dtopk_w"],
                                           dbalance=state["dbalance"], dz=state["dz"], counts=counts,
                                           seq_offsets=state["offsets"], scoring=c["scoring"])
            return {"balance": balance, "z": z, "counts": counts, "dlogits": d}
        return binding.moe_lora_add(state["y"], state["x"], state["a"], state["b"], state["ids"], state["scale"],
                                    out=torch.empty_like(state["y"]))
    if op == "norm":
        return _norm(state, c["fp8"])
    if op == "norm_train":
        got = _norm(state, False)
        r = got.get("residual", state["x"])
        got["dx"], got["dweight"] = _norm_backward(r, state["weight"], state["dout"], state["dresidual"])
        return got
    return _router(state) if op == "router" else _lora(state)


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """v in 64 bits to the nearest value of e4m3 (3 bits behind the leading one, subnormals from 2^-6 on), ties to even."""
    a = v.abs().clamp(1e-300, 448.0)
    e = torch.floor(torch.log2(a)).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), v) * (v != 0)


def _exact_norm(s, c):
    x = s["x"].double()
    if c["residual"]:
        new = (x + s["residual"].double()).to(torch.bfloat16)
        x = new.double()
    got = {"residual": new.double()} if c["residual"] else {}
    weight = s["weight"].double()
    if c["op"] == "norm_train":
        x, weight = x.requires_grad_(), weight.requires_grad_()
    y = x / torch.sqrt(torch.square(x).sum(1, keepdim=True) / c["H"] + EPS) * weight
    got["out"] = y.detach()
    if c["op"] == "norm_train":
        dx, got["dweight"] = torch.autograd.grad(y, (x, weight), s["dout"].double())
        got["dx"] = dx + s["dresidual"].double() if c["residual"] else dx
    elif c["fp8"]:
        codes, scales = torch.empty_like(y), []
        for at in range(0, c["H"], BLOCK):
            b = y[:, at:at + BLOCK]
            top = b.abs().max(1, keepdim=True).values
            top = torch.where(top > 0, top / 448, 1.0)
            codes[:, at:at + BLOCK] = _e4m3(b / top)
            scales.append(top)
        got["codes"], got["scales"] = codes, torch.cat(scales, 1)
    return got


def _exact_router(s, c):
    off, E, k = s["offsets"].tolist(), c["E"], c["k"]
    leaf = s["logits"].double().requires_grad_()
    balance, zs, counts, total = [], [], [], 0.0
    for q in range(c["seqs"]):
        l, i = leaf[off[q]:off[q + 1]], s["ids"][off[q]:off[q + 1]].long()
        n = torch.bincount(i[i >= 0], minlength=E)
        counts.append(n)
        if l.shape[0] == 0:
            balance.append(torch.zeros((), device=l.device, dtype=torch.float64))
            zs.append(balance[-1])
            continue
        score = torch.softmax(l, 1) if c["scoring"] == "softmax" else torch.sigmoid(l)
        mean = (score / score.sum(1, keepdim=True)).mean(0)
        balance.append(E * (n.double() / (k * l.shape[0]) * mean).sum())
        zs.append(torch.logsumexp(l, 1).square().mean())
    total = (torch.stack(balance) * s["dbalance"].double()).sum() + (torch.stack(zs) * s["dz"].double()).sum()
    rows = (s["ids"] >= 0).all(1).nonzero()[:, 0]
    picked = leaf[rows].gather(1, s["ids"][rows].long())
    w = torch.softmax(picked, 1)
    if c["scoring"] == "sigmoid":
        w = torch.sigmoid(picked)
        w = w / w.sum(1, keepdim=True)
    total = total + (w * s["dtopk_w"][rows].double()).sum()
    (d,) = torch.autograd.grad(total, leaf)
    return {"balance": torch.stack(balance).detach(), "z": torch.stack(zs).detach(), "counts": torch.stack(counts),
            "dlogits": d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s, case)
    if case["op"] == "router":
        return _exact_router(s, case)
    out = s["y"].double()
    for i in range(case["adapters"]):
        rows = (s["ids"] == i).nonzero()[:, 0]
        if rows.numel():
            low = torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][i].double())
            out[rows] += s["scale"][i].double() * torch.einsum("tr,nr->tn", low, s["b"][i].double())
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
