"""The norm, the router's losses and gradient, and low-rank adapters from their formulas in 64 bits,
with bounds on a kernel's error that count its roundings.

A result in bf16 is off by half a step, HALF of it; in e4m3 by 2^-4 of it, or 2^-10 of the scale below
the type's normal range.  An fp32 operation is off by F32 of its result, a sum of n terms by at most
n F32 of the sum of their magnitudes, expf and logf by 2 steps (2^-22).  What is left beside these
counts is covered by the factors SMALL = 2^-18 (64 fp32 roundings) that are named where they are used."""
import torch

HALF = 2.0 ** -8
F32 = 2.0 ** -24
SMALL = 2.0 ** -18
TINY = 2.0 ** -133  # half the smallest number of bf16


def norm(x, residual, weight, eps):
    """(out, r): 64 bits, r rounded to bf16 where there is a residual."""
    r = x.double()
    if residual is not None:
        r = (x.double() + residual.double()).float().to(torch.bfloat16).double()
    return r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * weight.double(), r


def norm_bound(out, h):
    """Of out in fp32 (the sum's roundings count half below the root; at most 24 + 5 + 32 terms in a row
    of them, then root, quotient, two products), and of it in bf16."""
    f32 = SMALL * out.abs()
    return f32, HALF * (out.abs() + f32) + f32 + TINY


def norm_backward(dout, r, weight, eps, dresidual):
    """(dx, dweight, bound of dx, bound of dweight)."""
    r, dout, w = r.double(), dout.double(), weight.double()
    rstd = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    n, g = r * rstd, dout * w
    mean = (g * n).mean(1, keepdim=True)
    dx = rstd * (g - n * mean)
    # the sum of g r: SMALL of its terms' magnitudes; then a few roundings of each term
    e = rstd * (2 * SMALL * (g.abs() + n.abs() * mean.abs()) + n.abs() * 2 * SMALL * (g * n).abs().mean(1, keepdim=True))
    if dresidual is not None:
        dx = dx + dresidual.double()
        e = e + F32 * (dx.abs() + dresidual.double().abs())
    terms = (dout * n).abs().sum(0)
    # n: SMALL; a column's sum: up to 64 rows of a block, 76 blocks of a warp, 8 warps
    return dx, (dout * n).sum(0), e + HALF * (dx.abs() + e) + TINY, terms * (SMALL + 160 * F32)


def e4m3(codes):
    """The values of e4m3 codes in 64 bits."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 8 * 2.0 ** -6)
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c >= 128, -v, v)


def sequences(m, off):
    return [(0, m)] if off is None else list(zip(off.tolist()[:-1], off.tolist()[1:]))


def router(logits, ids, off, sigmoid):
    """(balance, z, counts) per sequence, differentiable in logits (64 bits); rows that are all -inf have no part."""
    E, k = logits.shape[1], ids.shape[1]
    bal, zs, counts = [], [], []
    dead = (logits == -float("inf")).all(1)
    safe = torch.where(dead[:, None], torch.zeros_like(logits), logits)
    soft = torch.softmax(safe, 1)
    # sigma over its sum by logarithms: no underflow
    p = torch.softmax(torch.nn.functional.logsigmoid(safe), 1) if sigmoid else soft
    p = torch.where(dead[:, None], torch.zeros_like(p), p)
    z2 = torch.where(dead, torch.zeros_like(safe[:, 0]), torch.logsumexp(safe, 1).square())
    for a, b in sequences(logits.shape[0], off):
        i = ids[a:b].long()
        i = i[(i >= 0) & (i < E)]
        c = torch.bincount(i, minlength=E)
        counts.append(c)
        T = max(b - a, 1)
        bal.append(E / (k * T * T) * (c.double() * p[a:b].sum(0)).sum())
        zs.append(z2[a:b].sum() / T)
    return torch.stack(bal), torch.stack(zs), torch.stack(counts).int()


def router_bounds(logits, bal, z, off):
    """Of balance: terms of one sign, so relative: expf twice, at most 32 + 5 terms of a token, 4 + 5 of a
    chunk, a quotient or two -- within 2 SMALL.  Of z: lse is off by DL = 2^-21 (1 + the largest
    magnitude), its square by 2 |lse| DL + DL^2, the sum by SMALL."""
    zb = []
    safe = torch.where(torch.isinf(logits), torch.zeros_like(logits), logits)
    big = safe.abs().amax(1)
    lse = torch.logsumexp(logits, 1)
    lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse).abs()
    d = 2.0 ** -21 * (1 + big + lse)
    for a, b in sequences(logits.shape[0], off):
        zb.append(((2 * lse * d + d * d)[a:b].sum() / max(b - a, 1)))
    return 2 * SMALL * bal.abs() + 1e-37, torch.stack(zb) + SMALL * z + 1e-37


def route_weights(logits, ids, sigmoid, norm, scale):
    """moe_route's weights of the picks, differentiable; ids outside [0, E) have weight 0."""
    E = logits.shape[1]
    ok = (ids >= 0) & (ids < E)
    l = torch.gather(logits, 1, torch.where(ok, ids, torch.zeros_like(ids)).long())
    if sigmoid and not norm:
        return scale * torch.sigmoid(l) * ok
    l = torch.nn.functional.logsigmoid(l) if sigmoid else l
    ok = ok & (l != -float("inf"))
    some = ok.any(1, keepdim=True)
    l = torch.where(ok, l, torch.where(some, torch.full_like(l, -float("inf")), torch.zeros_like(l)))
    return torch.softmax(l, 1) * ok * (scale if sigmoid else 1.0)


def route_backward(logits, ids, off, sigmoid, norm, scale, dw, dbal, dz):
    """(dlogits, bound) in 64 bits."""
    m, E = logits.shape
    k = ids.shape[1]
    leaf = logits.double().requires_grad_()
    bal, z, counts = router(leaf, ids, off, sigmoid)
    total = leaf.sum() * 0 if torch.isfinite(logits).all() else torch.where(torch.isfinite(leaf), leaf, 0).sum() * 0
    if dw is not None:
        total = total + (route_weights(leaf, ids, sigmoid, norm, scale) * dw.double()).sum()
    if dbal is not None:
        total = total + (bal * dbal.double()).sum()
    if dz is not None:
        total = total + (z * dz.double()).sum()
    (d,) = torch.autograd.grad(total, leaf)
    # magnitudes of what is added up, each with some 64 fp32 roundings
    l = logits.double()
    dead = (l == -float("inf")).all(1)
    safe = torch.where(dead[:, None], torch.zeros_like(l), l)
    soft = torch.softmax(safe, 1)
    p = torch.softmax(torch.nn.functional.logsigmoid(safe), 1) if sigmoid else soft
    b = torch.zeros_like(l)
    lse = torch.logsumexp(safe, 1).abs()
    dl = 2.0 ** -21 * (1 + lse + torch.where(torch.isinf(safe), torch.zeros_like(safe), safe).abs().amax(1))
    for s, (a, e) in enumerate(sequences(m, off)):
        T = max(e - a, 1)
        if dbal is not None:
            c = (counts[s].double() - k * T / E).abs()
            pc = p[a:e]
            # an exponential below 2^-126 may count for nothing: over a sum of at least 1, p is off by that
            b[a:e] += dbal[s].double().abs() * E / (k * T * T) * (4 * SMALL * pc + 2.0 ** -126) * (
                c + (pc * c).sum(1, keepdim=True) + F32 * k * T)
        if dz is not None:
            b[a:e] += dz[s].double().abs() * 2 / T * (soft[a:e] * (4 * SMALL * lse[a:e] + dl[a:e])[:, None]
                                                      + 2.0 ** -126 * lse[a:e, None])
    if dw is not None:
        ok = (ids >= 0) & (ids < E)
        w = route_weights(l, ids, sigmoid, norm, scale)
        part = w * (dw.double().abs() + (w * dw.double().abs()).sum(1, keepdim=True)) * ok
        b.scatter_add_(1, torch.where(ok, ids, torch.zeros_like(ids)).long(), 4 * SMALL * part)
    return d, b + 4 * F32 * d.abs() + 1e-37


def lora(x, y, a, b, ids, scale):
    """(out, bound) in 64 bits: sums of k and of r terms, T as two bf16 parts (2^-16 of it), one rounding."""
    n, r, k = a.shape
    out = y.double().clone()
    e = torch.zeros_like(out)
    for i in range(n):
        rows = (ids == i).nonzero()[:, 0]
        if not rows.numel():
            continue
        xa, ai, bi = x[rows].double(), a[i].double(), b[i].double()
        s = 1.0 if scale is None else float(scale[i])
        t = s * (xa @ ai.T)
        et = abs(s) * (k + 160) * F32 * (xa.abs() @ ai.abs().T) + (2.0 ** -16 + 2 * F32) * t.abs()
        d = t @ bi.T
        out[rows] += d
        e[rows] = et @ bi.abs().T + (2 * r + 2) * F32 * (t.abs() @ bi.abs().T) + F32 * (y[rows].double().abs() + d.abs())
    return out, e + HALF * (out.abs() + e) + TINY
