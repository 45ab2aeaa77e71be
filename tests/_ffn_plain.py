"""The gated feed-forward block and MXFP4 from their formulas in 64 bits, with bounds on
what a correct kernel may be off by (no code of the package is used here)."""
from __future__ import annotations

import math

import torch

HALF = 2.0 ** -8      # half a step of bf16, relative: torch.finfo(torch.bfloat16).eps / 2
F32 = 2.0 ** -23      # one fp32 accumulation step, rounded or truncated
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# bounds of |act'| and |act''|: SiLU 1.0998 and 0.5, tanh-GELU 1.129 and 0.80
SLOPE, CURVE = 1.13, 0.81


def act(g, kind):
    return g * torch.sigmoid(arg(g, kind))


def arg(g, kind):
    return g if kind == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)


def act_slope(g, kind):
    s = torch.sigmoid(arg(g, kind))
    dt = 1.0 if kind == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    return g * s, s + g * s * (1 - s) * dt


def forward(x, w1, w3, w2, kind):
    x, w1, w3, w2 = (t.double() for t in (x, w1, w3, w2))
    return (act(x @ w1.T, kind) * (x @ w3.T)) @ w2.T


def backward(dout, x, w1, w3, w2, kind):
    dout, x, w1, w3, w2 = (t.double() for t in (dout, x, w1, w3, w2))
    g, u = x @ w1.T, x @ w3.T
    a, s = act_slope(g, kind)
    dh = dout @ w2
    dg, du = dh * u * s, dh * a
    return dg @ w1 + du @ w3, dg.T @ x, du.T @ x, dout.T @ (a * u)


def _h_parts(x, w1, w3, kind):
    """g, u, and how far a kernel's fp32 g, u may be from them."""
    n = x.shape[1]
    g, u = x @ w1.T, x @ w3.T
    return g, u, n * F32 * (x.abs() @ w1.abs().T), n * F32 * (x.abs() @ w3.abs().T)


def forward_bound(x, w1, w3, w2, kind, h_half=HALF):
    """|kernel - forward|, element by element, for h rounded by h_half of itself at most, out rounded
    to bf16 and fp32 sums; the activation is within 2^-20 of itself."""
    x, w1, w3, w2 = (t.double() for t in (x, w1, w3, w2))
    g, u, eg, eu = _h_parts(x, w1, w3, kind)
    a = act(g, kind)
    h = (a * u).abs()
    eh = SLOPE * eg * (u.abs() + eu) + (a.abs() + SLOPE * eg) * eu + 2.0 ** -20 * h
    eh = eh + h_half * (h + eh)
    eo = eh @ w2.abs().T + w2.shape[1] * F32 * ((h + eh) @ w2.abs().T)
    return eo + HALF * (((a * u) @ w2.T).abs() + eo)


def backward_bounds(dout, x, w1, w3, w2, kind):
    """The same of (dx, dw1, dw3, dw2): g and u saved in fp32, dg, du and h rounded to bf16."""
    dout, x, w1, w3, w2 = (t.double() for t in (dout, x, w1, w3, w2))
    g, u, eg, eu = _h_parts(x, w1, w3, kind)
    a, s = act_slope(g, kind)
    dh = dout @ w2
    ed = dout.shape[1] * F32 * (dout.abs() @ w2.abs())
    ea = SLOPE * eg + 2.0 ** -20 * a.abs()
    es = CURVE * eg + 2.0 ** -20

    def rounded(v, e):
        return e + HALF * (v.abs() + e)

    us, eus = u * s, u.abs() * es + eu * s.abs() + eu * es
    edg = rounded(dh * us, dh.abs() * eus + ed * us.abs() + ed * eus)
    edu = rounded(dh * a, dh.abs() * ea + ed * a.abs() + ed * ea)
    eh = rounded(a * u, a.abs() * eu + ea * u.abs() + ea * eu)
    dg, du, h = dh * us, dh * a, a * u

    def product(pairs):
        """Bound of the rounded sum of v^T w over (v, ev, w) pairs."""
        ref = sum(v.T @ w for v, _, w in pairs)
        mag = sum((v.abs() + ev).T @ w.abs() for v, ev, w in pairs)
        e = sum(ev.T @ w.abs() for _, ev, w in pairs) + sum(v.shape[0] for v, _, _ in pairs) * F32 * mag
        return e + HALF * (ref.abs() + e)

    ex = product([(dg.T, edg.T, w1), (du.T, edu.T, w3)])
    return ex, product([(dg, edg, x)]), product([(du, edu, x)]), product([(h, eh, dout)]).T


# ---------------------------------------------------------------- MXFP4

def mx_scales(v):
    """Scale bytes [rows, n/32] of v [rows, n] (fp32 or bf16), from the format's definition."""
    b = v.double().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    safe = torch.where(bad | (top == 0), torch.ones_like(top), top)
    _, e = torch.frexp(safe)
    s = (e - 1 - 2 + 127).clamp_min(0)
    s = torch.where(top == 0, torch.zeros_like(s), s)
    return torch.where(bad, torch.full_like(s, 255), s).to(torch.uint8)


def mx_codes(v, scales):
    """Codes [rows, n] (one a byte): the nearest of the grid, ties to even."""
    b = v.double().reshape(v.shape[0], -1, 32)
    bad = (scales == 255)[..., None]
    r = torch.where(bad, torch.zeros_like(b), b) / torch.exp2(scales.double() - 127)[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    d = (r.abs().clamp_max(6.0)[..., None] - grid).abs()
    # the lowest distance; of two equal ones the even code
    k = (d * 2 ** 20 + torch.tensor([0, 1] * 4, device=v.device) * 2.0 ** -20).argmin(-1)
    k = k + 8 * torch.signbit(r).long()
    return torch.where(bad, torch.zeros_like(k), k).reshape(v.shape).to(torch.uint8)


def mx_values(codes, scales):
    """64-bit values of codes (one a byte) and scale bytes in rows."""
    mag = torch.tensor(GRID, dtype=torch.float64, device=codes.device)[(codes & 7).long()]
    v = torch.where(codes > 7, -mag, mag).reshape(codes.shape[0], -1, 32)
    f = torch.exp2(scales.double() - 127)
    f = torch.where(scales == 255, torch.full_like(f, math.nan), f)
    return (v * f[..., None]).reshape(codes.shape)


def mx_round(v):
    s = mx_scales(v)
    return mx_values(mx_codes(v, s), s)


def mx_pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def mx_unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)


def mx_forward(x, w1, w3, w2, kind):
    """The block from the values w1, w3, w2 of MXFP4 weights, and a bound on a kernel's error: its
    fp32 h may fall on the other side of a rounding border."""
    x, w1, w3, w2 = mx_round(x), w1.double(), w3.double(), w2.double()
    g, u, eg, eu = _h_parts(x, w1, w3, kind)
    h = act(g, kind) * u
    eh = SLOPE * eg * (u.abs() + eu) + (act(g, kind).abs() + SLOPE * eg) * eu + 2.0 ** -20 * h.abs()
    q = mx_round(h)
    away = torch.where(h < 0, -eh, eh)
    e = torch.maximum((mx_round(h + away) - q).abs(), (mx_round(h - away) - q).abs())
    out = q @ w2.T
    eo = e @ w2.abs().T + w2.shape[1] * F32 * ((q.abs() + e) @ w2.abs().T)
    return out, eo + HALF * (out.abs() + eo)
