"""The gated feed-forward block, its backward pass, and the MXFP4 operators on the GPU, against
64-bit formulas with bounds derived from the roundings (tests/_ffn_plain.py)."""
import ctypes

import pytest
import torch

import _ffn_plain as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def _n(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _within(got, ref, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - bound
    i = int(over.argmax())
    assert over.max() <= 0, (f"off by {(got - ref).abs().flatten()[i]:.3e}, bound {bound.flatten()[i]:.3e} at {i} of "
                             f"{tuple(got.shape)}: {got.flatten()[i]:.6e} for {ref.flatten()[i]:.6e}")


def _weights(seed, H, I):
    return _n(seed, I, H, std=H ** -0.5), _n(seed + 1, I, H, std=H ** -0.5), _n(seed + 2, H, I, std=I ** -0.5)


def _quantised(B, w):
    """Weights as MXFP4 pairs, and their values in 64 bits (read by the plain code)."""
    pairs = [B.moe_mxfp4_quant(t) for t in w]
    vals = [P.mx_values(P.mx_unpack(c), B.mxfp4_unpack_scales(s, c.shape[0], c.shape[1] * 2)) for c, s in pairs]
    return pairs, vals


# ---------------------------------------------------------------- MXFP4 quantisation

def _check_quant(B, x):
    rows, n = x.shape
    codes, scales = B.moe_mxfp4_quant(x)
    want_s = P.mx_scales(x)
    want_c = P.mx_codes(x, want_s)
    assert torch.equal(B.mxfp4_unpack_scales(scales, rows, n), want_s)
    assert torch.equal(P.mx_unpack(codes), want_c)
    pad = scales.permute(0, 3, 2, 1, 4).reshape(-1, scales.shape[1] * 4)[:rows, n // 32:]
    assert not pad.any()
    want = P.mx_values(want_c, want_s)
    got = B.moe_mxfp4_dequant(codes, scales).double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))  # -0 equals 0 here


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 32), (3, 96), (37, 4128), (129, 256), (1000, 544), (2, 7168)])
def test_quant(B, rows, n, dtype):
    x = _n(rows + n, rows, n, dtype=torch.float32)
    x *= torch.exp2(torch.randint(-40, 40, (rows, 1), device="cuda").float())
    _check_quant(B, x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_borders(B, dtype):
    """Every rounding border and a step to either side, at small, middle and large scales; zeros,
    subnormals, infinities, NaN; the type's largest and lowest values."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.96875]
    rows = []
    for e in (-126, -60, -3, 0, 5, 100, 125):
        b = torch.tensor(mids, dtype=torch.float64) * 2.0 ** e
        b = b.to(dtype)
        up = torch.nextafter(b, torch.full_like(b, float("inf")))
        dn = torch.nextafter(b, torch.zeros_like(b))
        rows.append(torch.cat([b, -up, dn, torch.tensor([4.0 * 2.0 ** e, 0.0], dtype=dtype)]))
    z = torch.zeros(32, dtype=dtype)
    lim = torch.finfo(dtype)
    for v in (0.0, -0.0, lim.tiny, lim.tiny / 4, -lim.max, lim.max, float("inf"), float("-inf"), float("nan")):
        r = z.clone()
        r[5] = v
        r[9] = 1.0 if v not in (0.0, lim.tiny, lim.tiny / 4) else 0.0
        rows.append(r)
    x = torch.stack(rows).cuda()
    _check_quant(B, x)
    _check_quant(B, torch.cat([x, x.flip(0), x], 1))  # such blocks beside ordinary ones


def test_quant_strided_and_empty(B):
    base = _n(1, 40, 320)
    x = base[:, 64:160]  # rows 320 apart, 128-byte offset
    c, s = B.moe_mxfp4_quant(x)
    c2, s2 = B.moe_mxfp4_quant(x.contiguous())
    assert torch.equal(c, c2) and torch.equal(B.mxfp4_unpack_scales(s, 40, 96), B.mxfp4_unpack_scales(s2, 40, 96))
    c, s = B.moe_mxfp4_quant(base[:0])
    assert c.shape == (0, 160) and B.moe_mxfp4_dequant(c, s).shape == (0, 320)
    for bad in (base[:, 4:36], base.T, base[:, ::2], base.half()):
        with pytest.raises(ValueError):
            B.moe_mxfp4_quant(bad)
    with pytest.raises(B.MoeError):
        B.moe_mxfp4_quant(base[:, :40])


# ---------------------------------------------------------------- MXFP4 product

GEMM_SIZES = [(1, 8, 32), (1, 2048, 7168), (2, 136, 96), (5, 1000, 544), (16, 256, 256), (17, 128, 2080), (64, 520, 1024),
              (100, 384, 4128), (128, 256, 512), (129, 264, 288), (256, 256, 256), (300, 1032, 1568), (1000, 776, 928)]


@pytest.mark.parametrize("m,n,k", GEMM_SIZES)
def test_mx_linear(B, m, n, k):
    x = _n(m, m, k, dtype=torch.float32) * torch.exp2(torch.randint(-8, 8, (m, 1), device="cuda").float())
    (w,), (wv,) = _quantised(B, [_n(n + k, n, k, std=k ** -0.5)])
    xb = x.to(torch.bfloat16)
    xv = P.mx_round(xb)
    ref = xv @ wv.T
    bound = P.HALF * ref.abs() + (1 + P.HALF) * k * P.F32 * (xv.abs() @ wv.abs().T)
    _within(B.moe_mxfp4_linear(xb, *w), ref, bound)


def test_mx_gemm_scales_by_position(B):
    """Every block its own scale and every row its own sign pattern: a scale read for another row
    or block shows at once."""
    m, n, k = 200, 328, 640
    g = torch.Generator(device="cuda").manual_seed(5)
    def mat(rows):
        codes = torch.randint(0, 16, (rows, k), generator=g, device="cuda").to(torch.uint8)
        scales = torch.randint(117, 138, (rows, k // 32), generator=g, device="cuda").to(torch.uint8)
        return codes, scales
    (ac, as_), (bc, bs) = mat(m), mat(n)
    got = B.moe_mxfp4_gemm(P.mx_pack(ac), B.mxfp4_pack_scales(as_), P.mx_pack(bc), B.mxfp4_pack_scales(bs))
    a, b = P.mx_values(ac, as_), P.mx_values(bc, bs)
    ref = a @ b.T
    _within(got, ref, P.HALF * ref.abs() + (1 + P.HALF) * k * P.F32 * (a.abs() @ b.abs().T))


def test_mx_gemm_nan_scale_stays_in_its_row(B):
    x = _n(3, 40, 256)
    x[7, 33] = float("inf")
    x[21, 200] = float("nan")
    (w,), (wv,) = _quantised(B, [_n(4, 64, 256)])
    out = B.moe_mxfp4_linear(x, *w)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[7, 21]] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    assert B.mxfp4_device_status() == 0


def test_mx_linear_fp32_strided_and_streams(B):
    (w,), _ = _quantised(B, [_n(4, 72, 320)])
    base = _n(6, 30, 700, dtype=torch.float32)
    x = base[:, 4:324]
    want = B.moe_mxfp4_linear(x.contiguous(), *w)
    assert torch.equal(B.moe_mxfp4_linear(x, *w), want)
    assert torch.equal(B.moe_mxfp4_gemm(*B.moe_mxfp4_quant(x), *w), want)
    assert B.moe_mxfp4_linear(x[:0], *w).shape == (0, 72)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = B.moe_mxfp4_linear(x, *w, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        B.moe_mxfp4_linear(x[:, :300], *w)
    with pytest.raises(ValueError):
        B.moe_mxfp4_linear(x, w[0], w[1].reshape(-1))
    with pytest.raises(ValueError):
        B.moe_mxfp4_linear(x, w[0][:, ::2], w[1])


# ---------------------------------------------------------------- the block

def _saved_parts(saved, m, I):
    """act(g), u act'(g) and h [m, I] of what a forward pass saved."""
    n = (m + 31) // 32 * ((I + 31) // 32) * 1024
    blocks = [s.reshape((m + 31) // 32, (I + 31) // 32, 4, 32, 8) for s in (saved[:n], saved[n:2 * n])]
    a, d = (s.permute(0, 3, 1, 2, 4).reshape(s.shape[0] * 32, -1)[:m, :I] for s in blocks)
    return a, d, saved[2 * n:].view(torch.bfloat16)[:m * I].reshape(m, I)


FFN_SIZES = [(1, 2048, 768), (1, 8, 8), (3, 24, 40), (8, 264, 520), (9, 264, 520), (16, 256, 128), (17, 136, 264), (48, 1024, 512), (65, 520, 1032),
             (128, 256, 256), (200, 512, 384), (333, 1032, 2056), (777, 1016, 680), (130, 1032, 72), (256, 328, 200),
             (257, 4104, 64), (500, 200, 136)]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,H,I", FFN_SIZES)
def test_forward(B, m, H, I, kind):
    w = _weights(H + I, H, I)
    x = _n(m, m, H)
    blk = B.GatedFfn(*w, act=kind)
    out = blk.forward(x)
    ref = P.forward(x, *w, kind)
    out2, saved = blk.forward(x, save=True)
    _within(out2, ref, P.forward_bound(x, *w, kind))
    if m > 8:
        assert torch.equal(out, out2)
    else:  # h in two parts: half a step of the second one
        _within(out, ref, P.forward_bound(x, *w, kind, P.HALF ** 2))
    g, u = (x.double() @ v.double().T for v in w[:2])
    eg, eu = (H * P.F32 * (x.double().abs() @ v.double().abs().T) for v in w[:2])
    a, s = P.act_slope(g, kind)
    ea, es = P.SLOPE * eg + 2.0 ** -20 * a.abs(), P.CURVE * eg + 2.0 ** -20
    sa, sd, sh = _saved_parts(saved, m, I)
    _within(sa, a, ea)
    _within(sd, u * s, u.abs() * es + eu * s.abs() + eu * es + 2.0 ** -22 * (u * s).abs())
    eh = a.abs() * eu + ea * u.abs() + ea * eu + 2.0 ** -22 * (a * u).abs()
    _within(sh, a * u, eh + P.HALF * ((a * u).abs() + eh))
    assert blk.device_status() == 0


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,H,I", FFN_SIZES)
def test_backward(B, m, H, I, kind):
    w = _weights(H + I + 1, H, I)
    x, dout = _n(m, m, H), _n(m + 1, m, H)
    blk = B.GatedFfn(*w, act=kind)
    _, saved = blk.forward(x, save=True)
    got = blk.backward(dout, x, saved)
    ref = P.backward(dout, x, *w, kind)
    for g, r, b in zip(got, ref, P.backward_bounds(dout, x, *w, kind)):
        _within(g, r, b)
    assert blk.device_status() == 0
    # only the gradients asked for
    dx, *none = blk.backward(dout, x, saved, need_dw=False)
    assert torch.equal(dx, got[0]) and none == [None] * 3
    none, *dw = blk.backward(dout, x, saved, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dw, got[1:]))


def test_backward_against_differences(B):
    """The kernels' gradients along a direction against central differences of the 64-bit forward
    pass: off by no more than their bounds summed over the direction, and the difference's own error."""
    m, H, I = 24, 64, 96
    w = _weights(9, H, I)
    x, dout = _n(1, m, H), _n(2, m, H)
    blk = B.GatedFfn(*w, act="gelu")
    _, saved = blk.forward(x, save=True)
    got = blk.backward(dout, x, saved)
    leaves = [t.double() for t in (x, *w)]
    for i, (g, b) in enumerate(zip(got, P.backward_bounds(dout, x, *w, "gelu"))):
        v = torch.randn(leaves[i].shape, device="cuda", dtype=torch.float64)
        e = 1e-5
        hi, lo = ([t + s * e * v if j == i else t for j, t in enumerate(leaves)] for s in (1, -1))
        diff = ((P.forward(*hi, "gelu") - P.forward(*lo, "gelu")) * dout.double()).sum() / (2 * e)
        assert abs(diff - (g.double() * v).sum()) <= (b * v.abs()).sum() + 1e-6 * (1 + g.double().abs().sum())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,H,I", [(1, 7168, 2048), (1, 32, 32), (3, 96, 160), (16, 256, 128), (48, 1024, 512), (65, 544, 1056),
                                   (128, 256, 256), (200, 512, 416), (333, 1056, 2080)])
def test_mx_forward(B, m, H, I, kind):
    pairs, vals = _quantised(B, _weights(H + I, H, I))
    x = _n(m, m, H)
    blk = B.GatedFfn(*pairs, act=kind)
    ref, bound = P.mx_forward(x, *vals, kind)
    _within(blk.forward(x), ref, bound)
    assert blk.device_status() == 0


@pytest.mark.parametrize("mx", [False, True])
def test_forward_strided_rows_and_no_rows(B, mx):
    H, I = 256, 160
    w = _weights(5, H, I)
    blk = B.GatedFfn(*(_quantised(B, w)[0] if mx else w))
    base = _n(8, 70, 3 * H)
    x = base[:, H:2 * H]
    assert torch.equal(blk.forward(x), blk.forward(x.contiguous()))
    assert blk.forward(x[:0]).shape == (0, H)
    if not mx:
        dbase = _n(9, 70, 2 * H)
        dout = dbase[:, H:]
        _, saved = blk.forward(x, save=True)
        a, b = blk.backward(dout, x, saved), blk.backward(dout.contiguous(), x.contiguous(), saved)
        assert all(torch.equal(s, t) for s, t in zip(a, b))
        _, s0 = blk.forward(x[:0], save=True)
        dx, *dw = blk.backward(dout[:0], x[:0], s0)
        assert dx.shape == (0, H) and not any(t.any() for t in dw)


def test_a_bad_row_spoils_no_other(B):
    H, I = 264, 272
    w = _weights(11, H, I)
    blk = B.GatedFfn(*w)
    x = _n(12, 300, H)
    good = blk.forward(x)
    x2 = x.clone()
    x2[17, 3] = float("nan")
    x2[290, 5] = float("inf")
    out = blk.forward(x2)
    bad = torch.zeros(300, dtype=torch.bool, device="cuda")
    bad[[17, 290]] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.isnan(out[17]).all()


def test_extreme_pre_activations(B):
    """act and its slope where the exponential overflows and underflows: g of +-2^k up to 2^30."""
    H = I = 8
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    e = torch.tensor([-30, -3, 0, 2, 4, 6.5, 8, 30.0], device="cuda")
    x = torch.cat([torch.exp2(e), -torch.exp2(e)]).reshape(-1, 1).expand(-1, 8).to(torch.bfloat16).contiguous()
    dout = _n(3, 16, 8)
    for kind in ("silu", "gelu"):
        blk = B.GatedFfn(eye, eye, eye, act=kind)
        out, saved = blk.forward(x, save=True)
        w = (eye, eye, eye)
        xs = x.double()
        # h = act(g) g, rounded twice; below 2^-120 (exp(-t) past 2^126) the kernel may give 0
        ref = P.forward(x, *w, kind)
        assert torch.isfinite(out).all()
        assert ((out.double() - ref).abs() <= 3 * P.HALF * ref.abs() + 1e-30).all()
        got = blk.backward(dout, x, saved)
        want = P.backward(dout, x, *w, kind)
        assert all(torch.isfinite(t).all() for t in got)
        a, s = P.act_slope(xs, kind)
        # dx = dh (g s(g) + act(g)): each part rounded once, their sum once
        part = (dout.double() * xs * s).abs() + (dout.double() * a).abs()
        assert ((got[0].double() - want[0]).abs() <= 3 * P.HALF * part + 1e-30 + 2.0 ** -20 * (dout.double() * xs).abs()).all()


@pytest.mark.parametrize("mx", [False, True])
def test_offsets_past_32_bits(B, mx):
    """h has 2.4e9 elements (MXFP4: as many bytes of codes): the last rows against the formula, and
    alone; the last rows of dx likewise."""
    H, I, m, last = 64, 8192, 600_000 if mx else 300_000, 300
    w = _weights(7, H, I)
    x = _n(8, m, H)
    if mx:
        pairs, vals = _quantised(B, w)
        blk = B.GatedFfn(*pairs)
        ref, bound = P.mx_forward(x[-last:], *vals, "silu")
        _within(blk.forward(x)[-last:], ref, bound)
        return
    blk = B.GatedFfn(*w)
    tail = x[-last:].contiguous()
    out, saved = blk.forward(x, save=True)
    _within(out[-last:], P.forward(tail, *w, "silu"), P.forward_bound(tail, *w, "silu"))
    dx, *_ = blk.backward(x, x, saved, need_dw=False)
    _within(dx[-last:], P.backward(tail, tail, *w, "silu")[0], P.backward_bounds(tail, tail, *w, "silu")[0])
    assert blk.device_status() == 0


def test_quant_past_32_bits(B):
    rows, n = 300_000, 8192
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    x[-200:] = _n(5, 200, n)
    codes, scales = B.moe_mxfp4_quant(x)
    back = B.moe_mxfp4_dequant(codes, scales)[-200:].double()
    assert torch.equal(back, P.mx_round(x[-200:]))


def test_graph_capture_and_other_streams(B):
    """Forward and backward captured in a graph, replayed on new inputs, and run on a side stream:
    the same bits as eager calls."""
    H, I, m = 512, 384, 150
    w = _weights(21, H, I)
    blk = B.GatedFfn(*w)
    x, dout = _n(22, m, H), _n(23, m, H)
    blk.forward(x, save=True)
    blk.workspace(m, True, x.device)  # exists before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, saved = blk.forward(x, save=True)
        grads = blk.backward(dout, x, saved)
    for seed in (31, 32):
        x.copy_(_n(seed, m, H))
        dout.copy_(_n(seed + 10, m, H))
        g.replay()
        torch.cuda.synchronize()
        e_out, e_saved = blk.forward(x, save=True)
        e_grads = blk.backward(dout, x, e_saved)
        assert torch.equal(out, e_out) and torch.equal(_saved_parts(saved, m, I)[2], _saved_parts(e_saved, m, I)[2]) and all(torch.equal(a, b) for a, b in zip(grads, e_grads))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s_out = blk.forward(x, stream=st)
    st.synchronize()
    assert torch.equal(s_out, e_out)


def test_repeatable(B):
    H, I, m = 1032, 776, 555
    w = _weights(41, H, I)
    blk = B.GatedFfn(*w)
    x, dout = _n(42, m, H), _n(43, m, H)
    out, saved = blk.forward(x, save=True)
    first = (out, _saved_parts(saved, m, I)[2], *blk.backward(dout, x, saved))
    for _ in range(3):
        o, s = blk.forward(x, save=True)
        assert all(torch.equal(a, b) for a, b in zip(first, (o, _saved_parts(s, m, I)[2], *blk.backward(dout, x, s))))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("m", [3, 300])
def test_a_wait_that_runs_out(B, mx, m):
    """A stalled issuer ends its kernel by the wait limit with the error word set; the call after it
    is whole."""
    H, I = 256, 512
    w = _weights(2, H, I)
    blk = B.GatedFfn(*(_quantised(B, w)[0] if mx else w))
    x = _n(3, m, H)
    want = blk.forward(x)
    if not mx:
        _, saved = blk.forward(x, save=True)
        grads = blk.backward(x, x, saved)
    assert blk.device_status() == 0
    blk.set_wait_limit(20_000_000)
    blk.stall_test(True)
    blk.forward(x)
    assert blk.device_status() == 2  # read, and cleared
    if not mx:
        blk.backward(x, x, saved)
        assert blk.device_status() == 2
    blk.stall_test(False)
    blk.set_wait_limit(0)
    assert torch.equal(blk.forward(x), want)
    if not mx:
        assert all(torch.equal(a, b) for a, b in zip(blk.backward(x, x, saved), grads))
    assert blk.device_status() == 0


def test_refusals(B):
    H, I = 64, 96
    w1, w3, w2 = _weights(1, H, I)
    blk = B.GatedFfn(w1, w3, w2)
    x = _n(2, 10, H)
    _, saved = blk.forward(x, save=True)
    for bad in (x.float(), x[:, :56], x.T, x.cpu(), x[0], x[:, 1:].contiguous()):
        with pytest.raises(ValueError):
            blk.forward(bad)
    with pytest.raises(ValueError):
        blk.forward(x, out=torch.empty(9, H, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        blk.backward(x[:5], x, saved)
    with pytest.raises(ValueError):
        blk.backward(x, x, saved[:-4])
    with pytest.raises(ValueError):
        blk.backward(x, x, saved.bfloat16())
    with pytest.raises(ValueError):
        B.GatedFfn(w1, w3, w2.T)
    with pytest.raises(ValueError):
        B.GatedFfn(w1, w2, w2)
    pairs = _quantised(B, (w1, w3, w2))[0]
    mx = B.GatedFfn(*pairs)
    with pytest.raises(B.MoeError) as e:
        mx.forward(x, save=True)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(B.MoeError):
        mx.backward(x, x, saved)
    with pytest.raises(ValueError):
        B.moe_mxfp4_gemm(*pairs[0], *pairs[2])
    lib, p = B.load_library(), B._p
    ws = blk.workspace(10, True, x.device)
    out = torch.empty_like(x)
    assert lib.moe_ffn_forward(blk.handle, p(x), H, 10, p(out), None, p(ws), 256, None) == B.MOE_ERR_WORKSPACE
    assert lib.moe_ffn_forward(blk.handle, p(x), H - 8, 10, p(out), None, p(ws), ws.numel(), None) == 1
    assert lib.moe_ffn_forward(blk.handle, p(x), H, 10, p(out), saved.data_ptr() + 16, p(ws), ws.numel(), None) == 1
    assert lib.moe_ffn_forward(blk.handle, p(x), H, -1, p(out), None, p(ws), ws.numel(), None) == 1
    assert lib.moe_ffn_forward(blk.handle, p(x), H, 1 << 30, p(out), None, p(ws), ws.numel(), None) == 2
    assert lib.moe_ffn_backward(blk.handle, p(x), H, p(x), H, p(saved), 10, p(out), p(w1), None, None, p(ws),
                                ws.numel(), None) == 1


@pytest.mark.parametrize("m,k", [(1, 32), (1, 7168), (7, 544), (9, 4128), (16, 1056)])
def test_few_tokens_are_quantised_alike(B, m, k):
    """Up to 16 bf16 tokens are quantised inside the product's kernel: the same bits as by
    moe_mxfp4_quant, with zero, infinite and strided rows among them."""
    (w,), _ = _quantised(B, [_n(4, 520, k, std=k ** -0.5)])
    base = _n(6, m, k + 72, dtype=torch.float32) * torch.exp2(torch.randint(-30, 30, (m, 1), device="cuda").float())
    x = base.bfloat16()[:, 8:k + 8]
    if m > 5:
        x[1] = 0
        x[3, 5] = float("inf")
        x[4, k - 1] = float("nan")
    got = B.moe_mxfp4_linear(x, *w)
    want = B.moe_mxfp4_gemm(*B.moe_mxfp4_quant(x), *w)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    if m > 5:
        assert torch.isnan(got[3:5]).all() and not got[1].any() and torch.isfinite(got[5:]).all()


def test_capture_of_the_linear(B):
    """A product whose stream has no workspace yet, first called while a graph is captured."""
    (w,), _ = _quantised(B, [_n(4, 264, 320)])
    x = _n(6, 200, 320)
    want = B.moe_mxfp4_linear(x, *w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = B.moe_mxfp4_linear(x, *w)
    x.copy_(_n(7, 200, 320))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, B.moe_mxfp4_linear(x, *w)) and not torch.equal(got, want)
    assert B.mxfp4_device_status() == 0


def test_calls_on_a_given_stream_allocate_on_it(B):
    """Blocks freed on the current stream are not handed to a call that runs on another one."""
    H, I = 512, 256
    blk = B.GatedFfn(*_weights(3, H, I))
    x = _n(1, 64, H)
    want = blk.forward(x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    for _ in range(4):
        t = torch.empty(64, H, dtype=torch.bfloat16, device="cuda")
        busy.add_(1)
        t.copy_(x)  # still to come when t goes back to the current stream's pool
        del t
        outs = [blk.forward(x, stream=st) for _ in range(3)]
        st.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_example_trains_and_serves():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_and_serve_ffn.py")
    spec = importlib.util.spec_from_file_location("train_and_serve_ffn", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last, prompt, token = mod.run(hidden=256, inter=512, tokens=1024, steps=60, log=lambda s: None)
    assert last < 0.7 * first
    # two quantised operands per product: e2m1 steps of 1/4 to 1/2 of a value give about 0.1 each, in three products
    assert prompt < 0.35 and token < 0.5


@pytest.mark.parametrize("mx", [False, True])
def test_fewer_tokens_on_one_handle(B, mx):
    """A handle whose largest call had 9 to 15 tokens takes a call of 1 to 8 after it."""
    H, I = 256, 768
    w = _weights(13, H, I)
    w = _quantised(B, w)[0] if mx else w
    x = _n(14, 15, H)
    for first in (9, 12, 15):
        blk = B.GatedFfn(*w)
        for m in (first, 8, 1):
            assert torch.equal(blk.forward(x[:m]), B.GatedFfn(*w).forward(x[:m]))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_h_past_bf16_is_infinite_at_every_number_of_tokens(B, kind):
    """h that overflows fp32, and h that fp32 holds but bf16 does not, give infinities of W2's sign
    where h goes on in two bf16 parts (4 and 8 tokens) as where it does in one (9 and 12)."""
    eye = torch.eye(8, device="cuda")
    sign = torch.tensor([1.0, -1.0] * 4, device="cuda")
    blk = B.GatedFfn(eye.bfloat16(), 2 * eye.bfloat16(), sign[:, None].expand(8, 8).bfloat16().contiguous(), act=kind)
    x = torch.ones(12, 8, device="cuda")
    x[1, 3] = 2.0 ** 64                # h = 2^129
    x[2, 5] = 181 / 128 * 2.0 ** 63    # h = 1.9996 2^127: a step below 2^128 in fp32, 2^128 in bf16
    x = x.bfloat16()
    for m in (4, 8, 9, 12):
        out = blk.forward(x[:m]).float()
        assert torch.equal(out[1], sign * float("inf")) and torch.equal(out[2], sign * float("inf"))
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[3:]).all()
    assert blk.device_status() == 0


def _others(like, count=8):
    """Tensors that take up memory freed just now, filled with a pattern."""
    return [torch.full_like(like, 0x5A) for _ in range(count)]


@pytest.mark.parametrize("mx", [False, True])
def test_a_graph_survives_a_larger_call(B, mx):
    """Warm-up and capture of a small call, a large eager call, then replays: right outputs, and
    nothing written into memory that others have got since."""
    H, I, m = 512, 768, 40
    w = _weights(51, H, I)
    blk = B.GatedFfn(*(_quantised(B, w)[0] if mx else w))
    x, dout = _n(52, m, H), _n(53, m, H)

    def call():
        if mx:
            return (blk.forward(x),)
        out, saved = blk.forward(x, save=True)
        return (out, *blk.backward(dout, x, saved), blk.forward(x[:5]))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    small = blk.workspace(m, not mx, x.device)
    blk.forward(_n(54, 3000, H))
    if not mx:
        blk.backward(_n(54, 3000, H), _n(55, 3000, H), blk.forward(_n(55, 3000, H), save=True)[1])
    assert blk.workspace(m, not mx, x.device).numel() > small.numel()
    shape = torch.empty_like(small)
    del small
    others = [shape, *_others(shape)]
    shape.fill_(0x5A)
    for seed in (61, 62):
        x.copy_(_n(seed, m, H))
        dout.copy_(_n(seed + 10, m, H))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))
        assert all((t == 0x5A).all() for t in others)
    assert blk.device_status() == 0


def test_a_graph_of_products_survives_a_larger_call(B):
    """The same of moe_mxfp4_linear, warmed up on the stream that is then captured."""
    (w,), _ = _quantised(B, [_n(4, 264, 2048)])
    x = _n(6, 200, 2048)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.moe_mxfp4_linear(x, *w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = B.moe_mxfp4_linear(x, *w)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        B.moe_mxfp4_linear(_n(8, 5000, 2048), *w)
        others = _others(torch.empty(1024 + 200 * 1024 + 2 * 16 * 512, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    x.copy_(_n(7, 200, 2048))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, B.moe_mxfp4_linear(x, *w))
    assert all((t == 0x5A).all() for t in others)
    assert B.mxfp4_device_status() == 0 and B.mxfp4_device_status(st) == 0


@pytest.mark.parametrize("rows,n", [(1, 32), (5, 96), (300, 544)])
def test_buffers_aligned_to_16_bytes_alone(B, rows, n):
    """What the C entry points ask of their buffers is enough: all of them 16 bytes past a multiple
    of 32, with nothing written around the outputs."""
    def at16(nbytes):
        t = torch.full((nbytes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        assert t.data_ptr() % 32 == 0
        return t, t[16:16 + nbytes], t.data_ptr() + 16
    lib = B.load_library()
    for dtype, fn in ((torch.bfloat16, lib.moe_mxfp4_quant), (torch.float32, lib.moe_mxfp4_quant_f32)):
        x = _n(rows, rows, n, dtype=dtype)
        size = rows * n * x.element_size()
        _, xm, xp = at16(size)
        xm.copy_(x.reshape(-1).view(torch.uint8))
        want_c, want_s = B.moe_mxfp4_quant(x)
        codes, cm, cp = at16(want_c.numel())
        scales, sm, sp = at16(want_s.numel())
        out, om, op = at16(rows * n * 2)
        assert fn(xp, n, rows, n, cp, sp, None) == 0
        assert lib.moe_mxfp4_dequant(cp, sp, rows, n, op, None) == 0
        torch.cuda.synchronize()
        assert torch.equal(cm, want_c.reshape(-1))
        sm = sm.reshape(want_s.shape)
        assert torch.equal(B.mxfp4_unpack_scales(sm, rows, n), B.mxfp4_unpack_scales(want_s, rows, n))
        assert torch.equal(om.view(torch.bfloat16).reshape(rows, n), B.moe_mxfp4_dequant(want_c, want_s))
        for t, k in ((codes, cm.numel()), (scales, sm.numel()), (out, om.numel())):
            assert (t[:16] == 0x5A).all() and (t[16 + k:] == 0x5A).all()


def test_a_captured_header_is_not_taken_for_clean(B):
    """A workspace first seen by a captured call: its header is zeroed in the graph, and again for an
    eager call that comes before any replay."""
    H, I, m = 64, 96, 20
    blk = B.GatedFfn(*_weights(1, H, I))
    x = _n(2, m, H)
    want = blk.forward(x)
    lib, p = B.load_library(), B._p
    ws = torch.full((blk.workspace_size(m),), 0x5A, dtype=torch.uint8, device="cuda")
    out, code = torch.zeros_like(x), ctypes.c_int32()

    def call(stream):
        assert lib.moe_ffn_forward(blk.handle, p(x), H, m, p(out), None, p(ws), ws.numel(), B._stream(stream)) == 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(None)
    assert (ws == 0x5A).all()
    call(None)
    assert lib.moe_device_status(p(ws), B._stream(), ctypes.byref(code)) == 0 and code.value == 0
    assert torch.equal(out, want)
    ws.fill_(0x5A)
    out.zero_()
    g.replay()
    assert lib.moe_device_status(p(ws), B._stream(), ctypes.byref(code)) == 0 and torch.equal(out, want)


def test_an_error_is_read_after_the_workspace_has_grown(B):
    H, I = 256, 512
    blk = B.GatedFfn(*_weights(2, H, I))
    x = _n(3, 3, H)
    blk.workspace(3, False, x.device)
    assert blk.device_status() == 0  # before any call
    blk.set_wait_limit(20_000_000)
    blk.stall_test(True)
    blk.forward(x)
    blk.stall_test(False)
    blk.set_wait_limit(0)
    blk.forward(_n(4, 2000, H))
    assert blk.device_status() == 2 and blk.device_status() == 0


def test_products_of_two_threads_on_one_stream(B):
    import threading
    (w,), _ = _quantised(B, [_n(4, 256, 512)])
    xs = [_n(60 + i, 300, 512) for i in range(4)]
    want = [B.moe_mxfp4_linear(x, *w) for x in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]

    def work(i):
        for _ in range(200):
            got[i].append(B.moe_mxfp4_linear(xs[i], *w))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == 200 and all(torch.equal(o, v) for o in g) for g, v in zip(got, want))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("grow", [False, True])
def test_a_workspace_let_go_while_another_stream_uses_it(B, mx, grow):
    """A handle's workspace belongs to the stream of its first call.  Outgrown, or gone with the
    handle, while a call on another stream is still to run, it is not given to others before that."""
    H, I, m = 512, 2048, 300
    w = _weights(71, H, I)
    w = _quantised(B, w)[0] if mx else w
    x, big = _n(72, m, H), _n(73, 2000, H)
    blk = B.GatedFfn(*w)
    want = blk.forward(x)
    size = blk.workspace(m, False, x.device).numel()
    st, load = torch.cuda.Stream(), torch.zeros(1 << 28, device="cuda")
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            load.add_(1)  # some 6 ms before the call's turn comes
        blk.forward(x, out=out)
    if grow:
        blk.workspace(2000, False, x.device)
    else:
        del blk
    others = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all((t == 0x5A).all() for t in others) and torch.equal(out, want)


@pytest.mark.parametrize("m", [1, 3, 16, 40, 300])
def test_out_may_be_x(B, m):
    """In place: the linear (up to 16 tokens of bf16 are quantised by the kernel that writes out) and
    both forms of the block."""
    n = 2048
    (w,), _ = _quantised(B, [_n(4, n, n, std=n ** -0.5)])
    x = _n(5, m, n)
    want = B.moe_mxfp4_linear(x, *w)
    for _ in range(5):
        y = x.clone()
        assert B.moe_mxfp4_linear(y, *w, out=y) is y and torch.equal(y, want)
    if m > 1:  # rows of x are twice as long as the output's: out within x
        base = torch.cat([x, x], 1)
        y = base.reshape(-1)[:m * n].reshape(m, n)
        assert torch.equal(B.moe_mxfp4_linear(base[:, n:], *w, out=y), want)
    # x at the start of out's rows, in more row tiles than the device holds at once
    k, n2 = 512, 1 << 16
    (v,), _ = _quantised(B, [_n(4, n2, k, std=k ** -0.5)])
    want, y = B.moe_mxfp4_linear(x[:, :k], *v), torch.zeros(m, n2, dtype=torch.bfloat16, device="cuda")
    y[:, :k] = x[:, :k]
    assert torch.equal(B.moe_mxfp4_linear(y[:, :k], *v, out=y), want)
    ws = _weights(6, n, 512)
    for blk in (B.GatedFfn(*ws), B.GatedFfn(*_quantised(B, ws)[0])):
        want, y = blk.forward(x), x.clone()
        assert blk.forward(y, out=y) is y and torch.equal(y, want)


def test_read_back_past_bf16(B):
    """Scales 252 to 255 with every code: exact, infinite past bf16's range, or NaN."""
    codes = torch.arange(16, dtype=torch.uint8, device="cuda").repeat(4, 2)
    scales = torch.tensor([[252], [253], [254], [255]], dtype=torch.uint8, device="cuda")
    got = B.moe_mxfp4_dequant(P.mx_pack(codes), B.mxfp4_pack_scales(scales))
    want = P.mx_values(codes, scales).to(torch.bfloat16)
    assert torch.isinf(want[1:3]).any(1).all() and torch.isfinite(want[0]).all()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[:3], want[:3])
