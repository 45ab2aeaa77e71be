"""The norm with the residual's addition, the router's losses and gradient, and low-rank adapters on the
GPU, against 64-bit formulas with bounds derived from the roundings (tests/_ops_plain.py)."""
import pytest
import torch

import _ops_plain as P

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def _n(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _ints(seed, lo, hi, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _within(got, ref, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    i = int(over.argmax())
    assert over.max() <= 0, (f"{what} off by {(got - ref).abs().flatten()[i]:.3e}, bound {bound.flatten()[i]:.3e} at {i} of "
                             f"{tuple(got.shape)}: {got.flatten()[i]:.6e} for {ref.flatten()[i]:.6e}")


def _strided(t, extra=24, at=8):
    """The same rows inside a wider buffer."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), 77.0, dtype=t.dtype, device=t.device)
    wide[:, at:at + t.shape[1]] = t
    return wide[:, at:at + t.shape[1]], wide


# ---------------------------------------------------------------- norm

NORM_SIZES = [(1, 8), (3, 24), (1, 7168), (2, 1024), (9, 1032), (17, 256), (40, 264), (33, 520), (31, 776), (333, 1032),
              (5, 8200), (3, 16392), (2, 24576), (700, 2048), (2000, 128), (257, 4104)]


def _check_norm(B, n, x, res, w, eps, fp8):
    out, r = P.norm(x, res, w, eps)
    f32, bf = P.norm_bound(out, x.shape[1])
    if res is not None:
        assert torch.equal(n.residual, r.to(torch.bfloat16))
    if n.out is not None:
        _within(n.out, out, bf, "out")
    if fp8:
        h = x.shape[1]
        assert n.scales.shape == (x.shape[0], -(-h // 128))
        s = n.scales.double()
        top = torch.stack([out[:, c:c + 128].abs().amax(1) for c in range(0, h, 128)], 1)
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        _within(s, want, 2 * P.SMALL * want, "scales")
        each = s.repeat_interleave(128, 1)[:, :h]
        _within(P.e4m3(n.codes) * each, out, f32 + 2.0 ** -4 * (out.abs() + f32) + 2.0 ** -10 * each + P.SMALL * out.abs(), "codes")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("m,h", NORM_SIZES)
def test_norm(B, m, h, add, fp8):
    x = _n(m + h, m, h)
    res = _n(m + h + 1, m, h, std=4.0) if add else None
    w = 1 + _n(h, h, std=0.3, dtype=torch.float32)
    kept = res.clone() if add else None
    n = B.moe_add_rmsnorm(x, w, 1e-6, residual=res, fp8=fp8)
    _check_norm(B, n, x, res, w, 1e-6, fp8)
    if add:
        assert torch.equal(res, kept) and n.residual.data_ptr() != res.data_ptr()


def test_norm_codes_are_the_quantisers(B):
    """Where out is a bf16 number, its codes and scales are those that moe_act_quant_fp8 makes of it."""
    x = torch.ones(5, 1024, device="cuda", dtype=torch.bfloat16)  # rstd = 1 with eps = 0
    x[:, ::2] = -1
    w = _n(3, 1024, std=2.0).float()
    w[128:256] = 0
    n = B.moe_add_rmsnorm(x, w, 0.0, fp8=True)
    codes, scales = B.moe_act_quant_fp8(n.out)
    assert torch.equal(n.codes, codes) and torch.equal(n.scales, scales) and (scales[:, 1] == 1).all()


def test_norm_codes_of_values_too_small_for_a_scale(B):
    """Blocks whose largest value over 448 is below fp32's numbers: zero codes with a scale of 1, beside
    zeros and blocks of ordinary values."""
    x = torch.ones(3, 512, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(512, device="cuda")
    w[:128] = 1e-43
    w[5], w[128:256] = 0.0, 1e-40
    n = B.moe_add_rmsnorm(x, w, 0.0, fp8=True)
    assert (n.scales[:, 0] == 1).all() and not n.codes[:, :128].any()
    v = P.e4m3(n.codes) * n.scales.double().repeat_interleave(128, 1)
    # 1e-40 / 448 is 159 of fp32's smallest steps, off by half a one: 2^-8 of the value, and e4m3's 2^-4
    assert ((v[:, 128:256] - 1e-40).abs() <= 1e-40 * (2.0 ** -4 + 2.0 ** -7)).all()
    assert (n.codes[:, 256:] == 0x7E).all()  # 448


def test_norm_eight_bits_alone_and_in_place(B):
    m, h = 37, 1160
    x, res, w = _n(1, m, h), _n(2, m, h), _n(3, h, dtype=torch.float32)
    want = B.moe_add_rmsnorm(x, w, 1e-5, residual=res, fp8=True)
    only = B.moe_add_rmsnorm(x, w, 1e-5, residual=res, bf16=False, fp8=True)
    assert only.out is None and torch.equal(only.codes, want.codes) and torch.equal(only.residual, want.residual)
    x2, res2 = x.clone(), res.clone()
    n = B.moe_add_rmsnorm(x2, w, 1e-5, residual=res2, residual_out=res2, out=x2)
    assert n.out is x2 and n.residual is res2 and torch.equal(x2, want.out) and torch.equal(res2, want.residual)


def test_norm_strided_rows_and_no_rows(B):
    m, h = 41, 520
    x, res, w = _n(1, m, h), _n(2, m, h), _n(3, h, dtype=torch.float32)
    want = B.moe_add_rmsnorm(x, w, residual=res)
    xs, _ = _strided(x)
    rs, wide = _strided(res, 40, 16)
    got = B.moe_add_rmsnorm(xs, w, residual=rs, residual_out=rs)
    assert torch.equal(got.out, want.out) and torch.equal(rs, want.residual)
    assert (wide[:, :16] == 77).all() and (wide[:, 16 + h:] == 77).all()
    both = torch.cat((x, res), 1)  # x and residual side by side in one buffer, the residual updated there
    got = B.moe_add_rmsnorm(both[:, :h], w, residual=both[:, h:], residual_out=both[:, h:])
    assert torch.equal(got.out, want.out) and torch.equal(both[:, h:], want.residual) and torch.equal(both[:, :h], x)
    n = B.moe_add_rmsnorm(x[:0], w, residual=res[:0], fp8=True)
    assert n.out.shape == (0, h) and n.codes.shape == (0, h) and n.scales.shape == (0, 5)
    dx, dw = B.moe_add_rmsnorm_backward(x[:0], res[:0], w)
    assert dx.shape == (0, h) and not dw.any()


@pytest.mark.parametrize("h", [520, 2056])
def test_norm_rows_of_zeros_infinities_and_nan(B, h):
    """Zero rows stay zero (eps 0 makes them NaN, as the formula has it); a bad row spoils no other."""
    x, w = _n(1, 12, h), _n(2, h, dtype=torch.float32)
    x[2] = 0
    x[4, 3] = INF
    x[6, h - 1] = NAN
    n = B.moe_add_rmsnorm(x, w, fp8=True)
    good = [0, 1, 2, 3, 5, 7, 8, 9, 10, 11]
    ref = B.moe_add_rmsnorm(x[good].contiguous(), w, fp8=True)
    assert torch.equal(n.out[good], ref.out) and torch.equal(n.codes[good], ref.codes) and torch.equal(n.scales[good], ref.scales)
    assert not n.out[2].any() and not n.codes[2].any() and (n.scales[2] == 1).all()
    assert torch.isnan(n.out[4, 3]) and not n.out[4, 4:].any() and torch.isnan(n.out[6]).all()
    assert torch.isnan(P.e4m3(n.codes[6])).all() and torch.isnan(P.e4m3(n.codes[4]))[3]
    assert torch.isnan(B.moe_add_rmsnorm(x[2:3], w, 0.0).out).all()


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("m,h", NORM_SIZES)
def test_norm_backward(B, m, h, add):
    r, dout, w = _n(m, m, h, std=3.0), _n(h, m, h), 1 + _n(m + h, h, std=0.3, dtype=torch.float32)
    dres = _n(m + h + 2, m, h) if add else None
    dx, dw = B.moe_add_rmsnorm_backward(dout, r, w, 1e-6, dresidual=dres)
    want, wdw, bx, bw = P.norm_backward(dout, r, w, 1e-6, dres)
    _within(dx, want, bx, "dx")
    _within(dw, wdw, bw, "dweight")
    dx2, none = B.moe_add_rmsnorm_backward(dout, r, w, 1e-6, dresidual=dres, need_dw=False)
    assert none is None and torch.equal(dx, dx2)


def test_norm_backward_many_rows(B):
    """Blocks that go over many rows each, for rows of a warp and of a block; bounds as by their counts."""
    for m, h in ((40000, 264), (20000, 1544)):
        r, dout, w = _n(m, m, h), _n(h, m, h), _n(1, h, dtype=torch.float32)
        dx, dw = B.moe_add_rmsnorm_backward(dout, r, w)
        want, wdw, bx, bw = P.norm_backward(dout, r, w, 1e-6, None)
        _within(dx, want, bx, "dx")
        _within(dw, wdw, bw, "dweight")


def test_norm_backward_against_differences(B):
    """The gradient against differences of the forward formula in 64 bits: central ones of step d err
    by d^2 times a third derivative, which here stays below 1e-3 of d^2."""
    m, h = 4, 64
    r, dout, w = _n(1, m, h), _n(2, m, h), _n(3, h, dtype=torch.float32)
    dx, dw = B.moe_add_rmsnorm_backward(dout, r, w, 1e-5)
    _, _, bx, bw = P.norm_backward(dout, r, w, 1e-5, None)

    def loss(rr, ww):
        return (rr / torch.sqrt(rr.square().mean(1, keepdim=True) + 1e-5) * ww * dout.double()).sum()
    d = 1e-4
    for i, j in ((0, 0), (1, 33), (3, 63)):
        up, dn = r.double().clone(), r.double().clone()
        up[i, j] += d
        dn[i, j] -= d
        diff = (loss(up, w.double()) - loss(dn, w.double())) / (2 * d)
        assert (dx[i, j].double() - diff).abs() <= bx[i, j] + 1e-7
    for j in (0, 17, 63):
        up, dn = w.double().clone(), w.double().clone()
        up[j] += d
        dn[j] -= d
        diff = (loss(r.double(), up) - loss(r.double(), dn)) / (2 * d)
        assert (dw[j].double() - diff).abs() <= bw[j] + 1e-9


@pytest.mark.parametrize("h", [264, 2056])
@pytest.mark.parametrize("size", [2.0 ** -55, 2.0 ** 55])
def test_norm_of_very_small_and_large_rows(B, h, size):
    """Rows whose squares are still fp32's, without eps: forward and backward as for rows of any size."""
    r, dout, w = (_n(1, 5, h, dtype=torch.float32) * size).bfloat16(), _n(2, 5, h), _n(3, h, dtype=torch.float32)
    n = B.moe_add_rmsnorm(r, w, 0.0, fp8=True)
    _check_norm(B, n, r, None, w, 0.0, True)
    dout = (dout.float() * size).bfloat16()  # dx is then of ordinary size
    dx, dw = B.moe_add_rmsnorm_backward(dout, r, w, 0.0)
    want, wdw, bx, bw = P.norm_backward(dout, r, w, 0.0, None)
    _within(dx, want, bx, "dx")
    _within(dw, wdw, bw, "dweight")


def test_norm_backward_strided(B):
    m, h = 23, 1160
    r, dout, dres, w = _n(1, m, h), _n(2, m, h), _n(3, m, h), _n(4, h, dtype=torch.float32)
    want = B.moe_add_rmsnorm_backward(dout, r, w, dresidual=dres)
    got = B.moe_add_rmsnorm_backward(_strided(dout)[0], _strided(r, 8, 0)[0], w, dresidual=_strided(dres, 56, 48)[0])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- the router

ROUTER_SIZES = [(1, 1, 1), (5, 2, 2), (7, 3, 2), (333, 8, 2), (64, 16, 4), (129, 20, 5), (100, 64, 6), (130, 33, 3), (77, 128, 8),
                (200, 100, 32), (90, 130, 7), (300, 256, 8), (65, 257, 8), (50, 512, 8), (40, 513, 9), (37, 1024, 32), (21, 1023, 1),
                (3000, 8, 1), (5000, 60, 4)]


def _router_case(m, E, k, seed=0):
    logits = _n(seed + m, m, E, std=2.0, dtype=torch.float32) + _n(seed + E, E, dtype=torch.float32)
    return logits, torch.topk(logits, k, dim=1).indices.int().contiguous()


def _check_router(B, logits, ids, off, sigmoid, norm=True, scale=1.0, seed=5):
    name = "sigmoid" if sigmoid else "softmax"
    m, k = ids.shape
    S = 1 if off is None else off.numel() - 1
    bal, z, counts = B.moe_balance_loss(logits, ids, off, scoring=name)
    wb, wz, wc = P.router(logits.double(), ids, off, sigmoid)
    bb, bz = P.router_bounds(logits.double(), wb, wz, off)
    assert torch.equal(counts, wc)
    _within(bal, wb, bb, "balance")
    _within(z, wz, bz, "z")
    dw = _n(seed, m, k, dtype=torch.float32)
    db, dz = _n(seed + 1, S, dtype=torch.float32) * m, _n(seed + 2, S, dtype=torch.float32) * m
    for a, b, c in ((dw, db, dz), (dw, None, None), (None, db, None), (None, None, dz), (None, None, None)):
        d = B.moe_route_backward(logits, ids, a, b, c, counts if b is not None else None, off, name, norm, scale)
        want, bound = P.route_backward(logits, ids, off, sigmoid, norm, scale, a, b, c)
        _within(d, want, bound, f"dlogits {[t is not None for t in (a, b, c)]}")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("m,E,k", ROUTER_SIZES)
def test_router(B, m, E, k, sigmoid):
    _check_router(B, *_router_case(m, E, k), None, sigmoid)


@pytest.mark.parametrize("norm,scale", [(True, 2.5), (False, 1.0), (False, 0.5)])
def test_router_sigmoid_weights(B, norm, scale):
    _check_router(B, *_router_case(70, 48, 4), None, True, norm, scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("m,E,cuts", [
    (100, 8, [0, 100]), (100, 8, [0, 0, 1, 1, 64, 99, 99]), (300, 128, [0, 7, 128, 129, 250, 300]), (64, 30, [5, 20, 60]),
    (1000, 16, [0] + [3 * i for i in range(300)] + [950]), (40, 64, [0, 0, 0, 0]), (700, 32, list(range(0, 701))),
    (5000, 256, [0, 1, 4000, 4990]), (2000, 64, [0] * 600 + [1999])])
def test_router_sequences(B, m, E, cuts, sigmoid):
    """Sequences of one token and of many, empty ones, padding in front and behind, more of them than
    shared memory keeps the offsets of."""
    logits, ids = _router_case(m, E, min(4, E))
    _check_router(B, logits, ids, torch.tensor(cuts, dtype=torch.int32, device="cuda"), sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [12, 13, 256])
def test_router_ids_that_name_no_expert_or_one_twice(B, E, sigmoid):
    logits, ids = _router_case(50, E, 4)
    ids[3] = -1
    ids[4, 1:] = -1
    ids[5] = torch.tensor([2, 2, 2, 2], dtype=torch.int32)
    ids[6] = torch.tensor([7, 0, 7, 0], dtype=torch.int32)
    ids[7] = torch.tensor([E, E + 100, -2, 2 ** 31 - 1], dtype=torch.int32)
    ids[8, 0] = -2 ** 31
    _check_router(B, logits, ids, None, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [8, 60, 257])
def test_router_masked_logits(B, E, sigmoid):
    """-inf and the type's lowest value in masked places, rows that are masked whole."""
    logits, ids = _router_case(40, E, 3)
    logits[1, 2:] = -INF
    logits[2] = -INF
    logits[3, :E - 1] = torch.finfo(torch.float32).min
    logits[4, ::2] = -INF
    logits[5] = -200.0 - torch.arange(E, device="cuda")  # far below zero, each sigmoid underflows
    logits[6] = -30.0
    logits[7, 0] = 90.0
    bal, z, counts = B.moe_balance_loss(logits, ids, None, scoring="sigmoid" if sigmoid else "softmax")
    wb, wz, wc = P.router(logits.double(), ids, None, sigmoid)
    bb, bz = P.router_bounds(torch.where(logits < -1e30, torch.full_like(logits, -INF), logits).double(), wb, wz, None)
    assert torch.equal(counts, wc)
    _within(bal, wb, bb, "balance")
    _within(z, wz, bz, "z")
    one = torch.ones(1, device="cuda")
    dw = _n(3, 40, 3, dtype=torch.float32)
    d = B.moe_route_backward(logits, ids, dw, one * 40, one * 40, counts, None, "sigmoid" if sigmoid else "softmax")
    assert torch.isfinite(d).all() and not d[2].any() and not d[4, ::2].any() and not d[1, 2:].any()
    rows = [0, 6, 7, *range(8, 40)]
    lowest = torch.where(logits < -1e30, torch.full_like(logits, -1e5), logits)  # p = 0 in 64 bits too
    lowest[2] = 0
    want, bound = P.route_backward(lowest, ids, None, sigmoid, True, 1.0, dw, one * 40, one * 40)
    _within(d[rows], want[rows], bound[rows], "dlogits")
    rows = [1, 3, 4]
    live = logits[rows] > -1e30
    _within(d[rows] * live, want[rows] * live, bound[rows] + 1e-30, "dlogits of masked rows")
    _within(d[5:6], want[5:6], bound[5:6] + 2.0 ** -15 * want[5:6].abs(), "dlogits far below zero")


@pytest.mark.parametrize("E", [4, 48, 256])
def test_router_logits_of_any_alignment(B, E):
    """Logits that begin 4 bytes past a multiple of 16 give what aligned ones give, within the bounds
    of both (they are added up in another order)."""
    logits, ids = _router_case(90, E, 3)
    off = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    odd = torch.empty(90 * E + 1, device="cuda")[1:].view(90, E)
    odd.copy_(logits)
    assert odd.data_ptr() % 16 == 4 and odd.is_contiguous()
    for sigmoid in (False, True):
        _check_router(B, odd, ids, off, sigmoid)


def test_router_bad_rows_spoil_no_other(B):
    logits, ids = _router_case(30, 64, 4)
    off = torch.tensor([0, 10, 20, 28], dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    dw = torch.ones(30, 4, device="cuda")
    bal, z, counts = B.moe_balance_loss(logits, ids, off)
    d = B.moe_route_backward(logits, ids, dw, one, one, counts, off)
    logits[12, 5] = NAN
    logits[29] = NAN  # padding
    ids[29] = -1
    bal2, z2, counts2 = B.moe_balance_loss(logits, ids, off)
    d2 = B.moe_route_backward(logits, ids, dw, one, one, counts2, off)
    assert torch.equal(counts, counts2) and torch.isnan(bal2[1]) and torch.isnan(z2[1])
    assert torch.equal(bal[[0, 2]], bal2[[0, 2]]) and torch.equal(z[[0, 2]], z2[[0, 2]])
    rows = [i for i in range(29) if i != 12]
    assert torch.equal(d[rows], d2[rows]) and torch.isnan(d2[12]).all() and not d2[29].any()


def test_router_against_differences(B):
    """The gradient against central differences of the losses and weights in 64 bits (step 1e-4: their
    own error is below 1e-7 here)."""
    logits, ids = _router_case(20, 12, 3)
    off = torch.tensor([0, 8, 20], dtype=torch.int32, device="cuda")
    dw, db, dz = _n(1, 20, 3, dtype=torch.float32), _n(2, 2, dtype=torch.float32), _n(3, 2, dtype=torch.float32)
    for sigmoid in (False, True):
        _, _, counts = B.moe_balance_loss(logits, ids, off, scoring="sigmoid" if sigmoid else "softmax")
        d = B.moe_route_backward(logits, ids, dw, db, dz, counts, off, "sigmoid" if sigmoid else "softmax", True, 1.5)
        _, bound = P.route_backward(logits, ids, off, sigmoid, True, 1.5, dw, db, dz)

        def loss(l):
            bal, z, _ = P.router(l, ids, off, sigmoid)
            w = P.route_weights(l, ids, sigmoid, True, 1.5)
            return (bal * db.double()).sum() + (z * dz.double()).sum() + (w * dw.double()).sum()
        for t, e in ((0, 0), (7, 11), (8, 3), (19, 5)):
            up, dn = logits.double().clone(), logits.double().clone()
            up[t, e] += 1e-4
            dn[t, e] -= 1e-4
            assert (d[t, e].double() - (loss(up) - loss(dn)) / 2e-4).abs() <= bound[t, e] + 1e-7


def test_router_of_no_tokens(B):
    logits, ids = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    bal, z, counts = B.moe_balance_loss(logits, ids, off)
    assert not bal.any() and not z.any() and counts.shape == (3, 8) and not counts.any()
    assert B.moe_route_backward(logits, ids, seq_offsets=off, dz=z).shape == (0, 8)


def test_router_offsets_that_make_no_sense_touch_nothing_else(B):
    """Falling offsets and such outside the tokens: values unspecified, nothing written around the
    outputs and the right values in the calls after."""
    logits, ids = _router_case(300, 16, 2)
    good = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    want = B.moe_balance_loss(logits, ids, good)
    one = torch.ones(2, device="cuda")
    for bad in ([200, 100, 50], [-5, 1000, 40], [2 ** 31 - 1, -2 ** 31, 7], [-2 ** 31, 2 ** 31 - 1, -1]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        lib, p = B.load_library(), B._p
        out = torch.full((4096,), 7.0, device="cuda")
        counts = torch.full((4096,), 7, dtype=torch.int32, device="cuda")
        ws = torch.full((1 << 16,), 0x5A, dtype=torch.uint8, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        assert lib.moe_balance_loss(p(logits), p(ids), 300, 16, 2, p(off), 2, 0, p(out[1024:]), p(out[2048:]), p(counts[1024:]), p(ws), 1024, st) == 0
        d = B.moe_route_backward(logits, ids, dbalance=one, dz=one, counts=counts[1024:1056].view(2, 16), seq_offsets=off)
        torch.cuda.synchronize()
        assert (out[:1024] == 7).all() and (out[1026:2048] == 7).all() and (out[2050:] == 7).all()
        assert (counts[:1024] == 7).all() and (counts[1056:] == 7).all() and (ws[1024:] == 0x5A).all() and d.shape == (300, 16)
        assert all(torch.equal(a, b) for a, b in zip(B.moe_balance_loss(logits, ids, good), want))


def test_router_takes_what_the_layer_routes(B):
    """moe_route's weights are what the gradient is of, for both scorings."""
    from mixture_experts_ffn_gemv_gb300 import inputs as I
    for sigmoid in (False, True):
        shape = I.LayerShape(hidden=256, num_experts=16, top_k=4, inter=128, scoring="sigmoid" if sigmoid else "softmax",
                             routed_scaling=2.5 if sigmoid else 1.0)
        w = {n: torch.zeros(16, 128, 256, dtype=torch.bfloat16, device="cuda") for n in ("w1", "w3")}
        w["w2"] = torch.zeros(16, 256, 128, dtype=torch.bfloat16, device="cuda")
        layer = B.MoeLayer(shape, w)
        x, rw = _n(1, 60, 256), _n(2, 16, 256, std=0.1, dtype=torch.float32)
        ids, tw, logits = layer.moe_route(x, rw, logits=True)
        want = P.route_weights(logits.double(), ids, sigmoid, True, 2.5 if sigmoid else 1.0)
        _within(tw, want, 4 * P.SMALL * want, "topk_w")
        bal, z, counts = layer.moe_balance_loss(logits, ids)
        one, dw = torch.ones(1, device="cuda"), _n(3, 60, 4, dtype=torch.float32)
        d = layer.moe_route_backward(logits, ids, dw, one, one, counts)
        want, bound = P.route_backward(logits, ids, None, sigmoid, True, 2.5 if sigmoid else 1.0, dw, one, one)
        _within(d, want, bound, "dlogits")
        assert int(counts.sum()) == 240


# ---------------------------------------------------------------- adapters

LORA_SIZES = [(1, 7168, 2048, 16, 8), (1, 8, 8, 8, 1), (2, 72, 1032, 128, 3), (5, 8200, 264, 24, 4), (64, 2048, 712, 16, 40),
              (33, 136, 136, 72, 5), (64, 264, 8200, 64, 2), (65, 64, 64, 8, 1), (66, 264, 200, 8, 5), (128, 256, 128, 16, 3),
              (129, 520, 1032, 32, 2), (300, 1016, 680, 64, 4), (300, 72, 520, 128, 7), (200, 4104, 264, 24, 60),
              (1777, 1016, 2728, 8, 6), (513, 2048, 72, 72, 9), (2500, 328, 264, 48, 130),
              (130, 8, 8, 8, 3), (140, 264, 136, 16, 4), (90, 520, 264, 64, 5), (700, 64, 1032, 120, 20)]


def _lora_case(m, k, d, r, n, seed=0):
    x, y = _n(seed + m, m, k), _n(seed + d, m, d)
    a, b = _n(seed + r, n, r, k, std=k ** -0.5), _n(seed + n, n, d, r, std=r ** -0.5)
    scale = 0.5 + torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    return x, y, a, b, scale


def _requests(seed, m, n, count):
    """Tokens of requests that lie together, some without an adapter."""
    which = _ints(seed, -1, n, count)
    return which[torch.sort(_ints(seed + 1, 0, count, m)).values.long()].contiguous()


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("m,k,d,r,n", LORA_SIZES)
def test_lora(B, m, k, d, r, n, mixed):
    x, y, a, b, scale = _lora_case(m, k, d, r, n)
    ids = _ints(9, -1, n, m) if mixed else _requests(9, m, n, 5)
    out = torch.full_like(y, 5.0)
    got = B.moe_lora_add(y, x, a, b, ids, scale, out=out)
    want, bound = P.lora(x, y, a, b, ids, scale)
    assert got is out
    _within(got, want, bound)
    assert torch.equal(got[ids < 0], y[ids < 0])
    y2 = y.clone()
    assert B.moe_lora_add(y2, x, a, b, ids, scale) is y2 and torch.equal(y2, got)
    assert B.mxfp4_device_status() == 0


@pytest.mark.parametrize("m,k,d,r,n", [(129, 520, 136, 64, 5), (200, 4104, 264, 24, 60), (260, 1032, 1096, 128, 3), (384, 264, 2056, 16, 64),
                                       (97, 7176, 72, 72, 128), (515, 2048, 200, 128, 130)])
def test_lora_tokens_do_not_depend_on_the_others_adapters(B, m, k, d, r, n):
    """Few tokens of many adapters, which several blocks share: each token's result is, bit for bit, what it is
    where the others use none; in place, into strided rows, and beside adapters that hold NaN."""
    x, y, a, b, scale = _lora_case(m, k, d, r, n)
    ids = _ints(m + n, -1, n, m)
    ids[m // 2] = -1
    ids[0] = ids[m - 1] = 1
    got = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    want, bound = P.lora(x, y, a, b, ids, scale)
    _within(got, want, bound)
    for i in {-1, 0, 1, n - 1, int(ids[m // 3]), int(ids[m - 2])}:
        mine = ids == i
        alone = B.moe_lora_add(y, x, a, b, torch.where(mine, ids, -1).to(torch.int32), scale, out=torch.empty_like(y))
        assert torch.equal(alone[mine], got[mine]) and torch.equal(alone[~mine], y[~mine]), i
    place = y.clone()
    assert torch.equal(B.moe_lora_add(place, x, a, b, ids, scale), got)
    rows, wide = _strided(torch.zeros_like(y), 16, 8)
    B.moe_lora_add(y, x, a, b, ids, scale, out=rows)
    assert torch.equal(rows, got) and (wide[:, :8] == 77).all() and (wide[:, 8 + d:] == 77).all()
    a[1], b[0] = NAN, INF
    sound = (ids != 1) & (ids != 0)
    spoilt = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    assert torch.equal(spoilt[sound], got[sound]) and torch.isnan(spoilt[ids == 1]).all()
    assert B.mxfp4_device_status() == 0


@pytest.mark.parametrize("m", [3, 64, 65, 300])
def test_lora_no_scale_no_adapters_no_tokens(B, m):
    x, y, a, b, _ = _lora_case(m, 264, 328, 16, 3)
    ids = _ints(3, 0, 3, m)
    got = B.moe_lora_add(y, x, a, b, ids, out=torch.empty_like(y))
    want, bound = P.lora(x, y, a, b, ids, None)
    _within(got, want, bound)
    none = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    y[0, 0], y[m - 1, 5] = -0.0, NAN  # bit for bit
    out = torch.empty_like(y)
    B.moe_lora_add(y, x, a, b, none, out=out)
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))
    kept = y.clone()
    B.moe_lora_add(y, x, a, b, none)
    assert torch.equal(kept.view(torch.int16), y.view(torch.int16))
    empty = B.moe_lora_add(y[:0], x[:0], a, b, none[:0])
    assert empty.shape == (0, 328)


@pytest.mark.parametrize("m", [40, 200])
def test_lora_strided_rows(B, m):
    x, y, a, b, scale = _lora_case(m, 136, 200, 24, 4)
    ids = _requests(3, m, 4, 6)
    want = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    ys, wide = _strided(y, 56, 24)
    B.moe_lora_add(ys, _strided(x)[0], a, b, ids, scale)
    assert torch.equal(ys, want) and (wide[:, :24] == 77).all() and (wide[:, 224:] == 77).all()
    os, wide = _strided(torch.zeros_like(y), 16, 8)
    B.moe_lora_add(y, x, a, b, ids, scale, out=os)
    assert torch.equal(os, want) and (wide[:, :8] == 77).all() and (wide[:, 208:] == 77).all()
    both = torch.cat((x, y), 1)  # side by side
    B.moe_lora_add(both[:, 136:], both[:, :136], a, b, ids, scale)
    assert torch.equal(both[:, 136:], want) and torch.equal(both[:, :136], x)


@pytest.mark.parametrize("m", [40, 200])
def test_lora_bad_ids(B, m):
    x, y, a, b, scale = _lora_case(m, 136, 200, 16, 4)
    ids = _requests(3, m, 4, 6)
    good = ids.clone()
    for t, v in ((1, 4), (7, -2), (m - 1, 2 ** 31 - 1), (9, -2 ** 31)):
        ids[t], good[t] = v, -1
    want = B.moe_lora_add(y, x, a, b, good, scale, out=torch.empty_like(y))
    assert B.mxfp4_device_status() == 0
    got = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    assert torch.equal(got, want) and B.mxfp4_device_status() == 1 and B.mxfp4_device_status() == 0


@pytest.mark.parametrize("m", [40, 300])
def test_lora_bad_rows_spoil_no_other(B, m):
    x, y, a, b, scale = _lora_case(m, 264, 200, 16, 4)
    ids = _requests(3, m, 4, 6).clamp_min(0)
    want = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    x[5, 3], x[20, 200] = INF, NAN
    ids[33] = 3
    ids[34:] = ids[34:].clamp_max(2)
    a[3, 2, 7] = NAN
    ids[:33] = ids[:33].clamp_max(2)
    want = B.moe_lora_add(y, torch.nan_to_num(x, 0, 0, 0), torch.nan_to_num(a), b, ids, scale, out=torch.empty_like(y))
    got = B.moe_lora_add(y, x, a, b, ids, scale, out=torch.empty_like(y))
    rows = [i for i in range(m) if i not in (5, 20, 33)]
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[[20, 33]]).all() and not torch.isfinite(got[5]).any()


def test_lora_large_sums(B):
    """A x past what one bf16 part holds: the second part brings it to 16 bits (a bound of 2^-16 of
    each term, where one part would leave 2^-9)."""
    for m in (8, 200):
        x = torch.full((m, 64), 1.0, dtype=torch.bfloat16, device="cuda")
        a = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
        a[0, 0, 0], a[0, 0, 1] = 256.0, 1.0
        b = torch.ones(1, 8, 8, dtype=torch.bfloat16, device="cuda")
        y = torch.full((m, 8), -256.0, dtype=torch.bfloat16, device="cuda")
        ids = torch.zeros(m, dtype=torch.int32, device="cuda")
        assert (B.moe_lora_add(y, x, a, b, ids) == 1.0).all()


# ---------------------------------------------------------------- with what was there

@pytest.mark.parametrize("m", [1, 5, 64, 65, 300])
def test_linear_with_adapters(B, m):
    """moe_mxfp4_linear's adapters are moe_lora_add of its output, also in place of a buffer and on fewer
    tokens than the quantiser is fused for."""
    k, n = 544, 712
    w = B.moe_mxfp4_quant(_n(1, n, k, std=k ** -0.5))
    x, _, a, b, scale = _lora_case(m, k, n, 16, 4)
    ids = _requests(3, m, 4, 6)
    want = B.moe_lora_add(B.moe_mxfp4_linear(x, *w), x, a, b, ids, scale)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(B.moe_mxfp4_linear(x, *w, adapters=(a, b, scale), adapter_ids=ids), want)
    assert B.moe_mxfp4_linear(x, *w, out=out, adapters=(a, b, scale), adapter_ids=ids) is out and torch.equal(out, want)


def test_refusals(B):
    """What a call refuses, it refuses before anything is launched: the buffers stay as they are."""
    m, h = 10, 64
    x, res, w = _n(1, m, h), _n(2, m, h), _n(3, h, dtype=torch.float32)
    logits, ids = _router_case(m, 8, 2)
    a, b, one = _n(4, 3, 8, h), _n(5, 3, h, 8), torch.ones(1, device="cuda")
    which = torch.zeros(m, dtype=torch.int32, device="cuda")
    pair = B.moe_mxfp4_quant(_n(6, h, h))
    wide = torch.zeros(m, 2 * h, dtype=torch.bfloat16, device="cuda")
    kept = x.clone()
    value = [
        lambda: B.moe_add_rmsnorm(x.float(), w), lambda: B.moe_add_rmsnorm(x.T, w), lambda: B.moe_add_rmsnorm(x[0], w),
        lambda: B.moe_add_rmsnorm(x[:, 1:57], w[:56]), lambda: B.moe_add_rmsnorm(x, w.bfloat16()), lambda: B.moe_add_rmsnorm(x, w[:32]),
        lambda: B.moe_add_rmsnorm(x, w, residual=res[:5]), lambda: B.moe_add_rmsnorm(x, w, residual_out=res),
        lambda: B.moe_add_rmsnorm(x, w, bf16=False), lambda: B.moe_add_rmsnorm(x, w, out=wide[:, :h]),
        lambda: B.moe_add_rmsnorm(x, w, residual=res.cpu()), lambda: B.moe_add_rmsnorm(x, w, bf16=False, fp8=True, out=res),
        lambda: B.moe_add_rmsnorm_backward(x, res[:5], w), lambda: B.moe_add_rmsnorm_backward(x.float(), res, w),
        lambda: B.moe_add_rmsnorm_backward(x, res, w, dresidual=x[:, :32]),
        lambda: B.moe_balance_loss(logits.double(), ids), lambda: B.moe_balance_loss(logits, ids.long()),
        lambda: B.moe_balance_loss(logits, ids[:5]), lambda: B.moe_balance_loss(logits, ids, which[:1]),
        lambda: B.moe_balance_loss(logits, ids, which[:4].long()), lambda: B.moe_balance_loss(logits, ids, scoring="relu"),
        lambda: B.moe_route_backward(logits, ids, dbalance=one), lambda: B.moe_route_backward(logits, ids, dz=one[:0]),
        lambda: B.moe_route_backward(logits, ids, torch.ones(m, 3, device="cuda")),
        lambda: B.moe_lora_add(res, x, a, b, which.long()), lambda: B.moe_lora_add(res, x, a, b, which[:5]),
        lambda: B.moe_lora_add(res, x, a, b[:, :, :4], which), lambda: B.moe_lora_add(res, x, a.float(), b, which),
        lambda: B.moe_lora_add(res, x[:5], a, b, which), lambda: B.moe_lora_add(res, x, a, b, which, one),
        lambda: B.moe_mxfp4_linear(x, *pair, adapters=(a, b, None)), lambda: B.moe_mxfp4_linear(x, *pair, adapter_ids=which),
        lambda: B.moe_mxfp4_linear(x, *pair, out=x, adapters=(a, b, None), adapter_ids=which),
        lambda: B.moe_mxfp4_linear(x.float(), *pair, adapters=(a, b, None), adapter_ids=which),
    ]
    library = [
        (lambda: B.moe_add_rmsnorm(x, w, eps=-1.0), 1), (lambda: B.moe_add_rmsnorm(x, w, residual=res, out=res), 1),
        (lambda: B.moe_add_rmsnorm(x, w, residual=res, residual_out=x), 1),
        (lambda: B.moe_add_rmsnorm(torch.zeros(1, 24584, dtype=torch.bfloat16, device="cuda"), torch.ones(24584, device="cuda")), 2),
        (lambda: B.moe_route_backward(logits, ids, scoring="sigmoid", routed_scaling=0.0), 1),
        (lambda: B.moe_balance_loss(torch.zeros(m, 1032, device="cuda"), ids), 2),
        (lambda: B.moe_lora_add(x, x, a, b, which), 1), (lambda: B.moe_lora_add(res, x, a, b, which, out=x), 1),
        (lambda: B.moe_lora_add(res, x, _n(4, 3, 136, h), _n(5, 3, h, 136), which), 2),
        (lambda: B.moe_lora_add(res, x, _n(4, 3, 12, h), _n(5, 3, h, 12), which), 1),
    ]
    for call in value:
        with pytest.raises(ValueError):
            call()
    for call, status in library:
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.status == status
    assert torch.equal(x, kept)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("m", [1, 7, 200])
def test_experts_from_eight_bits(B, m, gate):
    """The experts of an fp8 layer from codes are, bit for bit, the experts of the x they were made of;
    and a layer behind the norm runs from the norm's codes."""
    import dataclasses
    from mixture_experts_ffn_gemv_gb300 import inputs as I
    shape = I.LayerShape(hidden=512, num_experts=8, top_k=2, inter=512, shared_inter=512, fp8=True)
    if gate:
        shape = dataclasses.replace(shape, shared_gate=True)
    wl = dataclasses.replace(I.WORKLOADS["tiny"], shape=shape)
    t = I.make_layer(wl, seed=0, device=torch.device("cuda", 0))
    layer = B.MoeLayer(shape, t)
    x, res, w = _n(1, m, 512), _n(2, m, 512), 1 + _n(3, 512, std=0.1, dtype=torch.float32)
    ids, tw = layer.moe_route(x, t["router_w"])
    for arm in ("gemv", "gemm"):
        want = layer.moe_experts(x, ids, tw, arm=arm)
        got = layer.moe_experts_fp8(*B.moe_act_quant_fp8(x), ids, tw, x=x if gate else None, arm=arm)
        assert torch.equal(got, want)
    n = B.moe_add_rmsnorm(x, w, residual=res, fp8=True)
    ids, tw = layer.moe_route(n.out, t["router_w"])
    a = layer.moe_experts_fp8(n.codes, n.scales, ids, tw, x=n.out).double()
    b = layer.moe_experts(n.out, ids, tw).double()
    # the two differ by x's rounding to bf16 ahead of its rounding to e4m3: at most one step of e4m3
    # in a code, 2^-3 of it, where it changes the code at all
    assert (a - b).norm() <= 2.0 ** -3 * b.norm() and layer.device_status() == 0


@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_router_step_behind_the_norm(B, sigmoid):
    """As a training step runs them: the norm, the layer's router and losses, the gradient of its logits,
    of its weight and of its input, and through the norm, against 64 bits over all of it.
    Roundings that the reference does not take: dlogits and the two products in fp32 (2^-18 of the sums of
    magnitudes, far below the rest), the router's input gradient to bf16 ahead of the norm's backward pass
    and that pass's result: 2^-9 of a value each on average at most, twice its own size through the norm
    (it takes away the part along n) -- 2^-7 of the whole, in the 2-norm."""
    from mixture_experts_ffn_gemv_gb300 import inputs as I
    m, H, E, k = 200, 256, 16, 4
    shape = I.LayerShape(hidden=H, num_experts=E, top_k=k, inter=128, scoring="sigmoid" if sigmoid else "softmax",
                         routed_scaling=2.5 if sigmoid else 1.0)
    ws = {n: _n(i, E, 128, H, std=0.05) for i, n in enumerate(("w1", "w3"))}
    ws["w2"] = _n(3, E, H, 128, std=0.05)
    layer = B.MoeLayer(shape, ws)
    x, res, w, rw = _n(1, m, H), _n(2, m, H, std=2.0), 1 + _n(3, H, std=0.2, dtype=torch.float32), _n(4, E, H, std=0.1, dtype=torch.float32)
    off = torch.tensor([0, 90, 190], dtype=torch.int32, device="cuda")
    dw, db, dz = _n(5, m, k, dtype=torch.float32), torch.full((2,), 3.0, device="cuda"), torch.full((2,), 0.5, device="cuda")
    n = B.moe_add_rmsnorm(x, w, residual=res)
    ids, tw, logits = layer.moe_route(n.out, rw, logits=True)
    assert torch.isfinite(layer.moe_experts(n.out, ids, tw)).all()
    bal, z, counts = layer.moe_balance_loss(logits, ids, off)
    d = layer.moe_route_backward(logits, ids, dw, db, dz, counts, off)
    drw = d.T @ n.out.float()
    dx, dweight = B.moe_add_rmsnorm_backward((d @ rw).to(torch.bfloat16), n.residual, w)

    r64, w64, rw64 = (t.double().requires_grad_() for t in (n.residual, w, rw))
    out = r64 / torch.sqrt(r64.square().mean(1, keepdim=True) + 1e-6) * w64
    out = out + (n.out.double() - out).detach()  # as the router saw it
    l = out @ rw64.T
    b2, z2, c2 = P.router(l, ids, off, sigmoid)
    total = (b2 * db.double()).sum() + (z2 * dz.double()).sum()
    total = total + (P.route_weights(l, ids, sigmoid, True, 2.5 if sigmoid else 1.0) * dw.double()).sum()
    want = torch.autograd.grad(total, (rw64, r64, w64))
    assert torch.equal(counts, c2)
    for got, ref, bound in zip((drw, dx, dweight), want, (2.0 ** -14, 2.0 ** -7, 2.0 ** -7)):
        assert (got.double() - ref).norm() <= bound * ref.norm()


def test_experts_from_eight_bits_refusals(B):
    import dataclasses
    from mixture_experts_ffn_gemv_gb300 import inputs as I
    shape = I.LayerShape(hidden=512, num_experts=4, top_k=2, inter=512, shared_inter=512, fp8=True, shared_gate=True)
    layer = B.MoeLayer(shape, I.make_layer(dataclasses.replace(I.WORKLOADS["tiny"], shape=shape), seed=0, device=torch.device("cuda", 0)))
    x = _n(1, 6, 512)
    codes, scales = B.moe_act_quant_fp8(x)
    ids, w = torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.ones(6, 2, device="cuda")
    assert layer.moe_experts_fp8(codes[:0], scales[:0], ids[:0], w[:0], x=x[:0]).shape == (0, 512)
    for bad in ((codes[:5], scales, ids, w, x), (codes, scales[:, :2], ids, w, x), (codes, scales, ids.long(), w, x),
                (codes, scales, ids, w[:, :1], x), (codes, scales, ids, w, x.float()), (x, scales, ids, w, x), (codes.cpu(), scales, ids, w, x)):
        with pytest.raises(ValueError):
            layer.moe_experts_fp8(*bad[:4], x=bad[4])
    with pytest.raises(B.MoeError) as e:  # its shared expert has a gate
        layer.moe_experts_fp8(codes, scales, ids, w)
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    plain = I.LayerShape(hidden=512, num_experts=4, top_k=2, inter=512)
    t = {k: torch.zeros(4, 512, 512, dtype=torch.bfloat16, device="cuda") for k in ("w1", "w3", "w2")}
    with pytest.raises(B.MoeError) as e:
        B.MoeLayer(plain, t).moe_experts_fp8(codes, scales, ids, w)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED


# ---------------------------------------------------------------- calls together

def _all(B, t):
    n = B.moe_add_rmsnorm(t["x"], t["w"], residual=t["res"], fp8=True)
    dx, dw = B.moe_add_rmsnorm_backward(t["dout"], n.residual, t["w"], dresidual=t["x"])
    bal, z, counts = B.moe_balance_loss(t["logits"], t["ids"], t["off"])
    d = B.moe_route_backward(t["logits"], t["ids"], t["dw"], t["one"], t["one"], counts, t["off"])
    y = B.moe_lora_add(t["x"], n.out, t["a"], t["b"], t["which"], out=torch.empty_like(t["x"]))
    few = B.moe_lora_add(t["x"][:9], n.out[:9], t["a"], t["b"], t["which"][:9], out=torch.empty_like(t["x"][:9]))
    return (*n, dx, dw, bal, z, counts, d, y, few)


def _state(seed, m=200, h=520):
    logits, ids = _router_case(m, 48, 4, seed)
    return {"x": _n(seed, m, h), "res": _n(seed + 1, m, h), "w": _n(seed + 2, h, dtype=torch.float32), "dout": _n(seed + 3, m, h),
            "logits": logits, "ids": ids, "off": torch.tensor([0, 30, 30, 180], dtype=torch.int32, device="cuda"),
            "dw": _n(seed + 4, m, 4, dtype=torch.float32), "one": torch.ones(3, device="cuda"),
            "a": _n(seed + 5, 5, 16, h, std=h ** -0.5), "b": _n(seed + 6, 5, h, 16, std=0.25),
            "which": _requests(seed, m, 5, 7)}


def _equal(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def test_repeatable(B):
    t = _state(1, 3000)
    want = _all(B, t)
    for _ in range(5):
        assert _equal(_all(B, t), want)


def test_graphs_and_other_streams(B):
    """Captured, replayed on new inputs in place, two graphs in turn, beside eager calls and after
    larger ones; on another stream than the tensors' own, and on a stream given to the call."""
    t, u = _state(1), _state(2, 333)
    st = torch.cuda.Stream()
    graphs = []
    _all(B, t), _all(B, u)
    torch.cuda.synchronize()
    for s in (t, u):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _all(B, s)
        graphs.append((g, s, out))
    _all(B, _state(3, 4000))
    others = [torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for seed in (11, 12):
        for g, s, out in graphs:
            for name, v in _state(seed, s["x"].shape[0]).items():
                s[name].copy_(v)
        for g, s, out in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for g, s, out in graphs:
            assert _equal(out, _all(B, s))
        assert all((o == 0x5A).all() for o in others)
    want = _all(B, t)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = _all(B, t)
    torch.cuda.synchronize()
    assert _equal(got, want)
    n = B.moe_add_rmsnorm(t["x"], t["w"], residual=t["res"], fp8=True, stream=st)
    dx = B.moe_add_rmsnorm_backward(t["dout"], want[1], t["w"], dresidual=t["x"], stream=st)
    bal = B.moe_balance_loss(t["logits"], t["ids"], t["off"], stream=st)
    d = B.moe_route_backward(t["logits"], t["ids"], t["dw"], t["one"], t["one"], want[8], t["off"], stream=st)
    y = B.moe_lora_add(t["x"], want[0], t["a"], t["b"], t["which"], out=torch.empty_like(t["x"]), stream=st)
    st.synchronize()
    assert _equal((*n, *dx, *bal, d, y), want[:-1])
    assert B.mxfp4_device_status() == 0 and B.mxfp4_device_status(st) == 0


def test_two_streams_at_once(B):
    """Calls of all operators on two streams, and products on tensor memory beside them: what runs at the
    same time shares neither workspaces nor tensor memory."""
    states = [_state(31, 300), _state(32, 1000)]
    w = [B.moe_mxfp4_quant(_n(40 + i, 520, 544, std=0.05)) for i in range(2)]
    xs = [_n(50 + i, 400, 544) for i in range(2)]
    want = [(*_all(B, t), B.moe_mxfp4_linear(x, *q)) for t, x, q in zip(states, xs, w)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((*_all(B, states[i]), B.moe_mxfp4_linear(xs[i], *w[i])))
    torch.cuda.synchronize()
    assert all(_equal(g, want[i]) for i in range(2) for g in got[i])
    assert all(B.mxfp4_device_status(st) == 0 for st in streams)


def test_threads_on_one_stream(B):
    import threading
    states = [_state(20 + i, 150 + 10 * i) for i in range(4)]
    want = [_all(B, s) for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(30):
            if not _equal(_all(B, states[i]), want[i]):
                bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not bad


def test_offsets_past_32_bits(B):
    """Tensors of more than 2^32 bytes and 2^31 elements: the last rows are right."""
    m, h = 300000, 8192
    x = torch.empty(m, h, dtype=torch.bfloat16, device="cuda")
    x[-3:], x[:3] = _n(1, 3, h), _n(2, 3, h)
    w = torch.ones(h, device="cuda")
    n = B.moe_add_rmsnorm(x, w, fp8=True)
    _check_norm(B, B.NormOut(n.out[-3:], None, n.codes[-3:], n.scales[-3:]), x[-3:], None, w, 1e-6, True)
    dx, _ = B.moe_add_rmsnorm_backward(n.out, x, w, need_dw=False)
    want, _, bound, _ = P.norm_backward(n.out[-3:], x[-3:], w, 1e-6, None)
    _within(dx[-3:], want, bound)
    del dx
    a, b = _n(3, 2, 8, h, std=h ** -0.5), _n(4, 2, h, 8)
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    ids[-200:] = 1
    want, bound = P.lora(n.out[-3:], x[-3:], a, b, ids[-3:], None)
    got = B.moe_lora_add(x, n.out, a, b, ids)
    _within(got[-3:], want, bound)


@pytest.mark.parametrize("m", [5, 200])
def test_adapters_past_32_bits(B, m):
    """Adapters that lie past 4 GB and rows of 2^20 columns: the last adapter, first and last columns."""
    n, r, d = 40, 64, 1 << 20
    b = torch.zeros(n, d, r, dtype=torch.bfloat16, device="cuda")
    b[-1] = _n(1, d, r, std=0.1)
    x, y, a = _n(2, m, 72), _n(3, m, d), _n(4, n, r, 72, std=0.1)
    ids = torch.full((m,), n - 1, dtype=torch.int32, device="cuda")
    ids[1] = 0
    out = B.moe_lora_add(y, x, a, b, ids, out=torch.empty_like(y))
    for cut in (slice(0, 1000), slice(d // 2, d // 2 + 1000), slice(d - 1000, d)):
        want, bound = P.lora(x, y[:, cut], a, b[:, cut], ids, None)
        _within(out[:, cut], want, bound)
    assert torch.equal(out[1], y[1])


def test_router_offsets_past_32_bits(B):
    m, E = 2200000, 1024
    logits = torch.zeros(m, E, device="cuda")
    ids = torch.zeros(m, 2, dtype=torch.int32, device="cuda")
    ids[:, 1] = 1023
    logits[-1, 5] = 3.0
    off = torch.tensor([0, m - 1, m], dtype=torch.int32, device="cuda")
    bal, z, counts = B.moe_balance_loss(logits, ids, off)
    assert counts[0, 0] == m - 1 and counts[0, 1023] == m - 1 and counts[1].sum() == 2
    wb, wz, _ = P.router(logits[-1:].double(), ids[-1:], None, False)
    bb, bz = P.router_bounds(logits[-1:].double(), wb, wz, None)
    _within(bal[1:], wb, bb)
    _within(z[1:], wz, bz)
    _within(bal[:1], torch.ones(1, device="cuda").double(), torch.full((1,), 2 * P.SMALL, device="cuda").double())
    one = torch.ones(2, device="cuda")
    d = B.moe_route_backward(logits, ids, None, one, one, counts, off)
    want, bound = P.route_backward(logits[-1:], ids[-1:], None, False, True, 1.0, None, one[:1], one[:1])
    _within(d[-1:], want, bound)
