"""How the products and adapters without a handle report what went wrong: the error words of captured
calls, refusals ahead of the first launch, and waits that run out."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def _n(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _adapters(m, k=136, d=200, r=16, n=4):
    """(y, x, a, b, ids): tokens of all adapters in turn, every fifth of none."""
    ids = torch.arange(m, dtype=torch.int32, device="cuda") % 5 - 1
    return _n(1, m, d), _n(2, m, k), _n(3, n, r, k, std=k ** -0.5), _n(4, n, d, r, std=r ** -0.5), ids


@pytest.mark.parametrize("m", [40, 300])
def test_errors_of_captured_calls_are_read(B, m):
    """An id that names no adapter, in a replayed graph: the word is there on whichever stream it is asked
    for, once, again after another replay, and not lost to a graph that is replayed in between without one."""
    y, x, a, b, ids = _adapters(m)
    good = ids.clone()
    out, sound = torch.empty_like(y), torch.empty_like(y)
    want = B.moe_lora_add(y, x, a, b, good, out=torch.empty_like(y))
    torch.cuda.synchronize()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_lora_add(y, x, a, b, ids, out=out)
        later = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")  # the pool may place it where the workspace was
    with torch.cuda.graph(h):
        B.moe_lora_add(y, x, a, b, good, out=sound)
    g.replay()
    assert B.mxfp4_device_status() == 0 and torch.equal(out, want)
    ids[3] = 4
    g.replay()
    h.replay()
    assert B.mxfp4_device_status() == 1 and B.mxfp4_device_status() == 0
    assert torch.equal(sound, want) and torch.equal(out[3], y[3]) and not later.any()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g.replay()
    assert B.mxfp4_device_status(st) == 1 and B.mxfp4_device_status() == 0
    g.replay()
    ids.copy_(good)
    g.replay()  # without an error: the word of the replay before stays
    assert B.mxfp4_device_status() == 1 and B.mxfp4_device_status() == 0 and torch.equal(out, want)


def test_eager_errors_stay_their_streams_own(B):
    """Captured calls beside them change nothing: an eager call's error is read on its stream alone."""
    y, x, a, b, ids = _adapters(40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_lora_add(y, x, a, b, ids, out=torch.empty_like(y))
    g.replay()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.moe_lora_add(y, x, a, b, torch.full_like(ids, 9), out=torch.empty_like(y))
    assert B.mxfp4_device_status() == 0 and B.mxfp4_device_status(st) == 1 and B.mxfp4_device_status(st) == 0


def test_captured_headers(B):
    """moe_captured_header leaves zeros but for where errors go, whatever was there, and nothing around it."""
    lib, code = B.load_library(), ctypes.c_int32()
    ws = torch.full((768,), 0x5A, dtype=torch.uint8, device="cuda")
    assert lib.moe_captured_header(ws.data_ptr() + 256, B._stream()) == 0
    torch.cuda.synchronize()
    words = ws[256:512].view(torch.int64)
    where = words.nonzero()[:, 0].tolist()  # an address and its complement
    assert len(where) == 2 and int(words[where[0]]) == ~int(words[where[1]]) and (ws[:256] == 0x5A).all() and (ws[512:] == 0x5A).all()
    assert lib.moe_captured_status(None, ctypes.byref(code)) == 0 and code.value == 0
    assert lib.moe_device_status(ws.data_ptr() + 256, None, ctypes.byref(code)) == 0 and code.value == 0


def test_linear_with_adapters_refuses_before_it_writes(B):
    """Whatever is refused of the adapters, out stays as it was, and so does y's memory where out is not given."""
    m, k, d = 70, 128, 104
    x, w, ids = _n(1, m, k), B.moe_mxfp4_quant(_n(2, d, k)), torch.zeros(m, dtype=torch.int32, device="cuda")

    def pair(r, n=2):
        return _n(3, n, r, k), _n(4, n, d, r), None
    a, b, _ = pair(16)
    askew = torch.zeros(a.numel() + 8, dtype=torch.bfloat16, device="cuda")
    cases = [(pair(12), ids, B.MoeError, 1), (pair(136), ids, B.MoeError, 2), (pair(16, 0), ids, B.MoeError, 1),
             ((askew[1:1 + a.numel()].view_as(a), b, None), ids, B.MoeError, 1),
             ((a, askew[4:4 + b.numel()].view_as(b), None), ids, B.MoeError, 1),
             ((a, b[:, :88], None), ids, ValueError, None), ((a, b, None), ids[:5], ValueError, None),
             ((a, b, torch.ones(3, device="cuda")), ids, ValueError, None), ((a[:, :, :64], b, None), ids, ValueError, None)]
    out = torch.full((m, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for adapters, which, error, status in cases:
        with pytest.raises(error) as e:
            B.moe_mxfp4_linear(x, *w, out=out, adapters=adapters, adapter_ids=which)
        assert status is None or e.value.status == status
        with pytest.raises(error):
            B.moe_mxfp4_linear(x, *w, adapters=adapters, adapter_ids=which)
    for bad in (x.float(), x[:, :64], x[0], _n(5, m, k + 4)[:, 4:]):
        with pytest.raises(ValueError):
            B.moe_mxfp4_linear(bad, *w, out=out, adapters=(a, b, None), adapter_ids=ids)
    torch.cuda.synchronize()
    assert (out == 7).all()
    none = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    assert B.moe_mxfp4_linear(x[:0], *w, out=none, adapters=(a, b, None), adapter_ids=ids[:0]) is none
    assert B.mxfp4_device_status() == 0


@pytest.fixture
def stall(B):
    """Sets the wait limit and what stalls; both are as they were afterwards."""
    lib = B.load_library()

    def set_to(kernel, ns=200_000):
        assert lib.moe_lora_set_wait_limit(ns if kernel else 0) == 0 and lib.moe_lora_stall_test(kernel) == 0
    yield set_to
    set_to(0)


# one adapter a tile; two; many, a box along r each; many, two boxes; many shared by several blocks, of one box and two
STALLS = [(300, 1016, 1032, 16, 1), (400, 264, 2056, 64, 2), (300, 520, 264, 24, 30), (500, 264, 520, 128, 6), (2600, 136, 264, 8, 5),
          (260, 520, 264, 16, 60), (140, 264, 136, 128, 20)]


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("m,k,d,r,n", STALLS)
def test_stalled_adapters_time_out_and_the_next_call_is_clean(B, stall, m, k, d, r, n, kernel):
    """A wait that runs out ends its kernel with the error word set, twice in a row; what lies around out is
    left alone; the call after it is right, also of a graph."""
    y, x, a, b, _ = _adapters(m, k, d, r, n)
    ids = torch.arange(m, dtype=torch.int32, device="cuda") % (n + 1) - 1
    want = B.moe_lora_add(y, x, a, b, ids, out=torch.empty_like(y))
    assert B.mxfp4_device_status() == 0
    wide = torch.full((m, d + 24), 77.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 8:8 + d]
    stall(kernel)
    for _ in range(2):
        B.moe_lora_add(y, x, a, b, ids, out=out)
        assert B.mxfp4_device_status() == 2
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_lora_add(y, x, a, b, ids, out=out)
    assert B.mxfp4_device_status() == 0
    g.replay()
    assert B.mxfp4_device_status() == 2
    stall(0)
    B.moe_lora_add(y, x, a, b, ids, out=out)
    assert B.mxfp4_device_status() == 0 and torch.equal(out, want)
    assert (wide[:, :8] == 77).all() and (wide[:, 8 + d:] == 77).all()


@pytest.mark.parametrize("m,n", [(300, 2), (260, 60), (2600, 5)])
def test_the_second_kernels_limit_starts_when_the_first_is_done(B, stall, m, n):
    """Stalled until its limit, the first kernel leaves no time of the second's waits, if those started with
    it: the second still completes, which rows without an adapter show, whose output needs no sums."""
    y, x, a, b, _ = _adapters(m, 264, 1032, 16, n)
    ids = torch.arange(m, dtype=torch.int32, device="cuda") % (n + 1) - 1
    B.moe_lora_add(y, x, a, b, ids, out=torch.empty_like(y))
    out = torch.full_like(y, 77.0)
    stall(1, 2_000_000)
    B.moe_lora_add(y, x, a, b, ids, out=out)
    assert B.mxfp4_device_status() == 2 and torch.equal(out[ids < 0], y[ids < 0])


def _owner(t):
    """The stream whose memory holds t."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_outputs_belong_to_the_stream_that_writes_them(B):
    """The layer's calls and the quantisers, given a stream: every tensor they return is of its memory, so
    that they write into none which the current stream has let go and still reads."""
    import dataclasses
    from mixture_experts_ffn_gemv_gb300 import inputs as I
    shape = I.LayerShape(hidden=512, num_experts=8, top_k=2, inter=512, fp8=True)
    t = I.make_layer(dataclasses.replace(I.WORKLOADS["tiny"], shape=shape), seed=0, device=torch.device("cuda", 0))
    layer = B.MoeLayer(shape, t)
    m = 70
    x, res, w = _n(1, m, 512), _n(2, m, 512), torch.ones(512, device="cuda")
    ids, tw = layer.moe_route(x, t["router_w"])
    codes, scales = B.moe_act_quant_fp8(x)
    calls = [lambda st: B.moe_act_quant_fp8(x, stream=st), lambda st: B.moe_act_quant_nvfp4(x, stream=st),
             lambda st: layer.moe_route(x, t["router_w"], logits=True, stream=st), lambda st: layer.moe_permute(ids, stream=st),
             lambda st: layer.moe_experts(x, ids, tw, stream=st), lambda st: layer.moe_experts_fp8(codes, scales, ids, tw, stream=st),
             lambda st: layer.moe_forward(x, t["router_w"], return_routing=True, stream=st),
             lambda st: layer.moe_forward_residual_rmsnorm(x, t["router_w"], res.clone(), w, return_routing=True, stream=st)]
    st = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        got = call(st)
        torch.cuda.synchronize()
        want, got = ((v,) if isinstance(v, torch.Tensor) else v for v in (want, got))
        for a, b in zip(want, got):
            assert torch.equal(a, b) and _owner(b) == st.cuda_stream != _owner(a)
    layer.prepare_router(t["router_w"], stream=st)
    assert _owner(layer._planes) == st.cuda_stream


def test_a_header_that_was_never_zeroed_is_no_address(B):
    """Errors go where a header says only if moe_captured_header wrote it: one full of anything takes them itself."""
    lib, code = B.load_library(), ctypes.c_int32()
    y, x, a, b, ids = _adapters(40)
    ids[3] = 4
    ws = torch.full((256,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    assert lib.moe_lora_add(x.data_ptr(), 136, 40, 136, y.data_ptr(), 200, 200, a.data_ptr(), b.data_ptr(), 4, 16, ids.data_ptr(),
                            None, y.data_ptr(), 200, ws.data_ptr(), 256, None) == 0
    assert lib.moe_device_status(ws.data_ptr(), None, ctypes.byref(code)) == 5 and code.value == 1


@pytest.mark.parametrize("h", [264, 2056])
def test_norm_past_the_range_of_its_sums(B, h):
    """Squares past fp32's range make zeros; below it a row counts as one of zeros, infinite with an eps of 0
    and, with an ordinary one, r / sqrt(eps) as the formula has it: two roundings of fp32 and bf16's half step."""
    w = 1 + _n(1, h, std=0.1).float()
    sign = torch.where(_n(2, 3, h) > 0, 1.0, -1.0)
    x = (sign * 1e20).bfloat16()
    assert not B.moe_add_rmsnorm(x, w).out.any()
    x = (sign * 1e-24).bfloat16()
    assert torch.isinf(B.moe_add_rmsnorm(x, w, 0.0).out).all()
    want = x.double() / 1e-6 ** 0.5 * w.double()
    assert ((B.moe_add_rmsnorm(x, w).out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18)).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [5, 64])
def test_router_losses_of_bad_logits(B, E, sigmoid):
    """A NaN makes its sequence's losses NaN, a +inf its z and, of softmax, its balance; other sequences are,
    bit for bit, as without them."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(30, E, device="cuda", generator=g)
    ids = torch.arange(60, dtype=torch.int32, device="cuda").view(30, 2) % E
    off = torch.tensor([0, 7, 15, 30], dtype=torch.int32, device="cuda")
    scoring = "sigmoid" if sigmoid else "softmax"
    good = B.moe_balance_loss(logits, ids, off, scoring)
    logits[3, 1], logits[9, 4] = float("nan"), float("inf")
    balance, z, counts = B.moe_balance_loss(logits, ids, off, scoring)
    assert torch.isnan(balance).tolist() == [True, not sigmoid, False] and torch.isnan(z).tolist() == [True, True, False]
    assert torch.isfinite(balance[1]) == sigmoid
    assert balance[2] == good[0][2] and z[2] == good[1][2] and torch.equal(counts, good[2])
