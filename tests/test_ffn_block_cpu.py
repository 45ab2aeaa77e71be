"""The gated feed-forward block and MXFP4 entry points without a GPU: refusals, sizes, the scale
order, and the formulas the GPU tests compare against."""
import ctypes
import threading
import time
import types
import weakref

import pytest
import torch

import _ffn_plain as P

FAKE = 0x10000  # never dereferenced: the calls fail before any device access


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def _create(B, ptrs=None, **kw):
    c = dict(hidden=256, inter=128, activation=0, weights=0)
    c.update(kw)
    cfg = B.MoeFfnConfig(*(c[k] for k in ("hidden", "inter", "activation", "weights")))
    if ptrs is None:
        ptrs = [FAKE] * (6 if c["weights"] == 3 else 3)
    w = B.MoeFfnWeights(*ptrs)
    out = ctypes.c_void_p()
    rc = B.load_library().moe_ffn_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(out))
    assert not out.value
    return rc


@pytest.mark.parametrize("kw,want", [
    (dict(hidden=0), 1), (dict(inter=-8), 1),
    (dict(hidden=100), 2), (dict(inter=12), 2),                      # bf16: multiples of 8
    (dict(weights=3, hidden=40), 2), (dict(weights=3, inter=48), 2),  # MXFP4: multiples of 32
    (dict(hidden=(1 << 20) + 8), 2),
    (dict(activation=2), 1), (dict(activation=-1), 1),
    (dict(weights=1), 1), (dict(weights=2), 1), (dict(weights=4), 1),
    (dict(ptrs=[FAKE, None, FAKE]), 1), (dict(ptrs=[FAKE, FAKE + 8, FAKE]), 1),
    (dict(ptrs=[FAKE] * 6), 1),                                      # scales with bf16 weights
    (dict(weights=3, ptrs=[FAKE] * 5), 1), (dict(weights=3, ptrs=[FAKE] * 5 + [FAKE + 4]), 1),
])
def test_create_refuses(B, kw, want):
    assert _create(B, **kw) == want


def test_null_arguments(B):
    lib = B.load_library()
    assert lib.moe_ffn_create(None, None, None) == 1
    n = ctypes.c_size_t()
    assert lib.moe_ffn_workspace_size(None, 1, 0, ctypes.byref(n)) == 1
    assert lib.moe_ffn_saved_size(None, 1, ctypes.byref(n)) == 1
    assert lib.moe_ffn_forward(None, FAKE, 8, 1, FAKE, None, FAKE, 1 << 20, None) == 1
    assert lib.moe_ffn_backward(None, FAKE, 8, FAKE, 8, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, None) == 1
    assert lib.moe_ffn_last_launch_count(None) == -1
    assert lib.moe_ffn_set_wait_limit(None, 0) == 1 and lib.moe_ffn_stall_test(None, 1) == 1
    assert lib.moe_ffn_destroy(None) == 0


@pytest.mark.parametrize("weights", [0, 3])
def test_workspace_sizes_never_fall(B, weights):
    """What holds m tokens holds fewer.  The sizes are computed from the config alone, with which a
    handle begins; there is no handle without a device."""
    lib, n = B.load_library(), ctypes.c_size_t()
    handle = ctypes.create_string_buffer(1 << 14)
    cfg = B.MoeFfnConfig(2048, 768, 0, weights)
    ctypes.memmove(handle, ctypes.byref(cfg), ctypes.sizeof(cfg))
    for backward in (0, 1) if weights == 0 else (0,):
        last = 0
        for m in range(600):
            assert lib.moe_ffn_workspace_size(handle, m, backward, ctypes.byref(n)) == 0
            assert n.value >= last, (m, n.value, last)
            last = n.value


def test_mxfp4_refusals(B):
    lib = B.load_library()
    n = ctypes.c_size_t()
    for rows, cols, rc in ((4, 33, 1), (-1, 32, 1), (4, 0, 1), (1 << 30, 32, 2), (4, 1 << 30, 2)):
        assert lib.moe_mxfp4_scales_size(rows, cols, ctypes.byref(n)) == rc
    for rows, cols, want in ((1, 32, 512), (128, 128, 512), (129, 128, 1024), (128, 160, 1024), (300, 416, 3 * 4 * 512)):
        assert lib.moe_mxfp4_scales_size(rows, cols, ctypes.byref(n)) == 0 and n.value == want
    for fn in (lib.moe_mxfp4_quant, lib.moe_mxfp4_quant_f32):
        assert fn(FAKE, 64, 4, 40, FAKE, FAKE, None) == 1       # n % 32
        assert fn(FAKE, 32, 4, 64, FAKE, FAKE, None) == 1       # ldx < n
        assert fn(FAKE, 66, 4, 64, FAKE, FAKE, None) == 1       # rows not 16-byte aligned
        assert fn(FAKE + 2, 64, 4, 64, FAKE, FAKE, None) == 1
        assert fn(FAKE, 64, 4, 64, FAKE, None, None) == 1
        assert fn(FAKE, 64, 1 << 40, 64, FAKE, FAKE, None) == 2
        assert fn(None, 64, 0, 64, None, None, None) == 0       # nothing to do
    assert lib.moe_mxfp4_dequant(FAKE, FAKE, 4, 48, FAKE, None) == 1
    assert lib.moe_mxfp4_dequant(FAKE, FAKE, 4, 64, None, None) == 1
    assert lib.moe_mxfp4_dequant(None, None, 0, 64, None, None) == 0
    assert lib.moe_mxfp4_gemm_workspace_size(4, 12, 64, ctypes.byref(n)) == 1
    assert lib.moe_mxfp4_gemm_workspace_size(4, 16, 64, ctypes.byref(n)) == 0
    need = n.value

    def gemm(m=4, n=16, k=64, a=FAKE, ws=FAKE, size=need, out=FAKE):
        return lib.moe_mxfp4_gemm(a, FAKE, m, FAKE, FAKE, n, k, out, ws, size, None)
    assert gemm(n=12) == 1 and gemm(k=48) == 1 and gemm(m=-1) == 1 and gemm(m=0) == 0
    assert gemm(ws=None) == 1 and gemm(ws=FAKE + 16) == 1 and gemm(size=128) == 3
    assert lib.moe_mxfp4_linear_workspace_size(4, 16, 48, ctypes.byref(n)) == 1
    assert lib.moe_mxfp4_linear_workspace_size(1, 16, 1 << 21, ctypes.byref(n)) == 2
    assert lib.moe_mxfp4_linear_workspace_size(130, 16, 160, ctypes.byref(n)) == 0
    assert n.value == 256 + -(-130 * 80 // 256) * 256 + 4 * 512
    for fn in (lib.moe_mxfp4_linear, lib.moe_mxfp4_linear_f32):
        assert fn(FAKE, 64, 0, FAKE, FAKE, 16, 64, FAKE, None, 0, None) == 0
        assert fn(FAKE, 64, 4, FAKE, FAKE, 12, 64, FAKE, FAKE, 1 << 20, None) == 1
        assert fn(FAKE, 64, 4, FAKE, FAKE, 16, 64, FAKE, FAKE, 256, None) == 3
        assert fn(FAKE, 32, 4, FAKE, FAKE, 16, 64, FAKE, FAKE, 1 << 20, None) == 1
        assert fn(FAKE, 64, 4, None, FAKE, 16, 64, FAKE, FAKE, 1 << 20, None) == 1
    assert gemm(a=None) == 1 and gemm(a=FAKE + 8) == 1 and gemm(out=None) == 1 and gemm(m=1 << 30) == 2


def test_binding_refuses_host_tensors(B):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.moe_mxfp4_quant(x)
    with pytest.raises(ValueError):
        B.moe_mxfp4_dequant(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8))
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.GatedFfn(w, w, w)
    with pytest.raises(ValueError):
        B.GatedFfn(w, w, w, act="relu")


@pytest.mark.parametrize("rows,n", [(1, 32), (128, 128), (130, 160), (300, 1056)])
def test_packed_scale_order(B, rows, n):
    s = torch.randint(0, 256, (rows, n // 32), dtype=torch.uint8)
    p = B.mxfp4_pack_scales(s)
    assert tuple(p.shape) == B.mxfp4_scales_shape(rows, n)
    flat, nkt = p.reshape(-1), p.shape[1]
    for r in range(0, rows, 7):
        for b in range(n // 32):
            at = (r // 128 * nkt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
            assert flat[at] == s[r, b]
    assert torch.equal(B.mxfp4_unpack_scales(p, rows, n), s)
    pad = p.permute(0, 3, 2, 1, 4).reshape(-1, nkt * 4)[:, n // 32:]
    assert not pad.any()


def test_grid_is_its_own_rounding():
    v = torch.tensor(P.GRID + tuple(-x for x in P.GRID) + (4.0,) * 16).reshape(1, 32)
    assert torch.equal(P.mx_round(v), v.double())
    # ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4; above 6 -> 6
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.75] * 4).reshape(1, 32)
    assert P.mx_round(t)[0, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_formula_against_differences(kind):
    """The formulas against central differences of the forward pass, in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    x, w1, w3, w2, dout = (torch.randn(s, generator=gen, dtype=torch.float64)
                           for s in ((5, 8), (16, 8), (16, 8), (8, 16), (5, 8)))
    grads = P.backward(dout, x, w1, w3, w2, kind)
    leaves = [x, w1, w3, w2]
    for i, grad in enumerate(grads):
        v = torch.randn(leaves[i].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        hi, lo = ([t + s * e * v if j == i else t for j, t in enumerate(leaves)] for s in (1, -1))
        diff = ((P.forward(*hi, kind) - P.forward(*lo, kind)) * dout).sum() / (2 * e)
        # a central difference is off by e^2 f''' / 6 and by rounding 1e-16 / e
        assert abs(diff - (grad * v).sum()) <= 1e-7 * (1 + grad.abs().sum())
    # and the bounds on slope and curvature that the tolerances use
    g = torch.linspace(-12, 12, 200001, dtype=torch.float64)
    _, s = P.act_slope(g, kind)
    assert s.abs().max() < P.SLOPE and (s.diff() / g.diff()).abs().max() < P.CURVE


# ---------------------------------------------------------------- workspaces (host memory stands in for the device's)

def _handle(B, monkeypatch, cls):
    """A handle of cls without a device: 256 bytes of workspace a token; and a call on m tokens, from
    which the workspace comes back."""
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(B, "_record", lambda ws, stream: None)
    h = object.__new__(cls)
    h.handle = None
    h.workspace_size = lambda m, backward=False: 256 * m
    h._new_workspaces()

    def call(m):
        ws = h.workspace(m, device="cpu") if cls is B.MoeLayer else h.workspace(m, False, "cpu")
        if ws is not h._past.used:
            ws[:256] = 0  # as the library does in the first call on it
        h._past.called(ws)
        return ws
    return h, call


@pytest.mark.parametrize("cls", ["GatedFfn", "MoeLayer"])
def test_a_captured_workspace_outlives_its_successor(B, monkeypatch, cls):
    """A CUDA graph replays into the workspace that its capture saw, also after a larger call."""
    capturing = False
    monkeypatch.setattr(B, "_capturing", lambda: capturing)
    h, space = _handle(B, monkeypatch, getattr(B, cls))
    first = weakref.ref(space(4))
    space(8)
    assert first() is None  # no graph knows it
    capturing = True
    used = weakref.ref(space(6))
    assert used() is space(8)
    capturing = False
    assert space(100).numel() >= 25600 and used() is not None
    at = used().data_ptr()
    assert space(200).data_ptr() != at and used() is not None
    if cls == "GatedFfn":
        assert h._ws_at == (space(200).data_ptr(), space(200).numel())
    capturing = True  # one that grows during a capture is kept too
    used = weakref.ref(space(400))
    capturing = False
    space(800)
    assert used() is not None


def test_captured_products_share_no_workspace(B, monkeypatch):
    """The products' hidden workspaces: a capture neither takes the one that eager calls on its
    stream share nor leaves its own to them."""
    capturing = False
    monkeypatch.setattr(B, "_capturing", lambda: capturing)
    monkeypatch.setattr(B, "_spaces", {})
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(B, "_record", lambda ws, stream: None)
    like = types.SimpleNamespace(get_device=lambda: 0, device="cpu")
    eager = B._space(like, 7, 1000)
    assert B._space(like, 7, 1000) is eager
    capturing = True
    a, b = B._space(like, 7, 1000), B._space(like, 7, 1000)
    assert len({t.data_ptr() for t in (eager, a, b)}) == 3 and not a[:256].any() and not b[:256].any()
    capturing = False
    assert B._space(like, 7, 1000) is eager


def _host_status(ws, stream, code):
    """moe_device_status of a workspace in host memory."""
    word = ctypes.c_int32.from_address(ws.value)
    code._obj.value, word.value = word.value, 0
    return 5 if code._obj.value else 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("cls", ["GatedFfn", "MoeLayer"])
def test_error_words_outlive_their_workspace(B, monkeypatch, cls, captured):
    """A workspace is not read before a call has used it, and an error that nobody has read is still
    there after the workspace has grown."""
    capturing = False
    monkeypatch.setattr(B, "_capturing", lambda: capturing)
    monkeypatch.setattr(B, "load_library", lambda: types.SimpleNamespace(moe_device_status=_host_status))
    monkeypatch.setattr(B, "_stream", lambda stream=None: None)
    h, space = _handle(B, monkeypatch, getattr(B, cls))
    assert h.device_status() == 0
    unused = h.workspace(2, False, "cpu") if cls == "GatedFfn" else h.workspace(2, "cpu")
    unused.fill_(0x5A)
    assert h.device_status() == 0
    first = space(4)
    assert h.device_status() == 0
    capturing = captured
    assert space(4) is first
    capturing = False
    first[0] = 2
    space(100)
    assert h.device_status() == 2 and h.device_status() == 0
    first[0] = 3  # a graph may set its own again
    space(200)
    assert h.device_status() == (3 if captured else 0) and h.device_status() == 0
    space(300)[0] = 1
    capturing = captured  # grown during a capture
    assert space(400)[0] == 0
    capturing = False
    assert h.device_status() == 1 and h.device_status() == 0


def test_error_words_of_products_outlive_their_workspace(B, monkeypatch):
    monkeypatch.setattr(B, "_capturing", lambda: False)
    monkeypatch.setattr(B, "_spaces", {})
    monkeypatch.setattr(B, "load_library", lambda: types.SimpleNamespace(moe_device_status=_host_status))
    monkeypatch.setattr(B, "_stream", lambda stream=None: None)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(B, "_record", lambda ws, stream: None)
    like = types.SimpleNamespace(get_device=lambda: 0, device="cpu")
    stream = types.SimpleNamespace(device=types.SimpleNamespace(index=0), cuda_stream=7)
    assert B.mxfp4_device_status(stream) == 0
    B._space(like, 7, 1000)[0] = 2
    B._space(like, 7, 1 << 20)
    assert B.mxfp4_device_status(stream) == 2 and B.mxfp4_device_status(stream) == 0


def test_operands_lie_on_the_current_device(B, monkeypatch):
    """The library launches on the current device: operands elsewhere are refused before a launch."""
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 40 + dev)
    there, here = (types.SimpleNamespace(get_device=lambda d=d: d, device=f"cuda:{d}") for d in (0, 1))
    assert B._on(here) == 41 and B._on(here, here, here) == 41
    block = object.__new__(B.GatedFfn)
    block._dev = 1
    assert block._stream_for(here, here) == 41
    for bad in ((there,), (here, there), (there, here), (here, here, here, there)):
        with pytest.raises(ValueError, match="cuda:0 in a call on cuda:1"):
            B._on(*bad)
        with pytest.raises(ValueError, match="cuda:0 in a call of a block on cuda:1"):
            block._stream_for(*bad)


def test_products_of_two_threads_do_not_interleave(B, monkeypatch):
    """A product of many tokens is two launches with the stream's shared workspace between them, and
    the interpreter runs other threads while the library launches."""
    inside, together, seen = 0, [], set()

    def linear(x, ld, m, codes, scales, n, k, out, ws, size, stream):
        nonlocal inside
        inside += 1
        time.sleep(0.002)
        together.append(inside)
        seen.add(ws)
        inside -= 1
        return 0
    monkeypatch.setattr(B, "_capturing", lambda: False)
    monkeypatch.setattr(B, "_spaces", {})
    monkeypatch.setattr(B, "_lib", types.SimpleNamespace(moe_mxfp4_linear=linear, moe_mxfp4_linear_f32=linear))
    monkeypatch.setattr(B, "_mx_matrix", lambda *a: (64, 64))
    monkeypatch.setattr(B, "_rows", lambda *a, **k: 64)
    monkeypatch.setattr(B, "_on", lambda *t: 7)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(B, "_record", lambda ws, stream: None)
    x = torch.zeros(20, 64, dtype=torch.bfloat16)
    threads = [threading.Thread(target=lambda: [B.moe_mxfp4_linear(x, x, x) for _ in range(10)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(together) == 40 and max(together) == 1 and len(seen) == 1


@pytest.mark.parametrize("cls", ["GatedFfn", "MoeLayer"])
def test_a_workspace_is_kept_until_its_successor_is_used(B, monkeypatch, cls):
    """The library takes a header for clean by its workspace's address, that of the last call: no
    other workspace may get that address before the next call."""
    monkeypatch.setattr(B, "_capturing", lambda: False)
    h, call = _handle(B, monkeypatch, getattr(B, cls))
    last = weakref.ref(call(4))
    for m in (8, 16, 32):
        h.workspace(m, False, "cpu") if cls == "GatedFfn" else h.workspace(m, "cpu")
        assert last() is not None
    call(32)
    assert last() is None


def test_streams_of_a_workspace_are_recorded_once_each(B, monkeypatch):
    recorded = []
    monkeypatch.setattr(B, "_capturing", lambda: False)
    past = B._Workspaces()
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(B, "_record", lambda ws, stream: recorded.append((id(ws), stream and stream.cuda_stream)))
    a, b = torch.zeros(256), torch.zeros(256)
    side = types.SimpleNamespace(cuda_stream=9)
    for stream in (None, None, side, side, None):
        past.called(a, stream)
    assert recorded == [(id(a), None), (id(a), 9)]
    recorded.clear()
    past.called(b)  # the copy of a's header is a use of a
    past.called(b)
    assert recorded == [(id(a), None), (id(b), None)]


@pytest.mark.parametrize("cls", ["GatedFfn", "MoeLayer"])
def test_making_a_workspace_writes_nothing(B, monkeypatch, cls):
    """A write from the stream that made a workspace could come late, amid a call on another one."""
    monkeypatch.setattr(B, "_capturing", lambda: False)
    h, _ = _handle(B, monkeypatch, getattr(B, cls))
    monkeypatch.setattr(B.torch, "empty", lambda n, **kw: torch.full((n,), 0x5A, dtype=torch.uint8))
    ws = h.workspace(4, False, "cpu") if cls == "GatedFfn" else h.workspace(4, "cpu")
    assert (ws == 0x5A).all()
