"""The norm, the router's operators and the adapters without a GPU: refusals, sizes, and what counts as
shared memory."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # never dereferenced: the calls fail before any device access
SZ = ctypes.c_size_t


@pytest.fixture(scope="module")
def B():
    from mixture_experts_ffn_gemv_gb300 import binding
    binding.load_library()
    return binding


def _call(fn, defaults, kw):
    args = dict(defaults)
    args.update(kw)
    return fn(*args.values())


NORM = dict(x=FAKE, ldx=64, res=FAKE + 4096, ldr=64, m=3, h=64, w=FAKE, eps=1e-6, res_out=FAKE + 8192, ldo=64, out=FAKE + 12288,
            codes=None, scales=None, st=None)
CODES = dict(codes=FAKE + 16384, scales=FAKE + 20480)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), 1), (dict(h=0), 1), (dict(h=60), 1), (dict(h=24584, ldx=24584, ldr=24584, ldo=24584), 2), (dict(m=1 << 30), 2),
    (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(ldx=56), 1), (dict(ldx=68), 1), (dict(ldx=1 << 40), 1),
    (dict(w=None), 1), (dict(w=FAKE + 4), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(res_out=None), 1), (dict(res=None), 1), (dict(ldr=56), 1), (dict(ldo=60), 1), (dict(res_out=FAKE + 4096, ldo=72), 1),
    (dict(out=None), 1), (dict(out=FAKE + 12290), 1), (dict(out=FAKE, ldx=72), 1),
    (dict(codes=FAKE), 1), (dict(scales=FAKE), 1), (dict(codes=FAKE + 8, scales=FAKE), 1), (dict(codes=FAKE, scales=FAKE + 2), 1),
    (dict(out=FAKE + 16), 1), (dict(out=FAKE + 4096), 1), (dict(out=FAKE + 8192), 1), (dict(res_out=FAKE), 1),
    (dict(res_out=FAKE + 4096 + 128), 1), (dict(CODES, codes=FAKE + 128), 1), (dict(CODES, scales=FAKE + 4096 + 256), 1),
    (dict(CODES, scales=FAKE + 16384 + 188), 1), (dict(CODES, codes=FAKE + 12288 + 368), 1),
    (dict(m=0, x=None, w=None), 0),
])
def test_norm_refuses(B, kw, want):
    assert _call(B.load_library().moe_add_rmsnorm, NORM, kw) == want


GRAD = dict(dout=FAKE, ldd=64, r=FAKE + 4096, ldr=64, m=3, h=64, w=FAKE, eps=1e-6, dres=FAKE + 8192, ldq=64, dx=FAKE + 12288,
            dw=FAKE, ws=FAKE, size=1 << 20, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), 1), (dict(h=12), 1), (dict(h=32768), 2), (dict(dout=None), 1), (dict(r=FAKE + 8), 1), (dict(ldd=32), 1),
    (dict(ldr=65), 1), (dict(w=None), 1), (dict(eps=-0.5), 1), (dict(ldq=8), 1), (dict(dx=None), 1), (dict(dx=FAKE + 8), 1),
    (dict(dx=FAKE, ldd=72), 1), (dict(dx=FAKE + 8192, ldq=72), 1), (dict(dx=FAKE + 4096), 1), (dict(dw=FAKE + 2), 1),
    (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(size=255), 3), (dict(m=0, dout=None), 0),
])
def test_norm_backward_refuses(B, kw, want):
    lib = B.load_library()
    assert _call(lib.moe_add_rmsnorm_backward, GRAD, kw) == want
    assert lib.moe_add_rmsnorm_backward_workspace_size(3, 64, None) == 1


LOSS = dict(logits=FAKE, ids=FAKE, m=10, e=8, k=2, off=FAKE, seqs=3, scoring=0, balance=FAKE, z=FAKE, counts=FAKE, ws=FAKE,
            size=1 << 20, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), 1), (dict(e=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(seqs=0), 1), (dict(off=None), 1), (dict(off=FAKE + 2), 1),
    (dict(scoring=2), 1), (dict(scoring=-1), 1), (dict(e=1025), 2), (dict(e=64, k=33), 2), (dict(m=1 << 30), 2),
    (dict(seqs=(1 << 24) + 1), 2), (dict(logits=None), 1), (dict(logits=FAKE + 2), 1), (dict(ids=None), 1), (dict(balance=None), 1),
    (dict(z=None), 1), (dict(counts=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 128), 1), (dict(size=511), 3), (dict(m=0, ws=None), 0),
])
def test_balance_loss_refuses(B, kw, want):
    lib = B.load_library()
    assert _call(lib.moe_balance_loss, LOSS, kw) == want
    n = SZ()
    assert lib.moe_balance_loss_workspace_size(10, 3, ctypes.byref(n)) == 0 and n.value == 512
    assert lib.moe_balance_loss_workspace_size(10, 0, ctypes.byref(n)) == 1


BACK = dict(logits=FAKE, ids=FAKE, m=10, e=8, k=2, scoring=1, norm=1, scale=2.0, dw=FAKE, off=None, seqs=1, counts=FAKE, db=FAKE,
            dz=FAKE, d=FAKE + 4096, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), 1), (dict(k=9), 1), (dict(seqs=2), 1), (dict(scoring=3), 1), (dict(norm=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(e=2048, k=2), 2), (dict(logits=None), 1), (dict(ids=None), 1),
    (dict(d=None), 1), (dict(d=FAKE), 1), (dict(d=FAKE + 2), 1), (dict(dw=FAKE + 2), 1), (dict(counts=None), 1), (dict(dz=FAKE + 1), 1),
    (dict(m=0, d=None), 0), (dict(m=0, scoring=0, scale=0.0, norm=5), 0),
])
def test_route_backward_refuses(B, kw, want):
    assert _call(B.load_library().moe_route_backward, BACK, kw) == want


LORA = dict(x=FAKE, ldx=64, m=200, k=64, y=FAKE + (1 << 20), ldy=128, d=128, a=FAKE, b=FAKE, n=4, r=16, ids=FAKE, scale=FAKE,
            out=FAKE + (2 << 20), ldo=128, ws=FAKE, size=1 << 30, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), 1), (dict(k=60), 1), (dict(k=0), 1), (dict(d=12), 1), (dict(d=0), 1), (dict(r=0), 1), (dict(r=12), 1), (dict(n=0), 1),
    (dict(r=136), 2), (dict(m=1 << 30), 2), (dict(k=(1 << 20) + 8), 2), (dict(d=(1 << 20) + 8), 2), (dict(n=(1 << 26) + 1), 2),
    (dict(x=None), 1), (dict(x=FAKE + 2), 1), (dict(ldx=56), 1), (dict(ldy=120), 1), (dict(ldo=132), 1),
    (dict(out=FAKE + (1 << 20), ldo=136), 1), (dict(out=FAKE), 1), (dict(a=None), 1), (dict(b=FAKE + 8), 1), (dict(ids=None), 1),
    (dict(ids=FAKE + 2), 1), (dict(scale=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 64), 1), (dict(size=256), 3),
    (dict(m=0, x=None), 0),
])
def test_lora_refuses(B, kw, want):
    assert _call(B.load_library().moe_lora_add, LORA, kw) == want


def test_experts_from_eight_bits_need_a_layer(B):
    lib = B.load_library()
    assert lib.moe_experts_fp8(None, FAKE, FAKE, None, 1, FAKE, FAKE, FAKE, 0, FAKE, 1 << 20, None) == 1


def test_workspaces_never_shrink_with_tokens(B):
    lib = B.load_library()
    for fn, args in ((lib.moe_lora_add_workspace_size, (4096, 64)), (lib.moe_add_rmsnorm_backward_workspace_size, (1032,)),
                     (lib.moe_balance_loss_workspace_size, (5,))):
        last = 0
        for m in (0, 1, 8, 64, 65, 128, 129, 1000, 19456, 19457, 100000):
            n = SZ()
            assert fn(m, *args, ctypes.byref(n)) == 0 and n.value >= last
            last = n.value


@pytest.mark.parametrize("kw,ok", [
    (dict(), True),
    (dict(y=FAKE + 128, out=FAKE + 128, ldx=192, ldy=192, ldo=192), True),          # side by side with x
    (dict(y=FAKE + 112, out=FAKE + 112, ldx=192, ldy=192, ldo=192), False),         # ... and into its last columns
    (dict(y=FAKE + 160, out=FAKE + 160, ldx=192, ldy=192, ldo=192), False),         # ... round to its next row's first
    (dict(x=FAKE + 256, y=FAKE, out=FAKE, ldx=192, ldy=192, ldo=192), True),        # the other way about
    (dict(out=FAKE + 4096 + 16, ldo=128), False),                                   # a part of y
    (dict(out=FAKE + 4096, ldo=136), False),                                        # y's start, other rows
    (dict(out=FAKE + 4096 + 200 * 256, ldo=128), True), (dict(out=FAKE + 4096 + 200 * 256 - 16, ldo=128), False),
    (dict(m=1, out=FAKE + 4096, ldo=136), True), (dict(m=1, y=FAKE + 128, out=FAKE + 128), True),
])
def test_what_shares_memory(B, kw, ok):
    """Calls refused for it fail there; the others come to the workspace that they lack."""
    args = dict(LORA, x=FAKE, y=FAKE + 4096 + (1 << 20), out=FAKE + 8192 + (2 << 20), size=255) | kw
    if "y" not in kw:
        args["y"] = FAKE + 4096
        args["x"] = FAKE + (1 << 24)
    assert B.load_library().moe_lora_add(*args.values()) == (3 if ok else 1)


@pytest.mark.parametrize("call,match", [
    (lambda B, t: B.moe_add_rmsnorm(t, t[0].float()), "x: "),
    (lambda B, t: B.moe_add_rmsnorm_backward(t, t, t[0].float()), "r: "),
    (lambda B, t: B.moe_balance_loss(t, t.int()), "logits: "),
    (lambda B, t: B.moe_balance_loss(t[0], t.int()), "logits: "),
    (lambda B, t: B.moe_route_backward(t.float(), t.int()), "logits: "),
    (lambda B, t: B.moe_lora_add(t, t, t, t, t[0].int()), "x: "),
    (lambda B, t: B.moe_lora_add(t, t, t[None], t[None], t[0].int()), "x: "),
    (lambda B, t: B.moe_mxfp4_linear(t, t, t, adapters=(t, t, None)), "adapter_ids"),
    (lambda B, t: B.moe_mxfp4_linear(t, t, t, adapter_ids=t), "adapters"),
])
def test_host_tensors_are_refused(B, call, match):
    with pytest.raises(ValueError, match=match):
        call(B, torch.zeros(4, 64, dtype=torch.bfloat16))
