"""ctypes binding of libmoe_ffn_gb300.so (argument marshalling only).

Every entry point keeps the C-ABI's name (moe_route, moe_permute,
moe_experts, moe_forward); the tensors' data pointers and the current torch
CUDA stream are passed straight through.  No computation happens here, and a
missing library is an error: there is no CPU or torch fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

from .build import LIB, build_library, up_to_date

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE = range(6)
MOE_WEIGHTS_BF16, MOE_WEIGHTS_FP8_E4M3_B128, MOE_WEIGHTS_NVFP4, MOE_WEIGHTS_MXFP4 = 0, 1, 2, 3
MOE_ACT_SILU, MOE_ACT_GELU_TANH = 0, 1
ACTIVATIONS = {"silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU_TANH}
MOE_SCORING_SOFTMAX, MOE_SCORING_SIGMOID = 0, 1
MOE_ARM_AUTO, MOE_ARM_GEMV, MOE_ARM_GEMM = 0, 1, 2
MOE_LORA_BY_TOKEN = 64  # up to so many tokens moe_lora_add needs no workspace but its header
ARMS = {"auto": MOE_ARM_AUTO, "gemv": MOE_ARM_GEMV, "gemm": MOE_ARM_GEMM}

EXPORTED = (
    "moe_layer_create", "moe_layer_destroy", "moe_workspace_size", "moe_select_arm", "moe_route",
    "moe_permute", "moe_permute_noalloc", "moe_experts", "moe_experts_fp8", "moe_shared_expert_add", "moe_forward",
    "moe_forward_residual_rmsnorm",
    "moe_act_quant_fp8", "moe_act_quant_nvfp4", "moe_act_quant_nvfp4_f32", "moe_device_status", "moe_router_planes_size",
    "moe_router_prepare", "moe_layer_set_wait_limit",
    "moe_layer_stall_test",
    "moe_last_launch_count", "moe_kernel_timing_enable", "moe_kernel_timing_read", "moe_kernel_count",
    "moe_kernel_name", "moe_status_string",
    "moe_ffn_create", "moe_ffn_destroy", "moe_ffn_workspace_size", "moe_ffn_saved_size", "moe_ffn_forward", "moe_ffn_backward",
    "moe_ffn_set_wait_limit", "moe_ffn_stall_test", "moe_ffn_last_launch_count", "moe_mxfp4_scales_size", "moe_mxfp4_quant", "moe_mxfp4_quant_f32",
    "moe_mxfp4_dequant", "moe_mxfp4_gemm_workspace_size", "moe_mxfp4_gemm",
    "moe_mxfp4_linear_workspace_size", "moe_mxfp4_linear", "moe_mxfp4_linear_f32",
    "moe_add_rmsnorm", "moe_add_rmsnorm_backward_workspace_size", "moe_add_rmsnorm_backward",
    "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_route_backward",
    "moe_lora_add_workspace_size", "moe_lora_add", "moe_lora_set_wait_limit", "moe_lora_stall_test",
    "moe_captured_header", "moe_captured_status",
)

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class MoeConfig(ctypes.Structure):
    _fields_ = [("hidden", _i32), ("num_experts", _i32), ("top_k", _i32), ("inter", _i32),
                ("shared_inter", _i32), ("weights", _i32), ("scoring", _i32), ("norm_topk_prob", _i32),
                ("routed_scaling_factor", ctypes.c_float), ("expert_begin", _i32), ("expert_end", _i32)]


class MoeExpertWeights(ctypes.Structure):
    _fields_ = [("w1", _vp), ("w3", _vp), ("w2", _vp), ("s1", _vp), ("s3", _vp), ("s2", _vp), ("gate", _vp),
                ("sb1", _vp), ("sb3", _vp), ("sb2", _vp)]


class MoeFfnConfig(ctypes.Structure):
    _fields_ = [("hidden", _i32), ("inter", _i32), ("activation", _i32), ("weights", _i32)]


class MoeFfnWeights(ctypes.Structure):
    _fields_ = [("w1", _vp), ("w3", _vp), ("w2", _vp), ("s1", _vp), ("s3", _vp), ("s2", _vp)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None
_lock = threading.Lock()


def load_library(path: str | None = None, build: bool = True):
    """Load (building first if stale) the CUDA library; raises if unavailable."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB
        if build and path is None and not up_to_date():
            build_library()
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library {p} is missing; build it with build_library()")
        lib = ctypes.CDLL(p)
        lib.moe_layer_create.argtypes = [ctypes.POINTER(MoeConfig), ctypes.POINTER(MoeExpertWeights),
                                         ctypes.POINTER(MoeExpertWeights), ctypes.POINTER(_vp)]
        lib.moe_layer_destroy.argtypes = [_vp]
        lib.moe_workspace_size.argtypes = [_vp, _i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.moe_select_arm.argtypes = [_vp, _i64]
        lib.moe_route.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        lib.moe_permute.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        lib.moe_permute_noalloc.argtypes = [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp]
        lib.moe_experts.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        lib.moe_experts_fp8.argtypes = [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        lib.moe_shared_expert_add.argtypes = [_vp, _vp, _i64, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        lib.moe_forward.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        lib.moe_forward_residual_rmsnorm.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp,
                                                     _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
        lib.moe_act_quant_fp8.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp]
        lib.moe_act_quant_nvfp4.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp]
        lib.moe_act_quant_nvfp4_f32.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp]
        lib.moe_device_status.argtypes = [_vp, _vp, ctypes.POINTER(_i32)]
        lib.moe_last_launch_count.argtypes = [_vp]
        lib.moe_router_planes_size.argtypes = [_vp, ctypes.POINTER(ctypes.c_size_t)]
        lib.moe_router_prepare.argtypes = [_vp, _vp, _vp, ctypes.c_size_t, _vp]
        lib.moe_layer_set_wait_limit.argtypes = [_vp, ctypes.c_uint64]
        lib.moe_layer_stall_test.argtypes = [_vp, ctypes.c_int]
        lib.moe_kernel_timing_enable.argtypes = [_vp, ctypes.c_int]
        lib.moe_kernel_timing_read.argtypes = [_vp, ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                               ctypes.POINTER(_i64)]
        lib.moe_kernel_count.argtypes = []
        lib.moe_kernel_name.argtypes = [ctypes.c_int]
        lib.moe_kernel_name.restype = ctypes.c_char_p
        lib.moe_status_string.argtypes = [ctypes.c_int]
        lib.moe_status_string.restype = ctypes.c_char_p
        sz = ctypes.c_size_t
        lib.moe_ffn_create.argtypes = [ctypes.POINTER(MoeFfnConfig), ctypes.POINTER(MoeFfnWeights),
                                       ctypes.POINTER(_vp)]
        lib.moe_ffn_destroy.argtypes = [_vp]
        lib.moe_ffn_workspace_size.argtypes = [_vp, _i64, ctypes.c_int, ctypes.POINTER(sz)]
        lib.moe_ffn_saved_size.argtypes = [_vp, _i64, ctypes.POINTER(sz)]
        lib.moe_ffn_forward.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, sz, _vp]
        lib.moe_ffn_backward.argtypes = [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, sz, _vp]
        lib.moe_ffn_set_wait_limit.argtypes = [_vp, ctypes.c_uint64]
        lib.moe_ffn_stall_test.argtypes = [_vp, ctypes.c_int]
        lib.moe_ffn_last_launch_count.argtypes = [_vp]
        lib.moe_mxfp4_scales_size.argtypes = [_i64, _i64, ctypes.POINTER(sz)]
        lib.moe_mxfp4_quant.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
        lib.moe_mxfp4_quant_f32.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
        lib.moe_mxfp4_dequant.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp]
        lib.moe_mxfp4_gemm_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(sz)]
        lib.moe_mxfp4_gemm.argtypes = [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, sz, _vp]
        lib.moe_mxfp4_linear_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(sz)]
        for fn in (lib.moe_mxfp4_linear, lib.moe_mxfp4_linear_f32):
            fn.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, sz, _vp]
        f32 = ctypes.c_float
        lib.moe_add_rmsnorm.argtypes = [_vp, _i64, _vp, _i64, _i64, _i64, _vp, f32, _vp, _i64, _vp, _vp, _vp, _vp]
        lib.moe_add_rmsnorm_backward_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(sz)]
        lib.moe_add_rmsnorm_backward.argtypes = [_vp, _i64, _vp, _i64, _i64, _i64, _vp, f32, _vp, _i64, _vp, _vp, _vp, sz,
                                                 _vp]
        lib.moe_balance_loss_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(sz)]
        lib.moe_balance_loss.argtypes = [_vp, _vp, _i64, _i32, _i32, _vp, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, sz, _vp]
        lib.moe_route_backward.argtypes = [_vp, _vp, _i64, _i32, _i32, ctypes.c_int, ctypes.c_int, f32, _vp, _vp, _i64, _vp,
                                           _vp, _vp, _vp, _vp]
        lib.moe_lora_add_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(sz)]
        lib.moe_lora_add.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp,
                                     sz, _vp]
        lib.moe_lora_set_wait_limit.argtypes = [ctypes.c_uint64]
        lib.moe_lora_stall_test.argtypes = [ctypes.c_int]
        lib.moe_captured_header.argtypes = [_vp, _vp]
        lib.moe_captured_status.argtypes = [_vp, ctypes.POINTER(_i32)]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load_library(build=False).moe_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - library absent
        return "status"


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _new(stream, device, dtype, *shape):
    """An empty tensor that belongs to the stream that writes it (None: the current one): its memory may
    have been let go a moment ago with work of its old stream still to come, which only that one waits for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_act_quant_fp8(x, stream=None):
    """x bf16 [rows, n] (device) -> (codes uint8 [rows, n], scales fp32 [rows, n/128])."""
    lib = load_library()
    rows, n = x.shape
    codes = _new(stream, x.device, torch.uint8, rows, n)
    scales = _new(stream, x.device, torch.float32, rows, n // 128)
    _check(lib.moe_act_quant_fp8(_p(x), rows, n, _p(codes), _p(scales), _stream(stream)), "moe_act_quant_fp8")
    return codes, scales


def moe_act_quant_nvfp4(x, stream=None):
    """x bf16 or fp32 [rows, n] (device) -> (packed codes uint8 [rows, n/2],
    e4m3 block-scale codes uint8 [rows, n/16], row scales fp32 [rows])."""
    lib = load_library()
    rows, n = x.shape
    codes = _new(stream, x.device, torch.uint8, rows, n // 2)
    sb = _new(stream, x.device, torch.uint8, rows, n // 16)
    g = _new(stream, x.device, torch.float32, rows)
    if x.dtype == torch.float32:
        fn, name = lib.moe_act_quant_nvfp4_f32, "moe_act_quant_nvfp4_f32"
    else:
        assert x.dtype == torch.bfloat16, x.dtype
        fn, name = lib.moe_act_quant_nvfp4, "moe_act_quant_nvfp4"
    _check(fn(_p(x), rows, n, _p(codes), _p(sb), _p(g), _stream(stream)), name)
    return codes, sb, g


_capturing = torch._C._cuda_isCurrentStreamCapturing
_raw_stream = torch._C._cuda_getCurrentRawStream  # of a device index
_current_device = torch._C._cuda_getDevice


def _record(ws, stream):
    """Tells torch that `stream` (None: the current one) uses ws: when ws is let go, its memory goes
    to others only after what that stream has been given."""
    ws.record_stream(stream if stream is not None else torch.cuda.current_stream(ws.device))


class _Workspaces:
    """The workspaces of a handle as its calls use them, one after another as each is outgrown.  A
    handle zeroes a workspace's header in the first call on it, on that call's stream; nothing here
    writes into one."""

    def __init__(self):
        self.used = None      # of the last call; kept until there is a call on another
        self.streams = set()  # that `used` is recorded on
        self.held = []        # those that captured graphs replay into
        self.headers = []     # of those outgrown that no graph uses

    def hold(self, ws):
        """Keeps ws for good if a CUDA graph is being captured, which will replay into it."""
        if _capturing() and not any(t is ws for t in self.held):
            self.held.append(ws)

    def called(self, ws, stream=None):
        """A call on `stream` (None: the current one) that uses ws has been launched."""
        raw = _raw_stream(ws.get_device()) if stream is None else stream.cuda_stream
        capturing = _capturing()
        if ws is not self.used:
            old, self.used, self.streams = self.used, ws, set()
            if old is not None and not any(t is old for t in self.held):
                if capturing:  # a copy would be made when the graph runs
                    self.headers.append(old)
                elif stream is None:
                    self.headers.append(old[:256].clone())
                    _record(old, None)
                else:
                    with torch.cuda.stream(stream):
                        self.headers.append(old[:256].clone())
                    _record(old, stream)
        if capturing:
            self.hold(ws)
        elif raw not in self.streams:
            _record(ws, stream)
            self.streams.add(raw)

    def status(self, stream) -> int:
        """The first device error (0: none) in the words of the workspaces that calls have used; a
        word that is set is cleared."""
        code, first = _i32(), 0
        for t in (*self.headers, *(t for t in self.held if t is not self.used), self.used):
            if t is None:
                continue
            rc = load_library().moe_device_status(_p(t), _stream(stream), ctypes.byref(code))
            if rc not in (MOE_OK, MOE_ERR_DEVICE):
                raise MoeError(rc, "moe_device_status")
            first = first or code.value
        self.headers.clear()
        return first


class MoeLayer:
    """A layer handle over caller-owned device weights (see include/moe_ffn.h).

    tensors: dict with w1, w3, w2 (and s1, s3, s2 for fp8; s1, s3, s2 and
    sb1, sb3, sb2 for NVFP4), optionally ws1, ws3, ws2 (+ ss1, ss3, ss2, and
    ssb1, ssb3, ssb2) for the shared expert, as produced by
    ``inputs.make_experts`` and moved to the device.
    """

    def __init__(self, shape, tensors: dict, expert_range=None):
        """expert_range: (begin, end) makes this handle one expert-parallel
        shard holding experts [begin, end) of shape.num_experts; its tensors
        w1, w3, w2 (and s*, sb*) are then stacked over those experts only."""
        self.lib = load_library()
        self.shape = shape
        self._keep = dict(tensors)
        sigmoid = getattr(shape, "scoring", "softmax") == "sigmoid"
        nvfp4 = bool(getattr(shape, "nvfp4", False))
        wfmt = MOE_WEIGHTS_NVFP4 if nvfp4 else (MOE_WEIGHTS_FP8_E4M3_B128 if shape.fp8 else MOE_WEIGHTS_BF16)
        cfg = MoeConfig(shape.hidden, shape.num_experts, shape.top_k, shape.inter, shape.shared_inter, wfmt,
                        MOE_SCORING_SIGMOID if sigmoid else MOE_SCORING_SOFTMAX,
                        int(bool(getattr(shape, "norm_topk_prob", True))),
                        float(getattr(shape, "routed_scaling", 1.0)),
                        *(expert_range if expert_range is not None else (0, 0)))
        sbn = ("sb1", "sb3", "sb2") if nvfp4 else ()
        routed = MoeExpertWeights(*[_p(tensors.get(n)) for n in ("w1", "w3", "w2", "s1", "s3", "s2")], None,
                                  *[_p(tensors.get(n)) for n in sbn])
        shared = None
        if shape.shared_inter:
            gate = _p(tensors.get("shared_gate")) if getattr(shape, "shared_gate", False) else None
            shared = MoeExpertWeights(*[_p(tensors.get(n)) for n in ("ws1", "ws3", "ws2", "ss1", "ss3", "ss2")],
                                      gate, *[_p(tensors.get("s" + n)) for n in sbn])
        self.expert_range = tuple(expert_range) if expert_range is not None else (0, shape.num_experts)
        handle = _vp()
        _check(self.lib.moe_layer_create(ctypes.byref(cfg), ctypes.byref(routed),
                                         ctypes.byref(shared) if shared is not None else None,
                                         ctypes.byref(handle)), "moe_layer_create")
        self.handle = handle
        self._new_workspaces()

    def _new_workspaces(self):
        self._ws = None
        self._past = _Workspaces()

    def close(self):
        if getattr(self, "handle", None):
            self.lib.moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- workspace
    def workspace_size(self, m: int) -> int:
        n = ctypes.c_size_t()
        _check(self.lib.moe_workspace_size(self.handle, int(m), ctypes.byref(n)), "moe_workspace_size")
        return n.value

    def workspace(self, m: int, device=None) -> torch.Tensor:
        """The handle's own workspace, grown to what a call on m tokens needs.  Those that captured
        graphs use live as long as the handle."""
        need = self.workspace_size(m)
        if self._ws is None or self._ws.numel() < need:
            self._grow(need, device)
        self._past.hold(self._ws)
        return self._ws

    def _grow(self, need: int, device=None):
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self._ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)

    def _call_space(self, m: int, stream) -> torch.Tensor:
        """The workspace for a call on `stream`."""
        need = self.workspace_size(m)
        if self._ws is None or self._ws.numel() < need:
            if stream is None:
                self._grow(need)
            else:
                with torch.cuda.stream(stream):  # what it allocates belongs to the stream that writes it
                    self._grow(need)
        return self._ws

    def select_arm(self, m: int) -> int:
        return self.lib.moe_select_arm(self.handle, int(m))

    def prepare_router(self, router_w, stream=None):
        """Split router_w once into planes this handle keeps (moe_router_prepare);
        router_w=None forgets them."""
        if router_w is None:
            _check(self.lib.moe_router_prepare(self.handle, None, None, 0, _stream(stream)), "moe_router_prepare")
            self._planes = None
            return
        n = ctypes.c_size_t()
        _check(self.lib.moe_router_planes_size(self.handle, ctypes.byref(n)), "moe_router_planes_size")
        self._planes = _new(stream, router_w.device, torch.uint8, max(n.value, 256))
        _check(self.lib.moe_router_prepare(self.handle, _p(router_w), _p(self._planes), self._planes.numel(),
                                           _stream(stream)), "moe_router_prepare")

    def set_wait_limit(self, ns: int):
        """Limit (ns) of the grouped GEMMs' bounded waits; 0 restores 2 s."""
        _check(self.lib.moe_layer_set_wait_limit(self.handle, int(ns)), "moe_layer_set_wait_limit")

    def stall_test(self, enable: bool):
        """Make the bf16 grouped GEMMs wait on a barrier nothing completes."""
        _check(self.lib.moe_layer_stall_test(self.handle, int(bool(enable))), "moe_layer_stall_test")

    def last_launch_count(self) -> int:
        return self.lib.moe_last_launch_count(self.handle)

    def kernel_timing(self, enable: bool):
        """Turn per-kernel event timing on or off (resets the totals)."""
        _check(self.lib.moe_kernel_timing_enable(self.handle, int(bool(enable))), "moe_kernel_timing_enable")

    def kernel_times(self) -> dict:
        """{kernel name: (total ms, launches)} for kernels launched while timing was on."""
        out = {}
        for k in range(self.lib.moe_kernel_count()):
            ms = ctypes.c_double()
            n = _i64()
            _check(self.lib.moe_kernel_timing_read(self.handle, k, ctypes.byref(ms), ctypes.byref(n)),
                   "moe_kernel_timing_read")
            if n.value:
                out[self.lib.moe_kernel_name(k).decode()] = (ms.value, n.value)
        return out

    def device_status(self, stream=None) -> int:
        """The first device error (0: none) of the handle's calls since it was last read; of a workspace
        that was made during a capture, from the graph's first run on."""
        return self._past.status(stream)

    # ---- entry points
    def moe_route(self, x, router_w, router_bias=None, logits=False, stream=None):
        m = x.shape[0]
        dev = x.device
        ids = _new(stream, dev, torch.int32, m, self.shape.top_k)
        w = _new(stream, dev, torch.float32, m, self.shape.top_k)
        lg = _new(stream, dev, torch.float32, m, self.shape.num_experts) if logits else None
        ws = self._call_space(m, stream)
        _check(self.lib.moe_route(self.handle, _p(x), m, _p(router_w), _p(router_bias), _p(lg), _p(ids), _p(w),
                                  _p(ws), ws.numel(), _stream(stream)), "moe_route")
        if m:
            self._past.called(ws, stream)
        return (ids, w, lg) if logits else (ids, w)

    def moe_permute(self, topk_ids, stream=None):
        m = topk_ids.shape[0]
        dev = topk_ids.device
        P = m * self.shape.top_k
        n_local = self.expert_range[1] - self.expert_range[0]  # this handle's experts
        off = _new(stream, dev, torch.int32, n_local + 1)
        sp = _new(stream, dev, torch.int32, P)
        sl = _new(stream, dev, torch.int32, P)
        ws = self._call_space(m, stream)
        _check(self.lib.moe_permute(self.handle, _p(topk_ids), m, _p(off), _p(sp), _p(sl), _p(ws), ws.numel(),
                                    _stream(stream)), "moe_permute")
        if m:
            self._past.called(ws, stream)
        return off, sp, sl

    def moe_experts(self, x, topk_ids, topk_w, arm="auto", out=None, stream=None):
        m = x.shape[0]
        if out is None:
            out = _new(stream, x.device, torch.bfloat16, m, self.shape.hidden)
        ws = self._call_space(m, stream)
        _check(self.lib.moe_experts(self.handle, _p(x), m, _p(topk_ids), _p(topk_w), _p(out), ARMS[arm], _p(ws),
                                    ws.numel(), _stream(stream)), "moe_experts")
        if m:
            self._past.called(ws, stream)
        return out

    def moe_experts_fp8(self, codes, scales, topk_ids, topk_w, x=None, arm="auto", out=None, stream=None):
        """moe_experts of an fp8 layer from x in 8 bits (codes uint8 [m, H], scales fp32 [m, H/128], as
        moe_add_rmsnorm and moe_act_quant_fp8 give them); x (bf16) only for a shared expert with a gate."""
        H, k = self.shape.hidden, self.shape.top_k
        _need(codes.dim() == 2, "codes: [m, H]")
        m = codes.shape[0]
        _dense(codes, _U8, (m, H), "codes")
        _dense(scales, _F32, (m, H // 128), "scales")
        _dense(topk_ids, torch.int32, (m, k), "topk_ids")
        _dense(topk_w, _F32, (m, k), "topk_w")
        _on(codes, scales, topk_ids, topk_w)
        if x is not None:
            _dense(x, _BF16, (m, H), "x")
            _on(x)
        if out is None:
            out = _new(stream, codes.device, torch.bfloat16, m, H)
        else:
            _dense(out, _BF16, (m, H), "out")
            _on(out)
        ws = self._call_space(m, stream)
        _check(self.lib.moe_experts_fp8(self.handle, _p(codes), _p(scales), _p(x), m, _p(topk_ids), _p(topk_w), _p(out),
                                        ARMS[arm], _p(ws), ws.numel(), _stream(stream)), "moe_experts_fp8")
        if m:
            self._past.called(ws, stream)
        return out

    def moe_balance_loss(self, logits, topk_ids, seq_offsets=None, stream=None):
        """moe_balance_loss of this layer's scoring."""
        return moe_balance_loss(logits, topk_ids, seq_offsets, getattr(self.shape, "scoring", "softmax"), stream)

    def moe_route_backward(self, logits, topk_ids, dtopk_w=None, dbalance=None, dz=None, counts=None, seq_offsets=None,
                           stream=None):
        """moe_route_backward of this layer's scoring and weights."""
        sh = self.shape
        return moe_route_backward(logits, topk_ids, dtopk_w, dbalance, dz, counts, seq_offsets,
                                  getattr(sh, "scoring", "softmax"), getattr(sh, "norm_topk_prob", True),
                                  float(getattr(sh, "routed_scaling", 1.0)), stream)

    def moe_shared_expert_add(self, x, out, arm="auto", stream=None):
        """out (bf16 [m, H], in place) += the shared expert of x."""
        m = x.shape[0]
        ws = self._call_space(m, stream)
        _check(self.lib.moe_shared_expert_add(self.handle, _p(x), m, _p(out), ARMS[arm], _p(ws), ws.numel(),
                                              _stream(stream)), "moe_shared_expert_add")
        if m:
            self._past.called(ws, stream)
        return out

    def moe_forward(self, x, router_w, router_bias=None, arm="auto", out=None, return_routing=False, stream=None):
        m = x.shape[0]
        dev = x.device
        if out is None:
            out = _new(stream, dev, torch.bfloat16, m, self.shape.hidden)
        ids = w = None
        if return_routing:
            ids = _new(stream, dev, torch.int32, m, self.shape.top_k)
            w = _new(stream, dev, torch.float32, m, self.shape.top_k)
        ws = self._call_space(m, stream)
        _check(self.lib.moe_forward(self.handle, _p(x), m, _p(router_w), _p(router_bias), _p(out), _p(ids), _p(w),
                                    ARMS[arm], _p(ws), ws.numel(), _stream(stream)), "moe_forward")
        if m:
            self._past.called(ws, stream)
        return (out, ids, w) if return_routing else out

    def moe_forward_residual_rmsnorm(self, x, router_w, residual, norm_w, eps=1e-6, router_bias=None, arm="auto",
                                     norm_out=None, return_routing=False, stream=None):
        """The layer with its tail: residual (bf16 [m, H], updated in place) +=
        the layer output, and norm_out = RMSNorm(residual) * norm_w (fp32 [H])."""
        m = x.shape[0]
        dev = x.device
        if norm_out is None:
            norm_out = _new(stream, dev, torch.bfloat16, m, self.shape.hidden)
        ids = w = None
        if return_routing:
            ids = _new(stream, dev, torch.int32, m, self.shape.top_k)
            w = _new(stream, dev, torch.float32, m, self.shape.top_k)
        ws = self._call_space(m, stream)
        _check(self.lib.moe_forward_residual_rmsnorm(self.handle, _p(x), m, _p(router_w), _p(router_bias),
                                                     _p(residual), _p(norm_w), float(eps), _p(norm_out), _p(ids),
                                                     _p(w), ARMS[arm], _p(ws), ws.numel(), _stream(stream)),
               "moe_forward_residual_rmsnorm")
        if m:
            self._past.called(ws, stream)
        return (norm_out, ids, w) if return_routing else norm_out


# ---------------------------------------------------------------- the gated feed-forward block and MXFP4
# (include/moe_ffn_block.h).  A decode step calls these once per layer, so the
# checks test the common case (dense rows) first and word the refusal after.

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_empty, _empty_like, _dense_rows = torch.empty, torch.empty_like, torch.contiguous_format


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _rows(t, n: int, what: str, f32: bool = False) -> int:
    """Checks a [rows, n] device matrix of bf16 (or fp32 where f32) whose rows are dense and
    16-byte aligned; returns its row stride."""
    if t.dtype is _BF16 and t.is_cuda and t.is_contiguous() and t.dim() == 2 and t.shape[1] == n \
            and t.data_ptr() % 16 == 0:
        return n
    _need(t.is_cuda and t.dim() == 2 and (t.dtype is _BF16 or (f32 and t.dtype is _F32)),
          f"{what}: a 2-d device tensor of bfloat16{' or float32' if f32 else ''}")
    _need(t.shape[1] == n, f"{what}: [rows, {n}], got {tuple(t.shape)}")
    ld = t.stride(0) if t.shape[0] > 1 else n
    _need(t.numel() == 0 or (t.stride(1) == 1 and ld >= n and ld * t.element_size() % 16 == 0
                             and t.data_ptr() % 16 == 0), f"{what}: rows must be dense and 16-byte aligned")
    return ld


def _dense(t, dtype, shape, what: str):
    if not (t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.shape == shape):
        raise ValueError(f"{what}: a contiguous device tensor of {dtype}, {tuple(shape)}")


def _on(*tensors) -> int:
    """The current CUDA stream of the device that every one of `tensors` lies on: the current
    device, on which the library launches.  A call that is given a stream makes it the current one
    first, so that what it allocates belongs to the stream that writes it."""
    dev = _current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"a tensor on {t.device} in a call on cuda:{dev}, the current device")
    return _raw_stream(dev)


def mxfp4_scales_shape(rows: int, n: int):
    """Shape of the packed scales of a [rows, n] matrix: [row tile, K tile, row % 32, row / 32, block]."""
    return (rows + 127) // 128, (n + 127) // 128, 32, 4, 4


def mxfp4_pack_scales(scales):
    """e8m0 scale bytes in rows (uint8 [rows, n/32], as checkpoints hold them) to the packed order."""
    rows, nb = scales.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    s = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=scales.device)
    s[:rows, :nb] = scales
    return s.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()


def mxfp4_unpack_scales(scales, rows: int, n: int):
    """The packed scales of a [rows, n] matrix back in rows, uint8 [rows, n/32]."""
    rt, kt = scales.shape[:2]
    return scales.permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, : n // 32].contiguous()


def _mx_matrix(codes, scales, what: str):
    """(rows, n) of a matrix held as codes and packed scales."""
    if codes.dim() != 2:
        raise ValueError(f"{what}: codes are [rows, n/2]")
    rows, half = codes.shape
    if not (codes.dtype is _U8 and codes.is_cuda and codes.is_contiguous()):
        raise ValueError(f"{what} codes: a contiguous device tensor of uint8")
    _dense(scales, _U8, ((rows + 127) // 128, (half + 63) // 64, 32, 4, 4), what + " scales")
    return rows, 2 * half


def moe_mxfp4_quant(x, stream=None):
    """x bf16 or fp32 [rows, n] (device; n a multiple of 32) -> (codes uint8 [rows, n/2], packed scales uint8)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_mxfp4_quant(x)
    lib = _lib or load_library()
    _need(x.dim() == 2, "x: [rows, n]")
    rows, n = x.shape
    ld = _rows(x, n, "x", f32=True)
    st = _on(x)
    dev = x.device
    codes = _empty((rows, n // 2), dtype=_U8, device=dev)
    scales = _empty(mxfp4_scales_shape(rows, n), dtype=_U8, device=dev)
    f32 = x.dtype is _F32
    rc = (lib.moe_mxfp4_quant_f32 if f32 else lib.moe_mxfp4_quant)(
        x.data_ptr(), ld, rows, n, codes.data_ptr(), scales.data_ptr(), st)
    if rc:
        raise MoeError(rc, "moe_mxfp4_quant_f32" if f32 else "moe_mxfp4_quant")
    return codes, scales


def moe_mxfp4_dequant(codes, scales, stream=None):
    """The values (bf16 [rows, n]) that codes and packed scales stand for; infinite past bf16's range."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_mxfp4_dequant(codes, scales)
    lib = _lib or load_library()
    rows, n = _mx_matrix(codes, scales, "x")
    st = _on(codes, scales)
    out = _empty((rows, n), dtype=_BF16, device=codes.device)
    rc = lib.moe_mxfp4_dequant(codes.data_ptr(), scales.data_ptr(), rows, n, out.data_ptr(), st)
    if rc:
        raise MoeError(rc, "moe_mxfp4_dequant")
    return out


_spaces = {}  # (device, stream) -> workspace of the operators without a handle launched on that stream, _Workspaces
# Held from the choice of such a workspace to the last launch that uses it: a product may be two
# launches, and other threads run during the library's calls.
_spaces_lock = threading.RLock()
_captured = set()  # devices on which a graph has captured calls of these operators


def _space(like, stream: int, need: int) -> torch.Tensor:
    """A workspace of at least `need` bytes for calls on `stream`, the current one, its header
    zeroed before first use.  A call that is captured into a graph gets one from the graph's own
    pool: the graph may be replayed beside eager calls, and after they have needed a larger one.
    The pool takes it back after the call, so that its errors go to the device's shared word."""
    key = (like.get_device(), stream)
    entry = _spaces.get(key)
    capturing = _capturing()
    if entry is not None and entry[0].numel() >= need and not capturing:
        return entry[0]
    ws = _empty((max(need, 1 << 16),), dtype=_U8, device=like.device)
    if capturing and ws.is_cuda:
        _check((_lib or load_library()).moe_captured_header(_p(ws), stream), "moe_captured_header")
        _captured.add(key[0])
    else:
        ws[:256].zero_()
    if not capturing:
        past = entry[1] if entry is not None else _Workspaces()
        past.called(ws)
        _spaces[key] = ws, past
    return ws


def _scratch(like, stream: int, need: int):
    """(address, what keeps it) of `need` bytes for a call on `stream` that keeps nothing in them: behind
    the header of the stream's workspace, or a captured graph's own."""
    if _capturing():
        ws = _empty((need,), dtype=_U8, device=like.device)
        return ws.data_ptr(), ws
    ws = _space(like, stream, need + 256)
    return ws.data_ptr() + 256, ws


def mxfp4_device_status(stream=None) -> int:
    """The first device error (0: none) of the MXFP4 products and adapters since it was last read: of
    eager calls on `stream`, and of captured ones on its device, whichever stream replays them (of
    other streams' replays, what has run by then)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    with _spaces_lock:
        ws, past = _spaces.get((s.device.index, s.cuda_stream), (None, None))
        first = 0 if ws is None else past.status(s)
        if s.device.index in _captured:
            code = _i32()
            with torch.cuda.device(s.device):
                rc = load_library().moe_captured_status(s.cuda_stream, ctypes.byref(code))
            if rc not in (MOE_OK, MOE_ERR_DEVICE):
                raise MoeError(rc, "moe_captured_status")
            first = first or code.value
        return first


def moe_mxfp4_gemm(a_codes, a_scales, b_codes, b_scales, out=None, stream=None):
    """A [m, k] times B [n, k] transposed, both MXFP4 (codes, packed scales) -> bf16 [m, n]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_mxfp4_gemm(a_codes, a_scales, b_codes, b_scales, out)
    lib = _lib or load_library()
    m, k = _mx_matrix(a_codes, a_scales, "a")
    n, kb = _mx_matrix(b_codes, b_scales, "b")
    _need(k == kb, f"k differs: {k} and {kb}")
    st = _on(a_codes, a_scales, b_codes, b_scales)
    if out is None:
        out = _empty((m, n), dtype=_BF16, device=a_codes.device)
    else:
        _dense(out, _BF16, (m, n), "out")
        _on(out)
    with _spaces_lock:
        ws = _space(a_codes, st, 256)
        rc = lib.moe_mxfp4_gemm(a_codes.data_ptr(), a_scales.data_ptr(), m, b_codes.data_ptr(), b_scales.data_ptr(), n,
                                k, out.data_ptr(), ws.data_ptr(), ws.numel(), st)
    if rc:
        raise MoeError(rc, "moe_mxfp4_gemm")
    return out


def moe_mxfp4_linear(x, codes, scales, out=None, stream=None, adapters=None, adapter_ids=None):
    """x (bf16 or fp32 [m, k]) quantised to MXFP4 per call, times a weight matrix [n, k] held in
    MXFP4 -> bf16 [m, n].  With adapters (a, b, scale), each token's low-rank adapter of x (bf16)
    is then added, moe_lora_add of adapter_ids; out may not be x there."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_mxfp4_linear(x, codes, scales, out, None, adapters, adapter_ids)
    if adapters is not None:
        _need(adapter_ids is not None, "adapters without adapter_ids")
        a, b, scale = adapters
        _need(codes.dim() == 2, "w: codes are [rows, n/2]")
        y = _empty((x.shape[0], codes.shape[0]), dtype=_BF16, device=x.device) if out is None else out
        _dense(y, _BF16, (x.shape[0], codes.shape[0]), "out")
        dev = _device_of(x, "x")
        _, args = _lora_args(y, x, a, b, adapter_ids, scale, None, dev)
        if out is not None and x.numel():
            at, to = x.data_ptr(), out.data_ptr()
            _need(to + 2 * out.numel() <= at or at + 2 * ((x.shape[0] - 1) * x.stride(0) + x.shape[1]) <= to,
                  "out: no part of x, where there are adapters")
        # What the library refuses of the adapters is refused before the product writes out: a call
        # without room for its workspace comes through all of its checks and launches nothing.
        rc = (_lib or load_library()).moe_lora_add(*args, 256, 0, None)  # 256: an address nobody looks at
        if rc not in (MOE_OK, MOE_ERR_WORKSPACE):
            raise MoeError(rc, "moe_lora_add")
        moe_mxfp4_linear(x, codes, scales, y)
        _lora_launch(x, args, dev)
        return y
    _need(adapter_ids is None, "adapter_ids without adapters")
    lib = _lib or load_library()
    n, k = _mx_matrix(codes, scales, "w")
    ld = _rows(x, k, "x", f32=True)
    m = x.shape[0]
    st = _on(x, codes, scales)
    if out is None:
        out = _empty((m, n), dtype=_BF16, device=x.device)
    else:
        _dense(out, _BF16, (m, n), "out")
        _on(out)
    f32 = x.dtype is _F32
    with _spaces_lock:
        # what moe_mxfp4_linear_workspace_size returns for a k that is a multiple of 32
        ws = _space(x, st, 1024 + m * k // 2 + (m + 127) // 128 * ((k + 127) // 128) * 512)
        rc = (lib.moe_mxfp4_linear_f32 if f32 else lib.moe_mxfp4_linear)(
            x.data_ptr(), ld, m, codes.data_ptr(), scales.data_ptr(), n, k, out.data_ptr(), ws.data_ptr(), ws.numel(),
            st)
    if rc:
        raise MoeError(rc, "moe_mxfp4_linear_f32" if f32 else "moe_mxfp4_linear")
    return out


class GatedFfn:
    """A dense gated feed-forward block over caller-owned device weights:
    out = (act(x w1^T) * (x w3^T)) w2^T, w1, w3 [I, H], w2 [H, I].

    Weights are bf16 tensors, or (codes, packed scales) pairs as
    moe_mxfp4_quant returns them; act is "silu" or "gelu" (tanh form).
    A handle keeps one workspace: order its calls, replays of graphs that
    captured them among these, as on one stream, and make them from one thread
    at a time.  Such graphs need the handle alive."""

    def __init__(self, w1, w3, w2, act="silu"):
        self.lib = load_library()
        _need(act in ACTIVATIONS, f"act: one of {sorted(ACTIVATIONS)}")
        self.mxfp4 = isinstance(w1, (tuple, list))
        if self.mxfp4:
            (I, H), shapes = _mx_matrix(*w1, "w1"), [_mx_matrix(*w, n) for w, n in ((w3, "w3"), (w2, "w2"))]
            _need(shapes == [(I, H), (H, I)], "w1, w3 [I, H], w2 [H, I]")
            ptrs = [_p(w[0]) for w in (w1, w3, w2)] + [_p(w[1]) for w in (w1, w3, w2)]
        else:
            _need(w1.dim() == 2, "w1: [I, H]")
            I, H = w1.shape
            for w, shape, name in ((w1, (I, H), "w1"), (w3, (I, H), "w3"), (w2, (H, I), "w2")):
                _dense(w, _BF16, shape, name)
            ptrs = [_p(w) for w in (w1, w3, w2)] + [None] * 3
        self._keep = (w1, w3, w2)
        _on(*(t for w in self._keep for t in (w if self.mxfp4 else (w,))))
        self._dev = (w1[0] if self.mxfp4 else w1).get_device()
        self.hidden, self.inter, self.act = H, I, act
        cfg = MoeFfnConfig(H, I, ACTIVATIONS[act], MOE_WEIGHTS_MXFP4 if self.mxfp4 else MOE_WEIGHTS_BF16)
        w = MoeFfnWeights(*ptrs)
        handle = _vp()
        _check(self.lib.moe_ffn_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(handle)), "moe_ffn_create")
        self.handle = handle
        self._saved = {}  # words saved, by tokens
        self._new_workspaces()

    def _new_workspaces(self):
        self._ws = None
        self._ws_at = (None, 0)
        self._fits = [-1, -1]  # tokens the workspace holds: forward, backward
        self._past = _Workspaces()

    def close(self):
        if getattr(self, "handle", None):
            self.lib.moe_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_size(self, m: int, backward: bool = False) -> int:
        n = ctypes.c_size_t()
        _check(self.lib.moe_ffn_workspace_size(self.handle, int(m), int(backward), ctypes.byref(n)),
               "moe_ffn_workspace_size")
        return n.value

    def workspace(self, m: int, backward: bool, device) -> torch.Tensor:
        """The handle's own workspace, grown to what a call on m tokens needs.  Those that captured
        graphs use live as long as the handle."""
        if m > self._fits[backward]:
            need = self.workspace_size(m, backward)
            if self._ws is None or self._ws.numel() < need:
                self._ws = torch.empty(max(need, 256), dtype=_U8, device=device)
                self._ws_at = (self._ws.data_ptr(), self._ws.numel())
            self._fits[backward] = m
        self._past.hold(self._ws)
        return self._ws

    def set_wait_limit(self, ns: int):
        """Limit (ns) of the kernels' bounded waits; 0 restores 2 s."""
        _check(self.lib.moe_ffn_set_wait_limit(self.handle, int(ns)), "moe_ffn_set_wait_limit")

    def stall_test(self, enable: bool):
        """Make the kernels wait on a barrier nothing completes."""
        _check(self.lib.moe_ffn_stall_test(self.handle, int(bool(enable))), "moe_ffn_stall_test")

    def last_launch_count(self) -> int:
        return self.lib.moe_ffn_last_launch_count(self.handle)

    def device_status(self, stream=None) -> int:
        """The first device error (0: none) of the handle's calls since it was last read; of a workspace
        that was made during a capture, from the graph's first run on."""
        return self._past.status(stream)

    def _stream_for(self, *tensors) -> int:
        """As _on, for tensors on the weights' device; that it is the current one the library checks."""
        dev = self._dev
        for t in tensors:
            if t.get_device() != dev:
                raise ValueError(f"a tensor on {t.device} in a call of a block on cuda:{dev}")
        return _raw_stream(dev)

    def saved_size(self, m: int) -> int:
        """Words of what a forward pass on m tokens saves (moe_ffn_saved_size, in 4-byte words)."""
        n = self._saved.get(m)
        if n is None:
            c = ctypes.c_size_t()
            _check(self.lib.moe_ffn_saved_size(self.handle, int(m), ctypes.byref(c)), "moe_ffn_saved_size")
            n = self._saved[m] = (c.value + 3) // 4
        return n

    def forward(self, x, save=False, out=None, stream=None):
        """x bf16 [m, H] (rows may be strided) -> out bf16 [m, H] (out may be x); with save (bf16
        weights), (out, saved) for backward: saved is fp32 [saved_size(m)], in moe_ffn_forward's own
        order.  Up to 8 tokens keep h in 16 bits unless it is saved, and differ from a saving call by
        h's rounding to bf16.  Given a stream, the call's inputs have to stay until that has run it."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, save, out)
        ld = _rows(x, self.hidden, "x")
        m = x.shape[0]
        st = self._stream_for(x)
        if out is None:
            out = _empty_like(x, memory_format=_dense_rows)
        else:
            _dense(out, _BF16, (m, self.hidden), "out")
            self._stream_for(out)
        if m > self._fits[0]:
            self.workspace(m, False, x.device)
        saved = _empty(self.saved_size(m), dtype=_F32, device=x.device) if save else None
        rc = self.lib.moe_ffn_forward(self.handle, x.data_ptr(), ld, m, out.data_ptr(),
                                      saved.data_ptr() if save else None, *self._ws_at, st)
        if rc:
            raise MoeError(rc, "moe_ffn_forward")
        past = self._past
        if m and (past.used is not self._ws or st not in past.streams or _capturing()):
            past.called(self._ws)
        return (out, saved) if save else out

    def backward(self, dout, x, saved, need_dx=True, need_dw=True, stream=None):
        """Gradients (dx, dw1, dw3, dw2), bf16, of the forward pass that saved `saved`; None
        for those not needed.  No tokens: the weight gradients are zero."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(dout, x, saved, need_dx, need_dw)
        H, I = self.hidden, self.inter
        ldd, ldx = _rows(dout, H, "dout"), _rows(x, H, "x")
        m = x.shape[0]
        _need(dout.shape[0] == m, "dout and x differ in rows")
        _dense(saved, _F32, (self.saved_size(m),), "saved")
        st = self._stream_for(dout, x, saved)
        dx = _empty_like(x, memory_format=_dense_rows) if need_dx else None
        dw1 = dw3 = dw2 = None
        if need_dw:
            new, dev = _empty if m else torch.zeros, x.device
            dw1 = new((I, H), dtype=_BF16, device=dev)
            dw3 = new((I, H), dtype=_BF16, device=dev)
            dw2 = new((H, I), dtype=_BF16, device=dev)
        if m > self._fits[1]:
            self.workspace(m, True, x.device)
        rc = self.lib.moe_ffn_backward(
            self.handle, dout.data_ptr(), ldd, x.data_ptr(), ldx, saved.data_ptr(), m,
            dx.data_ptr() if need_dx else None, *((dw1.data_ptr(), dw3.data_ptr(), dw2.data_ptr()) if need_dw else
                                                  (None, None, None)), *self._ws_at, st)
        if rc:
            raise MoeError(rc, "moe_ffn_backward")
        past = self._past
        if m and (past.used is not self._ws or st not in past.streams or _capturing()):
            past.called(self._ws)
        return dx, dw1, dw3, dw2


# ---------------------------------------------------------------- operators around the layer and the block
# (include/moe_ffn_ops.h)

class NormOut(NamedTuple):
    """What moe_add_rmsnorm gives; None for what was not asked for."""
    out: torch.Tensor | None       # bf16 [m, h]
    residual: torch.Tensor | None  # bf16 [m, h]: x + residual, what the norm was taken of
    codes: torch.Tensor | None     # uint8 [m, h], e4m3
    scales: torch.Tensor | None    # fp32 [m, ceil(h / 128)]


def _device_of(t, what: str) -> int:
    """The device of a call by its first tensor: the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: a device tensor")
    if dev != _current_device():
        _on(t)
    return dev


def _strided(t, n: int, rows: int, what: str) -> int:
    """Checks a bf16 matrix [rows, n] on the current device as _rows does; returns its row stride.
    Called where the common case, dense rows on that device, does not hold."""
    ld = _rows(t, n, what)
    _need(t.shape[0] == rows, f"{what}: {rows} rows, got {t.shape[0]}")
    _on(t)
    return ld


def _bad(t, dtype, shape, what: str):
    """Words the refusal of a tensor that is not dense, of that type and shape and on the current device."""
    _dense(t, dtype, shape, what)
    _on(t)
    raise ValueError(what)  # not reached: one of these refuses it


def moe_add_rmsnorm(x, weight, eps=1e-6, residual=None, residual_out=None, out=None, bf16=True, fp8=False,
                    stream=None) -> NormOut:
    """RMSNorm of x (bf16 [m, h], rows may be strided), or of r = x + residual, times weight (fp32
    [h]): to bf16 (out; it may be x) and, with fp8, to e4m3 codes and scales per 128 columns, of the
    values before they are rounded to bf16.  r goes to residual_out (a new tensor unless given; it may
    be residual)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_add_rmsnorm(x, weight, eps, residual, residual_out, out, bf16, fp8)
    lib = _lib or load_library()
    if x.dim() != 2:
        raise ValueError("x: [m, h]")
    dev = _device_of(x, "x")
    shape = m, h = x.shape
    dense = x.is_contiguous() and x.dtype is _BF16 and x.get_device() == dev
    ldx = h if dense else _strided(x, h, m, "x")
    if not (weight.dtype is _F32 and weight.is_contiguous() and weight.shape == (h,) and weight.get_device() == dev):
        _bad(weight, _F32, (h,), "weight")
    ldr = ldo = 0
    res = res_out = to = codes_at = scales_at = codes = scales = None
    if residual is not None:
        ldr = h
        if not (residual.shape == shape and residual.is_contiguous() and residual.dtype is _BF16
                and residual.get_device() == dev):
            ldr = _strided(residual, h, m, "residual")
        res = residual.data_ptr()
        if residual_out is None:
            residual_out = _empty_like(x, memory_format=_dense_rows)
            ldo = h
        else:
            ldo = _strided(residual_out, h, m, "residual_out")
        res_out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if out is not None:
        _need(bf16, "out: given, and bf16 not asked for")
        _dense(out, _BF16, (m, h), "out")
        _on(out)
        to = out.data_ptr()
    elif bf16:
        out = _empty_like(x, memory_format=_dense_rows)
        to = out.data_ptr()
    elif not fp8:
        raise ValueError("neither bf16 nor fp8 is asked for")
    if fp8:
        codes = _empty((m, h), dtype=_U8, device=x.device)
        scales = _empty((m, (h + 127) // 128), dtype=_F32, device=x.device)
        codes_at, scales_at = codes.data_ptr(), scales.data_ptr()
    rc = lib.moe_add_rmsnorm(x.data_ptr(), ldx, res, ldr, m, h, weight.data_ptr(), eps, res_out, ldo, to, codes_at,
                             scales_at, _raw_stream(dev))
    if rc:
        raise MoeError(rc, "moe_add_rmsnorm")
    return NormOut(out, residual_out, codes, scales)


_grad_space = {}  # (m, h) -> moe_add_rmsnorm_backward_workspace_size


def moe_add_rmsnorm_backward(dout, r, weight, eps=1e-6, dresidual=None, need_dw=True, stream=None):
    """Gradients (dx bf16 [m, h], dweight fp32 [h]) of moe_add_rmsnorm's out, given the r that it
    normalised (its residual, or x where there was none); dx is the gradient of x and of the residual
    alike, dresidual (bf16) what else flows into r.  dweight is None where not needed, zero of no rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_add_rmsnorm_backward(dout, r, weight, eps, dresidual, need_dw)
    lib = _lib or load_library()
    if r.dim() != 2:
        raise ValueError("r: [m, h]")
    dev = _device_of(r, "r")
    shape = m, h = r.shape
    ldr = h if r.is_contiguous() and r.dtype is _BF16 and r.get_device() == dev else _strided(r, h, m, "r")
    ldd = h
    if not (dout.shape == shape and dout.is_contiguous() and dout.dtype is _BF16 and dout.get_device() == dev):
        ldd = _strided(dout, h, m, "dout")
    if not (weight.dtype is _F32 and weight.is_contiguous() and weight.shape == (h,) and weight.get_device() == dev):
        _bad(weight, _F32, (h,), "weight")
    ldq, dres = 0, None
    if dresidual is not None:
        ldq = h
        if not (dresidual.shape == shape and dresidual.is_contiguous() and dresidual.dtype is _BF16
                and dresidual.get_device() == dev):
            ldq = _strided(dresidual, h, m, "dresidual")
        dres = dresidual.data_ptr()
    dx = _empty_like(r, memory_format=_dense_rows)
    st = _raw_stream(dev)
    if not need_dw:
        rc = lib.moe_add_rmsnorm_backward(dout.data_ptr(), ldd, r.data_ptr(), ldr, m, h, weight.data_ptr(), eps, dres,
                                          ldq, dx.data_ptr(), None, None, 0, st)
        if rc:
            raise MoeError(rc, "moe_add_rmsnorm_backward")
        return dx, None
    dw = _empty_like(weight) if m else torch.zeros_like(weight)
    need = _grad_space.get((m, h))
    if need is None:
        size = ctypes.c_size_t()
        rc = lib.moe_add_rmsnorm_backward_workspace_size(m, h, size)
        if rc:
            raise MoeError(rc, "moe_add_rmsnorm_backward")
        if len(_grad_space) >= 1024:
            _grad_space.clear()
        need = _grad_space[m, h] = size.value
    with _spaces_lock:
        ws, _kept = _scratch(r, st, need)
        rc = lib.moe_add_rmsnorm_backward(dout.data_ptr(), ldd, r.data_ptr(), ldr, m, h, weight.data_ptr(), eps, dres,
                                          ldq, dx.data_ptr(), dw.data_ptr(), ws, need, st)
    if rc:
        raise MoeError(rc, "moe_add_rmsnorm_backward")
    return dx, dw


SCORINGS = {"softmax": MOE_SCORING_SOFTMAX, "sigmoid": MOE_SCORING_SIGMOID}
_I32 = torch.int32


def _router_args(logits, topk_ids, seq_offsets, scoring, dev: int):
    """Checks what the router's operators share; returns (m, E, k, sequences, their offsets' address, scoring)."""
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("logits: [m, E], topk_ids: [m, k]")
    m, E = logits.shape
    rows, k = topk_ids.shape
    if not (logits.dtype is _F32 and logits.is_contiguous() and logits.get_device() == dev):
        _bad(logits, _F32, (m, E), "logits")
    if not (topk_ids.dtype is _I32 and topk_ids.is_contiguous() and rows == m and topk_ids.get_device() == dev):
        _bad(topk_ids, _I32, (m, k), "topk_ids")
    if scoring not in SCORINGS:
        raise ValueError(f"scoring: one of {sorted(SCORINGS)}")
    if seq_offsets is None:
        return m, E, k, 1, None, SCORINGS[scoring]
    if not (seq_offsets.dtype is _I32 and seq_offsets.dim() == 1 and seq_offsets.is_contiguous()
            and seq_offsets.get_device() == dev and seq_offsets.shape[0] >= 2):
        _need(seq_offsets.dim() == 1 and seq_offsets.shape[0] >= 2, "seq_offsets: [sequences + 1], at least one sequence")
        _bad(seq_offsets, _I32, tuple(seq_offsets.shape), "seq_offsets")
    return m, E, k, seq_offsets.shape[0] - 1, seq_offsets.data_ptr(), SCORINGS[scoring]


def moe_balance_loss(logits, topk_ids, seq_offsets=None, scoring="softmax", stream=None):
    """(balance, z, counts) of a router's logits (fp32 [m, E]) and picks (int32 [m, k]), for each
    sequence of tokens seq_offsets[s] .. seq_offsets[s + 1] (int32 on the device, not falling; None:
    one sequence of all): balance and z fp32 [S], counts int32 [S, E].  Tokens in no sequence and ids
    outside [0, E) count nowhere."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_balance_loss(logits, topk_ids, seq_offsets, scoring)
    lib = _lib or load_library()
    dev = _device_of(logits, "logits")
    m, E, k, S, off, mode = _router_args(logits, topk_ids, seq_offsets, scoring, dev)
    on = logits.device
    new = _empty if m else torch.zeros
    balance = new((S,), dtype=_F32, device=on)  # two tensors: rows of one cost more than its allocation
    z = _empty_like(balance) if m else torch.zeros_like(balance)
    counts = new((S, E), dtype=_I32, device=on)
    # what moe_balance_loss_workspace_size returns
    need = (4 * S + 255) // 256 * 256 + (((m + 7) // 8 + S) * 8 + 255) // 256 * 256
    st = _raw_stream(dev)
    with _spaces_lock:
        ws, _kept = _scratch(logits, st, need)
        rc = lib.moe_balance_loss(logits.data_ptr(), topk_ids.data_ptr(), m, E, k, off, S, mode, balance.data_ptr(),
                                  z.data_ptr(), counts.data_ptr(), ws, need, st)
    if rc:
        raise MoeError(rc, "moe_balance_loss")
    return balance, z, counts


def moe_route_backward(logits, topk_ids, dtopk_w=None, dbalance=None, dz=None, counts=None, seq_offsets=None,
                       scoring="softmax", norm_topk_prob=True, routed_scaling=1.0, stream=None):
    """The gradient of a router's logits, fp32 [m, E]: through the routing weights (dtopk_w fp32
    [m, k]) and through moe_balance_loss's balance and z (dbalance, dz fp32 [S], with the counts
    that it gave and the same seq_offsets)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_route_backward(logits, topk_ids, dtopk_w, dbalance, dz, counts, seq_offsets, scoring,
                                      norm_topk_prob, routed_scaling)
    lib = _lib or load_library()
    dev = _device_of(logits, "logits")
    m, E, k, S, off, mode = _router_args(logits, topk_ids, seq_offsets, scoring, dev)
    w = c = b = z = None
    if dtopk_w is not None:
        if not (dtopk_w.dtype is _F32 and dtopk_w.is_contiguous() and dtopk_w.shape == (m, k) and dtopk_w.get_device() == dev):
            _bad(dtopk_w, _F32, (m, k), "dtopk_w")
        w = dtopk_w.data_ptr()
    if dbalance is not None:
        if counts is None:
            raise ValueError("dbalance without counts")
        if not (dbalance.dtype is _F32 and dbalance.is_contiguous() and dbalance.shape == (S,) and dbalance.get_device() == dev):
            _bad(dbalance, _F32, (S,), "dbalance")
        b = dbalance.data_ptr()
    if dz is not None:
        if not (dz.dtype is _F32 and dz.is_contiguous() and dz.shape == (S,) and dz.get_device() == dev):
            _bad(dz, _F32, (S,), "dz")
        z = dz.data_ptr()
    if counts is not None:
        if not (counts.dtype is _I32 and counts.is_contiguous() and counts.shape == (S, E) and counts.get_device() == dev):
            _bad(counts, _I32, (S, E), "counts")
        c = counts.data_ptr()
    d = _empty_like(logits, memory_format=_dense_rows)
    rc = lib.moe_route_backward(logits.data_ptr(), topk_ids.data_ptr(), m, E, k, mode, 1 if norm_topk_prob else 0,
                                routed_scaling, w, off, S, c, b, z, d.data_ptr(), _raw_stream(dev))
    if rc:
        raise MoeError(rc, "moe_route_backward")
    return d


def _lora_args(y, x, a, b, ids, scale, out, dev: int):
    """Checks a call of moe_lora_add; returns its arguments up to out's stride, and out."""
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a: [n, r, k], b: [n, d, r]")
    n, r, k = a.shape
    d = b.shape[1]
    if not (a.dtype is _BF16 and a.is_contiguous() and a.get_device() == dev):
        _bad(a, _BF16, (n, r, k), "a")
    if not (b.dtype is _BF16 and b.is_contiguous() and b.shape == (n, d, r) and b.get_device() == dev):
        _bad(b, _BF16, (n, d, r), "b")
    m = x.shape[0] if x.dim() == 2 else -1
    ldx = k if x.is_contiguous() and x.dtype is _BF16 and x.shape == (m, k) and x.get_device() == dev else \
        _strided(x, k, m, "x")
    ldy = d
    if not (y.is_contiguous() and y.dtype is _BF16 and y.shape == (m, d) and y.get_device() == dev):
        ldy = _strided(y, d, m, "y")
    if not (ids.dtype is _I32 and ids.is_contiguous() and ids.shape == (m,) and ids.get_device() == dev):
        _bad(ids, _I32, (m,), "ids")
    s = None
    if scale is not None:
        if not (scale.dtype is _F32 and scale.is_contiguous() and scale.shape == (n,) and scale.get_device() == dev):
            _bad(scale, _F32, (n,), "scale")
        s = scale.data_ptr()
    if out is None:
        out, ldo = y, ldy
    else:
        ldo = d
        if not (out.is_contiguous() and out.dtype is _BF16 and out.shape == (m, d) and out.get_device() == dev):
            ldo = _strided(out, d, m, "out")
    return out, (x.data_ptr(), ldx, m, k, y.data_ptr(), ldy, d, a.data_ptr(), b.data_ptr(), n, r, ids.data_ptr(), s,
                 out.data_ptr(), ldo)


def _lora_launch(x, args, dev: int):
    """Launches what _lora_args has checked, on the current stream."""
    lib = _lib or load_library()
    need = 256
    if args[2] > MOE_LORA_BY_TOKEN:
        size = ctypes.c_size_t()
        rc = lib.moe_lora_add_workspace_size(args[2], args[3], args[10], size)
        if rc:
            raise MoeError(rc, "moe_lora_add")
        need = size.value
    st = _raw_stream(dev)
    with _spaces_lock:
        ws = _space(x, st, need)
        rc = lib.moe_lora_add(*args, ws.data_ptr(), ws.numel(), st)
    if rc:
        raise MoeError(rc, "moe_lora_add")


def moe_lora_add(y, x, a, b, ids, scale=None, out=None, stream=None):
    """y (bf16 [m, d], a projection's output for x, bf16 [m, k]; rows may be strided) plus each token's
    low-rank adapter: scale[i] b[i] (a[i] x[t]), i = ids[t] (int32 [m]; -1: none), a bf16 [n, r, k],
    b bf16 [n, d, r], scale fp32 [n] (None: 1).  Into y unless out is given.  Ids outside [-1, n) count
    as -1 and set the error word that mxfp4_device_status reads."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_lora_add(y, x, a, b, ids, scale, out)
    dev = _device_of(x, "x")
    out, args = _lora_args(y, x, a, b, ids, scale, out, dev)
    _lora_launch(x, args, dev)
    return out
