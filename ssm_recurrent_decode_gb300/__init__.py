"""Python binding of libgdn_decode.so, the GB300 (sm_103a) single-token gated delta-rule decode.

Argument marshalling only: every function here takes torch tensors that already live on the GPU,
passes their device pointers, sizes and strides through the C ABI declared in
``include/gdn_decode.h``, and launches on the current torch stream. Every step of the decode runs
in the library's CUDA kernels; there is no Python, PyTorch or CPU fallback, and a missing or
unbuildable library raises.

Entry points (same names as the C ABI):
  gdn_decode_step          row b on state slot b
  gdn_decode_step_indexed  row b on state slot cache_indices[b] (the packed decode over a pool)
  gdn_decode_buffered      output-only decode that writes the state back once every L steps
  gdn_decode_fused         conv1d update -> delta step (per-key or per-head decay) -> gated RMSNorm
  mamba_selective_scan_decode  the Mamba-1 selective-scan decode step (a diagonal recurrence)
  mamba_selective_scan     the same recurrence over whole sequences (prompts), packed end to end
  mamba_selective_scan_backward  its gradients
  gdn_beam_select          the best K of beams x vocabulary by cumulative log-probability
  gdn_beam_reorder         the chosen beams' states, moved within their slot pools
  gdn_linear_attention     linear attention with a decay for each head over whole sequences (prompts)
  gdn_linear_attention_backward  its gradients
  gdn_linear_attention_step  its single-token step over a pool of states
  gdn_rotary               rotary positions of q and k
plus ``fused_recurrent_gated_delta_rule_packed_decode``, the packed call with the keyword names
of "Microbenchmark: buffered output-only GDN decode (ReplaySSM Part A)" (_bench_cfg, run_packed).
"""
from __future__ import annotations

import contextlib
import ctypes
import threading

from . import _build

__all__ = [
    "lib", "build", "GdnError", "GdnStepArgs", "GdnRingArgs", "GdnFusedArgs",
    "gdn_decode_step", "gdn_decode_step_indexed", "gdn_decode_buffered", "gdn_decode_fused",
    "gdn_strerror", "split_mixed_qkv", "fused_recurrent_gated_delta_rule_packed_decode", "PreparedCall",
    "MambaArgs", "mamba_selective_scan_decode", "gdn_selftest_bounded_wait",
    "MambaScanArgs", "MambaScanGradArgs", "mamba_selective_scan", "mamba_selective_scan_backward",
    "mamba_scan_workspace",
    "BeamSelectArgs", "BeamPool", "BeamReorderArgs", "gdn_beam_select", "beam_select_workspace",
    "gdn_beam_reorder",
    "LinearArgs", "LinearGradArgs", "LinearStepArgs", "RotaryArgs", "gdn_linear_attention",
    "gdn_linear_attention_backward", "gdn_linear_attention_step", "linear_attention_workspace", "gdn_rotary",
    "rotary_frequencies",
    "GemvArgs", "gdn_gemv_bf16", "gemv_workspace",
    "GDN_F32", "GDN_BF16", "GDN_DEVERR_BAD_INDEX", "GDN_DEVERR_BAD_WRITE_POS", "GDN_DEVERR_TIMEOUT",
    "GDN_DEVERR_RANGE", "debug_lib", "using_debug_build",
    "EXPORTS",
]

GDN_F32, GDN_BF16 = 0, 1
GDN_GATE_RAW, GDN_GATE_DIRECT = 0, 1
GDN_FUSED_GATE_KDA, GDN_FUSED_GATE_GDN = 0, 1
GDN_ACT_SILU, GDN_ACT_SIGMOID = 0, 1
GDN_DEVERR_BAD_INDEX, GDN_DEVERR_BAD_WRITE_POS, GDN_DEVERR_TIMEOUT = 0x1, 0x2, 0x4
GDN_DEVERR_RANGE = 0x8
GDN_KERNEL = {"auto": 0, "tile": 1, "pipe": 2, "stage": 3}
ABI_VERSION = 9

# every function the header declares
EXPORTS = ("gdn_decode_step", "gdn_decode_step_indexed", "gdn_decode_buffered", "gdn_decode_fused",
           "gdn_strerror", "gdn_abi_struct_size", "gdn_abi_version", "mamba_selective_scan_decode",
           "gdn_selftest_bounded_wait", "gdn_gemv_bf16", "gdn_gemv_default_splits",
           "gdn_gemv_workspace_bytes", "gdn_gemv_bf16_noalloc", "gdn_decode_front",
           "gdn_front_proj_width", "gdn_gemv_set_wait_limit", "gdn_decode_step_indexed_chained",
           "mamba_selective_scan", "mamba_selective_scan_backward", "mamba_scan_workspace_bytes",
           "gdn_beam_select", "gdn_beam_select_workspace_bytes", "gdn_beam_reorder",
           "gdn_linear_attention", "gdn_linear_attention_backward", "gdn_linear_attention_step",
           "gdn_linear_workspace_bytes", "gdn_linear_set_wait_limit", "gdn_rotary")

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class GdnStepArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32),
                ("num_slots", _i32), ("in_dtype", _i32), ("out_dtype", _i32),
                ("q", _vp), ("k", _vp), ("v", _vp),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("gate_mode", _i32), ("a", _vp), ("b", _vp), ("A_log", _vp), ("dt_bias", _vp),
                ("g", _vp), ("beta", _vp), ("scale", _f32), ("use_qk_l2norm", _i32),
                ("state", _vp), ("out", _vp), ("err_flags", _vp), ("state_dtype", _i32)]


class GdnRingArgs(ctypes.Structure):
    _fields_ = [("L", _i32), ("ring_dtype", _i32), ("d_cache", _vp), ("k_cache", _vp),
                ("g_cache", _vp), ("write_pos", _vp), ("kernel", _i32)]


class GdnFusedArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("heads", _i32), ("head_dim", _i32), ("num_slots", _i32),
                ("x", _vp), ("x_stride", _i64), ("conv_w", _vp), ("conv_b", _vp),
                ("conv_state", _vp), ("cs_stride_slot", _i64), ("cs_stride_chan", _i64),
                ("cs_stride_tap", _i64), ("gate_kind", _i32), ("kda_gate_form", _i32),
                ("raw_g", _vp), ("raw_beta", _vp), ("A_log", _vp), ("dt_bias", _vp),
                ("lower_bound", _f32), ("scale", _f32), ("use_qk_l2norm", _i32),
                ("state", _vp), ("state_indices", _vp), ("pad_slot_id", _i32),
                ("out_gate", _vp), ("norm_w", _vp), ("norm_eps", _f32), ("gate_act", _i32),
                ("out", _vp), ("err_flags", _vp), ("kernel", _i32), ("raw_g_stride", _i64),
                ("raw_beta_stride", _i64), ("out_gate_stride", _i64)]


class GdnFrontArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("hidden", _i32), ("x", _vp), ("x_stride", _i64), ("W_in", _vp),
                ("W_out", _vp), ("z", _vp), ("o", _vp), ("y", _vp), ("y_dtype", _i32),
                ("y_stride", _i64), ("in_splits", _i32), ("out_splits", _i32), ("core", GdnFusedArgs)]


class MambaArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("D", _i32), ("N", _i32), ("in_dtype", _i32), ("out_dtype", _i32),
                ("x", _vp), ("dt", _vp), ("A", _vp), ("Bm", _vp), ("Cm", _vp), ("Dskip", _vp),
                ("z", _vp), ("h", _vp), ("h_out", _vp), ("y", _vp), ("err_flags", _vp)]


class MambaScanArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("S", _i32), ("D", _i32), ("N", _i32), ("in_dtype", _i32), ("out_dtype", _i32),
                ("x", _vp), ("x_stride", _i64), ("dt", _vp), ("dt_stride", _i64), ("A", _vp),
                ("Bm", _vp), ("B_stride", _i64), ("Cm", _vp), ("C_stride", _i64), ("Dskip", _vp),
                ("z", _vp), ("z_stride", _i64), ("cu_seqlens", _vp), ("state_indices", _vp),
                ("num_states", _i32), ("h0", _vp), ("h_last", _vp), ("y", _vp), ("y_stride", _i64),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("err_flags", _vp)]


class MambaScanGradArgs(ctypes.Structure):
    _fields_ = [("s", MambaScanArgs), ("dy", _vp), ("dy_stride", _i64), ("dh_last", _vp),
                ("dx", _vp), ("dx_stride", _i64), ("ddt", _vp), ("ddt_stride", _i64),
                ("dz", _vp), ("dz_stride", _i64), ("dBm", _vp), ("dB_stride", _i64),
                ("dCm", _vp), ("dC_stride", _i64), ("dA", _vp), ("dDskip", _vp), ("dh0", _vp)]


class GemvArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("N", _i32), ("Kd", _i32), ("out_dtype", _i32), ("x", _vp),
                ("x_stride", _i64), ("W", _vp), ("y", _vp), ("y_stride", _i64), ("splits", _i32),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("err_flags", _vp)]


class BeamSelectArgs(ctypes.Structure):
    _fields_ = [("batch", _i32), ("beams", _i32), ("vocab", _i32), ("K", _i32), ("logits_dtype", _i32),
                ("num_rows", _i32), ("logits", _vp), ("row_stride", _i64), ("rows", _vp), ("scores", _vp),
                ("finished", _vp), ("eos_token", _i32), ("out_scores", _vp), ("out_parents", _vp),
                ("out_tokens", _vp), ("out_finished", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("err_flags", _vp)]


class BeamPool(ctypes.Structure):
    _fields_ = [("base", _vp), ("slot_stride", _i64), ("slot_bytes", _i64)]


class BeamReorderArgs(ctypes.Structure):
    _fields_ = [("batch", _i32), ("beams", _i32), ("num_slots", _i32), ("num_pools", _i32),
                ("pools", ctypes.POINTER(BeamPool)), ("slots", _vp), ("parents", _vp), ("new_slots", _vp),
                ("err_flags", _vp)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("S", _i32), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32),
                ("in_dtype", _i32), ("out_dtype", _i32),
                ("q", _vp), ("q_stride", _i64), ("q_head_stride", _i64),
                ("k", _vp), ("k_stride", _i64), ("k_head_stride", _i64),
                ("v", _vp), ("v_stride", _i64), ("v_head_stride", _i64),
                ("g", _vp), ("g_stride", _i64), ("scale", _f32), ("cu_seqlens", _vp), ("state_indices", _vp),
                ("num_states", _i32), ("initial_state", _vp), ("final_state", _vp),
                ("o", _vp), ("o_stride", _i64), ("o_head_stride", _i64),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("err_flags", _vp)]


class LinearGradArgs(ctypes.Structure):
    _fields_ = [("s", LinearArgs), ("d_o", _vp), ("do_stride", _i64), ("do_head_stride", _i64), ("d_final_state", _vp),
                ("dq", _vp), ("dq_stride", _i64), ("dq_head_stride", _i64),
                ("dk", _vp), ("dk_stride", _i64), ("dk_head_stride", _i64),
                ("dv", _vp), ("dv_stride", _i64), ("dv_head_stride", _i64),
                ("dg", _vp), ("dg_stride", _i64), ("d_initial_state", _vp)]


class LinearStepArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32), ("num_slots", _i32),
                ("in_dtype", _i32), ("out_dtype", _i32), ("state_dtype", _i32),
                ("q", _vp), ("q_stride", _i64), ("q_head_stride", _i64),
                ("k", _vp), ("k_stride", _i64), ("k_head_stride", _i64),
                ("v", _vp), ("v_stride", _i64), ("v_head_stride", _i64),
                ("g", _vp), ("g_stride", _i64), ("scale", _f32), ("rotary_dim", _i32), ("interleaved", _i32),
                ("positions", _vp), ("frequencies", _vp), ("magnitude", _f32), ("state", _vp), ("out", _vp),
                ("err_flags", _vp)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("HK", _i32), ("D", _i32), ("rotary_dim", _i32), ("interleaved", _i32),
                ("inverse", _i32), ("dtype", _i32), ("magnitude", _f32), ("positions", _vp), ("frequencies", _vp),
                ("q", _vp), ("q_stride", _i64), ("q_head_stride", _i64),
                ("q_out", _vp), ("q_out_stride", _i64), ("q_out_head_stride", _i64),
                ("k", _vp), ("k_stride", _i64), ("k_head_stride", _i64),
                ("k_out", _vp), ("k_out_stride", _i64), ("k_out_head_stride", _i64)]


class GdnError(RuntimeError):
    """A non-zero status from the library (the message is gdn_strerror's)."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {gdn_strerror(status)} (status {status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile libgdn_decode.so in-tree (nvcc, sm_103a); returns its path."""
    return _build.build(force=force)


def _load(path: str):
    """Open one build of the library and declare its entry points' signatures."""
    L = ctypes.CDLL(path)
    for name in ("gdn_decode_step",):
        getattr(L, name).argtypes = [ctypes.POINTER(GdnStepArgs), _vp]
    L.gdn_decode_step_indexed.argtypes = [ctypes.POINTER(GdnStepArgs), _vp, _i32, _vp]
    L.gdn_decode_step_indexed_chained.argtypes = [ctypes.POINTER(GdnStepArgs), _vp, _i32, _vp]
    L.gdn_decode_buffered.argtypes = [ctypes.POINTER(GdnStepArgs), _vp, _i32,
                                      ctypes.POINTER(GdnRingArgs), _vp]
    L.gdn_decode_fused.argtypes = [ctypes.POINTER(GdnFusedArgs), _vp]
    L.mamba_selective_scan_decode.argtypes = [ctypes.POINTER(MambaArgs), _vp]
    L.mamba_selective_scan_decode.restype = ctypes.c_int
    L.mamba_selective_scan.argtypes = [ctypes.POINTER(MambaScanArgs), _vp]
    L.mamba_selective_scan.restype = ctypes.c_int
    L.mamba_selective_scan_backward.argtypes = [ctypes.POINTER(MambaScanGradArgs), _vp]
    L.mamba_selective_scan_backward.restype = ctypes.c_int
    L.mamba_scan_workspace_bytes.argtypes = [_i32] * 6
    L.mamba_scan_workspace_bytes.restype = ctypes.c_size_t
    L.gdn_beam_select.argtypes = [ctypes.POINTER(BeamSelectArgs), _vp]
    L.gdn_beam_select.restype = ctypes.c_int
    L.gdn_beam_select_workspace_bytes.argtypes = [_i32] * 4
    L.gdn_beam_select_workspace_bytes.restype = ctypes.c_size_t
    L.gdn_beam_reorder.argtypes = [ctypes.POINTER(BeamReorderArgs), _vp]
    L.gdn_beam_reorder.restype = ctypes.c_int
    L.gdn_linear_attention.argtypes = [ctypes.POINTER(LinearArgs), _vp]
    L.gdn_linear_attention.restype = ctypes.c_int
    L.gdn_linear_attention_backward.argtypes = [ctypes.POINTER(LinearGradArgs), _vp]
    L.gdn_linear_attention_backward.restype = ctypes.c_int
    L.gdn_linear_attention_step.argtypes = [ctypes.POINTER(LinearStepArgs), _vp, _i32, _vp]
    L.gdn_linear_attention_step.restype = ctypes.c_int
    L.gdn_linear_workspace_bytes.argtypes = [_i32] * 9
    L.gdn_linear_workspace_bytes.restype = ctypes.c_size_t
    L.gdn_linear_set_wait_limit.argtypes = [_i64]
    L.gdn_linear_set_wait_limit.restype = _i64
    L.gdn_rotary.argtypes = [ctypes.POINTER(RotaryArgs), _vp]
    L.gdn_rotary.restype = ctypes.c_int
    L.gdn_selftest_bounded_wait.argtypes = [_vp, _i64, _i32, _vp]
    L.gdn_decode_front.argtypes = [ctypes.POINTER(GdnFrontArgs), _vp]
    L.gdn_decode_front.restype = ctypes.c_int
    L.gdn_front_proj_width.argtypes = [_i32, _i32, _i32]
    L.gdn_front_proj_width.restype = _i64
    L.gdn_gemv_bf16.argtypes = [ctypes.POINTER(GemvArgs), _vp]
    L.gdn_gemv_bf16.restype = ctypes.c_int
    L.gdn_gemv_default_splits.argtypes = [_i32, _i32, _i32]
    L.gdn_gemv_default_splits.restype = _i32
    L.gdn_gemv_workspace_bytes.argtypes = [_i32, _i32, _i32]
    L.gdn_gemv_workspace_bytes.restype = ctypes.c_size_t
    L.gdn_gemv_bf16_noalloc.argtypes = [ctypes.POINTER(GemvArgs), _vp]
    L.gdn_gemv_bf16_noalloc.restype = ctypes.c_int
    L.gdn_gemv_set_wait_limit.argtypes = [_i64]
    L.gdn_gemv_set_wait_limit.restype = _i64
    L.gdn_selftest_bounded_wait.restype = ctypes.c_int
    for name in ("gdn_decode_step", "gdn_decode_step_indexed", "gdn_decode_buffered",
                 "gdn_decode_fused", "gdn_abi_version", "gdn_decode_step_indexed_chained"):
        getattr(L, name).restype = ctypes.c_int
    L.gdn_strerror.argtypes = [ctypes.c_int]
    L.gdn_strerror.restype = ctypes.c_char_p
    L.gdn_abi_struct_size.argtypes = [ctypes.c_int]
    L.gdn_abi_struct_size.restype = ctypes.c_size_t
    sizes = [L.gdn_abi_struct_size(i) for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 12, 13, 14, 15)]
    want = [ctypes.sizeof(c) for c in (GdnStepArgs, GdnRingArgs, GdnFusedArgs, GemvArgs, GdnFrontArgs, MambaArgs,
                                       MambaScanArgs, MambaScanGradArgs, BeamSelectArgs, BeamReorderArgs, BeamPool,
                                       LinearArgs, LinearGradArgs, LinearStepArgs, RotaryArgs)]
    if sizes != want or L.gdn_abi_version() != ABI_VERSION:
        raise RuntimeError(f"libgdn_decode.so ABI mismatch: struct sizes {sizes} vs {want}")
    return L


def lib():
    """The loaded library (built first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _load(_build.build())
    return _lib


_debug_lib = None


@contextlib.contextmanager
def using_debug_build():
    """Inside the with-block every entry point of this module calls the index-checking debug
    build (debug_lib) instead of the release library; prepared calls keep the library they were
    made with. For tests."""
    global _lib
    L = debug_lib()
    prev = lib()
    with _lock:
        _lib = L
    try:
        yield L
    finally:
        with _lock:
            _lib = prev


def debug_lib():
    """The index-checking debug build, libgdn_decode_debug.so (built first if needed): the same
    entry points, whose kernels report an out-of-range computed index through the error word
    (GDN_DEVERR_RANGE) instead of making the access. For tests; not for timing."""
    global _debug_lib
    with _lock:
        if _debug_lib is None:
            _debug_lib = _load(_build.build(debug=True))
    return _debug_lib


def gdn_strerror(status: int) -> str:
    return lib().gdn_strerror(int(status)).decode()


# ------------------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _ptr(t, name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _dense(t, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows(t, name: str, width: int):
    """A [B, width] or [B, heads, dim] view whose rows are dense: returns the row stride."""
    if t.dim() == 3:
        if t.stride(2) != 1 or t.stride(1) != t.shape[2] or t.shape[1] * t.shape[2] != width:
            raise ValueError(f"{name}: rows must be dense [heads, dim] of width {width}")
    elif t.dim() == 2:
        if t.stride(1) != 1 or t.shape[1] != width:
            raise ValueError(f"{name}: expected [B, {width}] with unit inner stride")
    else:
        raise ValueError(f"{name}: expected a 2-D or 3-D tensor")
    return t.stride(0)


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def split_mixed_qkv(mixed_qkv, H: int, HV: int, K: int, V: int):
    """Views q [B, H*K], k [B, H*K], v [B, HV*V] of a packed row [q | k | v] (no copy)."""
    hk = H * K
    return mixed_qkv[:, :hk], mixed_qkv[:, hk:2 * hk], mixed_qkv[:, 2 * hk:2 * hk + HV * V]


def _step_args(q, k, v, state, out, *, H, a, b, A_log, dt_bias, g, beta, scale, use_qk_l2norm,
               err_flags) -> GdnStepArgs:
    torch = _torch()
    if state.dim() != 4:
        raise ValueError("state must be [num_slots, HV, V, K]")
    _dense(state, "state")
    num_slots, HV, V, K = state.shape
    B = q.shape[0]
    if H is None:
        H = (q.shape[1] if q.dim() == 3 else q.shape[1] // K)
    _dense(out, "out")
    if out.numel() != B * HV * V:
        raise ValueError(f"out must hold B*HV*V = {B * HV * V} elements")
    s = GdnStepArgs()
    s.B, s.H, s.HV, s.K, s.V, s.num_slots = B, H, HV, K, V, num_slots
    s.in_dtype, s.out_dtype = _dtype_code(q), _dtype_code(out)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    s.q, s.k, s.v = _ptr(q, "q"), _ptr(k, "k"), _ptr(v, "v")
    s.q_stride, s.k_stride, s.v_stride = _rows(q, "q", H * K), _rows(k, "k", H * K), _rows(v, "v", HV * V)
    if g is not None or beta is not None:
        s.gate_mode = GDN_GATE_DIRECT
        s.g = _ptr(_dense(g, "g"), "g", torch.float32)
        s.beta = _ptr(_dense(beta, "beta"), "beta", torch.float32)
    else:
        s.gate_mode = GDN_GATE_RAW
        for t, n in ((a, "a"), (b, "b")):
            if t is None or t.dtype != q.dtype:
                raise TypeError(f"{n} must be given with the dtype of q")
        s.a, s.b = _ptr(_dense(a, "a"), "a"), _ptr(_dense(b, "b"), "b")
        s.A_log = _ptr(_dense(A_log, "A_log"), "A_log", torch.float32)
        s.dt_bias = _ptr(_dense(dt_bias, "dt_bias"), "dt_bias", torch.float32)
    s.scale = 0.0 if scale is None else float(scale)
    s.use_qk_l2norm = int(bool(use_qk_l2norm))
    s.state = _ptr(state, "state")
    s.state_dtype = _dtype_code(state)
    s.out = _ptr(out, "out")
    s.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    return s


def _check(fn: str, rc: int):
    if rc != 0:
        raise GdnError(fn, rc)


class PreparedCall:
    """A library call whose argument structs were built once (``prepare=True`` on an entry
    point). Calling it only launches, which takes a few microseconds of host time instead of
    re-marshalling every tensor; that matters for small batches, where the kernels take a few
    microseconds themselves. The tensors it was built from must stay alive with the same storage;
    each launch reads their current contents."""

    __slots__ = ("_name", "_fn", "_args", "_keep")

    def __init__(self, name, fn, args, keep):
        self._name, self._fn, self._args, self._keep = name, fn, args, keep

    def __call__(self, stream=None):
        _check(self._name, self._fn(*self._args, _stream(stream)))


def _run_or_prepare(name, args, keep, stream, prepare, result):
    fn = getattr(lib(), name)
    if prepare:
        return PreparedCall(name, fn, args, keep)
    _check(name, fn(*args, _stream(stream)))
    return result


# ------------------------------------------------------------------------------------------------
# entry points
# ------------------------------------------------------------------------------------------------
def gdn_decode_step(q, k, v, state, out, *, H=None, a=None, b=None, A_log=None, dt_bias=None,
                    g=None, beta=None, scale=None, use_qk_l2norm=True, err_flags=None, stream=None,
                    prepare=False):
    """One decode step, row b on slot b. q, k: [B, H*K] (or [B, H, K]) row views; v: [B, HV*V];
    gates either raw (a, b [B, HV] in the dtype of q; A_log, dt_bias [HV] fp32) or direct
    (g, beta [B, HV] fp32); state [num_slots, HV, V, K] fp32 (or bf16: stored in bf16, computed in
    fp32) updated in place; out [B, HV, V] (or [B, 1, HV, V]) fp32 or bf16.
    prepare=True returns a PreparedCall instead of launching (every entry point takes it)."""
    s = _step_args(q, k, v, state, out, H=H, a=a, b=b, A_log=A_log, dt_bias=dt_bias, g=g,
                   beta=beta, scale=scale, use_qk_l2norm=use_qk_l2norm, err_flags=err_flags)
    return _run_or_prepare("gdn_decode_step", (ctypes.byref(s),), (s,), stream, prepare, out)


def gdn_decode_step_indexed(q, k, v, state, out, cache_indices, *, pad_slot_id=-1, H=None, a=None,
                            b=None, A_log=None, dt_bias=None, g=None, beta=None, scale=None,
                            use_qk_l2norm=True, err_flags=None, chained=False, stream=None,
                            prepare=False):
    """As gdn_decode_step, with row b on slot cache_indices[b] (int32 [B] on the device); rows
    whose index is pad_slot_id are skipped (state untouched, out zeroed). chained=True calls
    gdn_decode_step_indexed_chained (a layer of a multi-layer decode: the launch may overlap the
    kernel before it on the stream, which must not write this call's state or cache_indices)."""
    torch = _torch()
    s = _step_args(q, k, v, state, out, H=H, a=a, b=b, A_log=A_log, dt_bias=dt_bias, g=g,
                   beta=beta, scale=scale, use_qk_l2norm=use_qk_l2norm, err_flags=err_flags)
    idx = _ptr(_dense(cache_indices, "cache_indices"), "cache_indices", torch.int32)
    return _run_or_prepare("gdn_decode_step_indexed_chained" if chained else "gdn_decode_step_indexed",
                           (ctypes.byref(s), ctypes.c_void_p(idx), ctypes.c_int32(int(pad_slot_id))),
                           (s,), stream, prepare, out)


def gdn_decode_buffered(q, k, v, state, out, d_cache, k_cache, g_cache, write_pos, *,
                        cache_indices=None, pad_slot_id=-1, H=None, a=None, b=None, A_log=None,
                        dt_bias=None, g=None, beta=None, scale=None, use_qk_l2norm=True,
                        err_flags=None, kernel="auto", stream=None, prepare=False):
    """Buffered output-only decode. state holds the checkpoints; d_cache [num_slots, HV, L, V],
    k_cache [num_slots, H, L, K] (both fp32 or both bf16), g_cache [num_slots, HV, L] fp32;
    write_pos int32 [B] is read, never advanced (the caller moves it to (p+1) % L).
    kernel: "auto" (the persistent pipelined kernel when K == V == 128, rows are 16-byte aligned
    and L > 1, else the per-tile kernel), "tile", "pipe" or "stage" (one CTA per tile staged in
    shared memory) to force one."""
    torch = _torch()
    s = _step_args(q, k, v, state, out, H=H, a=a, b=b, A_log=A_log, dt_bias=dt_bias, g=g,
                   beta=beta, scale=scale, use_qk_l2norm=use_qk_l2norm, err_flags=err_flags)
    r = GdnRingArgs()
    r.L = d_cache.shape[2]
    if k_cache.dtype != d_cache.dtype:
        raise TypeError("d_cache and k_cache must share one dtype")
    r.ring_dtype = _dtype_code(d_cache)
    expect = {"d_cache": (s.num_slots, s.HV, r.L, s.V), "k_cache": (s.num_slots, s.H, r.L, s.K),
              "g_cache": (s.num_slots, s.HV, r.L)}
    for name, t in (("d_cache", d_cache), ("k_cache", k_cache), ("g_cache", g_cache)):
        if tuple(t.shape) != expect[name]:
            raise ValueError(f"{name} must be {expect[name]}, got {tuple(t.shape)}")
        _dense(t, name)
    r.d_cache, r.k_cache = _ptr(d_cache, "d_cache"), _ptr(k_cache, "k_cache")
    r.g_cache = _ptr(g_cache, "g_cache", torch.float32)
    r.write_pos = _ptr(_dense(write_pos, "write_pos"), "write_pos", torch.int32)
    r.kernel = GDN_KERNEL[kernel]
    idx = None if cache_indices is None else _ptr(_dense(cache_indices, "cache_indices"),
                                                  "cache_indices", torch.int32)
    return _run_or_prepare("gdn_decode_buffered",
                           (ctypes.byref(s), ctypes.c_void_p(idx), ctypes.c_int32(int(pad_slot_id)),
                            ctypes.byref(r)), (s, r), stream, prepare, out)


def _fused_core(conv_w, conv_state, A_log, dt_bias, state, state_indices, norm_w, *, conv_b,
                pad_slot_id, gate_kind, kda_gate_form, lower_bound, scale, use_qk_l2norm, norm_eps,
                gate_act, err_flags, kernel):
    """The arguments of gdn_decode_fused that do not depend on the per-token inputs."""
    torch = _torch()
    _dense(state, "state")
    num_slots, heads, D, _ = state.shape
    f = GdnFusedArgs()
    f.heads, f.head_dim, f.num_slots = heads, D, num_slots
    f.conv_w = _ptr(_dense(conv_w, "conv_w"), "conv_w", torch.float32)
    f.conv_b = _ptr(conv_b, "conv_b", torch.float32)
    if tuple(conv_state.shape) != (num_slots, 3 * heads * D, 3):
        raise ValueError("conv_state must have logical shape [num_slots, 3*dim, 3]")
    f.conv_state = _ptr(conv_state, "conv_state", torch.bfloat16)
    f.cs_stride_slot, f.cs_stride_chan, f.cs_stride_tap = conv_state.stride()
    f.gate_kind = {"kda": GDN_FUSED_GATE_KDA, "gdn": GDN_FUSED_GATE_GDN}[gate_kind]
    f.kda_gate_form = int(kda_gate_form)
    f.A_log = _ptr(_dense(A_log, "A_log"), "A_log", torch.float32)
    f.dt_bias = _ptr(_dense(dt_bias, "dt_bias"), "dt_bias", torch.float32)
    f.lower_bound = float(lower_bound)
    f.scale = 0.0 if scale is None else float(scale)
    f.use_qk_l2norm = int(bool(use_qk_l2norm))
    f.state = _ptr(state, "state", torch.float32)
    f.state_indices = _ptr(_dense(state_indices, "state_indices"), "state_indices", torch.int32)
    f.pad_slot_id = int(pad_slot_id)
    f.norm_w = _ptr(_dense(norm_w, "norm_w"), "norm_w", torch.float32)
    f.norm_eps = float(norm_eps)
    f.gate_act = {"silu": GDN_ACT_SILU, "sigmoid": GDN_ACT_SIGMOID}[gate_act]
    f.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    f.kernel = GDN_KERNEL[kernel]
    return f


def front_proj_width(heads, head_dim, gate_kind="gdn"):
    """P, the width of the front's input projection output z (see gdn_decode_front)."""
    code = {"kda": GDN_FUSED_GATE_KDA, "gdn": GDN_FUSED_GATE_GDN}[gate_kind]
    return int(lib().gdn_front_proj_width(int(heads), int(head_dim), code))


def gdn_decode_front(x, W_in, W_out, z, o, y, conv_w, conv_state, A_log, dt_bias, state,
                     state_indices, norm_w, *, conv_b=None, pad_slot_id=0, gate_kind="gdn",
                     kda_gate_form=0, lower_bound=-5.0, scale=None, use_qk_l2norm=True,
                     norm_eps=1e-5, gate_act="silu", in_splits=0, out_splits=0, err_flags=None,
                     kernel="auto", stream=None, prepare=False):
    """One DeltaNet layer's decode forward (declared in include/gdn_front.h): z = x W_in^T (bf16
    z [T, P], columns q|k|v, out_gate, raw_g, raw_beta), o = conv -> step -> gated RMSNorm on views
    of z, y = o W_out^T. x bf16 [T, hidden] (row view allowed); W_in bf16 [P, hidden]; W_out bf16
    [hidden, dim]; z, o dense bf16 scratch [T, P], [T, dim]; y fp32 or bf16 [T, hidden]; the rest
    as for gdn_decode_fused."""
    torch = _torch()
    T, hidden = x.shape
    c = _fused_core(conv_w, conv_state, A_log, dt_bias, state, state_indices, norm_w,
                    conv_b=conv_b, pad_slot_id=pad_slot_id, gate_kind=gate_kind,
                    kda_gate_form=kda_gate_form, lower_bound=lower_bound, scale=scale,
                    use_qk_l2norm=use_qk_l2norm, norm_eps=norm_eps, gate_act=gate_act,
                    err_flags=err_flags, kernel=kernel)
    P = front_proj_width(c.heads, c.head_dim, gate_kind)
    dim = c.heads * c.head_dim
    if tuple(W_in.shape) != (P, hidden) or tuple(W_out.shape) != (hidden, dim):
        raise ValueError(f"expected W_in [{P}, {hidden}] and W_out [{hidden}, {dim}]")
    if tuple(z.shape) != (T, P) or tuple(o.shape) != (T, dim) or tuple(y.shape) != (T, hidden):
        raise ValueError(f"expected z [{T}, {P}], o [{T}, {dim}], y [{T}, {hidden}]")
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("x and y need unit inner stride")
    a = GdnFrontArgs()
    a.T, a.hidden = T, hidden
    a.x, a.x_stride = _ptr(x, "x", torch.bfloat16), x.stride(0)
    a.W_in = _ptr(_dense(W_in, "W_in"), "W_in", torch.bfloat16)
    a.W_out = _ptr(_dense(W_out, "W_out"), "W_out", torch.bfloat16)
    a.z = _ptr(_dense(z, "z"), "z", torch.bfloat16)
    a.o = _ptr(_dense(o, "o"), "o", torch.bfloat16)
    a.y, a.y_dtype, a.y_stride = _ptr(y, "y"), _dtype_code(y), y.stride(0)
    a.in_splits, a.out_splits = int(in_splits), int(out_splits)
    a.core = c
    return _run_or_prepare("gdn_decode_front", (ctypes.byref(a),), (a,), stream, prepare, y)


def gdn_decode_fused(x, conv_w, conv_state, raw_g, raw_beta, A_log, dt_bias, state, state_indices,
                     out_gate, norm_w, out, *, conv_b=None, pad_slot_id=0, gate_kind="kda",
                     kda_gate_form=0, lower_bound=-5.0, scale=None, use_qk_l2norm=True,
                     norm_eps=1e-5, gate_act="silu", err_flags=None, kernel="auto", stream=None,
                     prepare=False):
    """Fused decode: conv update -> delta step -> gated RMSNorm, one launch.
    kernel: "auto" (when head_dim is 128, the conv state is in the DS or SD layout, rows are
    16-byte aligned and there are more than two (token, head) tiles per SM: one CTA per tile
    staged in shared memory from sixteen tiles per SM, the persistent pipelined kernel below that;
    else the per-tile kernel), "tile", "pipe" or "stage" to force one.
    x bf16 [T, 3*dim]; conv_w fp32 [3*dim, 4]; conv_state bf16 with logical shape
    [num_slots, 3*dim, 3] (any strides: the "DS" layout is the plain tensor, the "SD" layout a
    transposed view of [num_slots, 3, 3*dim]); raw_g bf16 [T, heads, D] (kda) or [T, heads] (gdn);
    raw_beta bf16 [T, heads]; A_log fp32 [heads]; dt_bias fp32 [heads*D] (kda) or [heads] (gdn);
    state fp32 [num_slots, heads, D, D]; state_indices int32 [T]; out_gate bf16 [T, heads, D];
    norm_w fp32 [D]; out bf16 [T, heads, D]. raw_g, raw_beta and out_gate may be row views (any
    token stride, dense within a row), e.g. slices of one projection output."""
    torch = _torch()
    T = x.shape[0]
    f = _fused_core(conv_w, conv_state, A_log, dt_bias, state, state_indices, norm_w,
                    conv_b=conv_b, pad_slot_id=pad_slot_id, gate_kind=gate_kind,
                    kda_gate_form=kda_gate_form, lower_bound=lower_bound, scale=scale,
                    use_qk_l2norm=use_qk_l2norm, norm_eps=norm_eps, gate_act=gate_act,
                    err_flags=err_flags, kernel=kernel)
    heads, D = f.heads, f.head_dim
    f.T = T
    if x.stride(1) != 1:
        raise ValueError("x must have unit inner stride")
    f.x, f.x_stride = _ptr(x, "x", torch.bfloat16), x.stride(0)
    f.raw_g_stride = _rows(raw_g, "raw_g", heads * D if gate_kind == "kda" else heads)
    f.raw_g = _ptr(raw_g, "raw_g", torch.bfloat16)
    f.raw_beta_stride = _rows(raw_beta, "raw_beta", heads)
    f.raw_beta = _ptr(raw_beta, "raw_beta", torch.bfloat16)
    f.out_gate_stride = _rows(out_gate, "out_gate", heads * D)
    f.out_gate = _ptr(out_gate, "out_gate", torch.bfloat16)
    f.out = _ptr(_dense(out, "out"), "out", torch.bfloat16)
    return _run_or_prepare("gdn_decode_fused", (ctypes.byref(f),), (f,), stream, prepare, out)


def fused_recurrent_gated_delta_rule_packed_decode(mixed_qkv, a, b, A_log, dt_bias, scale,
                                                   initial_state, out, ssm_state_indices,
                                                   use_qk_l2norm_in_kernel=True, pad_slot_id=-1,
                                                   err_flags=None, stream=None):
    """The packed decode with the keyword names of the sglang microbenchmark's run_packed:
    mixed_qkv [B, 2*H*K + HV*V], a, b [B, HV], A_log, dt_bias [HV], initial_state
    [num_slots, HV, V, K] fp32 (updated in place), out [B, 1, HV, V], ssm_state_indices int32 [B].
    H is recovered from the row width."""
    _, HV, V, K = initial_state.shape
    H = _heads_from_width(mixed_qkv, HV, V, K)
    q, k, v = split_mixed_qkv(mixed_qkv, H, HV, K, V)
    return gdn_decode_step_indexed(q, k, v, initial_state, out, ssm_state_indices,
                                   pad_slot_id=pad_slot_id, H=H, a=a, b=b, A_log=A_log,
                                   dt_bias=dt_bias, scale=scale,
                                   use_qk_l2norm=use_qk_l2norm_in_kernel, err_flags=err_flags,
                                   stream=stream)


def _heads_from_width(mixed_qkv, HV, V, K):
    width = mixed_qkv.shape[1]
    if (width - HV * V) <= 0 or (width - HV * V) % (2 * K):
        raise ValueError("mixed_qkv width does not match 2*H*K + HV*V")
    return (width - HV * V) // (2 * K)


def fused_recurrent_gdn_replayssm_decode(mixed_qkv, a, b, A_log, dt_bias, scale, initial_state,
                                         d_cache, k_cache, g_cache, out, ssm_state_indices,
                                         write_pos, use_qk_l2norm_in_kernel=True, nk=2,
                                         pad_slot_id=-1, err_flags=None, stream=None):
    """The buffered output-only decode with the keyword names of the sglang microbenchmark's
    run_replay: initial_state [num_slots, HV, V, K] fp32 holds the checkpoints; d_cache
    [num_slots, HV, L, V], k_cache [num_slots, H, L, K], g_cache [num_slots, HV, L]; write_pos
    int32 [B] is read, not advanced. nk (the number of key chunks that page's kernel walks while
    replaying its ring) is accepted and has no effect: this library's replay is low-rank and
    never re-forms the state outside the flush step."""
    del nk
    _, HV, V, K = initial_state.shape
    H = _heads_from_width(mixed_qkv, HV, V, K)
    q, k, v = split_mixed_qkv(mixed_qkv, H, HV, K, V)
    return gdn_decode_buffered(q, k, v, initial_state, out, d_cache, k_cache, g_cache, write_pos,
                               cache_indices=ssm_state_indices, pad_slot_id=pad_slot_id, H=H, a=a,
                               b=b, A_log=A_log, dt_bias=dt_bias, scale=scale,
                               use_qk_l2norm=use_qk_l2norm_in_kernel, err_flags=err_flags,
                               stream=stream)


def conv_weight_from_stacked(weight):
    """Converts conv weights stacked per q/k/v part as [3, width, dim] (the layout the KDA
    microbenchmark passes to its fused op) to this library's [3*dim, width], channel-major. A
    one-time parameter conversion, not part of the decode step."""
    parts, width, dim = weight.shape
    return weight.permute(0, 2, 1).reshape(parts * dim, width).contiguous()


def fused_kda_decode(x, weight, bias, conv_state, raw_g, raw_beta, A_log, dt_bias, state_indices,
                     state, out, lower_bound, output_gate, norm_weight, norm_eps, *,
                     pad_slot_id=0, gate_act="silu", err_flags=None, stream=None):
    """The fused KDA decode with the keyword names of the KDA microbenchmark's `fused` call: x
    [T, 3*dim], weight [3*dim, 4] (conv_weight_from_stacked converts the stacked layout), bias or
    None, conv_state logical [num_slots, 3*dim, 3] (DS tensor or SD transposed view), raw_g
    [1, T, heads, D] or [T, heads, D], raw_beta [1, T, heads] or [T, heads], state [num_slots,
    heads, D, D], out [1, T, heads, D] or [T, heads, D], output_gate [T, heads, D], norm_weight
    [D] fp32. Slot 0 is the NULL (pad) slot, as on that page."""
    T = x.shape[0]
    heads, D = state.shape[1], state.shape[2]
    return gdn_decode_fused(x, weight, conv_state, raw_g.view(T, heads, D), raw_beta.view(T, heads),
                            A_log, dt_bias, state, state_indices, output_gate, norm_weight,
                            out.view(T, heads, D), conv_b=bias, pad_slot_id=pad_slot_id,
                            gate_kind="kda", lower_bound=lower_bound, norm_eps=norm_eps,
                            gate_act=gate_act, err_flags=err_flags, stream=stream)


def mamba_selective_scan_decode(x, dt, A, Bm, Cm, h, y, *, Dskip=None, z=None, h_out=None,
                                err_flags=None, stream=None, prepare=False):
    """Mamba-1 selective-scan decode step (declared in include/mamba_decode.h).
    x, dt: [B, D] and Bm, Cm: [B, N] (fp32 or bf16, one dtype); A: [D, N] fp32; Dskip: [D] fp32 or
    None; z: [B, D] or None; h: [B, D, N] fp32 state, updated in place unless h_out (same shape)
    is given; y: [B, D] fp32 or bf16; err_flags: an int32 CUDA tensor of one element or None."""
    torch = _torch()
    B, D = x.shape
    N = A.shape[1]
    m = MambaArgs()
    m.B, m.D, m.N = B, D, N
    m.in_dtype, m.out_dtype = _dtype_code(x), _dtype_code(y)
    for t, name in ((dt, "dt"), (Bm, "Bm"), (Cm, "Cm"), (z, "z")):
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{name} must have the dtype of x")
    if tuple(h.shape) != (B, D, N) or (h_out is not None and tuple(h_out.shape) != (B, D, N)):
        raise ValueError(f"h (and h_out) must be [{B}, {D}, {N}]")
    m.x, m.dt = _ptr(_dense(x, "x"), "x"), _ptr(_dense(dt, "dt"), "dt")
    m.A = _ptr(_dense(A, "A"), "A", torch.float32)
    m.Bm, m.Cm = _ptr(_dense(Bm, "Bm"), "Bm"), _ptr(_dense(Cm, "Cm"), "Cm")
    m.Dskip = _ptr(None if Dskip is None else _dense(Dskip, "Dskip"), "Dskip", torch.float32)
    m.z = _ptr(None if z is None else _dense(z, "z"), "z")
    m.h = _ptr(_dense(h, "h"), "h", torch.float32)
    m.h_out = _ptr(None if h_out is None else _dense(h_out, "h_out"), "h_out", torch.float32)
    m.y = _ptr(_dense(y, "y"), "y")
    m.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    return _run_or_prepare("mamba_selective_scan_decode", (ctypes.byref(m),), (m,), stream, prepare, y)


def _token_rows(t, name: str, T: int, width: int, dtype=None):
    """A [T, width] or [S, L, width] tensor whose T rows lie one stride apart: (pointer, row stride)."""
    if t.dim() not in (2, 3) or t.shape[-1] != width or t.numel() != T * width:
        raise ValueError(f"{name}: expected {T} rows of {width}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() == 0:
        return _ptr(t, name), width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: rows need unit inner stride")
    stride = t.stride(-2) if t.shape[-2] > 1 else t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else width
    if t.dim() == 3 and t.shape[0] > 1 and t.stride(0) != t.shape[1] * stride:
        raise ValueError(f"{name}: sequences must follow one another at the row stride")
    return _ptr(t, name), stride


def mamba_scan_workspace(T, D, N, *, sequences=1, uniform=True, backward=False, device=None):
    """A workspace tensor for mamba_selective_scan (or its backward pass) over T token rows of
    `sequences` sequences, of equal lengths (uniform) or given by cu_seqlens; None when the call needs none."""
    nbytes = lib().mamba_scan_workspace_bytes(int(T), int(sequences), int(D), int(N), int(uniform), int(backward))
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def _scan_args(x, dt, A, Bm, Cm, *, Dskip, z, sequences, cu_seqlens, state_indices, h0, other_states, workspace,
               err_flags):
    torch = _torch()
    D, N = A.shape
    T = x.numel() // D if D else 0
    m = MambaScanArgs()
    m.T, m.D, m.N = T, D, N
    if cu_seqlens is not None:
        if sequences is not None:
            raise ValueError("give cu_seqlens or sequences, not both")
        m.S = cu_seqlens.numel() - 1
    else:
        m.S = sequences if sequences is not None else (x.shape[0] if x.dim() == 3 else 1)
    m.in_dtype = _dtype_code(x)
    m.x, m.x_stride = _token_rows(x, "x", T, D)
    m.dt, m.dt_stride = _token_rows(dt, "dt", T, D, x.dtype)
    m.Bm, m.B_stride = _token_rows(Bm, "Bm", T, N, x.dtype)
    m.Cm, m.C_stride = _token_rows(Cm, "Cm", T, N, x.dtype)
    if z is not None:
        m.z, m.z_stride = _token_rows(z, "z", T, D, x.dtype)
    m.A = _ptr(_dense(A, "A"), "A", torch.float32)
    if Dskip is not None:
        if Dskip.numel() != D:
            raise ValueError(f"Dskip must have {D} entries")
        m.Dskip = _ptr(_dense(Dskip, "Dskip"), "Dskip", torch.float32)
    m.cu_seqlens = _ptr(None if cu_seqlens is None else _dense(cu_seqlens, "cu_seqlens"), "cu_seqlens", torch.int32)
    if state_indices is not None:
        if state_indices.numel() != m.S:
            raise ValueError(f"state_indices must have {m.S} entries")
        m.state_indices = _ptr(_dense(state_indices, "state_indices"), "state_indices", torch.int32)
    states = [t for t in (h0, *other_states) if t is not None]
    for t in states:
        if t.dim() != 3 or t.shape != states[0].shape or tuple(t.shape[1:]) != (D, N):
            raise ValueError(f"state buffers must be [num_states, {D}, {N}], all with the same num_states")
        _ptr(_dense(t, "a state buffer"), "a state buffer", torch.float32)
    m.num_states = states[0].shape[0] if states else 0
    m.h0 = None if h0 is None else h0.data_ptr()
    if workspace is not None:
        m.workspace = _ptr(_dense(workspace, "workspace"), "workspace")
        m.workspace_bytes = workspace.numel() * workspace.element_size()
    m.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    return m, T, D, N


def mamba_selective_scan(x, dt, A, Bm, Cm, y, *, Dskip=None, z=None, sequences=None, cu_seqlens=None,
                         state_indices=None, h0=None, h_last=None, workspace=None, err_flags=None, stream=None,
                         prepare=False):
    """Mamba-1 selective scan over whole sequences (declared in include/mamba_scan.h). x, dt, z, y: [T, D] (or
    [S, L, D]) and Bm, Cm: [T, N] row views, fp32 or bf16 (y of its own dtype); A: [D, N] and Dskip: [D] fp32. The T
    rows are `sequences` equal sequences (default: x's first axis of three, else one), or those of cu_seqlens
    (int32 [S + 1] on the device). h0 and h_last: [num_states, D, N] fp32 states at row state_indices[s] (int32;
    default s) of sequence s; h_last may be h0. workspace: see mamba_scan_workspace."""
    m, T, D, _ = _scan_args(x, dt, A, Bm, Cm, Dskip=Dskip, z=z, sequences=sequences, cu_seqlens=cu_seqlens,
                            state_indices=state_indices, h0=h0, other_states=(h_last,), workspace=workspace,
                            err_flags=err_flags)
    m.out_dtype = _dtype_code(y)
    m.y, m.y_stride = _token_rows(y, "y", T, D)
    m.h_last = None if h_last is None else h_last.data_ptr()
    keep = (m, x, dt, A, Bm, Cm, y, Dskip, z, cu_seqlens, state_indices, h0, h_last, workspace, err_flags)
    return _run_or_prepare("mamba_selective_scan", (ctypes.byref(m),), keep, stream, prepare, y)


def mamba_selective_scan_backward(x, dt, A, Bm, Cm, dy, *, Dskip=None, z=None, sequences=None, cu_seqlens=None,
                                  state_indices=None, h0=None, dh_last=None, dx=None, ddt=None, dz=None, dBm=None,
                                  dCm=None, dA=None, dDskip=None, dh0=None, workspace=None, err_flags=None,
                                  stream=None, prepare=False):
    """Gradients of mamba_selective_scan (declared in include/mamba_scan.h). dy: [T, D], dh_last: [num_states, D, N]
    fp32 or None (zero). Each gradient buffer given is written: dx, ddt, dz like x; dBm, dCm like Bm (all in the dtype
    of x), dA [D, N], dDskip [D] and dh0 [num_states, D, N] fp32 (also without h0: at a start from zero)."""
    torch = _torch()
    m, T, D, N = _scan_args(x, dt, A, Bm, Cm, Dskip=Dskip, z=z, sequences=sequences, cu_seqlens=cu_seqlens,
                            state_indices=state_indices, h0=h0, other_states=(dh_last, dh0), workspace=workspace,
                            err_flags=err_flags)
    a = MambaScanGradArgs()
    a.s = m
    a.dy, a.dy_stride = _token_rows(dy, "dy", T, D, x.dtype)
    for t, name, width, stride in ((dx, "dx", D, "dx_stride"), (ddt, "ddt", D, "ddt_stride"), (dz, "dz", D, "dz_stride"),
                                   (dBm, "dBm", N, "dB_stride"), (dCm, "dCm", N, "dC_stride")):
        if t is not None:
            p, st = _token_rows(t, name, T, width, x.dtype)
            setattr(a, name, p)
            setattr(a, stride, st)
    for t, name, shape in ((dA, "dA", (D, N)), (dDskip, "dDskip", (D,))):
        if t is not None:
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
            setattr(a, name, _ptr(_dense(t, name), name, torch.float32))
    a.dh_last = None if dh_last is None else dh_last.data_ptr()
    a.dh0 = None if dh0 is None else dh0.data_ptr()
    keep = (a, x, dt, A, Bm, Cm, dy, Dskip, z, cu_seqlens, state_indices, h0, dh_last, dx, ddt, dz, dBm, dCm, dA,
            dDskip, dh0, workspace, err_flags)
    return _run_or_prepare("mamba_selective_scan_backward", (ctypes.byref(a),), keep, stream, prepare, None)


def beam_select_workspace(batch, beams, vocab, K, device=None):
    """A workspace tensor for gdn_beam_select with these sizes."""
    nbytes = lib().gdn_beam_select_workspace_bytes(int(batch), int(beams), int(vocab), int(K))
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device or "cuda")


def _table(t, name, shape, dtype):
    if t is None:
        return None
    # (a flat table, or a row or column, is taken; two axes of other sizes are another table, a transposed one say)
    n = shape[0] * shape[1]
    if tuple(t.shape) != shape and (t.numel() != n or (t.dim() == 2 and max(t.shape) != n)):
        raise ValueError(f"{name} must be {list(shape)}")
    return _ptr(_dense(t, name), name, dtype)


def gdn_beam_select(logits, scores, out_scores, out_parents, out_tokens, *, rows=None, finished=None, eos_token=-1,
                    out_finished=None, workspace=None, err_flags=None, stream=None, prepare=False):
    """One beam-search selection (declared in include/gdn_beam.h). logits: [num_rows, vocab] fp32 or bf16 row view;
    scores: [batch, beams] fp32; rows: int32 [batch, beams], the logits row of each beam, or None (in order);
    finished: uint8 or bool [batch, beams] or None; out_scores fp32, out_parents and out_tokens int32, out_finished uint8
    or bool: [batch, K]. workspace: see beam_select_workspace."""
    torch = _torch()
    batch, beams = scores.shape
    K = out_scores.shape[1]
    a = BeamSelectArgs()
    a.batch, a.beams, a.K = batch, beams, K
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits: expected [rows, vocab] with unit inner stride")
    a.num_rows, a.vocab = logits.shape
    a.logits_dtype = _dtype_code(logits)
    a.logits = _ptr(logits, "logits")
    a.row_stride = logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]
    for t, name in ((finished, "finished"), (out_finished, "out_finished")):
        if t is not None and t.dtype not in (torch.uint8, torch.bool):
            raise TypeError(f"{name} must be uint8 or bool")
    a.rows = _table(rows, "rows", (batch, beams), torch.int32)
    a.scores = _table(scores, "scores", (batch, beams), torch.float32)
    a.finished = _table(finished, "finished", (batch, beams), None)
    a.eos_token = int(eos_token)
    a.out_scores = _table(out_scores, "out_scores", (batch, K), torch.float32)
    a.out_parents = _table(out_parents, "out_parents", (batch, K), torch.int32)
    a.out_tokens = _table(out_tokens, "out_tokens", (batch, K), torch.int32)
    a.out_finished = _table(out_finished, "out_finished", (batch, K), None)
    if workspace is not None:
        a.workspace = _ptr(_dense(workspace, "workspace"), "workspace")
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    keep = (a, logits, scores, out_scores, out_parents, out_tokens, rows, finished, out_finished, workspace, err_flags)
    return _run_or_prepare("gdn_beam_select", (ctypes.byref(a),), keep, stream, prepare,
                           (out_scores, out_parents, out_tokens))


def gdn_beam_reorder(pools, slots, parents, new_slots, *, err_flags=None, stream=None, prepare=False):
    """Moves the states of a beam search's chosen continuations (declared in include/gdn_beam.h). pools: tensors whose
    first axis is the slot and whose slots are dense (any dtype: states, convolution taps, rings), updated in place;
    slots, parents, new_slots: int32 [batch, beams]. new_slots gets each new beam's slot."""
    torch = _torch()
    batch, beams = slots.shape
    a = BeamReorderArgs()
    a.batch, a.beams = batch, beams
    a.num_pools = len(pools)
    table = (BeamPool * max(1, len(pools)))()
    num_slots = pools[0].shape[0] if pools else 1
    if any(t.dim() < 1 or t.shape[0] != num_slots for t in pools):
        raise ValueError("every pool must have the same number of slots")
    for q, t in zip(table, pools):
        if t.shape[0] > 0 and not t[0].is_contiguous():
            raise ValueError("a pool's slots must be dense")
        q.base = _ptr(t, "a pool")
        q.slot_bytes = t[0].numel() * t.element_size() if num_slots else 0
        q.slot_stride = t.stride(0) * t.element_size() if num_slots > 1 else q.slot_bytes
    a.num_slots = num_slots
    a.pools = table
    a.slots = _table(slots, "slots", (batch, beams), torch.int32)
    a.parents = _table(parents, "parents", (batch, beams), torch.int32)
    a.new_slots = _table(new_slots, "new_slots", (batch, beams), torch.int32)
    a.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    keep = (a, table, pools, slots, parents, new_slots, err_flags)
    return _run_or_prepare("gdn_beam_reorder", (ctypes.byref(a),), keep, stream, prepare, new_slots)


def _head_rows(t, name: str, rows=None, heads=None, dim=None, dtype=None):
    """A [rows, heads, dim] tensor (or [S, L, heads, dim], whose sequences follow one another at the row stride) of any
    row and head strides: pointer, row stride, head stride, and its sizes."""
    if t.dim() not in (3, 4):
        raise ValueError(f"{name}: expected [rows, heads, dim] or [S, L, heads, dim]")
    n, h, d = t.numel() // max(1, t.shape[-1] * t.shape[-2]), t.shape[-2], t.shape[-1]
    if 0 in t.shape[:-2]:
        n = 0
    for have, want, what in ((n, rows, "rows"), (h, heads, "heads"), (d, dim, "channels")):
        if want is not None and have != want:
            raise ValueError(f"{name}: expected {want} {what}, got {have}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: heads need unit inner stride")
    head = t.stride(-2) if h > 1 else d
    if t.dim() == 4 and n > 0:
        S, L = t.shape[0], t.shape[1]
        row = t.stride(1) if L > 1 else t.stride(0)
        if S > 1 and L > 1 and t.stride(0) != L * row:
            raise ValueError(f"{name}: sequences must follow one another at the row stride")
    else:
        row = t.stride(0) if t.dim() == 3 else h * d
    if n <= 1:
        row = h * d
    return _ptr(t, name), row, head, (n, h, d)


def _put_rows(a, field, t, name, stride=None, **kw):
    """Sets a struct's pointer, row stride and head stride of a tensor of head rows; returns its sizes."""
    stride = stride or field
    p, row, head, sizes = _head_rows(t, name, **kw)
    setattr(a, field, p)
    setattr(a, stride + "_stride", row)
    setattr(a, stride + "_head_stride", head)
    return sizes


def _log_decays(g, rows, heads):
    """g [HV], or [rows, HV] (or [S, L, HV]) fp32: pointer and row stride (0: one decay a head)."""
    torch = _torch()
    if g.dim() == 1:
        if g.shape[0] != heads or g.stride(0) != 1 and heads > 1:
            raise ValueError(f"g: expected {heads} dense entries")
        return _ptr(g, "g", torch.float32), 0
    p, stride = _token_rows(g, "g", rows, heads, torch.float32)
    if rows > 1 and stride == 0:
        raise ValueError("g: rows of one decay a head are given as a tensor [HV]")
    return p, stride if rows > 1 else max(stride, heads)


def linear_attention_workspace(T, H, HV, K, V, *, sequences=1, uniform=True, backward=False, dtype=None, device=None):
    """A workspace tensor for gdn_linear_attention (or its backward pass) over T token rows of `sequences` sequences,
    of equal lengths (uniform) or given by cu_seqlens, with inputs of `dtype` (default bfloat16); None when the call
    needs none. It is for these sizes: fewer tokens or sequences, cut otherwise, may need more. Calls that may run at the
    same time need one each."""
    torch = _torch()
    code = GDN_F32 if dtype == torch.float32 else GDN_BF16
    nbytes = lib().gdn_linear_workspace_bytes(int(T), int(sequences), int(H), int(HV), int(K), int(V), code, int(uniform),
                                              int(backward))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def _linear_args(q, k, v, g, *, scale, sequences, cu_seqlens, state_indices, states, workspace, err_flags):
    torch = _torch()
    a = LinearArgs()
    a.in_dtype = _dtype_code(q)
    a.T, a.H, a.K = _put_rows(a, "q", q, "q")
    _put_rows(a, "k", k, "k", rows=a.T, heads=a.H, dim=a.K, dtype=q.dtype)
    _, a.HV, a.V = _put_rows(a, "v", v, "v", rows=a.T, dtype=q.dtype)
    a.g, a.g_stride = _log_decays(g, a.T, a.HV)
    a.scale = 0.0 if scale is None else float(scale)
    if cu_seqlens is not None:
        if sequences is not None:
            raise ValueError("give cu_seqlens or sequences, not both")
        a.S = cu_seqlens.numel() - 1
        a.cu_seqlens = _ptr(_dense(cu_seqlens, "cu_seqlens"), "cu_seqlens", torch.int32)
    else:
        a.S = sequences if sequences is not None else (q.shape[0] if q.dim() == 4 else 1)
    if state_indices is not None:
        if state_indices.numel() != a.S:
            raise ValueError(f"state_indices must have {a.S} entries")
        a.state_indices = _ptr(_dense(state_indices, "state_indices"), "state_indices", torch.int32)
    states = [t for t in states if t is not None]
    for t in states:
        if t.dim() != 4 or t.shape != states[0].shape or tuple(t.shape[1:]) != (a.HV, a.V, a.K):
            raise ValueError(f"state buffers must be [num_states, {a.HV}, {a.V}, {a.K}], all with the same num_states")
        _ptr(_dense(t, "a state buffer"), "a state buffer", torch.float32)
    a.num_states = states[0].shape[0] if states else 0
    if workspace is not None:
        a.workspace = _ptr(_dense(workspace, "workspace"), "workspace")
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    return a


def gdn_linear_attention(q, k, v, g, o, *, scale=None, sequences=None, cu_seqlens=None, state_indices=None,
                         initial_state=None, final_state=None, workspace=None, err_flags=None, stream=None, prepare=False):
    """Linear attention with a decay for each head over whole sequences (declared in include/gdn_linear.h):
    S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t. q, k: [T, H, K] and v, o: [T, HV, V] (or [S, L, ..]) of any
    row and head strides, fp32 or bf16 (o of its own dtype); g: log decays fp32, [T, HV] or one per head [HV]. The T
    rows are `sequences` equal sequences (default: q's first axis of four, else one), or those of cu_seqlens (int32
    [S + 1] on the device; rows outside them are left as they are). initial_state and final_state: [num_states, HV, V, K]
    fp32 at row state_indices[s] (int32; default s) of sequence s; final_state may be initial_state. workspace: see
    linear_attention_workspace."""
    a = _linear_args(q, k, v, g, scale=scale, sequences=sequences, cu_seqlens=cu_seqlens, state_indices=state_indices,
                     states=(initial_state, final_state), workspace=workspace, err_flags=err_flags)
    a.out_dtype = _dtype_code(o)
    _put_rows(a, "o", o, "o", rows=a.T, heads=a.HV, dim=a.V)
    a.initial_state = None if initial_state is None else initial_state.data_ptr()
    a.final_state = None if final_state is None else final_state.data_ptr()
    keep = (a, q, k, v, g, o, cu_seqlens, state_indices, initial_state, final_state, workspace, err_flags)
    return _run_or_prepare("gdn_linear_attention", (ctypes.byref(a),), keep, stream, prepare, o)


def gdn_linear_attention_backward(q, k, v, g, do, *, scale=None, sequences=None, cu_seqlens=None, state_indices=None,
                                  initial_state=None, d_final_state=None, dq=None, dk=None, dv=None, dg=None,
                                  d_initial_state=None, workspace=None, err_flags=None, stream=None, prepare=False):
    """Gradients of gdn_linear_attention (declared in include/gdn_linear.h). do: like v; d_final_state: [num_states, HV,
    V, K] fp32 or None (zero). Each gradient buffer given is written: dq, dk like q, dv like v (in q's dtype, any row
    and head strides), dg fp32 like g, d_initial_state [num_states, HV, V, K] fp32 (also without initial_state: at a
    start from zero; not over initial_state or d_final_state)."""
    torch = _torch()
    s = _linear_args(q, k, v, g, scale=scale, sequences=sequences, cu_seqlens=cu_seqlens, state_indices=state_indices,
                     states=(initial_state, d_final_state, d_initial_state), workspace=workspace, err_flags=err_flags)
    s.initial_state = None if initial_state is None else initial_state.data_ptr()
    a = LinearGradArgs()
    a.s = s
    _put_rows(a, "d_o", do, "do", "do", rows=s.T, heads=s.HV, dim=s.V, dtype=q.dtype)
    for t, name, heads, dim in ((dq, "dq", s.H, s.K), (dk, "dk", s.H, s.K), (dv, "dv", s.HV, s.V)):
        if t is not None:
            _put_rows(a, name, t, name, rows=s.T, heads=heads, dim=dim, dtype=q.dtype)
    if dg is not None:
        if (dg.dim() == 1) != (g.dim() == 1):
            raise ValueError("dg must have the shape of g")
        a.dg, a.dg_stride = _log_decays(dg, s.T, s.HV)
    a.d_final_state = None if d_final_state is None else d_final_state.data_ptr()
    a.d_initial_state = None if d_initial_state is None else d_initial_state.data_ptr()
    keep = (a, q, k, v, g, do, cu_seqlens, state_indices, initial_state, d_final_state, dq, dk, dv, dg, d_initial_state,
            workspace, err_flags)
    return _run_or_prepare("gdn_linear_attention_backward", (ctypes.byref(a),), keep, stream, prepare, None)


def _rotary_table(frequencies):
    if frequencies.dim() != 1 or frequencies.numel() < 1:
        raise ValueError("frequencies must be [rotary_dim / 2]")
    return _ptr(_dense(frequencies, "frequencies"), "frequencies", _torch().float64), 2 * frequencies.numel()


def gdn_linear_attention_step(q, k, v, g, state, out, cache_indices=None, *, pad_slot_id=-1, scale=None, positions=None,
                              frequencies=None, interleaved=False, magnitude=1.0, err_flags=None, stream=None,
                              prepare=False):
    """One token of linear attention for each request row (declared in include/gdn_linear.h). q, k: [B, H, K] and v: [B,
    HV, V] of any row and head strides; g: log decays fp32, [B, HV] or [HV]; state: [num_slots, HV, V, K] fp32 or bf16,
    updated in place; out: [B, HV, V] dense. Row b is on slot cache_indices[b] (int32; default b); rows whose index is
    pad_slot_id are skipped (out zeroed). With frequencies (see gdn_rotary) q and k are turned to positions [B] first."""
    torch = _torch()
    if float(magnitude) == 0.0:
        raise ValueError("magnitude must not be 0")
    a = LinearStepArgs()
    a.in_dtype, a.out_dtype, a.state_dtype = _dtype_code(q), _dtype_code(out), _dtype_code(state)
    a.B, a.H, a.K = _put_rows(a, "q", q, "q")
    _put_rows(a, "k", k, "k", rows=a.B, heads=a.H, dim=a.K, dtype=q.dtype)
    _, a.HV, a.V = _put_rows(a, "v", v, "v", rows=a.B, dtype=q.dtype)
    a.g, a.g_stride = _log_decays(g, a.B, a.HV)
    if state.dim() != 4 or tuple(state.shape[1:]) != (a.HV, a.V, a.K):
        raise ValueError(f"state must be [num_slots, {a.HV}, {a.V}, {a.K}]")
    a.num_slots, a.state = state.shape[0], _ptr(_dense(state, "state"), "state")
    if out.numel() != a.B * a.HV * a.V:
        raise ValueError(f"out must hold {a.B * a.HV * a.V} elements")
    a.out = _ptr(_dense(out, "out"), "out")
    a.scale = 0.0 if scale is None else float(scale)
    if (positions is None) != (frequencies is None):
        raise ValueError("positions and frequencies go together")
    if frequencies is not None:
        a.frequencies, a.rotary_dim = _rotary_table(frequencies)
        if positions.numel() != a.B:
            raise ValueError(f"positions must have {a.B} entries")
        a.positions = _ptr(_dense(positions, "positions"), "positions", torch.int32)
        a.interleaved, a.magnitude = int(bool(interleaved)), float(magnitude)
    a.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    idx = None
    if cache_indices is not None:
        if cache_indices.numel() != a.B:
            raise ValueError(f"cache_indices must have {a.B} entries")
        idx = _ptr(_dense(cache_indices, "cache_indices"), "cache_indices", torch.int32)
    keep = (a, q, k, v, g, state, out, cache_indices, positions, frequencies, err_flags)
    return _run_or_prepare("gdn_linear_attention_step", (ctypes.byref(a), ctypes.c_void_p(idx), ctypes.c_int32(int(pad_slot_id))),
                           keep, stream, prepare, out)


def rotary_frequencies(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, original_length=None, keep_turns=32.0,
                       scale_turns=1.0, device=None):
    """fp64 frequencies [rotary_dim / 2] (radians a position) base^(-2i / rotary_dim) for gdn_rotary, scaled for contexts
    `factor` times as long as the trained one: None (as they are); "linear" (all divided by factor); "base" (a larger base, so
    that the slowest is divided by factor and the fastest kept); "parts" (what turns more than keep_turns times in
    original_length positions is kept, what turns less than scale_turns divided by factor, linearly between)."""
    torch = _torch()
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not factor > 0:
        raise ValueError("factor must be positive")
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_length is None:
            raise ValueError("scaling in parts needs original_length")
        turns = original_length * f / (2 * torch.pi)
        keep = ((turns - scale_turns) / (keep_turns - scale_turns)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device or "cuda")


def gdn_rotary(q, k, positions, frequencies, *, q_out=None, k_out=None, interleaved=False, inverse=False, magnitude=1.0,
               stream=None, prepare=False):
    """Rotary positions of q [T, H, D] and k [T, HK, D] (or None), fp32 or bf16 of any row and head strides (declared in
    include/gdn_rotary.h): the first 2 * len(frequencies) channels of every head are turned by positions[t] *
    frequencies[i] (int32 [T]; fp64, see rotary_frequencies) and multiplied by magnitude, as pairs (i, i + half) or
    (2i, 2i + 1) when interleaved. Without q_out and k_out in place. inverse=True turns back: the gradients of q and
    k from those of the outputs. Returns (q_out, k_out)."""
    torch = _torch()
    a = RotaryArgs()
    a.dtype = _dtype_code(q)
    a.T, a.H, a.D = _put_rows(a, "q", q, "q")
    q_out = q if q_out is None else q_out
    _put_rows(a, "q_out", q_out, "q_out", rows=a.T, heads=a.H, dim=a.D, dtype=q.dtype)
    if k is not None:
        _, a.HK, _ = _put_rows(a, "k", k, "k", rows=a.T, dim=a.D, dtype=q.dtype)
        k_out = k if k_out is None else k_out
        _put_rows(a, "k_out", k_out, "k_out", rows=a.T, heads=a.HK, dim=a.D, dtype=q.dtype)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if positions.numel() != a.T:
        raise ValueError(f"positions must have {a.T} entries")
    a.positions = _ptr(_dense(positions, "positions"), "positions", torch.int32)
    a.frequencies, a.rotary_dim = _rotary_table(frequencies)
    a.interleaved, a.inverse = int(bool(interleaved)), int(bool(inverse))
    a.magnitude = float(magnitude)
    if a.magnitude == 0.0:
        raise ValueError("magnitude must not be 0")
    keep = (a, q, k, q_out, k_out, positions, frequencies)
    return _run_or_prepare("gdn_rotary", (ctypes.byref(a),), keep, stream, prepare, (q_out, k_out))


def gdn_selftest_bounded_wait(err_flags, limit_cycles, arrive, stream=None):
    """Run the bounded-wait self-test kernel (see include/gdn_decode.h); err_flags is a CUDA int32
    tensor of one element that receives GDN_DEVERR_TIMEOUT when the wait gives up."""
    torch = _torch()
    _check("gdn_selftest_bounded_wait",
           lib().gdn_selftest_bounded_wait(_ptr(err_flags, "err_flags", torch.int32), int(limit_cycles),
                                           int(bool(arrive)), _stream(stream)))


def gemv_workspace(T, N, Kd, splits=0, device=None):
    """A workspace tensor for gdn_gemv_bf16 with this split count (0: the library's choice), or
    None when the call needs none."""
    torch = _torch()
    L = lib()
    s = splits or L.gdn_gemv_default_splits(int(T), int(N), int(Kd))
    nbytes = L.gdn_gemv_workspace_bytes(int(T), int(N), int(s))
    if nbytes == 0:
        return None
    return torch.empty(nbytes // 4, dtype=torch.float32, device=device or "cuda")


def gdn_gemv_bf16(x, W, y, *, splits=0, workspace=None, err_flags=None, stream=None, prepare=False):
    """Decode projection y [T, N] = x [T, Kd] W[N, Kd]^T (declared in include/gdn_gemv.h). x and W
    bf16 with dense rows (x may be a row view), y fp32 or bf16. With more than one K split (splits
    = 0 lets the library choose) a workspace is needed: see gemv_workspace. err_flags: optional
    int32 CUDA tensor of one element that a kernel giving up a bounded wait ORs a bit into."""
    torch = _torch()
    T, Kd = x.shape
    N = W.shape[0]
    if W.shape[1] != Kd or tuple(y.shape) != (T, N):
        raise ValueError(f"expected W [{N}, {Kd}] and y [{T}, {N}]")
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("x and y need unit inner stride")
    g = GemvArgs()
    g.T, g.N, g.Kd = T, N, Kd
    g.out_dtype = _dtype_code(y)
    g.x, g.x_stride = _ptr(x, "x", torch.bfloat16), x.stride(0)
    g.W = _ptr(_dense(W, "W"), "W", torch.bfloat16)
    g.y, g.y_stride = _ptr(y, "y"), y.stride(0)
    g.splits = int(splits)
    if workspace is not None:
        g.workspace = _ptr(_dense(workspace, "workspace"), "workspace", torch.float32)
        g.workspace_bytes = workspace.numel() * 4
    if err_flags is not None:
        g.err_flags = _ptr(err_flags, "err_flags", torch.int32)
    return _run_or_prepare("gdn_gemv_bf16", (ctypes.byref(g),), (g, workspace, err_flags), stream, prepare, y)
