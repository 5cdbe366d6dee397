"""ctypes binding of libmoe.so (C ABI in include/moe.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their device pointers and the current HIP stream to
the library, and raises MoEError when the library returns an error status.
No step of the computation runs here; if libmoe.so is missing or cannot be
loaded, ``load_library`` raises and nothing falls back to another path.

torch is imported before the library is loaded so that libmoe.so binds to the
HIP runtime torch already holds (both carry the soname libamdhip64.so.7); the
loader then checks that only one HIP runtime is mapped in the process.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmoe.so"
_lock = threading.Lock()
_lib = None

MOE_OK = 0
DTYPE_F32 = 0
DTYPE_BF16 = 1
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES of moe.h

_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
           3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_HIP"}


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class MoEProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("G", ctypes.c_int32), ("TG", ctypes.c_int32),
                ("k", ctypes.c_int32), ("scale", ctypes.c_float)]

    @classmethod
    def from_config(cls, cfg, T=None):
        return cls(cfg.T if T is None else T, cfg.H, cfg.I, cfg.E, cfg.G, cfg.TG, cfg.k,
                   cfg.scale)


class MoEGemmProblem(ctypes.Structure):
    """moe_gemm_problem of moe_gemm.h: P sorted positions, S activation rows,
    E experts, weights [E,N,K], k positions per activation row."""
    _fields_ = [("P", ctypes.c_int64), ("S", ctypes.c_int64), ("E", ctypes.c_int32),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("k", ctypes.c_int32)]


EXPORTS = ("moe_workspace_bytes", "moe_route", "moe_permute", "moe_expert_ffn",
           "moe_expert_gate_up", "moe_expert_down", "moe_combine", "moe_combine_residual",
           "moe_dense_mlp", "moe_expert_ffn_fp8", "moe_forward", "moe_forward_fp8",
           "moe_forward_noalloc", "moe_status_string", "moe_last_error",
           # grouped products (include/moe_gemm.h)
           "moe_gemm_workspace_bytes", "moe_grouped_gemm", "moe_grouped_gemm_dgrad",
           "moe_grouped_gemm_wgrad", "moe_quantize_rows_int8", "moe_grouped_gemm_int8",
           "moe_int8_workspace_bytes", "moe_expert_ffn_int8", "moe_forward_int8",
           "moe_backward_workspace_bytes", "moe_expert_ffn_backward",
           # experts in FP8 with a scale for each block of 128 (include/moe_fp8.h)
           "moe_fp8_block_scales", "moe_quantize_rows_fp8_block",
           "moe_quantize_weights_fp8_block", "moe_grouped_gemm_fp8_block",
           "moe_grouped_gemm_fp8_block_dgrad", "moe_expert_gate_up_fp8_block",
           "moe_fp8_block_workspace_bytes", "moe_expert_ffn_fp8_block", "moe_forward_fp8_block",
           "moe_fp8_block_backward_workspace_bytes", "moe_expert_ffn_fp8_block_backward",
           # the norm in front of the block (include/moe_norm.h)
           "moe_norm", "moe_norm_workspace_bytes", "moe_norm_backward",
           # measurement kernels (include/moe_peak.h)
           "moe_peak_stream_read", "moe_peak_mfma_bf16", "moe_peak_mfma_bf16_flops",
           "moe_peak_mfma_stream", "moe_peak_mfma_stream_flops", "moe_peak_mfma_stream_bytes")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _hip_runtimes_mapped():
    paths = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    paths.add(os.path.realpath(line.split()[-1]))
    except OSError:
        pass
    return paths


def load_library():
    """Load libmoe.so once and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m group_limited_routing_router_amd.build`")
        lib = ctypes.CDLL(path)
        rts = _hip_runtimes_mapped()
        if len(rts) > 1:
            raise ImportError(f"two HIP runtimes are mapped: {sorted(rts)}")
        P = ctypes.c_void_p
        prob = ctypes.POINTER(MoEProblem)
        st = ctypes.c_int
        lib.moe_workspace_bytes.argtypes = [prob]
        lib.moe_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_route.argtypes = [prob, P, P, P, P, P, P]
        lib.moe_route.restype = st
        lib.moe_permute.argtypes = [prob, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_permute.restype = st
        lib.moe_expert_ffn.argtypes = [prob, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_expert_ffn.restype = st
        lib.moe_expert_gate_up.argtypes = [prob, P, P, P, P, P, P, P]
        lib.moe_expert_gate_up.restype = st
        lib.moe_expert_down.argtypes = [prob, P, P, P, P, P]
        lib.moe_expert_down.restype = st
        lib.moe_combine.argtypes = [prob, P, P, P, P, ctypes.c_int, P]
        lib.moe_combine.restype = st
        lib.moe_combine_residual.argtypes = [prob, P, P, P, P, ctypes.c_float, ctypes.c_int32, P,
                                             P]
        lib.moe_combine_residual.restype = st
        lib.moe_expert_ffn_fp8.argtypes = [prob, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                           P]
        lib.moe_expert_ffn_fp8.restype = st
        lib.moe_forward_fp8.argtypes = [prob, P, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, P, P,
                                        P, ctypes.c_size_t, P]
        lib.moe_forward_fp8.restype = st
        lib.moe_dense_mlp.argtypes = [prob, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_dense_mlp.restype = st
        lib.moe_forward.argtypes = [prob, P, P, P, P, P, P, P, ctypes.c_int, P, P, P, P,
                                    ctypes.c_size_t, P]
        lib.moe_forward.restype = st
        lib.moe_forward_noalloc.argtypes = [prob, P, P, P, P, P, P, P, ctypes.c_int, P, P, P, P]
        lib.moe_forward_noalloc.restype = st
        gemm = ctypes.POINTER(MoEGemmProblem)
        i32, size = ctypes.c_int, ctypes.c_size_t
        lib.moe_gemm_workspace_bytes.argtypes = [gemm]
        lib.moe_gemm_workspace_bytes.restype = size
        lib.moe_grouped_gemm.argtypes = [gemm, P, P, P, P, P, i32, P, size, P]
        lib.moe_grouped_gemm.restype = st
        lib.moe_grouped_gemm_dgrad.argtypes = [gemm, P, P, P, P, i32, i32, P, size, P]
        lib.moe_grouped_gemm_dgrad.restype = st
        lib.moe_grouped_gemm_wgrad.argtypes = [gemm, P, P, P, P, P, i32, i32, P, size, P]
        lib.moe_grouped_gemm_wgrad.restype = st
        lib.moe_quantize_rows_int8.argtypes = [ctypes.c_int64, ctypes.c_int32, P, P, P, P]
        lib.moe_quantize_rows_int8.restype = st
        lib.moe_grouped_gemm_int8.argtypes = [gemm, P, P, P, P, P, P, P, i32, P, size, P]
        lib.moe_grouped_gemm_int8.restype = st
        lib.moe_int8_workspace_bytes.argtypes = [prob]
        lib.moe_int8_workspace_bytes.restype = size
        lib.moe_expert_ffn_int8.argtypes = [prob, P, P, P, P, P, P, P, P, P, P, P, size, P]
        lib.moe_expert_ffn_int8.restype = st
        lib.moe_forward_int8.argtypes = [prob, P, P, P, P, P, P, P, P, P, P, i32, P, P, P, P, size,
                                         P]
        lib.moe_forward_int8.restype = st
        lib.moe_backward_workspace_bytes.argtypes = [prob]
        lib.moe_backward_workspace_bytes.restype = size
        lib.moe_expert_ffn_backward.argtypes = [prob, P, P, P, P, P, P, P, P, P, P, P, i32, i32, P,
                                                size, P]
        lib.moe_expert_ffn_backward.restype = st
        i64, f32 = ctypes.c_int64, ctypes.c_float
        lib.moe_fp8_block_scales.argtypes = [ctypes.c_int32]
        lib.moe_fp8_block_scales.restype = ctypes.c_int32
        lib.moe_quantize_rows_fp8_block.argtypes = [i64, ctypes.c_int32, P, P, P, P]
        lib.moe_quantize_weights_fp8_block.argtypes = [ctypes.c_int32] * 3 + [P] * 4
        lib.moe_grouped_gemm_fp8_block.argtypes = [gemm] + [P] * 7 + [i32, P, size, P]
        lib.moe_grouped_gemm_fp8_block_dgrad.argtypes = [gemm] + [P] * 6 + [i32, i32, P, size, P]
        lib.moe_expert_gate_up_fp8_block.argtypes = [prob] + [P] * 11
        lib.moe_fp8_block_workspace_bytes.argtypes = [prob]
        lib.moe_fp8_block_workspace_bytes.restype = size
        lib.moe_expert_ffn_fp8_block.argtypes = [prob] + [P] * 10 + [i32, P, size, P]
        lib.moe_forward_fp8_block.argtypes = [prob] + [P] * 10 + [i32, P, P, P, P, size, P]
        lib.moe_fp8_block_backward_workspace_bytes.argtypes = [prob]
        lib.moe_fp8_block_backward_workspace_bytes.restype = size
        lib.moe_expert_ffn_fp8_block_backward.argtypes = ([prob] + [P] * 11 + [i32, P, P, P, i32, i32, P,
                                                                               size, P])
        lib.moe_norm.argtypes = [i64, ctypes.c_int32, P, i32, P, P, f32, i32, P, i32, P, P]
        lib.moe_norm_workspace_bytes.argtypes = [i64, ctypes.c_int32]
        lib.moe_norm_workspace_bytes.restype = size
        lib.moe_norm_backward.argtypes = [i64, ctypes.c_int32, P, i32, P, i32, P, P, i32, P, i32, P, P, i32,
                                          P, size, P]
        for name in ("moe_quantize_rows_fp8_block", "moe_quantize_weights_fp8_block",
                     "moe_grouped_gemm_fp8_block", "moe_grouped_gemm_fp8_block_dgrad",
                     "moe_expert_gate_up_fp8_block", "moe_expert_ffn_fp8_block",
                     "moe_forward_fp8_block", "moe_expert_ffn_fp8_block_backward", "moe_norm",
                     "moe_norm_backward"):
            getattr(lib, name).restype = st
        lib.moe_peak_stream_read.argtypes = [P, ctypes.c_size_t, ctypes.c_int, P, ctypes.c_int, P]
        lib.moe_peak_stream_read.restype = st
        lib.moe_peak_mfma_bf16.argtypes = [ctypes.c_int64, ctypes.c_int, P, ctypes.c_int, P]
        lib.moe_peak_mfma_bf16.restype = st
        lib.moe_peak_mfma_bf16_flops.argtypes = [ctypes.c_int64, ctypes.c_int]
        lib.moe_peak_mfma_bf16_flops.restype = ctypes.c_double
        lib.moe_peak_mfma_stream.argtypes = [P, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, P,
                                             ctypes.c_int, P]
        lib.moe_peak_mfma_stream.restype = st
        lib.moe_peak_mfma_stream_flops.argtypes = [ctypes.c_int64, ctypes.c_int]
        lib.moe_peak_mfma_stream_flops.restype = ctypes.c_double
        lib.moe_peak_mfma_stream_bytes.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
        lib.moe_peak_mfma_stream_bytes.restype = ctypes.c_double
        lib.moe_status_string.argtypes = [ctypes.c_int]
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_last_error.argtypes = []
        lib.moe_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status):
    if status != MOE_OK:
        raise MoEError(status, load_library().moe_last_error().decode())


def _dtype_code(out):
    if isinstance(out, int):
        raise TypeError("out must be a tensor")
    if out.dtype == torch.float32:
        return DTYPE_F32
    if out.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"out dtype {out.dtype} is not float32/bfloat16")


def moe_workspace_bytes(p: MoEProblem) -> int:
    return int(load_library().moe_workspace_bytes(ctypes.byref(p)))


def moe_route(p, x, w_router, bias, topk_ids, topk_weights, stream=None):
    _check(load_library().moe_route(ctypes.byref(p), _p(x), _p(w_router), _p(bias), _p(topk_ids),
                                     _p(topk_weights), _stream(stream)))


def moe_permute(p, topk_ids, expert_offsets, sorted_pairs, pair_rows, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_permute(ctypes.byref(p), _p(topk_ids), _p(expert_offsets),
                                       _p(sorted_pairs), _p(pair_rows), _p(ws), nbytes,
                                       _stream(stream)))


def moe_expert_ffn(p, x, sorted_pairs, expert_offsets, w_gate, w_up, w_down, y, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_expert_ffn(ctypes.byref(p), _p(x), _p(sorted_pairs),
                                          _p(expert_offsets), _p(w_gate), _p(w_up), _p(w_down),
                                          _p(y), _p(ws), nbytes, _stream(stream)))


def moe_expert_gate_up(p, x, sorted_pairs, expert_offsets, w_gate, w_up, h, stream=None):
    _check(load_library().moe_expert_gate_up(ctypes.byref(p), _p(x), _p(sorted_pairs),
                                              _p(expert_offsets), _p(w_gate), _p(w_up), _p(h),
                                              _stream(stream)))


def moe_expert_down(p, h, expert_offsets, w_down, y, stream=None):
    _check(load_library().moe_expert_down(ctypes.byref(p), _p(h), _p(expert_offsets),
                                           _p(w_down), _p(y), _stream(stream)))


def moe_combine(p, y, pair_rows, topk_weights, out, stream=None):
    _check(load_library().moe_combine(ctypes.byref(p), _p(y), _p(pair_rows), _p(topk_weights),
                                       _p(out), _dtype_code(out), _stream(stream)))


def moe_combine_residual(p, y, pair_rows, topk_weights, norm_weight, eps, step, residual,
                         stream=None):
    _check(load_library().moe_combine_residual(ctypes.byref(p), _p(y), _p(pair_rows),
                                                _p(topk_weights), _p(norm_weight), float(eps),
                                                int(step), _p(residual), _stream(stream)))


def moe_expert_ffn_fp8(p, x, sorted_pairs, expert_offsets, q_gate, s_gate, q_up, s_up, q_down,
                       s_down, y, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_expert_ffn_fp8(ctypes.byref(p), _p(x), _p(sorted_pairs),
                                              _p(expert_offsets), _p(q_gate), _p(s_gate), _p(q_up),
                                              _p(s_up), _p(q_down), _p(s_down), _p(y), _p(ws),
                                              nbytes, _stream(stream)))


def moe_forward_fp8(p, x, w_router, bias, q_gate, s_gate, q_up, s_up, q_down, s_down, out,
                    topk_ids, topk_weights, y, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_forward_fp8(ctypes.byref(p), _p(x), _p(w_router), _p(bias),
                                           _p(q_gate), _p(s_gate), _p(q_up), _p(s_up), _p(q_down),
                                           _p(s_down), _p(out), _dtype_code(out), _p(topk_ids),
                                           _p(topk_weights), _p(y), _p(ws), nbytes,
                                           _stream(stream)))


def moe_dense_mlp(p, x, w_gate, w_up, w_down, out, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_dense_mlp(ctypes.byref(p), _p(x), _p(w_gate), _p(w_up), _p(w_down),
                                         _p(out), _p(ws), nbytes, _stream(stream)))


def moe_forward(p, x, w_router, bias, w_gate, w_up, w_down, out, topk_ids, topk_weights, y, ws,
                stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().moe_forward(ctypes.byref(p), _p(x), _p(w_router), _p(bias), _p(w_gate),
                                       _p(w_up), _p(w_down), _p(out), _dtype_code(out),
                                       _p(topk_ids), _p(topk_weights), _p(y), _p(ws), nbytes,
                                       _stream(stream)))


def moe_forward_noalloc(p, x, w_router, bias, w_gate, w_up, w_down, out, topk_ids, topk_weights,
                        y, stream=None):
    _check(load_library().moe_forward_noalloc(ctypes.byref(p), _p(x), _p(w_router), _p(bias),
                                               _p(w_gate), _p(w_up), _p(w_down), _p(out),
                                               _dtype_code(out), _p(topk_ids), _p(topk_weights),
                                               _p(y), _stream(stream)))


# ---- grouped products (include/moe_gemm.h) ----
#
# These also check what the C side cannot see: that each tensor has the type
# and at least the elements the call takes, is contiguous and lies on the
# current device.  The calls are as short as the kernels they launch, so the
# device is asked for once and the library's functions are looked up once.

_BF16, _F32, _I32, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _arg(t, name, dtype, n, device, nullable=False):
    """The device address of tensor t after those checks."""
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is None")
    if t.dtype is not dtype:
        raise TypeError(f"{name} dtype {t.dtype} is not {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the current GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, needs {n}")
    return t.data_ptr()


def _ws_args(ws, device):
    if ws is None:
        return None, 0
    return _arg(ws, "ws", ws.dtype, 0, device), ws.numel() * ws.element_size()


def _on(stream, device):
    """The handle of `stream` (the current one of the device if None)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if isinstance(stream, int):
        return stream
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, not on the current GPU")
    return stream.cuda_stream


def moe_gemm_workspace_bytes(g: MoEGemmProblem) -> int:
    return int(load_library().moe_gemm_workspace_bytes(g))


def moe_grouped_gemm(g, a, sorted_pairs, expert_offsets, w, out, ws=None, stream=None):
    """out [P,N] (fp32 or bf16) = a[row(q)] . w[e]^T for each position q."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, E, N, K = g.P, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm(
        g, _arg(a, "a", _BF16, g.S * K, dev), _arg(sorted_pairs, "sorted_pairs", _I32, P, dev, True),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _arg(w, "w", _BF16, E * N * K, dev), _arg(out, "out", out.dtype, P * N, dev),
        _dtype_code(out), wp, wn, _on(stream, dev)))


def moe_grouped_gemm_dgrad(g, dout, expert_offsets, w, da, ws=None, accumulate=False,
                           stream=None):
    """da [P,K] (fp32 or bf16) = dout[q] . w[e]; da += with accumulate."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, E, N, K = g.P, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm_dgrad(
        g, _arg(dout, "dout", _BF16, P * N, dev),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _arg(w, "w", _BF16, E * N * K, dev), _arg(da, "da", da.dtype, P * K, dev),
        _dtype_code(da), 1 if accumulate else 0, wp, wn, _on(stream, dev)))


def moe_grouped_gemm_wgrad(g, dout, a, sorted_pairs, expert_offsets, dw, ws=None,
                           accumulate=False, stream=None):
    """dw [E,N,K] (fp32 or bf16) = sum over each expert's positions of
    dout[q]^T a[row(q)]; dw += with accumulate."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, E, N, K = g.P, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm_wgrad(
        g, _arg(dout, "dout", _BF16, P * N, dev, P == 0),
        _arg(a, "a", _BF16, g.S * K if P else 0, dev, P == 0),
        _arg(sorted_pairs, "sorted_pairs", _I32, P, dev, True),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _arg(dw, "dw", dw.dtype, E * N * K, dev), _dtype_code(dw), 1 if accumulate else 0, wp, wn,
        _on(stream, dev)))


def moe_quantize_rows_int8(x, codes, scales, stream=None):
    """The rows of x [rows,K] bf16 as int8 codes [rows,K] and fp32 scales
    [rows] (amax / 127)."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, needs 2")
    rows, K = x.shape
    _check(lib.moe_quantize_rows_int8(
        rows, K, _arg(x, "x", _BF16, 0, dev), _arg(codes, "codes", _I8, rows * K, dev),
        _arg(scales, "scales", _F32, rows, dev), _on(stream, dev)))


def moe_grouped_gemm_int8(g, a, a_scale, sorted_pairs, expert_offsets, w, w_scale, out, ws=None,
                          stream=None):
    """out [P,N] (fp32 or bf16) = a_scale[row(q)] w_scale[e] (a[row(q)] .
    w[e]^T) on int8 codes."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, S, E, N, K = g.P, g.S, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm_int8(
        g, _arg(a, "a", _I8, S * K, dev), _arg(a_scale, "a_scale", _F32, S, dev),
        _arg(sorted_pairs, "sorted_pairs", _I32, P, dev, True),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _arg(w, "w", _I8, E * N * K, dev), _arg(w_scale, "w_scale", _F32, E * N, dev),
        _arg(out, "out", out.dtype, P * N, dev), _dtype_code(out), wp, wn, _on(stream, dev)))


def moe_int8_workspace_bytes(p: MoEProblem) -> int:
    return int(load_library().moe_int8_workspace_bytes(p))


def _int8_weights(p, dev, q_gate, s_gate, q_up, s_up, q_down, s_down):
    n, gate, down = p.E * p.I * p.H, p.E * p.I, p.E * p.H
    return (_arg(q_gate, "q_gate", _I8, n, dev), _arg(s_gate, "s_gate", _F32, gate, dev),
            _arg(q_up, "q_up", _I8, n, dev), _arg(s_up, "s_up", _F32, gate, dev),
            _arg(q_down, "q_down", _I8, n, dev), _arg(s_down, "s_down", _F32, down, dev))


def moe_expert_ffn_int8(p, x, sorted_pairs, expert_offsets, q_gate, s_gate, q_up, s_up, q_down,
                        s_down, y, ws, stream=None):
    """The experts in 8-bit integers: y [T*k,H] fp32 in sorted order."""
    dev = torch.cuda.current_device()
    P = p.T * p.k
    wp, wn = _ws_args(ws, dev)
    _check(load_library().moe_expert_ffn_int8(
        p, _arg(x, "x", _BF16, p.T * p.H, dev), _arg(sorted_pairs, "sorted_pairs", _I32, P, dev),
        _arg(expert_offsets, "expert_offsets", _I32, p.E + 1, dev),
        *_int8_weights(p, dev, q_gate, s_gate, q_up, s_up, q_down, s_down),
        _arg(y, "y", _F32, P * p.H, dev), wp, wn, _on(stream, dev)))


def moe_forward_int8(p, x, w_router, bias, q_gate, s_gate, q_up, s_up, q_down, s_down, out,
                     topk_ids, topk_weights, y, ws, stream=None):
    """moe_forward with the experts in 8-bit integers."""
    dev = torch.cuda.current_device()
    P = p.T * p.k
    wp, wn = _ws_args(ws, dev)
    _check(load_library().moe_forward_int8(
        p, _arg(x, "x", _BF16, p.T * p.H, dev), _arg(w_router, "w_router", _BF16, p.E * p.H, dev),
        _arg(bias, "bias", _F32, p.E, dev, True),
        *_int8_weights(p, dev, q_gate, s_gate, q_up, s_up, q_down, s_down),
        _arg(out, "out", out.dtype, p.T * p.H, dev), _dtype_code(out),
        _arg(topk_ids, "topk_ids", _I32, P, dev, True),
        _arg(topk_weights, "topk_weights", _F32, P, dev, True), _arg(y, "y", _F32, P * p.H, dev),
        wp, wn, _on(stream, dev)))


def moe_backward_workspace_bytes(p: MoEProblem) -> int:
    return int(load_library().moe_backward_workspace_bytes(p))


def moe_expert_ffn_backward(p, x, sorted_pairs, expert_offsets, w_gate, w_up, w_down, dy, dx,
                            dw_gate, dw_up, dw_down, ws, accumulate=False, stream=None):
    """The gradients of moe_expert_ffn from dy [T*k,H] bf16: dx [T*k,H] fp32,
    both in sorted order, and dw_gate, dw_up [E,I,H], dw_down [E,H,I] (fp32 or
    bf16; += with accumulate)."""
    dev = torch.cuda.current_device()
    P, n, empty = p.T * p.k, p.E * p.I * p.H, p.T == 0
    wp, wn = _ws_args(ws, dev)
    _check(load_library().moe_expert_ffn_backward(
        p, _arg(x, "x", _BF16, p.T * p.H, dev, empty),
        _arg(sorted_pairs, "sorted_pairs", _I32, P, dev, empty),
        _arg(expert_offsets, "expert_offsets", _I32, p.E + 1, dev, empty and p.E == 1),
        _arg(w_gate, "w_gate", _BF16, n, dev), _arg(w_up, "w_up", _BF16, n, dev),
        _arg(w_down, "w_down", _BF16, n, dev), _arg(dy, "dy", _BF16, P * p.H, dev, empty),
        _arg(dx, "dx", _F32, P * p.H, dev, empty), _arg(dw_gate, "dw_gate", dw_gate.dtype, n, dev),
        _arg(dw_up, "dw_up", dw_gate.dtype, n, dev),
        _arg(dw_down, "dw_down", dw_gate.dtype, n, dev), _dtype_code(dw_gate),
        1 if accumulate else 0, wp, wn, _on(stream, dev)))


# ---- experts in FP8 with a scale for each block of 128 (include/moe_fp8.h) ----
#
# Codes are torch.float8_e4m3fn or, the same bytes, torch.uint8; scales (the
# exponent of a power of two + 127) torch.uint8.

_U8, _E4M3 = torch.uint8, torch.float8_e4m3fn


def _codes(t, name, n, device, nullable=False):
    if t is None or t.dtype is _U8:
        return _arg(t, name, _U8, n, device, nullable)
    return _arg(t, name, _E4M3, n, device, nullable)


def _blocks(n):
    return (n + 127) // 128


def moe_fp8_block_scales(C) -> int:
    """Bytes of a row's scales for C columns."""
    return int(load_library().moe_fp8_block_scales(C))


def _pitch(C):
    return (_blocks(C) + 3) // 4 * 4


def moe_quantize_rows_fp8_block(x, codes, scales, stream=None):
    """The rows of x [rows,K] bf16 as e4m3 codes [rows,K] and scales
    [rows,moe_fp8_block_scales(K)], one for each 128 columns."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, needs 2")
    rows, K = x.shape
    _check(lib.moe_quantize_rows_fp8_block(
        rows, K, _arg(x, "x", _BF16, 0, dev), _codes(codes, "codes", rows * K, dev),
        _arg(scales, "scales", _U8, rows * _pitch(K), dev), _on(stream, dev)))


def moe_quantize_weights_fp8_block(w, codes, scales, stream=None):
    """The matrices w [E,N,K] bf16 as e4m3 codes [E,N,K] and scales
    [E,ceil(N/128),ceil(K/128)], one for each 128 x 128."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    if w.dim() != 3:
        raise ValueError(f"w has {w.dim()} dimensions, needs 3")
    E, N, K = w.shape
    _check(lib.moe_quantize_weights_fp8_block(
        E, N, K, _arg(w, "w", _BF16, 0, dev), _codes(codes, "codes", E * N * K, dev),
        _arg(scales, "scales", _U8, E * _blocks(N) * _blocks(K), dev), _on(stream, dev)))


def moe_grouped_gemm_fp8_block(g, a, a_scale, sorted_pairs, expert_offsets, w, w_scale, out,
                               ws=None, stream=None):
    """out [P,N] (fp32 or bf16) = a[row(q)] . w[e]^T on dequantised codes."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, S, E, N, K = g.P, g.S, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm_fp8_block(
        g, _codes(a, "a", S * K, dev), _arg(a_scale, "a_scale", _U8, S * _pitch(K), dev),
        _arg(sorted_pairs, "sorted_pairs", _I32, P, dev, True),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _codes(w, "w", E * N * K, dev), _arg(w_scale, "w_scale", _U8, E * _blocks(N) * _blocks(K), dev),
        _arg(out, "out", out.dtype, P * N, dev), _dtype_code(out), wp, wn, _on(stream, dev)))


def moe_grouped_gemm_fp8_block_dgrad(g, dout, dout_scale, expert_offsets, w, w_scale, da, ws=None,
                                     accumulate=False, stream=None):
    """da [P,K] (fp32 or bf16) = dout[q] . w[e] on dequantised codes; da +=
    with accumulate."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, E, N, K = g.P, g.E, g.N, g.K
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_grouped_gemm_fp8_block_dgrad(
        g, _codes(dout, "dout", P * N, dev), _arg(dout_scale, "dout_scale", _U8, P * _pitch(N), dev),
        _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev, E == 1),
        _codes(w, "w", E * N * K, dev), _arg(w_scale, "w_scale", _U8, E * _blocks(N) * _blocks(K), dev),
        _arg(da, "da", da.dtype, P * K, dev), _dtype_code(da), 1 if accumulate else 0, wp, wn,
        _on(stream, dev)))


def _fp8_matrix(p, dev, q, s, name):
    n = p.E * p.I * p.H
    return (_codes(q, "q_" + name, n, dev),
            _arg(s, "s_" + name, _U8, p.E * _blocks(p.I) * _blocks(p.H), dev))


def _fp8_dispatch(p, dev, sorted_pairs, expert_offsets):
    dense = p.E == 1 and p.k == 1
    return (_arg(sorted_pairs, "sorted_pairs", _I32, p.T * p.k, dev, dense),
            _arg(expert_offsets, "expert_offsets", _I32, p.E + 1, dev, dense))


def moe_expert_gate_up_fp8_block(p, x, x_scale, sorted_pairs, expert_offsets, q_gate, s_gate, q_up,
                                 s_up, h, h_scale, stream=None):
    """h = silu(x . gate^T) (x . up^T) by position, quantised by rows: codes
    [T*k,I] and scales [T*k,moe_fp8_block_scales(I)], from x as codes [T,H] and
    scales."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P = p.T * p.k
    _check(lib.moe_expert_gate_up_fp8_block(
        p, _codes(x, "x", p.T * p.H, dev), _arg(x_scale, "x_scale", _U8, p.T * _pitch(p.H), dev),
        *_fp8_dispatch(p, dev, sorted_pairs, expert_offsets), *_fp8_matrix(p, dev, q_gate, s_gate, "gate"),
        *_fp8_matrix(p, dev, q_up, s_up, "up"), _codes(h, "h", P * p.I, dev),
        _arg(h_scale, "h_scale", _U8, P * _pitch(p.I), dev), _on(stream, dev)))


def moe_fp8_block_workspace_bytes(p: MoEProblem) -> int:
    return int(load_library().moe_fp8_block_workspace_bytes(p))


def moe_expert_ffn_fp8_block(p, x, sorted_pairs, expert_offsets, q_gate, s_gate, q_up, s_up, q_down,
                             s_down, y, ws, stream=None):
    """The experts in FP8: y [T*k,H] (fp32 or bf16) in sorted order from x
    [T,H] bf16."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_expert_ffn_fp8_block(
        p, _arg(x, "x", _BF16, p.T * p.H, dev), *_fp8_dispatch(p, dev, sorted_pairs, expert_offsets),
        *_fp8_matrix(p, dev, q_gate, s_gate, "gate"), *_fp8_matrix(p, dev, q_up, s_up, "up"),
        *_fp8_matrix(p, dev, q_down, s_down, "down"), _arg(y, "y", y.dtype, p.T * p.k * p.H, dev),
        _dtype_code(y), wp, wn, _on(stream, dev)))


def moe_forward_fp8_block(p, x, w_router, bias, q_gate, s_gate, q_up, s_up, q_down, s_down, out,
                          topk_ids, topk_weights, y, ws, stream=None):
    """moe_forward with the experts in FP8 by blocks."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P = p.T * p.k
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_forward_fp8_block(
        p, _arg(x, "x", _BF16, p.T * p.H, dev), _arg(w_router, "w_router", _BF16, p.E * p.H, dev),
        _arg(bias, "bias", _F32, p.E, dev, True), *_fp8_matrix(p, dev, q_gate, s_gate, "gate"),
        *_fp8_matrix(p, dev, q_up, s_up, "up"), *_fp8_matrix(p, dev, q_down, s_down, "down"),
        _arg(out, "out", out.dtype, p.T * p.H, dev), _dtype_code(out),
        _arg(topk_ids, "topk_ids", _I32, P, dev, True),
        _arg(topk_weights, "topk_weights", _F32, P, dev, True), _arg(y, "y", _F32, P * p.H, dev),
        wp, wn, _on(stream, dev)))


def moe_fp8_block_backward_workspace_bytes(p: MoEProblem) -> int:
    return int(load_library().moe_fp8_block_backward_workspace_bytes(p))


def moe_expert_ffn_fp8_block_backward(p, x, sorted_pairs, expert_offsets, q_gate, s_gate, q_up, s_up,
                                      q_down, s_down, dy, dx, dw_gate, dw_up, dw_down, ws,
                                      accumulate=False, stream=None):
    """The gradients of moe_expert_ffn_fp8_block from dy [T*k,H] bf16: dx
    [T*k,H] (fp32 or bf16), both in sorted order, and dw_gate, dw_up [E,I,H],
    dw_down [E,H,I] (all fp32 or all bf16; += with accumulate)."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    P, n, empty = p.T * p.k, p.E * p.I * p.H, p.T == 0
    wp, wn = _ws_args(ws, dev)
    dispatch = (None, None) if empty else _fp8_dispatch(p, dev, sorted_pairs, expert_offsets)
    if empty:
        dispatch = (None, _arg(expert_offsets, "expert_offsets", _I32, p.E + 1, dev, p.E == 1))
    _check(lib.moe_expert_ffn_fp8_block_backward(
        p, _arg(x, "x", _BF16, p.T * p.H, dev, empty), *dispatch,
        *_fp8_matrix(p, dev, q_gate, s_gate, "gate"), *_fp8_matrix(p, dev, q_up, s_up, "up"),
        *_fp8_matrix(p, dev, q_down, s_down, "down"), _arg(dy, "dy", _BF16, P * p.H, dev, empty),
        None if dx is None and empty else _arg(dx, "dx", dx.dtype, P * p.H, dev),
        DTYPE_F32 if dx is None and empty else _dtype_code(dx),
        _arg(dw_gate, "dw_gate", dw_gate.dtype, n, dev), _arg(dw_up, "dw_up", dw_gate.dtype, n, dev),
        _arg(dw_down, "dw_down", dw_gate.dtype, n, dev), _dtype_code(dw_gate),
        1 if accumulate else 0, wp, wn, _on(stream, dev)))


# ---- the norm in front of the block (include/moe_norm.h) ----


def _rows_of(x, name):
    if x.dim() != 2:
        raise ValueError(f"{name} has {x.dim()} dimensions, needs 2")
    return x.shape


def moe_norm(x, weight, bias, eps, out, stats=None, center=False, stream=None):
    """out = (x - mean) / sqrt(var + eps) weight + bias by rows of x [rows,H]
    (fp32 or bf16); without center the mean is left out (RMS norm).  stats
    [rows,2] fp32 takes mean and 1 / sqrt(var + eps) for moe_norm_backward."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    rows, H = _rows_of(x, "x")
    _check(lib.moe_norm(
        rows, H, _arg(x, "x", x.dtype, 0, dev), _dtype_code(x), _arg(weight, "weight", _F32, H, dev),
        _arg(bias, "bias", _F32, H, dev, True), eps, 1 if center else 0,
        _arg(out, "out", out.dtype, rows * H, dev), _dtype_code(out),
        _arg(stats, "stats", _F32, rows * 2, dev, True), _on(stream, dev)))


def moe_norm_workspace_bytes(rows, H) -> int:
    return int(load_library().moe_norm_workspace_bytes(rows, H))


def moe_norm_backward(dy, x, weight, stats, dx, dweight, dbias, ws, center=False, accumulate=False,
                      stream=None):
    """The gradients of moe_norm from dy [rows,H] and what the forward call was
    given and wrote: dx [rows,H], dweight [H] and dbias [H] (or None) fp32 (+=
    with accumulate)."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    rows, H = _rows_of(x, "x")
    wp, wn = _ws_args(ws, dev)
    _check(lib.moe_norm_backward(
        rows, H, _arg(dy, "dy", dy.dtype, rows * H, dev), _dtype_code(dy), _arg(x, "x", x.dtype, 0, dev),
        _dtype_code(x), _arg(weight, "weight", _F32, H, dev), _arg(stats, "stats", _F32, rows * 2, dev),
        1 if center else 0, _arg(dx, "dx", dx.dtype, rows * H, dev), _dtype_code(dx),
        _arg(dweight, "dweight", _F32, H, dev), _arg(dbias, "dbias", _F32, H, dev, True),
        1 if accumulate else 0, wp, wn, _on(stream, dev)))


def moe_peak_stream_read(buf, sink, workgroups, nontemporal=False, stream=None):
    """One streaming read of the whole of `buf` (a GPU tensor) by the
    measurement kernel; `sink` is a GPU tensor of at least 4 bytes."""
    nbytes = buf.numel() * buf.element_size()
    _check(load_library().moe_peak_stream_read(_p(buf), nbytes, int(bool(nontemporal)), _p(sink),
                                                int(workgroups), _stream(stream)))


def moe_peak_mfma_bf16(iters, sink, workgroups, random_operands=True, stream=None):
    """The back-to-back bf16 MFMA loop on pseudo-random (default) or fixed
    register operands; `sink` holds 4 * workgroups floats.  Returns the FLOPs
    of the call."""
    lib = load_library()
    _check(lib.moe_peak_mfma_bf16(int(iters), int(bool(random_operands)), _p(sink),
                                  int(workgroups), _stream(stream)))
    return float(lib.moe_peak_mfma_bf16_flops(int(iters), int(workgroups)))


def moe_peak_mfma_stream(buf, loads_per_step, steps, sink, workgroups, stream=None):
    """LDS-fed bf16 MFMAs with `loads_per_step` 16-byte HBM loads a lane per
    step from `buf` (a GPU tensor, or None with 0 loads); `sink` holds
    4 * workgroups floats.  Returns (FLOPs, bytes) of the call."""
    lib = load_library()
    nbytes = 0 if buf is None else buf.numel() * buf.element_size()
    _check(lib.moe_peak_mfma_stream(_p(buf) if buf is not None else None, nbytes,
                                    int(loads_per_step), int(steps), _p(sink), int(workgroups),
                                    _stream(stream)))
    return (float(lib.moe_peak_mfma_stream_flops(int(steps), int(workgroups))),
            float(lib.moe_peak_mfma_stream_bytes(int(steps), int(loads_per_step), int(workgroups))))


def alloc_buffers(p: MoEProblem, device="cuda", out_dtype=torch.float32):
    """Caller-side buffers for one forward pass (torch allocations)."""
    T, k, H, E = p.T, p.k, p.H, p.E
    ws_bytes = moe_workspace_bytes(p)
    if ws_bytes == 0 and T > 0:
        raise MoEError(1, load_library().moe_last_error().decode())
    return dict(
        out=torch.empty((T, H), dtype=out_dtype, device=device),
        topk_ids=torch.empty((T, k), dtype=torch.int32, device=device),
        topk_weights=torch.empty((T, k), dtype=torch.float32, device=device),
        expert_offsets=torch.empty((E + 1,), dtype=torch.int32, device=device),
        sorted_pairs=torch.empty((T * k,), dtype=torch.int32, device=device),
        pair_rows=torch.empty((T * k,), dtype=torch.int32, device=device),
        y=torch.empty((T * k, H), dtype=torch.float32, device=device),
        h=torch.empty((T * k, p.I), dtype=torch.bfloat16, device=device),
        ws=torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=device),
    )
