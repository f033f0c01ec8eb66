"""ctypes binding of ``libnvfp4_gemv.so`` (argument marshalling only).

Each C entry point of ``include/nvfp4_gemv.h``, ``include/nvfp4_quantize.h``,
``include/nvfp4_mma.h`` and ``include/nvfp4_ffn.h`` has a Python function of
the same name.  Pointer arguments accept a torch tensor (its ``data_ptr()``), a raw
integer device address, or None where the C side allows NULL; ``stream``
accepts None (torch's current stream), a ``torch.cuda.Stream`` or a raw
``hipStream_t`` integer.  A negative status raises :class:`Nvfp4GemvError`.
All arithmetic happens in the HIP kernels; nothing here falls back to the CPU.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnvfp4_gemv.so")

NVFP4_GEMV_OK = 0
NVFP4_GEMV_ERR_NULL_POINTER = -1
NVFP4_GEMV_ERR_BAD_SHAPE = -2
NVFP4_GEMV_ERR_WORKSPACE = -3
NVFP4_GEMV_ERR_LAUNCH = -4
NVFP4_GEMV_ERR_ALIAS = -5
NVFP4_GEMV_ERR_ALIGNMENT = -6
NVFP4_GEMV_ERR_DEVICE = -7
NVFP4_GEMV_ERR_BAD_TUNING = -8
NVFP4_GEMV_ERR_BAD_ARGUMENT = -9

NVFP4_ROUND_HALF_STEP = 0
NVFP4_ROUND_NEAREST_EVEN = 1
NVFP4_ROUND_NEAREST_LOWER = 2

NVFP4_OUT_F16 = 0
NVFP4_OUT_BF16 = 1
NVFP4_OUT_F32 = 2

NVFP4_W_ROW_MAJOR = 0
NVFP4_W_PACKED = 1

NVFP4_ACT_NONE = 0
NVFP4_ACT_RELU = 1
NVFP4_ACT_GELU = 2
NVFP4_ACT_GELU_TANH = 3
NVFP4_ACT_SILU = 4
NVFP4_ACT_GATED = 16

NVFP4_SCORE_SOFTMAX = 0
NVFP4_SCORE_SIGMOID = 1

NVFP4_MMA_FORM_MATRIX_CORES = 0
NVFP4_MMA_FORM_VALU_TILES = 1
NVFP4_MMA_FORM_LDS_STAGED = 2
NVFP4_MMA_FORM_LDS_VECTOR_REGS = 3

NVFP4_GEMV_PATH_AUTO = 0
NVFP4_GEMV_PATH_FAST = 1
NVFP4_GEMV_PATH_GENERIC = 2

NVFP4_GEMV_NOALLOC_SCRATCH_BYTES = 4 << 20

# Every symbol the header declares.
EXPORTED = (
    "nvfp4_gemv_status_string",
    "nvfp4_gemv_launch",
    "nvfp4_gemv_workspace_size",
    "nvfp4_gemv_launch_ws",
    "nvfp4_gemv_num_variants",
    "nvfp4_gemv_variant_info",
    "nvfp4_gemv_plan",
    "nvfp4_gemv_launch_tuned",
    "nvfp4_hbm_read_probe",
    "nvfp4_hbm_read_probe_rows",
    "nvfp4_workspace_reserve",
    "nvfp4_gemv_launch_noalloc",
    "nvfp4_quantize_activation",
    "nvfp4_quantize_weight",
    "nvfp4_gemv_bf16x_launch",
    "nvfp4_gemm_smalln_launch",
    "nvfp4_mma_num_variants",
    "nvfp4_mma_variant_info",
    "nvfp4_mma_variant_form",
    "nvfp4_gemm_smalln_plan",
    "nvfp4_grouped_gemv_plan",
    "nvfp4_gemm_smalln_launch_tuned",
    "nvfp4_grouped_gemv_launch",
    "nvfp4_grouped_gemv_launch_tuned",
    "nvfp4_mma_packed_sizes",
    "nvfp4_mma_pack_weight",
    "nvfp4_gemm_smalln_launch_packed",
    "nvfp4_grouped_gemv_launch_packed",
    "nvfp4_linear_workspace_size",
    "nvfp4_linear_launch_ws",
    "nvfp4_linear_launch",
    "nvfp4_moe_layer_workspace_size",
    "nvfp4_moe_layer_launch_ws",
    "nvfp4_moe_layer_launch",
)


class Nvfp4GemvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({nvfp4_gemv_status_string(status)})")


class Tuning(ctypes.Structure):
    """Mirror of ``nvfp4_gemv_tuning_t``."""
    _fields_ = [("path", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("ksplit", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def __repr__(self):
        return f"Tuning(path={self.path}, variant={self.variant}, ksplit={self.ksplit})"


class MmaTuning(ctypes.Structure):
    """Mirror of ``nvfp4_mma_tuning_t``."""
    _fields_ = [("path", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("ksplit", ctypes.c_int32), ("rows_per_block", ctypes.c_int32)]

    def __repr__(self):
        return (f"MmaTuning(path={self.path}, variant={self.variant}, ksplit={self.ksplit}, "
                f"rows_per_block={self.rows_per_block})")


class MoeLayerStruct(ctypes.Structure):
    """Mirror of ``nvfp4_moe_layer_t``."""
    _fields_ = [("router", ctypes.c_void_p), ("route_bias", ctypes.c_void_p),
                ("W13", ctypes.c_void_p), ("sf13", ctypes.c_void_p), ("alpha13", ctypes.c_void_p),
                ("W2", ctypes.c_void_p), ("sf2", ctypes.c_void_p), ("alpha2", ctypes.c_void_p),
                ("experts", ctypes.c_int64), ("hidden", ctypes.c_int64), ("inter", ctypes.c_int64),
                ("topk", ctypes.c_int32), ("x_type", ctypes.c_int32), ("w_layout", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64


def load():
    """Load the built library; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m precision_decode_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.nvfp4_gemv_status_string.restype = ctypes.c_char_p
    lib.nvfp4_gemv_status_string.argtypes = [ctypes.c_int]
    gemv_args = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64]
    lib.nvfp4_gemv_launch.restype = ctypes.c_int
    lib.nvfp4_gemv_launch.argtypes = gemv_args + [_P]
    lib.nvfp4_gemv_workspace_size.restype = ctypes.c_size_t
    lib.nvfp4_gemv_workspace_size.argtypes = [_I64, _I64, _I64]
    lib.nvfp4_gemv_launch_ws.restype = ctypes.c_int
    lib.nvfp4_gemv_launch_ws.argtypes = gemv_args + [_P, ctypes.c_size_t, _P]
    lib.nvfp4_gemv_num_variants.restype = ctypes.c_int
    lib.nvfp4_gemv_num_variants.argtypes = []
    lib.nvfp4_gemv_variant_info.restype = ctypes.c_int
    lib.nvfp4_gemv_variant_info.argtypes = [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int32)] * 4
    lib.nvfp4_gemv_plan.restype = ctypes.c_int
    lib.nvfp4_gemv_plan.argtypes = [_I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(Tuning),
                                    ctypes.POINTER(Tuning), ctypes.POINTER(ctypes.c_size_t)]
    lib.nvfp4_gemv_launch_tuned.restype = ctypes.c_int
    lib.nvfp4_gemv_launch_tuned.argtypes = gemv_args + [ctypes.POINTER(Tuning), _P, ctypes.c_size_t, _P]
    lib.nvfp4_gemv_launch_noalloc.restype = ctypes.c_int
    lib.nvfp4_gemv_launch_noalloc.argtypes = gemv_args + [_P]
    lib.nvfp4_workspace_reserve.restype = ctypes.c_int
    lib.nvfp4_workspace_reserve.argtypes = [ctypes.c_size_t, _P]
    lib.nvfp4_hbm_read_probe_rows.restype = ctypes.c_int
    lib.nvfp4_hbm_read_probe_rows.argtypes = [_P, _P, _I64, _I64, _P, _P]
    lib.nvfp4_hbm_read_probe.restype = ctypes.c_int
    lib.nvfp4_hbm_read_probe.argtypes = [_P, ctypes.c_size_t, _P, _P]
    lib.nvfp4_quantize_activation.restype = ctypes.c_int
    lib.nvfp4_quantize_activation.argtypes = [_P, _P, ctypes.c_int32, _P, _P, _I64, _I64,
                                              ctypes.c_int32, _P]
    lib.nvfp4_quantize_weight.restype = ctypes.c_int
    lib.nvfp4_quantize_weight.argtypes = [_P, _I64, _I64, _I64, ctypes.c_int32, _P, _P, _P, _P]
    lib.nvfp4_gemv_bf16x_launch.restype = ctypes.c_int
    lib.nvfp4_gemv_bf16x_launch.argtypes = [_P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P,
                                            _I64, _I64, _I64, _P]
    smalln_args = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int32]
    lib.nvfp4_gemm_smalln_launch.restype = ctypes.c_int
    lib.nvfp4_gemm_smalln_launch.argtypes = smalln_args + [_P]
    lib.nvfp4_mma_num_variants.restype = ctypes.c_int
    lib.nvfp4_mma_num_variants.argtypes = []
    lib.nvfp4_mma_variant_info.restype = ctypes.c_int
    lib.nvfp4_mma_variant_info.argtypes = [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int32)] * 3
    lib.nvfp4_mma_variant_form.restype = ctypes.c_int
    lib.nvfp4_mma_variant_form.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int32)]
    lib.nvfp4_grouped_gemv_plan.restype = ctypes.c_int
    lib.nvfp4_grouped_gemv_plan.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int,
                                            ctypes.POINTER(MmaTuning), ctypes.POINTER(MmaTuning)]
    lib.nvfp4_gemm_smalln_plan.restype = ctypes.c_int
    lib.nvfp4_gemm_smalln_plan.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int,
                                           ctypes.POINTER(MmaTuning), ctypes.POINTER(MmaTuning),
                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.nvfp4_gemm_smalln_launch_tuned.restype = ctypes.c_int
    lib.nvfp4_gemm_smalln_launch_tuned.argtypes = smalln_args + [ctypes.POINTER(MmaTuning), _P,
                                                                 ctypes.c_size_t, _P]
    grouped_args = [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int32]
    lib.nvfp4_grouped_gemv_launch.restype = ctypes.c_int
    lib.nvfp4_grouped_gemv_launch.argtypes = grouped_args + [_P]
    lib.nvfp4_grouped_gemv_launch_tuned.restype = ctypes.c_int
    lib.nvfp4_grouped_gemv_launch_tuned.argtypes = grouped_args + [ctypes.POINTER(MmaTuning), _P]
    lib.nvfp4_mma_packed_sizes.restype = ctypes.c_int
    lib.nvfp4_mma_packed_sizes.argtypes = [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_size_t)]
    lib.nvfp4_mma_pack_weight.restype = ctypes.c_int
    lib.nvfp4_mma_pack_weight.argtypes = [_P, _P, _I64, _I64, _I64, _P, _P, _P]
    lib.nvfp4_gemm_smalln_launch_packed.restype = ctypes.c_int
    lib.nvfp4_gemm_smalln_launch_packed.argtypes = smalln_args + [ctypes.POINTER(MmaTuning), _P]
    lib.nvfp4_grouped_gemv_launch_packed.restype = ctypes.c_int
    lib.nvfp4_grouped_gemv_launch_packed.argtypes = grouped_args + [ctypes.POINTER(MmaTuning), _P]
    I32 = ctypes.c_int32
    linear_args = [_P, I32, _I64, _P, _P, I32, _P, _P, _P, _I64, _P, I32, _I64, _I64, _I64, _I64, I32]
    lib.nvfp4_linear_workspace_size.restype = ctypes.c_size_t
    lib.nvfp4_linear_workspace_size.argtypes = [_I64, _I64, _I64, I32]
    lib.nvfp4_linear_launch_ws.restype = ctypes.c_int
    lib.nvfp4_linear_launch_ws.argtypes = linear_args + [_P, ctypes.c_size_t, _P]
    lib.nvfp4_linear_launch.restype = ctypes.c_int
    lib.nvfp4_linear_launch.argtypes = linear_args + [_P]
    moe_args = [ctypes.POINTER(MoeLayerStruct), _P, _I64, _P, _I64, _P, I32, _I64, _I64]
    lib.nvfp4_moe_layer_workspace_size.restype = ctypes.c_size_t
    lib.nvfp4_moe_layer_workspace_size.argtypes = [ctypes.POINTER(MoeLayerStruct), _I64]
    lib.nvfp4_moe_layer_launch_ws.restype = ctypes.c_int
    lib.nvfp4_moe_layer_launch_ws.argtypes = moe_args + [_P, ctypes.c_size_t, _P]
    lib.nvfp4_moe_layer_launch.restype = ctypes.c_int
    lib.nvfp4_moe_layer_launch.argtypes = moe_args + [_P]
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not getattr(t, "is_cuda", False):
        raise ValueError("device pointer expected: pass a CUDA/HIP tensor or an integer address")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        if torch.cuda.is_initialized():
            # the handle itself: building a Stream object around it takes longer than a launch
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current(device, stream):
    """Context with that GPU current, for a call on ``stream``."""
    import torch

    if stream is not None and isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise ValueError(f"stream is on GPU {stream.device_index}, the tensors on GPU {device}")
    return contextlib.nullcontext() if torch._C._cuda_getDevice() == device else torch.cuda.device(device)


def _allocate(shape, dtype, device, stream):
    """Tensor allocated on the stream that writes it: memory of another stream's tensors
    may still be in use by work queued there."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                           torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _enqueue(call, args, device, stream, where):
    """Makes the C call with the GPU that holds the tensors current, on ``stream``."""
    import torch

    handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if stream is None and torch._C._cuda_getDevice() == device:
        status = call(*args, handle)
    else:
        with _current(device, stream):
            status = call(*args, handle)
    _check(status, where)


def _check(status: int, where: str):
    if status != NVFP4_GEMV_OK:
        raise Nvfp4GemvError(status, where)


def nvfp4_gemv_status_string(status: int) -> str:
    return load().nvfp4_gemv_status_string(int(status)).decode()


def nvfp4_gemv_launch(A_packed, sfA, x_packed, sfx, alpha, c, l, m, k, stream=None):
    st = load().nvfp4_gemv_launch(_ptr(A_packed), _ptr(sfA), _ptr(x_packed), _ptr(sfx),
                                  _ptr(alpha), _ptr(c), l, m, k, _stream(stream))
    _check(st, "nvfp4_gemv_launch")


def nvfp4_gemv_workspace_size(l, m, k) -> int:
    return int(load().nvfp4_gemv_workspace_size(l, m, k))


def nvfp4_gemv_launch_ws(A_packed, sfA, x_packed, sfx, alpha, c, l, m, k, workspace,
                         workspace_bytes, stream=None):
    st = load().nvfp4_gemv_launch_ws(_ptr(A_packed), _ptr(sfA), _ptr(x_packed), _ptr(sfx),
                                     _ptr(alpha), _ptr(c), l, m, k, _ptr(workspace),
                                     int(workspace_bytes), _stream(stream))
    _check(st, "nvfp4_gemv_launch_ws")


def nvfp4_gemv_num_variants() -> int:
    return int(load().nvfp4_gemv_num_variants())


def nvfp4_gemv_variant_info(v: int):
    """(rows per wave, iterations in flight, waves per group, x staging: 0 fp16 in LDS,
    1 packed codes in LDS, 2 none)."""
    r, u, w, px = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().nvfp4_gemv_variant_info(v, ctypes.byref(r), ctypes.byref(u), ctypes.byref(w),
                                          ctypes.byref(px)), "nvfp4_gemv_variant_info")
    return r.value, u.value, w.value, px.value


def _tuning(t):
    if t is None:
        return None
    if isinstance(t, Tuning):
        return ctypes.byref(t)
    return ctypes.byref(Tuning(int(t.get("path", 0)), int(t.get("variant", 0)),
                               int(t.get("ksplit", 0)), 0))


def _mma_tuning(t):
    if t is None:
        return None
    if isinstance(t, MmaTuning):
        return ctypes.byref(t)
    return ctypes.byref(MmaTuning(int(t.get("path", 0)), int(t.get("variant", 0)),
                                  int(t.get("ksplit", 0)), int(t.get("rows_per_block", 0))))


def nvfp4_gemv_plan(l, m, k, aligned=True, tuning=None):
    """Returns (Tuning actually used, workspace bytes)."""
    out = Tuning()
    ws = ctypes.c_size_t()
    _check(load().nvfp4_gemv_plan(l, m, k, int(bool(aligned)), _tuning(tuning), ctypes.byref(out),
                                  ctypes.byref(ws)), "nvfp4_gemv_plan")
    return out, int(ws.value)


def nvfp4_gemv_launch_tuned(A_packed, sfA, x_packed, sfx, alpha, c, l, m, k, tuning, workspace,
                            workspace_bytes, stream=None):
    st = load().nvfp4_gemv_launch_tuned(_ptr(A_packed), _ptr(sfA), _ptr(x_packed), _ptr(sfx),
                                        _ptr(alpha), _ptr(c), l, m, k, _tuning(tuning),
                                        _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "nvfp4_gemv_launch_tuned")


def nvfp4_gemv_launch_noalloc(A_packed, sfA, x_packed, sfx, alpha, c, l, m, k, stream=None):
    st = load().nvfp4_gemv_launch_noalloc(_ptr(A_packed), _ptr(sfA), _ptr(x_packed), _ptr(sfx),
                                          _ptr(alpha), _ptr(c), l, m, k, _stream(stream))
    _check(st, "nvfp4_gemv_launch_noalloc")


def nvfp4_workspace_reserve(nbytes, stream=None):
    _check(load().nvfp4_workspace_reserve(int(nbytes), _stream(stream)), "nvfp4_workspace_reserve")


def nvfp4_hbm_read_probe(buffer, nbytes, sink, stream=None):
    _check(load().nvfp4_hbm_read_probe(_ptr(buffer), int(nbytes), _ptr(sink), _stream(stream)),
           "nvfp4_hbm_read_probe")


def nvfp4_hbm_read_probe_rows(A, sfA, rows, k, sink, stream=None):
    _check(load().nvfp4_hbm_read_probe_rows(_ptr(A), _ptr(sfA), rows, k, _ptr(sink),
                                            _stream(stream)), "nvfp4_hbm_read_probe_rows")


def nvfp4_quantize_activation(x_bf16, global_scale, scale_per_row, x_packed, sf, rows, d, rule,
                              stream=None):
    _check(load().nvfp4_quantize_activation(_ptr(x_bf16), _ptr(global_scale), int(scale_per_row),
                                            _ptr(x_packed), _ptr(sf), rows, d, int(rule),
                                            _stream(stream)), "nvfp4_quantize_activation")


def nvfp4_quantize_weight(w_bf16, groups, rows, d, rule, w_packed, sf, global_scale, stream=None):
    _check(load().nvfp4_quantize_weight(_ptr(w_bf16), groups, rows, d, int(rule), _ptr(w_packed),
                                        _ptr(sf), _ptr(global_scale), _stream(stream)),
           "nvfp4_quantize_weight")


def nvfp4_gemv_bf16x_launch(A_packed, sfA, A_scale, x_bf16, x_scale, rule, x_packed, sfx, alpha, c,
                            l, m, k, stream=None):
    _check(load().nvfp4_gemv_bf16x_launch(_ptr(A_packed), _ptr(sfA), _ptr(A_scale), _ptr(x_bf16),
                                          _ptr(x_scale), int(rule), _ptr(x_packed), _ptr(sfx),
                                          _ptr(alpha), _ptr(c), l, m, k, _stream(stream)),
           "nvfp4_gemv_bf16x_launch")


def nvfp4_gemm_smalln_launch(A_packed, sfA, B_packed, sfB, alpha, c, l, m, n, k,
                             out_type=NVFP4_OUT_F16, stream=None):
    _check(load().nvfp4_gemm_smalln_launch(_ptr(A_packed), _ptr(sfA), _ptr(B_packed), _ptr(sfB),
                                           _ptr(alpha), _ptr(c), l, m, n, k, int(out_type),
                                           _stream(stream)), "nvfp4_gemm_smalln_launch")


def nvfp4_mma_num_variants() -> int:
    return int(load().nvfp4_mma_num_variants())


def nvfp4_mma_variant_info(v: int):
    """Matrix-core variants: (row tiles of 16 per wave, windows in flight, waves
    per group); VALU row-tile variants: (rows per tile, vectors per pass, waves
    per group)."""
    r, u, w = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().nvfp4_mma_variant_info(v, ctypes.byref(r), ctypes.byref(u), ctypes.byref(w)),
           "nvfp4_mma_variant_info")
    return r.value, u.value, w.value


def nvfp4_mma_variant_form(v: int) -> int:
    """NVFP4_MMA_FORM_MATRIX_CORES (0), NVFP4_MMA_FORM_VALU_TILES (1),
    NVFP4_MMA_FORM_LDS_STAGED (2) or NVFP4_MMA_FORM_LDS_VECTOR_REGS (3)."""
    f = ctypes.c_int32()
    _check(load().nvfp4_mma_variant_form(v, ctypes.byref(f)), "nvfp4_mma_variant_form")
    return f.value


def nvfp4_gemm_smalln_plan(l, m, n, k, aligned=True, tuning=None):
    """Returns (MmaTuning actually used, workspace bytes)."""
    out = MmaTuning()
    ws = ctypes.c_size_t()
    _check(load().nvfp4_gemm_smalln_plan(l, m, n, k, int(bool(aligned)), _mma_tuning(tuning),
                                         ctypes.byref(out), ctypes.byref(ws)),
           "nvfp4_gemm_smalln_plan")
    return out, int(ws.value)


def nvfp4_grouped_gemv_plan(experts, n, k, tokens, aligned=True, packed=False, tuning=None):
    """Returns the MmaTuning the grouped GEMV would use for `tokens` routed tokens."""
    out = MmaTuning()
    _check(load().nvfp4_grouped_gemv_plan(experts, n, k, tokens, int(bool(aligned)),
                                          int(bool(packed)), _mma_tuning(tuning), ctypes.byref(out)),
           "nvfp4_grouped_gemv_plan")
    return out


def nvfp4_gemm_smalln_launch_tuned(A_packed, sfA, B_packed, sfB, alpha, c, l, m, n, k, out_type,
                                   tuning, workspace, workspace_bytes, stream=None):
    _check(load().nvfp4_gemm_smalln_launch_tuned(_ptr(A_packed), _ptr(sfA), _ptr(B_packed),
                                                 _ptr(sfB), _ptr(alpha), _ptr(c), l, m, n, k,
                                                 int(out_type), _mma_tuning(tuning), _ptr(workspace),
                                                 int(workspace_bytes), _stream(stream)),
           "nvfp4_gemm_smalln_launch_tuned")


def nvfp4_grouped_gemv_launch(X_packed, sfX, W_packed, sfW, offsets, gs_x, gs_w, c, tokens, experts,
                              n, k, out_type=NVFP4_OUT_BF16, stream=None):
    _check(load().nvfp4_grouped_gemv_launch(_ptr(X_packed), _ptr(sfX), _ptr(W_packed), _ptr(sfW),
                                            _ptr(offsets), _ptr(gs_x), _ptr(gs_w), _ptr(c), tokens,
                                            experts, n, k, int(out_type), _stream(stream)),
           "nvfp4_grouped_gemv_launch")


def nvfp4_grouped_gemv_launch_tuned(X_packed, sfX, W_packed, sfW, offsets, gs_x, gs_w, c, tokens,
                                    experts, n, k, out_type, tuning, stream=None):
    _check(load().nvfp4_grouped_gemv_launch_tuned(_ptr(X_packed), _ptr(sfX), _ptr(W_packed),
                                                  _ptr(sfW), _ptr(offsets), _ptr(gs_x), _ptr(gs_w),
                                                  _ptr(c), tokens, experts, n, k, int(out_type),
                                                  _mma_tuning(tuning), _stream(stream)),
           "nvfp4_grouped_gemv_launch_tuned")


def nvfp4_mma_packed_sizes(groups, rows, k):
    """(codes bytes, scales bytes) of packed weights for groups matrices of rows x k."""
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().nvfp4_mma_packed_sizes(groups, rows, k, ctypes.byref(cb), ctypes.byref(sb)),
           "nvfp4_mma_packed_sizes")
    return int(cb.value), int(sb.value)


def nvfp4_mma_pack_weight(W, sW, groups, rows, k, W_packed, sW_packed, stream=None):
    _check(load().nvfp4_mma_pack_weight(_ptr(W), _ptr(sW), groups, rows, k, _ptr(W_packed),
                                        _ptr(sW_packed), _stream(stream)), "nvfp4_mma_pack_weight")


def nvfp4_gemm_smalln_launch_packed(A_packed, sfA_packed, B_packed, sfB, alpha, c, l, m, n, k,
                                    out_type=NVFP4_OUT_F16, tuning=None, stream=None):
    _check(load().nvfp4_gemm_smalln_launch_packed(_ptr(A_packed), _ptr(sfA_packed), _ptr(B_packed),
                                                  _ptr(sfB), _ptr(alpha), _ptr(c), l, m, n, k,
                                                  int(out_type), _mma_tuning(tuning),
                                                  _stream(stream)),
           "nvfp4_gemm_smalln_launch_packed")


def nvfp4_grouped_gemv_launch_packed(X_packed, sfX, W_packed, sfW_packed, offsets, gs_x, gs_w, c,
                                     tokens, experts, n, k, out_type=NVFP4_OUT_BF16, tuning=None,
                                     stream=None):
    _check(load().nvfp4_grouped_gemv_launch_packed(_ptr(X_packed), _ptr(sfX), _ptr(W_packed),
                                                   _ptr(sfW_packed), _ptr(offsets), _ptr(gs_x),
                                                   _ptr(gs_w), _ptr(c), tokens, experts, n, k,
                                                   int(out_type), _mma_tuning(tuning),
                                                   _stream(stream)),
           "nvfp4_grouped_gemv_launch_packed")


def quantize_activation(x, global_scale, rule=NVFP4_ROUND_HALF_STEP, stream=None):
    """Tensor-level call: x (rows, d) bfloat16 (or its uint16/int16 bits),
    global_scale a float32 device tensor of 1 or ``rows`` values.  Returns
    (packed uint8 (rows, d/2), scales uint8 (rows, d/16))."""
    import torch

    if x.dim() != 2 or x.element_size() != 2 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous 2-D 16-bit device tensor (bf16 bits)")
    rows, d = x.shape
    device = x.get_device()
    if global_scale.dtype != torch.float32 or global_scale.get_device() != device or \
            global_scale.numel() not in (1, rows):
        raise ValueError(f"global_scale must be a float32 tensor of 1 or rows values on GPU {device}")
    per_row = 1 if (global_scale.numel() == rows and rows > 1) else 0
    q = _allocate((rows, d // 2), torch.uint8, x.device, stream)
    sf = _allocate((rows, d // 16), torch.uint8, x.device, stream)
    with _current(device, stream):
        nvfp4_quantize_activation(x, global_scale, per_row, q, sf, rows, d, rule, stream)
    return q, sf


def gemv(A_packed, sfA, x_packed, sfx, alpha=None, out=None, stream=None):
    """Tensor-level call: shapes (l,m,k/2), (l,m,k/16), (l,k/2), (l,k/16), (l,).

    Checks dtypes, shapes, contiguity and device, allocates ``out`` (uint16
    fp16 bits, (l, m)) if not given, and calls :func:`nvfp4_gemv_launch`.
    """
    import torch

    if A_packed.dim() != 3:
        raise ValueError("A_packed must be (l, m, k/2)")
    l, m, half = A_packed.shape
    k = 2 * half
    want = {"A_packed": (A_packed, (l, m, half)), "sfA": (sfA, (l, m, k // 16)),
            "x_packed": (x_packed, (l, half)), "sfx": (sfx, (l, k // 16))}
    device = A_packed.get_device()
    for name, (t, shape) in want.items():
        if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous uint8 device tensor of shape {shape}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on GPU {device}, as A_packed")
    if alpha is not None and (alpha.dtype != torch.float32 or tuple(alpha.shape) != (l,)
                              or alpha.get_device() != device):
        raise ValueError(f"alpha must be a float32 tensor of shape (l,) on GPU {device}")
    if out is None:
        out = _allocate((l, m), torch.uint16, A_packed.device, stream)
    elif (out.dtype not in (torch.uint16, torch.float16, torch.int16) or tuple(out.shape) != (l, m)
          or not out.is_contiguous() or out.get_device() != device):
        raise ValueError(f"out must be a contiguous 16-bit tensor of shape (l, m) on GPU {device}")
    with _current(device, stream):
        nvfp4_gemv_launch(A_packed, sfA, x_packed, sfx, alpha, out, l, m, k, stream)
    return out


def pack_weight(W, sW, stream=None):
    """Tensor-level call: W (groups, rows, k/2) and sW (groups, rows, k/16)
    uint8 device tensors -> (codes, scales), the packed layout of
    :func:`nvfp4_mma_pack_weight` as flat uint8 device tensors, for
    :func:`nvfp4_gemm_smalln_launch_packed` and
    :func:`nvfp4_grouped_gemv_launch_packed`.  A 2-D W is one group."""
    import torch

    if W.dim() == 2:
        W, sW = W.unsqueeze(0), sW.unsqueeze(0)
    if W.dim() != 3:
        raise ValueError("W must be (groups, rows, k/2) or (rows, k/2)")
    groups, rows, half = W.shape
    k = 2 * half
    for name, t, shape in (("W", W, (groups, rows, half)), ("sW", sW, (groups, rows, k // 16))):
        if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous uint8 device tensor of shape {shape}")
    device = W.get_device()
    if sW.get_device() != device:
        raise ValueError(f"sW must be on GPU {device}, as W")
    cb, sb = nvfp4_mma_packed_sizes(groups, rows, k)
    codes = _allocate(cb, torch.uint8, W.device, stream)
    scales = _allocate(sb, torch.uint8, W.device, stream)
    with _current(device, stream):
        nvfp4_mma_pack_weight(W, sW, groups, rows, k, codes, scales, stream)
    return codes, scales


# ---- feed-forward operators (include/nvfp4_ffn.h)

def nvfp4_linear_workspace_size(n, m, k, activation=NVFP4_ACT_NONE) -> int:
    return int(load().nvfp4_linear_workspace_size(n, m, k, int(activation)))


def nvfp4_linear_launch_ws(X, x_type, ldx, W, sfW, w_layout, alpha, bias, residual, ldr, Y, y_type,
                           ldy, n, m, k, activation, workspace, workspace_bytes, stream=None):
    _check(load().nvfp4_linear_launch_ws(_ptr(X), x_type, ldx, _ptr(W), _ptr(sfW), w_layout,
                                         _ptr(alpha), _ptr(bias), _ptr(residual), ldr, _ptr(Y), y_type,
                                         ldy, n, m, k, activation, _ptr(workspace),
                                         int(workspace_bytes), _stream(stream)),
           "nvfp4_linear_launch_ws")


def nvfp4_linear_launch(X, x_type, ldx, W, sfW, w_layout, alpha, bias, residual, ldr, Y, y_type, ldy,
                        n, m, k, activation, stream=None):
    _check(load().nvfp4_linear_launch(_ptr(X), x_type, ldx, _ptr(W), _ptr(sfW), w_layout, _ptr(alpha),
                                      _ptr(bias), _ptr(residual), ldr, _ptr(Y), y_type, ldy, n, m, k,
                                      activation, _stream(stream)), "nvfp4_linear_launch")


def nvfp4_moe_layer_workspace_size(layer, tokens) -> int:
    """``layer`` is a :class:`MoeLayerStruct` or a :class:`MoeLayer`."""
    return int(load().nvfp4_moe_layer_workspace_size(_moe_struct(layer), tokens))


def nvfp4_moe_layer_launch_ws(layer, X, ldx, residual, ldr, Y, y_type, ldy, tokens, workspace,
                              workspace_bytes, stream=None):
    _check(load().nvfp4_moe_layer_launch_ws(_moe_struct(layer), _ptr(X), ldx, _ptr(residual), ldr,
                                            _ptr(Y), y_type, ldy, tokens, _ptr(workspace),
                                            int(workspace_bytes), _stream(stream)),
           "nvfp4_moe_layer_launch_ws")


def nvfp4_moe_layer_launch(layer, X, ldx, residual, ldr, Y, y_type, ldy, tokens, stream=None):
    _check(load().nvfp4_moe_layer_launch(_moe_struct(layer), _ptr(X), ldx, _ptr(residual), ldr, _ptr(Y),
                                         y_type, ldy, tokens, _stream(stream)),
           "nvfp4_moe_layer_launch")


_ACTIVATIONS = {"none": NVFP4_ACT_NONE, "relu": NVFP4_ACT_RELU, "gelu": NVFP4_ACT_GELU,
                "gelu_tanh": NVFP4_ACT_GELU_TANH, "silu": NVFP4_ACT_SILU}
_SCORINGS = {"softmax": NVFP4_SCORE_SOFTMAX, "sigmoid": NVFP4_SCORE_SIGMOID}


def _named(table, name, what):
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}")
    return table[name]


_FLOAT_TYPES = {}   # torch.dtype -> NVFP4_OUT_*, filled on first use: torch is not imported before


def _float_type(dtype, what, f32=False):
    if not _FLOAT_TYPES:
        import torch

        _FLOAT_TYPES.update({torch.bfloat16: NVFP4_OUT_BF16, torch.float16: NVFP4_OUT_F16,
                             torch.float32: NVFP4_OUT_F32})
    code = _FLOAT_TYPES.get(dtype)
    if code is None or (code == NVFP4_OUT_F32 and not f32):
        raise ValueError(f"{what} must be bfloat16{', float16 or float32' if f32 else ' or float16'}")
    return code


def _rows(t, what, shape, device, dtype=None):
    """Element stride of the rows of a 2-D tensor on that GPU whose columns are contiguous."""
    if t.shape != shape or t.get_device() != device or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{what} must be a tensor on GPU {device} of shape {shape}"
                         f"{'' if dtype is None else f' and {dtype}'}")
    rows, cols = t.stride()
    if cols != 1 and shape[1] > 1:
        raise ValueError(f"{what} must have contiguous columns")
    # a single row's stride is free; torch reports anything there
    ld = rows if shape[0] > 1 else shape[1]
    if ld < shape[1]:
        raise ValueError(f"{what} must have rows that do not overlap")
    return ld


def _floats(t, count, what, device):
    if t is None:
        return
    import torch

    if t.dtype is not torch.float32 or t.numel() != count or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what} must be a contiguous float32 tensor of {count} values on GPU {device}")


def _weight(codes, scales, groups, rows, k, packed, what, device):
    """Checks codes and scales of ``groups`` matrices of rows x k in either layout."""
    import torch

    # packed: whole tiles of 16 rows and windows of 256 elements, as nvfp4_mma_packed_sizes says
    count = groups * (-(-rows // 16) * 16) * (-(-k // 256) * 256) if packed else groups * rows * k
    for t, want, name in ((codes, count // 2, "codes"), (scales, count // 16, "scales")):
        if t.dtype is not torch.uint8 or t.numel() != want or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"{what} {name} must be a contiguous uint8 tensor of {want} bytes on GPU {device}")


def _output(out, out_dtype, n, m, x, residual, stream):
    """Output tensor (allocated on the stream that writes it if not given), its
    type code and row strides of it and of the residual."""
    device = x.get_device()
    if out is None:
        dtype = x.dtype if out_dtype is None else out_dtype
        y_type = _float_type(dtype, "out_dtype", f32=True)
        out = _allocate((n, m), dtype, x.device, stream)
        ldy = m
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out_dtype differs from out's type")
        y_type = _float_type(out.dtype, "out", f32=True)
        ldy = _rows(out, "out", (n, m), device)
    ldr = 0 if residual is None else _rows(residual, "residual", (n, m), device, out.dtype)
    return out, y_type, ldy, ldr


def _address(t):
    """Address of a tensor that has been checked to be on a device, or None."""
    return None if t is None else t.data_ptr()


def linear(x, codes, scales, m, alpha=None, bias=None, residual=None, activation="none", gated=False,
           packed=False, out=None, out_dtype=None, stream=None):
    """Tensor-level linear layer: ``residual + f(alpha x W^T + bias)`` or, gated,
    ``residual + f(gate) * up``.

    x (n, k) bfloat16 or float16 with any row stride; codes and scales uint8:
    (m, k/2), (m, k/16), gated (2, m, k/2), (2, m, k/16), or with ``packed`` what
    :func:`pack_weight` returns for them; alpha float32 of 1 (gated 2) values,
    bias float32 of m (gated 2 m); residual (n, m) of the output's type, which
    may be ``out`` itself.  Returns (n, m) of ``out_dtype`` (default x's type).
    All tensors are on one GPU, which need not be the current one; the default
    stream is that GPU's current stream.
    """
    if x.dim() != 2:
        raise ValueError("x must be (n, k)")
    n, k = x.shape
    x_type = _float_type(x.dtype, "x")
    device = x.get_device()
    if device < 0:
        raise ValueError("x must be on a GPU")
    ldx = _rows(x, "x", (n, k), device)
    groups = 2 if gated else 1
    _weight(codes, scales, groups, m, k, packed, "weight", device)
    _floats(alpha, groups, "alpha", device)
    _floats(bias, groups * m, "bias", device)
    act = _named(_ACTIVATIONS, activation, "activation") | (NVFP4_ACT_GATED if gated else 0)
    out, y_type, ldy, ldr = _output(out, out_dtype, n, m, x, residual, stream)
    if n > 0:
        _enqueue(load().nvfp4_linear_launch, (
            x.data_ptr(), x_type, ldx, codes.data_ptr(), scales.data_ptr(),
            NVFP4_W_PACKED if packed else NVFP4_W_ROW_MAJOR, _address(alpha), _address(bias),
            _address(residual), ldr, out.data_ptr(), y_type, ldy, n, m, k, act), device, stream,
            "nvfp4_linear_launch")
    return out


class MoeLayer:
    """What stays the same from call to call of one mixture-of-experts layer
    (``nvfp4_moe_layer_t``); keeps the tensors it names alive, which are all on
    one GPU.

    router (experts, hidden) bfloat16 or float16; codes13 / scales13 the gate
    and up matrices, (2 experts, inter, .) with expert e's gate at 2 e; codes2 /
    scales2 the down matrices, (experts, hidden, .); with ``packed`` what
    :func:`pack_weight` returns for them.  alpha13 float32 (experts, 2),
    alpha2 (experts,), route_bias (experts,), each optional.
    """

    def __init__(self, router, codes13, scales13, codes2, scales2, inter, topk, alpha13=None,
                 alpha2=None, route_bias=None, activation="silu", scoring="softmax", renormalize=True,
                 routed_scale=1.0, packed=False):
        if router.dim() != 2 or not router.is_cuda or not router.is_contiguous():
            raise ValueError("router must be a contiguous (experts, hidden) device tensor")
        experts, hidden = router.shape
        self.device = router.get_device()
        _weight(codes13, scales13, 2 * experts, inter, hidden, packed, "gate and up", self.device)
        _weight(codes2, scales2, experts, hidden, inter, packed, "down", self.device)
        _floats(alpha13, 2 * experts, "alpha13", self.device)
        _floats(alpha2, experts, "alpha2", self.device)
        _floats(route_bias, experts, "route_bias", self.device)
        self.tensors = (router, codes13, scales13, codes2, scales2, alpha13, alpha2, route_bias)
        self.dtype, self.hidden = router.dtype, hidden
        self.struct = MoeLayerStruct(
            router=_ptr(router), route_bias=_ptr(route_bias), W13=_ptr(codes13), sf13=_ptr(scales13),
            alpha13=_ptr(alpha13), W2=_ptr(codes2), sf2=_ptr(scales2), alpha2=_ptr(alpha2),
            experts=experts, hidden=hidden, inter=inter, topk=topk,
            x_type=_float_type(router.dtype, "router"),
            w_layout=NVFP4_W_PACKED if packed else NVFP4_W_ROW_MAJOR,
            activation=_named(_ACTIVATIONS, activation, "activation"),
            scoring=_named(_SCORINGS, scoring, "scoring"), renormalize=int(bool(renormalize)),
            routed_scale=routed_scale, reserved=0)
        self.reference = ctypes.byref(self.struct)


def _moe_struct(layer):
    return ctypes.byref(layer.struct if isinstance(layer, MoeLayer) else layer)


def moe_layer(x, layer, residual=None, out=None, out_dtype=None, stream=None):
    """Tensor-level mixture-of-experts layer: x (tokens, hidden) of the
    router's type with any row stride, ``layer`` a :class:`MoeLayer`, residual
    (tokens, hidden) of the output's type, which may be ``out`` itself.  Returns
    (tokens, hidden) of ``out_dtype`` (default x's type).  GPU and stream as in
    :func:`linear`."""
    if x.dim() != 2 or x.shape[1] != layer.hidden:
        raise ValueError(f"x must be (tokens, {layer.hidden})")
    n = x.shape[0]
    ldx = _rows(x, "x", (n, layer.hidden), layer.device, layer.dtype)
    out, y_type, ldy, ldr = _output(out, out_dtype, n, layer.hidden, x, residual, stream)
    if n > 0:
        _enqueue(load().nvfp4_moe_layer_launch,
                 (layer.reference, x.data_ptr(), ldx, _address(residual), ldr, out.data_ptr(), y_type, ldy, n),
                 layer.device, stream, "nvfp4_moe_layer_launch")
    return out
