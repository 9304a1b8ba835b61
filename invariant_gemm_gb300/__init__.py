"""Python binding of the invariant_gemm C ABI (ctypes).

Argument marshalling only: every step of the path runs in the CUDA kernels of
`libinvariant_gemm.so`, built in-tree by `invariant_gemm_gb300.build`. There is
no fallback: if the library is missing, every call raises.

Tensors are torch CUDA tensors (device memory and streams come from torch);
their data pointers are handed to the library unchanged. Layouts:
  x        bf16  [M][K]
  A_stack  bf16  [L][slices][r][K]
  B_stack  bf16  [L][slices][N][r]
  z        f32   [slices][M][r]
  y        bf16  [M][slices*N]   (updated in place)
  idx      int32 [M]             (-1 = no adapter)
The calls around the adapters (mx4_quantize, mx4_dequantize, mx4_gemm,
block_norm) and those of the attention (qk_norm_rope, kv_append, kv_gather,
paged_attention) take their sizes and strides from the tensors and check them.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "MODE_DET", "MODE_ATOMIC", "MODE_UNSPLIT", "MODE_DET_TREE", "PATH_AUTO", "PATH_WARP", "PATH_MMA", "PATH_FMA",
    "FLAG_STATIC_WEIGHTS", "FLAG_UNFUSED", "FLAG_Z_FP32", "FLAG_TEST_COPY_TIMEOUT",
    "FLAG_INPUT_READY",
    "IGError", "Shape", "PlanInfo", "lib", "lib_path", "make_shape", "workspace_bytes",
    "plan_query", "workspace", "workspace_init", "map_tokens", "lora_shrink",
    "lora_expand", "lora_apply", "lora_shrink_noalloc", "check_status", "status_string",
    "EXPORTS",
    "NORM_WEIGHT_PLUS_ONE", "Mx4Shape", "NormShape", "mx4_scale_bytes", "mx4_quantize",
    "mx4_dequantize", "mx4_workspace", "mx4_gemm", "block_norm",
    "ROPE_INTERLEAVED", "qk_norm_rope", "kv_append", "kv_gather", "attention_workspace",
    "paged_attention",
]

MODE_DET, MODE_ATOMIC, MODE_UNSPLIT, MODE_DET_TREE = 0, 1, 2, 3
FLAG_STATIC_WEIGHTS = 1
FLAG_UNFUSED = 2
FLAG_Z_FP32 = 4
FLAG_TEST_COPY_TIMEOUT = 8   # testing only: the first A-copy wait of each block expires
FLAG_INPUT_READY = 16        # x not written by work still running on the stream
PATH_AUTO, PATH_WARP, PATH_MMA, PATH_FMA = 0, 1, 2, 3
NORM_WEIGHT_PLUS_ONE = 1     # block_norm, head norms: norm weights are stored as w - 1
ROPE_INTERLEAVED = 2         # rotated pairs are neighbours, not halves

STATUS = {
    0: "IG_OK", -1: "IG_ERR_ARG", -2: "IG_ERR_SHAPE", -3: "IG_ERR_ALIGN",
    -4: "IG_ERR_WS_SMALL", -5: "IG_ERR_CUDA", -6: "IG_ERR_WS_CORRUPT",
    -7: "IG_ERR_ADAPTER_RANGE", -8: "IG_ERR_TIMEOUT", -9: "IG_ERR_UNSUPPORTED",
    -10: "IG_ERR_INDEX_RANGE",
}

# every function declared in include/invariant_gemm.h
EXPORTS = [
    "ig_version", "ig_status_string", "ig_workspace_bytes", "ig_plan_query",
    "ig_workspace_init", "ig_map_tokens", "lora_shrink", "lora_expand", "lora_apply",
    "ig_check_status", "lora_shrink_noalloc", "ig_mx4_scale_bytes", "ig_mx4_workspace_bytes",
    "ig_mx4_quantize", "ig_mx4_dequantize", "ig_mx4_gemm", "ig_block_norm",
    "ig_qk_norm_rope", "ig_kv_append", "ig_kv_gather", "ig_attention_workspace_bytes",
    "ig_paged_attention",
]

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libinvariant_gemm.so")


class IGError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)} ({status_string(code)})")


class Shape(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
        ("r", ctypes.c_int64), ("slices", ctypes.c_int32), ("num_adapters", ctypes.c_int32),
        ("split_k", ctypes.c_int32), ("mode", ctypes.c_int32), ("path", ctypes.c_int32),
        ("flags", ctypes.c_int32),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("path", ctypes.c_int32), ("split_k", ctypes.c_int32), ("k_split", ctypes.c_int64),
        ("shrink_bm", ctypes.c_int32), ("shrink_bn", ctypes.c_int32),
        ("expand_bm", ctypes.c_int32), ("expand_bn", ctypes.c_int32),
        ("shrink_tiles_max", ctypes.c_int64), ("shrink_ctas_max", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64), ("determinism_key", ctypes.c_uint64),
        ("apply_kernels", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class Mx4Shape(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("ld_y", ctypes.c_int64), ("y_type", ctypes.c_int32), ("flags", ctypes.c_int32),
    ]


class NormShape(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("H", ctypes.c_int64), ("ld_h", ctypes.c_int64),
        ("ld_y", ctypes.c_int64), ("ld_h_out", ctypes.c_int64), ("ld_n", ctypes.c_int64),
        ("gate_row_stride", ctypes.c_int64), ("gate_col_stride", ctypes.c_int32),
        ("h_type", ctypes.c_int32), ("flags", ctypes.c_int32), ("eps", ctypes.c_float),
        ("scale", ctypes.c_float),
    ]


# The same structs as bytes: half the time of a ctypes.Structure.
_MX4_SHAPE = struct.Struct("qqqqii").pack
_NORM_SHAPE = struct.Struct("qqqqqqqiiiff").pack
# ig_rope_shape, ig_kv_cache, ig_batch and ig_attn_shape of the header
_ROPE_SHAPE = struct.Struct("qqqqqqiiiiif").pack
_KV_CACHE = struct.Struct("PPqqqiiii").pack
_BATCH = struct.Struct("PPPqii").pack
_ATTN_SHAPE = struct.Struct("qqqiifi").pack

_LIB = None
_P = ctypes.c_void_p
_SP = ctypes.POINTER(Shape)


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build it with `python -m invariant_gemm_gb300.build`")
        L = ctypes.CDLL(path, mode=ctypes.RTLD_LOCAL)
        L.ig_version.restype = ctypes.c_char_p
        L.ig_version.argtypes = []
        L.ig_status_string.restype = ctypes.c_char_p
        L.ig_status_string.argtypes = [ctypes.c_int]
        L.ig_workspace_bytes.restype = ctypes.c_size_t
        L.ig_workspace_bytes.argtypes = [_SP]
        L.ig_plan_query.restype = ctypes.c_int
        L.ig_plan_query.argtypes = [_SP, ctypes.POINTER(PlanInfo)]
        L.ig_workspace_init.restype = ctypes.c_int
        L.ig_workspace_init.argtypes = [_P, ctypes.c_size_t, _SP, _P]
        L.ig_map_tokens.restype = ctypes.c_int
        L.ig_map_tokens.argtypes = [_SP, _P, _P, ctypes.c_size_t, _P]
        L.lora_shrink.restype = ctypes.c_int
        L.lora_shrink.argtypes = [_SP, _P, _P, _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
        L.lora_expand.restype = ctypes.c_int
        L.lora_expand.argtypes = [_SP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.lora_apply.restype = ctypes.c_int
        L.lora_apply.argtypes = [_SP, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P,
                                 ctypes.c_size_t, _P]
        L.lora_shrink_noalloc.restype = ctypes.c_int
        L.lora_shrink_noalloc.argtypes = [_SP, _P, _P, _P, ctypes.c_float, _P, _P]
        L.ig_check_status.restype = ctypes.c_int
        L.ig_check_status.argtypes = [_P, ctypes.c_size_t, _P]
        i64 = ctypes.c_int64
        L.ig_mx4_scale_bytes.restype = ctypes.c_size_t
        L.ig_mx4_scale_bytes.argtypes = [i64, i64]
        L.ig_mx4_workspace_bytes.restype = ctypes.c_size_t
        L.ig_mx4_workspace_bytes.argtypes = []
        L.ig_mx4_quantize.restype = ctypes.c_int
        L.ig_mx4_quantize.argtypes = [i64, i64, _P, i64, ctypes.c_int, _P, _P, _P]
        L.ig_mx4_dequantize.restype = ctypes.c_int
        L.ig_mx4_dequantize.argtypes = [i64, i64, _P, _P, _P, i64, ctypes.c_int, _P]
        L.ig_mx4_gemm.restype = ctypes.c_int
        # the shape: Mx4Shape / NormShape by reference, or their bytes
        L.ig_mx4_gemm.argtypes = [_P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.ig_block_norm.restype = ctypes.c_int
        L.ig_block_norm.argtypes = [_P] * 11
        n = ctypes.c_size_t
        L.ig_qk_norm_rope.restype = ctypes.c_int
        L.ig_qk_norm_rope.argtypes = [_P] * 10 + [n, _P]
        L.ig_kv_append.restype = ctypes.c_int
        L.ig_kv_append.argtypes = [_P] * 5 + [i64] + [_P] * 7 + [n, _P]
        L.ig_kv_gather.restype = ctypes.c_int
        L.ig_kv_gather.argtypes = [_P, _P, i64, _P, i64, _P, i64, _P, n, _P]
        L.ig_attention_workspace_bytes.restype = n
        L.ig_attention_workspace_bytes.argtypes = [_P] * 3
        L.ig_paged_attention.restype = ctypes.c_int
        L.ig_paged_attention.argtypes = [_P] * 6 + [n, _P]
        _LIB = L
    return _LIB


def status_string(code: int) -> str:
    try:
        return lib().ig_status_string(int(code)).decode()
    except ImportError:
        return STATUS.get(code, "unknown")


def make_shape(M, K, N, r, *, slices=1, num_adapters=1, split_k=8, mode=MODE_DET,
               path=PATH_AUTO, flags=0) -> Shape:
    return Shape(int(M), int(K), int(N), int(r), int(slices), int(num_adapters),
                 int(split_k), int(mode), int(path), int(flags))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(ws):
    return ws.numel() * ws.element_size()


def _check(rc: int, what: str):
    if rc != 0:
        raise IGError(rc, what)


def workspace_bytes(shape: Shape) -> int:
    return int(lib().ig_workspace_bytes(ctypes.byref(shape)))


def plan_query(shape: Shape) -> dict:
    info = PlanInfo()
    _check(lib().ig_plan_query(ctypes.byref(shape), ctypes.byref(info)), "ig_plan_query")
    return {f: getattr(info, f) for f, _ in PlanInfo._fields_}


def workspace_init(shape: Shape, ws, stream=None):
    _check(lib().ig_workspace_init(_ptr(ws), _nbytes(ws), ctypes.byref(shape), _stream(stream)),
           "ig_workspace_init")


def workspace(shape: Shape, device="cuda", stream=None, min_bytes: int = 0):
    """Allocate (with torch) and initialise a workspace large enough for shape."""
    import torch
    n = workspace_bytes(shape)
    if n == 0:
        plan_query(shape)  # raises with the reason
        raise IGError(-2, "ig_workspace_bytes")
    ws = torch.empty(max(n, int(min_bytes)), dtype=torch.uint8, device=device)
    workspace_init(shape, ws, stream)
    return ws


def map_tokens(shape: Shape, adapter_idx, ws, stream=None):
    _check(lib().ig_map_tokens(ctypes.byref(shape), _ptr(adapter_idx), _ptr(ws), _nbytes(ws),
                               _stream(stream)), "ig_map_tokens")


def lora_shrink(shape: Shape, x, A_stack, adapter_idx, scale, z, ws, stream=None):
    _check(lib().lora_shrink(ctypes.byref(shape), _ptr(x), _ptr(A_stack), _ptr(adapter_idx),
                             float(scale), _ptr(z), _ptr(ws), _nbytes(ws), _stream(stream)),
           "lora_shrink")


def lora_expand(shape: Shape, z, B_stack, adapter_idx, y, ws, stream=None):
    _check(lib().lora_expand(ctypes.byref(shape), _ptr(z), _ptr(B_stack), _ptr(adapter_idx),
                             _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream)), "lora_expand")


def lora_apply(shape: Shape, x, y, adapter_idx, A_stack, B_stack, scale, z, ws, stream=None):
    _check(lib().lora_apply(ctypes.byref(shape), _ptr(x), _ptr(y), _ptr(adapter_idx),
                            _ptr(A_stack), _ptr(B_stack), float(scale), _ptr(z), _ptr(ws),
                            _nbytes(ws), _stream(stream)), "lora_apply")


def lora_shrink_noalloc(shape: Shape, x, A_stack, adapter_idx, scale, z, stream=None):
    """lora_shrink with the library's built-in 4 MiB scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _check(lib().lora_shrink_noalloc(ctypes.byref(shape), _ptr(x), _ptr(A_stack),
                                     _ptr(adapter_idx), float(scale), _ptr(z), _stream(stream)),
           "lora_shrink_noalloc")


def check_status(ws, stream=None) -> int:
    """Synchronise and return the device status (0 or a negative code)."""
    return int(lib().ig_check_status(_ptr(ws), _nbytes(ws), _stream(stream)))


# --- the block around the adapters: MX4 and the norms -------------------------
#
# Sizes and strides come from the tensors. A tensor of another type, size,
# device or inner stride than its place asks for raises IGError (IG_ERR_ARG or
# IG_ERR_SHAPE) before the library is called, and so do operands on a GPU that
# is not the current one; the library checks the rest.

# The checks of a call take longer than its launch. So each call tests all that
# is usual (right types, one device, contiguous) in expressions of its own, and
# goes through _rows and _flat, which take strides and name what is wrong, only
# when one of them is false.

def _rows(what, name, t, dev, dtype, shape):
    """Checks an operand of `shape` with contiguous rows on GPU `dev` (an index);
    returns its row stride. A single row's stride means nothing."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0:
        ld, inner = t.stride()
        if inner == 1 or shape[1] == 1:
            return ld if shape[0] > 1 else shape[1]
    _why(what, name, t, dev, dtype, shape)


def _flat(what, name, t, dev, dtype, count):
    """Checks a contiguous operand of at least `count` elements."""
    if not (t.dtype is dtype and t.numel() >= count and t.is_contiguous() and
            t.get_device() == dev >= 0):
        _why(what, name, t, dev, dtype, (count,))


def _vector(what, name, t, dev, dtype, count):
    """Checks a contiguous operand of `count` elements; returns its address."""
    if not (t.dtype is dtype and t.numel() == count and t.is_contiguous() and
            t.get_device() == dev >= 0):
        _why(what, name, t, dev, dtype, (count,))
    return t.data_ptr()


def _packed(what, name, codes, scales, dev, u8, rows, half):
    """Checks the two tensors of a [rows][2 half] MX4 matrix."""
    count = ((rows + 127) >> 7) * ((half + 63) >> 6) * 512
    if not (codes.dtype is u8 and scales.dtype is u8 and codes.shape == (rows, half) and
            codes.is_contiguous() and scales.is_contiguous() and scales.numel() >= count and
            codes.get_device() == scales.get_device() == dev >= 0):
        if codes.shape != (rows, half) or not codes.is_contiguous():
            _why(what, name + " codes", codes, dev, u8, (rows, half))
        _flat(what, name + " codes", codes, dev, u8, 0)
        _flat(what, name + " scales", scales, dev, u8, count)


def _why(what, name, t, dev, dtype, shape):
    if dev < 0:
        raise IGError(-1, f"{what}: operands are not on a GPU")
    code = -1 if t.dtype is not dtype or t.get_device() != dev else -2
    raise IGError(code, f"{what}: {name} is {t.dtype} {tuple(t.shape)} with strides {t.stride()} on "
                        f"{t.device}; {dtype} {tuple(shape)} with contiguous rows on GPU {dev} wanted")


def _values(what, name, t, torch):
    """(sizes, GPU, ig_type, row stride) of a 2-D bf16 or FP32 operand."""
    shape, dev, dtype = t.shape, t.get_device(), t.dtype
    if len(shape) != 2 or not (dtype is torch.bfloat16 or dtype is torch.float32):
        raise IGError(-1, f"{what}: {name} is {dtype} {tuple(shape)}, 2-D bf16 or FP32 wanted")
    ld = shape[1] if dev >= 0 and t.is_contiguous() else _rows(what, name, t, dev, dtype, shape)
    return shape, dev, int(dtype is torch.float32), ld


_ONE_GPU = False    # the process sees one GPU, which is then the current one


def _check_current(what, dev, torch):
    """The library launches on the current GPU: operands have to be there."""
    global _ONE_GPU
    _ONE_GPU = torch.cuda.device_count() == 1
    now = torch._C._cuda_getDevice()
    if now != dev:
        raise IGError(-1, f"{what}: operands are on GPU {dev}, the current one is GPU {now}")


def _stream_of(what, dev, stream, torch):
    """The stream's handle for a launch on GPU `dev`, checked to be current (with
    one GPU once: the look costs a call 0.3 us)."""
    if not _ONE_GPU:
        _check_current(what, dev, torch)
    # the current stream's handle without the Stream object around it, whose
    # construction costs 2 us a call
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def mx4_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the scales of a [rows][K] MX4 matrix."""
    n = int(lib().ig_mx4_scale_bytes(rows, K))
    if n == 0 and rows != 0:
        raise IGError(-2, "ig_mx4_scale_bytes")
    return n


def mx4_quantize(x, codes, scales, stream=None):
    """x [rows][K] (bf16 or FP32, rows may be strided) -> MX4: codes uint8
    [rows][K/2] and scales, uint8 of mx4_scale_bytes(rows, K) elements."""
    import torch
    what = "mx4_quantize"
    (rows, K), dev, t, ld = _values(what, "x", x, torch)
    _packed(what, "x", codes, scales, dev, torch.uint8, rows, (K + 1) >> 1)
    rc = (_LIB or lib()).ig_mx4_quantize(rows, K, x.data_ptr(), ld, t, codes.data_ptr(),
                                         scales.data_ptr(), _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def mx4_dequantize(codes, scales, out, stream=None):
    """The values of an MX4 matrix into out [rows][K] (bf16 or FP32)."""
    import torch
    what = "mx4_dequantize"
    (rows, K), dev, t, ld = _values(what, "out", out, torch)
    _packed(what, "input", codes, scales, dev, torch.uint8, rows, (K + 1) >> 1)
    rc = (_LIB or lib()).ig_mx4_dequantize(rows, K, codes.data_ptr(), scales.data_ptr(),
                                           out.data_ptr(), ld, t,
                                           _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def mx4_workspace(device="cuda"):
    """Allocate (with torch) a workspace for mx4_gemm. An initialised workspace
    of the LoRA calls serves as well."""
    import torch
    return torch.zeros(int(lib().ig_mx4_workspace_bytes()), dtype=torch.uint8, device=device)


def mx4_gemm(x_codes, x_scales, w_codes, w_scales, y, ws, flags=0, stream=None):
    """y [M][N] (bf16 or FP32) = x w^T, x [M][K] and w [N][K] in MX4. flags: 0 or
    FLAG_STATIC_WEIGHTS."""
    import torch
    what, u8 = "mx4_gemm", torch.uint8
    (M, N), dev, t, ld = _values(what, "y", y, torch)
    half = x_codes.shape[-1]
    _packed(what, "x", x_codes, x_scales, dev, u8, M, half)
    _packed(what, "w", w_codes, w_scales, dev, u8, N, half)
    if not (ws.dtype is u8 and ws.is_contiguous() and ws.get_device() == dev):
        _flat(what, "ws", ws, dev, u8, 0)
    rc = (_LIB or lib()).ig_mx4_gemm(_MX4_SHAPE(M, N, 2 * half, ld, t, flags), x_codes.data_ptr(),
                                     x_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
                                     y.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def _gate(what, gate, dev, b16, M, H):
    """(row stride, column stride) of a gate that broadcasts to [M][H]."""
    shape, strides = gate.shape, gate.stride()
    if len(shape) == 1:
        shape, strides = (1, *shape), (0, *strides)
    if gate.dtype is b16 and len(shape) == 2 and gate.get_device() == dev:
        rows, cols = shape
        rs, cs = strides
        if (rows == M or rows == 1) and (cols == H or cols == 1):
            if cols == 1:
                cs = 0
            if cs == 0 or cs == 1:
                return rs if rows > 1 else 0, cs
    _why(what, "gate", gate, dev, b16, (M, H))


def block_norm(h, y=None, w_post=None, w_pre=None, *, gate=None, scale=1.0, eps=1e-6,
               h_out=None, n_out=None, codes=None, scales=None, flags=0, stream=None):
    """t = rms_norm(y) w_post; h' = h + scale gate t; n = rms_norm(h') w_pre.

    h [M][H] bf16 or FP32 (None: 0), y [M][H] bf16 (None: h' = h), gate bf16
    that broadcasts to [M][H] from (H,), (1, H), (M, 1) or (M, H) (None: 1),
    w_post and w_pre bf16 [H] (None: no such norm). h_out (may be h) receives
    h', n_out n in bf16, codes and scales n in MX4; what is None is not
    written. flags: 0 or NORM_WEIGHT_PLUS_ONE."""
    import torch
    what, b16 = "block_norm", torch.bfloat16
    lead = h if h is not None else y
    if lead is None:
        raise IGError(-1, "block_norm: neither h nor y")
    shape, dev, t, ld = _values(what, "h" if h is not None else "y", lead, torch)
    M, H = shape
    h_type = lead.dtype
    ld_h = ld_y = ld_ho = ld_n = H
    ph = py = pg = p_post = p_pre = pho = pn = pc = ps = None
    grs = gcs = 0
    if h is not None:
        ld_h, ph = ld, h.data_ptr()
    elif h_out is not None:
        t, h_type = int(h_out.dtype is torch.float32), h_out.dtype
        if t == 0 and h_type is not b16:
            _why(what, "h_out", h_out, dev, b16, shape)
    if y is not None:
        if not (y.dtype is b16 and y.shape == shape and y.is_contiguous() and
                y.get_device() == dev):
            ld_y = _rows(what, "y", y, dev, b16, shape)
        py = y.data_ptr()
    if h_out is not None:
        if not (h_out.dtype is h_type and h_out.shape == shape and h_out.is_contiguous() and
                h_out.get_device() == dev):
            ld_ho = _rows(what, "h_out", h_out, dev, h_type, shape)
        pho = h_out.data_ptr()
    if n_out is not None:
        if not (n_out.dtype is b16 and n_out.shape == shape and n_out.is_contiguous() and
                n_out.get_device() == dev):
            ld_n = _rows(what, "n_out", n_out, dev, b16, shape)
        pn = n_out.data_ptr()
    if w_post is not None:
        p_post = _vector(what, "w_post", w_post, dev, b16, H)
    if w_pre is not None:
        p_pre = _vector(what, "w_pre", w_pre, dev, b16, H)
    if gate is not None:
        grs, gcs = _gate(what, gate, dev, b16, M, H)
        pg = gate.data_ptr()
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise IGError(-1, "block_norm: codes and scales go together")
        _packed(what, "n", codes, scales, dev, torch.uint8, M, (H + 1) >> 1)
        pc, ps = codes.data_ptr(), scales.data_ptr()
    rc = (_LIB or lib()).ig_block_norm(
        _NORM_SHAPE(M, H, ld_h, ld_y, ld_ho, ld_n, grs, gcs, t, flags, eps, scale), ph, py, pg,
        p_post, p_pre, pho, pn, pc, ps, _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


# --- the attention of a served layer -------------------------------------------
#
# Heads: bf16 [T][heads][D], dense but for the stride between tokens (so q, k
# and v may be columns of one buffer). Cache: codes uint8 [pages][2][heads][page]
# [D] and scales uint8 [pages][2][heads][page / 16], dense but for the stride
# between pages. Batch: cu int32 [B + 1], kv_len int32 [B], page_table int32
# [B][pages of the longest]; sequence b has the rows cu[b] .. cu[b + 1] - 1, its
# last tokens.

def _heads(what, name, t, dev, b16):
    """(sizes, stride between tokens) of an operand of heads."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 3 and t.dtype is b16 and t.get_device() == dev >= 0:
        _, heads, D = shape
        if strides[2] == 1 and (strides[1] == D or heads == 1) or 0 in shape:
            return shape, strides[0] if shape[0] > 1 else heads * D
    _why(what, name, t, dev, b16, shape)


def _like(what, name, t, dev, b16, shape):
    """Checks an operand of these heads; returns its stride."""
    if t.shape == shape:
        if t.dtype is b16 and t.is_contiguous() and t.get_device() == dev >= 0:
            return shape[1] * shape[2]
        return _heads(what, name, t, dev, b16)[1]
    _why(what, name, t, dev, b16, shape)


def _cache_of(what, cache, scales, dev, u8):
    """The cache's struct and its (heads, head_dim)."""
    shape = cache.shape
    if not (cache.dtype is u8 and len(shape) == 5 and shape[1] == 2 and cache.get_device() == dev):
        _why(what, "cache", cache, dev, u8, shape)
    pages, _, heads, page, D = shape
    blocks = page >> 4
    want = (pages, 2, heads, blocks)
    if not (scales.dtype is u8 and scales.shape == want and scales.get_device() == dev):
        _why(what, "scales", scales, dev, u8, want)
    ps, ss = 2 * heads * page * D, 2 * heads * blocks
    if not cache.is_contiguous() and pages:
        ps = cache.stride(0) if pages > 1 else ps
        if not cache[0].is_contiguous():
            _why(what, "cache", cache, dev, u8, shape)
    if not scales.is_contiguous() and pages:
        ss = scales.stride(0) if pages > 1 else ss
        if not scales[0].is_contiguous():
            _why(what, "scales", scales, dev, u8, want)
    return (_KV_CACHE(cache.data_ptr(), scales.data_ptr(), pages, ps, ss, page, heads, D, 0),
            heads, D)


def _batch_of(what, cu, kv_len, page_table, dev, i32, max_q):
    shape = page_table.shape
    if not (len(shape) == 2 and page_table.dtype is i32 and page_table.is_contiguous() and
            page_table.get_device() == dev):
        _why(what, "page_table", page_table, dev, i32, shape)
    B, cols = shape
    if not (cu.dtype is i32 and kv_len.dtype is i32 and cu.numel() == B + 1 and
            kv_len.numel() == B and cu.is_contiguous() and kv_len.is_contiguous() and
            cu.get_device() == kv_len.get_device() == dev):
        _vector(what, "cu", cu, dev, i32, B + 1)
        _vector(what, "kv_len", kv_len, dev, i32, B)
    return _BATCH(cu.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), cols, B, max_q)


def _angles(what, cos_sin, positions, dev, T, torch):
    """(rows, rotated values, addresses) of the rotation's operands."""
    rows = rot = 0
    pc = pp = None
    if cos_sin is not None:
        shape = cos_sin.shape
        if not (len(shape) == 2 and cos_sin.dtype is torch.float32 and cos_sin.is_contiguous() and
                cos_sin.get_device() == dev):
            _why(what, "cos_sin", cos_sin, dev, torch.float32, shape)
        rows, rot = shape
        pc = cos_sin.data_ptr()
    if positions is not None:
        pp = _vector(what, "positions", positions, dev, torch.int32, T)
    return rows, rot, pc, pp


def _status_ws(what, ws, dev, u8):
    if not (ws.dtype is u8 and ws.is_contiguous() and ws.get_device() == dev):
        _flat(what, "ws", ws, dev, u8, 0)


def qk_norm_rope(q, k, q_out, k_out, ws, *, w_q=None, w_k=None, cos_sin=None, positions=None,
                 eps=1e-6, flags=0, stream=None):
    """Norm of each head of q and k (w_q, w_k bf16 [D]; None: no norm) and the
    rotation of its first values by the angles of the token's position (cos_sin
    FP32 [positions][rotated values]: the cosines, then the sines; positions int32
    [T]; None: no rotation). q or k may be None, with their outputs; q_out may be
    q, k_out may be k. flags: NORM_WEIGHT_PLUS_ONE, ROPE_INTERLEAVED. ws: any
    workspace; a position outside the table is NaN there and in check_status."""
    import torch
    what, b16 = "qk_norm_rope", torch.bfloat16
    lead = q if q is not None else k
    if lead is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise IGError(-1, "qk_norm_rope: q and q_out, k and k_out go together, one pair at least")
    dev = lead.get_device()
    hq = hk = ld_q = ld_k = ld_qo = ld_ko = 0
    pq = pk = pqo = pko = pwq = pwk = None
    if q is not None:
        shape, ld_q = _heads(what, "q", q, dev, b16)
        T, hq, D = shape
        ld_qo = _like(what, "q_out", q_out, dev, b16, shape)
        pq, pqo = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        shape, ld_k = _heads(what, "k", k, dev, b16)
        if q is not None and (shape[0] != T or shape[2] != D):
            _why(what, "k", k, dev, b16, (T, shape[1], D))
        T, hk, D = shape
        ld_ko = _like(what, "k_out", k_out, dev, b16, shape)
        pk, pko = k.data_ptr(), k_out.data_ptr()
    if w_q is not None:
        pwq = _vector(what, "w_q", w_q, dev, b16, D)
    if w_k is not None:
        pwk = _vector(what, "w_k", w_k, dev, b16, D)
    rows, rot, pc, pp = _angles(what, cos_sin, positions, dev, T, torch)
    _status_ws(what, ws, dev, torch.uint8)
    rc = (_LIB or lib()).ig_qk_norm_rope(
        _ROPE_SHAPE(T, rows, ld_q, ld_k, ld_qo, ld_ko, hq, hk, D, rot, flags, eps), pq, pk, pwq,
        pwk, pc, pp, pqo, pko, ws.data_ptr(), ws.numel(), _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def kv_append(k, v, cache, scales, cu, kv_len, page_table, ws, *, w_k=None, cos_sin=None,
              positions=None, q=None, q_out=None, w_q=None, eps=1e-6, max_q=None, flags=0,
              stream=None):
    """k (normed and rotated as by qk_norm_rope) and v of the new tokens into the
    cache; q likewise into q_out (may be q) where given. positions None: the
    token's place in its sequence. max_q: no sequence has more new tokens (None:
    as many as there are)."""
    import torch
    what, b16 = "kv_append", torch.bfloat16
    dev = k.get_device()
    shape, ld_k = _heads(what, "k", k, dev, b16)
    T, hk, D = shape
    ld_v = _like(what, "v", v, dev, b16, shape)
    c, heads, Dc = _cache_of(what, cache, scales, dev, torch.uint8)
    if heads != hk or Dc != D:
        _why(what, "k", k, dev, b16, (T, heads, Dc))
    b = _batch_of(what, cu, kv_len, page_table, dev, torch.int32, T if max_q is None else max_q)
    hq = ld_q = ld_qo = 0
    pq = pqo = pwq = pwk = None
    if (q is None) != (q_out is None):
        raise IGError(-1, "kv_append: q and q_out go together")
    if q is not None:
        shape, ld_q = _heads(what, "q", q, dev, b16)
        hq = shape[1]
        if shape[0] != T or shape[2] != D:
            _why(what, "q", q, dev, b16, (T, hq, D))
        ld_qo = _like(what, "q_out", q_out, dev, b16, shape)
        pq, pqo = q.data_ptr(), q_out.data_ptr()
    if w_q is not None:
        pwq = _vector(what, "w_q", w_q, dev, b16, D)
    if w_k is not None:
        pwk = _vector(what, "w_k", w_k, dev, b16, D)
    rows, rot, pc, pp = _angles(what, cos_sin, positions, dev, T, torch)
    _status_ws(what, ws, dev, torch.uint8)
    rc = (_LIB or lib()).ig_kv_append(
        _ROPE_SHAPE(T, rows, ld_q, ld_k, ld_qo, 0, hq, hk, D, rot, flags, eps), c, b, k.data_ptr(),
        v.data_ptr(), ld_v, pq, pwq, pwk, pc, pp, pqo, ws.data_ptr(), ws.numel(),
        _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def kv_gather(cache, scales, cu, kv_len, page_table, k_out, v_out, ws, *, stream=None):
    """What the cache holds, in bf16: rows cu[b] .. cu[b + 1] - 1 of k_out and
    v_out [T][heads][D] are the last tokens of sequence b."""
    import torch
    what, b16 = "kv_gather", torch.bfloat16
    dev = cache.get_device()
    c, heads, D = _cache_of(what, cache, scales, dev, torch.uint8)
    shape, ld_k = _heads(what, "k_out", k_out, dev, b16)
    T = shape[0]
    if shape[1] != heads or shape[2] != D:
        _why(what, "k_out", k_out, dev, b16, (T, heads, D))
    ld_v = _like(what, "v_out", v_out, dev, b16, shape)
    b = _batch_of(what, cu, kv_len, page_table, dev, torch.int32, 0)
    _status_ws(what, ws, dev, torch.uint8)
    rc = (_LIB or lib()).ig_kv_gather(c, b, T, k_out.data_ptr(), ld_k, v_out.data_ptr(), ld_v,
                                      ws.data_ptr(), ws.numel(),
                                      _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)


def attention_workspace(q, cache, page_table, max_q=None):
    """Allocate (with torch) a workspace for paged_attention over up to the rows
    of q, the sequences and pages of page_table and max_q new tokens of one
    sequence (None: as many as q has, three times the bytes of max_q=1 for 256
    sequences of a token each). It serves the other calls as well."""
    import torch
    T, hq, D = q.shape
    _, _, heads, page, Dc = cache.shape
    B, cols = page_table.shape
    n = int(lib().ig_attention_workspace_bytes(
        _ATTN_SHAPE(T, hq * D, hq * D, hq, 0, 1.0, 0),
        _KV_CACHE(0, 0, 0, 0, 0, page, heads, Dc, 0),
        _BATCH(0, 0, 0, cols, B, T if max_q is None else max_q)))
    if n == 0 or Dc != D:
        raise IGError(-2, "ig_attention_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def paged_attention(q, cache, scales, cu, kv_len, page_table, out, ws, *, max_q=None, scale=None,
                    flags=0, stream=None):
    """Attention of the new tokens (q [T][heads][D]) over the cache, causal at the
    end of each sequence, into out (not q). scale None: 1 / sqrt(D). max_q: no
    sequence has more new tokens (None: as many as there are); it and the number
    of sequences and pages decide how large ws has to be (attention_workspace)."""
    import torch
    what, b16 = "paged_attention", torch.bfloat16
    dev = q.get_device()
    shape, ld_q = _heads(what, "q", q, dev, b16)
    T, hq, D = shape
    ld_o = _like(what, "out", out, dev, b16, shape)
    c, heads, Dc = _cache_of(what, cache, scales, dev, torch.uint8)
    if Dc != D:
        _why(what, "q", q, dev, b16, (T, hq, Dc))
    b = _batch_of(what, cu, kv_len, page_table, dev, torch.int32, T if max_q is None else max_q)
    _status_ws(what, ws, dev, torch.uint8)
    rc = (_LIB or lib()).ig_paged_attention(
        _ATTN_SHAPE(T, ld_q, ld_o, hq, flags, D ** -0.5 if scale is None else scale, 0), c, b,
        q.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_of(what, dev, stream, torch))
    if rc:
        raise IGError(rc, what)
