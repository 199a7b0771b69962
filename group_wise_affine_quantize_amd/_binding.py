"""ctypes binding of libnq.so: argument marshalling only.

Every function here takes torch tensors on the GPU, checks that their dtypes
and shapes describe the call, and passes raw device pointers and the current
HIP stream to the C entry point of the same name (include/nq.h).  All
arithmetic happens in libnq's HIP kernels; there is no fallback of any kind.
If libnq.so was not built, the first call raises.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libnq.so"

NQ_ROW_INDEPENDENT_ROWS = 8
NQ_F32, NQ_BF16 = 0, 1
NQ_ROUTE_GEMV, NQ_ROUTE_TILED = 1, 2
NQ_MXFP4, NQ_MXFP8, NQ_NVFP4 = 1, 2, 3
# floating-point mode -> (C enum, bits per code, group size)
FP_MODES = {"mxfp4": (NQ_MXFP4, 4, 32), "mxfp8": (NQ_MXFP8, 8, 32), "nvfp4": (NQ_NVFP4, 4, 16)}
NQ_KV_INT8, NQ_KV_FP8 = 1, 2
KV_FORMATS = {"int8": NQ_KV_INT8, "fp8": NQ_KV_FP8}
NQ_MOE_SOFTMAX, NQ_MOE_SIGMOID = 1, 2
ROPE_LAYOUTS = {"halves": 1, "pairs": 2}
MOE_SCORES = {"softmax": NQ_MOE_SOFTMAX, "sigmoid": NQ_MOE_SIGMOID}

_lib = None


class NQError(RuntimeError):
    """A libnq call returned a non-zero status."""

    def __init__(self, status, message):
        super().__init__(f"[{status}] {message}")
        self.status = status
        self.message = message


class Plan(ctypes.Structure):
    _fields_ = [("route", ctypes.c_int32), ("ksplit", ctypes.c_int32),
                ("rows_per_wave", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]

    def as_dict(self):
        return {"route": {1: "gemv", 2: "tiled"}.get(self.route, self.route),
                "ksplit": self.ksplit, "rows_per_wave": self.rows_per_wave,
                "tile_m": self.tile_m, "tile_n": self.tile_n}


def library_path():
    """libnq.so next to this file, or the build NQ_LIBRARY names (for
    instance the host-sanitizer build)."""
    return os.environ.get("NQ_LIBRARY") or os.path.join(HERE, _LIB_NAME)


_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_SIGNATURES = {
    "nq_quantize": [_P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P],
    "nq_dequantize": [_P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P, _I32, _P],
    "nq_qmm_plan": [_I64, _I64, _I64, _I32, _I32, _I32, _I32, _I32, ctypes.POINTER(Plan)],
    "nq_qmm_workspace_bytes": [_I64, _I64, _I64, _I32, _I32, _I32, _I32, _I32],
    "nq_qmm": [_P, _I32, _I64, _I64, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _P, _SZ, _P],
    "nq_qmm_row_exact": [_P, _I32, _I64, _I64, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _P, _SZ,
                         _P],
    "nq_qmm_with_plan": [ctypes.POINTER(Plan), _P, _I32, _I64, _I64, _P, _P, _P, _I32, _I64,
                         _I32, _I32, _P, _P, _SZ, _P],
    "nq_qmm_batched": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _P, _SZ,
                       _P],
    "nq_gather_qmm_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, _I32, _I32, _I32, _I32,
                                      _I32],
    "nq_gather_qmm": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P,
                      _I32, _P, _P, _SZ, _P],
    "nq_gather_qmm_noalloc": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P,
                              _I32, _P, _P],
    "nq_gather_qmm_row_exact": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _I64, _I32,
                                _I32, _P, _I32, _P, _P, _SZ, _P],
    "nq_gather_qmm_lhs": [_P, _I32, _I64, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _I64, _I32, _I32,
                          _P, _P, _I32, _I32, _P, _P, _SZ, _P],
    "nq_qmm_notrans_workspace_bytes": [_I64, _I64, _I64, _I32, _I32, _I32, _I32],
    "nq_qmm_notrans": [_P, _I32, _I64, _I64, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _P, _SZ, _P],
    "nq_qmm_notrans_row_exact": [_P, _I32, _I64, _I64, _P, _P, _P, _I32, _I64, _I32, _I32, _P, _P,
                                 _SZ, _P],
    "nq_qmm_grad_scales_biases": [_P, _P, _I32, _I64, _I64, _P, _I64, _I32, _I32, _P, _P, _I32, _P],
    "nq_fp_quantize": [_P, _I32, _I64, _I64, _I32, _P, _P, _P],
    "nq_fp_dequantize": [_P, _P, _I64, _I64, _I32, _P, _I32, _P],
    "nq_fp_qmm": [_P, _I32, _I64, _I64, _P, _P, _P, _I64, _I32, _I32, _P, _P],
    "nq_fp_gather_qmm_workspace_bytes": [_I64, _I64, _I64, _I64, _I64],
    "nq_fp_gather_qmm": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _P, _P,
                         _SZ, _P],
    "nq_fp_qmm_notrans_workspace_bytes": [_I64, _I64, _I64, _I32, _I32, _I32],
    "nq_fp_qmm_notrans": [_P, _I32, _I64, _I64, _P, _P, _P, _I64, _I32, _I32, _P, _P, _SZ, _P],
    "nq_kv_append": [_P, _P, _P, _I64, _P, _I64, _I32, _P],
    "nq_kv_read": [_P, _P, _P, _P, _I32, _P],
    "nq_kv_attention_workspace_bytes": [_P, _P, _I32, _I32],
    "nq_kv_attention": [_P, _P, _P, _I32, _I64, _I32, ctypes.c_float, _I32, _I64, _P, _P, _P, _SZ, _P],
    "nq_kv_attention_shared_workspace_bytes": [_P, _P, _P, _I32, _I32],
    "nq_kv_attention_shared": [_P, _P, _P, _P, _I32, _I64, _I32, ctypes.c_float, _I32, _P, _P, _P, _SZ, _P],
    "nq_moe_route": [_P, _P, _I32, _I64, _I64, _P, _P, _P, _P],
    "nq_moe_route_grad": [_P, _P, _I32, _I64, _I64, _P, _P, _P, _P],
    "nq_moe_sort_workspace_bytes": [_I64, _I32, _I32],
    "nq_moe_sort": [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P],
    "nq_moe_dispatch": [_P, _P, _I32, _I64, _I64, _P, _P],
    "nq_moe_dispatch_grad": [_P, _P, _I32, _I64, _P, _P],
    "nq_moe_combine": [_P, _P, _I32, _I64, _P, _P, _I64, _P, _P],
    "nq_moe_combine_grad": [_P, _P, _I32, _I64, _I64, _P, _P, _P, _P, _P],
    "nq_block_norm": [_P, _P, _I64, _P, _I64, _I32, _P, _P, _I64, _P, _I32, _P, _P, _P],
    "nq_block_norm_grad_workspace_bytes": [_P],
    "nq_block_norm_grad": [_P, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _P, _P, _I64, _P, _I32, _P, _P, _P, _P,
                           _P, _P, _SZ, _P],
    "nq_rope": [_P, _P, _I32, _I64, _I64, _I32, _I32, _P, _I64, _P, _I64, _P],
    "nq_rope_grad": [_P, _P, _I32, _I64, _I64, _I32, _I32, _P, _I64, _P, _I64, _P],
    "nq_status_string": [_I32],
    "nq_last_error": [],
    "nq_version": [],
}
_RESTYPES = {"nq_qmm_workspace_bytes": _SZ, "nq_gather_qmm_workspace_bytes": _SZ,
             "nq_qmm_notrans_workspace_bytes": _SZ, "nq_fp_gather_qmm_workspace_bytes": _SZ,
             "nq_fp_qmm_notrans_workspace_bytes": _SZ, "nq_kv_attention_workspace_bytes": _SZ,
             "nq_kv_attention_shared_workspace_bytes": _SZ, "nq_moe_sort_workspace_bytes": _SZ,
              "nq_block_norm_grad_workspace_bytes": _SZ,
             "nq_status_string": ctypes.c_char_p, "nq_last_error": ctypes.c_char_p,
             "nq_version": ctypes.c_char_p}


def load_library(path=None):
    """Loads libnq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m group_wise_affine_quantize_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _RESTYPES.get(name, ctypes.c_int)
    _lib = lib
    return lib


def _check(status):
    if status != 0:
        lib = load_library()
        raise NQError(status, lib.nq_last_error().decode())


def _torch():
    import torch
    return torch


def _dt(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return NQ_F32
    if t.dtype == torch.bfloat16:
        return NQ_BF16
    raise TypeError(f"libnq takes float32 or bfloat16 tensors, got {t.dtype}")


def _torch_dtype(dt):
    torch = _torch()
    return torch.float32 if dt == NQ_F32 else torch.bfloat16


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(stream, shape, dtype, device):
    """A new output or workspace tensor.  With a caller's stream it is
    allocated under that stream, so the caching allocator ties the memory to
    the stream the kernels run on and does not hand it to other work while
    they may still use it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _contig(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def words_per_row(k, bits):
    return k * bits // 32


def nq_quantize(w, group_size, bits, codes=None, scales=None, biases=None, stream=None):
    """w [..., k] (f32 or bf16) -> (codes uint32-as-int32 [..., k*bits/32],
    scales [..., k/gs], biases [..., k/gs]) in w's dtype."""
    torch = _torch()
    lib = load_library()
    _contig("w", w)
    k = w.shape[-1]
    n = w.numel() // k if k else 0
    lead = tuple(w.shape[:-1])
    if codes is None:
        codes = _empty(stream, lead + (words_per_row(k, bits),), torch.int32, w.device)
    if scales is None:
        scales = _empty(stream, lead + (k // group_size if group_size else 0,), w.dtype, w.device)
    if biases is None:
        biases = _empty(stream, scales.shape, scales.dtype, scales.device)
    _check(lib.nq_quantize(_ptr(w), _dt(w), n, k, group_size, bits, _ptr(codes), _ptr(scales),
                           _ptr(biases), _stream(stream)))
    return codes, scales, biases


def nq_dequantize(codes, scales, biases, group_size, bits, out_dtype=None, out=None, stream=None):
    """-> w_hat [..., k] in out_dtype (default: the scales' dtype)."""
    torch = _torch()
    lib = load_library()
    for name, t in (("codes", codes), ("scales", scales), ("biases", biases)):
        _contig(name, t)
    k = scales.shape[-1] * group_size
    n = scales.numel() // scales.shape[-1] if scales.shape[-1] else 0
    out_dtype = out_dtype or scales.dtype
    if out is None:
        out = _empty(stream, tuple(scales.shape[:-1]) + (k,), out_dtype, scales.device)
    _check(lib.nq_dequantize(_ptr(codes), _ptr(scales), _ptr(biases), _dt(scales), n, k,
                             group_size, bits, _ptr(out), _dt(out), _stream(stream)))
    return out


def nq_qmm_plan(m, n, k, group_size, bits, x_dtype, sb_dtype, row_exact=False):
    torch = _torch()
    lib = load_library()
    plan = Plan()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    sd = NQ_F32 if sb_dtype == torch.float32 else NQ_BF16
    _check(lib.nq_qmm_plan(m, n, k, group_size, bits, xd, sd, int(bool(row_exact)),
                           ctypes.byref(plan)))
    return plan


def nq_qmm_workspace_bytes(m, n, k, group_size, bits, x_dtype, sb_dtype, row_exact=False):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    sd = NQ_F32 if sb_dtype == torch.float32 else NQ_BF16
    return load_library().nq_qmm_workspace_bytes(m, n, k, group_size, bits, xd, sd,
                                                 int(bool(row_exact)))


def _qmm_call(entry, x, codes, scales, biases, group_size, bits, y, workspace, stream, plan=None):
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases)):
        _contig(name, t)
    m, k = x.shape
    n = scales.shape[0]
    if scales.shape[1] * group_size != k or codes.shape != (n, words_per_row(k, bits)):
        raise ValueError("codes/scales shapes do not match x and the quantization")
    if y is None:
        y = _empty(stream, (m, n), x.dtype, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = [_ptr(x), _dt(x), m, k, _ptr(codes), _ptr(scales), _ptr(biases), _dt(scales), n,
            group_size, bits, _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)]
    if plan is not None:
        _check(lib.nq_qmm_with_plan(ctypes.byref(plan), *args))
    else:
        _check(getattr(lib, entry)(*args))
    return y


def nq_qmm(x, codes, scales, biases, group_size, bits, y=None, workspace=None, stream=None):
    """y [m, n] = x [m, k] times the transposed dequantized weights, in x's dtype."""
    return _qmm_call("nq_qmm", x, codes, scales, biases, group_size, bits, y, workspace, stream)


def nq_qmm_row_exact(x, codes, scales, biases, group_size, bits, y=None, workspace=None,
                     stream=None):
    """nq_qmm whose every row is bit-equal to the one-row product."""
    return _qmm_call("nq_qmm_row_exact", x, codes, scales, biases, group_size, bits, y,
                     workspace, stream)


def nq_qmm_with_plan(plan, x, codes, scales, biases, group_size, bits, y=None, workspace=None,
                     stream=None):
    return _qmm_call(None, x, codes, scales, biases, group_size, bits, y, workspace, stream,
                     plan=plan)


def nq_qmm_batched(x, codes, scales, biases, group_size, bits, y=None, workspace=None,
                   stream=None):
    """x [batch, l, k] -> y [batch, l, n]: item i bit-equal to nq_qmm(x[i])."""
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases)):
        _contig(name, t)
    batch, l, k = x.shape
    n = scales.shape[0]
    if scales.shape[1] * group_size != k or codes.shape != (n, words_per_row(k, bits)):
        raise ValueError("codes/scales shapes do not match x and the quantization")
    if y is None:
        y = _empty(stream, (batch, l, n), x.dtype, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.nq_qmm_batched(_ptr(x), _dt(x), batch, l, k, _ptr(codes), _ptr(scales),
                              _ptr(biases), _dt(scales), n, group_size, bits, _ptr(y),
                              _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def nq_qmm_notrans_workspace_bytes(m, ni, nc, group_size, bits, x_dtype, row_exact=False):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    return load_library().nq_qmm_notrans_workspace_bytes(m, ni, nc, group_size, bits, xd,
                                                         int(bool(row_exact)))


def _notrans_call(entry, x, codes, scales, biases, group_size, bits, y, workspace, stream):
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases)):
        _contig(name, t)
    m, ni = x.shape
    nc = scales.shape[1] * group_size
    if scales.shape[0] != ni or codes.shape != (ni, words_per_row(nc, bits)):
        raise ValueError("codes/scales shapes do not match x and the quantization")
    if y is None:
        y = _empty(stream, (m, nc), x.dtype, x.device)
    if workspace is None:
        need = lib.nq_qmm_notrans_workspace_bytes(m, ni, nc, group_size, bits, _dt(x),
                                                  int(entry.endswith("row_exact")))
        if need:
            workspace = _empty(stream, need, torch.uint8, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(getattr(lib, entry)(_ptr(x), _dt(x), m, ni, _ptr(codes), _ptr(scales), _ptr(biases),
                               _dt(scales), nc, group_size, bits, _ptr(y), _ptr(workspace),
                               ws_bytes, _stream(stream)))
    return y


def nq_qmm_notrans(x, codes, scales, biases, group_size, bits, y=None, workspace=None, stream=None):
    """y [m, nc] = x [m, ni] times the dequantized weights as stored ([ni, nc],
    grouped along nc): the transpose = false product.  With the forward
    weights and x = dy it is the derivative for the activations."""
    return _notrans_call("nq_qmm_notrans", x, codes, scales, biases, group_size, bits, y, workspace,
                         stream)


def nq_qmm_notrans_row_exact(x, codes, scales, biases, group_size, bits, y=None, workspace=None,
                             stream=None):
    """nq_qmm_notrans whose every row is bit-equal to the one-row product."""
    return _notrans_call("nq_qmm_notrans_row_exact", x, codes, scales, biases, group_size, bits, y,
                         workspace, stream)


def nq_qmm_grad_scales_biases(x, dy, codes, group_size, bits, out_dtype=None, dscales=None,
                              dbiases=None, stream=None):
    """Derivatives of sum(dy * nq_qmm(x, w)) for w's scales and biases:
    x [m, k], dy [m, n] (same dtype), codes [n, k*bits/32] -> (dscales,
    dbiases) [n, k/gs] in out_dtype (default: x's dtype)."""
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("dy", dy), ("codes", codes)):
        _contig(name, t)
    m, k = x.shape
    n = dy.shape[1]
    if dy.shape[0] != m or dy.dtype != x.dtype or codes.shape != (n, words_per_row(k, bits)):
        raise ValueError("x, dy and codes do not match")
    od = out_dtype or x.dtype
    if dscales is None:
        dscales = _empty(stream, (n, k // group_size), od, x.device)
    if dbiases is None:
        dbiases = _empty(stream, (n, k // group_size), od, x.device)
    _check(lib.nq_qmm_grad_scales_biases(_ptr(x), _ptr(dy), _dt(x), m, k, _ptr(codes), n, group_size,
                                         bits, _ptr(dscales), _ptr(dbiases), _dt(dscales),
                                         _stream(stream)))
    return dscales, dbiases


def nq_gather_qmm_workspace_bytes(rows, l, k, e, n, group_size, bits, x_dtype, sb_dtype,
                                  sorted_hint=False):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    sd = NQ_F32 if sb_dtype == torch.float32 else NQ_BF16
    return load_library().nq_gather_qmm_workspace_bytes(rows, l, k, e, n, group_size, bits, xd,
                                                        sd, int(bool(sorted_hint)))


def _gather_call(entry, x, codes, scales, biases, group_size, bits, rhs_idx, sorted_hint, y,
                 workspace, stream):
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases),
                    ("rhs_idx", rhs_idx)):
        _contig(name, t)
    if rhs_idx.element_size() != 4:
        raise ValueError("rhs_idx must hold 32-bit ids")
    rows, l, k = x.shape
    e, n = scales.shape[0], scales.shape[1]
    if rhs_idx.numel() != rows:
        raise ValueError("rhs_idx must have one id per row")
    if y is None:
        y = _empty(stream, (rows, l, n), x.dtype, x.device)
    if workspace is None:
        need = lib.nq_gather_qmm_workspace_bytes(rows, l, k, e, n, group_size, bits, _dt(x),
                                                 _dt(scales), int(bool(sorted_hint)))
        if need:
            workspace = _empty(stream, need, torch.uint8, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(getattr(lib, entry)(_ptr(x), _dt(x), rows, l, k, _ptr(codes), _ptr(scales),
                               _ptr(biases), _dt(scales), e, n, group_size, bits, _ptr(rhs_idx),
                               int(bool(sorted_hint)), _ptr(y), _ptr(workspace), ws_bytes,
                               _stream(stream)))
    return y


def nq_gather_qmm(x, codes, scales, biases, group_size, bits, rhs_idx, sorted_hint=False, y=None,
                  workspace=None, stream=None):
    """x [rows, l, k]; codes [e, n, k*bits/32]; scales/biases [e, n, k/gs];
    rhs_idx [rows] (int32/uint32 bit patterns) -> y [rows, l, n] in x's dtype.
    A workspace is allocated when the call needs one and none is given."""
    return _gather_call("nq_gather_qmm", x, codes, scales, biases, group_size, bits, rhs_idx,
                        sorted_hint, y, workspace, stream)


def nq_gather_qmm_noalloc(x, codes, scales, biases, group_size, bits, rhs_idx, sorted_hint=False, y=None,
                          stream=None):
    """nq_gather_qmm with the grouping tables in the library's static device
    array: no workspace argument, and nothing allocated by the library (y is
    allocated here only when not given)."""
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases),
                    ("rhs_idx", rhs_idx)):
        _contig(name, t)
    if rhs_idx.element_size() != 4:
        raise ValueError("rhs_idx must hold 32-bit ids")
    rows, l, k = x.shape
    e, n = scales.shape[0], scales.shape[1]
    if rhs_idx.numel() != rows:
        raise ValueError("rhs_idx must have one id per row")
    if y is None:
        y = _empty(stream, (rows, l, n), x.dtype, x.device)
    _check(lib.nq_gather_qmm_noalloc(_ptr(x), _dt(x), rows, l, k, _ptr(codes), _ptr(scales), _ptr(biases),
                                     _dt(scales), e, n, group_size, bits, _ptr(rhs_idx), int(bool(sorted_hint)),
                                     _ptr(y), _stream(stream)))
    return y


def nq_gather_qmm_row_exact(x, codes, scales, biases, group_size, bits, rhs_idx, sorted_hint=False,
                            y=None, workspace=None, stream=None):
    """As nq_gather_qmm, every row bit-equal to its one-row product."""
    return _gather_call("nq_gather_qmm_row_exact", x, codes, scales, biases, group_size, bits,
                        rhs_idx, sorted_hint, y, workspace, stream)


def nq_gather_qmm_lhs(x, codes, scales, biases, group_size, bits, lhs_idx, rhs_idx,
                      sorted_hint=False, row_exact=False, y=None, workspace=None, stream=None):
    """x [x_items, l, k]; lhs_idx and rhs_idx [rows] (32-bit ids): row r of
    y [rows, l, n] is x[lhs_idx[r]] times expert rhs_idx[r]'s weights; an id
    past x_items or e gives a zero row."""
    torch = _torch()
    lib = load_library()
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("biases", biases),
                    ("lhs_idx", lhs_idx), ("rhs_idx", rhs_idx)):
        _contig(name, t)
    if lhs_idx.element_size() != 4 or rhs_idx.element_size() != 4:
        raise ValueError("lhs_idx and rhs_idx must hold 32-bit ids")
    x_items, l, k = x.shape
    e, n = scales.shape[0], scales.shape[1]
    rows = rhs_idx.numel()
    if lhs_idx.numel() != rows:
        raise ValueError("lhs_idx and rhs_idx must have one id per output row")
    if y is None:
        y = _empty(stream, (rows, l, n), x.dtype, x.device)
    if workspace is None:
        need = lib.nq_gather_qmm_workspace_bytes(rows, l, k, e, n, group_size, bits, _dt(x),
                                                 _dt(scales), int(bool(sorted_hint)))
        if need:
            workspace = _empty(stream, need, torch.uint8, x.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.nq_gather_qmm_lhs(_ptr(x), _dt(x), x_items, rows, l, k, _ptr(codes), _ptr(scales),
                                 _ptr(biases), _dt(scales), e, n, group_size, bits, _ptr(lhs_idx),
                                 _ptr(rhs_idx), int(bool(sorted_hint)), int(bool(row_exact)),
                                 _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)))
    return y


# ---------------------------------------------------------------- floating-point modes
def _fp(mode):
    if mode not in FP_MODES:
        raise ValueError(f"unknown floating-point mode {mode!r} (one of {sorted(FP_MODES)})")
    return FP_MODES[mode]


def nq_fp_quantize(w, mode, codes=None, scales=None, stream=None):
    """w [..., k] (f32 or bf16) -> (codes uint32-as-int32 [..., k*bits/32],
    scales uint8 [..., k/group]) in mode "mxfp4", "mxfp8" or "nvfp4"."""
    torch = _torch()
    lib = load_library()
    mid, bits, gs = _fp(mode)
    _contig("w", w)
    k = w.shape[-1]
    n = w.numel() // k if k else 0
    lead = tuple(w.shape[:-1])
    if codes is None:
        codes = _empty(stream, lead + (words_per_row(k, bits),), torch.int32, w.device)
    if scales is None:
        scales = _empty(stream, lead + (k // gs,), torch.uint8, w.device)
    _check(lib.nq_fp_quantize(_ptr(w), _dt(w), n, k, mid, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def nq_fp_dequantize(codes, scales, mode, out_dtype=None, out=None, stream=None):
    """-> w_hat [..., k] in out_dtype (default bf16)."""
    torch = _torch()
    lib = load_library()
    mid, bits, gs = _fp(mode)
    for name, t in (("codes", codes), ("scales", scales)):
        _contig(name, t)
    k = scales.shape[-1] * gs
    n = scales.numel() // scales.shape[-1] if scales.shape[-1] else 0
    if out is None:
        out = _empty(stream, tuple(scales.shape[:-1]) + (k,), out_dtype or torch.bfloat16, scales.device)
    _check(lib.nq_fp_dequantize(_ptr(codes), _ptr(scales), n, k, mid, _ptr(out), _dt(out),
                                _stream(stream)))
    return out


def nq_fp_qmm(x, codes, scales, mode, global_scale=None, row_exact=False, y=None, stream=None):
    """y [m, n] = x [m, k] times the transposed weights (times the fp32 global
    scale, a one-element GPU tensor, NVFP4 only), in x's dtype."""
    torch = _torch()
    lib = load_library()
    mid, bits, gs = _fp(mode)
    for name, t in (("x", x), ("codes", codes), ("scales", scales)):
        _contig(name, t)
    m, k = x.shape
    n = scales.shape[0]
    if scales.shape[1] * gs != k or codes.shape != (n, words_per_row(k, bits)):
        raise ValueError("codes/scales shapes do not match x and the mode")
    if y is None:
        y = _empty(stream, (m, n), x.dtype, x.device)
    _check(lib.nq_fp_qmm(_ptr(x), _dt(x), m, k, _ptr(codes), _ptr(scales), _ptr(global_scale), n, mid,
                         int(bool(row_exact)), _ptr(y), _stream(stream)))
    return y


def nq_fp_gather_qmm_workspace_bytes(rows, l, k, e, n):
    return load_library().nq_fp_gather_qmm_workspace_bytes(rows, l, k, e, n)


def nq_fp_gather_qmm(x, codes, scales, mode, rhs_idx, global_scales=None, row_exact=False, y=None,
                     workspace=None, stream=None):
    """x [rows, l, k], stacked experts codes [e, n, words] and scales [e, n,
    groups], rhs_idx [rows] (uint32 as int32), optional per-expert fp32 global
    scales [e] (NVFP4) -> y [rows, l, n]; row_exact keeps every row's
    one-row bits.  The workspace (bytes from nq_fp_gather_qmm_workspace_bytes)
    is allocated here when not given."""
    torch = _torch()
    lib = load_library()
    mid, bits, gs = _fp(mode)
    for name, t in (("x", x), ("codes", codes), ("scales", scales), ("rhs_idx", rhs_idx)):
        _contig(name, t)
    rows, l, k = x.shape
    e, n = scales.shape[0], scales.shape[1]
    if scales.shape[2] * gs != k or codes.shape != (e, n, words_per_row(k, bits)):
        raise ValueError("codes/scales shapes do not match x and the mode")
    if rhs_idx.numel() != rows:
        raise ValueError("rhs_idx must hold one expert per row")
    if y is None:
        y = _empty(stream, (rows, l, n), x.dtype, x.device)
    if workspace is None:
        need = lib.nq_fp_gather_qmm_workspace_bytes(rows, l, k, e, n)
        workspace = _empty(stream, need, torch.uint8, x.device) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.nq_fp_gather_qmm(_ptr(x), _dt(x), rows, l, k, _ptr(codes), _ptr(scales),
                                _ptr(global_scales), e, n, mid, _ptr(rhs_idx), int(bool(row_exact)), _ptr(y),
                                _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def nq_fp_qmm_notrans_workspace_bytes(m, ni, nc, mode, x_dtype, row_exact=False):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    return load_library().nq_fp_qmm_notrans_workspace_bytes(m, ni, nc, _fp(mode)[0], xd,
                                                            int(bool(row_exact)))


def nq_fp_qmm_notrans(x, codes, scales, mode, global_scale=None, row_exact=False, y=None, workspace=None,
                      stream=None):
    """y [m, nc] = x [m, ni] times the quantized matrix [ni, nc] as stored
    (codes [ni, nc*bits/32], scales [ni, nc/group]); with the forward weights
    this is the derivative for the activations.  The workspace is allocated
    here when not given."""
    torch = _torch()
    lib = load_library()
    mid, bits, gs = _fp(mode)
    for name, t in (("x", x), ("codes", codes), ("scales", scales)):
        _contig(name, t)
    m, ni = x.shape
    nc = scales.shape[1] * gs
    if scales.shape[0] != ni or codes.shape != (ni, words_per_row(nc, bits)):
        raise ValueError("codes/scales shapes do not match x and the mode")
    if y is None:
        y = _empty(stream, (m, nc), x.dtype, x.device)
    if workspace is None:
        need = lib.nq_fp_qmm_notrans_workspace_bytes(m, ni, nc, mid, _dt(x), int(bool(row_exact)))
        workspace = _empty(stream, need, torch.uint8, x.device) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.nq_fp_qmm_notrans(_ptr(x), _dt(x), m, ni, _ptr(codes), _ptr(scales), _ptr(global_scale), nc,
                                 mid, int(bool(row_exact)), _ptr(y), _ptr(workspace), ws_bytes,
                                 _stream(stream)))
    return y


# ---------------------------------------------------------------- key/value cache in 8 bits
# These calls are made once or twice per layer and serving step, where a
# microsecond on the host counts: outputs made here are not checked again, and
# the stream's handle is taken without making a Stream object.
def _raw_stream(stream=None):
    """The handle of `stream`, or of the current stream of the current device."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scales", _P), ("v_scales", _P), ("blocks", _I64),
                ("kv_heads", _I32), ("head_dim", _I32), ("block_tokens", _I32), ("format", _I32)]


class _KVSeqsStruct(ctypes.Structure):
    _fields_ = [("row_start", _P), ("lengths", _P), ("block_table", _P), ("batch", _I64), ("max_blocks", _I64),
                ("table_stride", _I64), ("rows", _I64)]


class _MoERouterStruct(ctypes.Structure):
    _fields_ = [("experts", _I32), ("score", _I32), ("groups", _I32), ("top_groups", _I32), ("group_best", _I32),
                ("top_k", _I32), ("renormalise", _I32), ("scale", ctypes.c_float)]


class _Described:
    """What a struct that calls pass describes.  Shapes are checked against the
    attributes and kernels go by the struct, so neither changes once it is made:
    a new description takes a new object."""

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} cannot be set; make a new {type(self).__name__}")
        object.__setattr__(self, name, value)


class KVCache(_Described):
    """A paged key/value cache in 8 bits (nq_kv_cache): k_codes [blocks,
    kv_heads, block_tokens, head_dim] and v_codes [blocks, kv_heads, head_dim,
    block_tokens] uint8, k_scales and v_scales [blocks, kv_heads] float32;
    format "int8" or "fp8".  The constructor allocates the arrays (contents
    undefined until written); wrap() takes existing ones."""

    def __init__(self, blocks, kv_heads, block_tokens, head_dim, format="int8", device="cuda"):
        torch = _torch()
        u8 = {"dtype": torch.uint8, "device": device}
        f32 = {"dtype": torch.float32, "device": device}
        self._bind(torch.empty((blocks, kv_heads, block_tokens, head_dim), **u8),
                   torch.empty((blocks, kv_heads), **f32),
                   torch.empty((blocks, kv_heads, head_dim, block_tokens), **u8),
                   torch.empty((blocks, kv_heads), **f32), format)

    @classmethod
    def wrap(cls, k_codes, k_scales, v_codes, v_scales, format):
        self = cls.__new__(cls)
        self._bind(k_codes, k_scales, v_codes, v_scales, format)
        return self

    def _bind(self, k_codes, k_scales, v_codes, v_scales, format):
        torch = _torch()
        if format not in KV_FORMATS:
            raise ValueError(f"unknown cache format {format!r} (one of {sorted(KV_FORMATS)})")
        for name, t, dt in (("k_codes", k_codes, torch.uint8), ("v_codes", v_codes, torch.uint8),
                            ("k_scales", k_scales, torch.float32), ("v_scales", v_scales, torch.float32)):
            _contig(name, t)
            if t.dtype != dt:
                raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        blocks, kv_heads, block_tokens, head_dim = k_codes.shape
        if tuple(v_codes.shape) != (blocks, kv_heads, head_dim, block_tokens) or \
                tuple(k_scales.shape) != (blocks, kv_heads) or tuple(v_scales.shape) != (blocks, kv_heads):
            raise ValueError("codes and scales do not describe one cache")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.blocks, self.kv_heads, self.block_tokens, self.head_dim = blocks, kv_heads, block_tokens, head_dim
        self.format = format
        self._struct = _KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                      v_scales.data_ptr(), blocks, kv_heads, head_dim, block_tokens,
                                      KV_FORMATS[format])
        self._ref = ctypes.byref(self._struct)


class KVSequences(_Described):
    """The sequences of a call (nq_kv_seqs): row_start [batch + 1], lengths
    [batch] and block_table [batch, max_blocks] int32 on the GPU, rows the
    number of rows of the call's arrays.  Row i of sequence b is token
    lengths[b] - row_start[b + 1] + i.  The tensors may be updated in place
    between calls; other tensors, or another number of rows, take a new
    object."""

    def __init__(self, row_start, lengths, block_table, rows):
        torch = _torch()
        for name, t in (("row_start", row_start), ("lengths", lengths)):
            _contig(name, t)
        for name, t in (("row_start", row_start), ("lengths", lengths), ("block_table", block_table)):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise TypeError(f"{name} must be an int32 GPU tensor")
        batch = lengths.numel()
        if row_start.numel() != batch + 1 or block_table.dim() != 2 or block_table.shape[0] != batch:
            raise ValueError("row_start, lengths and block_table do not describe one batch")
        max_blocks = block_table.shape[1]
        if max_blocks > 1 and block_table.stride(1) != 1:
            raise ValueError("the rows of block_table must be contiguous")
        stride = block_table.stride(0) if batch > 1 else max_blocks
        self.row_start, self.lengths, self.block_table, self.rows = row_start, lengths, block_table, rows
        self.batch = batch
        self._struct = _KVSeqsStruct(row_start.data_ptr(), lengths.data_ptr(), block_table.data_ptr(), batch,
                                     max_blocks, stride, rows)
        self._ref = ctypes.byref(self._struct)


def _row_stride(name, t, rows, heads, dim):
    """The row stride of a [rows, heads, dim] tensor whose rows are dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{name} must have shape {(rows, heads, dim)}, got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError(f"the rows of {name} must be contiguous")
    return s[0] if rows > 1 else heads * dim


def nq_kv_append(cache, seqs, k, v, stream=None):
    """Writes the keys and values of seqs' rows, k and v [rows, kv_heads,
    head_dim] (f32 or bf16, any row stride of whole 16 bytes), into cache."""
    lib = _lib or load_library()
    ldk = _row_stride("k", k, seqs.rows, cache.kv_heads, cache.head_dim)
    ldv = _row_stride("v", v, seqs.rows, cache.kv_heads, cache.head_dim)
    if k.dtype != v.dtype:
        raise TypeError("k and v must have the same dtype")
    status = lib.nq_kv_append(cache._ref, seqs._ref, k.data_ptr(), ldk, v.data_ptr(), ldv, _dt(k), _raw_stream(stream))
    if status:
        _check(status)


def nq_kv_read(cache, seqs, out_dtype=None, k=None, v=None, stream=None):
    """The tokens of seqs' rows -> (k, v) [rows, kv_heads, head_dim] in
    out_dtype (default bf16)."""
    torch = _torch()
    lib = _lib or load_library()
    shape = (seqs.rows, cache.kv_heads, cache.head_dim)
    dt = out_dtype or torch.bfloat16
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _contig(name, t)
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
            dt = t.dtype
    if k is None:
        k = _empty(stream, shape, dt, cache.k_codes.device)
    if v is None:
        v = _empty(stream, shape, dt, cache.k_codes.device)
    if k.dtype != v.dtype:
        raise TypeError("k and v must have the same dtype")
    status = lib.nq_kv_read(cache._ref, seqs._ref, k.data_ptr(), v.data_ptr(), _dt(k), _raw_stream(stream))
    if status:
        _check(status)
    return k, v


def nq_kv_attention_workspace_bytes(cache, seqs, q_heads, x_dtype):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    return load_library().nq_kv_attention_workspace_bytes(cache._ref, seqs._ref, q_heads, xd)


def nq_kv_attention(cache, seqs, q, scale=None, causal=True, window=0, out=None, lse=None, workspace=None,
                    stream=None):
    """Attention of q [rows, q_heads, head_dim] (f32 or bf16, any row stride of
    whole 16 bytes) over cache -> out, dense, in q's dtype.  scale: factor of
    the scores (default head_dim ** -0.5); window > 0: only the last `window`
    tokens of a row (with causal); lse: an optional [rows, q_heads] float32
    tensor for the log-sum-exp of the scores.  The workspace is allocated here
    when not given."""
    torch = _torch()
    lib = _lib or load_library()
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    heads = q.shape[1]
    ldq = _row_stride("q", q, seqs.rows, heads, cache.head_dim)
    dt = _dt(q)
    if out is None:
        out = _empty(stream, q.shape, q.dtype, q.device)
    else:
        _contig("out", out)
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
    if lse is not None:
        _contig("lse", lse)
        if tuple(lse.shape) != (seqs.rows, heads) or lse.dtype != torch.float32:
            raise ValueError("lse must be float32 [rows, q_heads]")
    if workspace is None:
        ws_bytes = lib.nq_kv_attention_workspace_bytes(cache._ref, seqs._ref, heads, dt)
        if ws_bytes:
            workspace = _empty(stream, ws_bytes, torch.uint8, q.device)
    else:
        _contig("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    status = lib.nq_kv_attention(cache._ref, seqs._ref, q.data_ptr(), dt, ldq, heads,
                                 cache.head_dim ** -0.5 if scale is None else scale, int(bool(causal)), window,
                                 out.data_ptr(), None if lse is None else lse.data_ptr(),
                                 None if workspace is None else workspace.data_ptr(), ws_bytes, _raw_stream(stream))
    if status:
        _check(status)
    return out


def nq_kv_attention_shared_workspace_bytes(cache, prefix, seqs, q_heads, x_dtype):
    torch = _torch()
    xd = NQ_F32 if x_dtype == torch.float32 else NQ_BF16
    return load_library().nq_kv_attention_shared_workspace_bytes(cache._ref, prefix._ref, seqs._ref, q_heads, xd)


def nq_kv_attention_shared(cache, prefix, seqs, q, scale=None, causal=True, out=None, lse=None, workspace=None,
                           stream=None):
    """nq_kv_attention for a batch whose sequences share prefixes, each read once
    for all of its rows.  prefix: a KVSequences over the same rows, of which rows
    row_start[p] .. row_start[p + 1] see all lengths[p] tokens of prefix p before
    those of their own sequence (seqs, whose lengths count own tokens only).  The
    workspace is allocated here when not given."""
    torch = _torch()
    lib = _lib or load_library()
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    heads = q.shape[1]
    ldq = _row_stride("q", q, seqs.rows, heads, cache.head_dim)
    dt = _dt(q)
    out = _empty(stream, q.shape, q.dtype, q.device) if out is None else _given("out", out, q.shape, q.dtype)
    if lse is not None:
        _given("lse", lse, (seqs.rows, heads), torch.float32)
    if workspace is None:
        ws_bytes = lib.nq_kv_attention_shared_workspace_bytes(cache._ref, prefix._ref, seqs._ref, heads, dt)
        if ws_bytes:
            workspace = _empty(stream, ws_bytes, torch.uint8, q.device)
    else:
        _contig("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    on = _launch_on(stream, cache.k_codes, prefix.lengths, seqs.lengths, q, out, lse, workspace)
    status = lib.nq_kv_attention_shared(cache._ref, prefix._ref, seqs._ref, q.data_ptr(), dt, ldq, heads,
                                        cache.head_dim ** -0.5 if scale is None else scale, int(bool(causal)),
                                        out.data_ptr(), _address(lse), _address(workspace), ws_bytes,
                                        on)
    if status:
        _check(status)
    return out


# ---------------------------------------------------------------- expert routing
class MoERouter(_Described):
    """How tokens choose experts (nq_moe_router): the top_k largest of score
    "softmax" or "sigmoid" (plus a bias), from the top_groups best of `groups`
    groups of neighbouring experts -- a group's score is its largest key
    (group_best 1) or the sum of its two largest (2); weights divided by their
    sum when renormalise, times scale."""

    def __init__(self, experts, top_k, score="softmax", groups=1, top_groups=None, group_best=1, renormalise=False,
                 scale=1.0):
        if score not in MOE_SCORES:
            raise ValueError(f"unknown score {score!r} (one of {sorted(MOE_SCORES)})")
        self.experts, self.top_k, self.score, self.groups = experts, top_k, score, groups
        self.top_groups = groups if top_groups is None else top_groups
        self.group_best, self.renormalise, self.scale = group_best, bool(renormalise), scale
        self._struct = _MoERouterStruct(experts, MOE_SCORES[score], groups, self.top_groups, group_best, top_k,
                                        int(self.renormalise), scale)
        self._ref = ctypes.byref(self._struct)


def _logits(router, logits):
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    if logits.dim() != 2 or logits.shape[1] != router.experts or (router.experts > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [tokens, experts] with contiguous rows")
    return logits.shape[0], logits.stride(0) if logits.shape[0] > 1 else router.experts


def nq_moe_route(router, logits, bias=None, ids=None, weights=None, stream=None):
    """logits [tokens, experts] (f32 or bf16, any row stride), bias [experts]
    float32 or None -> (ids [tokens, top_k] uint32-as-int32, weights [tokens,
    top_k] float32), the largest key first."""
    torch = _torch()
    lib = _lib or load_library()
    tokens, ld = _logits(router, logits)
    shape = (tokens, router.top_k)
    if bias is not None:
        _contig("bias", bias)
        if bias.dtype != torch.float32 or bias.numel() != router.experts:
            raise ValueError("bias must be float32 [experts]")
    for name, t, dt in (("ids", ids, torch.int32), ("weights", weights, torch.float32)):
        if t is not None:
            _contig(name, t)
            if t.shape != shape or t.dtype != dt:
                raise ValueError(f"{name} must be {dt} {shape}")
    if ids is None:
        ids = _empty(stream, shape, torch.int32, logits.device)
    if weights is None:
        weights = _empty(stream, shape, torch.float32, logits.device)
    status = lib.nq_moe_route(router._ref, logits.data_ptr(), _dt(logits), tokens, ld,
                              None if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                              _raw_stream(stream))
    if status:
        _check(status)
    return ids, weights


def nq_moe_route_grad(router, logits, ids, dweights, dlogits=None, stream=None):
    """The logits' gradient of sum(dweights * weights): ids from nq_moe_route,
    dweights [tokens, top_k] float32 -> dlogits [tokens, experts], dense, in
    the logits' dtype."""
    torch = _torch()
    lib = _lib or load_library()
    tokens, ld = _logits(router, logits)
    shape = (tokens, router.top_k)
    for name, t, dt in (("ids", ids, torch.int32), ("dweights", dweights, torch.float32)):
        _contig(name, t)
        if t.shape != shape or t.dtype != dt:
            raise ValueError(f"{name} must be {dt} {shape}")
    if dlogits is None:
        dlogits = _empty(stream, (tokens, router.experts), logits.dtype, logits.device)
    else:
        _contig("dlogits", dlogits)
        if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
            raise ValueError("dlogits must have the logits' shape and dtype")
    status = lib.nq_moe_route_grad(router._ref, logits.data_ptr(), _dt(logits), tokens, ld, ids.data_ptr(),
                                   dweights.data_ptr(), dlogits.data_ptr(), _raw_stream(stream))
    if status:
        _check(status)
    return dlogits


# ---------------------------------------------------------------- tokens sorted by expert
class _MoEOrderStruct(ctypes.Structure):
    _fields_ = [("starts", _P), ("place", _P), ("tokens", _I64), ("top_k", _I32), ("experts", _I32)]


class _BlockNormStruct(ctypes.Structure):
    _fields_ = [("rows", _I64), ("dim", _I64), ("gates", _I64), ("eps", ctypes.c_float), ("offset", ctypes.c_float),
                ("scale", ctypes.c_float)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("freq", _P), ("axis", _P), ("rotary_dim", _I32), ("axes", _I32), ("layout", _I32),
                ("scale", ctypes.c_float)]


# As for the cache, these calls are made for every layer and step: checks are kept
# to what the tensors cannot show by themselves, outputs made here are not
# checked, and each is one call of the allocator.
_TYPES = {}


def _type(t):
    """nq_dtype of a tensor."""
    if not _TYPES:
        torch = _torch()
        _TYPES.update({torch.float32: NQ_F32, torch.bfloat16: NQ_BF16})
    dt = _TYPES.get(t.dtype)
    return _dt(t) if dt is None else dt     # _dt refuses


def _launch_on(stream, *tensors):
    """The handle of the call's stream; all tensors (None left out) are on its GPU."""
    if stream is not None:
        at, handle = stream.device.index, stream.cuda_stream
    else:
        c = _torch()._C
        at = c._cuda_getDevice()
        handle = c._cuda_getCurrentRawStream(at)
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"a tensor on {t.device} in a call on cuda:{at}; make that device the current one "
                             "or pass a stream of it")
    return handle


def _given(name, t, shape, dtype):
    """A caller's dense tensor."""
    _contig(name, t)
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def _fresh(stream, like, shape, dtype=None):
    """A new dense tensor on the device of `like`, in its dtype unless given."""
    if stream is None:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    return _empty(stream, shape, dtype or like.dtype, like.device)


def _matrix(name, t, rows=None, dim=None, dtype=None):
    """The row stride of a [rows, dim] tensor whose rows are dense."""
    shape = t.shape
    if len(shape) != 2 or (rows is not None and (shape[0] != rows or shape[1] != dim)):
        raise ValueError(f"{name} must be " + ("a matrix" if rows is None else f"{(rows, dim)}") + f", got {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return ld if shape[0] > 1 else shape[1]


class MoEOrder(_Described):
    """Pairs (token, choice) in the order of their experts (nq_moe_order), int32
    tensors: starts [experts + 1], place [tokens, top_k] (each pair's row),
    row_token and row_expert [tokens * top_k] (each row's token and expert id,
    which nq_gather_qmm_lhs takes as lhs_idx and rhs_idx)."""

    def __init__(self, starts, place, row_token, row_expert):
        torch = _torch()
        if place.dim() != 2:
            raise ValueError("place must be [tokens, top_k]")
        pairs = place.numel()
        for name, t, n in (("starts", starts, starts.numel()), ("place", place, pairs), ("row_token", row_token, pairs),
                           ("row_expert", row_expert, pairs)):
            _contig(name, t)
            if t.dtype != torch.int32 or t.numel() != n:
                raise ValueError(f"{name} must hold {n} int32 numbers")
            if t.device != place.device:
                raise ValueError(f"{name} is not on place's device")
        self._bind(starts, place, row_token, row_expert, *place.shape, starts.numel() - 1)

    def _bind(self, starts, place, row_token, row_expert, tokens, top_k, experts):
        struct = _MoEOrderStruct(starts.data_ptr(), place.data_ptr(), tokens, top_k, experts)
        self.__dict__.update(starts=starts, place=place, row_token=row_token, row_expert=row_expert, tokens=tokens,
                             top_k=top_k, experts=experts, _struct=struct, _ref=ctypes.byref(struct))

    @classmethod
    def empty(cls, tokens, top_k, experts, device="cuda", stream=None):
        """An order of these sizes, its contents undefined until nq_moe_sort."""
        pairs = tokens * top_k
        buf = _empty(stream, (3 * pairs + experts + 1,), _torch().int32, device)
        place, row_token, row_expert, starts = buf.split_with_sizes((pairs, pairs, pairs, experts + 1))
        self = cls.__new__(cls)
        self._bind(starts, place.view(tokens, top_k), row_token, row_expert, tokens, top_k, experts)
        return self


def nq_moe_sort_workspace_bytes(tokens, top_k, experts):
    return load_library().nq_moe_sort_workspace_bytes(tokens, top_k, experts)


def nq_moe_sort(ids, experts, order=None, workspace=None, stream=None):
    """ids [tokens, top_k] (uint32 as int32) -> a MoEOrder: pairs in the stable order of
    their experts, ids outside 0 .. experts - 1 dropped (behind the others).
    order: an existing MoEOrder of these sizes to write to.  The workspace is
    allocated here when not given."""
    torch = _torch()
    lib = _lib or load_library()
    _contig("ids", ids)
    if ids.dim() != 2 or ids.dtype != torch.int32:
        raise ValueError("ids must be int32 [tokens, top_k]")
    tokens, top_k = ids.shape
    if order is None:
        if not 1 <= experts <= 1024:
            raise ValueError(f"experts must be 1 .. 1024, got {experts}")
        order = MoEOrder.empty(tokens, top_k, experts, ids.device, stream)
    elif (order.tokens, order.top_k, order.experts) != (tokens, top_k, experts):
        raise ValueError("order was made for other sizes")
    if workspace is None:
        ws_bytes = lib.nq_moe_sort_workspace_bytes(tokens, top_k, experts)
        if ws_bytes:
            workspace = _fresh(stream, ids, (ws_bytes,), torch.uint8)
    else:
        _contig("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    on = _launch_on(stream, ids, order.place, workspace)
    status = lib.nq_moe_sort(ids.data_ptr(), tokens, top_k, experts, order.starts.data_ptr(), order.place.data_ptr(),
                             order.row_token.data_ptr(), order.row_expert.data_ptr(),
                             None if workspace is None else workspace.data_ptr(), ws_bytes, on)
    if status:
        _check(status)
    return order


def nq_moe_dispatch(order, x, xs=None, stream=None):
    """x [tokens, hidden] (f32 or bf16, any row stride) -> xs [tokens * top_k,
    hidden], the tokens' rows in the order of their experts; rows of dropped
    pairs are zeros."""
    lib = _lib or load_library()
    ldx = _matrix("x", x)
    tokens, hidden = x.shape
    if tokens != order.tokens:
        raise ValueError(f"x must have {order.tokens} rows")
    shape = (tokens * order.top_k, hidden)
    xs = _fresh(stream, x, shape) if xs is None else _given("xs", xs, shape, x.dtype)
    on = _launch_on(stream, order.place, x, xs)
    status = lib.nq_moe_dispatch(order._ref, x.data_ptr(), _type(x), ldx, hidden, xs.data_ptr(), on)
    if status:
        _check(status)
    return xs


def _expert_rows(name, order, t):
    _contig(name, t)
    if t.dim() != 2 or t.shape[0] != order.tokens * order.top_k:
        raise ValueError(f"{name} must be [{order.tokens * order.top_k}, hidden]")
    return t.shape[1]


def nq_moe_dispatch_grad(order, dxs, dx=None, stream=None):
    """The gradient of x in nq_moe_dispatch: dxs [tokens * top_k, hidden] -> dx
    [tokens, hidden]."""
    lib = _lib or load_library()
    hidden = _expert_rows("dxs", order, dxs)
    shape = (order.tokens, hidden)
    dx = _fresh(stream, dxs, shape) if dx is None else _given("dx", dx, shape, dxs.dtype)
    on = _launch_on(stream, order.place, dxs, dx)
    status = lib.nq_moe_dispatch_grad(order._ref, dxs.data_ptr(), _type(dxs), hidden, dx.data_ptr(), on)
    if status:
        _check(status)
    return dx


def _pair_weights(order, weights):
    if weights is None:
        return None
    return _given("weights", weights, (order.tokens, order.top_k), _torch().float32).data_ptr()


def nq_moe_combine(order, ys, weights=None, residual=None, y=None, stream=None):
    """ys [tokens * top_k, hidden], weights [tokens, top_k] float32 (None: ones),
    residual [tokens, hidden] or None -> y [tokens, hidden] = residual + the
    weighted sum of each token's rows."""
    lib = _lib or load_library()
    hidden = _expert_rows("ys", order, ys)
    shape = (order.tokens, hidden)
    ldr = 0 if residual is None else _matrix("residual", residual, *shape, ys.dtype)
    y = _fresh(stream, ys, shape) if y is None else _given("y", y, shape, ys.dtype)
    on = _launch_on(stream, order.place, ys, weights, residual, y)
    status = lib.nq_moe_combine(order._ref, ys.data_ptr(), _type(ys), hidden, _pair_weights(order, weights),
                                None if residual is None else residual.data_ptr(), ldr, y.data_ptr(),
                                on)
    if status:
        _check(status)
    return y


def nq_moe_combine_grad(order, dy, ys=None, weights=None, dys=None, dweights=None, stream=None):
    """The gradients of nq_moe_combine: dy [tokens, hidden] (any row stride), ys and
    weights as there -> (dys [tokens * top_k, hidden], dweights [tokens, top_k]
    float32).  ys None: only dys, dweights is None.  The residual's gradient is dy."""
    torch = _torch()
    lib = _lib or load_library()
    ldd = _matrix("dy", dy)
    tokens, hidden = dy.shape
    if tokens != order.tokens:
        raise ValueError(f"dy must have {order.tokens} rows")
    if ys is not None and (_expert_rows("ys", order, ys) != hidden or ys.dtype != dy.dtype):
        raise ValueError("ys must have dy's columns and dtype")
    if ys is None and dweights is not None:
        raise ValueError("dweights needs ys")
    shape = (tokens * order.top_k, hidden)
    dys = _fresh(stream, dy, shape) if dys is None else _given("dys", dys, shape, dy.dtype)
    if ys is not None:
        shape = (tokens, order.top_k)
        dweights = _fresh(stream, dy, shape, torch.float32) if dweights is None else \
            _given("dweights", dweights, shape, torch.float32)
    on = _launch_on(stream, order.place, dy, ys, weights, dys, dweights)
    status = lib.nq_moe_combine_grad(order._ref, dy.data_ptr(), _type(dy), ldd, hidden,
                                     None if ys is None else ys.data_ptr(), _pair_weights(order, weights),
                                     dys.data_ptr(), None if dweights is None else dweights.data_ptr(),
                                     on)
    if status:
        _check(status)
    return dys, dweights


# ---------------------------------------------------------------- norms, gate and residual
def _address(t):
    return None if t is None else t.data_ptr()


def _norm_call(like, rows, dim, post, gate, pre, scale, offset, eps):
    """The shape struct, the parameters' dtype, and gate's row stride."""
    p = post if post is not None else gate if gate is not None else pre if pre is not None else like
    dtype = p.dtype
    if post is not None:
        _given("post", post, (dim,), dtype)
    if pre is not None:
        _given("pre", pre, (dim,), dtype)
    gates, ldg = 1, 0
    if gate is not None:
        if gate.dim() == 1:
            _given("gate", gate, (dim,), dtype)
            ldg = dim
        else:
            if gate.dim() != 2 or gate.shape[1] != dim:
                raise ValueError(f"gate must be [{dim}] or [gates, {dim}], got {tuple(gate.shape)}")
            gates = gate.shape[0]
            if gates == 0:
                if rows:
                    raise ValueError("gate has no rows")
                gates = 1
            ldg = _matrix("gate", gate, dtype=dtype)
    return _BlockNormStruct(rows, dim, gates, eps, offset, scale), _type(p), ldg


def nq_block_norm_grad_workspace_bytes(rows, dim, gates=1):
    return load_library().nq_block_norm_grad_workspace_bytes(
        ctypes.byref(_BlockNormStruct(rows, dim, gates, 1e-6, 0.0, 1.0)))


def nq_block_norm(h, y=None, post=None, gate=None, pre=None, scale=1.0, offset=0.0, eps=1e-6, h_out=None, z=None,
                  stream=None):
    """A block's output y joins the residual stream h, both [rows, dim] (f32 or
    bf16, any row stride), and the next block's input leaves it:
      h_out = h + scale * gate * norm(y) * (post + offset),
      z = norm(h_out) * (pre + offset),   norm(t) = t / sqrt(mean(t^2) + eps).
    post None: y itself; gate [dim], [gates, dim] (rows / gates neighbouring rows
    each) or None; y None: h_out is h; pre None: no z.  post, gate and pre share a
    dtype.  -> (h_out, z)."""
    lib = _lib or load_library()
    ldh = _matrix("h", h)
    rows, dim = h.shape
    shape, p_dt, ldg = _norm_call(h, rows, dim, post, gate, pre, scale, offset, eps)
    ldy = 0
    if y is not None:
        ldy = _matrix("y", y, rows, dim, h.dtype)
        h_out = _fresh(stream, h, (rows, dim)) if h_out is None else _given("h_out", h_out, (rows, dim), h.dtype)
    elif h_out is not None:
        raise ValueError("h_out needs y")
    if pre is not None:
        z = _fresh(stream, h, (rows, dim)) if z is None else _given("z", z, (rows, dim), h.dtype)
    elif z is not None:
        raise ValueError("z needs pre")
    on = _launch_on(stream, h, y, post, gate, pre, h_out, z)
    status = lib.nq_block_norm(ctypes.byref(shape), h.data_ptr(), ldh, _address(y), ldy, _type(h), _address(post),
                               _address(gate), ldg, _address(pre), p_dt, _address(h_out), _address(z),
                               on)
    if status:
        _check(status)
    return (h if y is None else h_out), z


def nq_block_norm_grad(h_out, y=None, dh_out=None, dz=None, post=None, gate=None, pre=None, scale=1.0, offset=0.0,
                       eps=1e-6, parameters=True, dh=None, dy=None, workspace=None, stream=None):
    """The gradients of nq_block_norm, from h_out as it returned it and the
    gradients dh_out and dz of its outputs (None: zero) -> (dh, dy, dpost,
    dgate, dpre), None where there is no such input; dpost, dgate and dpre in their
    parameters' dtype, None with parameters=False.  The workspace is allocated here
    when not given."""
    torch = _torch()
    lib = _lib or load_library()
    ldh = _matrix("h_out", h_out)
    rows, dim = h_out.shape
    dt = h_out.dtype
    shape, p_dt, ldg = _norm_call(h_out, rows, dim, post, gate, pre, scale, offset, eps)
    ldy = 0 if y is None else _matrix("y", y, rows, dim, dt)
    ldd = 0 if dh_out is None else _matrix("dh_out", dh_out, rows, dim, dt)
    ldz = 0 if dz is None else _matrix("dz", dz, rows, dim, dt)
    dh = _fresh(stream, h_out, (rows, dim)) if dh is None else _given("dh", dh, (rows, dim), dt)
    if y is not None:
        dy = _fresh(stream, h_out, (rows, dim)) if dy is None else _given("dy", dy, (rows, dim), dt)
    elif dy is not None:
        raise ValueError("dy needs y")
    dpost = dgate = dpre = None
    if parameters:
        if post is not None:
            dpost = _fresh(stream, post, (dim,))
        if gate is not None:
            dgate = _fresh(stream, gate, gate.shape)
        if pre is not None and dz is not None:
            dpre = _fresh(stream, pre, (dim,))
    if workspace is None:
        ws_bytes = lib.nq_block_norm_grad_workspace_bytes(ctypes.byref(shape))
        if ws_bytes:
            workspace = _fresh(stream, h_out, (ws_bytes,), torch.uint8)
    else:
        _contig("workspace", workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    on = _launch_on(stream, h_out, y, dh_out, dz, post, gate, pre, dh, dy, workspace)
    status = lib.nq_block_norm_grad(ctypes.byref(shape), h_out.data_ptr(), ldh, _address(y), ldy, _address(dh_out),
                                    ldd, _address(dz), ldz, _type(h_out), _address(post), _address(gate), ldg,
                                    _address(pre), p_dt, dh.data_ptr(), _address(dy), _address(dpost), _address(dgate),
                                    _address(dpre), _address(workspace), ws_bytes, on)
    if status:
        _check(status)
    return dh, dy, dpost, dgate, dpre


# ---------------------------------------------------------------- rotary positions
class Rope(_Described):
    """How heads are turned by their position (nq_rope_plan): the first rotary_dim
    columns of a head are pairs -- "halves": column i with column i + rotary_dim
    / 2, "pairs": neighbours -- and pair i is turned by freq[i] times the position
    on axis[i].  freq: rotary_dim / 2 numbers (default theta^(-2 i /
    rotary_dim)), kept in float64.  axis: the axis of each pair, or sections: how many
    neighbouring pairs each axis has; by default there is one axis.  scale multiplies
    the result."""

    def __init__(self, rotary_dim, theta=10000.0, sections=None, axis=None, freq=None, layout="halves", scale=1.0,
                 device="cuda"):
        torch = _torch()
        half = rotary_dim // 2
        if rotary_dim < 2 or rotary_dim % 2:
            raise ValueError("rotary_dim must be even and positive")
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"unknown layout {layout!r} (one of {sorted(ROPE_LAYOUTS)})")
        if sections is not None:
            if axis is not None:
                raise ValueError("give axis or sections, not both")
            axis = [a for a, n in enumerate(sections) for _ in range(n)]
            axes = len(sections)
        else:
            axis = None if axis is None else [int(a) for a in axis]
            axes = 1 if axis is None else max(axis, default=0) + 1
        if axis is not None and (len(axis) != half or min(axis) < 0):
            raise ValueError(f"axis (or sections) must give each of the {half} pairs an axis")
        if freq is None:
            freq = theta ** (-torch.arange(half, dtype=torch.float64) / half)
        self.freq = torch.as_tensor(freq, dtype=torch.float64).to(device).contiguous().clone()
        if tuple(self.freq.shape) != (half,):
            raise ValueError(f"freq must hold {half} numbers")
        if not self.freq.is_cuda:
            raise ValueError("a Rope lives on a GPU")
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.int32).to(self.freq.device)
        self.rotary_dim, self.axes, self.layout, self.scale = rotary_dim, axes, layout, scale
        self._struct = _RopeStruct(self.freq.data_ptr(), _address(self.axis), rotary_dim, axes, ROPE_LAYOUTS[layout],
                                   scale)
        self._ref = ctypes.byref(self._struct)


def _turn(name, rope, x, positions, out, stream, names):
    torch = _torch()
    lib = _lib or load_library()
    if x.dim() != 3:
        raise ValueError(f"{names[0]} must be [rows, heads, head_dim]")
    rows, heads, dim = x.shape
    ldx = _row_stride(names[0], x, rows, heads, dim)
    if positions.dtype != torch.int32 or not positions.is_cuda:
        raise TypeError("positions must be an int32 GPU tensor")
    if positions.dim() == 1 and rope.axes == 1:
        positions = positions[None]
    if tuple(positions.shape) != (rope.axes, rows):
        raise ValueError(f"positions must be [{rope.axes}, {rows}], got {tuple(positions.shape)}")
    if rows > 1 and positions.stride(1) != 1:
        raise ValueError("the positions of an axis must be contiguous")
    ldp = positions.stride(0) if rope.axes > 1 else rows
    if out is None:
        out = _fresh(stream, x, (rows, heads, dim))
        ldo = heads * dim
    else:
        if out.dtype != x.dtype:
            raise TypeError(f"{names[1]} must have {names[0]}'s dtype")
        ldo = _row_stride(names[1], out, rows, heads, dim)
    on = _launch_on(stream, rope.freq, x, positions, out)
    status = getattr(lib, name)(rope._ref, x.data_ptr(), _type(x), rows, ldx, heads, dim, positions.data_ptr(), ldp,
                                out.data_ptr(), ldo, on)
    if status:
        _check(status)
    return out


def nq_rope(rope, x, positions, out=None, stream=None):
    """x [rows, heads, head_dim] (f32 or bf16, any row stride, e.g. columns of a
    fused projection) turned by positions, int32 [axes, rows] (an expanded
    [rows] too, or [rows] itself with one axis) -> out, dense unless given; out=x turns in place."""
    return _turn("nq_rope", rope, x, positions, out, stream, ("x", "out"))


def nq_rope_grad(rope, dout, positions, dx=None, stream=None):
    """The gradient of x in nq_rope: dout [rows, heads, head_dim] turned back."""
    return _turn("nq_rope_grad", rope, dout, positions, dx, stream, ("dout", "dx"))
