"""ctypes binding of librq.so: argument marshalling only.

Each function checks that tensors live on the current CUDA device with the
expected dtype and contiguity, then passes raw device pointers, sizes and the
current stream to the C entry point of the same name.  All compute runs in the
library's kernels; a non-OK status raises :class:`RQError`.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "librq.so")

RQ_SIGNS_FIRST = 1
RQ_ATTN_ROTATED_OUT = 2
RQ_INT8_CODES = 4
RQ_GROUP_SCALES = 8
RQ_E4M3_CODES = 16      # rq_fwht_quant: INT4 codes as the product's E4M3 operand bytes
RQ_INT4_BYTES = 32      # rq_fwht_quant: INT4 codes, one int8 byte each (the W4A8 product's A operand)
RQ_A_E4M3 = 16          # rq_w4a4_gemm: a_q holds those bytes
RQ_KV_ROTATED_OUT = 2     # rq_kv_read: rows left in the rotated basis
RQ_ROPE_INTERLEAVED = 4   # rq_rope, rq_kv_append: pairs of neighbouring elements
RQ_ROPE_INVERSE = 8       # rq_rope: the transposed turn

_STATUS = {0: "RQ_OK", 1: "RQ_ERR_INVALID_ARG", 2: "RQ_ERR_UNSUPPORTED", 3: "RQ_ERR_MISALIGNED",
           4: "RQ_ERR_CUDA", 5: "RQ_ERR_TIMEOUT"}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.int32: 3}

_lib = None


class RQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load librq.so (built by ``__graft_entry__.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"librq.so not found at {_LIB_PATH}: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i64, u64, u32, i32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint32,
                             ctypes.c_int)
    lib.rq_fwht_quant.restype = i32
    lib.rq_fwht_quant.argtypes = [P, i32, i64, i64, i64, u64, u32, P, P, P, P]
    lib.rq_w4a4_gemm.restype = i32
    lib.rq_w4a4_gemm.argtypes = [P, P, P, P, i64, i64, i64, u64, u32, P, i32, P]
    lib.rq_kv_rotate_quant.restype = i32
    lib.rq_kv_rotate_quant.argtypes = [P, P, i32, i64, i64, i64, u64, u32, P, P, P, P, P]
    lib.rq_fwht_quant_gemm.restype = i32
    lib.rq_fwht_quant_gemm.argtypes = [P, i32, i64, i64, i64, u64, u32, P, P, i64, P, i32, P, P, P]
    lib.rq_w4a8_gemm.restype = i32
    lib.rq_w4a8_gemm.argtypes = [P, P, P, P, i64, i64, i64, i64, P, i32, P]
    lib.rq_attn_decode.restype = i32
    lib.rq_attn_decode.argtypes = [P, i32, i64, i64, i64, P, P, P, P, i64, u64, u32, ctypes.c_float, P, P]
    f32 = ctypes.c_float
    lib.rq_rope.restype = i32
    lib.rq_rope.argtypes = [P, i64, i64, i64, P, i64, i64] * 2 + [i32, i64, i64, i64, P, P, f32, u32, P]
    lib.rq_kv_append.restype = i32
    lib.rq_kv_append.argtypes = [P, i64, i64, P, i64, i64, i32, i64, i64, i64, P, P, P, i64, f32, u64, u32,
                                 P, P, P, P, i64, i64, P]
    lib.rq_kv_read.restype = i32
    lib.rq_kv_read.argtypes = [P, P, P, P, i64, i64, i64, i64, P, i64, P, P, i64, i64, u64, u32, P, P, i32, P]
    lib.rq_attn_tree_workspace.restype = i64
    lib.rq_attn_tree_workspace.argtypes = [i64]
    lib.rq_attn_tree.restype = i32
    lib.rq_attn_tree.argtypes = [P, i64, i64, i32, i64, i64, i64, P, P, P, P, i64, i64, i64, P, i64, P, P, i64, i64,
                                 P, i64, u64, u32, f32, P, P, i64, P]
    lib.rq_sync_status.restype = i32
    lib.rq_sync_status.argtypes = [P]
    lib.rq_selftest_wait_timeout.restype = i32
    lib.rq_selftest_wait_timeout.argtypes = [i64, P]
    lib.rq_probe_f8_mma.restype = i32
    lib.rq_probe_f8_mma.argtypes = [i64, P, P]
    lib.rq_status_string.restype = ctypes.c_char_p
    lib.rq_status_string.argtypes = [i32]
    lib.rq_version.restype = u32
    lib.rq_version.argtypes = []
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, st):
    if st != 0:
        raise RQError(fn, st)


def _dev(*tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors must be on one device")
    return dev


def _expect(t, name: str, shape, dtypes, *, optional: bool = False):
    """Check a tensor the caller passes in (an output buffer, a scale vector):
    exact shape, dtype and contiguity, so that no kernel reads or writes past the
    end of a buffer the C side cannot size-check."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    dtypes = dtypes if isinstance(dtypes, (tuple, list)) else (dtypes,)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_OUT_DTYPES = (torch.float16, torch.float32, torch.int32)


def fwht_quant(x: torch.Tensor, seed: int, flags: int = RQ_SIGNS_FIRST, *, q=None, scales=None,
               y=None, want_y: bool = False, stream=None):
    """Rotate each row of ``x`` (rows x n; row stride may exceed n) by the
    randomized Hadamard R and quantize it to packed INT4.

    Returns ``(q, scales)`` or ``(q, scales, y)`` when ``want_y``: q is
    (rows x n/2) uint8, scales (rows,) fp32, y (rows x n) fp32 = x R.  With
    RQ_INT8_CODES in flags q is (rows x n) int8; with RQ_GROUP_SCALES scales is
    (rows x n/128); with RQ_E4M3_CODES q is (rows x n) uint8, the same INT4 codes
    as the product's operand bytes (see include/rq.h), and scales (rows x 2)
    holds each row's scale and code sum; with RQ_INT4_BYTES q is
    (rows x n) int8, the INT4 codes one per byte (for w4a8_gemm: a W4A4 product
    with per-group weight scales)."""
    lib = load_library()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride in the last dimension")
    if x.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError("x must be float32, bfloat16 or float16")
    rows, n = x.shape
    if flags & (RQ_INT8_CODES | RQ_INT4_BYTES):
        q_shape, q_dtype = (rows, n), torch.int8
    elif flags & RQ_E4M3_CODES:
        q_shape, q_dtype = (rows, n), torch.uint8
    else:
        q_shape, q_dtype = (rows, n // 2), torch.uint8
    s_shape = (rows, n // 128) if flags & RQ_GROUP_SCALES else ((rows, 2) if flags & RQ_E4M3_CODES else (rows,))
    if q is None:
        q = torch.empty(q_shape, dtype=q_dtype, device=x.device)
    if scales is None:
        scales = torch.empty(s_shape, dtype=torch.float32, device=x.device)
    if want_y and y is None:
        y = torch.empty(rows, n, dtype=torch.float32, device=x.device)
    _expect(q, "q", q_shape, q_dtype)
    _expect(scales, "scales", s_shape, torch.float32)
    _expect(y, "y", (rows, n), torch.float32, optional=True)
    _dev(x, q, scales, y)
    with torch.cuda.device(x.device):
        st = lib.rq_fwht_quant(_ptr(x), _DTYPES[x.dtype], rows, n, x.stride(0), seed, flags,
                               _ptr(q), _ptr(scales), _ptr(y), _stream(stream))
    _check("rq_fwht_quant", st)
    return (q, scales, y) if y is not None else (q, scales)


def w4a4_gemm(a_q: torch.Tensor, a_scales, w_q: torch.Tensor, w_scales, *, out_dtype=torch.float16,
              seed: int = 0, out=None, stream=None):
    """y = dequant(Q(XR) . Q(R^T W)): a_q (M x K/2), w_q (N x K/2) packed codes,
    a_scales (M,), w_scales (N,).  out_dtype float16 / float32, or int32 for the
    raw accumulators.  a_q of shape (M x K) holds the activation codes in the
    operand form of fwht_quant(..., RQ_E4M3_CODES) (more than 64 rows); a_scales
    is then the (M x 2) scales-and-code-sums it returns, needed for int32 too.
    With operand-form activations, w_scales of shape (N x K/128) are per-group
    weight scales (fwht_quant(..., RQ_GROUP_SCALES) on the rows of W^T): fp16
    or fp32 output, N a multiple of 128, K <= 8192."""
    lib = load_library()
    M, ka = a_q.shape
    N, kb2 = w_q.shape
    if a_q.dtype != torch.uint8 or w_q.dtype != torch.uint8 or ka not in (kb2, 2 * kb2):
        raise ValueError("a_q (M x K/2, or M x K operand bytes) and w_q (N x K/2) must be uint8")
    if not (a_q.is_contiguous() and w_q.is_contiguous()):
        raise ValueError("packed operands must be contiguous")
    K = 2 * kb2
    flags = RQ_A_E4M3 if ka == K else 0
    if isinstance(w_scales, torch.Tensor) and w_scales.dim() == 2:
        if not flags:
            raise ValueError("per-group w_scales need the operand-form activations (a_q of shape M x K)")
        flags |= RQ_GROUP_SCALES
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=a_q.device)
    _expect(out, "out", (M, N), _OUT_DTYPES)
    raw = out.dtype == torch.int32       # raw accumulators: the scales are not read
    if flags & RQ_A_E4M3:
        _expect(a_scales, "a_scales", (M, 2), torch.float32)   # (scale, code sum) per row
    else:
        _expect(a_scales, "a_scales", (M,), torch.float32, optional=raw)
    if flags & RQ_GROUP_SCALES:
        if raw:
            raise ValueError("per-group scales give fp16 or fp32 output, not raw int32 accumulators")
        _expect(w_scales, "w_scales", (N, K // 128), torch.float32)
    else:
        _expect(w_scales, "w_scales", (N,), torch.float32, optional=raw)
    _dev(a_q, w_q, a_scales, w_scales, out)
    with torch.cuda.device(a_q.device):
        st = lib.rq_w4a4_gemm(_ptr(a_q), _ptr(a_scales), _ptr(w_q), _ptr(w_scales), M, N, K, seed, flags,
                              _ptr(out), _DTYPES[out.dtype], _stream(stream))
    _check("rq_w4a4_gemm", st)
    return out


def kv_rotate_quant(k, v, seed: int, flags: int = RQ_SIGNS_FIRST, *, out=None, stream=None):
    """K, V ([tokens][heads][head_dim], contiguous; either may be None) ->
    dict(kq, ks, vq, vs): packed codes [T][H][D/2] uint8 and scales [T][H] fp32."""
    lib = load_library()
    ref = k if k is not None else v
    if ref is None:
        raise ValueError("k and v cannot both be None")
    T, H, D = ref.shape
    for t in (k, v):
        if t is not None and (t.shape != ref.shape or t.dtype != ref.dtype or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous with the same shape and dtype")
    if out is None:
        out = {}
        if k is not None:
            out["kq"] = torch.empty(T, H, D // 2, dtype=torch.uint8, device=ref.device)
            out["ks"] = torch.empty(T, H, dtype=torch.float32, device=ref.device)
        if v is not None:
            out["vq"] = torch.empty(T, H, D // 2, dtype=torch.uint8, device=ref.device)
            out["vs"] = torch.empty(T, H, dtype=torch.float32, device=ref.device)
    for src, qk, sk in ((k, "kq", "ks"), (v, "vq", "vs")):
        if src is not None:
            _expect(out.get(qk), f"out[{qk!r}]", (T, H, D // 2), torch.uint8)
            _expect(out.get(sk), f"out[{sk!r}]", (T, H), torch.float32)
    _dev(k, v, *out.values())
    with torch.cuda.device(ref.device):
        st = lib.rq_kv_rotate_quant(_ptr(k), _ptr(v), _DTYPES[ref.dtype], T, H, D, seed, flags,
                                    _ptr(out.get("kq")), _ptr(out.get("ks")), _ptr(out.get("vq")),
                                    _ptr(out.get("vs")), _stream(stream))
    _check("rq_kv_rotate_quant", st)
    return out


def fwht_quant_gemm(x: torch.Tensor, seed: int, flags: int, w_q: torch.Tensor, w_scales, *,
                    out_dtype=torch.float16, out=None, a_q=None, a_scales=None, stream=None):
    """Decode-sized fusion of :func:`fwht_quant` and :func:`w4a4_gemm`: x (M x K,
    bf16/fp16, unit stride in the last dimension; M <= 16, K = 1024, 2048, 4096 or
    8192) is rotated,
    quantized and multiplied by w_q (N x K/2 packed codes, N a multiple of 128)
    in one launch.  Returns y (M x N, out_dtype float16 / float32 / int32 raw
    accumulators); a_q (M x K/2) and a_scales (M,), when given, receive the
    activation codes and scales."""
    lib = load_library()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride in the last dimension")
    M, K = x.shape
    N, kb = w_q.shape
    if kb * 2 != K or w_q.dtype != torch.uint8 or not w_q.is_contiguous():
        raise ValueError("w_q must be contiguous uint8 with K/2 columns")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("x must be bfloat16 or float16")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    _expect(out, "out", (M, N), _OUT_DTYPES)
    _expect(w_scales, "w_scales", (N,), torch.float32, optional=out.dtype == torch.int32)
    _expect(a_q, "a_q", (M, K // 2), torch.uint8, optional=True)
    _expect(a_scales, "a_scales", (M,), torch.float32, optional=True)
    _dev(x, w_q, w_scales, out, a_q, a_scales)
    with torch.cuda.device(x.device):
        st = lib.rq_fwht_quant_gemm(_ptr(x), _DTYPES[x.dtype], M, K, x.stride(0), seed, flags, _ptr(w_q),
                                    _ptr(w_scales), N, _ptr(out), _DTYPES[out.dtype], _ptr(a_q), _ptr(a_scales),
                                    _stream(stream))
    _check("rq_fwht_quant_gemm", st)
    return out


def attn_decode(q: torch.Tensor, cache: dict, seed: int, flags: int = RQ_SIGNS_FIRST, softmax_scale=None, *,
                out=None, stream=None):
    """Attention of query rows q ([M][heads][head_dim], contiguous fp32/bf16/fp16)
    over the rotated INT4 cache that :func:`kv_rotate_quant` wrote (a dict with kq,
    ks, vq, vs).  Returns out [M][heads][head_dim] fp32: (sum_t p_t v^_t) R^T, or the
    rotated sum with RQ_ATTN_ROTATED_OUT in flags.  softmax_scale defaults to
    1/sqrt(head_dim)."""
    lib = load_library()
    if q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [M][heads][head_dim] tensor")
    M, H, D = q.shape
    kq, ks, vq, vs = cache["kq"], cache["ks"], cache["vq"], cache["vs"]
    T = kq.shape[0]
    for t, shape, dt in ((kq, (T, H, D // 2), torch.uint8), (vq, (T, H, D // 2), torch.uint8),
                         (ks, (T, H), torch.float32), (vs, (T, H), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous():
            raise ValueError("cache tensors must be contiguous with the kv_rotate_quant layout")
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if q.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError("q must be float32, bfloat16 or float16")
    if out is None:
        out = torch.empty(M, H, D, dtype=torch.float32, device=q.device)
    _expect(out, "out", (M, H, D), torch.float32)
    _dev(q, kq, ks, vq, vs, out)
    with torch.cuda.device(q.device):
        st = lib.rq_attn_decode(_ptr(q), _DTYPES[q.dtype], M, H, D, _ptr(kq), _ptr(ks), _ptr(vq), _ptr(vs), T,
                                seed, flags, float(softmax_scale), _ptr(out), _stream(stream))
    _check("rq_attn_decode", st)
    return out


def w4a8_gemm(a_q: torch.Tensor, a_scales, w_q: torch.Tensor, w_scales, *, out_dtype=torch.float16, out=None,
              stream=None):
    """a_q (M x K int8) x w_q (N x K/2 packed INT4): y (M x N).  w_scales of shape (N,)
    are per channel, (N, K/128) per group of 128; out_dtype float16 / float32, or
    int32 (raw exact sums, per-channel scales only)."""
    lib = load_library()
    M, K = a_q.shape
    N, kb = w_q.shape
    if kb * 2 != K or a_q.dtype != torch.int8 or w_q.dtype != torch.uint8:
        raise ValueError("a_q must be int8 (M x K), w_q uint8 (N x K/2)")
    if not (a_q.is_contiguous() and w_q.is_contiguous()):
        raise ValueError("a_q and w_q must be contiguous")
    per_group = w_scales is not None and w_scales.dim() == 2 and w_scales.shape[1] != 1
    group = 128 if per_group else K
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=a_q.device)
    _expect(out, "out", (M, N), _OUT_DTYPES)
    raw = out.dtype == torch.int32
    _expect(a_scales, "a_scales", (M,), torch.float32, optional=raw)
    sw_shape = (N, K // 128) if per_group else ((N, 1) if w_scales is not None and w_scales.dim() == 2 else (N,))
    _expect(w_scales, "w_scales", sw_shape, torch.float32, optional=raw)
    _dev(a_q, a_scales, w_q, w_scales, out)
    with torch.cuda.device(a_q.device):
        st = lib.rq_w4a8_gemm(_ptr(a_q), _ptr(a_scales), _ptr(w_q), _ptr(w_scales), M, N, K, group, _ptr(out),
                              _DTYPES[out.dtype], _stream(stream))
    _check("rq_w4a8_gemm", st)
    return out


# ---- rotary positions, the paged cache and the attention over it ----

# Small calls cost what their checks cost, so these entry points ask for a tensor's
# properties once, compare device numbers, and take the raw stream handle.
# A torch that lacks the short forms of these has the public ones.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)


def _call(fn, name, dev: int, stream, *args):
    """Call a C entry point on device `dev` and its current (or the given) stream."""
    raw = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == _current_device():
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != 0:
        raise RQError(name, st)


def _empty(shape, dtype, device, stream):
    """New memory that a call on `stream` (None: the current one) writes: it has to come from that stream's pool, where
    earlier uses are ordered before the call and later ones behind it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _one_device(dev: int, *tensors):
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensors must be on one device")


def _expect_heads(t, name: str):
    """A [tokens][heads][head_dim] tensor: any token and head strides, unit stride inside a head.  Returns its shape and
    token and head strides; the stride of a dimension of size one, which nothing uses, is that of contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] != 1):
        raise ValueError(f"{name} must be [tokens][heads][head_dim] with unit stride in the last dimension")
    if t.dtype not in _FLOATS:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    H, D = shape[1], shape[2]
    return shape, (stride[0] if shape[0] != 1 else H * D, stride[1] if H != 1 else D)


def _expect_same(t, name: str, dtype, tokens: int):
    """The same, of a given dtype and number of tokens."""
    shape, stride = _expect_heads(t, name)
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if shape[0] != tokens:
        raise ValueError(f"{name}: expected {tokens} tokens, got {shape[0]}")
    return shape, stride


def _expect_vector(t, name: str, dtype, n: int, what: str):
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {what}")


def _expect_turns(turns, head_dim: int) -> int:
    if turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
        raise ValueError("turns must be a contiguous 1-D int64 tensor (rope_turns)")
    rot = 2 * turns.shape[0]
    if not 2 <= rot <= head_dim:
        raise ValueError(f"turns rotate {rot} of {head_dim} elements")
    return rot


def rope_turns(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
               original_length: int = 8192, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Rotary frequencies for :func:`rope` and :func:`kv_append`: ``(turns, mscale)``, turns an int64 tensor of
    rot_dim/2 frequencies in 2^-64 turns per position, mscale the factor the rotated values are multiplied by.

    w_i = base^(-2i/rot_dim) radians per position, scaled for contexts `factor` times longer:

    * ``"none"``: w_i;
    * ``"linear"``: w_i / factor (positions interpolated);
    * ``"base"``: base * factor^(rot_dim / (rot_dim - 2)), which leaves the fastest pair and interpolates the slowest;
    * ``"parts"``: pairs that turn more than `fast` times within original_length stay, those below `slow` turns
      are interpolated, with a ramp in the turns in between; mscale = 0.1 ln(factor) + 1 (Peng et al. 2023,
      "YaRN: Efficient Context Window Extension of Large Language Models");
    * ``"smooth"``: the same frequencies with mscale 1 (fast = 4, slow = 1 are usual there).
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if factor <= 0 or base <= 0 or not fast > slow:
        raise ValueError("factor and base must be positive, fast above slow")
    half, mscale = rot_dim // 2, 1.0
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    w = [base ** (-i / half) for i in range(half)]
    if scaling == "linear":
        w = [x / factor for x in w]
    elif scaling in ("parts", "smooth"):
        def kept(x):
            return min(1.0, max(0.0, (original_length * x / (2 * math.pi) - slow) / (fast - slow)))
        w = [x * kept(x) + x / factor * (1.0 - kept(x)) for x in w]
        if scaling == "parts" and factor > 1.0:
            mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    turns = [int(round(x / (2 * math.pi) * 2.0**64)) % (1 << 64) for x in w]
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device), mscale


def rope(q, k, positions: torch.Tensor, turns: torch.Tensor, *, interleaved: bool = False, inverse: bool = False,
         mscale: float = 1.0, out=None, stream=None):
    """Rotary positions on q and k ([tokens][heads][head_dim], strided views welcome; either may be None): the first
    2 * len(turns) elements of each head turn by positions[token] * turns, the others pass.  Returns (q', k'), new
    contiguous tensors or the pair given as `out` (which may be (q, k): in place).  ``inverse=True`` is the transposed
    turn, the gradient of the forward one, which backward() takes where q or k asks for a gradient (not with `out`).
    turns and mscale come from :func:`rope_turns`."""
    if (q is not None and q.requires_grad or k is not None and k.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot take part where gradients are asked for")
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            return _Rope.apply(q, k, positions, turns, interleaved, inverse, mscale)
    lib = _lib or load_library()
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q and k cannot both be None")
    dtype, dev, device = ref.dtype, ref.get_device(), ref.device
    T, D = ref.shape[0], ref.shape[-1]
    args, outs = [], []
    for i, x in enumerate((q, k)):
        if x is None:
            args += (None, 0, 0, 0, None, 0, 0)
            outs.append(None)
            continue
        name = "qk"[i]
        shape, xs = _expect_same(x, name, dtype, T)
        H = shape[1]
        if shape[2] != D:
            raise ValueError("q and k must have one head_dim")
        if out is None or out[i] is None:
            o, ot, oh = _empty(shape, dtype, device, stream), H * D, D
        else:
            o = out[i]
            oshape, os = _expect_same(o, f"out ({name})", dtype, T)
            if oshape != shape:
                raise ValueError(f"out ({name}): expected shape {tuple(shape)}, got {tuple(oshape)}")
            ot, oh = os[0], os[1]
            _one_device(dev, o)
        if x.get_device() != dev:
            raise ValueError("tensors must be on one device")
        args += (x.data_ptr(), H, xs[0], xs[1], o.data_ptr(), ot, oh)
        outs.append(o)
    _expect_vector(positions, "positions", torch.int64, T, "int64 tensor with one entry per token")
    rot = _expect_turns(turns, D)
    _one_device(dev, positions, turns)
    _call(lib.rq_rope, "rq_rope", dev, stream, *args, _DTYPES[dtype], T, D, rot, positions.data_ptr(), turns.data_ptr(),
          mscale, (RQ_ROPE_INTERLEAVED if interleaved else 0) | (RQ_ROPE_INVERSE if inverse else 0))
    return tuple(outs)


class _Rope(torch.autograd.Function):
    """rope of what asks for a gradient: backward is the transposed turn of the gradients that arrive."""

    @staticmethod
    def forward(ctx, q, k, positions, turns, interleaved, inverse, mscale):
        ctx.save_for_backward(positions, turns)
        ctx.turn = dict(interleaved=interleaved, inverse=not inverse, mscale=mscale)
        ctx.set_materialize_grads(False)
        out = rope(q, k, positions, turns, interleaved=interleaved, inverse=inverse, mscale=mscale)
        ctx.mark_non_differentiable(*(o for x, o in zip((q, k), out) if x is not None and not x.requires_grad))
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        gq, gk = (g.contiguous() if g is not None and ctx.needs_input_grad[i] else None for i, g in enumerate((gq, gk)))
        if gq is not None or gk is not None:
            gq, gk = rope(gq, gk, *ctx.saved_tensors, **ctx.turn)
        return gq, gk, None, None, None, None, None


def kv_cache(pages: int, heads: int, head_dim: int, page_size: int = 64, device="cuda") -> dict:
    """An empty paged cache: dict(kq, ks, vq, vs) with codes [pages][heads][page_size][head_dim/2] uint8 and scales
    [pages][heads][page_size] fp32."""
    cache = {}
    for n in "kv":
        cache[n + "q"] = torch.zeros(pages, heads, page_size, head_dim // 2, dtype=torch.uint8, device=device)
        cache[n + "s"] = torch.zeros(pages, heads, page_size, dtype=torch.float32, device=device)
    return cache


def _cache_parts(cache, head_dim=None):
    """The cache's tensors and its shape [pages][heads][page_size][head_dim/2]."""
    kq, ks, vq, vs = cache["kq"], cache["ks"], cache["vq"], cache["vs"]
    shape = kq.shape
    if len(shape) != 4 or (head_dim is not None and shape[3] * 2 != head_dim):
        raise ValueError(f"cache['kq']: expected [pages][heads][page_size][head_dim/2], got {tuple(shape)}")
    if not (kq.dtype is vq.dtype is torch.uint8 and ks.dtype is vs.dtype is torch.float32):
        raise ValueError("cache: codes are uint8 and scales float32")
    if vq.shape != shape or ks.shape != shape[:3] or vs.shape != ks.shape:
        raise ValueError("cache: kq and vq, ks and vs must agree in shape")
    if not (kq.is_contiguous() and ks.is_contiguous() and vq.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache tensors must be contiguous")
    return kq, ks, vq, vs, shape


def _expect_table(t):
    if t.dim() != 2 or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 tensor [seqs][width]")
    return t.shape


def kv_append(k, v, cache: dict, slots: torch.Tensor, seed: int, flags: int = RQ_SIGNS_FIRST, *, positions=None,
              turns=None, interleaved: bool = False, mscale: float = 1.0, stream=None) -> dict:
    """Quantise k and v ([tokens][heads][head_dim], strided views welcome) into the paged cache: row t goes to slot
    slots[t] = page * page_size + row (int64; outside the cache: skipped).  With positions and turns the keys take
    their rotary positions on the way (see :func:`rope`).  Returns the cache, which carries no gradient."""
    lib = _lib or load_library()
    kshape, kst = _expect_heads(k, "k")
    T, H, D = kshape
    dtype, dev = k.dtype, k.get_device()
    vshape, vst = _expect_same(v, "v", dtype, T)
    if vshape != kshape:
        raise ValueError(f"v: expected shape {tuple(kshape)}, got {tuple(vshape)}")
    kq, ks, vq, vs, shape = _cache_parts(cache, D)
    if shape[1] != H:
        raise ValueError(f"cache holds {shape[1]} heads, k has {H}")
    _expect_vector(slots, "slots", torch.int64, T, "int64 tensor with one entry per token")
    if (positions is None) != (turns is None):
        raise ValueError("positions and turns go together")
    rot, pp, tp = 0, None, None
    if turns is not None:
        _expect_vector(positions, "positions", torch.int64, T, "int64 tensor with one entry per token")
        rot, pp, tp = _expect_turns(turns, D), positions.data_ptr(), turns.data_ptr()
        _one_device(dev, positions, turns)
    _one_device(dev, v, kq, ks, vq, vs, slots)
    _call(lib.rq_kv_append, "rq_kv_append", dev, stream, k.data_ptr(), kst[0], kst[1], v.data_ptr(), vst[0], vst[1],
          _DTYPES[dtype], T, H, D, slots.data_ptr(), pp, tp, rot, mscale, seed,
          flags | RQ_ROPE_INTERLEAVED if interleaved else flags, kq.data_ptr(), ks.data_ptr(), vq.data_ptr(),
          vs.data_ptr(), shape[0], shape[2])
    return cache


def kv_read(cache: dict, block_table: torch.Tensor, starts, offsets: torch.Tensor, total: int, seed: int,
            flags: int = RQ_SIGNS_FIRST, *, dtype=torch.bfloat16, out=None, stream=None):
    """Sequences of the paged cache as dense rows (k, v), [total][heads][head_dim] of `dtype` (or the pair `out`), in
    the original basis, or the rotated one with RQ_KV_ROTATED_OUT in flags.  block_table [seqs][width] int32; starts
    [seqs] int32 (first token wanted; None: 0); offsets [seqs + 1] int32: sequence b fills rows offsets[b] to
    offsets[b + 1] - 1; rows at or past offsets[seqs] are left as they are."""
    lib = _lib or load_library()
    kq, ks, vq, vs, shape = _cache_parts(cache)
    pages, H, page, half = shape
    B, W = _expect_table(block_table)
    _expect_vector(offsets, "offsets", torch.int32, B + 1, "int32 tensor [seqs + 1]")
    dev, sp = kq.get_device(), None
    if starts is not None:
        _expect_vector(starts, "starts", torch.int32, B, "int32 tensor [seqs]")
        _one_device(dev, starts)
        sp = starts.data_ptr()
    if dtype not in _FLOATS:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if out is None:
        device = kq.device
        ko = _empty((total, H, 2 * half), dtype, device, stream)
        vo = _empty((total, H, 2 * half), dtype, device, stream)
    else:
        ko, vo = out
        _expect(ko, "out (k)", (total, H, 2 * half), dtype)
        _expect(vo, "out (v)", (total, H, 2 * half), dtype)
        _one_device(dev, ko, vo)
    _one_device(dev, ks, vq, vs, block_table, offsets)
    _call(lib.rq_kv_read, "rq_kv_read", dev, stream, kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), pages,
          H, page, 2 * half, block_table.data_ptr(), W, sp, offsets.data_ptr(), B, total, seed, flags, ko.data_ptr(), vo.data_ptr(), _DTYPES[dtype])
    return ko, vo


_workspace_bytes: dict = {}     # by device and head_dim: a size, asked for once


def attn_tree_workspace(head_dim: int) -> int:
    """Bytes of scratch that :func:`attn_tree` needs on the current device."""
    return int(load_library().rq_attn_tree_workspace(head_dim))


def attn_tree(q: torch.Tensor, cache: dict, block_table: torch.Tensor, context_lens: torch.Tensor,
              offsets: torch.Tensor, seed: int, flags: int = RQ_SIGNS_FIRST, *, tree_mask=None, max_nodes=None,
              softmax_scale=None, out=None, workspace=None, stream=None):
    """Attention of trees of drafted tokens over the paged cache.  Rows offsets[b] .. offsets[b + 1] - 1 of q
    ([rows][q_heads][head_dim], strided views welcome) are the nodes of sequence b, whose keys and values lie in the
    cache at places context_lens[b], context_lens[b] + 1, ...  A node sees the context and the nodes that its row of
    tree_mask (bool [rows][width], width >= the largest tree) names; without a mask, itself and those before it.
    max_nodes bounds the nodes of a sequence (default: the mask's width, or the number of rows).  One node per sequence
    is a plain decode step.  Returns [rows][q_heads][head_dim] of q's dtype; rows that see nothing are 0, rows of no
    sequence are not written.  The result carries no gradient."""
    lib = _lib or load_library()
    qshape, qs = _expect_heads(q, "q")
    N, Hq, D = qshape
    dtype, dev, device = q.dtype, q.get_device(), q.device
    kq, ks, vq, vs, shape = _cache_parts(cache, D)
    if Hq % shape[1]:
        raise ValueError(f"{Hq} query heads do not divide over {shape[1]} KV heads")
    B, W = _expect_table(block_table)
    _expect_vector(context_lens, "context_lens", torch.int32, B, "int32 tensor [seqs]")
    _expect_vector(offsets, "offsets", torch.int32, B + 1, "int32 tensor [seqs + 1]")
    mask_ptr, mask_stride = None, 0
    if tree_mask is not None:
        ms = tree_mask.shape
        if tree_mask.dtype is not torch.bool or len(ms) != 2 or ms[0] != N or (tree_mask.stride(1) != 1 and ms[1] > 1):
            raise ValueError("tree_mask must be bool [rows][width] with unit stride in the last dimension")
        mask_ptr = tree_mask.data_ptr()
        mask_stride = tree_mask.stride(0) if N > 1 else ms[1]     # the stride of a single row says nothing
        if max_nodes is None:
            max_nodes = ms[1]
        elif max_nodes > ms[1]:
            raise ValueError("tree_mask is narrower than max_nodes")
        _one_device(dev, tree_mask)
    elif max_nodes is None:
        max_nodes = N
    if out is None:
        out = _empty(qshape, dtype, device, stream)
    else:
        _expect(out, "out", (N, Hq, D), dtype)
        _one_device(dev, out)
    _one_device(dev, kq, ks, vq, vs, block_table, context_lens, offsets)
    if workspace is None:
        need = _workspace_bytes.get((dev, D))
        if need is None:
            with torch.cuda.device(dev):
                need = _workspace_bytes[dev, D] = lib.rq_attn_tree_workspace(D)
        workspace = _empty(need, torch.uint8, device, stream)
    else:
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        _one_device(dev, workspace)
        need = workspace.numel()
    _call(lib.rq_attn_tree, "rq_attn_tree", dev, stream, q.data_ptr(), qs[0], qs[1], _DTYPES[dtype], N, Hq, D,
          kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), shape[0], shape[1], shape[2],
          block_table.data_ptr(), W, context_lens.data_ptr(), offsets.data_ptr(), B, max_nodes, mask_ptr, mask_stride,
          seed, flags, D ** -0.5 if softmax_scale is None else softmax_scale, out.data_ptr(), workspace.data_ptr(), need)
    return out


def sync_status(stream=None) -> int:
    """Drain the stream and return the library's status word (0 = OK)."""
    return int(load_library().rq_sync_status(_stream(stream)))


def selftest_wait_timeout(limit_cycles: int, stream=None) -> None:
    """Launch the failure-detection self-test: a bounded device wait on a barrier
    that nothing arrives on.  The next :func:`sync_status` returns RQ_ERR_TIMEOUT."""
    _check("rq_selftest_wait_timeout", load_library().rq_selftest_wait_timeout(int(limit_cycles), _stream(stream)))


def probe_f8_mma(mmas_per_sm: int, stream=None) -> int:
    """Enqueue the tensor-pipe probe (back-to-back M128 N256 K32 FP8 MMAs, one CTA
    per SM); returns the number of CTAs.  Each MMA is 2,097,152 operations."""
    ctas = ctypes.c_int32(0)
    _check("rq_probe_f8_mma", load_library().rq_probe_f8_mma(int(mmas_per_sm), ctypes.byref(ctas), _stream(stream)))
    return int(ctas.value)
