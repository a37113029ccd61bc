"""Thin ctypes binding to liblowbit.so: the C ABI's entry points under the same names.

Argument marshalling only -- every step of every product runs in the HIP kernels behind the C ABI.
Tensors are torch device tensors (torch supplies device memory and streams); the stream defaults to
torch's current stream on the tensors' device.  A non-LB_OK status raises LowbitError.  If the shared
library is not built, importing this module raises ImportError: there is no other implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

Q1_0, Q2_0_G64, TERNARY_PLANAR, Q8_0, TERNARY_B3 = 1, 2, 3, 4, 5
ACT_Q8_0, ACT_I8_ROW, ACT_F32_Q8_0 = 1, 2, 3
F32, BF16, F16 = 0, 1, 2
LB_OK, LB_EINVAL, LB_ESHAPE, LB_EALIGN, LB_EUNSUPPORTED, LB_EDEVICE, LB_ENOMEM = range(7)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblowbit.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built (python -m bit_quantized_matvec_q1_amd.build); "
                      "the HIP library is the only implementation of this package")

_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float

lib = ctypes.CDLL(LIB_PATH)

# name -> (restype, argtypes), mirroring include/lowbit.h
SIGNATURES = {
    "lowbit_status_str": (ctypes.c_char_p, [_I]),
    "lowbit_last_error": (ctypes.c_char_p, []),
    "lowbit_weight_bytes": (_I64, [_I, _I64, _I64]),
    "lowbit_pack_weights": (_I, [_I, _P, _I64, _I64, _P, _P]),
    "lowbit_unpack_weights": (_I, [_I, _P, _I64, _I64, _P, _P]),
    "lowbit_quantize_act": (_I, [_I, _P, _I64, _I64, _P, _P, _P]),
    "lowbit_matvec": (_I, [_I, _P, _I64, _I64, _F, _I, _P, _P, _P, _P]),
    "lowbit_gemm": (_I, [_I, _P, _I64, _I64, _F, _I, _P, _P, _I64, _P, _P]),
    "lowbit_block_sums": (_I, [_I, _P, _I64, _I64, _I, _P, _P, _I64, _P, _P]),
    "dense_head_matvec": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "dense_head_matvec_i8": (_I, [_P, _P, _I64, _I64, _P, _P, _P]),
    "lowbit_matvec_popcount": (_I, [_P, _I64, _I64, ctypes.c_float, _P, _P, _P, _P, _P]),
    "lowbit_batch_create": (_I, [_P, ctypes.c_int32, _P]),
    "lowbit_matvec_batched": (_I, [_P, _P]),
    "lowbit_batch_launches": (ctypes.c_int32, [_P]),
    "lowbit_batch_destroy": (None, [_P]),
    "lowbit_matvec_batched_static": (_I, [_P, ctypes.c_int32, _P]),
    "lowbit_kv_cache_bytes": (_I64, [_I64, _I64, _I64, _I64]),
    "lowbit_kv_plan": (_I, [_P, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "lowbit_kv_release": (_I, [_P, _I64, _I64, _P, _P, _I64, _P, _I64, _P, _P, _P]),
    "lowbit_kv_append": (_I, [_I, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _I64, _I64, _P]),
    "lowbit_kv_read": (_I, [_I, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _P, _I64, _P]),
    "lowbit_kv_attention_workspace": (_I64, [_I64] * 8),
    "lowbit_kv_attention": (_I, [_I, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _I64, _I64, _I64, _F, _I64,
                                 _P, _I64, _P, _I64, _P]),
    "lowbit_logits_process": (_I, [_I, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _I64, _P, _I64, _P]),
    "lowbit_read_probe": (_I, [_P, _I64, _P, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.restype, _f.argtypes = _res, _args


class LowbitError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        msg = lib.lowbit_last_error().decode() or lib.lowbit_status_str(status).decode()
        super().__init__(f"{fn}: {lib.lowbit_status_str(status).decode()} ({msg})")


class lb_matvec_desc(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int32),
        ("afmt", ctypes.c_int32),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("W", ctypes.c_void_p),
        ("w_tensor_scale", ctypes.c_float),
        ("xq", ctypes.c_void_p),
        ("xscale", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
    ]


def _ptr(t):
    """A device tensor's address (ints pass through as raw addresses, unchecked).  Host tensors and strided
    views are refused: the kernels take dense device buffers, and a host address in a kernel is a memory
    fault."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"device tensor required, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor required (the C ABI takes dense row-major buffers)")
    return t.data_ptr()


_F16_BITS = (torch.uint16, torch.int16, torch.float16)  # binary16 scales travel as their 16-bit patterns
_BF16_BITS = (torch.uint16, torch.int16, torch.bfloat16)


def _check_arg(t, name, count, dtypes=None):
    """Check that tensor t holds at least `count` elements of one of `dtypes` (or, with dtypes None, at
    least `count` bytes of any dtype).  The kernels read and write exactly the extents the sizes imply, so
    a short buffer would be a read or write past its end: refused with ValueError.  None and raw int
    addresses are not checked (raw addresses are the caller's responsibility)."""
    if t is None or isinstance(t, int):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor, an int address or None is required")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not accepted (expected one of {[str(d) for d in dtypes]})")
    have = t.numel() if dtypes is not None else t.numel() * t.element_size()
    if count > 0 and have < count:
        unit = "elements" if dtypes is not None else "bytes"
        raise ValueError(f"{name}: needs at least {count} {unit}, has {have}")


def _args(*specs):
    """Addresses of the arguments (t, name, count[, dtypes]) after checking every one of them: all sizes and
    dtypes first, then the device and layout checks of _ptr."""
    for spec in specs:
        _check_arg(*spec)
    return [_ptr(spec[0]) for spec in specs]


def _pos(*vals):
    """Sizes as the C ABI sees them, for the extents checks: negative ones are left for the library to refuse
    (LB_ESHAPE), and a product with no rows (any size 0 but K) touches no buffer, so all extents are 0."""
    v = [max(int(x), 0) for x in vals]
    if len(v) > 1 and (v[0] == 0 or (len(v) > 2 and v[2] == 0)):  # (N, K[, M]): N == 0 or M == 0
        return [0] * len(v)
    return v


def _wbytes(fmt, N, K):
    n = lib.lowbit_weight_bytes(fmt, N, K)
    return max(n, 0)


def _scale_spec(t, name, afmt, M, K):
    """Activation scales: binary16 [M][K/32] for q8_0, fp32 [M] for per-row int8."""
    if afmt == ACT_I8_ROW:
        return (t, name, M, (torch.float32,))
    return (t, name, M * (K // 32), _F16_BITS)


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return torch.cuda.current_stream(t.device).cuda_stream
    return None


def _check(st: int, fn: str) -> None:
    if st != LB_OK:
        raise LowbitError(st, fn)


def lowbit_weight_bytes(fmt: int, N: int, K: int) -> int:
    return lib.lowbit_weight_bytes(fmt, N, K)


def lowbit_pack_weights(fmt, blocks, N, K, packed, stream=None):
    nb = _wbytes(fmt, N, K)  # the ggml block stream and the device layout have the same byte count
    pb, pp = _args((blocks, "blocks", nb), (packed, "packed", nb))
    _check(lib.lowbit_pack_weights(fmt, pb, N, K, pp, _stream(stream, packed)), "lowbit_pack_weights")


def lowbit_unpack_weights(fmt, packed, N, K, blocks, stream=None):
    nb = _wbytes(fmt, N, K)
    pp, pb = _args((packed, "packed", nb), (blocks, "blocks", nb))
    _check(lib.lowbit_unpack_weights(fmt, pp, N, K, pb, _stream(stream, packed)), "lowbit_unpack_weights")


def lowbit_quantize_act(afmt, x, M, K, xq, xscale, stream=None):
    m, k = _pos(M, K)
    px, pq, ps = _args((x, "x", m * k, (torch.float32,)), (xq, "xq", m * k, (torch.int8,)),
                       _scale_spec(xscale, "xscale", afmt, m, k))
    _check(lib.lowbit_quantize_act(afmt, px, M, K, pq, ps, _stream(stream, x)), "lowbit_quantize_act")


def lowbit_matvec(fmt, W, N, K, w_tensor_scale, afmt, xq, xscale, y, stream=None):
    n, k = _pos(N, K)
    pw, pq, ps, py = _args((W, "W", _wbytes(fmt, n, k)), (xq, "xq", k, (torch.int8,)),
                           _scale_spec(xscale, "xscale", afmt, 1, k), (y, "y", n, (torch.float32,)))
    _check(lib.lowbit_matvec(fmt, pw, N, K, float(w_tensor_scale), afmt, pq, ps, py, _stream(stream, y)),
           "lowbit_matvec")


def lowbit_gemm(fmt, W, N, K, w_tensor_scale, afmt, Xq, Xscale, M, Y, stream=None):
    n, k, m = _pos(N, K, M)
    pw, pq, ps, py = _args((W, "W", _wbytes(fmt, n, k)), (Xq, "Xq", m * k, (torch.int8,)),
                           _scale_spec(Xscale, "Xscale", afmt, m, k), (Y, "Y", m * n, (torch.float32,)))
    _check(lib.lowbit_gemm(fmt, pw, N, K, float(w_tensor_scale), afmt, pq, ps, M, py, _stream(stream, Y)),
           "lowbit_gemm")


def lowbit_block_sums(fmt, W, N, K, afmt, Xq, Xscale, M, sums, stream=None):
    n, k, m = _pos(N, K, M)
    per_row = fmt in (TERNARY_PLANAR, TERNARY_B3)  # one sum per row; else one per 32-block of K
    pw, pq, ps, pz = _args((W, "W", _wbytes(fmt, n, k)), (Xq, "Xq", m * k, (torch.int8,)),
                           _scale_spec(Xscale, "Xscale", afmt, m, k),
                           (sums, "sums", m * n * (1 if per_row else k // 32), (torch.int32,)))
    _check(lib.lowbit_block_sums(fmt, pw, N, K, afmt, pq, ps, M, pz, _stream(stream, sums)), "lowbit_block_sums")


def dense_head_matvec(W, N, K, x, y, stream=None):
    n, k = _pos(N, K)
    pw, px, py = _args((W, "W", n * k, _BF16_BITS), (x, "x", k, (torch.float32,)), (y, "y", n, (torch.float32,)))
    _check(lib.dense_head_matvec(pw, N, K, px, py, _stream(stream, y)), "dense_head_matvec")


def lowbit_matvec_popcount(W, N, K, w_tensor_scale, xq, xscale, y, row_sums=None, stream=None):
    n, k = _pos(N, K)
    pw, pq, ps, py, pr = _args((W, "W", _wbytes(TERNARY_PLANAR, n, k)), (xq, "xq", k, (torch.int8,)),
                               (xscale, "xscale", 1, (torch.float32,)), (y, "y", n, (torch.float32,)),
                               (row_sums, "row_sums", n, (torch.int32,)))
    _check(lib.lowbit_matvec_popcount(pw, N, K, float(w_tensor_scale), pq, ps, py, pr, _stream(stream, xq)),
           "lowbit_matvec_popcount")


def dense_head_matvec_i8(W, row_scale, N, K, x, y, stream=None):
    n, k = _pos(N, K)
    pw, pr, px, py = _args((W, "W", n * k, (torch.int8,)), (row_scale, "row_scale", n, (torch.float32,)),
                           (x, "x", k, (torch.float32,)), (y, "y", n, (torch.float32,)))
    _check(lib.dense_head_matvec_i8(pw, pr, N, K, px, py, _stream(stream, y)), "dense_head_matvec_i8")


def lowbit_read_probe(buf, nbytes, sink, stream=None):
    pb, ps = _args((buf, "buf", nbytes), (sink, "sink", 65536, (torch.int32, torch.uint32)))
    _check(lib.lowbit_read_probe(pb, nbytes, ps, _stream(stream, buf)), "lowbit_read_probe")


# ---- serving: block tables, the 4-bit cache, attention over it, logits ----------------------------

_DTYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
_I32 = (torch.int32,)


def _serve(fn, stream, tensors, call):
    """call(stream) on the tensors' device, which all of them have to share, whatever the current device is."""
    on = [t for t in tensors if isinstance(t, torch.Tensor)]
    for t in on:
        if not t.is_cuda:
            raise ValueError(f"device tensor required, got one on {t.device}")
        if t.device != on[0].device:
            raise ValueError(f"tensors on {on[0].device} and {t.device}: one device required")
    if not on or on[0].device.index == torch.cuda.current_device():
        _check(call(_stream(stream, *on)), fn)
        return
    with torch.cuda.device(on[0].device):
        _check(call(_stream(stream, *on)), fn)


def _row_arg(t, name, dtype, T, heads, D, stride):
    """Rows [T][heads][D]: (address, token stride).  A tensor may be a part of wider rows (any token stride, the
    row itself dense); an address takes `stride`, dense rows by default."""
    width = max(int(heads), 0) * max(int(D), 0)
    if t is None or isinstance(t, int):
        return t, width if stride is None else int(stride)
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor, an int address or None is required")
    if dtype in _DTYPES and t.dtype != _DTYPES[dtype]:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {_DTYPES[dtype]}")
    if T <= 0:
        return t.data_ptr(), width if stride is None else int(stride)
    if t.dim() == 2 and t.shape[1] == width:
        dense = t.stride(1) == 1 or width == 1
    elif t.dim() == 3 and tuple(t.shape[1:]) == (heads, D):
        dense = (t.stride(2) == 1 or D == 1) and (t.stride(1) == D or heads == 1)
    else:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, {heads}, {D}] or [T, {width}]")
    if t.shape[0] < T:
        raise ValueError(f"{name}: needs at least {T} rows, has {t.shape[0]}")
    step = t.stride(0) if T > 1 else max(t.stride(0), width)
    if not dense or step < width:
        raise ValueError(f"{name}: a row's elements have to be dense, and rows apart")
    if stride is not None and int(stride) != step:
        raise ValueError(f"{name}: stride {stride} given, the tensor's is {step}")
    return t.data_ptr(), step


def _flat(*specs):
    """Addresses of dense arguments (t, name, count[, dtypes]) after the checks of sizes, types and layout (the
    device is checked for all of a call's tensors together)."""
    out = []
    for t, name, count, *types in specs:
        _check_arg(t, name, count, *types)
        if isinstance(t, torch.Tensor) and not t.is_contiguous():
            raise ValueError(f"{name}: contiguous tensor required (the C ABI takes dense row-major buffers)")
        out.append(t.data_ptr() if isinstance(t, torch.Tensor) else t)
    return out


def _size(*v):
    """The sizes' product for the extents checks, 0 if one is not positive (the library refuses negative ones)."""
    n = 1
    for x in v:
        n *= max(int(x), 0)
    return n


def lowbit_kv_cache_bytes(pages: int, kv_heads: int, page_tokens: int, head_dim: int) -> int:
    return lib.lowbit_kv_cache_bytes(pages, kv_heads, page_tokens, head_dim)


def lowbit_kv_plan(new_lens, B, page_tokens, kv_lens, kv_lens_out, block_table, table_stride, free_pages, free_count,
                   free_count_out, cu_q, cu_pages, slots, positions, max_tokens, status, free_capacity=None, stream=None):
    """free_capacity: entries of free_pages (the tensor's size by default)."""
    if free_capacity is None:
        if not isinstance(free_pages, torch.Tensor):
            raise ValueError("free_capacity: needed where free_pages is no tensor")
        free_capacity = free_pages.numel()
    b, n = _size(B), _size(max_tokens)
    p = _flat((new_lens, "new_lens", b, _I32), (kv_lens, "kv_lens", b, _I32), (kv_lens_out, "kv_lens_out", b, _I32),
              (block_table, "block_table", _size(B, table_stride), _I32), (free_pages, "free_pages", _size(free_capacity), _I32),
              (free_count, "free_count", min(b, 1), _I32), (free_count_out, "free_count_out", min(b, 1), _I32),
              (cu_q, "cu_q", b and b + 1, _I32), (cu_pages, "cu_pages", b and b + 1, _I32), (slots, "slots", b and n, (torch.int64,)),
              (positions, "positions", b and n, _I32), (status, "status", b and 3, _I32))
    ts = (new_lens, kv_lens, kv_lens_out, block_table, free_pages, free_count, free_count_out, cu_q, cu_pages, slots, positions, status)
    _serve("lowbit_kv_plan", stream, ts, lambda s: lib.lowbit_kv_plan(
        p[0], B, page_tokens, p[1], p[2], p[3], table_stride, p[4], free_capacity, p[5], p[6], p[7], p[8], p[9], p[10], max_tokens,
        p[11], s))


def lowbit_kv_release(done, B, page_tokens, kv_lens, block_table, table_stride, free_pages, free_count, status, free_capacity=None,
                      stream=None):
    if free_capacity is None:
        if not isinstance(free_pages, torch.Tensor):
            raise ValueError("free_capacity: needed where free_pages is no tensor")
        free_capacity = free_pages.numel()
    b = _size(B)
    p = _flat((done, "done", b, _I32), (kv_lens, "kv_lens", b, _I32), (block_table, "block_table", _size(B, table_stride), _I32),
              (free_pages, "free_pages", _size(free_capacity), _I32), (free_count, "free_count", min(b, 1), _I32),
              (status, "status", b and 2, _I32))
    _serve("lowbit_kv_release", stream, (done, kv_lens, block_table, free_pages, free_count, status), lambda s: lib.lowbit_kv_release(
        p[0], B, page_tokens, p[1], p[2], table_stride, p[3], free_capacity, p[4], p[5], s))


def lowbit_kv_append(dtype, k, v, T, kv_heads, head_dim, slots, cache, pages, page_tokens, k_stride=None, v_stride=None, stream=None):
    """k, v: [T][kv_heads][head_dim] tensors (any token stride), or addresses with k_stride, v_stride."""
    nb = max(lib.lowbit_kv_cache_bytes(pages, kv_heads, page_tokens, head_dim), 0)
    (pk, sk), (pv, sv) = (_row_arg(t, n, dtype, T, kv_heads, head_dim, st) for t, n, st in ((k, "k", k_stride), (v, "v", v_stride)))
    ps, pc = _flat((slots, "slots", _size(T), (torch.int64,)), (cache, "cache", nb if T > 0 else 0))
    _serve("lowbit_kv_append", stream, (k, v, slots, cache), lambda s: lib.lowbit_kv_append(
        dtype, pk, sk, pv, sv, T, kv_heads, head_dim, ps, pc, pages, page_tokens, s))


def lowbit_kv_read(dtype, cache, pages, page_tokens, T, kv_heads, head_dim, slots, k, v, k_stride=None, v_stride=None, stream=None):
    """The rows of `slots` as the cache holds them, into k and v ([T][kv_heads][head_dim], any token stride)."""
    nb = max(lib.lowbit_kv_cache_bytes(pages, kv_heads, page_tokens, head_dim), 0)
    (pk, sk), (pv, sv) = (_row_arg(t, n, dtype, T, kv_heads, head_dim, st) for t, n, st in ((k, "k", k_stride), (v, "v", v_stride)))
    ps, pc = _flat((slots, "slots", _size(T), (torch.int64,)), (cache, "cache", nb if T > 0 else 0))
    _serve("lowbit_kv_read", stream, (k, v, slots, cache), lambda s: lib.lowbit_kv_read(
        dtype, pc, pages, page_tokens, T, kv_heads, head_dim, ps, pk, sk, pv, sv, s))


def lowbit_kv_attention_workspace(T, B, q_heads, kv_heads, head_dim, max_q, max_kv, window=0) -> int:
    return lib.lowbit_kv_attention_workspace(T, B, q_heads, kv_heads, head_dim, max_q, max_kv, window)


def lowbit_kv_attention(dtype, q, T, B, q_heads, kv_heads, head_dim, cu_q, kv_lens, block_table, table_stride, cache, pages,
                        page_tokens, max_q, max_kv, scale, out, window=0, workspace=None, q_stride=None, out_stride=None, stream=None):
    """q, out: [T][q_heads][head_dim] tensors (any token stride), or addresses with q_stride, out_stride.
    workspace: a tensor of at least lowbit_kv_attention_workspace(...) bytes; by default one is taken from torch's
    allocator for the stream the call runs on."""
    nb = max(lib.lowbit_kv_cache_bytes(pages, kv_heads, page_tokens, head_dim), 0)
    some = T > 0 and B > 0
    (pq, sq), (po, so) = (_row_arg(t, n, dtype, T, q_heads, head_dim, st) for t, n, st in ((q, "q", q_stride), (out, "out", out_stride)))
    pcu, pl, pt, pc = _flat((cu_q, "cu_q", _size(B) + 1 if some else 0, _I32), (kv_lens, "kv_lens", _size(B) if some else 0, _I32),
                            (block_table, "block_table", _size(B, table_stride) if some else 0, _I32),
                            (cache, "cache", nb if some else 0))
    need = lib.lowbit_kv_attention_workspace(T, B, q_heads, kv_heads, head_dim, max_q, max_kv, window)

    def call(s):
        ws = workspace
        if ws is None and need > 0:
            at = out if isinstance(out, torch.Tensor) else None
            dev = at.device if at is not None else torch.device("cuda", torch.cuda.current_device())
            if s == torch.cuda.current_stream(dev).cuda_stream:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
            else:  # of the other stream's own, so that nothing else gets it while that stream still works on it
                with torch.cuda.stream(torch.cuda.ExternalStream(s or 0, device=dev)):
                    ws = torch.empty(need, dtype=torch.uint8, device=dev)
        have = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else max(need, 0)
        (pw,) = _flat((ws, "workspace", max(need, 0)))
        return lib.lowbit_kv_attention(dtype, pq, sq, T, B, q_heads, kv_heads, head_dim, pcu, pl, pt, table_stride, pc, pages,
                                       page_tokens, max_q, max_kv, float(scale), window, po, so, pw, have, s)

    _serve("lowbit_kv_attention", stream, (q, out, cu_q, kv_lens, block_table, cache, workspace), call)


def _matrix(t, name, rows, width, types):
    """A [rows][>= width] matrix with dense rows: (address, row stride in elements).  width None: any."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.dtype not in types:
        raise ValueError(f"{name}: a tensor of one of {[str(d) for d in types]} is required")
    if t.dim() != 2 or t.shape[0] < rows or (width is not None and t.shape[1] < width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, needs at least [{rows}, {width if width is not None else 'any'}]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: dense rows required")
    step = t.stride(0) if rows > 1 else max(t.stride(0), t.shape[1])
    if rows > 1 and step < t.shape[1]:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), step


def lowbit_logits_process(dtype, logits, B, V, out, tokens=None, prompt_lens=None, total_lens=None, repetition=None, presence=None,
                          frequency=None, bias_tokens=None, bias_values=None, bias_lens=None, mask=None, stream=None):
    """logits, out [B][>= V] (out may be logits); tokens, bias_tokens, bias_values int32/int32/fp32 matrices with a
    row a request; mask: int32 or uint32 words [B][>= ceil(V / 32)]; the rest vectors of B (include/lowbit.h)."""
    b = _size(B)
    types = (_DTYPES[dtype],) if dtype in _DTYPES else tuple(_DTYPES.values())
    pin, sin = _matrix(logits, "logits", b, _size(V), types)
    po, so = _matrix(out, "out", b, _size(V), types)
    pt, st = _matrix(tokens, "tokens", b, None, _I32)
    pm, sm = _matrix(mask, "mask", b, (_size(V) + 31) // 32, (torch.int32, torch.uint32))
    f32 = (torch.float32,)
    pp, ptl, pr, pps, pf, pbl = _flat((prompt_lens, "prompt_lens", b, _I32), (total_lens, "total_lens", b, _I32),
                                      (repetition, "repetition", b, f32), (presence, "presence", b, f32),
                                      (frequency, "frequency", b, f32), (bias_lens, "bias_lens", b, _I32))
    pbt, sbt = _matrix(bias_tokens, "bias_tokens", b, None, _I32)
    pbv, sbv = _matrix(bias_values, "bias_values", b, None, f32)
    if bias_tokens is not None:
        if bias_values is None or bias_values.shape[1] != bias_tokens.shape[1] or sbv != sbt:
            raise ValueError("bias_values: the shape and row stride of bias_tokens are required")
        if sbt != bias_tokens.shape[1]:
            raise ValueError("bias_tokens: contiguous tensor required")
    if tokens is not None and st != tokens.shape[1]:
        raise ValueError("tokens: contiguous tensor required")
    ts = (logits, out, tokens, prompt_lens, total_lens, repetition, presence, frequency, bias_tokens, bias_values, bias_lens, mask)
    _serve("lowbit_logits_process", stream, ts, lambda s: lib.lowbit_logits_process(
        dtype, pin, sin, B, V, pt, st, pp, ptl, pr, pps, pf, pbt, pbv, sbt, pbl, pm, sm, po, so, s))


class Batch:
    """A work list of decode products prepared once (lowbit_batch_create) and launched by run().  The batch
    holds the tensors its descriptors point to until close(), so none of them can be freed (and its memory
    handed to another tensor) while the batch can still write into it."""

    def __init__(self, descs):
        arr = (lb_matvec_desc * len(descs))(*descs)
        handle = ctypes.c_void_p()
        _check(lib.lowbit_batch_create(ctypes.cast(arr, ctypes.c_void_p), len(descs), ctypes.byref(handle)),
               "lowbit_batch_create")
        self._h = handle
        self._keep = [getattr(d, "_tensors", ()) for d in descs]

    def run(self, stream=None):
        if not self._h:
            raise ValueError("batch is closed")
        s = _stream(stream) if stream is not None else torch.cuda.current_stream().cuda_stream
        _check(lib.lowbit_matvec_batched(self._h, s), "lowbit_matvec_batched")

    def launches(self):
        """Kernel launches one run() makes (lowbit_batch_launches)."""
        if not self._h:
            raise ValueError("batch is closed")
        return int(lib.lowbit_batch_launches(self._h))

    def close(self):
        if self._h:
            lib.lowbit_batch_destroy(self._h)
            self._h = None
        self._keep = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def desc(fmt, W, N, K, xq, xscale, y, w_tensor_scale=1.0, afmt=None, x=None) -> lb_matvec_desc:
    """One work-list entry, its buffers checked against the sizes like lowbit_matvec's.  With x (fp32
    activations) and afmt ACT_F32_Q8_0 the product quantises x to q8_0 in its own launch; xq and xscale
    are then ignored (pass None).  The entry keeps references to its tensors (a Batch built from it holds
    them)."""
    if afmt is None:
        afmt = ACT_F32_Q8_0 if x is not None else ACT_I8_ROW if fmt in (TERNARY_PLANAR, TERNARY_B3) else ACT_Q8_0
    n, k = _pos(N, K)
    if afmt == ACT_F32_Q8_0:
        pw, py, px = _args((W, "W", _wbytes(fmt, n, k)), (y, "y", n, (torch.float32,)), (x, "x", k, (torch.float32,)))
        pq, ps = _ptr(xq), _ptr(xscale)
    else:
        pw, py, pq, ps = _args((W, "W", _wbytes(fmt, n, k)), (y, "y", n, (torch.float32,)),
                               (xq, "xq", k, (torch.int8,)), _scale_spec(xscale, "xscale", afmt, 1, k))
        px = _ptr(x)
    d = lb_matvec_desc(fmt, afmt, N, K, pw, float(w_tensor_scale), pq, ps, py, px)
    d._tensors = tuple(t for t in (W, xq, xscale, y, x) if isinstance(t, torch.Tensor))
    return d
