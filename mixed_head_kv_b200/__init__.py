"""Python binding of libduo (include/duo.h): mixed-head (DuoAttention) attention on B200.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libduo.so. PyTorch supplies device memory and streams. The module
refuses to load when libduo.so has not been built (run
`python mixed_head_kv_b200/build.py` or `__graft_entry__.build()`); there is
no fallback path.

Functions keep the C names: duo_cache_alloc, duo_cache_free, duo_cache_append,
duo_prefill, duo_decode, duo_cache_len, duo_cache_set_len, duo_cache_views,
duo_cache_error, duo_status_str, the duo_paged_* calls. `DuoCache` bundles a
cache handle with the torch buffer that backs it; `PagedCache` a paged cache
with the torch tensors that are its pages, windows, page table and lengths.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libduo.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libduo.so is not built at {LIB_PATH}; run `python mixed_head_kv_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

DUO_OK = 0
DUO_ERR_INVALID_ARG = 1
DUO_ERR_CAPACITY = 2
DUO_ERR_ALIGNMENT = 3
DUO_ERR_CUDA = 4
DUO_ERR_STATE = 5
DUO_ERR_DEVICE = 6
DUO_ERR_SCRATCH_LIMIT = 7
DUO_ERR_HOST_MEMORY = 8
DUO_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024
DUO_MAX_Q_HEADS = 256
DUO_MAX_KV_HEADS = 128

DUO_MAX_RAGGED_BATCH = 64  # sequences of different lengths per batch (include/duo.h)
DUO_KV_BF16 = 0  # cache formats of the retrieval heads (include/duo.h)
DUO_KV_E4M3 = 1

EXPORTED = ("duo_cache_alloc", "duo_cache_free", "duo_cache_append", "duo_prefill", "duo_decode",
            "duo_cache_len", "duo_cache_set_len", "duo_cache_views", "duo_cache_error", "duo_status_str",
            "duo_decode_static_scratch", "duo_cache_append_ragged", "duo_cache_seq_lens",
            "duo_cache_set_seq_lens", "duo_prefill_ragged", "duo_cache_set_kv_scales",
            "duo_cache_test_wait_timeout",
            "duo_paged_size", "duo_paged_alloc", "duo_paged_free", "duo_paged_set_kv_scales", "duo_paged_extend",
            "duo_paged_append", "duo_paged_prefill", "duo_paged_decode", "duo_paged_fork", "duo_paged_copy",
            "duo_paged_release", "duo_paged_compact", "duo_paged_error", "duo_paged_test_wait_timeout")
DUO_PAGED_MAX_SEQS = 4096  # paged caches (include/duo.h)
DUO_PAGED_MAX_BATCH = 512
DUO_PAGED_MAX_GROUP = 8
DUO_ERR_BIT_PAGED_ARGUMENT = 4  # duo_paged_error bits
DUO_ERR_BIT_PAGED_CAPACITY = 8
DUO_ERR_BIT_PAGED_SHARED = 16
DUO_ERR_BIT_PAGED_WAIT = 32
DUO_TEST_WAIT_DECODE = 1  # duo_cache_test_wait_timeout kinds and duo_cache_error bits (include/duo.h)
DUO_TEST_WAIT_PREFILL = 2
DUO_ERR_BIT_PREFILL_WAIT = 1
DUO_ERR_BIT_DECODE_COPY = 2


class duo_layout(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("kv_format", ctypes.c_int32), ("max_len", ctypes.c_int64),
                ("softmax_scale", ctypes.c_float), ("reserved1", ctypes.c_int32)]


class duo_paged_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_layers", "max_seqs", "num_q_heads", "num_kv_heads", "head_dim", "sink",
                                              "recent", "kv_format", "page_size", "num_pages", "max_pages")]
    _fields_.append(("softmax_scale", ctypes.c_float))


class duo_paged_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("pages", "windows", "page_table", "seq_len", "page_ref", "workspace")]


class duo_paged_buffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_window", "v_window", "page_table", "seq_len",
                                               "page_ref", "workspace")]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_ST = ctypes.c_int

_lib.duo_status_str.restype = ctypes.c_char_p
_lib.duo_status_str.argtypes = [_ST]
_lib.duo_cache_alloc.restype = _ST
_lib.duo_cache_alloc.argtypes = [ctypes.POINTER(duo_layout), _P, _P, ctypes.c_size_t,
                                 ctypes.POINTER(ctypes.c_size_t), _P, ctypes.POINTER(_P)]
_lib.duo_cache_free.restype = _ST
_lib.duo_cache_free.argtypes = [_P]
_lib.duo_cache_append.restype = _ST
_lib.duo_cache_append.argtypes = [_P, _I32, _P, _P, _I64, _P]
_lib.duo_prefill.restype = _ST
_lib.duo_prefill.argtypes = [_P, _I32, _P, _P, _P, _P, _I64, _P]
_lib.duo_decode.restype = _ST
_lib.duo_decode.argtypes = [_P, _I32, _P, _P, _P, _P, _P]
_lib.duo_decode_static_scratch.restype = _ST
_lib.duo_decode_static_scratch.argtypes = [_P, _I32, _P, _P, _P, _P, _P]
_lib.duo_cache_len.restype = _ST
_lib.duo_cache_len.argtypes = [_P, _I32, ctypes.POINTER(_I64)]
_lib.duo_cache_set_len.restype = _ST
_lib.duo_cache_set_len.argtypes = [_P, _I32, _I64]
_lib.duo_cache_views.restype = _ST
_lib.duo_cache_views.argtypes = [_P, _I32, _I32, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_I64),
                                 ctypes.POINTER(_I32)]
_lib.duo_cache_append_ragged.restype = _ST
_lib.duo_cache_append_ragged.argtypes = [_P, _I32, _P, _P, ctypes.POINTER(_I64), _I64, _P]
_lib.duo_cache_set_kv_scales.restype = _ST
_lib.duo_cache_set_kv_scales.argtypes = [_P, _I32, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float), _P]
_lib.duo_prefill_ragged.restype = _ST
_lib.duo_prefill_ragged.argtypes = [_P, _I32, _P, _P, _P, _P, ctypes.POINTER(_I64), _I64, _P]
_lib.duo_cache_seq_lens.restype = _ST
_lib.duo_cache_seq_lens.argtypes = [_P, _I32, ctypes.POINTER(_I64)]
_lib.duo_cache_set_seq_lens.restype = _ST
_lib.duo_cache_set_seq_lens.argtypes = [_P, _I32, ctypes.POINTER(_I64)]
_lib.duo_cache_test_wait_timeout.restype = _ST
_lib.duo_cache_test_wait_timeout.argtypes = [_P, _I32, ctypes.c_uint64]
_lib.duo_cache_error.restype = _ST
_lib.duo_cache_error.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]

_lib.duo_paged_size.restype = _ST
_lib.duo_paged_size.argtypes = [ctypes.POINTER(duo_paged_layout), _P, ctypes.POINTER(duo_paged_sizes)]
_lib.duo_paged_alloc.restype = _ST
_lib.duo_paged_alloc.argtypes = [ctypes.POINTER(duo_paged_layout), _P, ctypes.POINTER(duo_paged_buffers), _P,
                                 ctypes.POINTER(_P)]
_lib.duo_paged_free.restype = _ST
_lib.duo_paged_free.argtypes = [_P]
_lib.duo_paged_set_kv_scales.restype = _ST
_lib.duo_paged_set_kv_scales.argtypes = [_P, _I32, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float), _P]
_lib.duo_paged_extend.restype = _ST
_lib.duo_paged_extend.argtypes = [_P, _I32, _P, _P, _P]
_lib.duo_paged_append.restype = _ST
_lib.duo_paged_append.argtypes = [_P, _I32, _I32, _P, _P, _P, _P, _I64, _I64, _P]
_lib.duo_paged_prefill.restype = _ST
_lib.duo_paged_prefill.argtypes = [_P, _I32, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]
_lib.duo_paged_decode.restype = _ST
_lib.duo_paged_decode.argtypes = [_P, _I32, _I32, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]
_lib.duo_paged_fork.restype = _ST
_lib.duo_paged_fork.argtypes = [_P, _I32, _P, _P, _P]
_lib.duo_paged_copy.restype = _ST
_lib.duo_paged_copy.argtypes = [_P, _I32, _P, _P, _P]
_lib.duo_paged_release.restype = _ST
_lib.duo_paged_release.argtypes = [_P, _I32, _P, _P]
_lib.duo_paged_compact.restype = _ST
_lib.duo_paged_compact.argtypes = [_P, _P]
_lib.duo_paged_test_wait_timeout.restype = _ST
_lib.duo_paged_test_wait_timeout.argtypes = [_P, _I32]
_lib.duo_paged_error.restype = _ST
_lib.duo_paged_error.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]


class DuoError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {duo_status_str(status)} (status {status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != DUO_OK:
        raise DuoError(status, where)


def _ptr(x) -> Optional[int]:
    """Device pointer of a tensor, or an int/None passed through."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # the current stream's handle without building a Stream object
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def duo_status_str(status: int) -> str:
    return _lib.duo_status_str(status).decode()


def make_layout(num_layers, batch, num_q_heads, num_kv_heads, head_dim, sink, recent, max_len,
                softmax_scale=0.0, kv_format=0) -> duo_layout:
    return duo_layout(num_layers, batch, num_q_heads, num_kv_heads, head_dim, sink, recent, kv_format, max_len,
                      softmax_scale, 0)


def _mask_buf(is_retrieval: Sequence[int]):
    vals = [int(x) for x in is_retrieval]
    return (ctypes.c_uint8 * max(1, len(vals)))(*vals)


def duo_cache_alloc(layout: duo_layout, is_retrieval: Sequence[int], dev_buf=None, buf_bytes: int = 0,
                    stream=None):
    """Returns (status, required_bytes, handle). With dev_buf None only sizes the cache."""
    req = ctypes.c_size_t(0)
    handle = _P()
    mask = _mask_buf(is_retrieval)
    s = _stream(stream) if dev_buf is not None else None
    st = _lib.duo_cache_alloc(ctypes.byref(layout), ctypes.cast(mask, _P), _ptr(dev_buf), buf_bytes,
                              ctypes.byref(req), s, ctypes.byref(handle))
    return st, req.value, handle.value


def duo_cache_free(handle) -> int:
    return _lib.duo_cache_free(handle)


def duo_cache_append(handle, layer, k, v, n_tok, stream=None) -> int:
    return _lib.duo_cache_append(handle, layer, _ptr(k), _ptr(v), n_tok, _stream(stream))


def duo_prefill(handle, layer, q, k, v, out, n_tok, stream=None) -> int:
    return _lib.duo_prefill(handle, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), n_tok, _stream(stream))


def duo_decode(handle, layer, q, k_new, v_new, out, stream=None) -> int:
    return _lib.duo_decode(handle, layer, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _stream(stream))


def duo_decode_static_scratch(handle, layer, q, k_new, v_new, out, stream=None) -> int:
    """duo_decode with its split-KV scratch in the library's static device array
    (for callers that cannot allocate device memory at call time)."""
    return _lib.duo_decode_static_scratch(handle, layer, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                          _stream(stream))


def duo_cache_len(handle, layer):
    n = _I64(0)
    st = _lib.duo_cache_len(handle, layer, ctypes.byref(n))
    return st, n.value


def duo_cache_set_len(handle, layer, length) -> int:
    return _lib.duo_cache_set_len(handle, layer, length)


def duo_cache_append_ragged(handle, layer, k, v, n_tok: Sequence[int], max_tok: int, stream=None) -> int:
    """Sequence b appends rows [0, n_tok[b]) of k/v [batch][max_tok][Hkv][D]."""
    n = (_I64 * max(1, len(n_tok)))(*[int(x) for x in n_tok])
    return _lib.duo_cache_append_ragged(handle, layer, _ptr(k), _ptr(v), n, max_tok,
                                        _stream(stream) if k is not None else None)


def duo_prefill_ragged(handle, layer, q, k, v, out, n_tok: Sequence[int], max_tok: int, stream=None) -> int:
    """Sequence b's chunk is rows [0, n_tok[b]) of q/k/v [batch][max_tok][H][D]."""
    n = (_I64 * max(1, len(n_tok)))(*[int(x) for x in n_tok])
    return _lib.duo_prefill_ragged(handle, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), n, max_tok,
                                   _stream(stream) if q is not None else None)


def duo_cache_set_kv_scales(handle, layer, k_scale: Sequence[float], v_scale: Sequence[float], stream=None) -> int:
    """Per-KV-head scales of an E4M3 cache (host lists [num_kv_heads])."""
    k = (ctypes.c_float * max(1, len(k_scale)))(*[float(x) for x in k_scale])
    v = (ctypes.c_float * max(1, len(v_scale)))(*[float(x) for x in v_scale])
    return _lib.duo_cache_set_kv_scales(handle, layer, k, v, _stream(stream))


def duo_cache_seq_lens(handle, layer, batch: int):
    lens = (_I64 * batch)()
    st = _lib.duo_cache_seq_lens(handle, layer, lens)
    return st, list(lens)


def duo_cache_set_seq_lens(handle, layer, lens: Sequence[int]) -> int:
    arr = (_I64 * max(1, len(lens)))(*[int(x) for x in lens])
    return _lib.duo_cache_set_seq_lens(handle, layer, arr)


def duo_cache_views(handle, layer, kv_head):
    k, v, slots, r = _P(), _P(), _I64(0), _I32(0)
    st = _lib.duo_cache_views(handle, layer, kv_head, ctypes.byref(k), ctypes.byref(v), ctypes.byref(slots),
                              ctypes.byref(r))
    return st, k.value, v.value, slots.value, r.value


def duo_cache_test_wait_timeout(handle, launches: int, timeout_ns: int) -> int:
    """Arm the next launch of the given kinds to test the bounded waits (include/duo.h)."""
    return _lib.duo_cache_test_wait_timeout(handle, launches, timeout_ns)


def duo_cache_error(handle, stream=None):
    f = ctypes.c_uint32(0)
    st = _lib.duo_cache_error(handle, _stream(stream), ctypes.byref(f))
    return st, f.value


def make_paged_layout(num_layers, max_seqs, num_q_heads, num_kv_heads, head_dim, sink, recent, page_size, num_pages,
                      max_pages, softmax_scale=0.0, kv_format=0) -> duo_paged_layout:
    return duo_paged_layout(num_layers, max_seqs, num_q_heads, num_kv_heads, head_dim, sink, recent, kv_format, page_size,
                            num_pages, max_pages, softmax_scale)


def duo_paged_size(layout: duo_paged_layout, is_retrieval: Sequence[int]):
    """(status, duo_paged_sizes): bytes of each device buffer."""
    sizes = duo_paged_sizes()
    if len(is_retrieval) < layout.num_layers * layout.num_kv_heads:  # the library reads that many
        return DUO_ERR_INVALID_ARG, sizes
    st = _lib.duo_paged_size(ctypes.byref(layout), ctypes.cast(_mask_buf(is_retrieval), _P), ctypes.byref(sizes))
    return st, sizes


def duo_paged_alloc(layout: duo_paged_layout, is_retrieval: Sequence[int], buffers: duo_paged_buffers, stream=None):
    """(status, handle)."""
    handle = _P()
    if len(is_retrieval) < layout.num_layers * layout.num_kv_heads:
        return DUO_ERR_INVALID_ARG, None
    st = _lib.duo_paged_alloc(ctypes.byref(layout), ctypes.cast(_mask_buf(is_retrieval), _P), ctypes.byref(buffers),
                              _stream(stream), ctypes.byref(handle))
    return st, handle.value


def duo_paged_free(handle) -> int:
    return _lib.duo_paged_free(handle)


def duo_paged_set_kv_scales(handle, layer, k_scale: Sequence[float], v_scale: Sequence[float], stream=None) -> int:
    k = (ctypes.c_float * max(1, len(k_scale)))(*[float(x) for x in k_scale])
    v = (ctypes.c_float * max(1, len(v_scale)))(*[float(x) for x in v_scale])
    return _lib.duo_paged_set_kv_scales(handle, layer, k, v, _stream(stream))


def duo_paged_extend(handle, n, seqs, n_tok=None, stream=None) -> int:
    return _lib.duo_paged_extend(handle, n, _ptr(seqs), _ptr(n_tok), _stream(stream))


def duo_paged_append(handle, layer, n, seqs, row_start, k, v, n_rows, kv_stride=0, stream=None) -> int:
    return _lib.duo_paged_append(handle, layer, n, _ptr(seqs), _ptr(row_start), _ptr(k), _ptr(v), n_rows, kv_stride,
                                 _stream(stream))


def duo_paged_prefill(handle, layer, n, row_start, q, k, v, out, n_rows, q_stride=0, kv_stride=0, out_stride=0,
                      stream=None) -> int:
    return _lib.duo_paged_prefill(handle, layer, n, _ptr(row_start), _ptr(q), _ptr(k), _ptr(v), _ptr(out), n_rows,
                                  q_stride, kv_stride, out_stride, _stream(stream))


def duo_paged_decode(handle, layer, n, seqs, q, k_new, v_new, out, q_stride=0, kv_stride=0, out_stride=0,
                     stream=None) -> int:
    return _lib.duo_paged_decode(handle, layer, n, _ptr(seqs), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), q_stride,
                                 kv_stride, out_stride, _stream(stream))


def duo_paged_fork(handle, n, src, dst, stream=None) -> int:
    return _lib.duo_paged_fork(handle, n, _ptr(src), _ptr(dst), _stream(stream))


def duo_paged_copy(handle, n, src, dst, stream=None) -> int:
    return _lib.duo_paged_copy(handle, n, _ptr(src), _ptr(dst), _stream(stream))


def duo_paged_release(handle, n, seqs, stream=None) -> int:
    return _lib.duo_paged_release(handle, n, _ptr(seqs), _stream(stream))


def duo_paged_compact(handle, stream=None) -> int:
    return _lib.duo_paged_compact(handle, _stream(stream))


def duo_paged_test_wait_timeout(handle, launches: int) -> int:
    """Arm the next launch of the given kinds to test the bounded waits (include/duo.h)."""
    return _lib.duo_paged_test_wait_timeout(handle, launches)


def duo_paged_error(handle, stream=None):
    f = ctypes.c_uint32(0)
    st = _lib.duo_paged_error(handle, _stream(stream), ctypes.byref(f))
    return st, f.value


class DuoCache:
    """A cache handle plus the torch uint8 buffer that backs it (owned here)."""

    def __init__(self, num_layers, batch, num_q_heads, num_kv_heads, head_dim, sink, recent, max_len,
                 is_retrieval: Sequence[int], softmax_scale=0.0, device="cuda", stream=None, kv_format=0):
        import torch
        self.layout = make_layout(num_layers, batch, num_q_heads, num_kv_heads, head_dim, sink, recent, max_len,
                                  softmax_scale, kv_format)
        self.is_retrieval = [int(x) for x in is_retrieval]
        st, req, _ = duo_cache_alloc(self.layout, self.is_retrieval)
        _check(st, "duo_cache_alloc(size)")
        self.nbytes = req
        self.buffer = torch.empty(req + 256, dtype=torch.uint8, device=device)
        off = (-self.buffer.data_ptr()) % 256
        self._base = self.buffer.data_ptr() + off
        st, _, handle = duo_cache_alloc(self.layout, self.is_retrieval, self._base, req, stream)
        _check(st, "duo_cache_alloc")
        self.handle = handle

    def close(self):
        if getattr(self, "handle", None):
            duo_cache_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: module globals may already be gone
            pass

    def append(self, layer, k, v, stream=None):
        _check(duo_cache_append(self.handle, layer, k, v, k.shape[1], stream), "duo_cache_append")

    def append_ragged(self, layer, k, v, n_tok, stream=None):
        """Per-sequence token counts n_tok[b] <= k.shape[1] (rows past them are not read)."""
        _check(duo_cache_append_ragged(self.handle, layer, k, v, n_tok, k.shape[1], stream),
               "duo_cache_append_ragged")

    def prefill_ragged(self, layer, q, k, v, out, n_tok, stream=None):
        _check(duo_prefill_ragged(self.handle, layer, q, k, v, out, n_tok, q.shape[1], stream), "duo_prefill_ragged")

    def seq_lens(self, layer):
        st, lens = duo_cache_seq_lens(self.handle, layer, self.layout.batch)
        _check(st, "duo_cache_seq_lens")
        return lens

    def set_seq_lens(self, layer, lens):
        _check(duo_cache_set_seq_lens(self.handle, layer, lens), "duo_cache_set_seq_lens")

    def prefill(self, layer, q, k, v, out, stream=None):
        _check(duo_prefill(self.handle, layer, q, k, v, out, q.shape[1], stream), "duo_prefill")

    def decode(self, layer, q, k_new, v_new, out, stream=None):
        _check(duo_decode(self.handle, layer, q, k_new, v_new, out, stream), "duo_decode")

    def length(self, layer) -> int:
        st, n = duo_cache_len(self.handle, layer)
        _check(st, "duo_cache_len")
        return n

    def set_length(self, layer, n):
        _check(duo_cache_set_len(self.handle, layer, n), "duo_cache_set_len")

    def error_flags(self, stream=None) -> int:
        st, f = duo_cache_error(self.handle, stream)
        _check(st, "duo_cache_error")
        return f

    def head_view(self, layer, kv_head):
        """(k, v, is_retrieval): torch views [batch, slots, head_dim] of one KV head's cache
        (bf16, or uint8 E4M3 codes for the retrieval heads of an E4M3 cache)."""
        import torch
        st, kp, vp, slots, r = duo_cache_views(self.handle, layer, kv_head)
        _check(st, "duo_cache_views")
        B, D = self.layout.batch, self.layout.head_dim
        codes = bool(r) and self.layout.kv_format == DUO_KV_E4M3
        n = B * slots * D * (1 if codes else 2)  # bytes

        def view(ptr):
            start = ptr - self.buffer.data_ptr()
            raw = self.buffer[start:start + n]
            return (raw if codes else raw.view(torch.bfloat16)).view(B, slots, D)
        return view(kp), view(vp), r

    def set_kv_scales(self, layer, k_scale, v_scale, stream=None):
        _check(duo_cache_set_kv_scales(self.handle, layer, k_scale, v_scale, stream), "duo_cache_set_kv_scales")


class PagedCache:
    """A paged mixed-head cache (include/duo.h, duo_paged_*) and the tensors that hold it.

    Tensors (attributes; pass `tensors`, a dict with these names, to use your own):
      k_pages, v_pages    [num_pages, R, page_size, head_dim] bfloat16 or float8_e4m3fn, R = retrieval heads of all layers
      k_window, v_window  [max_seqs, S, sink + recent, head_dim] bfloat16, S = streaming heads of all layers
      page_table          int32 [max_seqs, max_pages]; seq_len int32 [max_seqs]; page_ref int32 [num_pages]
    Sequences are numbers in [0, max_seqs), empty at first (seq_len 0). Entry lists (seqs, n_tok, row_start, src, dst)
    are int32 tensors on the cache's device. Rows (q, k, v, out) are bfloat16 [rows, heads, head_dim]; the stride
    between rows is free (a slice of a fused projection), a row itself is dense. A step is: extend once, then per layer
    prefill + append (whole prompts) or decode (one token). Calls run on the current stream and must be ordered among
    themselves; nothing waits for the device except error_flags. A captured CUDA graph of a step may be replayed.
    `stream`: where the cache is set up, behind what the current stream holds by then. A cache that was used on other
    streams than that one (or in a graph) is closed, or dropped, when their work has ended.
    """

    _NAMES = ("k_pages", "v_pages", "k_window", "v_window", "page_table", "seq_len", "page_ref")

    def __init__(self, num_layers, max_seqs, num_q_heads, num_kv_heads, head_dim, sink, recent, page_size, num_pages,
                 max_pages, is_retrieval: Sequence[int], softmax_scale=0.0, kv_format=DUO_KV_BF16, device="cuda",
                 tensors=None, stream=None):
        import torch
        self.handle = None
        self.layout = make_paged_layout(num_layers, max_seqs, num_q_heads, num_kv_heads, head_dim, sink, recent, page_size,
                                        num_pages, max_pages, softmax_scale, kv_format)
        mask = [int(x) for x in is_retrieval]
        if len(mask) != num_layers * num_kv_heads:
            raise ValueError(f"is_retrieval has {len(mask)} entries, not num_layers * num_kv_heads")
        self.is_retrieval = mask
        st, sizes = duo_paged_size(self.layout, mask)
        _check(st, "duo_paged_size")
        retr = sum(mask)
        strm = len(mask) - retr
        page = torch.float8_e4m3fn if kv_format == DUO_KV_E4M3 else torch.bfloat16
        shapes = {"k_pages": ((num_pages, retr, page_size, head_dim), page),
                  "k_window": ((max_seqs, strm, sink + recent, head_dim), torch.bfloat16),
                  "page_table": ((max_seqs, max_pages), torch.int32), "seq_len": ((max_seqs,), torch.int32),
                  "page_ref": ((num_pages,), torch.int32)}
        shapes["v_pages"], shapes["v_window"] = shapes["k_pages"], shapes["k_window"]
        if tensors is None:
            tensors = {n: torch.zeros(shapes[n][0], dtype=shapes[n][1], device=device) for n in self._NAMES}
        self.device = tensors["seq_len"].device
        buffers = duo_paged_buffers()
        for n in self._NAMES:
            t = tensors[n]
            shape, dtype = shapes[n]
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{n}: expected a contiguous {dtype} tensor {shape} on {self.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
            setattr(self, n, t)
            setattr(buffers, n, t.data_ptr() or None)
        if self.device.type != "cuda":
            raise ValueError("a paged cache lives on a CUDA device")
        self._workspace = torch.empty(sizes.workspace, dtype=torch.uint8, device=self.device)
        buffers.workspace = self._workspace.data_ptr()
        self._constants()
        with torch.cuda.device(self.device):
            here, raw = torch.cuda.current_stream(), _stream(stream)
            if raw != here.cuda_stream:  # the tensors are allocated and filled on the current stream
                other = torch.cuda.ExternalStream(raw) if isinstance(stream, int) else stream
                other.wait_stream(here)
                if not isinstance(stream, int):
                    for t in (self._workspace, *(tensors[n] for n in self._NAMES)):
                        t.record_stream(other)
            st, handle = duo_paged_alloc(self.layout, mask, buffers, raw)
        _check(st, "duo_paged_alloc")
        self.handle = handle

    def _constants(self):
        """What the argument checks compare with on every call."""
        import torch
        self._int32, self._bf16 = torch.int32, torch.bfloat16
        self._index = -1 if self.device.type == "cpu" else self.device.index
        self._raw_stream = None if self.device.type == "cpu" else getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._dim, self._q_heads, self._kv_heads = (self.layout.head_dim, self.layout.num_q_heads,
                                                    self.layout.num_kv_heads)

    def _on(self, stream):
        """The stream's handle; by default the current one of the cache's device."""
        if stream is None and self._raw_stream is not None:
            return self._raw_stream(self._index)
        return _stream(stream)

    def close(self):
        if getattr(self, "handle", None):
            duo_paged_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: module globals may already be gone
            pass

    def _entries(self, name, t, n=None):
        if t.dtype is not self._int32 or t.dim() != 1 or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name}: expected a contiguous 1-d int32 tensor on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name}: expected {n} entries, got {t.shape[0]}")
        return t.data_ptr()

    def _rows(self, name, t, heads, n=None):
        """(address, row stride) of packed rows [n, heads, head_dim]."""
        d = self._dim
        rows, h, w = t.shape if t.dim() == 3 else (0, -1, -1)
        if h != heads or w != d or t.dtype is not self._bf16 or t.get_device() != self._index:
            raise ValueError(f"{name}: expected bfloat16 rows [*, {heads}, {d}] on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        if n is not None and rows != n:
            raise ValueError(f"{name}: expected {n} rows, got {rows}")
        if t.is_contiguous():
            return t.data_ptr(), 0
        s = t.stride()
        if rows and (s[2] != 1 or (heads > 1 and s[1] != d) or (rows > 1 and s[0] < heads * d)):
            raise ValueError(f"{name}: rows must be dense and must not overlap, got strides {s}")
        return t.data_ptr(), (s[0] if rows > 1 else 0)

    def _kv(self, k, v, n):
        heads = self._kv_heads
        kp, ks = self._rows("k", k, heads, n)
        vp, vs = self._rows("v", v, heads, n)
        if ks != vs:
            raise ValueError(f"k and v must have the same row stride, got {ks} and {vs}")
        return kp, vp, ks

    def set_kv_scales(self, layer, k_scale, v_scale, stream=None):
        heads = self.layout.num_kv_heads
        if len(k_scale) != heads or len(v_scale) != heads:
            raise ValueError(f"expected {heads} scales for k and for v")
        _check(duo_paged_set_kv_scales(self.handle, layer, k_scale, v_scale, self._on(stream)), "duo_paged_set_kv_scales")

    def extend(self, seqs, n_tok=None, stream=None):
        """Sequence seqs[i] gets n_tok[i] (default 1) more tokens."""
        a = self._entries("seqs", seqs)
        n = seqs.shape[0]
        b = None if n_tok is None else self._entries("n_tok", n_tok, n)
        _check(_lib.duo_paged_extend(self.handle, n, a, b, self._on(stream)), "duo_paged_extend")

    def append(self, layer, seqs, row_start, k, v, stream=None):
        """Rows [row_start[i], row_start[i + 1]) of k and v are the newest tokens of seqs[i]."""
        a = self._entries("seqs", seqs)
        n = seqs.shape[0]
        b = self._entries("row_start", row_start, n + 1)
        rows = k.shape[0]
        kp, vp, ks = self._kv(k, v, rows)
        _check(_lib.duo_paged_append(self.handle, layer, n, a, b, kp, vp, rows, ks, self._on(stream)), "duo_paged_append")

    def prefill(self, layer, row_start, q, k, v, out, stream=None):
        """Whole prompts: rows [row_start[i], row_start[i + 1]) of q, k, v and out."""
        b = self._entries("row_start", row_start)
        n = row_start.shape[0] - 1
        if n < 0:
            raise ValueError("row_start: expected one entry more than there are prompts")
        rows, heads = q.shape[0], self._q_heads
        qp, qs = self._rows("q", q, heads)
        kp, vp, ks = self._kv(k, v, rows)
        op, os_ = self._rows("out", out, heads, rows)
        _check(_lib.duo_paged_prefill(self.handle, layer, n, b, qp, kp, vp, op, rows, qs, ks, os_, self._on(stream)),
               "duo_paged_prefill")

    def decode(self, layer, seqs, q, k_new, v_new, out, stream=None):
        """Row i of k_new and v_new is the newest token of seqs[i]; out[i] = attention of q[i]."""
        a = self._entries("seqs", seqs)
        n, heads = seqs.shape[0], self._q_heads
        qp, qs = self._rows("q", q, heads, n)
        kp, vp, ks = self._kv(k_new, v_new, n)
        op, os_ = self._rows("out", out, heads, n)
        _check(_lib.duo_paged_decode(self.handle, layer, n, a, qp, kp, vp, op, qs, ks, os_, self._on(stream)),
               "duo_paged_decode")

    def _pairs(self, src, dst):
        a = self._entries("src", src)
        return src.shape[0], a, self._entries("dst", dst, src.shape[0])

    def fork(self, src, dst, stream=None):
        """Empty sequence dst[i] shares the pages of src[i]."""
        n, a, b = self._pairs(src, dst)
        _check(_lib.duo_paged_fork(self.handle, n, a, b, self._on(stream)), "duo_paged_fork")

    def copy(self, src, dst, stream=None):
        """Empty sequence dst[i] becomes a copy of src[i] in pages of its own."""
        n, a, b = self._pairs(src, dst)
        _check(_lib.duo_paged_copy(self.handle, n, a, b, self._on(stream)), "duo_paged_copy")

    def release(self, seqs, stream=None):
        a = self._entries("seqs", seqs)
        _check(_lib.duo_paged_release(self.handle, seqs.shape[0], a, self._on(stream)), "duo_paged_release")

    def compact(self, stream=None):
        _check(_lib.duo_paged_compact(self.handle, self._on(stream)), "duo_paged_compact")

    def error_flags(self, stream=None) -> int:
        st, f = duo_paged_error(self.handle, self._on(stream))
        _check(st, "duo_paged_error")
        return f
