"""Python binding of libqgemv (the MI355X compressed-weight product).

Thin marshalling over the C ABI in include/qgemv.h and include/qcache.h: every function here has
the name of the C entry point it calls, takes torch tensors that already
live on the GPU, allocates outputs with torch when none are given, passes
raw device pointers and torch's current HIP stream, and raises QError on a
non-zero status.  All arithmetic runs in the HIP kernels; there is no CPU
fallback, and any call fails loudly when the shared library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

__all__ = [
    "QError", "load", "lib_path", "q_abi_version", "q_format_version", "q_status_str",
    "qgroup_sizes", "qpack_group", "qunpack_group", "qgemv_group",
    "qgroup_outlier_ws", "qpack_group_outlier", "qgemv_group_outlier", "qgemv_group_multi",
    "qcodebook_default", "qpack_group_cb", "qgemv_group_cb",
    "qtq_centroids", "qtq_rotation", "qtq_quant_keys", "qtq_project", "qtq_logits", "qtq_quant_values", "qtq_attend",
    "qbinlr_sizes", "qpack_binlr", "qunpack_binlr", "qgemv_binlr", "qgemv_binlr_noalloc",
    "qstream_read", "qgemm_prefill_ws", "qgemm_prefill", "Q_F32", "Q_BF16", "Q_FMT_GROUP", "Q_FMT_BINLR",
    "qcache_sizes", "make_qcache", "qcache_write", "qcache_read", "qcache_attend_ws", "qcache_attend",
    "qcache_attend_shared",
]

Q_OK, Q_EINVAL, Q_EALIGN, Q_EUNSUPPORTED, Q_ERANGE, Q_EWORKSPACE, Q_EHIP = 0, -1, -2, -3, -4, -5, -6
Q_F32, Q_BF16, Q_F16 = 0, 1, 2
Q_FMT_GROUP, Q_FMT_BINLR = 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB: Optional[ctypes.CDLL] = None


def lib_path() -> str:
    return os.path.join(_HERE, "libqgemv.so")


class QError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({q_status_str(status)})")


class qweight(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("bits", ctypes.c_int), ("group", ctypes.c_int),
        ("codes", ctypes.c_void_p), ("meta", ctypes.c_void_p),
        ("r", ctypes.c_int64), ("ubits", ctypes.c_void_p), ("vtbits", ctypes.c_void_p),
        ("s1", ctypes.c_void_p), ("s2", ctypes.c_void_p),
        ("side", ctypes.c_void_p), ("oidx", ctypes.c_void_p), ("n_out", ctypes.c_int64),
        ("book_ids", ctypes.c_void_p), ("books", ctypes.c_void_p), ("n_books", ctypes.c_int),
    ]


class qgroup_mat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("meta", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("y", ctypes.c_void_p)]


class qcache(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("bits", ctypes.c_int),
        ("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p), ("v_meta", ctypes.c_void_p),
    ]


class qseqs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("max_pages", ctypes.c_int64),
        ("pages", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
    ]


def load() -> ctypes.CDLL:
    """Load libqgemv.so from the package directory (raises if it is missing)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libqgemv.so not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    I64, I32, P, SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "q_abi_version": (I32, []),
        "q_format_version": (I32, []),
        "q_status_str": (ctypes.c_char_p, [I32]),
        "qgroup_sizes": (I32, [I64, I64, I32, I32, SZ, SZ]),
        "qpack_group": (I32, [P, I64, I64, I32, I32, P, P, P]),
        "qunpack_group": (I32, [P, P, I64, I64, I32, I32, P, P, P]),
        "qgemv_group": (I32, [P, P, I64, I64, I32, I32, P, I32, I64, P, I32, P]),
        "qgroup_outlier_ws": (I32, [I64, I64, SZ]),
        "qgemv_group_multi": (I32, [ctypes.POINTER(qgroup_mat), I32, I64, I32, I32, P, I32, I64, I32, P]),
        "qpack_group_outlier": (I32, [P, I64, I64, I32, I32, I64, P, P, P, P, P, ctypes.c_size_t, P]),
        "qgemv_group_outlier": (I32, [P, P, P, P, I64, I64, I64, I32, I32, P, I32, I64, P, I32, P]),
        "qcodebook_default": (I32, [I32, P, ctypes.POINTER(ctypes.c_int)]),
        "qpack_group_cb": (I32, [P, I64, I64, I32, I32, P, I32, P, P, P, P]),
        "qgemv_group_cb": (I32, [P, P, P, P, I32, I64, I64, I32, I32, P, I32, I64, P, I32, P]),
        "qtq_centroids": (I32, [I32, I32, ctypes.POINTER(ctypes.c_float), P]),
        "qtq_rotation": (I32, [I32, P, P]),
        "qtq_sizes": (I32, [I64, I32, SZ, SZ, SZ]),
        "qtq_quant_keys": (I32, [P, I64, I32, P, P, ctypes.c_float, P, P, P, P, P]),
        "qtq_logits_ws": (I32, [I64, I64, SZ]),
        "qtq_project": (I32, [P, P, P, P]),
        "qtq_logits": (I32, [P, P, P, I64, I64, I32, ctypes.c_float, P, P, P, P, I64, P, P, ctypes.c_size_t, P]),
        "qtq_quant_values": (I32, [P, I64, I32, P, ctypes.c_float, P, P, P, P]),
        "qtq_attend_ws": (I32, [I64, I64, I64, SZ]),
        "qtq_attend": (I32, [P, P, I64, I64, I32, ctypes.c_float, P, P, P, I64, P, P, ctypes.c_size_t, P]),
        "qbinlr_sizes": (I32, [I64, I64, I64, I64, SZ, SZ, SZ]),
        "qpack_binlr": (I32, [P, P, I64, I64, I64, P, P, P]),
        "qunpack_binlr": (I32, [P, P, I64, I64, I64, P, P, P]),
        "qgemv_binlr": (I32, [P, P, P, P, I64, I64, I64, P, I32, I64, P, I32, P, ctypes.c_size_t, P]),
        "qgemv_binlr_noalloc": (I32, [P, P, P, P, I64, I64, I64, P, I32, I64, P, I32, P]),
        "qstream_read": (I32, [P, ctypes.c_size_t, P, P]),
        "qgemm_prefill_ws": (I32, [ctypes.POINTER(qweight), I64, SZ]),
        "qgemm_prefill": (I32, [ctypes.POINTER(qweight), P, I32, I64, P, I32, P, ctypes.c_size_t, P]),
    }
    CA, SQ, U64, F32 = ctypes.POINTER(qcache), ctypes.POINTER(qseqs), ctypes.c_size_t, ctypes.c_float
    sig.update({
        "qcache_sizes": (I32, [I64, I32, I32, I32, I32, SZ, SZ]),
        "qcache_write": (I32, [CA, SQ, P, I64, P, I64, I32, P]),
        "qcache_read": (I32, [CA, SQ, P, I64, P, I64, I32, P]),
        "qcache_attend_ws": (I32, [CA, SQ, I32, I64, SZ]),
        "qcache_attend": (I32, [CA, SQ, P, I64, I32, F32, P, I64, I32, P, U64, P]),
        "qcache_attend_shared": (I32, [CA, SQ, P, I64, P, I64, I32, F32, P, I64, I32, P, U64, P]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(status: int, what: str):
    if status != Q_OK:
        raise QError(status, what)


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return Q_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return Q_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA (HIP) tensors")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _need_bytes(t: Optional[torch.Tensor], nbytes: int, what: str):
    """A buffer the kernels read or write nbytes of: it must hold them (the C
    ABI receives bare pointers and cannot check).  Every wrapper checks all
    sizes first and then, with _need_cuda, that every tensor is on the
    device."""
    if t is None:
        raise ValueError(f"{what}: missing")
    if _nbytes(t) < nbytes:
        raise ValueError(f"{what}: {_nbytes(t)} bytes, needs {nbytes}")


def _need_numel(t: Optional[torch.Tensor], numel: int, what: str, dtypes=None, exact=True):
    """An array argument with numel elements (at least numel when not exact:
    a longer table of which the kernels read the first numel entries) and one
    of dtypes."""
    if t is None:
        raise ValueError(f"{what}: missing")
    if t.numel() != numel if exact else t.numel() < numel:
        raise ValueError(f"{what}: {t.numel()} elements, expected {'' if exact else 'at least '}{numel}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {dtypes}")


_ACT = (torch.float32, torch.bfloat16, torch.int16, torch.uint16)   # activations (bf16 as 16-bit bits)
_OUT = (torch.float32, torch.bfloat16)
_Q16 = (torch.bfloat16,)
_H16 = (torch.int16, torch.uint16, torch.float16)                    # fp16 bit patterns


def _batch(x: torch.Tensor, K: int, what: str = "x") -> int:
    """Rows of an activation tensor [B][K] (or [K] for one row)."""
    if x.dtype not in _ACT:
        raise ValueError(f"{what}: dtype {x.dtype} is not fp32 or bf16")
    if x.dim() == 1:
        B = 1
    elif x.dim() == 2:
        B = x.shape[0]
    else:
        raise ValueError(f"{what}: expected [B][K] or [K], got shape {tuple(x.shape)}")
    if x.numel() != B * K:
        raise ValueError(f"{what}: shape {tuple(x.shape)} does not match K = {K}")
    return B


def q_abi_version() -> int:
    return load().q_abi_version()


def q_format_version() -> int:
    return load().q_format_version()


def q_status_str(status: int) -> str:
    return load().q_status_str(status).decode()


# ------------------------------------------------------------------ group RTN
def qgroup_sizes(N: int, K: int, bits: int, group: int):
    c, m = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qgroup_sizes(N, K, bits, group, ctypes.byref(c), ctypes.byref(m)), "qgroup_sizes")
    return c.value, m.value


def qpack_group(W: torch.Tensor, bits: int, group: int, codes=None, meta=None, stream=None):
    """Quantize + pack fp32 W[N][K] -> (codes uint8[N*K*b/8], meta int32[N*K/g])."""
    _need_cuda(W)
    if W.dim() != 2 or W.dtype != torch.float32:
        raise ValueError("W must be fp32 [N][K]")
    N, K = W.shape
    cb, mb = qgroup_sizes(N, K, bits, group)
    if codes is None:
        codes = torch.empty(cb, dtype=torch.uint8, device=W.device)
    if meta is None:
        meta = torch.empty(mb // 4, dtype=torch.int32, device=W.device)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    _need_cuda(codes, meta)
    _check(load().qpack_group(_ptr(W), N, K, bits, group, _ptr(codes), _ptr(meta), _stream(stream)),
           "qpack_group")
    return codes, meta


def qunpack_group(codes, meta, N: int, K: int, bits: int, group: int, want_w: bool = False, stream=None):
    cb, mb = qgroup_sizes(N, K, bits, group)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    q = torch.empty((N, K), dtype=torch.uint8, device=codes.device)
    w = torch.empty((N, K), dtype=torch.float32, device=codes.device) if want_w else None
    _need_cuda(codes, meta)
    _check(load().qunpack_group(_ptr(codes), _ptr(meta), N, K, bits, group, _ptr(q), _ptr(w),
                                _stream(stream)), "qunpack_group")
    return (q, w) if want_w else q


def qgemv_group(codes, meta, N: int, K: int, bits: int, group: int, x: torch.Tensor,
                y: Optional[torch.Tensor] = None, y_dtype=torch.float32, stream=None):
    """y[B][N] = x[B][K] W_hat^T; x is bf16 (or int16/uint16 bf16 bits) or fp32."""
    cb, mb = qgroup_sizes(N, K, bits, group)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    B = _batch(x, K)
    if y is None:
        y = torch.empty((B, N), dtype=y_dtype, device=x.device)
    _need_numel(y, B * N, "y", _OUT)
    _need_cuda(codes, meta, x, y)
    _check(load().qgemv_group(_ptr(codes), _ptr(meta), N, K, bits, group, _ptr(x), _dtype_code(x), B,
                              _ptr(y), _dtype_code(y), _stream(stream)), "qgemv_group")
    return y


def qgemv_group_multi(mats, K: int, bits: int, group: int, x: torch.Tensor, ys=None,
                      y_dtype=torch.float32, stream=None):
    """[y_i] for mats = [(codes_i, meta_i, N_i)] sharing x, K, bits, group, in
    one launch."""
    B = _batch(x, K)
    if ys is None:
        ys = [torch.empty((B, n), dtype=y_dtype, device=x.device) for (_, _, n) in mats]
    if len(ys) != len(mats):
        raise ValueError("one output per matrix")
    for (c, m, n), y in zip(mats, ys):
        cb, mb = qgroup_sizes(n, K, bits, group)
        _need_bytes(c, cb, "codes")
        _need_bytes(m, mb, "meta")
        _need_numel(y, B * n, "y", _OUT)
        if y.dtype != ys[0].dtype:
            raise ValueError("all outputs of a grouped call share one dtype")
    arr = (qgroup_mat * len(mats))(*[qgroup_mat(c.data_ptr(), m.data_ptr(), n, y.data_ptr())
                                     for (c, m, n), y in zip(mats, ys)])
    _need_cuda(x, *[t for (c, m, _), y in zip(mats, ys) for t in (c, m, y)])
    _check(load().qgemv_group_multi(arr, len(mats), K, bits, group, _ptr(x), _dtype_code(x), B,
                                    _dtype_code(ys[0]), _stream(stream)), "qgemv_group_multi")
    return ys


# ------------------------------------------------ group RTN + outlier columns
def qgroup_outlier_ws(K: int, n_out: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qgroup_outlier_ws(K, n_out, ctypes.byref(n)), "qgroup_outlier_ws")
    return n.value


def qpack_group_outlier(W: torch.Tensor, bits: int, group: int, n_out: int, stream=None):
    """(codes, meta, side uint16[N][n_out] fp16 bits, idx int32[n_out]) for fp32 W[N][K]."""
    _need_cuda(W)
    if W.dim() != 2 or W.dtype != torch.float32:
        raise ValueError("W must be fp32 [N][K]")
    N, K = W.shape
    cb, mb = qgroup_sizes(N, K, bits, group)
    codes = torch.empty(cb, dtype=torch.uint8, device=W.device)
    meta = torch.empty(mb // 4, dtype=torch.int32, device=W.device)
    side = torch.empty((N, n_out), dtype=torch.int16, device=W.device)
    idx = torch.empty(n_out, dtype=torch.int32, device=W.device)
    ws = torch.empty(qgroup_outlier_ws(K, n_out), dtype=torch.uint8, device=W.device)
    _check(load().qpack_group_outlier(_ptr(W), N, K, bits, group, n_out, _ptr(codes), _ptr(meta),
                                      _ptr(side), _ptr(idx), _ptr(ws), ws.numel(), _stream(stream)),
           "qpack_group_outlier")
    return codes, meta, side, idx


def qgemv_group_outlier(codes, meta, side, idx, N: int, K: int, bits: int, group: int, x: torch.Tensor,
                        y: Optional[torch.Tensor] = None, y_dtype=torch.float32, stream=None):
    """y[B][N] = x W_rest_hat^T + x[:, idx] side^T."""
    cb, mb = qgroup_sizes(N, K, bits, group)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    n_out = idx.numel()
    _need_numel(idx, n_out, "idx", (torch.int32,))
    _need_numel(side, N * n_out, "side", _H16, exact=False)
    B = _batch(x, K)
    if y is None:
        y = torch.empty((B, N), dtype=y_dtype, device=x.device)
    _need_numel(y, B * N, "y", _OUT)
    _need_cuda(codes, meta, side, idx, x, y)
    _check(load().qgemv_group_outlier(_ptr(codes), _ptr(meta), _ptr(side), _ptr(idx), idx.numel(), N, K, bits,
                                      group, _ptr(x), _dtype_code(x), B, _ptr(y), _dtype_code(y),
                                      _stream(stream)), "qgemv_group_outlier")
    return y


# ------------------------------------------------- group codes with codebooks
def qcodebook_default(bits: int) -> torch.Tensor:
    """The library's default dictionary for b-bit codes: uint8 [8][2^b] (host)."""
    L = 1 << bits
    out = torch.zeros((8, L), dtype=torch.uint8)
    n = ctypes.c_int()
    _check(load().qcodebook_default(bits, ctypes.c_void_p(out.data_ptr()), ctypes.byref(n)), "qcodebook_default")
    return out[: n.value]


def qpack_group_cb(W: torch.Tensor, bits: int, group: int, books: torch.Tensor, stream=None):
    """(codes, meta, book_ids uint8[N][K/g]) for fp32 W[N][K] with the
    dictionary books (uint8 [D][2^b], on the device)."""
    if W.dim() != 2 or W.dtype != torch.float32:
        raise ValueError("W must be fp32 [N][K]")
    _need_numel(books, books.shape[0] << bits, "books", (torch.uint8,), exact=False)
    _need_cuda(W, books)
    N, K = W.shape
    cb, mb = qgroup_sizes(N, K, bits, group)
    codes = torch.empty(cb, dtype=torch.uint8, device=W.device)
    meta = torch.empty(mb // 4, dtype=torch.int32, device=W.device)
    ids = torch.empty((N, K // group), dtype=torch.uint8, device=W.device)
    _check(load().qpack_group_cb(_ptr(W), N, K, bits, group, _ptr(books), books.shape[0], _ptr(codes),
                                 _ptr(meta), _ptr(ids), _stream(stream)), "qpack_group_cb")
    return codes, meta, ids


def qgemv_group_cb(codes, meta, book_ids, books, N: int, K: int, bits: int, group: int, x: torch.Tensor,
                   y: Optional[torch.Tensor] = None, y_dtype=torch.float32, stream=None):
    """y[B][N] = x W_hat^T with w_hat = s * books[id][q] / 2^(7-b) + o."""
    cb, mb = qgroup_sizes(N, K, bits, group)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    _need_numel(book_ids, N * (K // group), "book_ids", (torch.uint8,), exact=False)
    _need_numel(books, books.shape[0] << bits, "books", (torch.uint8,), exact=False)
    B = _batch(x, K)
    if y is None:
        y = torch.empty((B, N), dtype=y_dtype, device=x.device)
    _need_numel(y, B * N, "y", _OUT)
    _need_cuda(codes, meta, book_ids, books, x, y)
    _check(load().qgemv_group_cb(_ptr(codes), _ptr(meta), _ptr(book_ids), _ptr(books), books.shape[0], N, K,
                                 bits, group, _ptr(x), _dtype_code(x), B, _ptr(y), _dtype_code(y),
                                 _stream(stream)), "qgemv_group_cb")
    return y


# ------------------------------------------------- key-cache quantization
def qtq_centroids(d: int, mbits: int):
    """(delta, table uint8 numpy [2^mbits]) on the 7-bit centroid grid."""
    import numpy as np
    t = np.zeros(1 << mbits, dtype=np.uint8)
    dl = ctypes.c_float()
    _check(load().qtq_centroids(d, mbits, ctypes.byref(dl), t.ctypes.data_as(ctypes.c_void_p)), "qtq_centroids")
    return dl.value, t


def qtq_rotation(G):
    """Q of G = QR, diag(R) > 0, for a host fp64 array G [d][d]."""
    import numpy as np
    G = np.ascontiguousarray(G, dtype=np.float64)
    out = np.empty_like(G)
    _check(load().qtq_rotation(G.shape[0], G.ctypes.data_as(ctypes.c_void_p), out.ctypes.data_as(ctypes.c_void_p)),
           "qtq_rotation")
    return out


def qtq_quant_keys(K: torch.Tensor, bits: int, Pi: torch.Tensor, S: torch.Tensor, delta: float, table,
                   stream=None):
    """(codes int32[n*4*(bits-1)], signs int32[n][4], norms int32[n]) for fp32 keys K[n][128]."""
    import numpy as np
    if K.dim() != 2 or K.shape[1] != 128 or K.dtype != torch.float32:
        raise ValueError("keys must be fp32 [n][128]")
    _need_numel(Pi, 128 * 128, "Pi", (torch.float64,))
    _need_numel(S, 128 * 128, "S", (torch.float64,))
    _need_cuda(K, Pi, S)
    n = K.shape[0]
    cb, sb, nb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qtq_sizes(n, bits, ctypes.byref(cb), ctypes.byref(sb), ctypes.byref(nb)), "qtq_sizes")
    codes = torch.empty(cb.value // 4, dtype=torch.int32, device=K.device)
    signs = torch.empty((n, 4), dtype=torch.int32, device=K.device)
    norms = torch.empty(n, dtype=torch.int32, device=K.device)
    t = np.ascontiguousarray(table, dtype=np.uint8)
    _check(load().qtq_quant_keys(_ptr(K), n, bits, _ptr(Pi), _ptr(S), float(delta), t.ctypes.data_as(ctypes.c_void_p),
                                 _ptr(codes), _ptr(signs), _ptr(norms), _stream(stream)), "qtq_quant_keys")
    return codes, signs, norms


def qtq_project(S: torch.Tensor, Pi: torch.Tensor, stream=None) -> torch.Tensor:
    """S Pi (fp64, device), the second matrix qtq_logits takes."""
    _need_numel(S, 128 * 128, "S", (torch.float64,))
    _need_numel(Pi, 128 * 128, "Pi", (torch.float64,))
    _need_cuda(S, Pi)
    out = torch.empty((128, 128), dtype=torch.float64, device=S.device)
    _check(load().qtq_project(_ptr(S), _ptr(Pi), _ptr(out), _stream(stream)), "qtq_project")
    return out


def qtq_logits(codes, signs, norms, n: int, heads: int, bits: int, delta: float, table, Pi, SPi, Qv: torch.Tensor,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """out[heads][nq][n] fp32 logits for queries Qv[heads][nq][128] (fp32);
    SPi = qtq_project(S, Pi)."""
    import numpy as np
    if Qv.dim() != 3 or Qv.shape[0] != heads or Qv.shape[2] != 128 or Qv.dtype != torch.float32:
        raise ValueError(f"queries must be fp32 [{heads}][nq][128]")
    nq = Qv.shape[1]
    cb, sb, nb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qtq_sizes(n * heads, bits, ctypes.byref(cb), ctypes.byref(sb), ctypes.byref(nb)), "qtq_sizes")
    _need_bytes(codes, cb.value, "codes")
    _need_bytes(signs, sb.value, "signs")
    _need_bytes(norms, nb.value, "norms")
    _need_numel(Pi, 128 * 128, "Pi", (torch.float64,))
    _need_numel(SPi, 128 * 128, "SPi", (torch.float64,))
    if out is None:
        out = torch.empty((heads, nq, n), dtype=torch.float32, device=Qv.device)
    _need_numel(out, heads * nq * n, "out", (torch.float32,))
    need = ctypes.c_size_t()
    _check(load().qtq_logits_ws(heads, nq, ctypes.byref(need)), "qtq_logits_ws")
    if ws is None:
        ws = torch.empty(need.value, dtype=torch.uint8, device=Qv.device)
    _need_bytes(ws, need.value, "ws")
    t = np.ascontiguousarray(table, dtype=np.uint8)
    _need_cuda(codes, signs, norms, Pi, SPi, Qv, out, ws)
    _check(load().qtq_logits(_ptr(codes), _ptr(signs), _ptr(norms), n, heads, bits, float(delta),
                             t.ctypes.data_as(ctypes.c_void_p), _ptr(Pi), _ptr(SPi), _ptr(Qv), nq, _ptr(out), _ptr(ws),
                             ws.numel(), _stream(stream)), "qtq_logits")
    return out


def qtq_quant_values(V: torch.Tensor, bits: int, Pi: torch.Tensor, delta: float, table, stream=None):
    """(codes int32[n*4*bits], norms int32[n]) for fp32 values V[n][128]."""
    import numpy as np
    if V.dim() != 2 or V.shape[1] != 128 or V.dtype != torch.float32:
        raise ValueError("values must be fp32 [n][128]")
    _need_numel(Pi, 128 * 128, "Pi", (torch.float64,))
    _need_cuda(V, Pi)
    n = V.shape[0]
    codes = torch.empty(n * 4 * bits, dtype=torch.int32, device=V.device)
    norms = torch.empty(n, dtype=torch.int32, device=V.device)
    t = np.ascontiguousarray(table, dtype=np.uint8)
    _check(load().qtq_quant_values(_ptr(V), n, bits, _ptr(Pi), float(delta), t.ctypes.data_as(ctypes.c_void_p),
                                   _ptr(codes), _ptr(norms), _stream(stream)), "qtq_quant_values")
    return codes, norms


def qtq_attend_ws(n: int, heads: int, nq: int) -> int:
    need = ctypes.c_size_t()
    _check(load().qtq_attend_ws(n, heads, nq, ctypes.byref(need)), "qtq_attend_ws")
    return need.value


def qtq_attend(codes, norms, n: int, heads: int, bits: int, delta: float, table, Pi, P: torch.Tensor,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """out[heads][nq][128] = P[heads][nq][n] times the dequantized values."""
    import numpy as np
    if P.dim() != 3 or P.shape[0] != heads or P.shape[2] != n or P.dtype != torch.float32:
        raise ValueError(f"weights must be fp32 [{heads}][nq][{n}]")
    nq = P.shape[1]
    _need_bytes(codes, n * heads * 16 * bits, "codes")
    _need_bytes(norms, n * heads * 4, "norms")
    _need_numel(Pi, 128 * 128, "Pi", (torch.float64,))
    if out is None:
        out = torch.empty((heads, nq, 128), dtype=torch.float32, device=P.device)
    _need_numel(out, heads * nq * 128, "out", (torch.float32,))
    need = qtq_attend_ws(n, heads, nq)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=P.device)
    _need_bytes(ws, need, "ws")
    t = np.ascontiguousarray(table, dtype=np.uint8)
    _need_cuda(codes, norms, Pi, P, out, ws)
    _check(load().qtq_attend(_ptr(codes), _ptr(norms), n, heads, bits, float(delta), t.ctypes.data_as(ctypes.c_void_p),
                             _ptr(Pi), _ptr(P), nq, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "qtq_attend")
    return out


# ---------------------------------------------------------------- binary LR
def qbinlr_sizes(N: int, K: int, r: int, B: int = 1):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qbinlr_sizes(N, K, r, B, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "qbinlr_sizes")
    return a.value, b.value, c.value


def qpack_binlr(U: torch.Tensor, V: torch.Tensor, ubits=None, vtbits=None, stream=None):
    if U.dim() != 2 or V.dim() != 2 or U.dtype != torch.int8 or V.dtype != torch.int8 or U.shape[1] != V.shape[1]:
        raise ValueError("U [N][r] and V [K][r] must be int8 with the same r")
    N, r = U.shape
    K = V.shape[0]
    ub, vb, _ = qbinlr_sizes(N, K, r)
    if ubits is None:
        ubits = torch.empty(ub // 4, dtype=torch.int32, device=U.device)
    if vtbits is None:
        vtbits = torch.empty(vb // 4, dtype=torch.int32, device=U.device)
    _need_bytes(ubits, ub, "ubits")
    _need_bytes(vtbits, vb, "vtbits")
    _need_cuda(U, V, ubits, vtbits)
    _check(load().qpack_binlr(_ptr(U), _ptr(V), N, K, r, _ptr(ubits), _ptr(vtbits), _stream(stream)),
           "qpack_binlr")
    return ubits, vtbits


def qunpack_binlr(ubits, vtbits, N: int, K: int, r: int, stream=None):
    ub, vb, _ = qbinlr_sizes(N, K, r)
    _need_bytes(ubits, ub, "ubits")
    _need_bytes(vtbits, vb, "vtbits")
    U = torch.empty((N, r), dtype=torch.int8, device=ubits.device)
    V = torch.empty((K, r), dtype=torch.int8, device=ubits.device)
    _need_cuda(ubits, vtbits)
    _check(load().qunpack_binlr(_ptr(ubits), _ptr(vtbits), N, K, r, _ptr(U), _ptr(V), _stream(stream)),
           "qunpack_binlr")
    return U, V


def qgemv_binlr(ubits, vtbits, s1, s2, N: int, K: int, r: int, x: torch.Tensor,
                y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                y_dtype=torch.float32, stream=None):
    B = _batch(x, K)
    ub, vb, wsb = qbinlr_sizes(N, K, r, B)
    _need_bytes(ubits, ub, "ubits")
    _need_bytes(vtbits, vb, "vtbits")
    _need_numel(s1, N, "s1", _H16, exact=False)
    _need_numel(s2, K, "s2", _H16, exact=False)
    if ws is None:
        ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    _need_bytes(ws, wsb, "ws")
    if y is None:
        y = torch.empty((B, N), dtype=y_dtype, device=x.device)
    _need_numel(y, B * N, "y", _OUT)
    _need_cuda(ubits, vtbits, s1, s2, x, y, ws)
    _check(load().qgemv_binlr(_ptr(ubits), _ptr(vtbits), _ptr(s1), _ptr(s2), N, K, r, _ptr(x),
                              _dtype_code(x), B, _ptr(y), _dtype_code(y), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "qgemv_binlr")
    return y


def qgemv_binlr_noalloc(ubits, vtbits, s1, s2, N: int, K: int, r: int, x: torch.Tensor,
                        y: Optional[torch.Tensor] = None, y_dtype=torch.float32, stream=None):
    """qgemv_binlr with the library's per-device scratch array as workspace
    (no workspace argument; the C call allocates nothing).  Pass y to keep
    the whole call free of allocations."""
    B = _batch(x, K)
    ub, vb, _ = qbinlr_sizes(N, K, r, B)
    _need_bytes(ubits, ub, "ubits")
    _need_bytes(vtbits, vb, "vtbits")
    _need_numel(s1, N, "s1", _H16, exact=False)
    _need_numel(s2, K, "s2", _H16, exact=False)
    if y is None:
        y = torch.empty((B, N), dtype=y_dtype, device=x.device)
    _need_numel(y, B * N, "y", _OUT)
    _need_cuda(ubits, vtbits, s1, s2, x, y)
    _check(load().qgemv_binlr_noalloc(_ptr(ubits), _ptr(vtbits), _ptr(s1), _ptr(s2), N, K, r, _ptr(x),
                                      _dtype_code(x), B, _ptr(y), _dtype_code(y), _stream(stream)),
           "qgemv_binlr_noalloc")
    return y


# -------------------------------------------------------------- measurement
def qstream_read(buf: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Read buf once as a plain 16-byte nontemporal stream (bandwidth
    reference); out is a device int32 scratch word."""
    nbytes = _nbytes(buf)
    if nbytes % 16:
        raise ValueError("buf: size not a multiple of 16 bytes")
    _need_bytes(out, 4, "out")
    _need_cuda(buf, out)
    _check(load().qstream_read(_ptr(buf), nbytes, _ptr(out), _stream(stream)), "qstream_read")


# ------------------------------------------------------------------ prefill
def make_qweight_group(codes, meta, N, K, bits, group, side=None, idx=None, book_ids=None,
                       books=None) -> qweight:
    """A qweight descriptor (optionally with outlier side columns, or with
    per-group books of a dictionary); it keeps references to the tensors it
    points into."""
    n_out = 0 if idx is None else idx.numel()
    cb, mb = qgroup_sizes(N, K, bits, group)
    _need_bytes(codes, cb, "codes")
    _need_bytes(meta, mb, "meta")
    if n_out:
        _need_numel(idx, n_out, "idx", (torch.int32,))
        _need_numel(side, N * n_out, "side", _H16, exact=False)
    if books is not None:
        _need_numel(books, books.shape[0] << bits, "books", (torch.uint8,), exact=False)
        _need_numel(book_ids, N * (K // group), "book_ids", (torch.uint8,), exact=False)
    _need_cuda(codes, meta, side, idx, book_ids, books)
    w = qweight(Q_FMT_GROUP, N, K, bits, group, codes.data_ptr(), meta.data_ptr(), 0, None, None, None, None,
                side.data_ptr() if n_out else None, idx.data_ptr() if n_out else None, n_out,
                None if book_ids is None else book_ids.data_ptr(), None if books is None else books.data_ptr(),
                0 if books is None else books.shape[0])
    w._tensors = (codes, meta, side, idx, book_ids, books)
    return w


def make_qweight_binlr(ubits, vtbits, s1, s2, N, K, r) -> qweight:
    """A qweight descriptor; it keeps references to the tensors it points into."""
    ub, vb, _ = qbinlr_sizes(N, K, r)
    _need_bytes(ubits, ub, "ubits")
    _need_bytes(vtbits, vb, "vtbits")
    _need_numel(s1, N, "s1", _H16, exact=False)
    _need_numel(s2, K, "s2", _H16, exact=False)
    _need_cuda(ubits, vtbits, s1, s2)
    w = qweight(Q_FMT_BINLR, N, K, 0, 0, None, None, r, ubits.data_ptr(), vtbits.data_ptr(),
                s1.data_ptr(), s2.data_ptr())
    w._tensors = (ubits, vtbits, s1, s2)
    return w


def qgemm_prefill_ws(w: qweight, M: int) -> int:
    n = ctypes.c_size_t()
    _check(load().qgemm_prefill_ws(ctypes.byref(w), M, ctypes.byref(n)), "qgemm_prefill_ws")
    return n.value


def qgemm_prefill(w: qweight, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, y_dtype=torch.float32, stream=None):
    if X.dim() != 2 or X.shape[1] != w.K:
        raise ValueError(f"X must be [M][{w.K}], got shape {tuple(X.shape)}")
    M = X.shape[0]
    need = qgemm_prefill_ws(w, M)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=X.device)
    if need:
        _need_bytes(ws, need, "ws")
    if Y is None:
        Y = torch.empty((M, w.N), dtype=y_dtype, device=X.device)
    _need_numel(Y, M * w.N, "Y", _OUT)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _need_cuda(X, Y, ws, *w._tensors)
    _check(load().qgemm_prefill(ctypes.byref(w), _ptr(X), _dtype_code(X), M, _ptr(Y), _dtype_code(Y),
                                _ptr(ws), nbytes, _stream(stream)), "qgemm_prefill")
    return Y


# ------------------------------------------------- quantized, paged KV cache
def qcache_sizes(n_pages: int, page_size: int, heads: int, head_dim: int, bits: int):
    """(codes, meta) bytes of one buffer each; K and V have one of both."""
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qcache_sizes(n_pages, page_size, heads, head_dim, bits, ctypes.byref(a), ctypes.byref(b)),
           "qcache_sizes")
    return a.value, b.value


def make_qcache(n_pages: int, page_size: int, heads: int, head_dim: int, bits: int, k_codes=None, k_meta=None,
                v_codes=None, v_meta=None, device=None) -> qcache:
    """A cache descriptor over the given buffers, or over new ones (zeros) on
    device when none are given; it keeps references to the tensors it points
    into (._tensors: k_codes, k_meta, v_codes, v_meta).  Buffers that hold
    anything but what qcache_write put there keep to its range: see
    include/qcache.h."""
    cb, mb = qcache_sizes(n_pages, page_size, heads, head_dim, bits)
    given = (k_codes, k_meta, v_codes, v_meta)
    if all(t is None for t in given):
        device = torch.device("cuda") if device is None else device
        given = tuple(torch.zeros(n, dtype=d, device=device)
                      for n, d in ((cb, torch.uint8), (mb // 4, torch.int32)) * 2)
    for t, n, what in zip(given, (cb, mb, cb, mb), ("k_codes", "k_meta", "v_codes", "v_meta")):
        _need_bytes(t, n, what)
    _need_cuda(*given)
    _one_device(*given)
    c = qcache(n_pages, page_size, heads, head_dim, bits, *(t.data_ptr() for t in given))
    c._tensors = given
    c._device, c._index = given[0].device, given[0].get_device()
    return c


def _one_device(first, *rest):
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")


def _cache_seqs(cache: qcache, T: int, pages, lens, starts) -> qseqs:
    if pages.dim() != 2 or pages.dtype != torch.int32:
        raise ValueError("pages must be int32 [B][max_pages]")
    B, width = pages.shape
    if lens is None or lens.dtype != torch.int32 or lens.numel() != B:
        _need_numel(lens, B, "lens", (torch.int32,))
    if starts is not None:
        _need_numel(starts, B + 1, "starts", (torch.int32,))
    elif T != B:
        raise ValueError(f"starts: missing, and {T} rows are not one for each of {B} sequences")
    return qseqs(B, T, width, pages.data_ptr(), lens.data_ptr(), None if starts is None else starts.data_ptr())


def _cache_rows(t: torch.Tensor, heads: int, D: int, dtypes, what: str) -> int:
    """Token stride (elements) of rows [T][heads][D]: dense within a token,
    any stride between tokens that keeps 16-byte alignment."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{what}: expected [T][{heads}][{D}], got shape {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {dtypes}")
    token, head, one = t.stride()
    if one != 1 or (heads > 1 and head != D) or (shape[0] > 1 and token < heads * D):
        raise ValueError(f"{what}: the rows of one token must be contiguous, got strides {t.stride()}")
    return token if shape[0] > 1 else heads * D


def _on_device(cache: qcache, dense: bool, *ts):
    """Every tensor is on the cache's device (and contiguous, where dense)."""
    for t in ts:
        if t is None:
            continue
        if t.get_device() != cache._index:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA (HIP) tensors")
            raise ValueError(f"tensors on different devices: {cache._device} and {t.device}")
        if dense and not t.is_contiguous():
            raise ValueError("pages, lens, starts and ws must be contiguous")


def _stream_of(cache: qcache, stream):
    if stream.device != cache._device:
        raise ValueError(f"stream on {stream.device}, tensors on {cache._device}")
    return stream


def _fresh(cache: qcache, stream, shape, dtype, returned: bool) -> torch.Tensor:
    """A tensor for a call on `stream` (None: the current one), out of that
    stream's memory pool: a block that the current stream's pool hands out may
    still be used by work queued there, which `stream` does not wait for.  A
    result is recorded on the current stream as well, where the caller goes on
    to use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache._device)
    with torch.cuda.stream(_stream_of(cache, stream)):
        t = torch.empty(shape, dtype=dtype, device=cache._device)
    if returned:
        t.record_stream(torch.cuda.current_stream(cache._device))
    return t


def _cache_call(cache: qcache, stream, what, fn, *args):
    """fn(cache, *args, stream) on the cache's device."""
    idx = cache._index
    if stream is None and idx == torch._C._cuda_getDevice():
        status = fn(cache, *args, torch._C._cuda_getCurrentRawStream(idx))
    else:
        stream = torch.cuda.current_stream(cache._device) if stream is None else _stream_of(cache, stream)
        with torch.cuda.device(cache._device):
            status = fn(cache, *args, stream.cuda_stream)
    if status != Q_OK:
        raise QError(status, what)


def qcache_write(cache: qcache, K: torch.Tensor, V: torch.Tensor, pages, lens, starts=None, stream=None) -> None:
    """Quantize rows K, V [T][heads][head_dim] (bf16 or fp32) into the cache:
    the newest tokens of sequences with page tables pages int32
    [B][max_pages] and lengths lens int32 [B] (the new tokens included); rows
    starts[b] .. starts[b+1]-1 are sequence b's, one row each without starts."""
    ks = _cache_rows(K, cache.heads, cache.head_dim, _OUT, "K")
    vs = _cache_rows(V, cache.heads, cache.head_dim, (K.dtype,), "V")
    T = K.shape[0]
    if V.shape[0] != T:
        raise ValueError(f"V: {V.shape[0]} rows, K has {T}")
    seqs = _cache_seqs(cache, T, pages, lens, starts)
    _on_device(cache, True, pages, lens, starts)
    _on_device(cache, False, K, V)
    if T == 0:
        return
    _cache_call(cache, stream, "qcache_write", load().qcache_write, seqs, K.data_ptr(), ks, V.data_ptr(), vs,
                _dtype_code(K))


def qcache_read(cache: qcache, pages, lens, starts=None, rows: Optional[int] = None, K: Optional[torch.Tensor] = None,
                V: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None):
    """(K, V) [rows][heads][head_dim] of the cache as values: the last
    starts[b+1] - starts[b] tokens of each sequence, the last one without
    starts.  rows: starts[B] when no outputs are given (host knowledge; the
    call does not look at device data).  Rows no sequence owns are not
    written.  Outputs allocated here belong to `stream`: another stream waits
    for it before it reads them."""
    heads, D = cache.heads, cache.head_dim
    given = K is not None or V is not None
    if not given:
        if rows is None:
            if starts is not None:
                raise ValueError("rows: missing, and no outputs given")
            rows = pages.shape[0]
        if dtype not in _OUT:
            raise ValueError(f"dtype {dtype}, expected one of {_OUT}")
        T, ks, vs = rows, heads * D, heads * D
    elif K is None or V is None:
        raise ValueError("K and V: both outputs or neither")
    else:
        ks = _cache_rows(K, heads, D, _OUT, "K")
        vs = _cache_rows(V, heads, D, (K.dtype,), "V")
        T = K.shape[0]
        if V.shape[0] != T:
            raise ValueError(f"V: {V.shape[0]} rows, K has {T}")
        _on_device(cache, False, K, V)
    seqs = _cache_seqs(cache, T, pages, lens, starts)
    _on_device(cache, True, pages, lens, starts)
    if not given:
        K, V = _fresh(cache, stream, (2, T, heads, D), dtype, True).unbind(0)
    if T == 0:
        return K, V
    _cache_call(cache, stream, "qcache_read", load().qcache_read, seqs, K.data_ptr(), ks, V.data_ptr(), vs,
                _dtype_code(K))
    return K, V


@functools.lru_cache(maxsize=1024)
def _attend_ws(page_size, heads, head_dim, bits, B, T, max_pages, q_heads, prefix_len) -> int:
    n = ctypes.c_size_t()
    c, seqs = qcache(1, page_size, heads, head_dim, bits), qseqs(B, T, max_pages)
    _check(load().qcache_attend_ws(ctypes.byref(c), ctypes.byref(seqs), q_heads, prefix_len, ctypes.byref(n)),
           "qcache_attend_ws")
    return n.value


def qcache_attend_ws(cache: qcache, B: int, T: int, max_pages: int, q_heads: int, prefix_len: int = 0) -> int:
    """Workspace bytes for B sequences with T rows and page tables of
    max_pages entries (prefix_len: of qcache_attend_shared)."""
    return _attend_ws(cache.page_size, cache.heads, cache.head_dim, cache.bits, B, T, max_pages, q_heads, prefix_len)


def _cache_attend(what, cache, Q, prefix, pages, lens, starts, scale, out, out_dtype, ws, stream):
    """prefix: () or (prefix_pages, prefix_len)."""
    heads, D = cache.heads, cache.head_dim
    shape = Q.shape
    if len(shape) != 3 or shape[1] < 1 or shape[1] % heads:
        raise ValueError(f"Q: expected [T][q_heads][{D}] with q_heads a multiple of {heads}, got shape {tuple(shape)}")
    T, q_heads, _ = shape
    q_stride = _cache_rows(Q, q_heads, D, _Q16, "Q")
    seqs = _cache_seqs(cache, T, pages, lens, starts)
    if out is None:
        if out_dtype not in _OUT:
            raise ValueError(f"out_dtype {out_dtype}, expected one of {_OUT}")
        o_stride = q_heads * D
    else:
        o_stride = _cache_rows(out, q_heads, D, _OUT, "out")
        if out.shape[0] != T:
            raise ValueError(f"out: {out.shape[0]} rows, Q has {T}")
    _on_device(cache, True, pages, lens, starts)
    _on_device(cache, False, Q, out)
    if out is None:
        out = _fresh(cache, stream, (T, q_heads, D), out_dtype, True)
    if T == 0:
        return out
    n_prefix = prefix[1] if prefix else 0
    need = _attend_ws(cache.page_size, heads, D, cache.bits, seqs.B, T, seqs.max_pages, q_heads, n_prefix)
    if ws is None:
        ws = _fresh(cache, stream, need, torch.uint8, False)
        ws_bytes = need
    else:
        _need_bytes(ws, need, "ws")
        _on_device(cache, True, ws)
        ws_bytes = _nbytes(ws)
    rest = (Q.data_ptr(), q_stride, q_heads, D ** -0.5 if scale is None else scale, out.data_ptr(), o_stride,
            Q_F32 if out.dtype == torch.float32 else Q_BF16, ws.data_ptr(), ws_bytes)
    if prefix:
        _on_device(cache, True, prefix[0])
        _cache_call(cache, stream, what, load().qcache_attend_shared, seqs, prefix[0].data_ptr(), n_prefix, *rest)
    else:
        _cache_call(cache, stream, what, load().qcache_attend, seqs, *rest)
    return out


def qcache_attend(cache: qcache, Q: torch.Tensor, pages, lens, starts=None, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, ws: Optional[torch.Tensor] = None,
                  stream=None):
    """out [T][q_heads][head_dim] (bf16 or fp32): causal attention of rows Q
    (bf16) over the cached tokens of their sequences; pages, lens and starts
    as qcache_write's, whose rows these are.  scale: head_dim^-1/2 by
    default.  Calls that may overlap need a workspace each.  An output that is
    allocated here belongs to `stream`: another stream waits for it first."""
    return _cache_attend("qcache_attend", cache, Q, (), pages, lens, starts, scale, out, out_dtype, ws, stream)


def qcache_attend_shared(cache: qcache, Q: torch.Tensor, prefix_pages, prefix_len: int, pages, lens, starts=None,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         out_dtype=torch.bfloat16, ws: Optional[torch.Tensor] = None, stream=None):
    """qcache_attend behind a prefix of prefix_len tokens (pages prefix_pages,
    int32) that all rows see, read once for every 256 rows of a KV head and not
    for every sequence.  pages and lens describe the sequences' own tokens
    only."""
    if prefix_pages is None or prefix_pages.dtype != torch.int32:
        raise ValueError("prefix_pages must be int32")
    if prefix_len < 1:
        raise ValueError(f"prefix_len: {prefix_len}, must be at least 1")
    _need_numel(prefix_pages, -(-prefix_len // cache.page_size), "prefix_pages", (torch.int32,), exact=False)
    return _cache_attend("qcache_attend_shared", cache, Q, (prefix_pages, prefix_len), pages, lens, starts, scale, out,
                         out_dtype, ws, stream)
