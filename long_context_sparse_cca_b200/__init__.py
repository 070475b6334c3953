"""CCA-Attention on NVIDIA B200: Python binding of the C library libcca.

Thin ctypes layer over ``include/cca.h``: it checks tensor devices, dtypes
and layouts, allocates outputs with PyTorch when the caller passes none, and
hands raw device pointers and the current CUDA stream to the library.  Every
step of the computation runs in the library's CUDA kernels; there is no
other code path.  If ``libcca.so`` is missing, every call raises.

Build the library with ``python -m long_context_sparse_cca_b200.build``.

Entry points (same names as the C ABI):
    cca_pool, cca_attn_prefill, cca_cache_prefill, cca_cache_append,
    cca_attn_prefill_lse (forward that keeps each row's log-sum-exp),
    cca_attn_backward, cca_attn_backward_workspace_bytes (training),
    cca_attn_decode, cca_decode_step (append + decode in one launch),
    cca_decode_workspace_bytes, cca_attn_decode_noalloc,
    cca_cache_append_rows, cca_attn_decode_rows (per-row lengths in device
    memory), cca_lca_pool, cca_lca_cache_prefill, cca_lca_cache_append (the
    LCA variant's condensation; ``lca_query_sums`` allocates the running
    query sums its cache calls keep), cca_pool_packed,
    cca_packed_workspace_bytes, cca_attn_prefill_packed (prompts of different
    lengths without padding), cca_paged_workspace_bytes, cca_paged_reserve
    (cca_paged_reserve_held of the C ABI), cca_paged_fill, cca_attn_decode_paged, cca_paged_step, cca_paged_fork,
    cca_paged_compact (a decode cache whose rows share memory in pages),
    cca_selftest_wait_timeout, cca_device_status
and the ``Cache`` and ``PagedCache`` classes holding a decode cache's device
buffers.

Every call runs on ``stream`` (None: the current one).  What it allocates
(outputs, a workspace) belongs to that stream, as with PyTorch calls made
under ``torch.cuda.stream(stream)``: before another stream uses an output it
waits for that stream, and ``record_stream`` tells PyTorch of a use that may
outlast the tensor.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcca.so")

CCA_OK = 0
CCA_ERR_INVALID_ARG = 1
CCA_ERR_UNSUPPORTED = 2
CCA_ERR_CAPACITY = 3
CCA_ERR_CUDA = 4
CCA_ERR_TIMEOUT = 5
CCA_ERR_RANGE = 6
CCA_ERR_SCRATCH = 7
CCA_ERR_SEQLENS = 8
CCA_ERR_PAGE = 9
CCA_BF16 = 0
CCA_F32 = 1
NOALLOC_SCRATCH_BYTES = 4 << 20  # CCA_NOALLOC_SCRATCH_BYTES of include/cca.h

# Every symbol include/cca.h declares.
EXPORTS = ("cca_pool", "cca_attn_prefill", "cca_cache_prefill",
           "cca_cache_append", "cca_decode_workspace_bytes", "cca_attn_decode",
           "cca_device_status", "cca_status_string", "cca_version", "cca_last_error",
           "cca_attn_decode_noalloc", "cca_selftest_wait_timeout",
           "cca_cache_append_rows", "cca_attn_decode_rows", "cca_decode_step",
           "cca_attn_prefill_lse", "cca_attn_backward", "cca_attn_backward_workspace_bytes",
           "cca_lca_pool", "cca_lca_cache_prefill", "cca_lca_cache_append",
           "cca_pool_packed", "cca_packed_workspace_bytes", "cca_attn_prefill_packed",
           "cca_paged_workspace_bytes", "cca_paged_reserve", "cca_paged_reserve_held",
           "cca_paged_fill",
           "cca_attn_decode_paged", "cca_paged_step", "cca_paged_fork", "cca_paged_compact")


class CCAError(RuntimeError):
    """A nonzero status from libcca."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_core", ctypes.c_void_p), ("v_core", ctypes.c_void_p),
                ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("g", ctypes.c_int), ("w", ctypes.c_int),
                ("core_cap", ctypes.c_int64), ("tail_cap", ctypes.c_int64),
                ("len", ctypes.c_int64)]


class _RowsStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class _PagedStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in
                 ("k_core", "v_core", "k_raw", "v_raw", "core_table", "raw_table", "core_ref",
                  "raw_ref", "lens")] +
                [(n, ctypes.c_int) for n in
                 ("layers", "B", "Hq", "Hkv", "d", "g", "w", "page", "core_cols", "raw_cols",
                  "core_pages", "raw_pages")])


_lib = None


def lib():
    """Load libcca.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"libcca.so not found at {LIB_PATH}; build it with "
            "`python -m long_context_sparse_cca_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i, i64, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int
    CP = ctypes.POINTER(_CacheStruct)
    L.cca_pool.argtypes = [P, P, P, P, P, i, i, i, i64, i, i, P]
    L.cca_pool.restype = st
    L.cca_attn_prefill.argtypes = [P, P, P, P, P, P, i, i, i, i, i64, i, i, i, P]
    L.cca_attn_prefill.restype = st
    L.cca_attn_prefill_lse.argtypes = [P, P, P, P, P, P, i, P, i, i, i, i64, i, i, i, P]
    L.cca_attn_prefill_lse.restype = st
    L.cca_attn_backward_workspace_bytes.argtypes = [i, i, i, i64, i, i]
    L.cca_attn_backward_workspace_bytes.restype = ctypes.c_size_t
    L.cca_attn_backward.argtypes = [P, P, P, P, P, P, i, P, P, P, P, P, i, i, i, i64, i, i, i,
                                    P, ctypes.c_size_t, P]
    L.cca_attn_backward.restype = st
    L.cca_lca_pool.argtypes = [P, P, P, P, P, i, i, i, i64, i, i, i, P]
    L.cca_lca_pool.restype = i
    L.cca_lca_cache_prefill.argtypes = [CP, P, P, P, P, i64, i, P]
    L.cca_lca_cache_prefill.restype = i
    L.cca_lca_cache_append.argtypes = [CP, P, P, P, P, i, P]
    L.cca_lca_cache_append.restype = i
    L.cca_cache_prefill.argtypes = [CP, P, P, P, i64, P]
    L.cca_cache_prefill.restype = st
    L.cca_cache_append.argtypes = [CP, P, P, P, P]
    L.cca_cache_append.restype = st
    L.cca_decode_workspace_bytes.argtypes = [CP]
    L.cca_decode_workspace_bytes.restype = ctypes.c_size_t
    L.cca_attn_decode.argtypes = [CP, P, P, i, P, ctypes.c_size_t, P]
    L.cca_attn_decode.restype = st
    L.cca_attn_decode_noalloc.argtypes = [CP, P, P, i, P]
    L.cca_attn_decode_noalloc.restype = st
    L.cca_decode_step.argtypes = [CP, P, P, P, P, i, P, ctypes.c_size_t, P]
    L.cca_decode_step.restype = st
    L.cca_cache_append_rows.argtypes = [CP, P, P, P, P, P]
    L.cca_cache_append_rows.restype = st
    L.cca_attn_decode_rows.argtypes = [CP, P, P, P, i, P, ctypes.c_size_t, P]
    L.cca_attn_decode_rows.restype = st
    RP, PP, sz = ctypes.POINTER(_RowsStruct), ctypes.POINTER(_PagedStruct), ctypes.c_size_t
    L.cca_pool_packed.argtypes = [RP, RP, RP, P, P, P, i, i, i, i64, i, i, P]
    L.cca_pool_packed.restype = st
    L.cca_packed_workspace_bytes.argtypes = [i, i64]
    L.cca_packed_workspace_bytes.restype = sz
    L.cca_attn_prefill_packed.argtypes = [RP, RP, RP, P, P, P, RP, i, i, i, i, i64, i, i, i,
                                          P, sz, P]
    L.cca_attn_prefill_packed.restype = st
    L.cca_paged_workspace_bytes.argtypes = [PP]
    L.cca_paged_workspace_bytes.restype = sz
    L.cca_paged_reserve.argtypes = [PP, P, ctypes.c_longlong, P]
    L.cca_paged_reserve.restype = st
    L.cca_paged_reserve_held.argtypes = [PP, P, ctypes.c_longlong, P, sz, P]
    L.cca_paged_reserve_held.restype = st
    L.cca_paged_fill.argtypes = [PP, i, RP, RP, P, P, P, P, i, i64, P]
    L.cca_paged_fill.restype = st
    L.cca_attn_decode_paged.argtypes = [PP, i, P, P, i, P, sz, P]
    L.cca_attn_decode_paged.restype = st
    L.cca_paged_step.argtypes = [PP, i, P, P, P, P, i, P, sz, P]
    L.cca_paged_step.restype = st
    L.cca_paged_fork.argtypes = [PP, P, P, sz, P]
    L.cca_paged_fork.restype = st
    L.cca_paged_compact.argtypes = [PP, P, P, sz, P]
    L.cca_paged_compact.restype = st
    L.cca_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
    L.cca_selftest_wait_timeout.restype = st
    L.cca_device_status.argtypes = [P]
    L.cca_device_status.restype = st
    L.cca_status_string.argtypes = [i]
    L.cca_status_string.restype = ctypes.c_char_p
    L.cca_version.argtypes = []
    L.cca_version.restype = ctypes.c_char_p
    L.cca_last_error.argtypes = []
    L.cca_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().cca_status_string(int(status)).decode()


def version() -> str:
    return lib().cca_version().decode()


def last_error() -> str:
    """CUDA error text behind this thread's last CCA_ERR_CUDA."""
    return lib().cca_last_error().decode()


def _check(status: int, what: str) -> None:
    if status != CCA_OK:
        if status == CCA_ERR_CUDA:
            what = f"{what} ({last_error()})"
        raise CCAError(status, what)


def _torch():
    import torch
    return torch


def _stream(stream) -> ctypes.c_void_p:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Context in which ``stream`` is the current one."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _new(like, shape, dtype, stream, fill=None):
    """A tensor on the device of ``like`` for a call on ``stream`` (None: the
    current one), from that stream's pool: memory of another stream's pool
    could still be in use by work queued there, and would go back to it while
    the call's own work has yet to run."""
    if stream is None:
        t = like.new_empty(shape, dtype=dtype)
        return t if fill is None else t.fill_(fill)
    with _on(stream):
        return _new(like, shape, dtype, None, fill)


def _dev(t, name: str, dtype=None):
    """Pointer of a contiguous CUDA tensor (None passes NULL)."""
    if t is None:
        return None
    torch = _torch()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    want = dtype or torch.bfloat16
    if t.dtype != want:
        raise ValueError(f"{name} must be {want}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _workspace(t):
    """Address and bytes of a caller's workspace: contiguous, so that as many
    bytes as it has elements lie behind its address (an expanded tensor has
    less memory than that)."""
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not t.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr()), t.numel() * t.element_size()


def _int(x, name: str, bits: int = 32) -> int:
    """A number for a C integer of so many bits, to which ctypes would cut it
    without a word."""
    x = int(x)
    if x >> (bits - 1) not in (0, -1):
        raise ValueError(f"{name} = {x} does not fit in {bits} bits")
    return x


def _odtype(out_dtype) -> int:
    torch = _torch()
    if out_dtype in (torch.bfloat16, "bf16"):
        return CCA_BF16
    if out_dtype in (torch.float32, "f32", "fp32"):
        return CCA_F32
    raise ValueError(f"unsupported output dtype {out_dtype}")


def cca_pool(Q, K, V, g: int, Kc=None, Vc=None, stream=None):
    """Globally-aware pooling: Q [B,Hq,T,d], K/V [B,Hkv,T,d] (bf16, CUDA).

    Returns (Kc, Vc) [B, Hkv, T // g, d] fp16.
    """
    torch = _torch()
    B, Hq, T, d = Q.shape
    Hkv = K.shape[1]
    m = T // g
    if Kc is None:
        Kc = _new(Q, (B, Hkv, m, d), torch.float16, stream)
    if Vc is None:
        Vc = _new(Q, (B, Hkv, m, d), torch.float16, stream)
    if tuple(K.shape) != (B, Hkv, T, d) or tuple(V.shape) != (B, Hkv, T, d):
        raise ValueError("K and V must be [B, Hkv, T, d]")
    if tuple(Kc.shape) != (B, Hkv, m, d) or tuple(Vc.shape) != (B, Hkv, m, d):
        raise ValueError("Kc and Vc must be [B, Hkv, T // g, d]")
    _check(lib().cca_pool(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"),
                          _dev(Kc, "Kc", torch.float16), _dev(Vc, "Vc", torch.float16),
                          B, Hq, Hkv, T, d,
                          _int(g, "g"), _stream(stream)), "cca_pool")
    return Kc, Vc


def cca_attn_prefill(Q, K, V, Kc, Vc, g: int, w: int, O=None,
                     out_dtype=None, stream=None):
    """Fused core + local attention over the whole sequence.

    Q [B,Hq,T,d], K/V [B,Hkv,T,d] (bf16), Kc/Vc [B,Hkv,T//g,d] (fp16).
    Returns O [B, Hq, T, d] in ``out_dtype`` (bf16 default, or fp32).
    """
    torch = _torch()
    B, Hq, T, d = Q.shape
    Hkv = K.shape[1]
    if O is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        O = _new(Q, (B, Hq, T, d), dt, stream)
    od = _odtype(O.dtype)
    if tuple(O.shape) != (B, Hq, T, d):
        raise ValueError("O must be [B, Hq, T, d]")
    _check(lib().cca_attn_prefill(
        _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(Kc, "Kc", torch.float16),
        _dev(Vc, "Vc", torch.float16), _dev(O, "O", O.dtype), od, B, Hq, Hkv, T, d, _int(g, "g"),
        _int(w, "w"), _stream(stream)), "cca_attn_prefill")
    return O


def cca_attn_prefill_lse(Q, K, V, Kc, Vc, g: int, w: int, O=None, out_dtype=None,
                         lse=None, stream=None):
    """cca_attn_prefill that also returns each row's log-sum-exp (fp32
    [B, Hq, T], log2 units), as cca_attn_backward needs: (O, lse)."""
    torch = _torch()
    B, Hq, T, d = Q.shape
    Hkv = K.shape[1]
    if O is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        O = _new(Q, (B, Hq, T, d), dt, stream)
    if lse is None:
        lse = _new(Q, (B, Hq, T), torch.float32, stream)
    od = _odtype(O.dtype)
    if tuple(O.shape) != (B, Hq, T, d) or tuple(lse.shape) != (B, Hq, T):
        raise ValueError("O must be [B, Hq, T, d] and lse [B, Hq, T]")
    _check(lib().cca_attn_prefill_lse(
        _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(Kc, "Kc", torch.float16),
        _dev(Vc, "Vc", torch.float16), _dev(O, "O", O.dtype), od,
        _dev(lse, "lse", torch.float32), B, Hq, Hkv, T, d, _int(g, "g"), _int(w, "w"),
        _stream(stream)), "cca_attn_prefill_lse")
    return O, lse


def cca_attn_backward_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int, g: int) -> int:
    return int(lib().cca_attn_backward_workspace_bytes(int(B), int(Hq), int(Hkv), int(T),
                                                       int(d), _int(g, "g")))


def cca_attn_backward(Q, K, V, Kc, Vc, O, lse, dO, g: int, w: int, dQ=None, dK=None,
                      dV=None, workspace=None, stream=None):
    """Gradients (dQ, dK, dV), fp32, of sum(dO * O) for the CCA attention
    O = attention(Q, K, V) with its pooled Kc, Vc (from cca_pool) and the
    forward's O and lse (from cca_attn_prefill_lse).  dO: bf16 like Q."""
    torch = _torch()
    B, Hq, T, d = Q.shape
    Hkv = K.shape[1]
    dQ = _new(Q, (B, Hq, T, d), torch.float32, stream) if dQ is None else dQ
    dK = _new(Q, (B, Hkv, T, d), torch.float32, stream) if dK is None else dK
    dV = _new(Q, (B, Hkv, T, d), torch.float32, stream) if dV is None else dV
    nbytes = cca_attn_backward_workspace_bytes(B, Hq, Hkv, T, d, g)
    if workspace is None:
        workspace = _new(Q, max(nbytes, 256), torch.uint8, stream)
    _check(lib().cca_attn_backward(
        _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(Kc, "Kc", torch.float16),
        _dev(Vc, "Vc", torch.float16), _dev(O, "O", O.dtype), _odtype(O.dtype),
        _dev(lse, "lse", torch.float32), _dev(dO, "dO"), _dev(dQ, "dQ", torch.float32),
        _dev(dK, "dK", torch.float32), _dev(dV, "dV", torch.float32), B, Hq, Hkv, T, d,
        _int(g, "g"), _int(w, "w"), *_workspace(workspace), _stream(stream)),
        "cca_attn_backward")
    return dQ, dK, dV


class Cache:
    """A decode cache: core slots of completed groups (fp16) plus a raw ring
    of ``tail_cap`` tokens (bf16, default w + g), device buffers owned here."""

    def __init__(self, B: int, Hq: int, Hkv: int, d: int, g: int, w: int,
                 core_cap: int, tail_cap: Optional[int] = None, device="cuda"):
        torch = _torch()
        tail_cap = w + g if tail_cap is None else int(tail_cap)
        kw = dict(dtype=torch.bfloat16, device=device)
        kh = dict(dtype=torch.float16, device=device)
        self.k_core = torch.zeros((B, Hkv, core_cap, d), **kh)
        self.v_core = torch.zeros((B, Hkv, core_cap, d), **kh)
        self.k_tail = torch.zeros((B, Hkv, tail_cap, d), **kw)
        self.v_tail = torch.zeros((B, Hkv, tail_cap, d), **kw)
        self.struct = _CacheStruct(self.k_core.data_ptr(), self.v_core.data_ptr(),
                                   self.k_tail.data_ptr(), self.v_tail.data_ptr(),
                                   *(_int(x, "a size of Cache") for x in (B, Hq, Hkv, d, g, w)),
                                   core_cap, tail_cap, 0)
        self.workspace = None

    def row(self, b: int) -> "Cache":
        """Row b alone: a B = 1 cache over the same device buffers (for
        example to fill rows from prefixes of different lengths with
        cca_cache_prefill before decoding them with per-row lengths)."""
        v = object.__new__(Cache)
        v.k_core, v.v_core = self.k_core[b:b + 1], self.v_core[b:b + 1]
        v.k_tail, v.v_tail = self.k_tail[b:b + 1], self.v_tail[b:b + 1]
        st = self.struct
        v.struct = _CacheStruct(v.k_core.data_ptr(), v.v_core.data_ptr(),
                                v.k_tail.data_ptr(), v.v_tail.data_ptr(),
                                1, st.Hq, st.Hkv, st.d, st.g, st.w, st.core_cap,
                                st.tail_cap, 0)
        v.workspace = None
        return v

    def state_dict(self) -> dict:
        """Host copy of the cache (core slots, ring, shape, length), for
        saving and later restoring a decode session."""
        st = self.struct
        return {"shape": {n: int(getattr(st, n)) for n in
                          ("B", "Hq", "Hkv", "d", "g", "w", "core_cap", "tail_cap")},
                "len": int(st.len),
                "k_core": self.k_core.cpu(), "v_core": self.v_core.cpu(),
                "k_tail": self.k_tail.cpu(), "v_tail": self.v_tail.cpu()}

    @classmethod
    def from_state_dict(cls, state: dict, device="cuda") -> "Cache":
        """A cache on ``device`` holding what ``state_dict`` saved."""
        sh = state["shape"]
        c = cls(sh["B"], sh["Hq"], sh["Hkv"], sh["d"], sh["g"], sh["w"], sh["core_cap"],
                sh["tail_cap"], device=device)
        for n in ("k_core", "v_core", "k_tail", "v_tail"):
            getattr(c, n).copy_(state[n])
        c.len = state["len"]
        return c

    @property
    def len(self) -> int:
        return int(self.struct.len)

    @len.setter
    def len(self, n: int) -> None:
        self.struct.len = int(n)

    def __getattr__(self, name):
        if name in ("B", "Hq", "Hkv", "d", "g", "w", "core_cap", "tail_cap"):
            return getattr(self.struct, name)
        raise AttributeError(name)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.k_core, self.v_core, self.k_tail, self.v_tail))


def cca_cache_prefill(cache: Cache, Q, K, V, stream=None) -> None:
    """Fill ``cache`` from a prefix Q [B,Hq,T,d], K/V [B,Hkv,T,d]."""
    T = Q.shape[2]
    _check(lib().cca_cache_prefill(ctypes.byref(cache.struct), _dev(Q, "Q"),
                                   _dev(K, "K"), _dev(V, "V"), T,
                                   _stream(stream)), "cca_cache_prefill")


def cca_cache_append(cache: Cache, q_t, k_t, v_t, stream=None) -> None:
    """Append one token: q_t [B,Hq,d], k_t/v_t [B,Hkv,d] (bf16, CUDA)."""
    _check(lib().cca_cache_append(ctypes.byref(cache.struct), _dev(q_t, "q_t"),
                                  _dev(k_t, "k_t"), _dev(v_t, "v_t"),
                                  _stream(stream)), "cca_cache_append")


# ---- the LCA variant: latent-condensed pooling with a positional anchor

def cca_lca_pool(Q, K, V, g: int, d_rope: int, Kc=None, Vc=None, stream=None):
    """LCA condensation: Q [B,Hq,T,d], K/V [B,Hkv,T,d] (bf16, CUDA); the last
    d_rope entries of a key row are its positional part.

    Returns (Kc, Vc) [B, Hkv, T // g, d] fp16, for cca_attn_prefill.
    """
    torch = _torch()
    B, Hq, T, d = Q.shape
    Hkv = K.shape[1]
    m = T // g
    if Kc is None:
        Kc = _new(Q, (B, Hkv, m, d), torch.float16, stream)
    if Vc is None:
        Vc = _new(Q, (B, Hkv, m, d), torch.float16, stream)
    if tuple(K.shape) != (B, Hkv, T, d) or tuple(V.shape) != (B, Hkv, T, d):
        raise ValueError("K and V must be [B, Hkv, T, d]")
    if tuple(Kc.shape) != (B, Hkv, m, d) or tuple(Vc.shape) != (B, Hkv, m, d):
        raise ValueError("Kc and Vc must be [B, Hkv, T // g, d]")
    _check(lib().cca_lca_pool(_dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"),
                              _dev(Kc, "Kc", torch.float16), _dev(Vc, "Vc", torch.float16),
                              B, Hq, Hkv, T, d, _int(g, "g"), _int(d_rope, "d_rope"),
                              _stream(stream)), "cca_lca_pool")
    return Kc, Vc


def lca_query_sums(cache: Cache):
    """A zeroed q_sum [B, Hq, d] fp32 buffer for the LCA cache calls."""
    torch = _torch()
    return torch.zeros((cache.B, cache.Hq, cache.d), dtype=torch.float32, device="cuda")


def _qsum(cache: Cache, q_sum):
    torch = _torch()
    if tuple(q_sum.shape) != (cache.B, cache.Hq, cache.d):
        raise ValueError("q_sum must be [B, Hq, d]")
    return _dev(q_sum, "q_sum", torch.float32)


def cca_lca_cache_prefill(cache: Cache, q_sum, Q, K, V, d_rope: int, stream=None) -> None:
    """Fill ``cache`` from a prefix with LCA condensation; sets q_sum to the
    open group's query sums."""
    T = Q.shape[2]
    _check(lib().cca_lca_cache_prefill(ctypes.byref(cache.struct), _qsum(cache, q_sum),
                                       _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), T,
                                       _int(d_rope, "d_rope"), _stream(stream)),
           "cca_lca_cache_prefill")


def cca_lca_cache_append(cache: Cache, q_sum, q_t, k_t, v_t, d_rope: int, stream=None) -> None:
    """Append one token with LCA condensation of the group it completes."""
    _check(lib().cca_lca_cache_append(ctypes.byref(cache.struct), _qsum(cache, q_sum),
                                      _dev(q_t, "q_t"), _dev(k_t, "k_t"), _dev(v_t, "v_t"),
                                      _int(d_rope, "d_rope"), _stream(stream)),
           "cca_lca_cache_append")


def cca_decode_workspace_bytes(cache: Cache) -> int:
    return int(lib().cca_decode_workspace_bytes(ctypes.byref(cache.struct)))


def cca_attn_decode(cache: Cache, q_t, o_t=None, out_dtype=None,
                    workspace=None, stream=None):
    """Attention of the newest token: q_t [B,Hq,d] -> o_t [B,Hq,d]."""
    torch = _torch()
    if o_t is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        o_t = _new(q_t, tuple(q_t.shape), dt, stream)
    od = _odtype(o_t.dtype)
    if workspace is None:
        workspace = _cache_workspace(cache, q_t, stream)
    _check(lib().cca_attn_decode(
        ctypes.byref(cache.struct), _dev(q_t, "q_t"), _dev(o_t, "o_t", o_t.dtype),
        od, *_workspace(workspace), _stream(stream)), "cca_attn_decode")
    return o_t


def _cache_workspace(cache: Cache, like, stream):
    """The cache's own decode workspace, zero-filled when (re)allocated, as
    cca_decode_step requires before its first use, on the call's stream."""
    nbytes = cca_decode_workspace_bytes(cache)
    if cache.workspace is None or cache.workspace.numel() < nbytes:
        cache.workspace = _new(like, max(nbytes, 256), _torch().uint8, stream, fill=0)
    return cache.workspace


def cca_decode_step(cache: Cache, q_t, k_t, v_t, o_t=None, out_dtype=None,
                    workspace=None, stream=None):
    """Append token t = cache.len and return its attention output, in one
    launch: q_t [B,Hq,d], k_t/v_t [B,Hkv,d] (bf16) -> o_t [B,Hq,d].  A
    caller-provided workspace must have been zero-filled before its first
    use with this cache."""
    torch = _torch()
    if o_t is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        o_t = _new(q_t, tuple(q_t.shape), dt, stream)
    od = _odtype(o_t.dtype)
    if workspace is None:
        workspace = _cache_workspace(cache, q_t, stream)
    _check(lib().cca_decode_step(
        ctypes.byref(cache.struct), _dev(q_t, "q_t"), _dev(k_t, "k_t"), _dev(v_t, "v_t"),
        _dev(o_t, "o_t", o_t.dtype), od, *_workspace(workspace), _stream(stream)),
        "cca_decode_step")
    return o_t


def _lens(lens):
    torch = _torch()
    if not (isinstance(lens, torch.Tensor) and lens.is_cuda and lens.dtype == torch.int64
            and lens.is_contiguous()):
        raise ValueError("lens must be a contiguous int64 CUDA tensor of B entries")
    return ctypes.c_void_p(lens.data_ptr())


def cca_cache_append_rows(cache: Cache, lens, q_t, k_t, v_t, stream=None) -> None:
    """Append one token per row, row b at position lens[b]; lens (int64,
    CUDA, [B]) is advanced on the device.  cache.len is not used."""
    if lens.numel() != cache.B:
        raise ValueError("lens needs one entry per batch row")
    _check(lib().cca_cache_append_rows(ctypes.byref(cache.struct), _lens(lens),
                                       _dev(q_t, "q_t"), _dev(k_t, "k_t"), _dev(v_t, "v_t"),
                                       _stream(stream)), "cca_cache_append_rows")


def cca_attn_decode_rows(cache: Cache, lens, q_t, o_t=None, out_dtype=None,
                         workspace=None, stream=None):
    """Attention of token lens[b] - 1 of every row b (lens: int64, CUDA, [B]):
    q_t [B,Hq,d] -> o_t [B,Hq,d].  Capturable in a CUDA graph."""
    torch = _torch()
    if lens.numel() != cache.B:
        raise ValueError("lens needs one entry per batch row")
    if o_t is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        o_t = _new(q_t, tuple(q_t.shape), dt, stream)
    od = _odtype(o_t.dtype)
    if workspace is None:
        workspace = _cache_workspace(cache, q_t, stream)
    _check(lib().cca_attn_decode_rows(
        ctypes.byref(cache.struct), _lens(lens), _dev(q_t, "q_t"),
        _dev(o_t, "o_t", o_t.dtype), od, *_workspace(workspace), _stream(stream)),
        "cca_attn_decode_rows")
    return o_t


def cca_attn_decode_noalloc(cache: Cache, q_t, o_t=None, out_dtype=None, stream=None):
    """As cca_attn_decode, with the library's fixed device scratch in place
    of a workspace (for callers that cannot allocate device memory)."""
    torch = _torch()
    if o_t is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        o_t = _new(q_t, tuple(q_t.shape), dt, stream)
    od = _odtype(o_t.dtype)
    _check(lib().cca_attn_decode_noalloc(
        ctypes.byref(cache.struct), _dev(q_t, "q_t"), _dev(o_t, "o_t", o_t.dtype), od,
        _stream(stream)), "cca_attn_decode_noalloc")
    return o_t


# ---- packed prompts: sequences of different lengths without padding

def _device(t, name: str) -> int:
    """The device of a call's first tensor, which has to be the current one
    (the library launches on that)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _torch().cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return dev


def _here(t, name: str, dev: int) -> int:
    """Pointer of a tensor on the call's device."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor of device {dev}, is on {t.device}")
    return t.data_ptr()


def _raw_stream(stream, dev: int) -> int:
    """The stream's handle; None: the current one (in a call of a few
    microseconds, cheaper than a Stream object)."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _tensor(t, name: str, shape, dtype, dev: int) -> int:
    """Pointer of a contiguous tensor of this shape on the current device."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return _here(t, name, dev)


def _rows(t, name: str, shape, dtype, dev: int):
    """A [heads, total, d] tensor of any row and head strides as the
    library's packed tensor."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    head, row, one = t.stride()
    if one != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return _RowsStruct(_here(t, name, dev), row, head)


def _offsets(cu, dev: int) -> int:
    if cu.dtype != _torch().int32 or cu.dim() != 1 or cu.shape[0] < 2 or not cu.is_contiguous():
        raise ValueError("cu must be a contiguous int32 tensor of S + 1 offsets")
    return _here(cu, "cu", dev)


def _packed_shapes(Q, K):
    if Q.dim() != 3 or K.dim() != 3:
        raise ValueError("Q, K and V must be [heads, total, d]")
    Hq, total, d = Q.shape
    return Hq, K.shape[0], total, d


def cca_pool_packed(Q, K, V, cu, g: int, Kc=None, Vc=None, stream=None):
    """cca_pool for packed prompts: Q [Hq,total,d], K/V [Hkv,total,d] (bf16,
    rows of any stride: views of [total,heads,d] included), sequence s in
    rows cu[s] .. cu[s + 1] - 1 (cu: int32, CUDA, [S + 1]).

    Returns (Kc, Vc) [Hkv, total // g, d] fp16; the groups of sequence s
    start at row cu[s] // g, rows without a group are zero.
    """
    torch = _torch()
    bf, dev = torch.bfloat16, _device(Q, "Q")
    Hq, Hkv, total, d = _packed_shapes(Q, K)
    shape = (Hkv, total // int(g) if g > 0 else 0, d)
    if Kc is None and Vc is None:
        Kc, Vc = _new(Q, (2, *shape), torch.float16, stream).unbind(0)
    elif Kc is None or Vc is None:
        raise ValueError("give both Kc and Vc, or neither")
    _check(lib().cca_pool_packed(
        _rows(Q, "Q", (Hq, total, d), bf, dev), _rows(K, "K", (Hkv, total, d), bf, dev),
        _rows(V, "V", (Hkv, total, d), bf, dev), _offsets(cu, dev),
        _tensor(Kc, "Kc", shape, torch.float16, dev), _tensor(Vc, "Vc", shape, torch.float16, dev),
        cu.shape[0] - 1, Hq, Hkv, total, d, _int(g, "g"),
        _raw_stream(stream, dev)), "cca_pool_packed")
    return Kc, Vc


def cca_packed_workspace_bytes(S: int, total: int) -> int:
    return int(lib().cca_packed_workspace_bytes(int(S), int(total)))


def cca_attn_prefill_packed(Q, K, V, Kc, Vc, cu, g: int, w: int, O=None, out_dtype=None,
                            workspace=None, stream=None):
    """cca_attn_prefill for packed prompts (cca_pool_packed gives the
    layout, Kc and Vc).  w >= total is plain causal attention: Kc and Vc may
    then be None.  Returns O [Hq, total, d] in ``out_dtype`` (bf16 default,
    or fp32), in Q's memory order when allocated here; rows that belong to
    no sequence are not written.
    """
    torch = _torch()
    bf, dev = torch.bfloat16, _device(Q, "Q")
    Hq, Hkv, total, d = _packed_shapes(Q, K)
    S = cu.shape[0] - 1
    if O is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        if not Q.is_contiguous() and Q.stride(0) < Q.stride(1):  # [total, Hq, d] in memory
            O = _new(Q, (total, Hq, d), dt, stream).transpose(0, 1)
        else:
            O = _new(Q, (Hq, total, d), dt, stream)
    ws, nbytes = None, 0
    if workspace is not None:
        _here(workspace, "workspace", dev)
        ws, nbytes = _workspace(workspace)
    elif S > 0:
        nbytes = lib().cca_packed_workspace_bytes(S, total)
        if nbytes:
            workspace = _new(Q, nbytes, torch.uint8, stream)
            ws = workspace.data_ptr()
    core = (Hkv, total // int(g) if g > 0 else 0, d)
    _check(lib().cca_attn_prefill_packed(
        _rows(Q, "Q", (Hq, total, d), bf, dev), _rows(K, "K", (Hkv, total, d), bf, dev),
        _rows(V, "V", (Hkv, total, d), bf, dev),
        None if Kc is None else _tensor(Kc, "Kc", core, torch.float16, dev),
        None if Vc is None else _tensor(Vc, "Vc", core, torch.float16, dev), _offsets(cu, dev),
        _rows(O, "O", (Hq, total, d), O.dtype, dev), _odtype(O.dtype), S, Hq, Hkv, total, d,
        _int(g, "g"), _int(w, "w"), ws, nbytes, _raw_stream(stream, dev)),
        "cca_attn_prefill_packed")
    return O


# ---- the paged decode cache

class PagedCache:
    """A decode cache for B rows of any lengths that share their memory in
    pages of ``page`` rows: core rows (fp16) in ``core_pages`` pages, raw
    rows (bf16) in ``raw_pages`` pages, the same page numbers in every one of
    ``layers`` layers.  ``max_len``: the longest row the tables take.
    core_pages = 0 gives a cache of plain causal attention.

    ``lens`` (int64 [B]), ``core_table`` and ``raw_table`` (int32 [B, cols],
    -1: no page), ``core_ref`` and ``raw_ref`` (int32, table entries per
    page) are views of one tensor, ``tables``; ``pools`` holds k_core,
    v_core, k_raw, v_raw [layers, pages, Hkv, page, d].
    """

    def __init__(self, B: int, Hq: int, Hkv: int, d: int, g: int, w: int, page: int,
                 core_pages: int, raw_pages: int, max_len: int, layers: int = 1, device="cuda"):
        torch = _torch()
        if min(B, Hkv, d, g, page, raw_pages, max_len, layers) < 1 or core_pages < 0:
            raise ValueError("sizes of a PagedCache must be positive")
        core_cols = max(-(-(max_len // g) // page), 1) if core_pages else 0
        kh = dict(dtype=torch.float16, device=device)
        kw = dict(dtype=torch.bfloat16, device=device)
        pools = (torch.zeros((layers, core_pages, Hkv, page, d), **kh),
                 torch.zeros((layers, core_pages, Hkv, page, d), **kh),
                 torch.zeros((layers, raw_pages, Hkv, page, d), **kw),
                 torch.zeros((layers, raw_pages, Hkv, page, d), **kw))
        self._set(B, core_cols, -(-max_len // page), pools, Hq, g, w)
        for t in (self.lens, self.core_ref, self.raw_ref):
            t.zero_()
        self.core_table.fill_(-1)
        self.raw_table.fill_(-1)

    def _set(self, B, core_cols, raw_cols, pools, Hq, g, w):
        torch = _torch()
        self.pools = pools
        self.k_core, self.v_core, self.k_raw, self.v_raw = pools
        layers, core_pages, Hkv, page, d = self.k_core.shape
        raw_pages = self.k_raw.shape[1]
        device = self.k_raw.device
        n = (2 * B, B * core_cols, B * raw_cols, core_pages, raw_pages)
        self.tables = torch.empty(sum(n), dtype=torch.int32, device=device)
        parts = self.tables.split(n)
        self.lens = parts[0].view(torch.int64)
        self.core_table = parts[1].view(B, core_cols)
        self.raw_table = parts[2].view(B, raw_cols)
        self.core_ref, self.raw_ref = parts[3], parts[4]
        self.struct = _PagedStruct(
            *(t.data_ptr() for t in (*pools, self.core_table, self.raw_table, self.core_ref,
                                     self.raw_ref, self.lens)),
            layers, B, _int(Hq, "Hq"), Hkv, d, _int(g, "g"), _int(w, "w"), page, core_cols,
            raw_cols, core_pages, raw_pages)
        # zero-filled once, as the library asks for
        self.workspace = torch.zeros(max(cca_paged_workspace_bytes(self), 256),
                                     dtype=torch.uint8, device=device)
        self.workspace_at = self.workspace.data_ptr(), self.workspace.numel()
        self.q_shape, self.kv_shape = (B, int(Hq), d), (B, Hkv, d)

    @classmethod
    def from_tensors(cls, core_table, raw_table, core_ref, raw_ref, lens, k_core, v_core, k_raw,
                     v_raw, Hq: int, g: int, w: int) -> "PagedCache":
        """A cache over the given pools (kept, not copied) with a copy of the
        given tables, counts and lengths."""
        torch = _torch()
        B = lens.numel()
        for name, t, dt, shape in (
                ("core_table", core_table, torch.int32, (B, core_table.shape[-1])),
                ("raw_table", raw_table, torch.int32, (B, raw_table.shape[-1])),
                ("core_ref", core_ref, torch.int32, k_core.shape[1:2]),
                ("raw_ref", raw_ref, torch.int32, k_raw.shape[1:2]),
                ("lens", lens, torch.int64, (B,)),
                ("k_core", k_core, torch.float16, k_core.shape),
                ("v_core", v_core, torch.float16, k_core.shape),
                ("k_raw", k_raw, torch.bfloat16, k_raw.shape),
                ("v_raw", v_raw, torch.bfloat16, k_raw.shape)):
            if t.dtype != dt or t.shape != shape or not t.is_contiguous() or \
                    t.device != k_raw.device:
                raise ValueError(f"{name} must be a contiguous {dt} tensor {tuple(shape)} on "
                                 f"{k_raw.device}")
        if k_core.dim() != 5 or k_raw.dim() != 5 or k_core.shape[:1] != k_raw.shape[:1] or \
                k_core.shape[2:] != k_raw.shape[2:]:
            raise ValueError("pools must be [layers, pages, Hkv, page, d]")
        c = object.__new__(cls)
        c._set(B, core_table.shape[1], raw_table.shape[1], (k_core, v_core, k_raw, v_raw), Hq, g, w)
        for mine, given in ((c.lens, lens), (c.core_table, core_table), (c.raw_table, raw_table),
                            (c.core_ref, core_ref), (c.raw_ref, raw_ref)):
            mine.copy_(given)
        return c

    def state_dict(self) -> dict:
        """Host copy of the cache, for saving and later restoring a session."""
        st = self.struct
        return {"shape": {n: int(getattr(st, n)) for n in ("Hq", "g", "w")},
                **{n: getattr(self, n).to("cpu", copy=True) for n in self._TENSORS}}

    @classmethod
    def from_state_dict(cls, state: dict, device="cuda") -> "PagedCache":
        """A cache on ``device`` holding what ``state_dict`` saved."""
        return cls.from_tensors(*(state[n].to(device, copy=True) for n in cls._TENSORS),
                                **state["shape"])

    _TENSORS = ("core_table", "raw_table", "core_ref", "raw_ref", "lens", "k_core", "v_core",
                "k_raw", "v_raw")

    def __getattr__(self, name):
        if name in ("layers", "B", "Hq", "Hkv", "d", "g", "w", "page", "core_cols", "raw_cols",
                    "core_pages", "raw_pages"):
            return getattr(self.struct, name)
        raise AttributeError(name)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (*self.pools, self.tables))


def cca_paged_workspace_bytes(cache: PagedCache) -> int:
    return int(lib().cca_paged_workspace_bytes(ctypes.byref(cache.struct)))


def _paged_workspace(cache: PagedCache, workspace, dev: int):
    if workspace is None:  # (on the cache's device)
        return cache.workspace_at
    _here(workspace, "workspace", dev)
    return _workspace(workspace)


def cca_paged_reserve(cache: PagedCache, n, stream=None, workspace=None) -> None:
    """Lengthen rows and give them the pages of their new tokens: ``n`` is a
    number of tokens for every row that is not free, or an int64 CUDA tensor
    [B] of each row's.  Raw pages before the new window are given back.  A row
    that held tokens and is given more than one has to be filled again as a
    whole (cca_paged_fill) before anything reads it.  A row that does not fit keeps its length and pages (CCA_ERR_CAPACITY of
    cca_device_status), and cca_paged_step with the same workspace leaves it
    as it is until a later call gives it room."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    if isinstance(n, torch.Tensor):
        each, n = _tensor(n, "n", (cache.B,), torch.int64, dev), 0
    else:
        each = None
    _check(lib().cca_paged_reserve_held(cache.struct, each, _int(n, "n", 64),
                                        *_paged_workspace(cache, workspace, dev),
                                        _raw_stream(stream, dev)), "cca_paged_reserve")


def cca_paged_fill(cache: PagedCache, K, V, Kc, Vc, cu, rows, layer: int = 0,
                   stream=None) -> None:
    """Fill one layer's pages from packed prompts K/V [Hkv,total,d] with
    their core rows Kc/Vc (cca_pool_packed; None without core pages):
    sequence s becomes row rows[s] (int32, CUDA, [S]), which
    cca_paged_reserve has given the sequence's length."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    total = K.shape[1]
    S = cu.shape[0] - 1
    shape, core = (cache.Hkv, total, cache.d), (cache.Hkv, total // cache.g, cache.d)
    _check(lib().cca_paged_fill(
        cache.struct, _int(layer, "layer"), _rows(K, "K", shape, torch.bfloat16, dev),
        _rows(V, "V", shape, torch.bfloat16, dev),
        None if Kc is None else _tensor(Kc, "Kc", core, torch.float16, dev),
        None if Vc is None else _tensor(Vc, "Vc", core, torch.float16, dev), _offsets(cu, dev),
        _tensor(rows, "rows", (S,), torch.int32, dev), S, total, _raw_stream(stream, dev)),
        "cca_paged_fill")


def cca_attn_decode_paged(cache: PagedCache, q_t, layer: int = 0, o_t=None, out_dtype=None,
                          workspace=None, stream=None):
    """Attention of the newest token of every row: q_t [B,Hq,d] -> o_t
    [B,Hq,d]; free rows get zeros.  Capturable in a CUDA graph.  A workspace
    other than the cache's own (for calls at the same time) must have been
    zero-filled before its first use."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    shape = cache.q_shape
    if o_t is None:
        o_t = _new(q_t, shape, torch.bfloat16 if out_dtype is None else out_dtype, stream)
    _check(lib().cca_attn_decode_paged(
        cache.struct, _int(layer, "layer"), _tensor(q_t, "q_t", shape, torch.bfloat16, dev),
        _tensor(o_t, "o_t", shape, o_t.dtype, dev), _odtype(o_t.dtype),
        *_paged_workspace(cache, workspace, dev), _raw_stream(stream, dev)),
        "cca_attn_decode_paged")
    return o_t


def cca_paged_step(cache: PagedCache, q_t, k_t, v_t, layer: int = 0, o_t=None, out_dtype=None,
                   workspace=None, stream=None):
    """One decode step of one layer in one launch: append the newest token of
    every row (q_t [B,Hq,d], k_t/v_t [B,Hkv,d]; cca_paged_reserve(cache, 1)
    has made room for it, once for all layers) and return its attention
    output o_t [B,Hq,d].  A row that cca_paged_reserve refused stays as it is
    and gets zeros.  Capturable in a CUDA graph."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    shape, kv = cache.q_shape, cache.kv_shape
    if o_t is None:
        o_t = _new(q_t, shape, torch.bfloat16 if out_dtype is None else out_dtype, stream)
    _check(lib().cca_paged_step(
        cache.struct, _int(layer, "layer"), _tensor(q_t, "q_t", shape, torch.bfloat16, dev),
        _tensor(k_t, "k_t", kv, torch.bfloat16, dev), _tensor(v_t, "v_t", kv, torch.bfloat16, dev),
        _tensor(o_t, "o_t", shape, o_t.dtype, dev), _odtype(o_t.dtype),
        *_paged_workspace(cache, workspace, dev), _raw_stream(stream, dev)), "cca_paged_step")
    return o_t


def cca_paged_fork(cache: PagedCache, parent, workspace=None, stream=None) -> None:
    """Row b becomes what row parent[b] was (int32, CUDA, [B]; b: keeps it,
    -1: frees it), for all layers.  Full pages are shared, partly filled last
    ones copied: samples of one prompt, beams that change places, rows that
    are done.  Called between steps, before the next cca_paged_reserve."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    _check(lib().cca_paged_fork(
        cache.struct, _tensor(parent, "parent", (cache.B,), torch.int32, dev),
        *_paged_workspace(cache, workspace, dev), _raw_stream(stream, dev)), "cca_paged_fork")


def cca_paged_compact(cache: PagedCache, live=None, workspace=None, stream=None):
    """Move the pages in use to the front of their pools, for all layers.
    Returns ``live`` (int64, CUDA, [2]): pages in use of the core and of the
    raw pool."""
    torch, dev = _torch(), _device(cache.tables, "cache")
    if live is None:
        live = _new(cache.tables, 2, torch.int64, stream)
    _check(lib().cca_paged_compact(
        cache.struct, _tensor(live, "live", (2,), torch.int64, dev),
        *_paged_workspace(cache, workspace, dev), _raw_stream(stream, dev)), "cca_paged_compact")
    return live


def cca_selftest_wait_timeout(limit_us: int = 1000, stream=None) -> None:
    """Launch the failure-path self-test kernel: a bounded wait on a barrier
    that nothing completes.  cca_device_status() afterwards returns
    CCA_ERR_TIMEOUT; the context stays usable."""
    _check(lib().cca_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "cca_selftest_wait_timeout")


def cca_device_status(stream=None) -> int:
    """Synchronise the stream; return the library's device status
    (CCA_OK, CCA_ERR_TIMEOUT, CCA_ERR_RANGE or CCA_ERR_CUDA)."""
    return int(lib().cca_device_status(_stream(stream)))
