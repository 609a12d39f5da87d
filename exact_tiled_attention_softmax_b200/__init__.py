"""Python binding of the exact tiled masked softmax attention library.

Thin ctypes marshalling over the C ABI declared in include/attn.h: the same
entry-point names, torch tensors turned into attn_tensor views, outputs and
workspace allocated by torch on the current device, launches on torch's
current stream. All arithmetic runs in the CUDA library; there is no CPU
path. A missing or unloadable libattn.so raises immediately.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

__all__ = [
    "AllowedSet", "AttentionFunction", "AttnError", "PagedCache", "attention", "attn_cache_read", "attn_cache_write",
    "attn_paged_fwd", "attn_paged_workspace_size", "attn_fwd", "attn_bwd", "attn_bwd_noalloc", "attn_fwd_workspace_size",
    "attn_bwd_workspace_size", "attn_get_status", "attn_selftest_wait_timeout", "attn_set_kernel_events",
    "attn_status_string",
    "attn_version", "library_path", "load_library",
]

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_WORKSPACE = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_DEVICE = 5

ATTN_DEVERR_TOPK_INDEX = 0x1
ATTN_DEVERR_OVERFLOW = 0x2
ATTN_DEVERR_TIMEOUT = 0x4
ATTN_DEVERR_TOPK_CAUSAL = 0x8
ATTN_DEVERR_PAGE = 0x10
ATTN_DEVERR_RAGGED = 0x20

ATTN_F32 = 0
ATTN_BF16 = 1
ATTN_F16 = 2
ATTN_E4M3 = 3  # paged caches only

ATTN_MASK_CAUSAL = 0x1
ATTN_MASK_WINDOW = 0x2
ATTN_MASK_BLOCK = 0x4
ATTN_MASK_TOPK = 0x8
ATTN_MASK_LENGTHS = 0x10
ATTN_MASK_STARTS = 0x20
ATTN_MASK_TOPK_CHECK_CAUSAL = 0x40
ATTN_MASK_FIRST = 0x80
ATTN_LSE_KV_ONLY = 0x1
ATTN_LSE_NEG_LOG2 = 0x2
ATTN_BWD_DETERMINISTIC = 0x1

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "libattn.so")


class AttnTensorC(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class AttnMaskC(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("window_left", ctypes.c_int64),
                ("block_mask", ctypes.c_void_p), ("block_q", ctypes.c_int32),
                ("block_k", ctypes.c_int32), ("bm_stride_b", ctypes.c_int64),
                ("bm_stride_h", ctypes.c_int64), ("bm_stride_q", ctypes.c_int64),
                ("topk_idxs", ctypes.c_void_p), ("topk_stride", ctypes.c_int64),
                ("topk_max", ctypes.c_int32), ("topk_length", ctypes.c_void_p),
                ("sink", ctypes.c_void_p), ("dropout_p", ctypes.c_float),
                ("dropout_seed", ctypes.c_uint64), ("lengths", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("starts_stride_b", ctypes.c_int64),
                ("lse_format", ctypes.c_uint32), ("bwd_flags", ctypes.c_uint32),
                ("window_first", ctypes.c_int64)]


class AttnCacheC(ctypes.Structure):
    _fields_ = [("k", AttnTensorC), ("v", AttnTensorC), ("k_scale", AttnTensorC), ("v_scale", AttnTensorC),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("batch", ctypes.c_int32), ("seq_lens", ctypes.c_void_p)]


_LIB = None


def load_library():
    """Load libattn.so once; raise if it is absent (no fallback exists)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run python -m exact_tiled_attention_softmax_b200.build)")
    lib = ctypes.CDLL(path)
    M, vp, sz = ctypes.POINTER(AttnMaskC), ctypes.c_void_p, ctypes.c_size_t
    T = C = vp  # attn_tensor and attn_cache descriptors: packed bytes, or a structure by reference
    lib.attn_version.restype = ctypes.c_int
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_status_string.argtypes = [ctypes.c_int]
    lib.attn_fwd_workspace_size.restype = sz
    lib.attn_fwd_workspace_size.argtypes = [T, T, T, M]
    lib.attn_bwd_workspace_size.restype = sz
    lib.attn_bwd_workspace_size.argtypes = [T, T, T, M]
    lib.attn_fwd.restype = ctypes.c_int
    lib.attn_fwd.argtypes = [T, T, T, M, ctypes.c_float, T, T, vp, sz, vp]
    lib.attn_bwd.restype = ctypes.c_int
    lib.attn_bwd.argtypes = [T, T, T, T, T, T, M, ctypes.c_float, T, T, T, vp, vp, sz, vp]
    lib.attn_bwd_noalloc.restype = ctypes.c_int
    lib.attn_bwd_noalloc.argtypes = [T, T, T, T, T, T, M, ctypes.c_float, T, T, T, vp, vp]
    lib.attn_cache_write.restype = ctypes.c_int
    lib.attn_cache_write.argtypes = [T, T, vp, C, vp, sz, vp]
    lib.attn_cache_read.restype = ctypes.c_int
    lib.attn_cache_read.argtypes = [C, T, T, vp, sz, vp]
    lib.attn_paged_workspace_size.restype = sz
    lib.attn_paged_workspace_size.argtypes = [T, C, M]
    lib.attn_paged_fwd.restype = ctypes.c_int
    lib.attn_paged_fwd.argtypes = [T, vp, C, M, ctypes.c_float, ctypes.c_int32, T, T, vp, sz, vp]
    lib.attn_get_status.restype = ctypes.c_int
    lib.attn_get_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.attn_selftest_wait_timeout.restype = ctypes.c_int
    lib.attn_selftest_wait_timeout.argtypes = [vp, sz, vp]
    lib.attn_set_kernel_events.restype = ctypes.c_int
    lib.attn_set_kernel_events.argtypes = [vp, vp]
    _LIB = lib
    return lib


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {attn_status_string(code)} (status {code})")
        self.code = code


def attn_status_string(code: int) -> str:
    return load_library().attn_status_string(int(code)).decode()


def attn_version() -> int:
    return int(load_library().attn_version())


_DTYPES = {torch.float32: ATTN_F32, torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16,
           torch.float8_e4m3fn: ATTN_E4M3}


# attn_tensor and attn_cache as packed bytes: filling a ctypes structure field
# by field costs several microseconds a tensor, more than a small kernel runs.
_TENSOR = struct.Struct("@Pii4q4q")
_CACHE = struct.Struct("@" + 4 * "Pii4q4q" + "PqiiP")
assert _TENSOR.size == ctypes.sizeof(AttnTensorC) and _CACHE.size == ctypes.sizeof(AttnCacheC)
_PAD = tuple((0,) * (4 - n) for n in range(5))
_NO_TENSOR = (0,) * 11


def _fields(t: torch.Tensor) -> tuple:
    """attn_tensor's fields for t, in order."""
    n = t.dim()
    if n > 4:
        raise ValueError("at most 4 dimensions")
    pad = _PAD[n]
    return (t.data_ptr() if t.numel() else 0, _DTYPES.get(t.dtype, -1), n, *t.shape, *pad, *t.stride(), *pad)


def _packed(t: torch.Tensor | None) -> bytes | None:
    """The attn_tensor of t (NULL for None)."""
    return None if t is None else _TENSOR.pack(*_fields(t))


def _check_on(device: torch.device, *tensors) -> None:
    """Every tensor a kernel reads or writes must sit on `device`, a CUDA
    device: the library receives raw pointers and cannot tell a host
    pointer, or another GPU's, from its own."""
    if device.type != "cuda":
        raise ValueError(f"attention tensors must be CUDA tensors (got {device})")
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, the query on {device}")


_INT32, _ONE_DIM, _TWO_DIMS = (torch.int32,), (1,), (2,)


def _check_mask_tensor(t: torch.Tensor, name: str, dtypes, dims) -> None:
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.dim() not in dims:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {' or '.join(map(str, dims))}")
    if not t.is_contiguous() and t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the innermost dimension must be contiguous")


@dataclass
class AllowedSet:
    """The allowed-set descriptor (attn_mask). Tensors must live on the GPU.

    block_mask: uint8 [nq_blocks, nk_blocks], or with leading [B, H] dims
    (size-1 dims broadcast). topk_idxs int32 [Tq, >= topk_max],
    topk_length int32 [Tq], sink float32 [Hq] (a shorter one is refused). lengths int32 [B] (active
    cells per batch row, Tq == Tk); starts int32 [B, Tq] or [Tq] (lowest
    allowed key of each query row, e.g. its packed segment's first cell).
    lse_kv_only / lse_neg_log2 select the LSE format that attn_fwd writes
    and attn_bwd expects: the sink left out, and/or stored as -log2 Z.
    deterministic makes every gradient of attn_bwd bitwise reproducible.
    window_first keeps the first keys visible outside the window (needs
    window_left; not with starts).
    topk_check_causal turns on the debug check of the top-k lists against
    each token's causal position (ATTN_DEVERR_TOPK_CAUSAL in the status).
    """
    causal: bool = False
    window_left: int = 0
    block_mask: torch.Tensor | None = None
    block_q: int = 128
    block_k: int = 128
    topk_idxs: torch.Tensor | None = None
    topk_length: torch.Tensor | None = None
    topk_max: int | None = None
    sink: torch.Tensor | None = None
    dropout_p: float = 0.0
    dropout_seed: int = 0
    lengths: torch.Tensor | None = None
    starts: torch.Tensor | None = None
    lse_kv_only: bool = False
    lse_neg_log2: bool = False
    deterministic: bool = False
    topk_check_causal: bool = False
    window_first: int = 0

    def tensors(self) -> list:
        """The device tensors the descriptor points at."""
        return [t for t in (self.block_mask, self.topk_idxs, self.topk_length, self.sink, self.lengths,
                            self.starts) if t is not None]

    def to_c(self) -> AttnMaskC:
        """The C descriptor. Checks each tensor's dtype and rank first, since
        the library sees only its pointer and strides."""
        for t, name, dtypes, dims in (
                (self.block_mask, "block_mask", (torch.uint8, torch.bool), (2, 4)),
                (self.topk_idxs, "topk_idxs", (torch.int32,), (2,)),
                (self.topk_length, "topk_length", (torch.int32,), (1,)),
                (self.sink, "sink", (torch.float32,), (1,)),
                (self.lengths, "lengths", (torch.int32,), (1,)),
                (self.starts, "starts", (torch.int32,), (1, 2))):
            if t is not None:
                _check_mask_tensor(t, name, dtypes, dims)
        m = AttnMaskC()
        flags = 0
        if self.causal:
            flags |= ATTN_MASK_CAUSAL
        if self.window_left:
            flags |= ATTN_MASK_WINDOW
            m.window_left = int(self.window_left)
        if self.window_first:
            flags |= ATTN_MASK_FIRST
            m.window_first = int(self.window_first)
        if self.block_mask is not None:
            bm = self.block_mask
            flags |= ATTN_MASK_BLOCK
            m.block_mask = bm.data_ptr()
            m.block_q, m.block_k = int(self.block_q), int(self.block_k)
            if bm.dim() == 2:
                m.bm_stride_b = m.bm_stride_h = 0
                m.bm_stride_q = bm.stride(0)
            else:
                m.bm_stride_b = bm.stride(0) if bm.shape[0] > 1 else 0
                m.bm_stride_h = bm.stride(1) if bm.shape[1] > 1 else 0
                m.bm_stride_q = bm.stride(2)
        if self.topk_idxs is not None:
            flags |= ATTN_MASK_TOPK
            m.topk_idxs = self.topk_idxs.data_ptr()
            m.topk_stride = self.topk_idxs.stride(0)
            m.topk_max = int(self.topk_max if self.topk_max is not None else self.topk_idxs.shape[1])
            m.topk_length = self.topk_length.data_ptr() if self.topk_length is not None else 0
            if self.topk_check_causal:
                flags |= ATTN_MASK_TOPK_CHECK_CAUSAL
        if self.lengths is not None:
            flags |= ATTN_MASK_LENGTHS
            m.lengths = self.lengths.data_ptr()
        if self.starts is not None:
            st = self.starts
            if st.stride(-1) != 1:
                raise ValueError("starts rows must be contiguous")
            flags |= ATTN_MASK_STARTS
            m.starts = st.data_ptr()
            m.starts_stride_b = st.stride(0) if st.dim() == 2 and st.shape[0] > 1 else 0
        if self.sink is not None:
            m.sink = self.sink.data_ptr()
        if self.lse_kv_only or self.lse_neg_log2:
            m.lse_format = (ATTN_LSE_KV_ONLY if self.lse_kv_only else 0) | \
                (ATTN_LSE_NEG_LOG2 if self.lse_neg_log2 else 0)
        if self.deterministic:
            m.bwd_flags = ATTN_BWD_DETERMINISTIC
        if self.dropout_p or self.dropout_seed:
            m.dropout_p = float(self.dropout_p)
            m.dropout_seed = int(self.dropout_seed) & 0xFFFFFFFFFFFFFFFF
        m.flags = flags
        return m


def _stream_handle(stream) -> int:
    if stream is None:  # torch's current stream of the current device, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _workspace(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned: the caching allocator hands out 512-byte aligned blocks.
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _on_stream(stream, make):
    """make()'s new tensors (a tuple) for a call on `stream` (None: the current
    one). They are allocated, and filled, on that stream, so that neither a
    fill nor an earlier use of their memory is still at work when the call's
    kernels run, and recorded for the current stream, on which the caller may
    go on with them (and drop them)."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        made = make()
    if here != stream:
        for t in made:
            t.record_stream(here)
    return made


def _is_topk(allowed: AllowedSet | None) -> bool:
    return allowed is not None and allowed.topk_idxs is not None


def _mask_of(allowed: AllowedSet | None, q, dsink=None) -> AttnMaskC | None:
    """The descriptor of a call on q, whose second dimension is its heads: the
    kernels read a sink logit, and write a sink gradient, for each of them."""
    for t, name in ((dsink, "dsink"), (allowed.sink if allowed else None, "sink")):
        if t is not None and q.dim() > 1 and t.numel() < q.shape[1]:
            raise ValueError(f"{name}: {t.numel()} entries for {q.shape[1]} query heads")
    return allowed.to_c() if allowed else None


def attn_fwd_workspace_size(q, k, v, allowed: AllowedSet | None = None) -> int:
    cq, ck, cv = _packed(q), _packed(k), _packed(v)
    m = allowed.to_c() if allowed else None
    return int(load_library().attn_fwd_workspace_size(cq, ck, cv, m))


def attn_bwd_workspace_size(q, k, v, allowed: AllowedSet | None = None) -> int:
    cq, ck, cv = _packed(q), _packed(k), _packed(v)
    m = allowed.to_c() if allowed else None
    return int(load_library().attn_bwd_workspace_size(cq, ck, cv, m))


def attn_fwd(q, k, v, allowed: AllowedSet | None = None, scale: float | None = None, *,
             out=None, lse=None, workspace=None, stream=None):
    """Forward pass. Dense: q [B,Hq,Tq,d], k [B,Hkv,Tk,d], v [B,Hkv,Tk,dv];
    with Tq != Tk query row i sits at key position i + Tk - Tq.
    Top-k: q [Tq,H,Dqk], k = KV [Tkv,Dqk], v = KV[:, :Dv].
    Returns (o, lse); lse is fp32, natural log, sink-inclusive."""
    lib = load_library()
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if out is None:
        out, = _on_stream(stream, lambda: (q.new_empty((*q.shape[:-1], v.shape[-1])),))
    if lse is None:
        lse, = _on_stream(stream, lambda: (q.new_empty(q.shape[:-1], dtype=torch.float32),))
    m = _mask_of(allowed, q)
    cq, ck, cv, co, cl = (_packed(x) for x in (q, k, v, out, lse))
    need = lib.attn_fwd_workspace_size(cq, ck, cv, m)
    if workspace is None:
        workspace, = _on_stream(stream, lambda: (_workspace(need, q.device),))
    _check_on(q.device, k, v, out, lse, workspace, *(allowed.tensors() if allowed else ()))
    rc = lib.attn_fwd(cq, ck, cv, m, scale, co, cl,
                      workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return out, lse


def attn_bwd(q, k, v, o, do, lse, allowed: AllowedSet | None = None, scale: float | None = None, *,
             dq=None, dk=None, dv=None, dsink=None, workspace=None, stream=None):
    """Reverse pass. Returns (dq, dk, dv, dsink). Top-k: dk is dKV [Tkv,Dqk]
    and dv is None. dsink is None unless the allowed set carries a sink."""
    lib = load_library()
    if scale is None:
        scale = q.shape[-1] ** -0.5
    topk = _is_topk(allowed)
    if dq is None:
        dq, = _on_stream(stream, lambda: (torch.empty_like(q),))
    if dk is None:
        dk, = _on_stream(stream, lambda: (torch.empty_like(k),))
    if dv is None and not topk:
        dv, = _on_stream(stream, lambda: (torch.empty_like(v),))
    if dsink is None and allowed is not None and allowed.sink is not None:
        dsink, = _on_stream(stream, lambda: (torch.empty_like(allowed.sink, dtype=torch.float32),))
    m = _mask_of(allowed, q, dsink)
    cq, ck, cv, co, cdo, cl = (_packed(x) for x in (q, k, v, o, do, lse))
    cdq, cdk, cdv = _packed(dq), _packed(dk), _packed(dv)
    need = lib.attn_bwd_workspace_size(cq, ck, cv, m)
    if workspace is None:
        workspace, = _on_stream(stream, lambda: (_workspace(need, q.device),))
    _check_on(q.device, k, v, o, do, lse, dq, dk, dv, dsink, workspace,
              *(allowed.tensors() if allowed else ()))
    rc = lib.attn_bwd(cq, ck, cv, co, cdo, cl, m,
                      scale, cdq, cdk, cdv,
                      dsink.data_ptr() if dsink is not None else None,
                      workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd")
    return dq, dk, (None if topk else dv), dsink


def attn_bwd_noalloc(q, k, v, o, do, lse, allowed: AllowedSet | None = None, scale: float | None = None, *,
                     dq, dk, dv=None, dsink=None, stream=None):
    """Reverse pass whose scratch is the library's fixed 64 MiB device array
    (for callers that cannot allocate device memory). The caller passes every
    output buffer; nothing is allocated here or in the library. Returns
    (dq, dk, dv, dsink)."""
    lib = load_library()
    if scale is None:
        scale = q.shape[-1] ** -0.5
    m = _mask_of(allowed, q, dsink)
    cq, ck, cv, co, cdo, cl = (_packed(x) for x in (q, k, v, o, do, lse))
    cdq, cdk, cdv = _packed(dq), _packed(dk), _packed(dv)
    _check_on(q.device, k, v, o, do, lse, dq, dk, dv, dsink, *(allowed.tensors() if allowed else ()))
    rc = lib.attn_bwd_noalloc(cq, ck, cv, co, cdo, cl, m,
                              scale, cdq, cdk, cdv,
                              dsink.data_ptr() if dsink is not None else None, _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_noalloc")
    return dq, dk, dv, dsink


def attn_get_status(workspace: torch.Tensor | None, stream=None) -> int:
    """Synchronise and return (then clear) the device status bits of a
    workspace, or with workspace=None those of attn_bwd_noalloc's fixed
    scratch array on the current device."""
    bits = ctypes.c_uint32(0)
    ptr = workspace.data_ptr() if workspace is not None else None
    rc = load_library().attn_get_status(ptr, _stream_handle(stream), ctypes.byref(bits))
    if rc not in (ATTN_OK, ATTN_ERR_DEVICE):
        raise AttnError(rc, "attn_get_status")
    return int(bits.value)


def attn_selftest_wait_timeout(workspace: torch.Tensor, stream=None) -> None:
    """Enqueue the failure-detection self-test: a wait that nothing completes
    runs out after its limit (2 s) and sets ATTN_DEVERR_TIMEOUT in the status
    word of `workspace` (a device tensor of at least 256 bytes); read it with
    attn_get_status."""
    rc = load_library().attn_selftest_wait_timeout(workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                                   _stream_handle(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_selftest_wait_timeout")


def attn_set_kernel_events(begin: "torch.cuda.Event | None", end: "torch.cuda.Event | None") -> None:
    """Have the next attn_fwd / attn_bwd call on this thread record `begin`
    and `end` around its main kernel (timing events created with
    enable_timing=True). Each event is recorded once here first so that its
    CUDA handle exists; None, None cancels."""
    if begin is None or end is None:
        load_library().attn_set_kernel_events(None, None)
        return
    for ev in (begin, end):
        if not ev.cuda_event:
            ev.record()
    load_library().attn_set_kernel_events(ctypes.c_void_p(begin.cuda_event), ctypes.c_void_p(end.cuda_event))


@dataclass
class PagedCache:
    """A paged K/V cache (attn_cache) on one GPU.

    k [num_pages, page_size, Hkv, d] and v [num_pages, page_size, Hkv, dv]
    (float32, bfloat16, float16 or float8_e4m3fn; any stride order, the last
    dimension contiguous), k_scale and v_scale float32 [num_pages, page_size,
    Hkv] with an e4m3 pool. block_table int32 [batch, max_pages]: the pages of
    each sequence, in order; seq_lens int32 [batch]: its cached positions, the
    tokens of the step in hand included.
    """
    k: torch.Tensor
    v: torch.Tensor
    block_table: torch.Tensor
    seq_lens: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, kv_heads: int, d: int, batch: int, max_pages: int, *,
                 dv: int | None = None, dtype=torch.bfloat16, device="cuda") -> "PagedCache":
        """An empty cache: zeroed pool (each head's rows of a page next to one
        another, the order the attention kernels read), table and lengths."""
        def pool(*inner, dtype):
            return torch.zeros(num_pages, kv_heads, page_size, *inner, dtype=dtype, device=device).transpose(1, 2)

        quant = dtype == torch.float8_e4m3fn
        return cls(pool(d, dtype=dtype), pool(d if dv is None else dv, dtype=dtype),
                   torch.zeros(batch, max_pages, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device),
                   pool(dtype=torch.float32) if quant else None, pool(dtype=torch.float32) if quant else None)

    def tensors(self) -> list:
        return [t for t in (self.k, self.v, self.block_table, self.seq_lens, self.k_scale, self.v_scale)
                if t is not None]

    def to_c(self) -> AttnCacheC:
        """The C descriptor, after the checks that raw pointers cannot carry."""
        return AttnCacheC.from_buffer_copy(self.packed())

    def packed(self) -> bytes:
        """to_c's bytes."""
        table, lens = self.block_table, self.seq_lens
        _check_mask_tensor(table, "block_table", _INT32, _TWO_DIMS)
        _check_mask_tensor(lens, "seq_lens", _INT32, _ONE_DIM)
        B, pages = table.shape
        if B != lens.shape[0]:
            raise ValueError("block_table and seq_lens hold different numbers of sequences")
        _check_on(self.k.device, self.v, table, lens, self.k_scale, self.v_scale)
        return _CACHE.pack(
            *_fields(self.k), *_fields(self.v),
            *(_NO_TENSOR if self.k_scale is None else _fields(self.k_scale)),
            *(_NO_TENSOR if self.v_scale is None else _fields(self.v_scale)),
            table.data_ptr(), table.stride(0), pages, B, lens.data_ptr())


def _cu_q_ptr(cu_q, cache: PagedCache):
    if cu_q is None:
        return None
    _check_mask_tensor(cu_q, "cu_q", _INT32, _ONE_DIM)
    if cu_q.shape[0] != cache.seq_lens.shape[0] + 1:
        raise ValueError(f"cu_q holds {cu_q.shape[0]} entries, expected one more than the sequences")
    _check_on(cache.k.device, cu_q)
    return cu_q.data_ptr()


def _on_device(device: torch.device, call, stream, *args) -> int:
    """call(*args, stream handle) with `device` current: the library launches
    on the current device, and the default stream is that device's current
    one."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return call(*args, _stream_handle(stream))
    return call(*args, _stream_handle(stream))


def _workspace_args(workspace) -> tuple:
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def attn_cache_write(k, v, cache: PagedCache, cu_q=None, *, workspace=None, stream=None) -> PagedCache:
    """Write new tokens' rows k [rows, Hkv, d], v [rows, Hkv, dv] at the ends
    of the cache's sequences (cu_q int32 [batch + 1]; None: the same number
    each), quantised when the cache is e4m3. With a workspace of at least 256
    bytes, attn_get_status reports bad pages and lengths. Returns the cache."""
    device = cache.k.device
    c, cu = cache.packed(), _cu_q_ptr(cu_q, cache)
    _check_on(device, k, v, workspace)
    rc = _on_device(device, load_library().attn_cache_write, stream, _packed(k), _packed(v), cu, c,
                    *_workspace_args(workspace))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_write")
    return cache


def attn_cache_read(cache: PagedCache, max_len: int | None = None, *, dtype=None, k=None, v=None, workspace=None,
                    stream=None):
    """Read the cache back as dense (k [batch, Hkv, T, d], v [batch, Hkv, T,
    dv]), T = max_len (default: all that the table can hold). Rows past a
    sequence's length are left as they were in k and v given by the caller and
    are zero in new ones. dtype (new tensors): default the pool's, bfloat16
    for an e4m3 pool."""
    device = cache.k.device
    if k is None or v is None:
        _, page, H, d = cache.k.shape
        given = k if k is not None else v
        T = given.shape[2] if given is not None else \
            int(max_len) if max_len is not None else cache.block_table.shape[1] * page
        if given is not None:
            dtype = given.dtype
        elif dtype is None:
            dtype = torch.bfloat16 if cache.k.dtype == torch.float8_e4m3fn else cache.k.dtype
        B = cache.seq_lens.shape[0]
        widths = ([d] if k is None else []) + ([cache.v.shape[3]] if v is None else [])
        new = _on_stream(stream, lambda: [torch.zeros(B, H, T, w, dtype=dtype, device=device) for w in widths])
        k = new[0] if k is None else k
        v = new[-1] if v is None else v
    c = cache.packed()
    _check_on(device, k, v, workspace)
    rc = _on_device(device, load_library().attn_cache_read, stream, c, _packed(k), _packed(v),
                    *_workspace_args(workspace))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_read")
    return k, v


def attn_paged_workspace_size(q, cache: PagedCache, allowed: AllowedSet | None = None) -> int:
    m = allowed.to_c() if allowed else None
    with torch.cuda.device(q.device):
        return int(load_library().attn_paged_workspace_size(_packed(q), cache.packed(), m))


def attn_paged_fwd(q, cache: PagedCache, cu_q=None, allowed: AllowedSet | None = None, scale: float | None = None, *,
                   max_q: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens q [rows, Hq, d] over a paged cache that already
    holds them: query i of a sequence's n new tokens sits at position
    seq_len - n + i. allowed: causal, window_left, window_first, sink and the
    LSE formats. max_q: the largest number of new tokens of a sequence, when
    known. It only chooses between kernels, but matters for speed: left out
    with cu_q, all rows count as one sequence's, and a batch of single tokens
    takes the kernel for long chunks (64 sequences of 8192 keys: 461 us
    instead of 325 in bf16, 667 instead of 206 in e4m3). Returns (o [rows, Hq, dv], lse
    [rows, Hq])."""
    lib, device = load_library(), q.device
    rows, heads, d = q.shape
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out, = _on_stream(stream, lambda: (q.new_empty((rows, heads, cache.v.shape[3])),))
    if lse is None:
        lse, = _on_stream(stream, lambda: (q.new_empty((rows, heads), dtype=torch.float32),))
    m = _mask_of(allowed, q)
    cq, c, cu = _packed(q), cache.packed(), _cu_q_ptr(cu_q, cache)
    _check_on(device, cache.k, out, lse, workspace, *(allowed.tensors() if allowed else ()))

    def call(s):
        ws = workspace
        if ws is None:
            need = lib.attn_paged_workspace_size(cq, c, m)
            if stream is None:
                ws = q.new_empty(need, dtype=torch.uint8)
            else:  # from that stream's pool: freed here, reused there after the call
                with torch.cuda.stream(stream):
                    ws = _workspace(need, device)
        return lib.attn_paged_fwd(cq, cu, c, m, scale, int(max_q), _packed(out), _packed(lse), *_workspace_args(ws), s)

    rc = _on_device(device, call, stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged_fwd")
    return out, lse


class AttentionFunction(torch.autograd.Function):
    """attn_fwd / attn_bwd as one autograd node. Saves Q, K, V, O and the LSE
    (never P); the reverse pass recomputes the scores tile by tile.

    Inputs: q, k, v, sink (float32 [Hq] or None, so that its gradient is
    routed), the allowed set and the scale. Outputs: O and the LSE; the LSE is
    not differentiable through this node. Top-k (shared KV): pass k = KV and
    v = KV[:, :Dv]; the whole dKV comes back as k's gradient and v's is None,
    so a KV leaf that both were sliced from receives the tied gradient once.
    """

    @staticmethod
    def forward(ctx, q, k, v, sink, allowed, scale):
        import dataclasses
        al = dataclasses.replace(allowed, sink=sink.detach() if sink is not None else None)
        o, lse = attn_fwd(q, k, v, al, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.allowed, ctx.scale, ctx.has_sink = al, scale, sink is not None
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    def backward(ctx, d_o, d_lse):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv, dsink = attn_bwd(q, k, v, o, d_o.contiguous(), lse, ctx.allowed, ctx.scale)
        return dq, dk, dv, (dsink if ctx.has_sink else None), None, None


def attention(q, k, v, allowed: AllowedSet | None = None, scale: float | None = None, sink=None):
    """Differentiable exact masked attention: returns (O, LSE). The allowed
    set's own sink field is ignored here; pass the sink tensor as `sink`."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return AttentionFunction.apply(q, k, v, sink, allowed if allowed is not None else AllowedSet(), scale)
