"""Python binding over the C ABI: turns torch CUDA tensors into the raw
pointers, sizes and stream the C calls take.  Every step of the path runs in
libsls.so kernels; this module only marshals arguments and, where asked,
allocates output tensors with torch (the C library itself allocates
nothing).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.SLS_DTYPE_F32, torch.bfloat16: L.SLS_DTYPE_BF16}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the current device's current stream, without building a torch.cuda.Stream (3 us of a call on the host)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_sink(sink, heads: int, index: int):
    """A sink for a step on device `index`."""
    _need(sink, "sink", torch.float32, (heads,))
    if sink.get_device() != index:
        raise ValueError("sink must be on the step's device")


def _list_width(page_idx) -> int:
    """Entries a row of optional page lists.  Lists without columns have no memory, and no pointer to one means every page."""
    if page_idx is None:
        return 0
    if page_idx.dim() != 2 or page_idx.shape[1] < 1:
        raise ValueError("page_idx must be [rows, entries] with at least one entry a row (count says how many hold), got "
                         f"{tuple(page_idx.shape)}")
    return int(page_idx.shape[1])


def make_desc(batch, num_q_heads, num_kv_heads, head_dim, page_size, capacity, dtype,
              scale: float = 0.0, cuda_cores: bool = False, no_tma: bool = False,
              test_wait_timeout: bool = False) -> L.AttnDesc:
    """Descriptor of one layer's decode shapes (the C ABI's sls_attn_desc); dtype is a torch dtype
    or an SLS_DTYPE_* code, scale 0 means 1/sqrt(head_dim).  test_wait_timeout sets the
    bounded-wait test hook (SLS_FLAG_TEST_WAIT_TIMEOUT; tests only)."""
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    flags = ((L.SLS_FLAG_CUDA_CORES if cuda_cores else 0) | (L.SLS_FLAG_NO_TMA if no_tma else 0)
             | (L.SLS_FLAG_TEST_WAIT_TIMEOUT if test_wait_timeout else 0))
    return L.AttnDesc(batch, num_q_heads, num_kv_heads, head_dim, page_size, capacity, code,
                      flags, float(scale))


def get_stats(reset: bool = False) -> dict:
    """Counters of the paths the library took (synchronises the device)."""
    st = L.Stats()
    L.call("sls_get_stats", ctypes.byref(st), int(bool(reset)))
    return {name: int(getattr(st, name)) for name, _ in L.Stats._fields_}


def pipeline_check() -> None:
    """Synchronises the device and reads the device status words; raises
    SlsError with code SLS_ETIMEOUT if a pipelined kernel gave up waiting for
    its copies, or SLS_EDEVICE if a kernel met (and skipped) page-list entries
    that are neither a page of the pool nor -1, since the last check."""
    L.call("sls_pipeline_check")


def desc_for(k_cache: torch.Tensor, num_q_heads: int, page_size: int, scale: float = 0.0,
             cuda_cores: bool = False) -> L.AttnDesc:
    """Descriptor read off a [B, Hkv, Cap, D] key cache."""
    B, Hkv, Cap, D = k_cache.shape
    return make_desc(B, num_q_heads, Hkv, D, page_size, Cap, k_cache.dtype, scale, cuda_cores)


def default_splits(desc: L.AttnDesc, max_entries: int) -> int:
    """The library's split count: one wave of attend CTAs, >= 64 tokens each."""
    return int(L.load().sls_attend_default_splits(ctypes.byref(desc), int(max_entries)))


# ----------------------------------------------------------------- metadata

def pagemeta_build(desc: L.AttnDesc, k_cache, ctx_len, kmin=None, kmax=None):
    """Per-page min and max of the valid keys (sls_pagemeta_build); allocates
    kmin/kmax [B, Hkv, Cap/P, D] when not given.  Returns (kmin, kmax)."""
    _need(k_cache, "k_cache")
    _need(ctx_len, "ctx_len", torch.int32)
    B, Hkv, Cap, D = k_cache.shape
    shape = (B, Hkv, Cap // desc.page_size, D)
    kmin = torch.empty(shape, dtype=k_cache.dtype, device=k_cache.device) if kmin is None else kmin
    kmax = torch.empty(shape, dtype=k_cache.dtype, device=k_cache.device) if kmax is None else kmax
    _need(kmin, "kmin", k_cache.dtype, shape)
    _need(kmax, "kmax", k_cache.dtype, shape)
    L.call("sls_pagemeta_build", ctypes.byref(desc), _ptr(k_cache), _ptr(ctx_len), _ptr(kmin),
           _ptr(kmax), _stream())
    return kmin, kmax


def pagemeta_update(desc: L.AttnDesc, k_cache, pos, kmin, kmax):
    """Folds the key at pos[b] of every sequence into its page's min/max
    (sls_pagemeta_update)."""
    _need(pos, "pos", torch.int32)
    L.call("sls_pagemeta_update", ctypes.byref(desc), _ptr(k_cache), _ptr(pos), _ptr(kmin),
           _ptr(kmax), _stream())


def thumb_build(desc: L.AttnDesc, k_cache, ctx_len, block: int, codes=None, scales=None):
    """2-bit thumbnails of every complete block (sls_thumb_build); allocates
    codes [B, Hkv, Cap, D/4] u8 and scales [B, Hkv, Cap/block, D] when not given.
    Returns (codes, scales)."""
    _need(k_cache, "k_cache")
    _need(ctx_len, "ctx_len", torch.int32)
    B, Hkv, Cap, D = k_cache.shape
    if codes is None:
        codes = torch.zeros((B, Hkv, Cap, D // 4), dtype=torch.uint8, device=k_cache.device)
    if scales is None:
        scales = torch.zeros((B, Hkv, Cap // block, D), dtype=k_cache.dtype, device=k_cache.device)
    _need(codes, "codes", torch.uint8, (B, Hkv, Cap, D // 4))
    _need(scales, "scales", k_cache.dtype, (B, Hkv, Cap // block, D))
    L.call("sls_thumb_build", ctypes.byref(desc), _ptr(k_cache), _ptr(ctx_len), int(block),
           _ptr(codes), _ptr(scales), _stream())
    return codes, scales


def thumb_update(desc: L.AttnDesc, k_cache, pos, block: int, codes, scales):
    """Quantises the block that the key at pos[b] completes (sls_thumb_update)."""
    _need(pos, "pos", torch.int32)
    L.call("sls_thumb_update", ctypes.byref(desc), _ptr(k_cache), _ptr(pos), int(block),
           _ptr(codes), _ptr(scales), _stream())


def thumb_residual_build(desc: L.AttnDesc, k_cache, ctx_len, block: int, codes=None, scales=None, res=None):
    """Thumbnails plus 8-bit residuals of every complete block."""
    B, H, Cap, D = desc.batch, desc.num_kv_heads, desc.capacity, desc.head_dim
    dev = k_cache.device
    codes = torch.zeros((B, H, Cap, D // 4), dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.zeros((B, H, Cap // block, D), dtype=k_cache.dtype, device=dev) if scales is None else scales
    res = torch.zeros((B, H, Cap, D), dtype=torch.int8, device=dev) if res is None else res
    L.call("sls_thumb_residual_build", ctypes.byref(desc), _ptr(k_cache), _ptr(ctx_len), int(block), _ptr(codes),
           _ptr(scales), _ptr(res), _stream())
    return codes, scales, res


def thumb_residual_update(desc: L.AttnDesc, k_cache, pos, block: int, codes, scales, res):
    """Thumbnail and 8-bit residuals of the block that the key at pos[b]
    completes (sls_thumb_residual_update)."""
    _need(pos, "pos", torch.int32)
    L.call("sls_thumb_residual_update", ctypes.byref(desc), _ptr(k_cache), _ptr(pos), int(block), _ptr(codes),
           _ptr(scales), _ptr(res), _stream())


# ---------------------------------------------------------------- selection

def select_pages_workspace(desc: L.AttnDesc, device="cuda"):
    """Scratch buffer of select_pages (sls_select_pages_workspace_size bytes)."""
    n = L.load().sls_select_pages_workspace_size(ctypes.byref(desc))
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def select_pages(desc: L.AttnDesc, q, kmin, kmax, ctx_len, k: int, n_sink_pages: int = 0,
                 n_local_tokens: int = 0, out=None, workspace=None):
    """Quest selection (sls_select_pages): per (sequence, KV head) the k pages
    with the highest min/max bound, forced sink and local pages included,
    ascending, -1 padded.  Returns page_idx [B*Hkv, k] int32."""
    _need(q, "q")
    rows = desc.batch * desc.num_kv_heads
    out = torch.empty((rows, k), dtype=torch.int32, device=q.device) if out is None else out
    _need(out, "page_idx", torch.int32, (rows, k))
    workspace = select_pages_workspace(desc, q.device) if workspace is None else workspace
    L.call("sls_select_pages", ctypes.byref(desc), _ptr(q), _ptr(kmin), _ptr(kmax), _ptr(ctx_len),
           int(k), int(n_sink_pages), int(n_local_tokens), _ptr(out), _ptr(workspace),
           workspace.numel(), _stream())
    return out


def select_delta_workspace(desc: L.AttnDesc, block: int, device="cuda"):
    """Scratch buffer of select_delta (sls_select_delta_workspace_size bytes)."""
    n = L.load().sls_select_delta_workspace_size(ctypes.byref(desc), int(block))
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def select_delta(desc: L.AttnDesc, q, k_cache, codes, scales, ctx_len, block: int, delta: float,
                 count=None, block_idx=None, workspace=None):
    """Top-delta selection (sls_select_delta): the blocks whose thumbnail
    scores come within delta of the pseudo-max, plus the first and newest
    block.  Returns (count [B*Hkv], block_idx [B*Hkv, Cap/block])."""
    rows = desc.batch * desc.num_kv_heads
    nblk = desc.capacity // block
    count = torch.empty(rows, dtype=torch.int32, device=q.device) if count is None else count
    block_idx = torch.empty((rows, nblk), dtype=torch.int32, device=q.device) if block_idx is None else block_idx
    workspace = select_delta_workspace(desc, block, q.device) if workspace is None else workspace
    _need(block_idx, "block_idx", torch.int32)
    L.call("sls_select_delta", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(codes), _ptr(scales),
           _ptr(ctx_len), int(block), float(delta), _ptr(count), _ptr(block_idx),
           int(block_idx.shape[1]), _ptr(workspace), workspace.numel(), _stream())
    return count, block_idx


# ---------------------------------------------------------------- attention

def partials(desc: L.AttnDesc, num_splits: int, device="cuda"):
    """Split partials (o [B, Hq, S, D], m and l [B, Hq, S], fp32) for
    sparse_decode_attend and combine_splits."""
    B, Hq, D = desc.batch, desc.num_q_heads, desc.head_dim
    return (torch.empty((B, Hq, num_splits, D), dtype=torch.float32, device=device),
            torch.empty((B, Hq, num_splits), dtype=torch.float32, device=device),
            torch.empty((B, Hq, num_splits), dtype=torch.float32, device=device))


def sparse_decode_attend(desc: L.AttnDesc, q, k_cache, v_cache, page_idx, ctx_len, num_splits: int,
                         count=None, k_fixed: Optional[int] = None, parts=None):
    """page_idx [rows, stride] int32 (or None for every page); count [rows]
    int32 or None (then k_fixed, default stride, entries per row)."""
    _need(q, "q")
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache")
    o, m, l = partials(desc, num_splits, q.device) if parts is None else parts
    stride = _list_width(page_idx)
    kf = stride if k_fixed is None else int(k_fixed)
    L.call("sls_sparse_decode_attend", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
           _ptr(page_idx), stride, _ptr(count), kf, _ptr(ctx_len), int(num_splits), _ptr(o),
           _ptr(m), _ptr(l), _stream())
    return o, m, l


def attend_combine_workspace(desc: L.AttnDesc, num_splits: int, device="cuda"):
    """Zero-filled workspace of sparse_decode_attend_combine (reusable)."""
    n = L.load().sls_attend_combine_workspace_size(ctypes.byref(desc), int(num_splits))
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def sparse_decode_attend_combine(desc: L.AttnDesc, q, k_cache, v_cache, page_idx, ctx_len,
                                 num_splits: int, count=None, k_fixed: Optional[int] = None,
                                 sink=None, out=None, lse=None, workspace=None, want_lse: bool = True):
    """Attend and combine in one launch; returns (out, lse)."""
    _need(q, "q")
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache")
    B, Hq, D = desc.batch, desc.num_q_heads, desc.head_dim
    dtype = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
    out = torch.empty((B, Hq, D), dtype=dtype, device=q.device) if out is None else out
    if want_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if sink is not None:
        _need(sink, "sink", torch.float32, (Hq,))
    workspace = attend_combine_workspace(desc, num_splits, q.device) if workspace is None else workspace
    stride = _list_width(page_idx)
    kf = stride if k_fixed is None else int(k_fixed)
    L.call("sls_sparse_decode_attend_combine", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
           _ptr(page_idx), stride, _ptr(count), kf, _ptr(ctx_len), int(num_splits), _ptr(sink),
           _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream())
    return out, lse


def refined_workspace(desc: L.AttnDesc, device="cuda"):
    """Zero-filled workspace of refined_decode_attend_combine (reusable)."""
    n = L.load().sls_refined_decode_attend_workspace_size(ctypes.byref(desc))
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def refined_decode_attend_combine(desc: L.AttnDesc, q, k_cache, v_cache, codes, scales, res, block_idx, count,
                                  ctx_len, sink=None, out=None, lse=None, workspace=None, want_lse: bool = True):
    """Attention over the kept blocks of every row, the rows' lists cut into
    equal work items, combine fused; complete blocks are scored with the
    refined (2-bit + 8-bit) keys, or with the bf16 keys when codes, scales
    and res are None.  Returns (out, lse)."""
    for t, nm in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (block_idx, "block_idx"),
                  (count, "count")):
        _need(t, nm)
    B, Hq, D = desc.batch, desc.num_q_heads, desc.head_dim
    out = torch.empty((B, Hq, D), dtype=q.dtype, device=q.device) if out is None else out
    if want_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if sink is not None:
        _need(sink, "sink", torch.float32, (Hq,))
    workspace = refined_workspace(desc, q.device) if workspace is None else workspace
    L.call("sls_refined_decode_attend_combine", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
           _ptr(codes), _ptr(scales), _ptr(res), _ptr(block_idx), int(block_idx.shape[-1]), _ptr(count),
           _ptr(ctx_len), _ptr(sink), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream())
    return out, lse


def combine_splits(desc: L.AttnDesc, parts, sink=None, out=None, lse=None, want_lse: bool = True):
    """Log-sum-exp merge of the split partials with the optional sink
    (sls_combine_splits).  Returns (out [B, Hq, D], lse [B, Hq] or None)."""
    o, m, l = parts
    B, Hq, S, D = o.shape
    dtype = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
    out = torch.empty((B, Hq, D), dtype=dtype, device=o.device) if out is None else out
    if want_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=o.device)
    if sink is not None:
        _need(sink, "sink", torch.float32, (Hq,))
    L.call("sls_combine_splits", ctypes.byref(desc), _ptr(o), _ptr(m), _ptr(l), int(S), _ptr(sink),
           _ptr(out), _ptr(lse), _stream())
    return out, lse


def decode_append(desc: L.AttnDesc, k_new, v_new, k_cache, v_cache, ctx_len, kmin=None, kmax=None,
                  pos_out=None):
    """Writes one new token per sequence at ctx_len, keeps the page min/max
    current and advances ctx_len (all on the device)."""
    for t, nm in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, nm)
    L.call("sls_decode_append", ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
           _ptr(kmin), _ptr(kmax), _ptr(ctx_len), _ptr(pos_out), _stream())


def quest_step_workspace(desc: L.AttnDesc, k: int, num_splits: int = 0, device="cuda"):
    """Zero-filled workspace of quest_decode_step (reusable)."""
    n = L.load().sls_quest_decode_step_workspace_size(ctypes.byref(desc), int(k), int(num_splits))
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def quest_step_splits(desc: L.AttnDesc, k: int) -> int:
    """Cluster size of the one-launch step for this shape (0: two launches)."""
    return int(L.load().sls_quest_decode_step_splits(ctypes.byref(desc), int(k)))


def quest_decode_step(desc: L.AttnDesc, q, k_cache, v_cache, kmin, kmax, ctx_len, k: int,
                      n_sink_pages: int = 0, n_local_tokens: int = 0, sink=None, page_idx=None,
                      out=None, lse=None, num_splits: int = 0, workspace=None, want_lse: bool = True,
                      min_sparsity: float = 0.0):
    """The whole Quest step (select + attend + combine), one launch where the
    shape allows; returns (out, lse).  page_idx, if given, receives the list."""
    for t, nm in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (kmin, "kmin"), (kmax, "kmax")):
        _need(t, nm)
    B, Hq, D = desc.batch, desc.num_q_heads, desc.head_dim
    dtype = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
    out = torch.empty((B, Hq, D), dtype=dtype, device=q.device) if out is None else out
    if want_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if sink is not None:
        _need(sink, "sink", torch.float32, (Hq,))
    if page_idx is not None:
        _need(page_idx, "page_idx", torch.int32, (desc.batch * desc.num_kv_heads, int(k)))
    workspace = quest_step_workspace(desc, k, num_splits, q.device) if workspace is None else workspace
    L.call("sls_quest_decode_step", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kmin),
           _ptr(kmax), _ptr(ctx_len), int(k), int(n_sink_pages), int(n_local_tokens), _ptr(sink),
           _ptr(page_idx), _ptr(out), _ptr(lse), int(num_splits), float(min_sparsity), _ptr(workspace),
           workspace.numel(), _stream())
    return out, lse


def selection_recall(desc: L.AttnDesc, q, k_cache, page_idx, ctx_len, count=None,
                     k_fixed: Optional[int] = None, recall=None, workspace=None):
    """Attention-mass recall of each query head's page list: [B, Hq] float32."""
    _need(q, "q")
    _need(k_cache, "k_cache")
    recall = torch.empty((desc.batch, desc.num_q_heads), dtype=torch.float32, device=q.device) \
        if recall is None else recall
    n = L.load().sls_selection_recall_workspace_size(ctypes.byref(desc))
    workspace = torch.empty(max(int(n), 1), dtype=torch.uint8, device=q.device) if workspace is None else workspace
    stride = _list_width(page_idx)
    kf = stride if k_fixed is None else int(k_fixed)
    L.call("sls_selection_recall", ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(page_idx), stride, _ptr(count),
           kf, _ptr(ctx_len), _ptr(recall), _ptr(workspace), workspace.numel(), _stream())
    return recall


# ------------------------------------------------- per-head norm and rotation

_fast = None


def _binding():
    """The tensor binding of the calls below (csrc/binding.cpp), bound to the loaded library."""
    global _fast
    if _fast is None:
        L.load()
        try:
            from . import _binding as fast
        except ImportError as e:
            raise RuntimeError("the tensor binding of the norm/rotation, 8-bit and paged cache calls is missing or does not load: "
                               f"build it first (python -m sparse_long_context_gb300.build): {e}") from e
        fast.bind(L.LIB_PATH)
        _fast = fast
    return _fast


def make_rope(num_q_heads: int, num_kv_heads: int, head_dim: int, dtype, rotary_dim: Optional[int] = None,
              theta: float = 10000.0, interleaved: bool = False, eps: float = 1e-6, inv_freq=None) -> L.RopeDesc:
    """Descriptor of qk_norm_rope (sls_rope_desc).  rotary_dim defaults to head_dim; inv_freq, if given, holds the
    rotary_dim / 2 frequencies in radians per position (any host sequence of numbers)."""
    rotary_dim = head_dim if rotary_dim is None else int(rotary_dim)
    freq = None
    if inv_freq is not None:
        values = [float(f) for f in inv_freq]
        if len(values) != rotary_dim // 2:
            raise ValueError(f"inv_freq must hold rotary_dim / 2 = {rotary_dim // 2} values, got {len(values)}")
        freq = (ctypes.c_double * max(len(values), 1))(*values)
    rope = L.RopeDesc(int(num_q_heads), int(num_kv_heads), int(head_dim), rotary_dim, int(bool(interleaved)),
                      _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype), float(eps), float(theta), freq)
    rope.keep_alive = freq
    return rope


def qk_norm_rope(rope: L.RopeDesc, q, k, positions, q_weight=None, k_weight=None, q_out=None, k_out=None):
    """Per-head RMS norm (where a weight is given) and rotation by the token's position (sls_qk_norm_rope).
    q [N, Hq, D] and k [N, Hkv, D] may be strided views of one projection's output; positions [N] int32, negative
    ones skipped.  The outputs default to new contiguous tensors and may be q and k themselves.  A side with no
    heads is passed as None.  Returns (q_out, k_out)."""
    if rope.num_q_heads and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if rope.num_kv_heads and k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    status = (_fast or _binding()).qk_norm_rope(rope, q, k, positions, q_weight, k_weight, q_out, k_out)
    if status:
        L.check("sls_qk_norm_rope", status)
    return q_out if rope.num_q_heads else None, k_out if rope.num_kv_heads else None


# -------------------------------------------------------------- 8-bit KV cache

_KV8_FORMATS = {"int8": L.SLS_KV8_INT8, "e4m3": L.SLS_KV8_E4M3}


class Kv8Cache:
    """A K/V cache in 8 bits with one scale per block of tokens and KV head (sls_kv8_cache): codes
    [B, Hkv, Cap, D] uint8, scales [B, Hkv, Cap/block] fp32, and the bf16 tail buffers [B, Hkv, block, D] in which
    the tokens of the newest, partial block wait.  fmt is "int8" or "e4m3"."""

    def __init__(self, desc: L.AttnDesc, fmt: str, block: int, k_codes, v_codes, k_scales, v_scales, k_tail, v_tail):
        B, H, Cap, D = desc.batch, desc.num_kv_heads, desc.capacity, desc.head_dim
        block = int(block)
        if fmt not in _KV8_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(_KV8_FORMATS)}, got {fmt!r}")
        if block < 1 or Cap % block:
            raise ValueError(f"block {block} must divide the capacity {Cap}")
        for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _need(t, name, torch.uint8, (B, H, Cap, D))
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _need(t, name, torch.float32, (B, H, Cap // block))
        for t, name in ((k_tail, "k_tail"), (v_tail, "v_tail")):
            _need(t, name, torch.bfloat16, (B, H, block, D))
        self.index = k_codes.get_device()
        if any(t.get_device() != self.index for t in (v_codes, k_scales, v_scales, k_tail, v_tail)):
            raise ValueError("the cache's tensors must be on one device")
        self.fmt, self.block, self.shape = fmt, block, (B, H, Cap, D)
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.k_tail, self.v_tail = k_tail, v_tail
        self.c = L.Kv8CacheDesc(_KV8_FORMATS[fmt], block, *(t.data_ptr() for t in (
            k_codes, v_codes, k_scales, v_scales, k_tail, v_tail)))

    @classmethod
    def empty(cls, desc: L.AttnDesc, fmt: str = "int8", block: int = 64, device="cuda") -> "Kv8Cache":
        """A new cache of the descriptor's shape (zero-filled)."""
        B, H, Cap, D = desc.batch, desc.num_kv_heads, desc.capacity, desc.head_dim
        new = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        return cls(desc, fmt, block, new((B, H, Cap, D), torch.uint8), new((B, H, Cap, D), torch.uint8),
                   new((B, H, Cap // block), torch.float32), new((B, H, Cap // block), torch.float32),
                   new((B, H, block, D), torch.bfloat16), new((B, H, block, D), torch.bfloat16))

    def _beside(self, t: torch.Tensor, desc: L.AttnDesc) -> L.Kv8CacheDesc:
        """The C structure, for a call with this descriptor on t's device."""
        if t.get_device() != self.index:
            raise ValueError("the cache must be on the device of the other tensors")
        if (desc.batch, desc.num_kv_heads, desc.capacity, desc.head_dim) != self.shape:
            raise ValueError(f"the descriptor's shape is not that of the cache, {self.shape}")
        return self.c

    def values(self):
        """The complete blocks' K and V as fp32 [B, H, Cap, D] (codes times scales; for inspection)."""
        dt = torch.int8 if self.fmt == "int8" else torch.float8_e4m3fn
        def one(codes, scales):
            B, H, Cap, D = codes.shape
            x = codes.view(dt).float().view(B, H, Cap // self.block, self.block, D)
            return (x * scales[..., None, None]).view(B, H, Cap, D)
        return one(self.k_codes, self.k_scales), one(self.v_codes, self.v_scales)


def kv8_append(desc: L.AttnDesc, cache: Kv8Cache, k_new, v_new, ctx_len, new_len=None, kmin=None, kmax=None,
               mass=None, ctx_out=None, pos_out=None):
    """Appends the first new_len[b] (None: all) tokens of k_new, v_new [B, T, Hkv, D] to every sequence
    (sls_kv8_append): complete blocks are quantised, the rest waits in the tail.  ctx_out defaults to ctx_len
    (advanced in place).  The new tensors may be strided views with contiguous channels."""
    status = (_fast or _binding()).kv8_append(desc, cache._beside(k_new, desc), k_new, v_new, ctx_len, new_len, kmin, kmax,
                                              mass, ctx_out, pos_out)
    if status:
        L.check("sls_kv8_append", status)
    return ctx_len if ctx_out is None else ctx_out


def kv8_attend_workspace(desc: L.AttnDesc, cache: Kv8Cache, mass: bool = False, device="cuda"):
    """Zero-filled workspace of kv8_decode_attend (reusable, also by calls of other shapes that need no more bytes, one
    after the other); mass: for calls that sum the blocks' weights."""
    n = L.load().sls_kv8_decode_attend_workspace_size(ctypes.byref(desc), ctypes.byref(cache.c), int(bool(mass)))
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def kv8_decode_attend(desc: L.AttnDesc, cache: Kv8Cache, q, ctx_len, page_idx=None, count=None,
                      k_fixed: Optional[int] = None, sink=None, mass_in=None, mass_out=None, out=None, lse=None,
                      workspace=None, want_lse: bool = True):
    """Decode attention over an 8-bit cache (sls_kv8_decode_attend): dense, or over page lists [rows, stride].
    mass_out, if given, receives every complete block's summed softmax weight added to mass_in.  Returns
    (out, lse)."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = kv8_attend_workspace(desc, cache, mass_out is not None, q.device)
    status = (_fast or _binding()).kv8_decode_attend(desc, cache._beside(q, desc), q, ctx_len, page_idx, count, k_fixed, sink,
                                                     mass_in, mass_out, out, lse, workspace)
    if status:
        L.check("sls_kv8_decode_attend", status)
    return out, lse


def kv8_evict(desc: L.AttnDesc, cache: Kv8Cache, ctx_len, mass, keep: int, n_sink_blocks: int = 0,
              n_recent_blocks: int = 0, dst_desc: Optional[L.AttnDesc] = None, dst: Optional[Kv8Cache] = None,
              ctx_out=None, mass_out=None, kept_idx=None, kmin=None, kmax=None, kmin_out=None, kmax_out=None):
    """Keeps at most `keep` complete blocks of every row by accumulated attention weight (sls_kv8_evict), in place
    (dst None) or into another cache of dst_desc's capacity.  The outputs default to the inputs' buffers in place,
    and ctx_out to ctx_len in place only.  Returns (ctx_out, kept_idx)."""
    if (dst is None) != (dst_desc is None):
        raise ValueError("dst and dst_desc: both or neither")
    if dst is None:
        dcap, to = desc.capacity, None
        mass_out = mass if mass_out is None else mass_out
        kmin_out = kmin if kmin_out is None else kmin_out
        kmax_out = kmax if kmax_out is None else kmax_out
        ctx_out = ctx_len if ctx_out is None else ctx_out
    else:
        dcap, to = dst_desc.capacity, dst._beside(ctx_len, dst_desc)
        if (dst_desc.batch, dst_desc.num_kv_heads, dst_desc.head_dim, dst_desc.page_size, dst_desc.dtype) != (
                desc.batch, desc.num_kv_heads, desc.head_dim, desc.page_size, desc.dtype):
            raise ValueError("dst_desc must describe the same rows and pages as desc")
        if ctx_out is None:
            ctx_out = torch.empty_like(ctx_len)
    if kept_idx is None:
        kept_idx = torch.empty((desc.batch * desc.num_kv_heads, max(int(keep), 0)), dtype=torch.int32,
                               device=ctx_len.device)
    status = (_fast or _binding()).kv8_evict(desc, cache._beside(ctx_len, desc), dcap, to, keep, n_sink_blocks,
                                             n_recent_blocks, mass, mass_out, kmin, kmax, kmin_out, kmax_out, kept_idx,
                                             ctx_len, ctx_out)
    if status:
        L.check("sls_kv8_evict", status)
    return ctx_out, kept_idx


# ------------------------------------------------------------- paged KV cache

class PagedCache:
    """A K/V cache whose pages lie in a pool and may be shared (sls_paged_cache): k_pages, v_pages [N, Hkv, P, D], and
    optionally the pages' key summaries kmin, kmax [N, Hkv, D].  The lengths ctx_len [B], the table [B, Cap/P] and the
    counts refs [N] are views of one int32 tensor, meta, which also holds the free pages: a copy of meta is a copy of
    what the cache's sequences are.  A new cache holds no token."""

    def __init__(self, desc: L.AttnDesc, k_pages, v_pages, kmin=None, kmax=None):
        B, H, D, P = desc.batch, desc.num_kv_heads, desc.head_dim, desc.page_size
        dt = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
        N = int(k_pages.shape[0])
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            _need(t, name, dt, (N, H, P, D))
        if (kmin is None) != (kmax is None):
            raise ValueError("kmin and kmax: both or neither")
        for t, name in ((kmin, "kmin"), (kmax, "kmax")):
            if t is not None:
                _need(t, name, dt, (N, H, D))
        self.index = k_pages.get_device()
        if any(t is not None and t.get_device() != self.index for t in (v_pages, kmin, kmax)):
            raise ValueError("the cache's tensors must be on one device")
        words = int(L.load().sls_paged_state_words(ctypes.byref(desc), N))
        if not words:
            raise ValueError(f"no paged cache of this descriptor and {N} pages: " + L.load().sls_last_error().decode())
        mp, up = desc.capacity // P, lambda n: -(-n // 4) * 4  # the parts of meta start at 16 bytes
        at = [0, up(B), up(B) + up(B * mp), up(B) + up(B * mp) + up(N)]
        self.meta = torch.zeros(at[3] + words, dtype=torch.int32, device=k_pages.device)
        self.ctx_len, self.table = self.meta[:B], self.meta[at[1]:at[1] + B * mp].view(B, mp)
        self.refs, state = self.meta[at[2]:at[2] + N], self.meta[at[3]:]
        self.shape = (B, H, desc.capacity, D, P, desc.dtype)
        self.num_pages, self.k_pages, self.v_pages, self.kmin, self.kmax = N, k_pages, v_pages, kmin, kmax
        self.c = L.PagedCacheDesc(N, *(None if t is None else t.data_ptr() for t in (
            k_pages, v_pages, kmin, kmax, self.ctx_len, self.table, self.refs, state)))
        paged_init(desc, self)

    @classmethod
    def empty(cls, desc: L.AttnDesc, num_pages: int, summaries: bool = False, device="cuda") -> "PagedCache":
        """A new cache with a pool of num_pages pages (zero-filled); summaries: with kmin and kmax."""
        H, D = desc.num_kv_heads, desc.head_dim
        dt = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
        new = lambda *shape: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        pool = (int(num_pages), H, desc.page_size, D)
        return cls(desc, new(*pool), new(*pool), *((new(num_pages, H, D), new(num_pages, H, D)) if summaries else ()))

    def load(self, table, ctx_len):
        """Takes over a table [B, Cap/P] and lengths [B] made elsewhere (paged_init)."""
        self._beside(torch._C._cuda_getDevice(), self.desc())  # before anything changes
        both = ((table, self.table, "table"), (ctx_len, self.ctx_len, "ctx_len"))
        for t, mine, name in both:
            if t.shape != mine.shape or t.dtype not in (torch.int64, torch.int32, torch.int16, torch.int8, torch.uint8):
                raise ValueError(f"{name} must be integers of shape {tuple(mine.shape)}, got {t.dtype} {tuple(t.shape)}")
        for t, mine, _ in both:  # numbers that 32 bits cannot hold stay out of range
            mine.copy_(t.clamp(-1 << 31, (1 << 31) - 1) if t.dtype == torch.int64 else t)
        paged_init(self.desc(), self)

    def desc(self) -> L.AttnDesc:
        """A descriptor of the cache's shape, with as many query heads as KV heads."""
        B, H, cap, D, P, dtype = self.shape
        return make_desc(B, H, H, D, P, cap, dtype)

    def _beside(self, index: int, desc: L.AttnDesc) -> L.PagedCacheDesc:
        """The C structure, for a call with this descriptor on device `index`."""
        if index != self.index:
            raise ValueError("the cache must be on the device of the other tensors")
        if (desc.batch, desc.num_kv_heads, desc.capacity, desc.head_dim, desc.page_size, desc.dtype) != self.shape:
            raise ValueError(f"the descriptor's shape is not that of the cache, {self.shape}")
        return self.c

    def values(self, b: int):
        """Sequence b's K and V [Hkv, n, D] in order (for inspection: reads its length)."""
        n, P = int(self.ctx_len[b]), self.shape[4]
        pages = self.table[b, :-(-n // P)].long()
        return tuple(x[pages].transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n] for x in (self.k_pages, self.v_pages))


def paged_init(desc: L.AttnDesc, cache: PagedCache):
    """Derives the counts and the free pages from the cache's table and lengths (sls_paged_init)."""
    L.call("sls_paged_init", ctypes.byref(desc), ctypes.byref(cache._beside(torch._C._cuda_getDevice(), desc)), _stream())


def paged_append(desc: L.AttnDesc, cache: PagedCache, k_new, v_new, new_len=None, pos_out=None):
    """Appends the first new_len[b] (None: all) tokens of k_new, v_new [B, T, Hkv, D] to every sequence, on pages taken
    from the pool (sls_paged_append).  The new tensors may be strided views with contiguous channels.  Returns the
    cache's ctx_len, advanced in place."""
    status = (_fast or _binding()).paged_append(desc, cache._beside(k_new.get_device(), desc), k_new, v_new, new_len, pos_out)
    if status:
        L.check("sls_paged_append", status)
    return cache.ctx_len


def paged_select_workspace(desc: L.AttnDesc, cache: PagedCache):
    """Scratch buffer of paged_select_pages (that of select_pages)."""
    return select_pages_workspace(desc, cache.k_pages.device)


def paged_select_pages(desc: L.AttnDesc, cache: PagedCache, q, k: int, n_sink_pages: int = 0, n_local_tokens: int = 0,
                       out=None, workspace=None):
    """Quest selection over a paged cache's summaries (sls_paged_select_pages).  Returns the logical pages
    [B*Hkv, k] int32, ascending, -1 padded."""
    if out is None:
        out = torch.empty((desc.batch * desc.num_kv_heads, max(int(k), 0)), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = paged_select_workspace(desc, cache)
    status = (_fast or _binding()).paged_select_pages(desc, cache._beside(q.get_device(), desc), q, k, n_sink_pages,
                                                      n_local_tokens, out, workspace)
    if status:
        L.check("sls_paged_select_pages", status)
    return out


def paged_attend_workspace(desc: L.AttnDesc, cache: PagedCache):
    """Zero-filled workspace of paged_decode_attend (reusable, also by calls of other shapes that need no more bytes, one
    after the other)."""
    n = L.load().sls_paged_decode_attend_workspace_size(ctypes.byref(desc))
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=cache.k_pages.device)


def paged_decode_attend(desc: L.AttnDesc, cache: PagedCache, q, page_idx=None, count=None, k_fixed: Optional[int] = None,
                        sink=None, out=None, lse=None, workspace=None, want_lse: bool = True):
    """Decode attention over a paged cache (sls_paged_decode_attend): dense, or over lists [rows, stride] of logical
    pages.  Returns (out, lse)."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = paged_attend_workspace(desc, cache)
    status = (_fast or _binding()).paged_decode_attend(desc, cache._beside(q.get_device(), desc), q, page_idx, count, k_fixed,
                                                       sink, out, lse, workspace)
    if status:
        L.check("sls_paged_decode_attend", status)
    return out, lse


def paged_fork_workspace(desc: L.AttnDesc, cache: PagedCache):
    """Workspace of paged_fork (reusable)."""
    n = L.load().sls_paged_fork_workspace_size(ctypes.byref(desc))
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=cache.k_pages.device)


def paged_fork(desc: L.AttnDesc, cache: PagedCache, parent, keep_len=None, done=None, workspace=None):
    """Makes every sequence b the first keep_len[b] (None: all) tokens of what sequence parent[b] was (sls_paged_fork):
    forks, reorders, cuts, and with parent[b] = -1 frees.  done [1] int32, if given, becomes 1, or 0 when the pool
    lacked pages for the copies of partial pages (nothing has changed then)."""
    if workspace is None:
        workspace = paged_fork_workspace(desc, cache)
    status = (_fast or _binding()).paged_fork(desc, cache._beside(parent.get_device(), desc), parent, keep_len, done, workspace)
    if status:
        L.check("sls_paged_fork", status)


def paged_compact_workspace(desc: L.AttnDesc, cache: PagedCache):
    """Workspace of paged_compact (reusable)."""
    n = L.load().sls_paged_compact_workspace_size(cache.num_pages)
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=cache.k_pages.device)


def paged_compact(desc: L.AttnDesc, cache: PagedCache, moved=None, workspace=None):
    """Moves the used pages to the front of the pool (sls_paged_compact).  moved [N] int32, if given, receives every
    page's new number (-1: it was free)."""
    if workspace is None:
        workspace = paged_compact_workspace(desc, cache)
    status = (_fast or _binding()).paged_compact(desc, cache._beside(workspace.get_device(), desc), moved, workspace)
    if status:
        L.check("sls_paged_compact", status)


# ------------------------------------------------------------ decode step

class QuestDecode:
    """One Quest decode step (select + attend + combine) over preallocated
    buffers, capturable in a CUDA graph.  one_launch: the whole step in one
    kernel where the shape allows (quest_decode_step); otherwise select, then
    attend with the combine fused (fused=True) or as its own launch."""

    def __init__(self, desc: L.AttnDesc, k_budget: int, n_sink_pages: int, n_local_tokens: int,
                 num_splits: Optional[int] = None, device="cuda", fused: bool = True,
                 one_launch: bool = True, min_sparsity: float = 0.0):
        self.desc = desc
        self.k = int(k_budget)
        self.n_sink, self.n_local = int(n_sink_pages), int(n_local_tokens)
        self.fused = fused
        self.one_launch = fused and one_launch
        self.min_sparsity = float(min_sparsity)
        rows = desc.batch * desc.num_kv_heads
        self.S = num_splits or default_splits(desc, self.k)
        self.step_splits = int(num_splits or 0)
        self.step_workspace = quest_step_workspace(desc, self.k, self.step_splits, device)
        self.page_idx = torch.empty((rows, self.k), dtype=torch.int32, device=device)
        self.workspace = select_pages_workspace(desc, device)
        self.parts = partials(desc, self.S, device)
        self.ac_workspace = attend_combine_workspace(desc, self.S, device)
        dtype = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
        self.out = torch.empty((desc.batch, desc.num_q_heads, desc.head_dim), dtype=dtype, device=device)
        self.lse = torch.empty((desc.batch, desc.num_q_heads), dtype=torch.float32, device=device)

    def select(self, q, kmin, kmax, ctx_len):
        return select_pages(self.desc, q, kmin, kmax, ctx_len, self.k, self.n_sink, self.n_local,
                            out=self.page_idx, workspace=self.workspace)

    def attend(self, q, k_cache, v_cache, ctx_len, sink=None):
        if self.fused:
            return sparse_decode_attend_combine(self.desc, q, k_cache, v_cache, self.page_idx, ctx_len,
                                                self.S, sink=sink, out=self.out, lse=self.lse,
                                                workspace=self.ac_workspace)
        sparse_decode_attend(self.desc, q, k_cache, v_cache, self.page_idx, ctx_len, self.S,
                             parts=self.parts)
        return combine_splits(self.desc, self.parts, sink, out=self.out, lse=self.lse)

    def __call__(self, q, k_cache, v_cache, kmin, kmax, ctx_len, sink=None):
        if self.one_launch:
            return quest_decode_step(self.desc, q, k_cache, v_cache, kmin, kmax, ctx_len, self.k, self.n_sink,
                                     self.n_local, sink=sink, page_idx=self.page_idx, out=self.out,
                                     lse=self.lse, num_splits=self.step_splits, workspace=self.step_workspace,
                                     min_sparsity=self.min_sparsity)
        self.select(q, kmin, kmax, ctx_len)
        return self.attend(q, k_cache, v_cache, ctx_len, sink)


class DeltaDecode:
    """One top-delta decode step (select_delta + attend + combine).

    balanced=True (the default where the shape allows: bf16, G <= 8, no path
    flag in the descriptor) attends
    with the work-item kernel, which spreads rows of very different list
    lengths evenly over the GPU; otherwise the split-K attend with num_splits
    per row.  With refined=True the attend scores complete blocks with the
    refined keys (2-bit thumbnail + 8-bit residual, "Faster Than Flash"
    eq. 4): the call then takes the residuals as well."""

    def __init__(self, desc: L.AttnDesc, block: int, delta: float, num_splits: Optional[int] = None,
                 device="cuda", fused: bool = True, refined: bool = False, balanced: Optional[bool] = None):
        if desc.page_size != block:
            raise ValueError("attend page_size must equal the thumbnail block")
        self.desc, self.block, self.delta = desc, int(block), float(delta)
        self.fused = fused
        self.refined = refined
        ok = (desc.dtype == L.SLS_DTYPE_BF16 and desc.num_q_heads // desc.num_kv_heads <= 8
              and desc.batch * desc.num_kv_heads <= 4096)  # the work-item kernel's row limit
        # the default for the fast path only: the descriptor's path flags select the split-K attends
        self.balanced = (fused and ok and desc.flags == 0) if balanced is None else balanced
        if refined and not ok:
            raise ValueError("the refined attend needs bf16 and G <= 8")
        self.bal_workspace = refined_workspace(desc, device) if (self.balanced or refined) else None
        rows = desc.batch * desc.num_kv_heads
        nblk = desc.capacity // block
        self.S = num_splits or default_splits(desc, nblk)
        self.count = torch.empty(rows, dtype=torch.int32, device=device)
        self.block_idx = torch.empty((rows, nblk), dtype=torch.int32, device=device)
        self.workspace = select_delta_workspace(desc, block, device)
        self.parts = partials(desc, self.S, device)
        self.ac_workspace = attend_combine_workspace(desc, self.S, device)
        dtype = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
        self.out = torch.empty((desc.batch, desc.num_q_heads, desc.head_dim), dtype=dtype, device=device)
        self.lse = torch.empty((desc.batch, desc.num_q_heads), dtype=torch.float32, device=device)

    def select(self, q, k_cache, codes, scales, ctx_len):
        return select_delta(self.desc, q, k_cache, codes, scales, ctx_len, self.block, self.delta,
                            count=self.count, block_idx=self.block_idx, workspace=self.workspace)

    def attend(self, q, k_cache, v_cache, ctx_len, sink=None):
        if self.balanced:
            return refined_decode_attend_combine(self.desc, q, k_cache, v_cache, None, None, None, self.block_idx,
                                                 self.count, ctx_len, sink=sink, out=self.out, lse=self.lse,
                                                 workspace=self.bal_workspace)
        if self.fused:
            return sparse_decode_attend_combine(self.desc, q, k_cache, v_cache, self.block_idx, ctx_len,
                                                self.S, count=self.count, sink=sink, out=self.out,
                                                lse=self.lse, workspace=self.ac_workspace)
        sparse_decode_attend(self.desc, q, k_cache, v_cache, self.block_idx, ctx_len, self.S,
                             count=self.count, parts=self.parts)
        return combine_splits(self.desc, self.parts, sink, out=self.out, lse=self.lse)

    def attend_refined(self, q, k_cache, v_cache, codes, scales, res, ctx_len, sink=None):
        return refined_decode_attend_combine(self.desc, q, k_cache, v_cache, codes, scales, res, self.block_idx,
                                             self.count, ctx_len, sink=sink, out=self.out, lse=self.lse,
                                             workspace=self.bal_workspace)

    def __call__(self, q, k_cache, v_cache, codes, scales, ctx_len, sink=None, res=None):
        self.select(q, k_cache, codes, scales, ctx_len)
        if self.refined:
            if res is None:
                raise ValueError("the refined step needs the residuals")
            return self.attend_refined(q, k_cache, v_cache, codes, scales, res, ctx_len, sink)
        return self.attend(q, k_cache, v_cache, ctx_len, sink)


class Kv8Decode:
    """One decode step over an 8-bit cache from the projected heads on: norm and rotation of q and k
    (qk_norm_rope), append of the token (kv8_append), and the attention, dense or, with k_budget > 0, over the
    k_budget pages per KV head that Quest selection picks from page min/max kept of the unquantised keys.  The
    buffers are preallocated, so a step can be captured in a CUDA graph.  With mass=True every block's attention
    weight is summed (dense only), and evict() cuts the cache to a budget of blocks by it.

    As with decode_append, a sequence at capacity is left unchanged: the step appends nothing to it and ctx_len
    stays (its query attends to what is held), so a caller that counts tokens evicts, or stops, before that.  The
    same holds for a piece of a prompt that does not fit.  The weight sums are those of decode steps: after a prefill
    they are 0, and an eviction then keeps the first blocks."""

    def __init__(self, desc: L.AttnDesc, rope: L.RopeDesc, fmt: str = "int8", block: int = 64, k_budget: int = 0,
                 n_sink_pages: int = 0, n_local_tokens: int = 0, mass: bool = False, device="cuda",
                 q_weight=None, k_weight=None):
        if (rope.num_q_heads, rope.num_kv_heads, rope.head_dim, rope.dtype) != (
                desc.num_q_heads, desc.num_kv_heads, desc.head_dim, desc.dtype):
            raise ValueError("rope and desc must describe the same heads")
        if mass and k_budget:
            raise ValueError("weight sums need dense attention (k_budget 0)")
        if desc.flags & ~L.SLS_FLAG_TEST_WAIT_TIMEOUT:
            raise ValueError("the 8-bit attend has one kernel: no path flags")
        if k_budget:  # what the first step would refuse only after it has appended its token
            if desc.page_size < 16:
                raise ValueError(f"page lists over an 8-bit cache need pages of >= 16 tokens, got {desc.page_size}")
            forced = n_sink_pages + (-(-n_local_tokens // desc.page_size) + 1 if n_local_tokens > 0 else 0)
            if min(n_sink_pages, n_local_tokens) < 0 or not max(1, forced) <= k_budget <= desc.capacity // desc.page_size:
                raise ValueError(f"k_budget {k_budget} must hold the forced pages (up to {forced}) and be at most the "
                                 f"{desc.capacity // desc.page_size} pages of a row")
        B, Hq, H, D, P = desc.batch, desc.num_q_heads, desc.num_kv_heads, desc.head_dim, desc.page_size
        self.desc, self.rope = desc, rope
        self.k, self.n_sink, self.n_local = int(k_budget), int(n_sink_pages), int(n_local_tokens)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.cache = Kv8Cache.empty(desc, fmt, block, device)
        new = lambda shape, dt=torch.bfloat16: torch.zeros(shape, dtype=dt, device=device)  # noqa: E731
        self.ctx_len = new(B, torch.int32)      # tokens held
        self.evicted = new(B, torch.int32)      # tokens evicted before them: position = evicted + index held
        self.positions = new(B, torch.int32)    # position of the step's token
        self.q, self.k_new = new((B, Hq, D)), new((B, H, D))
        self.out, self.lse = new((B, Hq, D)), new((B, Hq), torch.float32)
        self.kmin = self.kmax = self.page_idx = self.select_workspace = self.mass = None
        if self.k:
            self.kmin, self.kmax = new((B, H, desc.capacity // P, D)), new((B, H, desc.capacity // P, D))
            self.page_idx = new((B * H, self.k), torch.int32)
            self.select_workspace = select_pages_workspace(desc, device)
        if mass:
            self.mass = new((B, H, desc.capacity // block), torch.float32)
        if not L.load().sls_kv8_decode_attend_workspace_size(ctypes.byref(desc), ctypes.byref(self.cache.c), int(mass)):
            raise ValueError("the 8-bit attend does not take this descriptor or block")
        self.workspace = kv8_attend_workspace(desc, self.cache, mass, device)

    def prefill(self, qkv, new_len=None):
        """Writes the keys and values of a prompt (or of its next piece): qkv [B, T, Hq + 2 Hkv, D], of which
        sequence b has its first new_len[b] tokens.  Returns the rotated queries [B, T, Hq, D]."""
        Hq, H, D = self.desc.num_q_heads, self.desc.num_kv_heads, self.desc.head_dim
        B, T = qkv.shape[:2]
        step = torch.arange(T, dtype=torch.int32, device=qkv.device)
        pos = (self.ctx_len + self.evicted)[:, None] + step
        if new_len is not None:
            pos = torch.where(step < new_len[:, None], pos, -1)  # padding is skipped
        flat = qkv[:, :, :Hq + H].reshape(B * T, Hq + H, D)  # a view, or a copy where qkv is a slice of a longer batch
        q, k = qk_norm_rope(self.rope, flat[:, :Hq], flat[:, Hq:], pos.reshape(-1), self.q_weight, self.k_weight)
        kv8_append(self.desc, self.cache, k.view(B, T, H, D), qkv[:, :, Hq + H:], self.ctx_len, new_len=new_len,
                   kmin=self.kmin, kmax=self.kmax, mass=self.mass)
        return q.view(B, T, Hq, D)

    def __call__(self, qkv, sink=None):
        """qkv [B, Hq + 2 Hkv, D]: the projected heads of one token per sequence.  Returns (out, lse)."""
        d, Hq, H = self.desc, self.desc.num_q_heads, self.desc.num_kv_heads
        if sink is not None:
            _need_sink(sink, Hq, self.cache.index)  # before the token is appended
        torch.add(self.ctx_len, self.evicted, out=self.positions)
        qk_norm_rope(self.rope, qkv[:, :Hq], qkv[:, Hq:Hq + H], self.positions, self.q_weight, self.k_weight,
                     q_out=self.q, k_out=self.k_new)
        kv8_append(d, self.cache, self.k_new[:, None], qkv[:, None, Hq + H:], self.ctx_len, kmin=self.kmin,
                   kmax=self.kmax, mass=self.mass)
        if self.k:
            select_pages(d, self.q, self.kmin, self.kmax, self.ctx_len, self.k, self.n_sink, self.n_local,
                         out=self.page_idx, workspace=self.select_workspace)
        return kv8_decode_attend(d, self.cache, self.q, self.ctx_len, page_idx=self.page_idx, sink=sink,
                                 mass_in=self.mass, mass_out=self.mass, out=self.out, lse=self.lse,
                                 workspace=self.workspace)

    def evict(self, keep: int, n_sink_blocks: int = 0, n_recent_blocks: int = 0):
        """Cuts every sequence to its keep heaviest complete blocks (kv8_evict in place).  Returns their numbers."""
        if self.mass is None:
            raise ValueError("evict needs the weight sums (mass=True)")
        held = self.ctx_len.clone()
        kept = kv8_evict(self.desc, self.cache, self.ctx_len, self.mass, keep, n_sink_blocks, n_recent_blocks)[1]
        self.evicted += held - self.ctx_len  # after the call: one that is refused moves no position
        return kept


class PagedDecode:
    """One decode step over a paged cache from the projected heads on: norm and rotation of q and k (qk_norm_rope),
    append of the token on pages of the pool (paged_append), and the attention, dense or, with k_budget > 0, over the
    k_budget pages per KV head that Quest selection picks (paged_select_pages).  The buffers are preallocated, so a step
    can be captured in a CUDA graph.

    A sequence at capacity, or for whose token the pool has no page left, is left unchanged: pos[b] is then -1, and its
    query attends to what is held.  The same holds for a piece of a prompt."""

    def __init__(self, desc: L.AttnDesc, rope: L.RopeDesc, num_pages: int, k_budget: int = 0, n_sink_pages: int = 0,
                 n_local_tokens: int = 0, device="cuda", q_weight=None, k_weight=None):
        if (rope.num_q_heads, rope.num_kv_heads, rope.head_dim, rope.dtype) != (
                desc.num_q_heads, desc.num_kv_heads, desc.head_dim, desc.dtype):
            raise ValueError("rope and desc must describe the same heads")
        if desc.flags & ~L.SLS_FLAG_TEST_WAIT_TIMEOUT:
            raise ValueError("the paged attend has one kernel: no path flags")
        if k_budget:  # what the first step would refuse only after it has appended its token
            forced = n_sink_pages + (-(-n_local_tokens // desc.page_size) + 1 if n_local_tokens > 0 else 0)
            if min(n_sink_pages, n_local_tokens) < 0 or not max(1, forced) <= k_budget <= desc.capacity // desc.page_size:
                raise ValueError(f"k_budget {k_budget} must hold the forced pages (up to {forced}) and be at most the "
                                 f"{desc.capacity // desc.page_size} pages of a sequence")
            if not L.load().sls_select_pages_workspace_size(ctypes.byref(desc)):
                raise ValueError("the selection does not take this descriptor (262144 pages a sequence at most, got "
                                 f"{desc.capacity // desc.page_size})")
        if not L.load().sls_paged_decode_attend_workspace_size(ctypes.byref(desc)):
            raise ValueError("the paged attend does not take this descriptor")
        B, Hq, H, D = desc.batch, desc.num_q_heads, desc.num_kv_heads, desc.head_dim
        dt = torch.bfloat16 if desc.dtype == L.SLS_DTYPE_BF16 else torch.float32
        self.desc, self.rope = desc, rope
        self.k, self.n_sink, self.n_local = int(k_budget), int(n_sink_pages), int(n_local_tokens)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.cache = PagedCache.empty(desc, num_pages, summaries=self.k > 0, device=device)
        new = lambda shape, dtype=dt: torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        self.q, self.k_new = new((B, Hq, D)), new((B, H, D))
        self.out, self.lse = new((B, Hq, D)), new((B, Hq), torch.float32)
        self.pos = new(B, torch.int32)  # positions written by the last step or piece of a prompt
        self.done = new(1, torch.int32)
        self.page_idx = self.select_workspace = None
        if self.k:
            self.page_idx = new((B * H, self.k), torch.int32)
            self.select_workspace = paged_select_workspace(desc, self.cache)
        self.workspace = paged_attend_workspace(desc, self.cache)
        self.fork_workspace = paged_fork_workspace(desc, self.cache)
        self.compact_workspace = paged_compact_workspace(desc, self.cache)

    @property
    def ctx_len(self):
        """Tokens held by each sequence [B] int32 (the cache's own)."""
        return self.cache.ctx_len

    def prefill(self, qkv, new_len=None):
        """Writes the keys and values of a prompt (or of its next piece): qkv [B, T, Hq + 2 Hkv, D], of which
        sequence b has its first new_len[b] tokens.  Returns the rotated queries [B, T, Hq, D]."""
        Hq, H, D = self.desc.num_q_heads, self.desc.num_kv_heads, self.desc.head_dim
        B, T = qkv.shape[:2]
        step = torch.arange(T, dtype=torch.int32, device=qkv.device)
        pos = self.ctx_len[:, None] + step
        if new_len is not None:
            pos = torch.where(step < new_len[:, None], pos, -1)  # padding is skipped
        flat = qkv[:, :, :Hq + H].reshape(B * T, Hq + H, D)  # a view, or a copy where qkv is a slice of a longer batch
        q, k = qk_norm_rope(self.rope, flat[:, :Hq], flat[:, Hq:], pos.reshape(-1), self.q_weight, self.k_weight)
        paged_append(self.desc, self.cache, k.view(B, T, H, D), qkv[:, :, Hq + H:], new_len=new_len, pos_out=self.pos)
        return q.view(B, T, Hq, D)

    def __call__(self, qkv, sink=None):
        """qkv [B, Hq + 2 Hkv, D]: the projected heads of one token per sequence.  Returns (out, lse)."""
        d, Hq, H = self.desc, self.desc.num_q_heads, self.desc.num_kv_heads
        if sink is not None:
            _need_sink(sink, Hq, self.cache.index)  # before the token is appended
        qk_norm_rope(self.rope, qkv[:, :Hq], qkv[:, Hq:Hq + H], self.ctx_len, self.q_weight, self.k_weight, q_out=self.q,
                     k_out=self.k_new)
        paged_append(d, self.cache, self.k_new[:, None], qkv[:, None, Hq + H:], pos_out=self.pos)
        if self.k:
            paged_select_pages(d, self.cache, self.q, self.k, self.n_sink, self.n_local, out=self.page_idx,
                               workspace=self.select_workspace)
        return paged_decode_attend(d, self.cache, self.q, page_idx=self.page_idx, sink=sink, out=self.out, lse=self.lse,
                                   workspace=self.workspace)

    def fork(self, parent, keep_len=None):
        """Forks, reorders, cuts and frees sequences (paged_fork).  Returns done [1]: 1, or 0 when the pool lacked pages
        and nothing has changed."""
        paged_fork(self.desc, self.cache, parent, keep_len=keep_len, done=self.done, workspace=self.fork_workspace)
        return self.done

    def compact(self):
        """Moves the used pages to the front of the pool (paged_compact)."""
        paged_compact(self.desc, self.cache, workspace=self.compact_workspace)
