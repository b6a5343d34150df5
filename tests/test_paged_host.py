"""What the paged cache's calls refuse, before any launch: shapes, types, workspaces, alignment, and buffers that share
memory.  (No call of this file may pass: it would be launched.)"""
import ctypes

import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops

P = lambda x: ctypes.c_void_p(x)  # noqa: E731  never dereferenced
NAMES = ("k_pages", "v_pages", "kmin", "kmax", "ctx_len", "table", "refs", "state")
PAGES = 64  # [64, 2, 16, 128] bf16: 512 KB
AT = {n: (1 + i) << 24 for i, n in enumerate(NAMES)}
SIZES = dict(k_pages=PAGES << 13, v_pages=PAGES << 13, kmin=PAGES << 9, kmax=PAGES << 9, ctx_len=12, table=3 * 64 * 4, refs=PAGES * 4,
             state=(16 + 2 + 6) * 4)
X = {n: (21 + i) << 24 for i, n in enumerate(
    ("k", "v", "len", "pos", "q", "out", "lse", "ws", "idx", "count", "sink", "parent", "keep", "done", "moved"))}


def desc(**kw):
    d = dict(batch=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, capacity=1024, dtype=L.SLS_DTYPE_BF16, flags=0,
             scale=0.0)
    d.update(kw)
    return L.AttnDesc(*d.values())


def cache(pages=PAGES, **kw):
    return L.PagedCacheDesc(pages, *({**AT, **kw}[n] for n in NAMES))


def init(lib, d=None, c=None):
    return lib.sls_paged_init(ctypes.byref(d or desc()), ctypes.byref(c or cache()), None)


def append(lib, d=None, c=None, strides=(8 * 256, 256, 128), max_new=8, **kw):
    x = {**X, **kw}
    return lib.sls_paged_append(ctypes.byref(d or desc()), ctypes.byref(c or cache()), P(x["k"]), *strides, P(x["v"]), *strides,
                                max_new, P(x["len"]), P(x["pos"]), None)


def select(lib, d=None, c=None, k=8, sinks=1, local=16, size=None, **kw):
    x, d = {**X, **kw}, d or desc()
    size = lib.sls_select_pages_workspace_size(ctypes.byref(d)) if size is None else size
    return lib.sls_paged_select_pages(ctypes.byref(d), ctypes.byref(c or cache()), P(x["q"]), k, sinks, local, P(x["idx"]),
                                      P(x["ws"]), size, None)


def attend(lib, d=None, c=None, size=1 << 22, stride=8, fixed=8, **kw):
    x = {**X, **kw}
    return lib.sls_paged_decode_attend(ctypes.byref(d or desc()), ctypes.byref(c or cache()), P(x["q"]), P(x["idx"]), stride,
                                       P(x["count"]), fixed, P(x["sink"]), P(x["out"]), P(x["lse"]), P(x["ws"]), size, None)


def fork(lib, d=None, c=None, size=1 << 20, **kw):
    x = {**X, **kw}
    return lib.sls_paged_fork(ctypes.byref(d or desc()), ctypes.byref(c or cache()), P(x["parent"]), P(x["keep"]), P(x["done"]),
                              P(x["ws"]), size, None)


def compact(lib, d=None, c=None, size=1 << 20, **kw):
    x = {**X, **kw}
    return lib.sls_paged_compact(ctypes.byref(d or desc()), ctypes.byref(c or cache()), P(x["moved"]), P(x["ws"]), size, None)


CALLS = [init, append, select, attend, fork, compact]


def error(lib):
    return lib.sls_last_error().decode()


@pytest.mark.parametrize("call", CALLS)
def test_descriptors_and_caches(lib, call):
    for bad, code in ((dict(page_size=8), L.SLS_EUNSUPPORTED), (dict(page_size=1), L.SLS_EUNSUPPORTED),
                      (dict(page_size=24), L.SLS_EINVAL), (dict(page_size=512, capacity=1024), L.SLS_EINVAL),
                      (dict(head_dim=96), L.SLS_EUNSUPPORTED), (dict(dtype=2), L.SLS_EUNSUPPORTED), (dict(batch=0), L.SLS_EINVAL),
                      (dict(batch=4097), L.SLS_EUNSUPPORTED), (dict(num_q_heads=18), L.SLS_EUNSUPPORTED),
                      (dict(num_q_heads=7), L.SLS_EINVAL), (dict(capacity=1000), L.SLS_EINVAL),
                      (dict(batch=4096, capacity=1 << 24), L.SLS_EOVERFLOW)):
        assert call(lib, d=desc(**bad)) == code, bad
    for pages in (0, -1, (1 << 24) + 1):
        assert call(lib, c=cache(pages)) == L.SLS_EINVAL
    assert call(lib, d=desc(num_kv_heads=8), c=cache(1 << 24)) == L.SLS_EOVERFLOW
    for n in ("k_pages", "v_pages", "ctx_len", "table", "refs", "state"):
        assert call(lib, c=cache(**{n: None})) == L.SLS_EINVAL and "NULL" in error(lib)
    for n in NAMES:
        step = 2 if n in ("ctx_len", "table", "refs") else 8
        assert call(lib, c=cache(**{n: AT[n] + step})) == L.SLS_EINVAL and "aligned" in error(lib), n
    assert call(lib, c=cache(kmin=None)) == L.SLS_EINVAL and "both" in error(lib)


@pytest.mark.parametrize("call", CALLS)
def test_a_caches_buffers_share_no_memory(lib, call):
    for i, a in enumerate(NAMES):
        for b in NAMES[:i]:
            for at in (AT[b], AT[b] + (SIZES[b] - 4) // 16 * 16):
                assert call(lib, c=cache(**{a: at})) == L.SLS_EINVAL and "share memory" in error(lib), (a, b)


ARGS = {append: ("k", "v", "len", "pos"), select: ("q", "idx", "ws"), fork: ("parent", "keep", "done", "ws"),
        attend: ("q", "idx", "count", "sink", "out", "lse", "ws"), compact: ("moved", "ws")}
WRITTEN = {append: ("pos",), select: ("idx", "ws"), attend: ("out", "lse", "ws"), fork: ("done", "ws"), compact: ("moved", "ws")}


@pytest.mark.parametrize("call", CALLS[1:])
def test_arguments_share_no_memory_and_are_aligned(lib, call):
    for n in ARGS[call]:
        for b in NAMES:
            for at in (AT[b], AT[b] + (SIZES[b] - 4) // 16 * 16):
                assert call(lib, **{n: at}) == L.SLS_EINVAL and "memory with the cache" in error(lib), (n, b)
        assert call(lib, **{n: X[n] + 2}) == L.SLS_EINVAL and "aligned" in error(lib), n
    for n in WRITTEN[call]:
        for other in ARGS[call]:
            if other != n:
                assert call(lib, **{n: X[other]}) == L.SLS_EINVAL and "shares memory with another" in error(lib), (n, other)


def test_append(lib):
    assert append(lib, max_new=-1) == L.SLS_EINVAL
    for n in ("k", "v"):
        assert append(lib, **{n: None}) == L.SLS_EINVAL
    for st in ((-8, 256, 128), (2048, 256, 4), (2048, 4, 128), (1 << 41, 256, 128)):
        assert append(lib, strides=st) == L.SLS_EINVAL
    assert append(lib, d=desc(dtype=L.SLS_DTYPE_F32), strides=(2048, 256, 2)) == L.SLS_EINVAL
    # a strided tensor that reaches into the cache
    assert append(lib, k=AT["refs"] - 4 * 2048, strides=(2048, 256, 128)) == L.SLS_EINVAL and "cache" in error(lib)
    assert append(lib, v=AT["refs"] - (1 << 20), strides=(1 << 22, 256, 128)) == L.SLS_EINVAL and "cache" in error(lib)


def test_select(lib):
    assert select(lib, c=cache(kmin=None, kmax=None)) == L.SLS_EINVAL and "kmin" in error(lib)
    for bad in (dict(k=0), dict(k=65), dict(sinks=-1), dict(local=-1), dict(k=2, sinks=3, local=0), dict(k=3, sinks=1, local=32)):
        assert select(lib, **bad) == L.SLS_EINVAL, bad
    assert select(lib, size=100) == L.SLS_EWORKSPACE and select(lib, ws=None) == L.SLS_EWORKSPACE
    for n in ("q", "idx"):
        assert select(lib, **{n: None}) == L.SLS_EINVAL
    assert select(lib, d=desc(capacity=16 << 20)) == L.SLS_EUNSUPPORTED


def test_attend(lib):
    for flag in (L.SLS_FLAG_CUDA_CORES, L.SLS_FLAG_NO_TMA):
        assert attend(lib, d=desc(flags=flag)) == L.SLS_EUNSUPPORTED
    assert attend(lib, d=desc(batch=4096)) == L.SLS_EUNSUPPORTED  # 8192 rows
    assert lib.sls_paged_decode_attend_workspace_size(ctypes.byref(desc(batch=4096))) == 0
    assert lib.sls_paged_decode_attend_workspace_size(ctypes.byref(desc(page_size=8))) == 0
    for bad in (dict(stride=0), dict(fixed=-1, count=None), dict(fixed=9, count=None)):
        assert attend(lib, **bad) == L.SLS_EINVAL, bad
    assert attend(lib, stride=1 << 28) == L.SLS_EOVERFLOW
    assert attend(lib, size=64) == L.SLS_EWORKSPACE and attend(lib, ws=None) == L.SLS_EWORKSPACE
    for n in ("q", "out"):
        assert attend(lib, **{n: None}) == L.SLS_EINVAL
        assert attend(lib, **{n: X[n] + 4}) == L.SLS_EINVAL


def test_fork_and_compact(lib):
    assert fork(lib, parent=None) == L.SLS_EINVAL
    assert fork(lib, size=100) == L.SLS_EWORKSPACE and fork(lib, ws=None) == L.SLS_EWORKSPACE
    assert fork(lib, size=lib.sls_paged_fork_workspace_size(ctypes.byref(desc())) - 1) == L.SLS_EWORKSPACE
    assert compact(lib, size=lib.sls_paged_compact_workspace_size(PAGES) - 1) == L.SLS_EWORKSPACE
    assert lib.sls_paged_fork_workspace_size(ctypes.byref(desc(batch=5000))) == 0
    assert lib.sls_paged_compact_workspace_size(0) == 0
    assert fork(lib, ws=X["ws"] + 4) == L.SLS_EINVAL and compact(lib, ws=X["ws"] + 8) == L.SLS_EINVAL


def test_words_of_state(lib):
    for pages, want in ((1, 16 + 2 + 6), (32, 16 + 2 + 6), (64, 16 + 2 + 6), (65, 16 + 4 + 6), (1 << 24, 16 + (1 << 19) + 6)):
        assert lib.sls_paged_state_words(ctypes.byref(desc()), pages) == want
    assert lib.sls_paged_state_words(ctypes.byref(desc(page_size=8)), 64) == 0
    assert lib.sls_paged_state_words(ctypes.byref(desc()), 0) == 0


def test_python_side():
    d = ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16)
    cpu = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.PagedCache(d, cpu, cpu)
    rope = ops.make_rope(4, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError, match="same heads"):
        ops.PagedDecode(d, ops.make_rope(4, 1, 64, torch.bfloat16), 8)
    with pytest.raises(ValueError, match="path flags"):
        ops.PagedDecode(ops.make_desc(2, 4, 2, 64, 16, 256, torch.bfloat16, cuda_cores=True), rope, 8)
    for k, sinks, local in ((17, 0, 0), (2, 3, 0), (2, 0, 32), (4, -1, 0)):
        with pytest.raises(ValueError, match="k_budget"):
            ops.PagedDecode(d, rope, 8, k_budget=k, n_sink_pages=sinks, n_local_tokens=local)
    with pytest.raises(ValueError, match="does not take"):
        ops.PagedDecode(ops.make_desc(2, 4, 2, 64, 8, 256, torch.bfloat16), rope, 8)
