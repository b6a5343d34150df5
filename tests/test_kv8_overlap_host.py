"""Buffers that share memory where a call of the 8-bit cache could not give the documented result (or could follow an
overwritten list): refused on the host, before any launch."""
import ctypes

import pytest

from sparse_long_context_gb300 import _lib as L

P = lambda x: ctypes.c_void_p(x)  # noqa: E731  never dereferenced
NAMES = ("k_codes", "v_codes", "k_scales", "v_scales", "k_tail", "v_tail")
DESC = L.AttnDesc(2, 8, 2, 128, 16, 1024, L.SLS_DTYPE_BF16, 0, 0.0)  # 4 rows of 16 blocks of 64 tokens
AT = {n: (1 + i) << 24 for i, n in enumerate(NAMES)}
TO = {n: (11 + i) << 24 for i, n in enumerate(NAMES)}
SIZES = dict(k_codes=4 << 17, v_codes=4 << 17, k_scales=256, v_scales=256, k_tail=4 << 14, v_tail=4 << 14)
X = {n: (21 + i) << 24 for i, n in enumerate(
    ("mass", "mass_out", "kmin", "kmax", "kmin_out", "kmax_out", "kept", "ctx", "ctx_out", "pos", "k", "v", "len", "q",
     "out", "lse", "ws", "idx", "count", "sink"))}


def cache(at):
    return L.Kv8CacheDesc(0, 64, *(at[n] for n in NAMES))


def evict(lib, in_place, src=None, dst=None, **kw):
    x = {**X, **kw}
    a = {**AT, **(src or {})}
    b = a if in_place else {**TO, **(dst or {})}
    if in_place:
        x.update({n + "_out": x[n] for n in ("mass", "kmin", "kmax") if n + "_out" not in kw})
    sc, dc = cache(a), cache(b)
    status = lib.sls_kv8_evict(ctypes.byref(DESC), ctypes.byref(sc), 1024, ctypes.byref(dc), 4, 1, 1, P(x["mass"]),
                             P(x["mass_out"]), P(x["kmin"]), P(x["kmax"]), P(x["kmin_out"]), P(x["kmax_out"]), P(x["kept"]),
                             P(x["ctx"]), P(x["ctx_out"]), None)
    assert b"memory" in lib.sls_last_error()  # refused for this reason (no call of this file may pass: it would be launched)
    return status


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_lists_and_lengths_are_memory_of_their_own(lib, in_place):
    """(The moving kernel reads the list as it is: a list overwritten on the way would lead out of the cache.)"""
    others = {**AT, **{n: X[n] for n in ("mass", "kmin", "kmax", "ctx", "ctx_out")}}
    if not in_place:
        others.update({n + " of dst": v for n, v in TO.items()})
        others.update({n: X[n] for n in ("mass_out", "kmin_out", "kmax_out")})
    for name, at in others.items():
        if name not in ("ctx", "ctx_out"):
            for own in ("kept", "ctx", "ctx_out"):
                assert evict(lib, in_place, **{own: at}) == L.SLS_EINVAL, (own, name)
        assert evict(lib, in_place, kept=at) == L.SLS_EINVAL, name
        assert evict(lib, in_place, kept=at - 60) == L.SLS_EINVAL, name  # 4 rows of 4 entries: the last one


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_buffers_do_not_share_memory(lib, in_place):
    for i, a in enumerate(NAMES):
        for b in NAMES[:i]:
            assert evict(lib, in_place, src={a: AT[b]}) == L.SLS_EINVAL, (a, b)
            assert evict(lib, in_place, src={a: AT[b] + SIZES[b] - 16}) == L.SLS_EINVAL, (a, b)
            if not in_place:
                assert evict(lib, in_place, dst={a: TO[b]}) == L.SLS_EINVAL, (a, b)
    assert evict(lib, in_place, kmax=X["kmin"]) == L.SLS_EINVAL
    assert evict(lib, in_place, mass=AT["k_scales"]) == L.SLS_EINVAL
    if not in_place:
        assert evict(lib, in_place, kmax_out=X["kmin_out"]) == L.SLS_EINVAL
        assert evict(lib, in_place, mass_out=TO["v_scales"] + 252) == L.SLS_EINVAL


def append(lib, src=None, **kw):
    x, c = {**X, **kw}, cache({**AT, **(src or {})})
    st = [8 * 256, 256, 128]
    status = lib.sls_kv8_append(ctypes.byref(DESC), ctypes.byref(c), P(x["k"]), *st, P(x["v"]), *st, 8, P(x["len"]),
                                P(x["kmin"]), P(x["kmax"]), P(x["mass"]), P(x["ctx"]), P(x["ctx_out"]), P(x["pos"]), None)
    assert b"memory" in lib.sls_last_error()
    return status


def test_append_buffers_do_not_share_memory(lib):
    for i, a in enumerate(NAMES):
        for b in NAMES[:i]:
            assert append(lib, {a: AT[b]}) == L.SLS_EINVAL, (a, b)
    for name in ("kmin", "kmax", "mass", "ctx_out", "pos"):
        for n, at in AT.items():
            assert append(lib, **{name: at + SIZES[n] - 16}) == L.SLS_EINVAL, (name, n)
        for other in ("kmin", "kmax", "mass", "ctx_out", "pos"):
            if other != name:
                assert append(lib, **{name: X[other]}) == L.SLS_EINVAL, (name, other)
    for name in ("ctx", "len"):
        for at in [*AT.values(), X["kmin"], X["kmax"], X["mass"]]:
            assert append(lib, **{name: at}) == L.SLS_EINVAL, name


def attend(lib, src=None, pages=False, **kw):
    x, c = {**X, **kw}, cache({**AT, **(src or {})})
    status = lib.sls_kv8_decode_attend(
        ctypes.byref(DESC), ctypes.byref(c), P(x["q"]), P(x["idx"]) if pages else None, 8, P(x["count"]) if pages else None, 8,
        P(x["ctx"]), P(x["sink"]), P(x["out"]), P(x["lse"]), None if pages else P(x["mass"]),
        None if pages else P(x["mass_out"]), P(x["ws"]), 1 << 40, None)
    assert b"memory" in lib.sls_last_error()
    return status


@pytest.mark.parametrize("pages", [False, True])
def test_attend_buffers_do_not_share_memory(lib, pages):
    for i, a in enumerate(NAMES):
        for b in NAMES[:i]:
            assert attend(lib, {a: AT[b]}, pages) == L.SLS_EINVAL, (a, b)
    read = ["q", "ctx", "sink"] + (["idx", "count"] if pages else ["mass"])
    written = ["out", "lse", "ws"] + ([] if pages else ["mass_out"])
    for name in written:
        for n, at in AT.items():
            assert attend(lib, None, pages, **{name: at + SIZES[n] - 16}) == L.SLS_EINVAL, (name, n)
        for other in read + written:
            if other != name and (name, other) != ("mass_out", "mass"):  # sums in place are allowed
                assert attend(lib, None, pages, **{name: X[other]}) == L.SLS_EINVAL, (name, other)
