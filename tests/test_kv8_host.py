"""Refusals of the norm/rotation and 8-bit cache calls: host-side checks, no kernel runs."""
import ctypes

import pytest
import torch

from sparse_long_context_gb300 import _lib as L
from sparse_long_context_gb300 import ops

P = lambda x: ctypes.c_void_p(x)  # noqa: E731  never dereferenced: validation fails first
A = P(0x10000)


def desc(**kw):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, capacity=1024,
             dtype=L.SLS_DTYPE_BF16, flags=0, scale=0.0)
    d.update(kw)
    return L.AttnDesc(**d)


def cache(at=1 << 20, fmt=0, block=64, **kw):
    c = dict(k_codes=at, v_codes=at + (1 << 24), k_scales=at + (2 << 24), v_scales=at + (3 << 24),
             k_tail=at + (4 << 24), v_tail=at + (5 << 24))
    c.update(kw)
    return L.Kv8CacheDesc(fmt, block, *(c[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales", "k_tail", "v_tail")))


def rope_call(lib, n=4, q=A, k=A, qs=(1024, 128), ks=(256, 128), pos=A, qo=A, qos=(1024, 128), ko=A, kos=(256, 128),
              w=None, **kw):
    r = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, rotary_dim=128, interleaved=0, dtype=1, eps=1e-6, theta=1e4)
    r.update(kw)
    d = L.RopeDesc(**r)
    return lib.sls_qk_norm_rope(ctypes.byref(d), n, q, *qs, k, *ks, w, None, pos, qo, *qos, ko, *kos, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_q_heads=-1), L.SLS_EINVAL), (dict(num_q_heads=0, num_kv_heads=0), L.SLS_EINVAL),
    (dict(head_dim=96), L.SLS_EUNSUPPORTED), (dict(rotary_dim=24), L.SLS_EUNSUPPORTED),
    (dict(rotary_dim=144), L.SLS_EUNSUPPORTED), (dict(rotary_dim=-16), L.SLS_EUNSUPPORTED),
    (dict(interleaved=2), L.SLS_EINVAL), (dict(dtype=9), L.SLS_EUNSUPPORTED), (dict(eps=-1.0), L.SLS_EINVAL),
    (dict(eps=float("nan")), L.SLS_EINVAL), (dict(theta=0.0), L.SLS_EINVAL), (dict(theta=float("inf")), L.SLS_EINVAL),
    (dict(n=-1), L.SLS_EINVAL), (dict(q=None), L.SLS_EINVAL), (dict(k=None), L.SLS_EINVAL), (dict(pos=None), L.SLS_EINVAL),
    (dict(qo=None), L.SLS_EINVAL), (dict(q=P(0x10002)), L.SLS_EINVAL), (dict(w=P(0x10008)), L.SLS_EINVAL),
    (dict(qs=(1023, 128)), L.SLS_EINVAL), (dict(qs=(-1024, 128)), L.SLS_EINVAL),
    (dict(qos=(512, 128)), L.SLS_EINVAL),      # tokens' outputs overlap
    (dict(qos=(1024, 64)), L.SLS_EINVAL),      # heads' outputs overlap
    (dict(kos=(0, 128)), L.SLS_EINVAL),
])
def test_rope_refusals(lib, kw, code):
    assert rope_call(lib, **kw) == code
    assert lib.sls_last_error()


def test_rope_null_desc_and_no_tokens(lib):
    assert lib.sls_qk_norm_rope(None, 1, A, 0, 0, A, 0, 0, None, None, A, A, 0, 0, A, 0, 0, None) == L.SLS_EINVAL
    assert rope_call(lib, n=0, q=None, k=None, pos=None) == L.SLS_OK  # nothing to do


@pytest.mark.parametrize("d,c,code", [
    (dict(dtype=L.SLS_DTYPE_F32), {}, L.SLS_EUNSUPPORTED), (dict(head_dim=32), {}, L.SLS_EUNSUPPORTED),
    ({}, dict(fmt=2), L.SLS_EUNSUPPORTED), ({}, dict(block=8), L.SLS_EINVAL), ({}, dict(block=48), L.SLS_EINVAL),
    ({}, dict(block=512), L.SLS_EINVAL), (dict(capacity=1040), {}, L.SLS_EINVAL), ({}, dict(k_codes=0), L.SLS_EINVAL),
    ({}, dict(v_tail=0), L.SLS_EINVAL), ({}, dict(v_codes=(1 << 20) + 8), L.SLS_EINVAL),
    ({}, dict(k_tail=(1 << 20) + 8), L.SLS_EINVAL), ({}, dict(k_scales=(1 << 20) + 2), L.SLS_EINVAL),
])
def test_cache_refusals_in_every_call(lib, d, c, code):
    dd, cc = desc(**d), cache(**c)
    st = [2048, 256, 128]
    assert lib.sls_kv8_append(ctypes.byref(dd), ctypes.byref(cc), A, *st, A, *st, 4, None, None, None, None, A, A, None,
                              None) == code
    assert lib.sls_kv8_decode_attend(ctypes.byref(dd), ctypes.byref(cc), A, None, 0, None, 0, A, None, A, None, None,
                                     None, A, 1 << 40, None) == code
    assert lib.sls_kv8_decode_attend_workspace_size(ctypes.byref(dd), ctypes.byref(cc), 1) == 0
    assert lib.sls_kv8_evict(ctypes.byref(dd), ctypes.byref(cc), dd.capacity, None, 4, 0, 0, A, A, None, None, None,
                             None, A, A, A, None) == code


def append(lib, dd=None, st=(2048, 256, 128), new=4, k=A, kmin=None, kmax=None, ctx=A, out=A, v=A, n=None, pos=None):
    dd = dd or desc()
    c = cache()
    return lib.sls_kv8_append(ctypes.byref(dd), ctypes.byref(c), k, *st, v, *st, new, n, kmin, kmax, None, ctx, out,
                              pos, None)


def test_append_refusals(lib):
    assert append(lib, new=-1) == L.SLS_EINVAL
    assert append(lib, k=None) == L.SLS_EINVAL
    assert append(lib, v=P(0x10008)) == L.SLS_EINVAL
    assert append(lib, ctx=None) == L.SLS_EINVAL
    assert append(lib, out=None) == L.SLS_EINVAL
    assert append(lib, st=(2048, 250, 128)) == L.SLS_EINVAL
    assert append(lib, st=(-2048, 256, 128)) == L.SLS_EINVAL
    assert append(lib, kmin=A) == L.SLS_EINVAL
    assert append(lib, dd=desc(page_size=1), kmin=A, kmax=A) == L.SLS_EINVAL
    assert append(lib, dd=desc(batch=1 << 20), new=1 << 20) == L.SLS_EOVERFLOW
    assert append(lib, dd=desc(batch=1, num_q_heads=1, num_kv_heads=1, capacity=(1 << 30) + 64)) == L.SLS_EUNSUPPORTED
    assert append(lib, out=P(0x10004)) == L.SLS_EINVAL                     # partly ctx_len's memory
    assert append(lib, out=P(0x20000), n=P(0x20004)) == L.SLS_EINVAL
    assert append(lib, pos=A) == L.SLS_EINVAL
    assert append(lib, out=P(0x20000), pos=P(0x20004)) == L.SLS_EINVAL


def attend(lib, dd=None, q=A, idx=None, stride=0, count=None, k=0, ctx=A, out=P(0x80000), mi=None, mo=None, ws=A, wsb=1 << 40):
    dd = dd or desc()
    c = cache()
    return lib.sls_kv8_decode_attend(ctypes.byref(dd), ctypes.byref(c), q, idx, stride, count, k, ctx, None, out, None, mi,
                                     mo, ws, wsb, None)


def test_attend_refusals(lib):
    assert attend(lib, q=None) == L.SLS_EINVAL
    assert attend(lib, ctx=None) == L.SLS_EINVAL
    assert attend(lib, out=P(0x10004)) == L.SLS_EINVAL
    assert attend(lib, dd=desc(flags=L.SLS_FLAG_CUDA_CORES)) == L.SLS_EUNSUPPORTED
    assert attend(lib, dd=desc(flags=L.SLS_FLAG_NO_TMA)) == L.SLS_EUNSUPPORTED
    assert attend(lib, dd=desc(batch=4097, num_q_heads=1, num_kv_heads=1)) == L.SLS_EUNSUPPORTED
    assert attend(lib, dd=desc(batch=2048, capacity=1 << 20)) == L.SLS_EUNSUPPORTED   # 2^32 cache slots
    assert attend(lib, dd=desc(page_size=8), idx=A, stride=4, k=4) == L.SLS_EUNSUPPORTED
    assert attend(lib, idx=A, stride=0) == L.SLS_EINVAL
    assert attend(lib, idx=A, stride=4, k=5) == L.SLS_EINVAL
    assert attend(lib, idx=A, stride=1 << 28, k=1) == L.SLS_EOVERFLOW
    assert attend(lib, idx=A, stride=4, k=4, mo=A) == L.SLS_EUNSUPPORTED
    assert attend(lib, mi=A) == L.SLS_EINVAL
    assert attend(lib, mi=P(0x100000), mo=P(0x100004)) == L.SLS_EINVAL     # partly the same memory
    assert attend(lib, q=P(0x100000), out=P(0x100010)) == L.SLS_EINVAL
    need = lib.sls_kv8_decode_attend_workspace_size(ctypes.byref(desc()), ctypes.byref(cache()), 0)
    with_mass = lib.sls_kv8_decode_attend_workspace_size(ctypes.byref(desc()), ctypes.byref(cache()), 1)
    assert 0 < need < with_mass
    assert attend(lib, ws=None) == L.SLS_EWORKSPACE
    assert attend(lib, wsb=need - 1) == L.SLS_EWORKSPACE
    assert attend(lib, mo=A, wsb=with_mass - 1) == L.SLS_EWORKSPACE
    assert attend(lib, ws=P(0x10008)) == L.SLS_EINVAL


def evict(lib, dst=None, dcap=1024, keep=4, sink=1, recent=1, mass=A, mass_out=A, km=(None,) * 4, kept=A, ctx=A, out=A,
          dd=None, src=None):
    dd, c = dd or desc(), src or cache()
    return lib.sls_kv8_evict(ctypes.byref(dd), ctypes.byref(c), dcap, None if dst is None else ctypes.byref(dst), keep,
                             sink, recent, mass, mass_out, *km, kept, ctx, out, None)


def test_evict_refusals(lib):
    far = 1 << 30
    for kw in (dict(keep=0), dict(sink=-1), dict(keep=4, sink=2, recent=3), dict(keep=16), dict(mass=None), dict(kept=None),
               dict(ctx=None), dict(out=None), dict(out=P(0x10004)), dict(mass_out=P(0x20000)), dict(mass_out=None), dict(dcap=512),
               dict(km=(A, None, None, None)), dict(km=(A, A, P(0x30000), A)),
               dict(dst=cache(fmt=1), dcap=1024), dict(dst=cache(far, block=32)), dict(dst=cache(far), dcap=1000),
               dict(dst=cache(far), dcap=256, keep=4),
               dict(dst=cache(far, v_codes=1 << 20)),                      # shares memory with the source
               dict(dst=cache((1 << 20) + 4096), mass_out=P(far)),         # overlaps it
               dict(dst=cache(far), mass_out=A)):                          # sums over the ones being read
        assert evict(lib, **kw) == L.SLS_EINVAL, kw
        assert lib.sls_last_error()
    pages = (P(0x40000000), P(0x41000000), P(0x42000000), P(0x43000000))
    assert evict(lib, dd=desc(page_size=128), dst=cache(1 << 31), mass_out=P(0x50000000), km=pages) == L.SLS_EUNSUPPORTED


def test_binding_refuses_host_tensors_and_bad_shapes():
    d = ops.make_desc(1, 2, 1, 64, 16, 64, torch.bfloat16)
    z = torch.zeros((1, 1, 64, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.Kv8Cache(d, "int8", 16, z, z, z, z, z, z)
    with pytest.raises(ValueError):
        ops.Kv8Cache(d, "int4", 16, z, z, z, z, z, z)
    with pytest.raises(ValueError):
        ops.make_rope(1, 1, 64, torch.bfloat16, rotary_dim=32, inv_freq=[1.0])
    rope = ops.make_rope(1, 1, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(rope, torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32))


def test_cache_of_another_shape_is_refused():
    """A cache is used with the shape it was made for: a larger descriptor would reach past its buffers."""
    cache = object.__new__(ops.Kv8Cache)  # without a GPU there are no buffers; the check comes before they are used
    cache.index, cache.shape, cache.c = -1, (2, 1, 64, 64), L.Kv8CacheDesc()
    x = torch.zeros((2, 1, 1, 64), dtype=torch.bfloat16)
    ctx = torch.zeros(2, dtype=torch.int32)
    for b, h, cap, d in ((2, 1, 128, 64), (3, 1, 64, 64), (2, 2, 64, 64), (2, 1, 64, 128)):
        wrong = ops.make_desc(b, 2, h, d, 16, cap, torch.bfloat16)
        with pytest.raises(ValueError, match="shape is not that of the cache"):
            ops.kv8_append(wrong, cache, x, x, ctx)
        with pytest.raises(ValueError, match="shape is not that of the cache"):
            ops.kv8_decode_attend(wrong, cache, x[:, 0], ctx, out=x, lse=ctx, workspace=ctx)
        with pytest.raises(ValueError, match="shape is not that of the cache"):
            ops.kv8_evict(wrong, cache, ctx, x, 1)
        right = ops.make_desc(2, 2, 1, 64, 16, 64, torch.bfloat16)
        if (b, h, d) == (2, 1, 64):
            with pytest.raises(ValueError, match="shape is not that of the cache"):
                ops.kv8_evict(right, cache, ctx, x, 1, dst_desc=wrong, dst=cache)
