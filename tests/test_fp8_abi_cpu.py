"""Refusals of the 8-bit cache's functions: on the host, before any CUDA work, and the binding's own (runs without a GPU)."""
import ctypes
import os

import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300 import _lib
from tests.test_mxfp4_abi_cpu import fake

INV, MIS = _lib.EA_ERR_INVALID_ARG, _lib.EA_ERR_MISALIGNED
WS = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def h():
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_attention_long_gb300 import build
        build.build()
    return ea.lib()


def rows(h, a, n=1, row0=0, n_rows=4, Smax=128, dtype=0, hs=512, rs=128, read=False):
    return (h.expert_attn_read_fp8 if read else h.expert_attn_write_fp8)(a, n, row0, n_rows, Smax, dtype, hs, rs, None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw", [dict(n=0), dict(row0=-1), dict(n_rows=-1), dict(row0=125), dict(n_rows=129), dict(row0=2 ** 31 - 1),
                                dict(Smax=0, n_rows=0), dict(Smax=64), dict(Smax=192), dict(Smax=(1 << 22) + 128), dict(dtype=3), dict(dtype=-1),
                                dict(hs=-8), dict(rs=-128), dict(hs=1 << 41), dict(rs=1 << 41)])
def test_rows_bad_sizes(h, kw, read):
    assert rows(h, fake(_lib.EaFp8Rows), read=read, **kw) == INV


@pytest.mark.parametrize("read", [False, True])
def test_rows_bad_pointers(h, read):
    for name, _ in _lib.EaFp8Rows._fields_:
        assert rows(h, fake(_lib.EaFp8Rows, **{name: None}), read=read) == INV, name
        assert rows(h, fake(_lib.EaFp8Rows, **{name: 0x700002}), read=read) == MIS, name
        ok = rows(h, fake(_lib.EaFp8Rows, **{name: 0x700004}), read=read)
        assert (ok not in (INV, MIS)) if "scale" in name else ok == MIS, name
    assert rows(h, None, read=read) == INV
    assert rows(h, fake(_lib.EaFp8Rows), hs=516, read=read) == MIS and rows(h, fake(_lib.EaFp8Rows), rs=132, read=read) == MIS
    assert rows(h, fake(_lib.EaFp8Rows), dtype=2, hs=516, rs=132, read=read) != MIS  # 4-byte elements


def test_read_refuses_rows_that_overlap(h):
    a = fake(_lib.EaFp8Rows)
    for hs, rs in ((512, 64), (0, 128), (128, 128), (384, 128), (256, 1024), (0, 0)):
        assert rows(h, a, hs=hs, rs=rs, read=True) == INV, (hs, rs)
    for hs, rs in ((512, 128), (128, 1024), (1000, 128), (136, 1080)):
        assert rows(h, a, hs=hs, rs=rs, read=True) not in (INV, MIS), (hs, rs)


def test_what_is_written_twice_is_refused(h):
    for n, over in ((1, dict(k_cache=0x900000, v_cache=0x900000)), (2, dict(k_cache=0x900000)), (3, dict(v_scale=0x900000)), (70, dict(k_scale=0x90000000))):
        assert rows(h, fake(_lib.EaFp8Rows, n, **over), n=n) == INV
        assert rows(h, fake(_lib.EaFp8Rows, n, **over), n=n, read=True) not in (INV, MIS)  # a cache that is read may
        assert h.text_decode_attention_fp8(fake(_lib.EaDecodeFp8Args, n, **over), n, 10, 128, 0, WS, 1 << 40, None) == INV
    for n, over in ((1, dict(k=0x900000, v=0x900000)), (2, dict(k=0x900000)), (66, dict(v=0x90000000))):
        assert rows(h, fake(_lib.EaFp8Rows, n, **over), n=n, read=True) == INV
        assert rows(h, fake(_lib.EaFp8Rows, n, **over), n=n) not in (INV, MIS)
    for name in ("out", "k_new", "v_new", "weight_out", "weight_in"):
        assert h.text_decode_attention_fp8(fake(_lib.EaDecodeFp8Args, 2, **{name: 0x900000}), 2, 10, 128, 0, WS, 1 << 40, None) == INV, name
    for name in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma"):  # inputs may be shared
        assert h.text_decode_attention_fp8(fake(_lib.EaDecodeFp8Args, 2, **{name: 0x900000}), 2, 10, 128, 0, WS, 1 << 40, None) not in (INV, MIS)
    for name in ("k_dst", "v_dst", "k_scale_dst", "v_scale_dst", "weight_dst", "kept"):
        assert evict(h, spread(2, **{name: 1 << 45}), n=2) == INV, name


def test_decode_refusals(h):
    f = h.text_decode_attention_fp8
    call = lambda a=None, n=1, pos=10, Smax=128, delta=0, w=WS: f(  # noqa: E731
        fake(_lib.EaDecodeFp8Args) if a is None else a, n, pos, Smax, delta, w, 1 << 40, None)
    for kw in (dict(n=0), dict(pos=-1), dict(pos=128), dict(Smax=64), dict(Smax=192), dict(Smax=(1 << 22) + 128),
               dict(delta=1 << 24), dict(delta=-(1 << 24) - 10), dict(delta=2 ** 31 - 1), dict(w=None)):
        assert call(**kw) == INV, kw
    assert call(w=ctypes.c_void_p(0x100010)) == MIS
    for name, _ in _lib.EaDecodeFp8Args._fields_:
        got = call(a=fake(_lib.EaDecodeFp8Args, **{name: None}))
        if name in ("k_new", "v_new", "weight_in"):
            assert got not in (INV, MIS), name
        else:  # (weight_out: with weight_in there)
            assert got == INV, name
        assert call(a=fake(_lib.EaDecodeFp8Args, **{name: 0x700002})) == MIS, name
    assert call(a=fake(_lib.EaDecodeFp8Args, weight_in=None, weight_out=None)) not in (INV, MIS)
    assert call(a=fake(_lib.EaDecodeFp8Args, weight_in=0x900000, weight_out=0x900000)) not in (INV, MIS)  # in place
    last = (1 << 24) - 1
    assert call(delta=last - 10) not in (INV, MIS) and call(delta=-last - 10) not in (INV, MIS)
    assert call(delta=last - 9) == INV and call(delta=-last - 11) == INV
    assert h.text_decode_fp8_workspace_size(0, 128, 0) == 0 and h.text_decode_fp8_workspace_size(1, 100, 0) == 0


def spread(n=1, **over):
    """Eviction's arrays, far enough apart for the largest caches."""
    a = (_lib.EaEvictFp8Args * n)()
    for i in range(n):
        for j, (name, _) in enumerate(_lib.EaEvictFp8Args._fields_):
            setattr(a[i], name, (1 << 40) * (i + 1) + (1 << 34) * j)
        for k, v in over.items():
            setattr(a[i], k, v)
    return a


def evict(h, a=None, n=1, rows=100, keep=60, first=4, recent=10, Smax=128, ws=WS):
    return h.expert_attn_evict_fp8(spread(n) if a is None else a, n, rows, keep, first, recent, Smax, ws, 1 << 40, None)


def test_evict_refusals(h):
    for kw in (dict(n=0), dict(rows=-1), dict(rows=129), dict(keep=-1), dict(keep=101), dict(first=-1), dict(recent=-1), dict(first=61),
               dict(first=51), dict(recent=57), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), dict(Smax=192), dict(Smax=0), dict(Smax=(1 << 22) + 128), dict(ws=None)):
        assert evict(h, **kw) == INV, kw
    assert evict(h, ws=ctypes.c_void_p(0x100010)) == MIS
    assert evict(h) not in (INV, MIS) and evict(h, keep=100) not in (INV, MIS) and evict(h, keep=14) not in (INV, MIS)
    for name, _ in _lib.EaEvictFp8Args._fields_:
        assert evict(h, spread(**{name: None})) == INV, name
        assert evict(h, spread(**{name: 0x700002})) == MIS, name
    assert h.expert_attn_evict_fp8_workspace_size(0, 128) == 0 and h.expert_attn_evict_fp8_workspace_size(1, 100) == 0


def test_evict_in_place_or_elsewhere(h):
    pairs = (("k_cache", "k_dst"), ("v_cache", "v_dst"), ("k_scale", "k_scale_dst"), ("v_scale", "v_scale_dst"), ("weight", "weight_dst"))
    a = spread()
    for s, d in pairs:
        setattr(a[0], d, getattr(a[0], s))
    assert evict(h, a) not in (INV, MIS)  # all five in place
    for s, d in pairs:  # one alone, all but one, one that overlaps
        assert evict(h, spread(**{d: getattr(spread()[0], s)})) == INV, d
        b = spread()
        for t, e in pairs:
            setattr(b[0], e, getattr(b[0], t) if e != d else (1 << 45))
        assert evict(h, b) == INV, d
        assert evict(h, spread(**{d: getattr(spread()[0], s) + 32})) == INV, d
    # one layer's destination is another's source
    b = spread(2)
    b[0].k_dst = b[1].k_cache
    assert evict(h, b, n=2) == INV


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    cache, k, q = ea.alloc_fp8_cache(128, "cpu"), z(8, 4, 128, dt=torch.bfloat16), z(64, 128, dt=torch.bfloat16)
    for make, layer in ((ea.make_fp8_rows_args, ea.Fp8Rows(k, k, cache)),
                        (ea.make_decode_fp8_args, ea.DecodeFp8Buffers(q, q[:8], q[:8], q[0], q[0], cache, q)),
                        (ea.make_evict_fp8_args, ea.EvictFp8Buffers(cache, z(8, 128, dt=torch.float32), z(8, 5, dt=torch.int32)))):
        with pytest.raises(TypeError):
            make([layer], 128)
        with pytest.raises(ValueError):
            make([], 128)
