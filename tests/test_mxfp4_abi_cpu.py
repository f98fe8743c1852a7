"""Refusals of the 4-bit cache's functions: on the host, before any CUDA work (runs without a GPU)."""
import ctypes
import os

import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300 import _lib

INV, MIS = _lib.EA_ERR_INVALID_ARG, _lib.EA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def h():
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_attention_long_gb300 import build
        build.build()
    return ea.lib()


def fake(struct, n=1, **over):
    """Aligned fake device pointers, all different: validation never follows them."""
    a = (struct * n)()
    for i in range(n):
        for j, (name, _) in enumerate(struct._fields_):
            setattr(a[i], name, 0x100000 * (i + 1) + 0x1000 * j)
        for k, v in over.items():
            setattr(a[i], k, v)
    return a


def rows(h, a, n=1, row0=0, n_rows=4, Smax=64, dtype=0, hs=512, rs=128, read=False):
    f = h.expert_attn_read_mxfp4 if read else h.expert_attn_write_mxfp4
    return f(a, n, row0, n_rows, Smax, dtype, hs, rs, None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw", [dict(n=0), dict(row0=-1), dict(n_rows=-1), dict(row0=61), dict(n_rows=65), dict(row0=2 ** 31 - 1),
                                dict(Smax=0, n_rows=0), dict(Smax=(1 << 22) + 1), dict(dtype=3), dict(dtype=-1),
                                dict(hs=-8), dict(rs=-128), dict(hs=1 << 41), dict(rs=1 << 41)])
def test_rows_bad_sizes(h, kw, read):
    assert rows(h, fake(_lib.EaMxfp4Rows), read=read, **kw) == INV


@pytest.mark.parametrize("read", [False, True])
def test_rows_bad_pointers(h, read):
    for name, _ in _lib.EaMxfp4Rows._fields_:
        assert rows(h, fake(_lib.EaMxfp4Rows, **{name: None}), read=read) == INV, name
        assert rows(h, fake(_lib.EaMxfp4Rows, **{name: 0x700008}), read=read) == MIS, name
    assert rows(h, None, read=read) == INV
    assert rows(h, fake(_lib.EaMxfp4Rows), hs=516, read=read) == MIS
    assert rows(h, fake(_lib.EaMxfp4Rows), rs=132, read=read) == MIS
    assert rows(h, fake(_lib.EaMxfp4Rows), dtype=2, hs=516, rs=132, read=read) != MIS  # 4-byte elements


def test_read_refuses_rows_that_overlap(h):
    a = fake(_lib.EaMxfp4Rows)
    for hs, rs in ((512, 64), (0, 128), (128, 128), (384, 128), (256, 1024), (0, 0)):
        assert rows(h, a, hs=hs, rs=rs, read=True) == INV, (hs, rs)
    for hs, rs in ((512, 128), (128, 1024), (1000, 128), (136, 1080)):
        assert rows(h, a, hs=hs, rs=rs, read=True) not in (INV, MIS), (hs, rs)
    assert rows(h, a, n_rows=1, hs=0, rs=0, read=True) == INV  # eight heads into one row


def test_one_cache_twice_is_refused(h):
    ws = ctypes.c_void_p(0x100000)
    for n, over in ((1, dict(k_codes=0x900000, v_codes=0x900000)), (2, dict(k_codes=0x900000)), (3, dict(v_codes=0x900000))):
        assert rows(h, fake(_lib.EaMxfp4Rows, n, **over), n=n) == INV
        a = fake(_lib.EaAttnMxfp4Args, n, **over)
        assert h.text_decode_attention_mxfp4(a, n, 10, 128, 0, ws, 1 << 40, None) == INV
        assert h.expert_attn_layers_mxfp4(a, n, 10, 128, 0, ws, 1 << 40, None) == INV


@pytest.mark.parametrize("fn", ["text_decode_attention_mxfp4", "expert_attn_layers_mxfp4"])
def test_attention_refusals(h, fn):
    f, ws = getattr(h, fn), ctypes.c_void_p(0x100000)
    call = lambda a=None, n=1, pos=10, Smax=128, delta=0, w=ws: f(  # noqa: E731
        fake(_lib.EaAttnMxfp4Args) if a is None else a, n, pos, Smax, delta, w, 1 << 40, None)
    last = 128 if "decode" in fn else 65
    for kw in (dict(n=0), dict(pos=-1), dict(pos=last), dict(Smax=64), dict(Smax=100), dict(Smax=(1 << 22) + 64),
               dict(delta=1 << 24), dict(delta=-(1 << 24) - 10), dict(delta=2 ** 31 - 1), dict(w=None)):
        assert call(**kw) == INV, kw
    assert call(w=ctypes.c_void_p(0x100010)) == MIS
    for name, _ in _lib.EaAttnMxfp4Args._fields_:
        want = INV if name not in ("k_new", "v_new") else None
        got = call(a=fake(_lib.EaAttnMxfp4Args, **{name: None}))
        assert (got == INV) if want else (got not in (INV, MIS)), name
        assert call(a=fake(_lib.EaAttnMxfp4Args, **{name: 0x700008})) == MIS, name


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    cache = ea.Mxfp4Cache(z(8, 64, 64), z(8, 64, 4), z(8, 64, 64), z(8, 64, 4))
    k = z(8, 4, 128, dt=torch.bfloat16)
    with pytest.raises(TypeError):
        ea.make_rows_args([ea.Mxfp4Rows(k, k, cache)], 64)
    q = z(64, 128, dt=torch.bfloat16)
    with pytest.raises(TypeError):
        ea.make_decode_mxfp4_args([ea.DecodeMxfp4Buffers(q, q[:8], q[:8], q[0], q[0], cache, q)], 64)
    for f in (ea.make_rows_args, ea.make_decode_mxfp4_args, ea.make_mxfp4_args):
        with pytest.raises(ValueError):
            f([], 64)


def test_scales_twice_are_refused(h):
    ws = ctypes.c_void_p(0x100000)
    for n, over in ((1, dict(k_scales=0x900000, v_scales=0x900000)), (2, dict(k_scales=0x900000)), (70, dict(v_scales=0x90000000))):
        assert rows(h, fake(_lib.EaMxfp4Rows, n, **over), n=n) == INV
        a = fake(_lib.EaAttnMxfp4Args, n, **over)
        assert h.text_decode_attention_mxfp4(a, n, 10, 128, 0, ws, 1 << 40, None) == INV
        assert h.expert_attn_layers_mxfp4(a, n, 10, 128, 0, ws, 1 << 40, None) == INV
    a = fake(_lib.EaAttnMxfp4Args, 70)
    assert h.text_decode_attention_mxfp4(a, 70, 10, 128, 0, ws, 1 << 40, None) not in (INV, MIS)


def test_rows_read_into_one_place_twice_are_refused(h):
    for n, over in ((1, dict(k=0x900000, v=0x900000)), (2, dict(k=0x900000)), (66, dict(v=0x90000000))):
        assert rows(h, fake(_lib.EaMxfp4Rows, n, **over), n=n, read=True) == INV
        assert rows(h, fake(_lib.EaMxfp4Rows, n, **over), n=n) not in (INV, MIS)  # a source may
    one = fake(_lib.EaMxfp4Rows, 2, k_codes=0x900000, k_scales=0xA00000)
    assert rows(h, one, n=2, read=True) not in (INV, MIS)  # as may a cache that is read


@pytest.mark.parametrize("fn,tok", [("text_decode_attention_mxfp4", 1), ("expert_attn_layers_mxfp4", 64)])
def test_positions_up_to_the_documented_ends(h, fn, tok):
    call = lambda p0: getattr(h, fn)(fake(_lib.EaAttnMxfp4Args), 1, 10, 128, p0 - 10, ctypes.c_void_p(0x100000), 1 << 40, None)  # noqa: E731
    last, first = (1 << 24) - tok, 1 - (1 << 24)
    assert call(last) not in (INV, MIS) and call(first) not in (INV, MIS)
    assert call(last + 1) == INV and call(first - 1) == INV
