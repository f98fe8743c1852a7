"""The binding's checks of marshalled arguments, with a library that only notes its calls (runs without a GPU)."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300 import _lib


class Ws:
    """A workspace on the same (missing) device as CPU tensors."""
    dtype = torch.uint8
    get_device = staticmethod(lambda: None)
    is_contiguous = staticmethod(lambda: True)
    data_ptr = numel = staticmethod(lambda: 1 << 20)


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(_lib, "_lib_handle", Lib())
    monkeypatch.setattr(_lib, "_device_now", lambda: None)
    monkeypatch.setattr(_lib, "_stream_now", lambda d: 0)
    monkeypatch.setattr(_lib, "_ptr", lambda t, name, dtype=None, numel=None: None if t is None else t.data_ptr())
    return seen


def bufs(cls, hq, tok, Smax=128):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return cls(z(hq, tok, 128), z(8, tok, 128), z(8, tok, 128), z(128), z(128), ea.alloc_mxfp4_cache(Smax, "cpu"), z(hq, tok, 128))


def test_arguments_of_one_attention_are_refused_by_the_other(calls):
    """Both are arrays of the same struct: a decode step's, given to the expert, would have it read 64 rows where there is one."""
    dec = ea.make_decode_mxfp4_args([bufs(ea.DecodeMxfp4Buffers, 64, 1)], 128)
    exp = ea.make_mxfp4_args([bufs(ea.LayerMxfp4Buffers, 16, 64)], 128)
    with pytest.raises(TypeError, match="make_mxfp4_args"):
        ea.expert_attn_layers_mxfp4(None, 10, 128, 0, Ws, _arr=dec)
    with pytest.raises(TypeError, match="make_decode_mxfp4_args"):
        ea.text_decode_attention_mxfp4(None, 10, 128, 0, Ws, _arr=exp)
    for f in (ea.expert_attn_write_mxfp4, ea.expert_attn_read_mxfp4):
        with pytest.raises(TypeError, match="make_rows_args"):
            f(None, 0, 1, 128, _arr=exp)
    assert calls == []
    ea.text_decode_attention_mxfp4(None, 10, 128, 0, Ws, _arr=dec)
    ea.expert_attn_layers_mxfp4(None, 10, 128, 0, Ws, _arr=exp)
    assert calls == ["text_decode_attention_mxfp4", "expert_attn_layers_mxfp4"]


def test_arguments_for_another_cache_length_are_refused(calls):
    dec = ea.make_decode_mxfp4_args([bufs(ea.DecodeMxfp4Buffers, 64, 1)], 128)
    with pytest.raises(ValueError, match="128 rows"):
        ea.text_decode_attention_mxfp4(None, 10, 192, 0, Ws, _arr=dec)
    assert calls == []


@pytest.mark.parametrize("far", [1 << 31, (1 << 32) + 3, -(1 << 32) + 3])
def test_numbers_past_32_bits_are_refused(calls, far):
    """ctypes would cut them: row 2^32 + 3 is not row 3."""
    dec = ea.make_decode_mxfp4_args([bufs(ea.DecodeMxfp4Buffers, 64, 1)], 128)
    exp = ea.make_mxfp4_args([bufs(ea.LayerMxfp4Buffers, 16, 64)], 128)
    z = torch.zeros(8, 4, 128)
    c = ea.alloc_mxfp4_cache(128, "cpu")
    a = _lib._Arr("make_rows_args", (_lib.EaMxfp4Rows * 1)(), [z, c], None, 2, (512, 128), 4, 128)
    for f in (lambda: ea.text_decode_attention_mxfp4(None, far, 128, 0, Ws, _arr=dec),
              lambda: ea.text_decode_attention_mxfp4(None, 10, 128, far, Ws, _arr=dec),
              lambda: ea.expert_attn_layers_mxfp4(None, far, 128, 0, Ws, _arr=exp),
              lambda: ea.expert_attn_layers_mxfp4(None, 10, 128, far, Ws, _arr=exp),
              lambda: ea.expert_attn_write_mxfp4(None, far, 1, 128, _arr=a),
              lambda: ea.expert_attn_read_mxfp4(None, far, 1, 128, _arr=a),
              lambda: ea.expert_attn_write_mxfp4(None, 0, -abs(far) - 1, 128, _arr=a)):
        with pytest.raises(ValueError, match="32 bits"):
            f()
    assert calls == []
