"""The binding's checks of the 8-bit cache's marshalled arguments, with a library that only notes its calls (runs without a GPU)."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300 import _lib
from tests.test_mxfp4_binding_cpu import Ws, calls  # noqa: F401


def decode_args(Smax=128):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return ea.make_decode_fp8_args([ea.DecodeFp8Buffers(z(64, 128), z(8, 128), z(8, 128), z(128), z(128), ea.alloc_fp8_cache(Smax, "cpu"), z(64, 128))], Smax)


def evict_args(keep=50, Smax=128):
    return ea.make_evict_fp8_args([ea.EvictFp8Buffers(ea.alloc_fp8_cache(Smax, "cpu"), torch.zeros(8, Smax), torch.zeros(8, keep, dtype=torch.int32))], Smax)


def rows_args(maker="make_fp8_rows_args"):
    return _lib._Arr(maker, (_lib.EaFp8Rows * 1)(), [], None, 2, (512, 128), 4, 128)


def test_calls_reach_the_library(calls):  # noqa: F811
    ea.text_decode_attention_fp8(None, 10, 128, 0, Ws, _arr=decode_args())
    ea.expert_attn_evict_fp8(None, 100, 50, 4, 10, 128, Ws, _arr=evict_args())
    ea.expert_attn_write_fp8(None, 0, 4, 128, _arr=rows_args())
    ea.expert_attn_read_fp8(None, 0, 4, 128, _arr=rows_args())
    assert calls == ["text_decode_attention_fp8", "expert_attn_evict_fp8", "expert_attn_write_fp8", "expert_attn_read_fp8"]


def test_arguments_of_another_call_are_refused(calls):  # noqa: F811
    for f in (lambda: ea.text_decode_attention_fp8(None, 10, 128, 0, Ws, _arr=evict_args()),
              lambda: ea.text_decode_attention_mxfp4(None, 10, 128, 0, Ws, _arr=decode_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 50, 4, 10, 128, Ws, _arr=decode_args()),
              lambda: ea.expert_attn_write_fp8(None, 0, 4, 128, _arr=rows_args("make_rows_args")),
              lambda: ea.expert_attn_write_mxfp4(None, 0, 4, 128, _arr=rows_args())):
        with pytest.raises(TypeError, match="expected"):
            f()
    assert calls == []


def test_sizes_that_do_not_fit_the_arguments_are_refused(calls):  # noqa: F811
    for f in (lambda: ea.text_decode_attention_fp8(None, 10, 256, 0, Ws, _arr=decode_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 50, 4, 10, 256, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 51, 4, 10, 128, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 49, 4, 10, 128, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_write_fp8(None, 0, 5, 128, _arr=rows_args())):
        with pytest.raises(ValueError):
            f()
    assert calls == []


@pytest.mark.parametrize("far", [1 << 31, (1 << 32) + 3, -(1 << 32) + 3])
def test_numbers_past_32_bits_are_refused(calls, far):  # noqa: F811
    for f in (lambda: ea.text_decode_attention_fp8(None, far, 128, 0, Ws, _arr=decode_args()),
              lambda: ea.text_decode_attention_fp8(None, 10, 128, far, Ws, _arr=decode_args()),
              lambda: ea.expert_attn_evict_fp8(None, far, 50, 4, 10, 128, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 50, far, 10, 128, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_evict_fp8(None, 100, 50, 4, far, 128, Ws, _arr=evict_args()),
              lambda: ea.expert_attn_write_fp8(None, far, 1, 128, _arr=rows_args()),
              lambda: ea.expert_attn_read_fp8(None, far, 1, 128, _arr=rows_args())):
        with pytest.raises(ValueError):
            f()
    assert calls == []
