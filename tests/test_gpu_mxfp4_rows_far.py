"""The 4-bit cache's writer and reader at offsets past 32 bits: the last rows of the largest cache, rows and heads further apart
than 2^31 bytes or elements."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
import oracle
from tests._mxfp4_util import DEV, quantise

pytestmark = pytest.mark.gpu


def stored(x: torch.Tensor) -> torch.Tensor:
    c, e = quantise(x.float().cpu().numpy())
    return torch.from_numpy(np.asarray(oracle.dequantize_rows(c, e)))


def test_the_largest_cache():
    Smax, n = 1 << 22, 5
    cache = ea.alloc_mxfp4_cache(Smax)
    k, v = (torch.randn(8, n, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(k, v, cache)], Smax - n, n, Smax)
    bk, bv = torch.empty_like(k), torch.empty_like(v)
    ea.expert_attn_read_mxfp4([ea.Mxfp4Rows(bk, bv, cache)], Smax - n, n, Smax)
    assert torch.equal(bk.cpu().double(), stored(k)) and torch.equal(bv.cpu().double(), stored(v))
    assert int(cache.k_codes[:, :Smax - n].count_nonzero()) == 0 and int(cache.v_scales[:, :Smax - n].count_nonzero()) == 0


@pytest.mark.parametrize("shape", [(1 << 30, 128), (128, 1 << 30)])  # strides of heads and rows, in elements
def test_rows_far_apart(shape):
    hs, rs = shape
    n = 3
    buf = torch.zeros(max(7 * hs + (n - 1) * rs, (n - 1) * rs + 7 * hs) + 128 + 4096, device=DEV, dtype=torch.bfloat16)
    k, v = (buf[i:].as_strided((8, n, 128), (hs, rs, 1)) for i in (0, 2048))
    src = [torch.randn(8, n, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    k.copy_(src[0])
    v.copy_(src[1])
    cache = ea.alloc_mxfp4_cache(64)
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(k, v, cache)], 7, n, 64)
    k.zero_()
    v.zero_()
    ea.expert_attn_read_mxfp4([ea.Mxfp4Rows(k, v, cache)], 7, n, 64)
    assert torch.equal(k.cpu().double(), stored(src[0])) and torch.equal(v.cpu().double(), stored(src[1]))
