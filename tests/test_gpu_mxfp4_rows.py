"""GPU parity of the 4-bit cache's writer and reader (expert_attn_write_mxfp4, expert_attn_read_mxfp4).
Both are exact: the codes and exponents equal the oracle quantiser's, the values read back equal
code * 2^e (rounded once to fp16), and no other byte changes."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
import oracle
from tests._mxfp4_util import DEV, quantise, random_cache, unpacked

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _rows(seed, n, dtype, order, wide=True):
    """k and v [8, n, 128] on the device: head-major, or columns of a fused [n][extra | k | v] buffer."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, 8, n, 128))
    if wide and dtype is not FP16:
        x *= np.exp2(rng.integers(-20, 20, (2, 8, n, 4))).repeat(32, -1)
    x[0, 0, 0, :32] = 0.0                                                    # an all-zero block
    x[0, 3, n - 1, 32:64] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * 2.0 ** -3  # ties
    x[1, 2, n // 2] *= -0.0                                                  # negative zeros
    if dtype is not FP16:
        x[1, 7, 0, 64:96] *= 2.0 ** -133                                     # subnormals: exponent clamped
    t = torch.from_numpy(x).to(FP32).to(dtype)
    if order == "head":
        return [a.to(DEV) for a in t]
    fused = torch.full((n, 3 * 1024), 99.0, dtype=dtype, device=DEV)
    for i in range(2):
        fused[:, 1024 * (i + 1):1024 * (i + 2)] = t[i].transpose(0, 1).reshape(n, 1024).to(DEV)
    return [fused[:, 1024 * (i + 1):1024 * (i + 2)].view(n, 8, 128).transpose(0, 1) for i in range(2)]


def _untouched(before, after, row0, n):
    keep = [r for r in range(before.shape[1]) if not row0 <= r < row0 + n]
    assert torch.equal(before[:, keep].cpu(), after[:, keep].cpu())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("row0,n,Smax,order", [(0, 1, 1, "head"), (5, 1, 64, "token"), (3, 17, 20, "head"), (64, 64, 128, "token"),
                                               (1, 333, 512, "token"), (0, 1000, 1000, "head")])
def test_rows_written_bit_exact(dtype, row0, n, Smax, order):
    k, v = _rows(row0 + n, n, dtype, order)
    cache = random_cache(1, Smax, 0).device()
    before = [t.clone() for t in cache.__dict__.values()]
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(k, v, cache)], row0, n, Smax)
    torch.cuda.synchronize()
    for src, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        want_c, want_e = quantise(src.float().cpu().numpy())
        got_c, got_e = unpacked(codes[:, row0:row0 + n], scales[:, row0:row0 + n])
        assert np.array_equal(got_e, want_e) and np.array_equal(got_c, want_c)
    for a, b in zip(before, cache.__dict__.values()):
        _untouched(a, b, row0, n)


def test_rows_written_like_the_whole_cache_quantiser():
    # bf16 rows, infinities and NaN among them: byte for byte what expert_attn_quantize_cache_mxfp4 makes
    Smax = 192
    k, v = _rows(7, Smax, BF16, "head")
    k[1, 4, 7], k[1, 4, 99], v[0, 9, 3], v[0, 9, 4] = float("inf"), float("nan"), float("-inf"), float("nan")
    v[5, 5, 32:64] = float("nan")
    cache = ea.alloc_mxfp4_cache(Smax)
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(k, v, cache)], 0, Smax, Smax)
    for src, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        c, s = torch.empty_like(codes), torch.empty_like(scales)
        ea.expert_attn_quantize_cache_mxfp4(src.contiguous(), Smax, Smax, c, s)
        assert torch.equal(c, codes) and torch.equal(s, scales)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("row0,n,Smax,order", [(0, 1, 1, "head"), (5, 1, 64, "token"), (3, 17, 20, "head"), (1, 333, 512, "token")])
def test_rows_read_back_exact(dtype, row0, n, Smax, order):
    c = random_cache(11, Smax, Smax, k_gain=3.0, v_gain=2.0 ** -9)
    k, v = (torch.full_like(t, 55.0) for t in _rows(1, n + 2, dtype, "head")) if order == "head" else _rows(1, n + 2, dtype, order)
    guard = [t[:, n:].clone() for t in (k, v)]
    ea.expert_attn_read_mxfp4([ea.Mxfp4Rows(k, v, c.device())], row0, n, Smax)
    torch.cuda.synchronize()
    for got, (codes, exps), g in ((k, c.k, guard[0]), (v, c.v, guard[1])):
        want = torch.from_numpy(oracle.dequantize_rows(codes[:, row0:row0 + n], exps[:, row0:row0 + n]))
        assert torch.equal(got[:, :n].cpu().double(), want.to(dtype).double())
        assert torch.equal(got[:, n:], g)  # rows past n are not written


def test_every_code_and_scale_read_back():
    # all 16 codes under all 255 numeric scale bytes, and NaN for 255
    codes = torch.arange(256, dtype=torch.uint8).repeat(8, 256, 1)[:, :, :64].contiguous()
    for r in range(256):
        codes[:, r] = torch.arange(64, dtype=torch.uint8) + 64 * (r % 4)
    scales = torch.arange(256, dtype=torch.uint8)[None, :, None].expand(8, 256, 4).contiguous()
    cache = ea.Mxfp4Cache(codes.to(DEV), scales.to(DEV), codes.to(DEV), scales.to(DEV))
    k, v = (torch.empty(8, 256, 128, device=DEV) for _ in range(2))
    ea.expert_attn_read_mxfp4([ea.Mxfp4Rows(k, v, cache)], 0, 256, 256)
    c, e = unpacked(codes, scales)
    want = torch.from_numpy(oracle.dequantize_rows(c[:, :255], e[:, :255])).float()
    assert torch.equal(k[:, :255].cpu(), want) and torch.equal(v[:, :255].cpu(), want)
    assert torch.isnan(k[:, 255]).all()


def test_many_layers_in_one_call_and_over_64():
    n, Smax = 70, 64
    src = [_rows(100 + l, 2, BF16, "head") for l in range(n)]
    caches = [ea.alloc_mxfp4_cache(Smax) for _ in range(n)]
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(k, v, c) for (k, v), c in zip(src, caches)], 30, 2, Smax)
    back = [[torch.empty_like(t) for t in kv] for kv in src]
    ea.expert_attn_read_mxfp4([ea.Mxfp4Rows(k, v, c) for (k, v), c in zip(back, caches)], 30, 2, Smax)
    for kv, b in zip(src, back):
        for x, y in zip(kv, b):
            c, e = quantise(x.float().cpu().numpy())
            assert np.array_equal(y.double().cpu().numpy(), oracle.dequantize_rows(c, e))


def test_one_source_row_for_every_head():
    # a source may repeat (stride 0): the same row for all heads
    row = torch.randn(1, 1, 128, device=DEV, dtype=FP32)
    cache = ea.alloc_mxfp4_cache(64)
    x = row.expand(8, 1, 128)
    ea.expert_attn_write_mxfp4([ea.Mxfp4Rows(x, x, cache)], 63, 1, 64)
    assert (cache.k_codes[:, 63] == cache.k_codes[:1, 63]).all() and torch.equal(cache.k_codes, cache.v_codes)


def test_rows_captured_in_a_graph():
    Smax, n = 128, 5
    k, v = _rows(3, n, BF16, "token")
    cache = ea.alloc_mxfp4_cache(Smax)
    bk, bv = (torch.zeros(8, n, 128, dtype=BF16, device=DEV) for _ in range(2))
    src, dst = ea.make_rows_args([ea.Mxfp4Rows(k, v, cache)], Smax), ea.make_rows_args([ea.Mxfp4Rows(bk, bv, cache)], Smax)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ea.expert_attn_write_mxfp4(None, 7, n, Smax, _arr=src)
        ea.expert_attn_read_mxfp4(None, 7, n, Smax, _arr=dst)
    k.mul_(2.0)  # the replay reads what the tensors hold then
    g.replay()
    c, e = quantise(k.float().cpu().numpy())
    assert np.array_equal(bk.double().cpu().numpy(), oracle.dequantize_rows(c, e))
