"""The 8-bit cache's writer and reader on the GPU: codes and scales bit for bit against the rule written out on the host, rows
read back exactly, at sizes that begin, fill and cross blocks."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV, F32, HostCache, random_cache, same_cache

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def rows(seed, n, dtype, order="head", gain=1.0):
    x = torch.from_numpy((np.random.default_rng(seed).standard_normal((8, n, 128)) * gain).astype(F32)).to(dtype)
    return x if order == "head" else x.transpose(0, 1).contiguous().transpose(0, 1)


def write(cache, k, v, row0, Smax):
    ea.expert_attn_write_fp8([ea.Fp8Rows(k.to(DEV), v.to(DEV), cache)], row0, k.shape[1], Smax)


def host_write(h, k, v, row0):
    h.append(0, k.float().numpy(), row0)
    h.append(1, v.float().numpy(), row0)


def read(cache, row0, n, Smax, dtype):
    k, v = (torch.full((8, n, 128), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    ea.expert_attn_read_fp8([ea.Fp8Rows(k, v, cache)], row0, n, Smax)
    return k, v


def values(h, i, row0, n, dtype):
    """What the reader gives: the fp32 product, rounded to the rows' type."""
    x = h.values(i, row0 + n)[:, row0:]
    return torch.from_numpy(x.astype(F32)).to(dtype)


@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("row0,n,Smax", [(0, 1, 128), (0, 128, 128), (0, 129, 256), (1, 1, 128), (127, 1, 128), (127, 2, 256),
                                         (128, 5, 384), (77, 300, 512), (300, 84, 384), (250, 261, 640)])
def test_append(row0, n, Smax, dtype, order):
    h = random_cache(row0 + n, Smax, row0)
    cache = h.device()
    k, v = rows(1, n, dtype, order, 2.0), rows(2, n, dtype, order, 0.5)  # K's need larger scales, V's do not
    write(cache, k, v, row0, Smax)
    host_write(h, k, v, row0)
    same_cache(cache, h)
    first = row0 // 128 * 128
    for back in DTYPES:
        got = read(cache, first, row0 + n - first, Smax, back)
        for i in range(2):
            assert torch.equal(got[i].cpu(), values(h, i, first, row0 + n - first, back))


def test_a_row_at_a_time_gives_what_the_rule_says():
    """A block filled row by row, each row twice the size of the last at first: its scale grows, its codes move."""
    h, Smax = HostCache(256), 256
    cache = h.device()
    for r in range(140):
        gain = 2.0 ** min(r, 30) * 1e-4
        k, v = rows(r, 1, torch.float32, gain=gain), rows(1000 + r, 1, torch.float32, gain=1.0)
        write(cache, k, v, r, Smax)
        host_write(h, k, v, r)
    same_cache(cache, h)


def test_values_survive_a_growing_scale():
    """Doubling a scale changes no value but those among the subnormals, which move by at most half of 2^-9 of it."""
    Smax = 128
    cache = HostCache(Smax).device()
    k = rows(3, 64, torch.float32)
    write(cache, k, k, 0, Smax)
    before, s0 = read(cache, 0, 64, Smax, torch.float32)[0].cpu(), cache.k_scale[:, 0].cpu()
    write(cache, rows(4, 1, torch.float32, gain=40.0), rows(5, 1, torch.float32), 64, Smax)
    after, s1 = read(cache, 0, 64, Smax, torch.float32)[0].cpu(), cache.k_scale[:, 0].cpu()
    assert (s1 > s0).all()
    normal = before.abs() >= s1[:, None, None] * 2.0 ** -6
    assert torch.equal(before[normal], after[normal]) and normal.float().mean() > 0.9
    assert ((after - before).abs() <= s1[:, None, None] * 2.0 ** -10).all()


@pytest.mark.parametrize("gain", [1e-37, 1e-29, 1e-20, 1e20, 1e37, 3e38])
def test_magnitudes_from_end_to_end(gain):
    x = torch.from_numpy(np.clip(np.random.default_rng(5).standard_normal((8, 130, 128)) * gain, -3.4e38, 3.4e38).astype(F32))
    h = HostCache(256)
    cache = h.device()
    write(cache, x, x, 0, 256)
    host_write(h, x, x, 0)
    same_cache(cache, h)
    assert torch.isfinite(read(cache, 0, 130, 256, torch.float32)[0]).all()


def test_zeros_infinities_and_nan():
    x = rows(6, 20, torch.bfloat16).clone()
    x[0] = 0
    x[1, 3, 5], x[1, 4, 6] = float("inf"), -float("inf")
    x[2, 7, 9] = float("nan")
    x[3] = float("nan")
    h = HostCache(128)
    cache = h.device()
    write(cache, x, x, 0, 128)
    host_write(h, x, x, 0)
    same_cache(cache, h)
    got = read(cache, 0, 20, 128, torch.float32)[0].cpu()
    assert (got[0] == 0).all() and got[1, 3, 5] > 1e38 and got[1, 4, 6] < -1e38 and torch.isnan(got[2, 7, 9])
    assert torch.isnan(got[2]).sum() == 1 and torch.isnan(got[3]).all()
    y = rows(7, 3, torch.bfloat16)  # a block of zeros takes any rows after it
    write(cache, y, y, 20, 128)
    host_write(h, y, y, 20)
    same_cache(cache, h)


def test_no_rows_writes_nothing():
    h = random_cache(8, 256, 100)
    cache = h.device()
    z = rows(0, 0, torch.bfloat16)
    write(cache, z, z, 100, 256)
    ea.expert_attn_read_fp8([ea.Fp8Rows(z.to(DEV), z.to(DEV), cache)], 0, 0, 256)
    same_cache(cache, h)


def test_rows_written_again_from_an_earlier_one():
    """Taking rows back is writing from an earlier row: the block's scale stays as large as it was."""
    h = random_cache(9, 256, 200)
    cache = h.device()
    k, v = rows(10, 30, torch.float16), rows(11, 30, torch.float16)
    write(cache, k, v, 150, 256)
    host_write(h, k, v, 150)
    same_cache(cache, h)


@pytest.mark.parametrize("layers", [3, 64, 67])
def test_layers_and_strided_rows(layers):
    """k and v cut out of one buffer with padding between rows and heads; every layer its own cache."""
    Smax, row0, n = 256, 60, 90
    hs = [random_cache(20 + l % 4, Smax, row0) for l in range(layers)]
    caches = [h.device() for h in hs]
    fused = torch.from_numpy(np.random.default_rng(12).standard_normal((layers, n, 2, 8, 136)).astype(F32)).to(torch.bfloat16).to(DEV)
    L = [ea.Fp8Rows(fused[l, :, 0, :, :128].transpose(0, 1), fused[l, :, 1, :, :128].transpose(0, 1), caches[l]) for l in range(layers)]
    ea.expert_attn_write_fp8(L, row0, n, Smax)
    back = torch.zeros(layers, n, 2, 8, 136, dtype=torch.bfloat16, device=DEV)
    B = [ea.Fp8Rows(back[l, :, 0, :, :128].transpose(0, 1), back[l, :, 1, :, :128].transpose(0, 1), caches[l]) for l in range(layers)]
    ea.expert_attn_read_fp8(B, row0, n, Smax)
    assert (back[..., 128:] == 0).all()
    for l in sorted({0, layers // 2, layers - 1}):
        host_write(hs[l], L[l].k.cpu(), L[l].v.cpu(), row0)
        same_cache(caches[l], hs[l], f"layer {l}")
        assert torch.equal(B[l].k.cpu(), values(hs[l], 0, row0, n, torch.bfloat16))


def test_offsets_past_32_bits():
    """The largest cache: 8 heads x 2^22 rows x 128 bytes; its last rows, of the last head too."""
    Smax, n = 1 << 22, 200
    row0 = Smax - n
    cache = ea.alloc_fp8_cache(Smax)
    k, v = rows(13, n, torch.bfloat16), rows(14, n, torch.bfloat16)
    write(cache, k, v, row0, Smax)
    h = HostCache(256, fill=0)  # the last two blocks, which held zeros under a scale of 1
    for s in h.scales:
        s[:] = 1
    host_write(h, k, v, 256 - n)
    for i, (c, s) in enumerate(((cache.k_cache, cache.k_scale), (cache.v_cache, cache.v_scale))):
        assert np.array_equal(c[:, -256:].cpu().numpy(), h.codes[i])
        assert np.array_equal(s[:, -3:-1].cpu().numpy(), h.scales[i][:, :2])
        assert not c[:, :-256].any() and (s[:, -1] == 1).all() and (s[:, :-3] == 1).all()
    assert torch.equal(read(cache, row0, n, Smax, torch.bfloat16)[1].cpu(), values(h, 1, 256 - n, n, torch.bfloat16))


def test_captured_and_on_another_stream():
    Smax, h = 256, random_cache(15, 256, 100)
    cache, s = h.device(), torch.cuda.Stream()
    k, v = rows(16, 20, torch.bfloat16).to(DEV), rows(17, 20, torch.bfloat16).to(DEV)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    w, b = [ea.Fp8Rows(k, v, cache)], [ea.Fp8Rows(kb, vb, cache)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ea.expert_attn_write_fp8(w, 100, 20, Smax)
        ea.expert_attn_read_fp8(b, 100, 20, Smax)
    for seed in (18, 19):
        x = rows(seed, 20, torch.bfloat16, gain=float(seed - 17))
        k.copy_(x.to(DEV))
        v.copy_(x.to(DEV))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        host_write(h, x, x, 100)
        same_cache(cache, h)
        assert torch.equal(kb.cpu(), values(h, 0, 100, 20, torch.bfloat16))
