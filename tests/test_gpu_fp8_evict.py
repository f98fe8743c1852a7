"""Eviction from an 8-bit cache against the rule written out on the host: which rows stay (equal weights, zeros, NaN), their
codes, scales and weights to the bit, in place and into another cache."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV, F32, HostCache, evict_oracle, random_cache, same_cache
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu


def heavy(seed, Smax):
    """Weights as steps leave them: a few rows with most of it, many with next to none, some with none, some alike."""
    rng = np.random.default_rng(seed)
    w = rng.gamma(0.05, 3.0, (8, Smax)).astype(F32)
    w[rng.random((8, Smax)) < 0.1] = 0
    w[rng.random((8, Smax)) < 0.1] = 0.25
    return w


def pow2_scales(h, seed):
    """Blocks' scales a few powers of two apart, as appended blocks have them."""
    rng = np.random.default_rng(seed)
    for s in h.scales:
        s *= np.exp2(rng.integers(-3, 4, s.shape)).astype(F32)
    return h


def check(h, w, n_rows, n_keep, first, recent, in_place, layers=1):
    Smax = h.Smax
    kept, to, wk = evict_oracle(h, w, n_rows, n_keep, first, recent)
    L = []
    for _ in range(layers):
        src, wd = h.device(), torch.from_numpy(w.copy()).to(DEV)
        out = torch.full((8, n_keep), -1, dtype=torch.int32, device=DEV)
        L.append(ea.EvictFp8Buffers(src, wd, out) if in_place else
                 ea.EvictFp8Buffers(src, wd, out, HostCache(Smax).device(), torch.full_like(wd, -7.0)))
    ws = ea.alloc_evict_fp8_workspace(layers, Smax)
    ea.expert_attn_evict_fp8(L, n_rows, n_keep, first, recent, Smax, ws)
    check_status(ws)
    nb = -(-n_keep // 128)
    for x in L:
        assert np.array_equal(x.kept.cpu().numpy(), kept)
        if in_place:  # what lies behind the kept rows stays as it was
            want = h.copy()
            for i in range(2):
                want.codes[i][:, :n_keep], want.scales[i][:, :nb] = to.codes[i][:, :n_keep], to.scales[i][:, :nb]
            same_cache(x.cache, want)
            wo, rest = x.weight.cpu().numpy(), w
        else:
            same_cache(x.cache, h)
            same_cache(x.to, to)
            assert np.array_equal(x.weight.cpu().numpy(), w, equal_nan=True)
            wo, rest = x.weight_to.cpu().numpy(), np.full_like(w, -7.0)
        assert np.array_equal(wo[:, :n_keep], wk, equal_nan=True) and np.array_equal(wo[:, n_keep:], rest[:, n_keep:], equal_nan=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_rows,n_keep,first,recent,Smax", [
    (1, 1, 0, 0, 128), (2, 1, 0, 0, 128), (2, 1, 1, 0, 128), (2, 1, 0, 1, 128), (128, 127, 0, 0, 128), (129, 128, 4, 30, 256),
    (300, 256, 4, 64, 512), (300, 1, 0, 0, 384), (300, 299, 0, 0, 384), (300, 300, 10, 10, 384), (512, 129, 64, 64, 512),
    (640, 200, 100, 100, 640), (1025, 700, 0, 700, 1152), (1025, 700, 700, 0, 1152), (2047, 1000, 3, 128, 2048), (4700, 4096, 4, 512, 8192),
    (5000, 100, 0, 10, 5120)])
def test_sizes(n_rows, n_keep, first, recent, Smax, in_place):
    h = pow2_scales(random_cache(n_rows + n_keep, Smax, n_rows), n_rows)
    check(h, heavy(n_rows, Smax), n_rows, n_keep, first, recent, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_equal_weights_go_to_the_lowest_rows(in_place):
    for w in (np.zeros((8, 512), F32), np.full((8, 512), 3.5, F32), np.tile(np.array([0.0, -0.0, 1.0, 1.0], F32), (8, 128))):
        check(random_cache(1, 512, 500), w, 500, 300, 2, 50, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_weights_that_are_no_sums(in_place):
    """Negative ones, infinities, subnormals, and NaN, which is above all."""
    rng = np.random.default_rng(2)
    w = rng.choice(np.array([-np.inf, -2.5, -1e-40, -0.0, 0.0, 1e-45, 1e-40, 1.0, 3e38, np.inf, np.nan, -np.nan], F32), (8, 1024))
    for n_keep in (60, 130, 500, 900):
        check(random_cache(3, 1024, 1000), w, 1000, n_keep, 0, 20, in_place)


def test_weights_that_differ_in_their_last_bits():
    """Neighbouring numbers: the last of the threshold's bits decide."""
    rng = np.random.default_rng(4)
    w = (0x3F800000 + rng.integers(0, 4000, (8, 2048))).astype(np.uint32).view(F32)
    check(random_cache(5, 2048, 2000), w, 2000, 1500, 1, 9, True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layers,n_rows,n_keep", [(3, 1000, 800), (64, 300, 200), (66, 260, 130), (20, 3000, 2900)])
def test_layers(layers, n_rows, n_keep, in_place):
    """Every layer alike: none waits for another's blocks, none is left out."""
    Smax = -(-n_rows // 128) * 128
    check(random_cache(6, Smax, n_rows), heavy(7, Smax), n_rows, n_keep, 5, 100, in_place, layers)


@pytest.mark.parametrize("in_place", [False, True])
def test_kept_rows_at_either_end(in_place):
    """All that stays from the cache's beginning (nothing moves), from its end (everything does), and every other row."""
    up, n = np.tile(np.arange(2000, dtype=F32), (8, 1)), 1900
    up = np.concatenate([up, np.zeros((8, 48), F32)], 1)
    for w in (up, -up, (np.arange(2048) % 2).astype(F32)[None].repeat(8, 0)):
        check(random_cache(8, 2048, n), w, n, 950, 0, 0, in_place)


def test_long_cache():
    """131000 rows to a quarter; heads keep different rows."""
    Smax, n = 131072, 131000
    rng = np.random.default_rng(9)
    h = HostCache(Smax, fill=0)
    for i in range(2):
        h.codes[i][:, :n] = rng.integers(0, 0x7F, (8, n, 128), dtype=np.uint8)
        h.scales[i][:, :-1] = np.exp2(rng.integers(-4, 4, (8, Smax // 128))).astype(F32)
    check(h, heavy(10, Smax), n, 32769, 16, 4097, True)


def test_none_kept_does_nothing():
    h, w = random_cache(11, 256, 200), heavy(12, 256)
    L = [ea.EvictFp8Buffers(h.device(), torch.from_numpy(w).to(DEV), torch.empty(8, 0, dtype=torch.int32, device=DEV))]
    ea.expert_attn_evict_fp8(L, 200, 0, 0, 0, 256, ea.alloc_evict_fp8_workspace(1, 256))
    same_cache(L[0].cache, h)


def test_a_workspace_serves_smaller_calls_and_captured_ones():
    """One workspace: an eager call, a captured one of another shape, replayed twice around it."""
    ws, s = ea.alloc_evict_fp8_workspace(3, 1024), torch.cuda.Stream()
    shapes = [(3, 1000, 700, 1024), (1, 250, 130, 256)]
    made = []
    for layers, n, keep, Smax in shapes:
        h, w = random_cache(n, Smax, n), heavy(n, Smax)
        L = [ea.EvictFp8Buffers(h.device(), torch.from_numpy(w).to(DEV), torch.full((8, keep), -1, dtype=torch.int32, device=DEV),
                                HostCache(Smax).device(), torch.zeros(8, Smax, device=DEV)) for _ in range(layers)]
        made.append((h, w, L))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ea.expert_attn_evict_fp8(made[0][2], 1000, 700, 3, 100, 1024, ws)
    with torch.cuda.stream(s):
        for _ in range(2):
            g.replay()
            ea.expert_attn_evict_fp8(made[1][2], 250, 130, 0, 20, 256, ws)
        g.replay()
    torch.cuda.synchronize()
    check_status(ws)
    for (h, w, L), (layers, n, keep, Smax), (first, recent) in zip(made, shapes, ((3, 100), (0, 20))):
        kept, to, wk = evict_oracle(h, w, n, keep, first, recent)
        for x in L:
            assert np.array_equal(x.kept.cpu().numpy(), kept)
            same_cache(x.to, to)


def test_two_streams_at_once():
    h, w = random_cache(13, 2048, 2000), heavy(14, 2048)
    kept, to, wk = evict_oracle(h, w, 2000, 1500, 4, 100)
    runs = []
    for layers in (2, 9, 1):
        L = [ea.EvictFp8Buffers(h.device(), torch.from_numpy(w.copy()).to(DEV), torch.full((8, 1500), -1, dtype=torch.int32, device=DEV))
             for _ in range(layers)]
        runs.append((L, ea.alloc_evict_fp8_workspace(layers, 2048), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for L, ws, s in runs:
        with torch.cuda.stream(s):
            ea.expert_attn_evict_fp8(L, 2000, 1500, 4, 100, 2048, ws)
    torch.cuda.synchronize()
    for L, ws, _ in runs:
        check_status(ws)
        for x in L:
            assert np.array_equal(x.kept.cpu().numpy(), kept)
            for i, (c, s) in enumerate(((x.cache.k_cache, x.cache.k_scale), (x.cache.v_cache, x.cache.v_scale))):
                assert np.array_equal(c[:, :1500].cpu().numpy(), to.codes[i][:, :1500])
                assert np.array_equal(s[:, :12].cpu().numpy(), to.scales[i][:, :12])
