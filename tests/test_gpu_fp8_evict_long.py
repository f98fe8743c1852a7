"""Eviction from long caches (a head's weights shared by clusters of two, three, four and eight, kept on chip and read again) and of
layers that differ, against the rule in plain torch calls. Every scale is one, so that rows move as they are."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu


def weights(seed, Smax, alike):
    """Sums as steps leave them, or a few values only: many rows at the threshold, in every slice."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if alike:
        return torch.randint(0, 4, (8, Smax), generator=g, device=DEV).float() * 0.25
    return torch.exp(2 * torch.randn(8, Smax, generator=g, device=DEV)) * (torch.rand(8, Smax, generator=g, device=DEV) > 0.1)


def cache(seed, Smax):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = ea.alloc_fp8_cache(Smax)
    for t in (c.k_cache, c.v_cache):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


def rule(w, n_rows, keep, first, recent):
    among = w[:, first:n_rows - recent].double().sort(dim=1, descending=True, stable=True)[1][:, :keep - first - recent] + first
    ends = torch.cat([torch.arange(first, device=DEV), torch.arange(n_rows - recent, n_rows, device=DEV)]).expand(8, -1)
    return torch.cat([among, ends], 1).sort(1)[0]


def check(layers, n_rows, keep, first, recent, in_place):
    """layers: (cache, weights) of each."""
    L, want = [], []
    Smax = layers[0][1].shape[1]
    for c, w in layers:
        kept = torch.full((8, keep), -1, dtype=torch.int32, device=DEV)
        L.append(ea.EvictFp8Buffers(c, w, kept) if in_place else ea.EvictFp8Buffers(c, w, kept, ea.alloc_fp8_cache(Smax), torch.full_like(w, -7.0)))
        r = rule(w, n_rows, keep, first, recent)
        rows = r[..., None].expand(-1, -1, 128)
        behind = [t[:, keep:].clone() for t in ((c.k_cache, c.v_cache, w) if in_place else (L[-1].to.k_cache, L[-1].to.v_cache, L[-1].weight_to))]
        want.append((r, c.k_cache.gather(1, rows), c.v_cache.gather(1, rows), w.gather(1, r), behind))
    ws = ea.alloc_evict_fp8_workspace(len(L), Smax)
    ea.expert_attn_evict_fp8(L, n_rows, keep, first, recent, Smax, ws)
    check_status(ws)
    for l, (x, (r, k, v, w, behind)) in enumerate(zip(L, want)):
        got = (x.cache.k_cache, x.cache.v_cache, x.weight) if in_place else (x.to.k_cache, x.to.v_cache, x.weight_to)
        assert torch.equal(x.kept.long(), r), f"layer {l}"
        assert all(torch.equal(t[:, :keep], u) for t, u in zip(got, (k, v, w))), f"layer {l}"
        assert all(torch.equal(t[:, keep:], u) for t, u in zip(got, behind)), f"layer {l}"
        scales = (x.cache.k_scale, x.cache.v_scale) if in_place else (x.to.k_scale, x.to.v_scale)
        assert all((s == 1).all() for s in scales)


@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_rows,keep,first,recent", [
    (8192, 5000, 0, 0), (8193, 5000, 4300, 600), (8193, 8192, 0, 0), (16384, 9000, 10, 8200), (16385, 7000, 5700, 100),
    (20000, 300, 4, 100), (24576, 24000, 9000, 9000), (24577, 6000, 0, 6000), (24577, 6000, 6000, 0), (40000, 20000, 0, 1000)])
def test_clusters_of_two_three_and_four(n_rows, keep, first, recent, in_place, alike):
    Smax = n_rows // 128 * 128 + 256
    check([(cache(n_rows + l, Smax), weights(n_rows + 10 * l, Smax, alike)) for l in range(2)], n_rows, keep, first, recent, in_place)


@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("n_rows,keep,first,recent,in_place", [
    (131072, 3000, 5, 100, False), (131073, 3000, 5, 100, False), (131073, 20000, 17000, 100, True), (262144, 2000, 0, 0, True),
    (262145, 2000, 0, 0, False), (262145, 40000, 33000, 5000, True)])
def test_clusters_of_eight(n_rows, keep, first, recent, in_place, alike):
    """Past 262144 rows a slice's weights no longer stay on chip."""
    Smax = n_rows // 128 * 128 + 256
    check([(cache(n_rows, Smax), weights(keep, Smax, alike))], n_rows, keep, first, recent, in_place)


@pytest.mark.parametrize("alike", [False, True])
def test_the_longest_cache(alike):
    Smax = 1 << 22
    check([(cache(1, Smax), weights(2, Smax, alike))], Smax, 100001, 16, 5000, True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layers,n_rows,keep", [(3, 1000, 800), (64, 300, 200), (66, 260, 130), (70, 900, 513), (9, 9000, 4000)])
def test_layers_that_differ(layers, n_rows, keep, in_place):
    """No two layers alike, also beyond the 64 of one launch."""
    Smax = -(-n_rows // 128) * 128
    check([(cache(l, Smax), weights(100 + l, Smax, l % 2)) for l in range(layers)], n_rows, keep, 5, 100, in_place)


def test_layers_that_share_sources():
    """Several layers thinned by one weight array, and one cache thinned by two."""
    Smax, n = 1024, 1000
    w, c = weights(1, Smax, False), cache(2, Smax)
    check([(cache(l, Smax), w) for l in range(3)] + [(c, w), (c, weights(3, Smax, True))], n, 600, 4, 50, False)
