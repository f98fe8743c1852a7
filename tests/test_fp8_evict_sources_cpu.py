"""What layers of one eviction may share: sources that are only read may stand in several layers, nothing that is written may be read or
written by another one (runs without a GPU)."""
import pytest

from gqa_attention_long_gb300 import _lib
from tests.test_fp8_abi_cpu import INV, MIS, evict, h, spread  # noqa: F401

SOURCES = ("k_cache", "v_cache", "k_scale", "v_scale", "weight")
WRITTEN = ("k_dst", "v_dst", "k_scale_dst", "v_scale_dst", "weight_dst", "kept")


@pytest.mark.parametrize("n", [2, 64, 70, 130])
def test_sources_may_be_shared(h, n):  # noqa: F811
    for name in SOURCES:
        assert evict(h, spread(n, **{name: 1 << 50}), n=n) not in (INV, MIS), name
    assert evict(h, spread(n, **{s: (1 << 50) + (i << 36) for i, s in enumerate(SOURCES)}), n=n) not in (INV, MIS)
    for name in WRITTEN:
        assert evict(h, spread(n, **{name: 1 << 50}), n=n) == INV, name


@pytest.mark.parametrize("n,reader,writer", [(2, 0, 1), (2, 1, 0), (70, 0, 69), (70, 69, 0), (70, 66, 68), (130, 129, 63), (130, 63, 64)])
def test_what_is_written_is_no_source(h, n, reader, writer):  # noqa: F811
    for s in SOURCES:
        for w in WRITTEN:
            a = spread(n)
            setattr(a[reader], s, getattr(a[writer], w))
            assert evict(h, a, n=n) == INV, (s, w)
    # a layer in place, and another one that reads what it moves
    a = spread(n)
    for s, d in zip(SOURCES, WRITTEN):
        setattr(a[writer], d, getattr(a[writer], s))
    assert evict(h, a, n=n) not in (INV, MIS)
    a[reader].weight = a[writer].weight
    assert evict(h, a, n=n) == INV
