"""NaN and infinities in the decode step over an 8-bit cache, in its kernel for little work (one layer) and in the other one: they stay
in the heads, rows and channels that the formula gives them. Other outputs have the bar of the step's own tests."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV, decode_buffers, decode_inputs, decode_oracle, f64, random_cache
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu
REL = 2.0 ** -8 + 2.0 ** -12
NAN = float("nan")
# (layers, pos): one CTA, a cluster, many parts; whole units with their weights formed, cut ones, long ones
SHAPES = [(1, 200), (1, 700), (1, 4700), (64, 900), (20, 2500), (5, 20000)]


def call(pairs, pos, weights=True):
    """pairs: (inputs, host cache) of each layer; outputs and weights."""
    Smax = pairs[0][1].Smax
    bufs = [decode_buffers(x, h.device(), None, torch.zeros(8, Smax, device=DEV) if weights else None) for x, h in pairs]
    ws = ea.alloc_decode_fp8_workspace(len(bufs), Smax, weights=weights)
    ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
    check_status(ws)
    return [(f64(b.out), f64(b.weight_out)[:, :pos + 1] if weights else None) for b in bufs]


def check(got, want, nan):
    """nan [64, 128]: where the output is not a number."""
    assert np.array_equal(np.isnan(got), nan), f"{np.isnan(got).sum()} outputs are NaN, {nan.sum()} are expected"
    assert np.linalg.norm((got - want)[~nan]) <= REL * np.linalg.norm(want[~nan])


def setup(layers, pos):
    """Layers alike but for the middle one, which a test changes; its index."""
    Smax = pos // 128 * 128 + 256
    x, h = decode_inputs(1), random_cache(2, Smax, pos)
    at = layers // 2
    return [(x, h)] * at + [({k: v.clone() for k, v in x.items()}, h.copy())] + [(x, h)] * (layers - at - 1), at


@pytest.mark.parametrize("layers,pos", SHAPES)
def test_nan_codes_of_held_rows(layers, pos):
    """In K: its key's scores, so every channel of the group's heads; in V: its channel of the group's heads."""
    pairs, at = setup(layers, pos)
    x, h = pairs[at]
    h.codes[0][2, pos // 2, 3] = 0x7F
    h.codes[1][5, pos - 1, 9] = 0xFF
    h.codes[1][7, 0, 127] = 0x7F
    got = call(pairs, pos)
    nan = np.zeros((64, 128), bool)
    nan[16:24], nan[40:48, 9], nan[56:, 127] = True, True, True
    want = [decode_oracle(*(p if i else (p[0], p[1].copy())), pos, 0) for i, p in ((0, (pairs[0][0], random_cache(2, h.Smax, pos))), (1, (x, h.copy())))]
    for i, (out, w) in enumerate(got):
        check(out, want[i == at]["out"], nan if i == at else np.zeros_like(nan))
        bad = np.isnan(w).all(1)
        assert np.array_equal(bad, np.arange(8) == 2 if i == at else np.zeros(8, bool)) and np.isfinite(w[~bad]).all()


@pytest.mark.parametrize("layers,pos", SHAPES)
@pytest.mark.parametrize("name,heads", [("q_raw", slice(9, 10)), ("k_raw", slice(48, 56))])
def test_nan_rows_of_the_step(layers, pos, name, heads):
    """One query row, or the new key of one KV head."""
    pairs, at = setup(layers, pos)
    x, h = pairs[at]
    clean = decode_oracle(pairs[at][0], random_cache(2, h.Smax, pos), pos, 0)["out"]
    x[name][9 if name == "q_raw" else 6].view(-1)[5] = NAN
    for i, (out, w) in enumerate(call(pairs, pos)):
        nan = np.zeros((64, 128), bool)
        if i == at:
            nan[heads] = True
        check(out, clean, nan)
        groups = np.isnan(w).any(1)
        assert np.array_equal(groups, nan.reshape(8, -1).any(1))


@pytest.mark.parametrize("layers,pos", SHAPES)
def test_an_infinite_query_gain_gives_nan(layers, pos):
    """Scores of plus and minus infinity: their softmax is not a number, in whichever kernel."""
    pairs, at = setup(layers, pos)
    x, h = pairs[at]
    clean = decode_oracle(x, random_cache(2, h.Smax, pos), pos, 0)["out"]
    x["q_gamma"].view(-1)[77] = float("inf")
    for i, (out, _) in enumerate(call(pairs, pos, weights=False)):
        check(out, clean, np.full((64, 128), i == at))
