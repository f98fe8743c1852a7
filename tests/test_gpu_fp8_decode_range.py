"""The decode step over an 8-bit cache at the ends of V's range: sums over many keys stay finite where their mean is. Outputs are
bf16: at most half a step, 2^-8, off; with what weights and scores add (2^-12 in all) the bar of the step's own tests."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV, F32, HostCache, decode_buffers, decode_inputs, decode_oracle, f64, same_cache
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu
REL = 2.0 ** -8 + 2.0 ** -12
# (layers, pos): little work in one CTA, a cluster and many parts; whole units, cut ones, and both
SHAPES = [(1, 200), (1, 1000), (1, 4700), (3, 400), (20, 2500), (5, 20000), (64, 900)]


def run(x, h, pos, layers, weights=True):
    bufs = [decode_buffers(x, h.device(), None, torch.full((8, h.Smax), -7.0, device=DEV) if weights else None) for _ in range(layers)]
    ws = ea.alloc_decode_fp8_workspace(layers, h.Smax, weights=weights)
    ea.text_decode_attention_fp8(bufs, pos, h.Smax, -pos, ws)
    check_status(ws)
    want = decode_oracle(x, h, pos, -pos)
    for b in bufs:
        same_cache(b.cache, h, signs=False)
        got = f64(b.out)
        assert np.isfinite(got).all()
        off = np.abs(got - want["out"])
        assert (off <= REL * np.abs(want["out"])).all(), float((off / np.abs(want["out"])).max())
        if weights:
            w = f64(b.weight_out)[:, :pos + 1]
            assert (np.abs(w - want["weight"]) <= 1.5e-4 * want["weight"] + 1e-37).all()


def alike(pos, e):
    """Keys that all weigh the same, V = 448 2^e in every channel."""
    h, x = HostCache((pos // 128 + 2) * 128), decode_inputs(2)
    for i in range(2):
        h.codes[i][:, :pos] = 0x7E
        h.scales[i][:] = F32(2.0 ** (e if i else -20))
    for n in ("q_raw", "k_raw"):
        x[n].zero_()
    x["v_raw"].fill_(2.0 ** (e + 8))
    return x, h


@pytest.mark.parametrize("e", [118, 94, 93, -100])
@pytest.mark.parametrize("layers,pos", SHAPES)
def test_sums_past_fp32(layers, pos, e):
    """448 x 2^118 is 1.5e38, three of them are past fp32; at 2^-100 their mean is still 45 powers of two above fp32's end."""
    x, h = alike(pos, e)
    run(x, h, pos, layers)


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("layers,pos", SHAPES)
def test_scales_that_rise_and_fall(layers, pos, up):
    """Blocks' scales from 2^80 to 2^118 in turn, rising or falling, V of one sign: every block's share is in the sum."""
    x, h = alike(pos, 118)
    e = np.linspace(80, 118, pos // 128 + 1).round()
    h.scales[1][:, :len(e)] = np.exp2(e if up else e[::-1]).astype(F32)
    if not up:
        x["v_raw"].fill_(2.0 ** 80)
    run(x, h, pos, layers)


@pytest.mark.parametrize("layers,pos", SHAPES)
def test_a_large_scale_over_codes_of_zero(layers, pos):
    """Half of the blocks hold zeros under 2^118; the output is the other half's, whose scale is 1."""
    x, h = alike(pos, 0)
    x["v_raw"].fill_(256.0)
    for b in range(0, pos // 128, 2):
        h.codes[1][:, 128 * b:128 * b + 128] = 0
        h.scales[1][:, b] = F32(2.0 ** 118)
    run(x, h, pos, layers)
