"""Softmax weights of the decode step over an 8-bit cache, to more bits than the bf16 output shows of them."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import DEV, F32, HostCache, decode_buffers, decode_inputs, decode_oracle, f64
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,pos", [(1, 2000), (20, 2000), (5, 20000)])
def test_outputs_that_cancel(layers, pos):
    """Keys of two kinds in turn, V = 1 under a tile's largest weight and V = -1 under a somewhat smaller one, w: out = (1 - w) / (1 + w),
    w = 0.94 to 1 or lower by head. A weight may be off by 2^-14 of itself (one at the tile's largest is exact), scores, which these
    inputs keep under 1, by 1.5 x 2^-18, of either kind: |out's error| <= 2^-8 |out| + 2^-14 w / (1 + w) + 2^-17. With weights held to 2^-9
    it would be 2^-10 for some head."""
    Smax = pos // 128 * 128 + 256
    h, x = HostCache(Smax), decode_inputs(1)
    for i in range(2):
        h.codes[i][:, :pos] = 0
        h.scales[i][:] = F32(1)
    h.codes[0][:, 0:pos:2, 0] = 0x38
    h.scales[0][:] = np.exp2(np.linspace(-4, 0, 8)).astype(F32)[:, None]  # by kv head
    h.codes[1][:, 0:pos:2] = 0x38
    h.codes[1][:, 1:pos:2] = 0xB8
    for n in ("q_gamma", "k_gamma"):
        x[n].fill_(1.0)
    x["k_raw"].zero_()
    x["v_raw"].zero_()
    q = x["q_raw"].view(64, 128)
    q.zero_()
    q[:, 0] = torch.linspace(0.1, 1.0, 64)
    q[:, 1] = 1.0 - q[:, 0].float() ** 2
    bufs = [decode_buffers(x, h.device()) for _ in range(layers)]
    ws = ea.alloc_decode_fp8_workspace(layers, Smax)
    ea.text_decode_attention_fp8(bufs, pos, Smax, -pos, ws)
    check_status(ws)
    want = decode_oracle(x, h, pos, -pos)["out"]
    assert (want > 0).all() and want.max() < 0.6
    w = (1 - want) / (1 + want)
    for b in bufs:
        off = np.abs(f64(b.out) - want) - (2.0 ** -8 * want + 2.0 ** -14 * w / (1 + w) + 2.0 ** -17)
        assert (off <= 0).all(), f"{(off > 0).sum()} outputs, the worst by {off.max():.1e}"
