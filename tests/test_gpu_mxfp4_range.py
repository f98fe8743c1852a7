"""The attentions over a 4-bit cache where scales differ by far more than 16-bit numbers hold: between the channel blocks
of the values or the keys, between rows, and between queries and keys. Outputs are compared 32 channels at a time, so that
small channels count beside large ones. The bar is that of the attentions' other tests, relative L2 <= 5e-3 (its terms are
added up there); the references are fp64."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._gpu_util import check_status
from tests._mxfp4_util import HostCache, decode_oracle, device_buffers, expert_oracle, f64, step_inputs
from tests.test_gpu_mxfp4_attention import REL

pytestmark = pytest.mark.gpu
FORMS = {"decode": (ea.text_decode_attention_mxfp4, ea.alloc_decode_mxfp4_workspace, decode_oracle, 64, 1),
         "expert": (ea.expert_attn_layers_mxfp4, ea.alloc_mxfp4_workspace, expert_oracle, 16, 64)}


def close_by_block(got: torch.Tensor, want: np.ndarray, what: str):
    g = f64(got)
    assert np.isfinite(g).all(), what
    for b in range(4):
        c = slice(32 * b, 32 * b + 32)
        rel = np.linalg.norm(g[..., c] - want[..., c]) / np.linalg.norm(want[..., c])
        assert rel <= REL, f"{what}: channels {32 * b} to {32 * b + 31}: rel-L2 {rel:.2e}"


def run(form, x, h, n, delta, layers):
    """The same layer `layers` times in one call: with 20 of them a CTA's keys are many tiles of a unit, with one layer a
    unit is cut over all of them."""
    call, alloc, ref, _, _ = FORMS[form]
    bufs = [device_buffers(x, h.device()) for _ in range(layers)]
    ws = alloc(layers)
    call(bufs, n, h.Smax, delta, ws)
    check_status(ws)
    want = ref(x, h, n, delta)["out"]
    for l in {0, layers // 2, layers - 1}:
        close_by_block(bufs[l].out, want, f"layer {l}")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [1, 72, 200, 127, 300])
@pytest.mark.parametrize("size", [1e-6, 1e-8, 1e-12])
def test_small_queries_over_zero_keys(form, n, size):
    """Rows that were never written before the last key, and a query of next to nothing: every key counts the same."""
    _, _, _, hq, tok = FORMS[form]
    x = step_inputs(n, hq, tok)
    x["q_raw"] = (x["q_raw"].float() * size).to(torch.bfloat16)
    v = np.random.default_rng(n).standard_normal((8, 512, 128))
    run(form, x, HostCache(np.zeros_like(v), v, n), n, 0, 1)


def one_sided(seed, hq, tok):
    """Queries that all point the same way in channels 63 and 127 (which hardly rotate at positions 0 to 63)."""
    x = step_inputs(seed, hq, tok)
    q = 0.25 * x["q_raw"].float()
    q[..., 63] = q[..., 127] = 1.0
    x["q_raw"] = q.to(torch.bfloat16)
    return x


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layers", [1, 20])
@pytest.mark.parametrize("steps", [(0, -8, -16, -24), (45, 15, -15, -45), (-30, 0, -2, -32), (60, -60, 0, 0)])
def test_values_of_blocks_far_apart(form, layers, steps):
    _, _, _, hq, tok = FORMS[form]
    x = step_inputs(17, hq, tok)
    k, v = np.random.default_rng(17).standard_normal((2, 8, 896, 128))
    by = np.exp2(steps).repeat(32)
    v *= by
    x["v_raw"] = (x["v_raw"].float() * torch.from_numpy(by)).to(torch.bfloat16)
    run(form, x, HostCache(k, v, 700), 700, 0, layers)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layers", [1, 20])
@pytest.mark.parametrize("at", [0, 333, 699])
@pytest.mark.parametrize("by", [30, 60, 100])
def test_large_value_without_weight(form, layers, at, by):
    """A row whose values are 2^by above the others', at a key that no query looks at."""
    _, _, _, hq, tok = FORMS[form]
    x = one_sided(at, hq, tok)
    k, v = np.random.default_rng(at + by).standard_normal((2, 8, 896, 128))
    k[:, at, [63, 127]] = -512.0
    v[:, at] *= 2.0 ** by
    run(form, x, HostCache(k, v, 700), 700, -700, layers)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layers", [1, 20])
def test_values_spread_at_random(form, layers):
    _, _, _, hq, tok = FORMS[form]
    x = step_inputs(23, hq, tok)
    rng = np.random.default_rng(23)
    k, v = rng.standard_normal((2, 8, 896, 128))
    v *= np.exp2(rng.integers(-60, 1, (8, 896, 4)) + np.array([0, -20, 30, 7])).repeat(32, -1)
    run(form, x, HostCache(k, v, 700), 700, 0, layers)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layers", [1, 20])
@pytest.mark.parametrize("by", [26, 50, 90])
def test_keys_of_blocks_far_apart(form, layers, by):
    """Blocks 0 and 2 of the keys 2^by above blocks 1 and 3, in channels where the queries are zero."""
    _, _, _, hq, tok = FORMS[form]
    x = step_inputs(29, hq, tok)
    x["q_gamma"][0:32] = x["q_gamma"][64:96] = 0.0
    k, v = np.random.default_rng(29).standard_normal((2, 8, 896, 128))
    k[..., 0:32] *= 2.0 ** by
    k[..., 64:96] *= 2.0 ** by
    x["k_gamma"][0:32] = x["k_gamma"][64:96] = 2.0 ** by
    run(form, x, HostCache(k, v, 700), 700, 0, layers)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layers", [1, 20])
@pytest.mark.parametrize("at", [0, 333, 699])
@pytest.mark.parametrize("by", [26, 60])
def test_large_key_against_every_query(form, layers, at, by):
    _, _, _, hq, tok = FORMS[form]
    x = one_sided(at, hq, tok)
    k, v = np.random.default_rng(at).standard_normal((2, 8, 896, 128))
    k[:, at, [63, 127]] = -2.0 ** by
    run(form, x, HostCache(k, v, 700), 700, -700, layers)


@pytest.mark.parametrize("layers,n", [(1, 700), (20, 700), (3, 1500)])
@pytest.mark.parametrize("high", [16, 12])
def test_weights_far_below_the_largest(layers, n, high):
    """One key in every 32 is a sink, 8 (high + 8 - 2) / sqrt(128) nats above the rest, with values of zero: the output is what
    the rest add. Decode holds weights in f16 with a warp's largest at 2^8 at least, to 2^-25 of absolute error."""
    x = step_inputs(1, 64, 1)
    for name in ("q_gamma", "k_gamma"):
        x[name].fill_(1.0)
    x["q_raw"].zero_()
    x["q_raw"][..., 63] = x["q_raw"][..., 127] = 1.0  # normed: 8 in both
    x["k_raw"].zero_()
    x["v_raw"].fill_(1.0)
    Smax = -(-(n + 1) // 64) * 64
    k, v = np.zeros((8, Smax, 128)), np.ones((8, Smax, 128))
    k[:, ::32, 63], k[:, ::32, 127] = high, 8.0
    v[:, ::32] = 0.0
    h = HostCache(k, v, n)
    bufs = [device_buffers(x, h.device()) for _ in range(layers)]
    ws = ea.alloc_decode_mxfp4_workspace(layers)
    ea.text_decode_attention_mxfp4(bufs, n, Smax, -n, ws)
    check_status(ws)
    small = np.exp2(-8 * (high + 8) / 128 ** 0.5 / np.log(2))  # a rest key's weight, the sink's being 1
    sinks = -(-n // 32)
    rest = n + 1 - sinks
    want = rest * small / (sinks + rest * small)
    # bf16's half step, the weight's (2^-25 at 2^8), and 1e-4 for fp32 sums and exponentials
    bar = 2.0 ** -9 + 2.0 ** -33 / small + 1e-4
    for b in bufs:
        off = float((b.out.double() / want - 1).abs().max())
        assert off <= bar, f"off by {off:.2e}, bar {bar:.2e}"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [0, 1, 130, 384])
def test_few_rows_far_apart(form, n):
    """Blocks of keys and values far apart where the own rows are all there is, or a whole unit is one CTA's."""
    _, _, _, hq, tok = FORMS[form]
    x = step_inputs(n + 3, hq, tok)
    x["q_gamma"][0:32] = x["q_gamma"][64:96] = 0.0
    x["k_gamma"][0:32] = x["k_gamma"][64:96] = 2.0 ** 40
    by = np.exp2([0, -12, 25, -40]).repeat(32)
    x["v_raw"] = (x["v_raw"].float() * torch.from_numpy(by)).to(torch.bfloat16)
    k, v = np.random.default_rng(n).standard_normal((2, 8, 512, 128))
    k[..., 0:32] *= 2.0 ** 40
    k[..., 64:96] *= 2.0 ** 40
    run(form, x, HostCache(k, v * by, n), n, 0, 3)


@pytest.mark.parametrize("form", FORMS)
def test_far_apart_again_and_captured(form):
    """The same bits from every call, and from a graph's replay."""
    call, alloc, _, hq, tok = FORMS[form]
    x = step_inputs(5, hq, tok)
    k, v = np.random.default_rng(5).standard_normal((2, 8, 1088, 128))
    by = np.exp2([0, -30, -15, 5]).repeat(32)
    h = HostCache(k * by[::-1], v * by, 1000)
    bufs, ws = [device_buffers(x, h.device()) for _ in range(9)], alloc(9)
    call(bufs, 1000, 1088, 0, ws)
    outs = [b.out.clone() for b in bufs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(bufs, 1000, 1088, 0, ws)
    for _ in range(3):
        for b in bufs:
            b.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check_status(ws)
        assert all(torch.equal(b.out, o) for b, o in zip(bufs, outs))
