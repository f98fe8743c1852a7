"""GPU parity of the attentions over a 4-bit cache (text_decode_attention_mxfp4 and
expert_attn_layers_mxfp4) against the fp64 oracle on the dequantised values.

The new rows are exact: their codes and exponents equal the oracle quantiser's. The output's bar is
that of the other caches, relative L2 <= 5e-3. What it has to hold: the bf16 output's rounding, at most
2^-8 of each value, uniform within its step, so about 2^-8 / sqrt(3) * 3/4 = 1.7e-3 in the L2 norm; q
and the softmax weights in 16 bits (at most 2^-11 each way in fp16): a score of these inputs, a sum of
128 products of about unit variance over sqrt(128), moves by about 2^-11 / sqrt(3), 3e-4, and so do
the weights; fp32 accumulation, below 1e-5. Together under 2e-3; the bar is 2.5 times that."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._gpu_util import check_status
from tests._mxfp4_util import (DEV, HostCache, decode_oracle, device_buffers, expert_oracle, f64, quantise,
                               random_cache, step_inputs, unpacked)

pytestmark = pytest.mark.gpu
REL = 5e-3


def close(got: torch.Tensor, want: np.ndarray, what: str = "out"):
    g = f64(got)
    assert np.isfinite(g).all(), what
    rel = np.linalg.norm(g - want) / max(np.linalg.norm(want), 1e-300)
    # no single value is further off than 8 times the bar's share of the largest one
    big = np.abs(g - want).max() / max(np.abs(want).max(), 1e-300)
    assert rel <= REL and big <= 8 * REL, f"{what}: rel-L2 {rel:.2e}, largest {big:.2e}"


def check_new_rows(b, ref, row0, n):
    c = b.cache
    for name, codes, scales, new in (("k", c.k_codes, c.k_scales, b.k_new), ("v", c.v_codes, c.v_scales, b.v_new)):
        want_c, want_e = ref[name]
        got_c, got_e = unpacked(codes[:, row0:row0 + n], scales[:, row0:row0 + n])
        assert np.array_equal(got_e.reshape(want_e.shape), want_e), name
        assert np.array_equal(got_c.reshape(want_c.shape), want_c), name
        if new is not None:
            import oracle
            assert np.array_equal(f64(new), oracle.dequantize_rows(want_c, want_e).reshape(new.shape)), name


def check_untouched(h: HostCache, c, lo, hi):
    keep = [r for r in range(h.Smax) if not lo <= r < hi]
    for want, got in zip(h.bytes, c.__dict__.values()):
        assert torch.equal(want[:, keep], got[:, keep].cpu())


def decode(xs, hs, pos, Smax, delta=0, values=True):
    bufs = [device_buffers(x, h.device(), values) for x, h in zip(xs, hs)]
    ws = ea.alloc_decode_mxfp4_workspace(len(bufs))
    ea.text_decode_attention_mxfp4(bufs, pos, Smax, delta, ws)
    torch.cuda.synchronize()
    check_status(ws)
    return bufs


def expert(xs, hs, S, Smax, delta=0, values=True):
    bufs = [device_buffers(x, h.device(), values) for x, h in zip(xs, hs)]
    ws = ea.alloc_mxfp4_workspace(len(bufs))
    ea.expert_attn_layers_mxfp4(bufs, S, Smax, delta, ws)
    torch.cuda.synchronize()
    check_status(ws)
    return bufs


# ------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("pos,Smax,delta", [(0, 128, 0), (1, 128, 5), (7, 128, -7), (63, 128, 0), (64, 128, 0), (127, 128, 0), (128, 192, 0),
                                            (129, 192, -200), (300, 512, 0), (511, 512, 9), (1027, 1088, 0),
                                            (2500, 4096, 100000)])
def test_decode_one_layer(pos, Smax, delta):
    x, h = step_inputs(10 * pos, 64, 1), random_cache(pos, Smax, pos, k_gain=1.5)
    (b,) = decode([x], [h], pos, Smax, delta)
    ref = decode_oracle(x, h, pos, delta)
    check_new_rows(b, ref, pos, 1)
    check_untouched(h, b.cache, pos, pos + 1)
    close(b.out, ref["out"])


@pytest.mark.parametrize("pos", [4700, 8191])
def test_decode_long(pos):
    x, h = step_inputs(pos, 64, 1), random_cache(pos, 8192, pos)
    (b,) = decode([x], [h], pos, 8192)
    close(b.out, decode_oracle(x, h, pos, 0)["out"])


@pytest.mark.parametrize("layers,pos,Smax", [(3, 130, 192), (9, 1000, 1024), (65, 77, 128), (20, 2047, 2048)])
def test_decode_several_layers(layers, pos, Smax):
    xs = [step_inputs(1000 + 7 * l, 64, 1) for l in range(layers)]
    hs = [random_cache(50 + l, Smax, pos) for l in range(layers)]
    bufs = decode(xs, hs, pos, Smax, 3, values=False)
    for l in {0, 1, layers // 2, layers - 1}:
        ref = decode_oracle(xs[l], hs[l], pos, 3)
        check_new_rows(bufs[l], ref, pos, 1)
        close(bufs[l].out, ref["out"], f"layer {l}")


@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFE, 0xFF])
def test_decode_never_uses_rows_after_pos(fill):
    x = step_inputs(5, 64, 1)
    outs = [decode([x], [random_cache(6, 512, 300, fill=f)], 300, 512)[0].out for f in (0x33, fill)]
    assert torch.equal(*outs)


# ------------------------------------------------------------------------------------ expert
@pytest.mark.parametrize("S,Smax,delta", [(0, 128, 0), (1, 128, 0), (63, 128, -5), (64, 128, 0), (65, 192, 0), (127, 256, 0), (128, 192, 7),
                                          (129, 512, 0), (256, 512, 0), (300, 384, -300), (1000, 1088, 0), (1961, 2048, 50000)])
def test_expert_one_layer(S, Smax, delta):
    x, h = step_inputs(20 * S + 1, 16, 64), random_cache(S + 3, Smax, S, k_gain=1.5)
    (b,) = expert([x], [h], S, Smax, delta)
    ref = expert_oracle(x, h, S, delta)
    check_new_rows(b, ref, Smax - 64, 64)
    check_untouched(h, b.cache, Smax - 64, Smax)
    close(b.out, ref["out"])


@pytest.mark.parametrize("S,Smax", [(4700, 8192), (8128, 8192)])
def test_expert_long(S, Smax):
    x, h = step_inputs(S, 16, 64), random_cache(S, Smax, S)
    (b,) = expert([x], [h], S, Smax)
    close(b.out, expert_oracle(x, h, S, 0)["out"])


@pytest.mark.parametrize("layers,S,Smax", [(3, 130, 256), (9, 700, 768), (66, 77, 192), (21, 1500, 1600)])
def test_expert_several_layers(layers, S, Smax):
    xs = [step_inputs(3000 + 7 * l, 16, 64) for l in range(layers)]
    hs = [random_cache(90 + l, Smax, S) for l in range(layers)]
    bufs = expert(xs, hs, S, Smax, 3, values=False)
    for l in {0, 1, layers // 2, layers - 1}:
        ref = expert_oracle(xs[l], hs[l], S, 3)
        check_new_rows(bufs[l], ref, Smax - 64, 64)
        close(bufs[l].out, ref["out"], f"layer {l}")


@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFE, 0xFF])
def test_expert_never_uses_hidden_rows(fill):
    x = step_inputs(15, 16, 64)
    outs = [expert([x], [random_cache(16, 512, 200, fill=f)], 200, 512)[0].out for f in (0x33, fill)]
    assert torch.equal(*outs)


# --------------------------------------------------------------------------------- both forms
FORMS = {"decode": (decode, decode_oracle, 64, 1), "expert": (expert, expert_oracle, 16, 64)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", ["tiny values", "huge values", "zero values", "zero blocks", "spread scales", "one large key",
                                  "values grow", "values shrink", "zero keys", "zero queries", "large gains"])
def test_magnitudes(form, case):
    """Cache contents whose scales differ by far: between blocks of a row, rows and tiles of rows."""
    run, ref, hq, tok = FORMS[form]
    n, Smax = 700, 896
    rng = np.random.default_rng(len(case))
    k, v = rng.standard_normal((2, 8, Smax, 128))
    x = step_inputs(len(case), hq, tok)
    if case == "tiny values":
        v *= 2.0 ** -110
        x["v_raw"] = (x["v_raw"].float() * 2.0 ** -110).to(torch.bfloat16)
    elif case == "huge values":
        v *= 2.0 ** 110
        x["v_raw"] = (x["v_raw"].float() * 2.0 ** 110).to(torch.bfloat16)
    elif case == "zero values":
        v[:, :600] = 0.0
    elif case == "zero blocks":
        v *= 2.0 ** -40
        v[:, :, 32:64] = 0.0
        x["v_raw"] = (x["v_raw"].float() * 2.0 ** -40).to(torch.bfloat16)
        x["v_raw"][..., 32:64] = 0.0
    elif case == "spread scales":
        v *= np.exp2(rng.integers(-6, 7, (8, Smax, 4))).repeat(32, -1)
        k *= np.exp2(rng.integers(-3, 2, (8, Smax, 4))).repeat(32, -1)
    elif case == "one large key":
        k[:, 5] *= 8.0
        k[:, 400] *= 16.0
    elif case == "values grow":
        v *= np.exp2(np.arange(Smax) // 64)[None, :, None]
    elif case == "values shrink":
        v *= np.exp2(-(np.arange(Smax) // 64))[None, :, None]
    elif case == "zero keys":
        k[:] = 0.0
    elif case == "zero queries":
        x["q_raw"].zero_()
    elif case == "large gains":
        x["q_gamma"] = (x["q_gamma"].float() * 2.0 ** 10).to(torch.bfloat16)
        k *= 2.0 ** -10
        x["k_gamma"] = (x["k_gamma"].float() * 2.0 ** -10).to(torch.bfloat16)
    h = HostCache(k, v, n)
    (b,) = run([x], [h], n, Smax)
    want = ref(x, h, n, 0)
    check_new_rows(b, want, n if form == "decode" else Smax - 64, tok)
    close(b.out, want["out"], case)


@pytest.mark.parametrize("form", FORMS)
def test_same_bits_again_and_from_a_used_workspace(form):
    run, _, hq, tok = FORMS[form]
    n, Smax = 1500, 2048
    xs = [step_inputs(40 + l, hq, tok) for l in range(3)]
    hs = [random_cache(70 + l, Smax, n) for l in range(3)]
    bufs = [device_buffers(x, h.device()) for x, h in zip(xs, hs)]
    alloc, call = ((ea.alloc_decode_mxfp4_workspace, ea.text_decode_attention_mxfp4) if form == "decode" else
                   (ea.alloc_mxfp4_workspace, ea.expert_attn_layers_mxfp4))
    ws = alloc(3)
    outs = []
    for _ in range(4):
        call(bufs, n, Smax, 0, ws)
        outs.append([b.out.clone() for b in bufs])
    check_status(ws)
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


@pytest.mark.parametrize("form", FORMS)
def test_a_run_of_them_together(form):
    """Prefill rows written into an empty cache, attention over them, the step's new rows read back: on a
    stream of its own, captured and replayed."""
    _, ref, hq, tok = FORMS[form]
    n, Smax = 333, 512
    x = step_inputs(77, hq, tok)
    rng = np.random.default_rng(5)
    k, v = (torch.from_numpy(rng.standard_normal((8, n, 128)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    cache = ea.alloc_mxfp4_cache(Smax)
    b = device_buffers(x, cache)
    row0 = n if form == "decode" else Smax - 64
    back = ea.Mxfp4Rows(*(torch.zeros(8, tok, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)), cache)
    alloc, call, args = ((ea.alloc_decode_mxfp4_workspace, ea.text_decode_attention_mxfp4, ea.make_decode_mxfp4_args)
                         if form == "decode" else (ea.alloc_mxfp4_workspace, ea.expert_attn_layers_mxfp4, ea.make_mxfp4_args))
    ws = alloc(1)
    keep = [k.to(DEV), v.to(DEV)]
    src = ea.make_rows_args([ea.Mxfp4Rows(*keep, cache)], Smax)
    dst, step = ea.make_rows_args([back], Smax), args([b], Smax)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        ea.expert_attn_write_mxfp4(None, 0, n, Smax, _arr=src)
        call(None, n, Smax, 0, ws, _arr=step)
        ea.expert_attn_read_mxfp4(None, row0, tok, Smax, _arr=dst)
    with torch.cuda.stream(s):
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    check_status(ws)
    pad = lambda t: np.concatenate([t.float().numpy(), np.zeros((8, Smax - n, 128), np.float32)], 1)  # noqa: E731
    want = ref(x, HostCache(pad(k), pad(v), Smax), n, 0)
    check_new_rows(b, want, row0, tok)
    close(b.out, want["out"])
    assert torch.equal(back.k.reshape(b.k_new.shape), b.k_new) and torch.equal(back.v.reshape(b.v_new.shape), b.v_new)


def test_decode_then_expert_over_one_cache():
    """The text model writes token after token, then the expert attends over what it left."""
    Smax, first = 512, 200
    h = random_cache(8, Smax, first)
    cache = h.device()
    k, v = [np.array(a[0]) for a in (h.k, h.v)], [np.array(a[1]) for a in (h.k, h.v)]
    for t in range(3):
        x = step_inputs(500 + t, 64, 1)
        b = device_buffers(x, cache)
        ws = ea.alloc_decode_mxfp4_workspace(1)
        ea.text_decode_attention_mxfp4([b], first + t, Smax, 0, ws)
        ref = decode_oracle(x, h, first + t, 0)
        close(b.out, ref["out"], f"token {t}")
        for i, name in enumerate(("k", "v")):
            k[i][:, first + t], v[i][:, first + t] = ref[name]
        h.k, h.v = (k[0], v[0]), (k[1], v[1])
    x = step_inputs(600, 16, 64)
    b = device_buffers(x, cache)
    ws = ea.alloc_mxfp4_workspace(1)
    ea.expert_attn_layers_mxfp4([b], first + 3, Smax, 0, ws)
    close(b.out, expert_oracle(x, h, first + 3, 0)["out"])


@pytest.mark.parametrize("form", FORMS)
def test_workspace_too_small_is_refused(form):
    _, _, hq, tok = FORMS[form]
    b = device_buffers(step_inputs(1, hq, tok), random_cache(1, 128, 10).device())
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    with pytest.raises(ea.ExpertAttnError, match="WORKSPACE"):
        (ea.text_decode_attention_mxfp4 if form == "decode" else ea.expert_attn_layers_mxfp4)([b], 10, 128, 0, ws)
    assert torch.isnan(b.out).all()


def test_quantise_helper_is_the_oracles():
    import oracle
    x = np.random.default_rng(0).standard_normal((3, 128)).astype(np.float32)
    c, e = oracle.quantize_rows(x)
    a, b = quantise(x)
    assert np.array_equal(a, c) and np.array_equal(b, e)
