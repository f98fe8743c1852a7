"""The attentions over a 4-bit cache where a call can go wrong besides its sizes: a cache whose offsets pass 32 bits, one
key far above a million others, a query row that is not a number, the ends of the positions, one workspace in two
captured graphs, two streams. The bar is that of the attentions' other tests, relative L2 <= 5e-3 (its terms are added
up there); the references are fp64."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._gpu_util import check_status
from tests._mxfp4_util import DEV, decode_oracle, device_buffers, expert_oracle, random_cache, step_inputs
from tests.test_gpu_mxfp4_attention import REL, close

pytestmark = pytest.mark.gpu
FORMS = {"decode": (ea.text_decode_attention_mxfp4, ea.alloc_decode_mxfp4_workspace, decode_oracle, 64, 1),
         "expert": (ea.expert_attn_layers_mxfp4, ea.alloc_mxfp4_workspace, expert_oracle, 16, 64)}
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values of a head's rows, on the device."""
    lut = torch.tensor(VALUES + [-x for x in VALUES], dtype=torch.float64, device=codes.device)
    x = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).reshape(codes.shape[0], 4, 32)
    return (x * torch.exp2(scales.double() - 127)[..., None]).reshape(codes.shape[0], 128)


def attend(q, cache, g, spans):
    """softmax(q K^T / sqrt(128)) V over head g's rows of `spans`, in pieces that fit the card."""
    m = torch.full((q.shape[0], 1), -torch.inf, dtype=torch.float64, device=q.device)
    den, num = torch.zeros_like(m), torch.zeros_like(q)
    for lo, hi in spans:
        for r in range(lo, hi, 1 << 18):
            c = slice(r, min(r + (1 << 18), hi))
            s = q @ values(cache.k_codes[g, c], cache.k_scales[g, c]).T / 128 ** 0.5
            top = torch.maximum(m, s.max(1, keepdim=True).values)
            p, a = torch.exp(s - top), torch.exp(m - top)
            den, num, m = den * a + p.sum(1, keepdim=True), num * a + p @ values(cache.v_codes[g, c], cache.v_scales[g, c]), top
    return num / den


@pytest.mark.parametrize("form", FORMS)
def test_offsets_past_32_bits(form):
    """The largest cache: 8 heads x 2^22 rows x 64 bytes of codes; the last rows are keys."""
    call, alloc, _, hq, tok = FORMS[form]
    Smax = 1 << 22
    n = Smax - tok
    gen = torch.Generator(DEV).manual_seed(3)
    byte = lambda lo, hi, w: torch.randint(lo, hi, (8, Smax, w), dtype=torch.uint8, device=DEV, generator=gen)  # noqa: E731
    cache = ea.Mxfp4Cache(byte(0, 256, 64), byte(124, 127, 4), byte(0, 256, 64), byte(122, 130, 4))
    x = step_inputs(9, hq, tok)
    x["q_gamma"] = x["q_gamma"] * 2
    b, ws = device_buffers(x, cache), alloc(1)
    last = [t[7, -tok - 1].clone() for t in cache.__dict__.values()]
    call([b], n, Smax, 0, ws)
    check_status(ws)
    assert all(torch.equal(t[7, -tok - 1], w) for t, w in zip(cache.__dict__.values(), last))
    import oracle
    f = lambda name: x[name].double().numpy()  # noqa: E731
    args = [f(i) for i in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")]
    q = torch.from_numpy(np.asarray((oracle.decode_prologue if form == "decode" else oracle.prologue)(*args, n, 0)[0])).to(DEV)
    got = b.out.double().reshape(8, -1, 128)
    for g in (0, 7):
        want = attend(q.reshape(8, -1, 128)[g], cache, g, [(0, Smax)])
        assert torch.linalg.norm(got[g] - want) <= REL * torch.linalg.norm(want), g


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("first", [True, False])
def test_half_a_million_keys_far_below_one(form, first):
    """One key e^16.97 above 2^19 equal ones: each weighs 2^-24.5 of it, all together 2 % of the whole. Twenty layers, so
    that a part of the keys that one CTA takes is a head's whole cache."""
    call, alloc, _, hq, tok = FORMS[form]
    Smax, layers = (1 << 19) + 64, 20
    n = Smax - 64
    x = step_inputs(1, hq, tok)
    for name in ("q_gamma", "k_gamma"):
        x[name].fill_(1.0)
    x["q_raw"].zero_()
    x["q_raw"][..., 63] = x["q_raw"][..., 127] = 1.0  # normed: 8 in both; channels that hardly rotate
    x["k_raw"].zero_()
    x["v_raw"].fill_(1.0)
    at = 5 if first else n - 5
    bufs = []
    for _ in range(layers):
        cache = ea.alloc_mxfp4_cache(Smax)
        cache.v_codes.fill_(0x22)          # 1 in every channel
        for t in (cache.k_scales, cache.v_scales):
            t.fill_(127)
        cache.k_codes[:, at, 31] = 0x60    # channel 63: code 6 is 4, times 2^2
        cache.k_codes[:, at, 63] = 0x40    # channel 127: 2, times 2^2
        cache.k_scales[:, at] = 129
        cache.v_codes[:, at] = 0xAA        # -1
        bufs.append(device_buffers(x, cache))
    ws = alloc(layers)
    call(bufs, n, Smax, -n, ws)
    check_status(ws)
    # position 0 (to 63): the rotation by 63 * 5e6^(-63/64) = 1.6e-5 moves the score by less than 1e-3 of a nat
    big, rest = np.exp(8 * (16 + 8) / 128 ** 0.5), n - 1 + tok
    for b in bufs:
        # the output's bf16 rounding, at most 2^-8 of it, and 1e-3 for the rest (the rotation, f16 and fp32)
        want = torch.full(b.out.shape, float((rest - big) / (rest + big)), dtype=torch.float64)
        off, bar = float((b.out.cpu().double() - want).abs().max()), (2.0 ** -8 + 1e-3) * float(want.abs().max())
        assert off <= bar


@pytest.mark.parametrize("layers,pos,Smax", [(10, 8191, 8192), (5, 20000, 20032), (40, 1500, 1536)])
def test_decode_units_cut_anywhere(layers, pos, Smax):
    """Shapes whose units are cut over several CTAs at any chunk, a CTA working on more than one unit; two calls, so that the
    second meets the counters that the first left."""
    call, alloc, ref, hq, tok = FORMS["decode"]
    picks = sorted({0, layers // 2, layers - 1})
    xs = [step_inputs(50 + l, hq, tok) for l in range(layers)]
    hs = [random_cache(60 + l % 3, Smax, pos) for l in range(3)]
    bufs = [device_buffers(x, hs[l % 3].device()) for l, x in enumerate(xs)]
    ws = alloc(layers)
    for _ in range(2):
        for b in bufs:
            b.out.fill_(float("nan"))
        call(bufs, pos, Smax, 0, ws)
        check_status(ws)
        for l in picks:
            close(bufs[l].out, ref(xs[l], hs[l % 3], pos, 0)["out"], f"layer {l}")
        assert all(torch.isfinite(b.out).all() for b in bufs)


@pytest.mark.parametrize("form", FORMS)
def test_a_query_that_is_not_a_number_stays_alone(form):
    call, alloc, ref, hq, tok = FORMS[form]
    x, h = step_inputs(77, hq, tok), random_cache(78, 1024, 700)
    want = ref(x, h, 700, 0)["out"]
    row = (9,) if form == "decode" else (3, 21)
    x["q_raw"][row + (5,)] = float("nan")
    b, ws = device_buffers(x, h.device()), alloc(1)
    call([b], 700, 1024, 0, ws)
    check_status(ws)
    assert torch.isnan(b.out[row]).all()
    b.out[row] = torch.from_numpy(np.asarray(want[row])).to(b.out)
    close(b.out, want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("end", [False, True])
def test_first_and_last_position(form, end):
    call, alloc, ref, hq, tok = FORMS[form]
    x, h = step_inputs(31, hq, tok), random_cache(32, 256, 100)
    delta = (1 << 24) - tok - 100 if end else 1 - (1 << 24) - 100
    b, ws = device_buffers(x, h.device()), alloc(1)
    call([b], 100, 256, delta, ws)
    check_status(ws)
    close(b.out, ref(x, h, 100, delta)["out"])


@pytest.mark.parametrize("form", FORMS)
def test_two_graphs_share_a_workspace(form):
    """Captured at different layer counts and lengths, replayed in turn with inputs that change, an eager call between."""
    call, alloc, ref, hq, tok = FORMS[form]
    shapes = [(1, 1500, 2048), (3, 400, 512)]
    xs = [[step_inputs(10 * i + l, hq, tok) for l in range(n)] for i, (n, _, _) in enumerate(shapes)]
    hs = [[random_cache(20 * i + l, Smax, rows) for l in range(n)] for i, (n, rows, Smax) in enumerate(shapes)]
    bufs = [[device_buffers(x, h.device()) for x, h in zip(a, b)] for a, b in zip(xs, hs)]
    ws, s = alloc(3), torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for b, (_, rows, Smax) in zip(bufs, shapes):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                call(b, rows, Smax, 0, ws)
        for turn in range(2):
            for i in (0, 1, 1, 0):
                x2 = [step_inputs(100 * turn + 10 * i + l, hq, tok) for l in range(shapes[i][0])]
                for b, x in zip(bufs[i], x2):
                    for name, t in x.items():
                        getattr(b, name).copy_(t)
                    b.out.fill_(float("nan"))
                graphs[i].replay()
                outs = [b.out.clone() for b in bufs[i]]
                call(bufs[1 - i], *shapes[1 - i][1:], 0, ws)
                s.synchronize()
                for o, x, h in zip(outs, x2, hs[i]):
                    close(o, ref(x, h, shapes[i][1], 0)["out"], f"turn {turn}, graph {i}")
    check_status(ws)


def test_two_streams_at_once():
    """Both attentions, each with its own workspace and cache, on streams of their own: what they give alone."""
    runs = []
    for form, (call, alloc, ref, hq, tok) in FORMS.items():
        for n, rows, Smax in ((2, 3000, 4096), (9, 300, 384)):
            xs = [step_inputs(7 * l + n, hq, tok) for l in range(n)]
            hs = [random_cache(9 * l + n, Smax, rows) for l in range(n)]
            bufs = [device_buffers(x, h.device()) for x, h in zip(xs, hs)]
            ws = alloc(n)
            call(bufs, rows, Smax, 0, ws)
            runs.append((call, bufs, rows, Smax, ws, [b.out.clone() for b in bufs], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for call, bufs, rows, Smax, ws, _, s in runs:
            with torch.cuda.stream(s):
                call(bufs, rows, Smax, 0, ws)
    torch.cuda.synchronize()
    for _, bufs, _, _, ws, alone, _ in runs:
        check_status(ws)
        for b, o in zip(bufs, alone):
            assert torch.equal(b.out, o)


@pytest.mark.parametrize("form", FORMS)
def test_one_workspace_for_calls_of_different_layer_counts(form):
    """A workspace made for 64 layers serves smaller calls in between: whatever they keep there stays out of the way."""
    call, alloc, ref, hq, tok = FORMS[form]
    ws = alloc(64)
    h = [random_cache(3 + l, 512, 400) for l in range(3)]
    many = [device_buffers(step_inputs(l, hq, tok), h[l % 3].device()) for l in range(64)]
    few = [device_buffers(step_inputs(100 + l, hq, tok), random_cache(8 + l, 1088, 1000).device()) for l in range(3)]
    outs = []
    for _ in range(2):
        for b in many:
            b.out.fill_(float("nan"))
        call(many, 400, 512, 0, ws)
        outs.append([b.out.clone() for b in many])
        call(few, 1000, 1088, 0, ws)
    check_status(ws)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for l in (0, 40, 63):
        close(outs[1][l], ref(step_inputs(l, hq, tok), h[l % 3], 400, 0)["out"], f"layer {l}")
