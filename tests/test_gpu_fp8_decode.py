"""The decode step over an 8-bit cache against the oracle in fp64 over the appended cache's values.

Bars. The output is bf16: at most half a step off, 2^-8 of it, and 2^-8 / sqrt(3) of it in relative L2 over mantissas of every size; softmax
weights are held to 2^-9 (rounded to nearest, of either sign), which adds no more than 2^-9 / sqrt(3) over keys whose V is random, and q to
2^-19 of a row's largest channel: relative L2 <= REL = 2^-8 + 2^-12. A weight is fp32: its relative error is the
error of its score and of the log-sum-exp, each at most (2^-18 + 2^-19) times sum |q k| / sqrt(128), which these inputs keep
under 12: 2 x 12 x 1.5 x 2^-18 < 1.5e-4 = WREL. The stored rows are those of the rule, bit for bit."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._fp8_util import (DEV, F32, HostCache, decode_buffers, decode_inputs, decode_oracle, f64, random_cache, same_cache)
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu
REL, WREL = 2.0 ** -8 + 2.0 ** -12, 1.5e-4


def close(got: torch.Tensor, want: np.ndarray, what: str = "out") -> None:
    got = f64(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= REL, f"{what}: relative L2 {rel:.2e}"


def weights_close(got: torch.Tensor, base, want: np.ndarray, pos: int) -> None:
    """got [8, Smax] against base + want (rows [0, pos)) and want alone (row pos)."""
    got, sums = f64(got)[:, :pos + 1], want.copy()
    if base is not None:
        sums[:, :pos] += f64(base)[:, :pos]
    off = np.abs(got - sums)
    assert (off <= WREL * want + 2.0 ** -23 * np.abs(sums) + 1e-37).all(), float((off / (want + 1e-30)).max())


def step(x, h, pos, delta=0, layers=1, base=None, in_place=False, ws=None):
    """One layer's step (other layers get copies), checked whole; base: weights before it."""
    bufs, Smax = [], h.Smax
    for _ in range(layers):
        wo = None
        if base is not None:
            wo = base.clone() if in_place else torch.full_like(base, -7.0)
        bufs.append(decode_buffers(x, h.device(), base if base is None or not in_place else wo, wo))
    if layers > 1 and base is not None and not in_place:
        for b in bufs:
            b.weight_in = base.clone()
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=base is not None) if ws is None else ws
    ea.text_decode_attention_fp8(bufs, pos, Smax, delta, ws)
    check_status(ws)
    r = decode_oracle(x, h, pos, delta)
    for b in bufs:
        same_cache(b.cache, h, signs=False)
        close(b.out, r["out"])
        assert torch.equal(b.k_new.cpu(), torch.from_numpy(r["k"].astype(F32)).to(torch.bfloat16))
        assert torch.equal(b.v_new.cpu(), torch.from_numpy(r["v"].astype(F32)).to(torch.bfloat16))
        if base is not None:
            weights_close(b.weight_out, base, r["weight"], pos)
            assert torch.equal(b.weight_out[:, pos + 1:], base[:, pos + 1:]) if in_place else (b.weight_out[:, pos + 1:] == -7.0).all()
    return bufs, r


def sums(seed, Smax):
    return torch.from_numpy(np.random.default_rng(seed).gamma(0.3, 2.0, (8, Smax)).astype(F32)).to(DEV)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("pos,Smax,delta", [(0, 128, 0), (1, 128, 5), (31, 128, -31), (127, 128, 0), (128, 256, 0), (129, 384, 7),
                                            (255, 256, -3), (300, 512, 0), (1000, 1024, 4000), (1023, 1024, 0), (1024, 1152, 0),
                                            (2500, 4096, -400), (4700, 8192, -37)])
def test_lengths(pos, Smax, delta, weights):
    """Rows behind pos are NaN codes, under NaN scales where a block holds nothing."""
    step(decode_inputs(pos), random_cache(pos + 1, Smax, pos), pos, delta, base=sums(pos, Smax) if weights else None)


@pytest.mark.parametrize("layers,pos,Smax", [(2, 700, 1024), (3, 4700, 4736), (8, 130, 256), (9, 2000, 2048), (20, 1500, 1536), (64, 200, 256), (70, 383, 384)])
def test_layers(layers, pos, Smax):
    """Units cut anywhere over the CTAs; more than 64 layers are more than one launch."""
    step(decode_inputs(layers), random_cache(layers, Smax, pos), pos, 0, layers, sums(1, Smax), in_place=layers % 2 == 0)


@pytest.mark.parametrize("layers,pos,Smax", [(20, 4000, 4096), (40, 2303, 2304), (64, 1200, 1280), (33, 1024, 1152), (5, 20000, 20096)])
def test_units_cut_anywhere(layers, pos, Smax):
    """More than 14 key tiles to an SM: CTAs that work on several units, whole and in parts; layers that differ, new rows that need
    larger scales; a second call meets the counters that the first left."""
    hs = [random_cache(60 + l, Smax, pos, v_gain=4.0 ** -l) for l in range(3)]
    xs = [decode_inputs(50 + l) for l in range(3)]
    for l, x in enumerate(xs):
        x["k_gamma"] = x["k_gamma"] * (1 + 2 * l)
    base = [sums(l, Smax) for l in range(3)]
    bufs = [decode_buffers(xs[l % 3], hs[l % 3].device(), base[l % 3].clone(), torch.full((8, Smax), -7.0, device=DEV)) for l in range(layers)]
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=True)
    want = [decode_oracle(xs[l], hs[l], pos, 0) for l in range(3)]
    for _ in range(2):  # (the second call's rows are there already, and fit)
        for b in bufs:
            b.out.fill_(float("nan"))
            b.weight_out.fill_(-7.0)
        ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
        check_status(ws)
        for l, b in enumerate(bufs):
            if l < 3 or l % 7 == 0 or l == layers - 1:
                same_cache(b.cache, hs[l % 3], f"layer {l}")
            close(b.out, want[l % 3]["out"], f"layer {l}")
            weights_close(b.weight_out, base[l % 3], want[l % 3]["weight"], pos)
            assert (b.weight_out[:, pos + 1:] == -7.0).all()


@pytest.mark.parametrize("pos,Smax,layers", [(900, 1024, 5), (4000, 4096, 14)])
def test_weights_of_some_layers_only(pos, Smax, layers):
    h, base = random_cache(3, Smax, pos), sums(2, Smax)
    bufs = [decode_buffers(decode_inputs(4), h.device(), None, torch.full_like(base, -7.0) if l % 3 == 1 else None) for l in range(layers)]
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=True)
    ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
    check_status(ws)
    r = decode_oracle(decode_inputs(4), h, pos, 0)
    for b in bufs:
        close(b.out, r["out"])
        if b.weight_out is not None:
            weights_close(b.weight_out, None, r["weight"], pos)  # without sums before it: this step's alone
            assert (b.weight_out[:, pos + 1:] == -7.0).all()


def test_a_generation_fills_blocks():
    """Steps across a block's end, k growing: scales grow, codes move, sums add up in place."""
    Smax, h, ws = 256, random_cache(5, 256, 120), ea.alloc_decode_fp8_workspace(1, 256, weights=True)
    cache, base = h.device(), sums(6, Smax)
    want = f64(base).copy()
    for i, pos in enumerate(range(120, 134)):
        x = decode_inputs(100 + i)
        x["k_gamma"] = x["k_gamma"] * (1 + i)
        x["v_raw"] = x["v_raw"] * (1 + i)
        b = decode_buffers(x, cache, base, base)
        ea.text_decode_attention_fp8([b], pos, Smax, 0, ws)
        r = decode_oracle(x, h, pos, 0)
        same_cache(cache, h, f"pos {pos}")
        close(b.out, r["out"], f"pos {pos}")
        want[:, :pos] += r["weight"][:, :pos]
        want[:, pos] = r["weight"][:, pos]
    check_status(ws)
    assert (np.abs(f64(base)[:, :134] - want[:, :134]) <= 14 * 2.0 ** -23 * want[:, :134] + 14 * WREL).all()


@pytest.mark.parametrize("k_range,v_range", [(0, 60), (8, 8), (0, 200)])
def test_scales_far_apart(k_range, v_range):
    """Blocks whose V scales (and K scales) differ by up to 2^200: each tile's share is formed by itself, in fp32."""
    Smax, pos = 1280, 1200
    h = random_cache(7, Smax, pos)
    rng = np.random.default_rng(8)
    for i, span in enumerate((k_range, v_range)):
        if span:
            e = rng.integers(-span // 2, span // 2 + 1, h.scales[i].shape)
            if i == 0:
                e = -np.abs(e)  # keys that are all but zero: no score leaves the softmax's range
            h.scales[i] = (h.scales[i] * np.exp2(e)).astype(F32)
    h.scales[1][:, 9] = np.maximum(h.scales[1][:, 9], F32(2.0 ** -20))  # (the block that the new row joins)
    step(decode_inputs(9), h, pos, base=sums(3, Smax))


def test_one_key_that_decides_and_a_block_that_outweighs_it():
    """A block of V 2^40 larger under keys e^-25 lower still decides the output."""
    Smax, pos = 384, 300
    h = random_cache(10, Smax, pos, k_gain=0.01)
    x = decode_inputs(11)
    for n in ("q_gamma", "k_gamma"):
        x[n].fill_(1.0)
    x["q_raw"].fill_(1.0)  # after the norm: ones; the rotation at position 0 leaves them
    h.scales[0][:, :2] = F32(2.0 ** -9)
    h.codes[0][:, 5] = 0x7E  # 448 in every channel: 448 * 2^-9 * 128 / 11.3 = 9.9
    h.codes[0][:, 5, 64:] = 0x7E
    h.scales[1][:, 1] *= F32(2.0 ** 40)
    step(x, h, pos, -pos, base=sums(4, Smax))


def test_infinite_and_nan_codes_of_held_rows():
    """A NaN in a held row makes its heads NaN (K: all channels; V: its channel), and no other head."""
    Smax, pos = 256, 200
    h = random_cache(12, Smax, pos)
    h.codes[0][2, 17, 3] = 0x7F
    h.codes[1][5, 140, 9] = 0xFF
    x = decode_inputs(13)
    b, ws = decode_buffers(x, h.device(), None, torch.zeros(8, Smax, device=DEV)), ea.alloc_decode_fp8_workspace(1, Smax, weights=True)
    ea.text_decode_attention_fp8([b], pos, Smax, 0, ws)
    check_status(ws)
    r = decode_oracle(x, h, pos, 0)
    out = b.out.cpu()
    assert torch.isnan(out[16:24]).all() and torch.isnan(out[40:48, 9]).all()
    rest = ~np.isnan(r["out"])
    assert np.array_equal(torch.isnan(out).numpy(), ~rest)
    assert np.linalg.norm((f64(out) - r["out"])[rest]) <= REL * np.linalg.norm(r["out"][rest])
    w = b.weight_out.cpu()[:, :pos + 1]
    assert torch.isnan(w[2]).all() and torch.isfinite(w[[0, 1, 3, 4, 5, 6, 7]]).all()


def test_a_query_that_is_not_a_number_stays_alone():
    Smax, pos, x = 1024, 700, decode_inputs(77)
    h = random_cache(78, Smax, pos)
    r = decode_oracle(x, h.copy(), pos, 0)
    x["q_raw"][9, 5] = float("nan")
    b, ws = decode_buffers(x, h.device()), ea.alloc_decode_fp8_workspace(1, Smax)
    ea.text_decode_attention_fp8([b], pos, Smax, 0, ws)
    check_status(ws)
    assert torch.isnan(b.out[9]).all()
    b.out[9] = torch.from_numpy(r["out"][9]).to(b.out)
    close(b.out, r["out"])


@pytest.mark.parametrize("end", [False, True])
def test_first_and_last_position(end):
    step(decode_inputs(31), random_cache(32, 256, 100), 100, (1 << 24) - 1 - 100 if end else 1 - (1 << 24) - 100)


def test_zero_query_and_zero_rows():
    """A query of zeros weighs all keys alike; zero k and v rows are stored as zeros."""
    x, h = decode_inputs(33), random_cache(34, 256, 130)
    for n in ("q_raw", "k_raw", "v_raw"):
        x[n].zero_()
    step(x, h, 130, base=sums(5, 256))


def test_long_cache_with_a_far_maximum():
    """70001 keys; the largest scores come last, then first."""
    Smax, pos = 70144, 70000
    for at in (5, pos - 3):
        h = HostCache(Smax)
        rng = np.random.default_rng(35)
        for i in range(2):
            h.codes[i][:, :pos] = rng.integers(0, 0x60, (8, pos, 128), dtype=np.uint8) | (rng.integers(0, 2, (8, pos, 128), dtype=np.uint8) << 7)
            h.scales[i][:, :-1] = F32(2.0 ** -6)
        h.codes[0][:, at] = 0x6C
        x = decode_inputs(36)
        x["q_raw"].fill_(1.0)
        step(x, h, pos, -pos, base=sums(7, Smax))


def test_offsets_past_32_bits():
    """The largest cache: 8 heads x 2^22 rows; the last rows are keys that decide."""
    Smax = 1 << 22
    pos = Smax - 1
    cache = ea.alloc_fp8_cache(Smax)
    cache.k_scale.fill_(2.0 ** -7)
    cache.v_scale.fill_(2.0 ** -7)
    h = HostCache(128)
    rng = np.random.default_rng(37)
    for i, c in enumerate((cache.k_cache, cache.v_cache)):
        h.codes[i][:] = rng.integers(0, 0x70, h.codes[i].shape, dtype=np.uint8)
        h.scales[i][:] = F32(2.0 ** -7)
        c[:, -128:] = torch.from_numpy(h.codes[i]).to(DEV)
    x = decode_inputs(38)
    w = torch.full((8, Smax), -7.0, device=DEV)
    b, ws = decode_buffers(x, cache, None, w), ea.alloc_decode_fp8_workspace(1, Smax, weights=True)
    ea.text_decode_attention_fp8([b], pos, Smax, 0, ws)
    check_status(ws)
    import oracle
    q, k, v = oracle.decode_prologue(*(f64(x[n]) for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")), pos, 0)
    h.append(0, k.astype(F32)[:, None], 127)
    h.append(1, v.astype(F32)[:, None], 127)
    keys, vals, rest = h.values(0, 128), h.values(1, 128), Smax - 128  # the others: zero keys and values
    for g in range(8):
        s = q[8 * g:8 * g + 8] @ keys[g].T / np.sqrt(128)
        top = np.maximum(s.max(1, keepdims=True), 0)
        p = np.exp(s - top)
        den = p.sum(1, keepdims=True) + rest * np.exp(-top)
        close(b.out[8 * g:8 * g + 8], p @ vals[g] / den, f"head {g}")
        ww = f64(w[g])
        assert np.allclose(ww[-128:], (p / den).sum(0), rtol=WREL, atol=0)
        assert np.allclose(ww[:-128], (np.exp(-top) / den).sum(), rtol=WREL, atol=0)
    assert torch.equal(cache.k_cache[7, -1].cpu(), torch.from_numpy(h.codes[0][7, -1]))


def test_two_graphs_share_a_workspace():
    """Captured at different layer counts and lengths, replayed in turn with inputs that change, an eager call between."""
    shapes = [(1, 1500, 2048), (3, 400, 512)]
    hs = [[random_cache(20 * i + l, Smax, pos) for l in range(n)] for i, (n, pos, Smax) in enumerate(shapes)]
    bufs = [[decode_buffers(decode_inputs(10 * i + l), h.device(), None, torch.zeros(8, shapes[i][2], device=DEV)) for l, h in enumerate(b)] for i, b in enumerate(hs)]
    ws, s = ea.alloc_decode_fp8_workspace(3, 2048, weights=True), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for b, (_, pos, Smax) in zip(bufs, shapes):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            ea.text_decode_attention_fp8(b, pos, Smax, 0, ws)
    with torch.cuda.stream(s):
        for turn in range(2):
            for i in (0, 1, 1, 0):
                xs = [decode_inputs(100 * turn + 10 * i + l) for l in range(shapes[i][0])]
                for b, x in zip(bufs[i], xs):
                    for name, t in x.items():
                        getattr(b, name).copy_(t)
                    b.out.fill_(float("nan"))
                graphs[i].replay()
                got = [(b.out.clone(), b.weight_out.clone()) for b in bufs[i]]
                j = 1 - i
                ea.text_decode_attention_fp8(bufs[j], shapes[j][1], shapes[j][2], 0, ws)
                s.synchronize()
                for (o, w), x, h in zip(got, xs, hs[i]):
                    r = decode_oracle(x, h, shapes[i][1], 0)
                    close(o, r["out"], f"turn {turn}, graph {i}")
                    weights_close(w, None, r["weight"], shapes[i][1])
                for b, h in zip(bufs[j], hs[j]):  # the eager call appended, too
                    decode_oracle({n: getattr(b, n).cpu() for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")}, h, shapes[j][1], 0)
    check_status(ws)


def test_two_streams_at_once():
    """Calls with a workspace and caches of their own, on streams of their own: what they give alone, to the bit."""
    runs = []
    for n, pos, Smax in ((2, 3000, 3200), (20, 2000, 2048), (1, 4000, 4096)):
        bufs = [decode_buffers(decode_inputs(7 * l + n), random_cache(9 * l % 4 + n, Smax, pos).device(), None, torch.zeros(8, Smax, device=DEV)) for l in range(n)]
        ws = ea.alloc_decode_fp8_workspace(n, Smax, weights=True)
        for _ in range(2):
            ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
        runs.append((bufs, pos, Smax, ws, [(b.out.clone(), b.weight_out.clone()) for b in bufs], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for bufs, pos, Smax, ws, _, s in runs:
            with torch.cuda.stream(s):
                ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
    torch.cuda.synchronize()
    for bufs, _, _, ws, alone, _ in runs:
        check_status(ws)
        for b, (o, w) in zip(bufs, alone):
            assert torch.equal(b.out, o) and torch.equal(b.weight_out, w)


def test_one_workspace_for_calls_of_different_layer_counts():
    ws = ea.alloc_decode_fp8_workspace(64, 1152, weights=True)
    hs = [random_cache(3 + l, 1024, 900) for l in range(3)]
    many = [decode_buffers(decode_inputs(l), hs[l % 3].device(), None, torch.zeros(8, 1024, device=DEV)) for l in range(64)]
    few = [decode_buffers(decode_inputs(100 + l), random_cache(8 + l, 1152, 1000).device()) for l in range(3)]
    ea.text_decode_attention_fp8(many, 900, 1024, 0, ws)  # (a first one: what a second appends is there already)
    outs = []
    for _ in range(2):
        for b in many:
            b.out.fill_(float("nan"))
        ea.text_decode_attention_fp8(many, 900, 1024, 0, ws)
        outs.append([(b.out.clone(), b.weight_out.clone()) for b in many])
        ea.text_decode_attention_fp8(few, 1000, 1152, 0, ws)
    check_status(ws)
    for (a, v), (b, w) in zip(*outs):
        assert torch.equal(a, b) and torch.equal(v, w)
    for l in (0, 40, 63):
        close(outs[1][l][0], decode_oracle(decode_inputs(l), hs[l % 3].copy(), 900, 0)["out"], f"layer {l}")


def test_workspace_too_small_is_refused():
    b = decode_buffers(decode_inputs(1), random_cache(1, 256, 100).device(), None, torch.zeros(8, 256, device=DEV))
    ws = ea.alloc_decode_fp8_workspace(1, 256, weights=False)
    with pytest.raises(ea.ExpertAttnError, match="workspace"):
        ea.text_decode_attention_fp8([b], 100, 256, 0, ws)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("layers", [1, 20])
def test_many_keys_far_below_one(layers, first):
    """One key e^16.97 above the others, which all together weigh 2 % of it (2^19 keys), or 2^-9 (2^14 keys, twenty layers): a weight
    that its own tile's largest outweighs by 2^24 may count as zero, those of the other tiles must not."""
    n = 1 << (19 if layers == 1 else 14)
    Smax, at = n + 128, 5 if first else n - 5
    x = decode_inputs(1)
    for name in ("q_gamma", "k_gamma"):
        x[name].fill_(1.0)
    x["q_raw"].zero_()
    x["q_raw"][..., 63] = x["q_raw"][..., 127] = 1.0  # normed: 8 in both
    x["k_raw"].zero_()
    x["v_raw"].fill_(1.0)
    bufs = []
    for _ in range(layers):
        cache = ea.alloc_fp8_cache(Smax)
        cache.v_cache.fill_(0x38)        # 1 in every channel, under scales of 1
        cache.k_cache[:, at, 63] = 0x58  # 16
        cache.k_cache[:, at, 127] = 0x50  # 8: 8 * 24 / sqrt(128) = 16.97
        cache.v_cache[:, at] = 0xB8      # -1
        bufs.append(decode_buffers(x, cache, None, torch.zeros(8, Smax, device=DEV)))
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=True)
    ea.text_decode_attention_fp8(bufs, n, Smax, -n, ws)
    check_status(ws)
    big, rest = np.exp(8 * 24 / 128 ** 0.5), n
    for b in bufs:
        want = (rest - big) / (rest + big)
        assert float((b.out.double() - want).abs().max()) <= (2.0 ** -8 + 2.0 ** -12) * abs(want)
        w = f64(b.weight_out)
        assert np.allclose(w[:, at], 8 * big / (rest + big), rtol=WREL) and np.allclose(w[:, at + 1:n + 1], 8 / (rest + big), rtol=WREL)


@pytest.mark.parametrize("layers,pos", [(29, 39 * 128 - 1), (29, 39 * 128), (30, 39 * 128 - 127), (64, 5 * 128 - 1), (64, 1300), (40, 2561),
                                        (65, 38 * 128 + 77)])
def test_weights_of_many_layers(layers, pos):
    """One to three whole units and parts of two more to a CTA, with sums before in place, elsewhere, nowhere, and layers without weights."""
    Smax = (pos // 128 + 1) * 128 + 128
    x, h = decode_inputs(11), random_cache(5, Smax, pos)
    g = torch.Generator(device=DEV).manual_seed(9)
    base = torch.rand(8, Smax, generator=g, device=DEV)
    bufs, kinds = [], []
    for i in range(layers):
        kind = ("in place", "elsewhere", "nowhere", "elsewhere", "none")[i % 5 if i < layers - 6 else 1]
        wo = {"in place": base.clone(), "none": None}.get(kind, torch.full_like(base, -7.0))
        wi = {"in place": wo, "elsewhere": base.clone()}.get(kind)
        bufs.append(decode_buffers(x, h.device(), wi, wo))
        kinds.append(kind)
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=True)
    ea.text_decode_attention_fp8(bufs, pos, Smax, 3, ws)
    check_status(ws)
    r = decode_oracle(x, h, pos, 3)
    for b, kind in zip(bufs, kinds):
        same_cache(b.cache, h, signs=False)
        close(b.out, r["out"])
        if kind != "none":
            weights_close(b.weight_out, None if kind == "nowhere" else base, r["weight"], pos)
            assert torch.equal(b.weight_out[:, pos + 1:], base[:, pos + 1:]) if kind == "in place" else (b.weight_out[:, pos + 1:] == -7.0).all()


def test_weights_of_many_layers_in_captured_steps():
    """In place, thirty layers, a captured step replayed four times while another stream has calls of its own: each adds the same weights
    (four fp32 additions, each off by at most half a step)."""
    n, pos, Smax = 30, 1400, 1536
    x, h = decode_inputs(21), random_cache(22, Smax, pos)
    base = torch.rand(8, Smax, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    mine, others = ([decode_buffers(x, h.device(), w, w) for w in (base.clone() for _ in range(n))] for _ in range(2))
    ws, ws2 = (ea.alloc_decode_fp8_workspace(n, Smax, weights=True) for _ in range(2))
    s, s2, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        ea.text_decode_attention_fp8(mine, pos, Smax, 0, ws)
    for _ in range(4):
        with torch.cuda.stream(s):
            graph.replay()
        with torch.cuda.stream(s2):
            ea.text_decode_attention_fp8(others, pos, Smax, 0, ws2)
    torch.cuda.synchronize()
    check_status(ws)
    check_status(ws2)
    r = decode_oracle(x, h, pos, 0)
    want = f64(base)[:, :pos] + 4 * r["weight"][:, :pos]
    for b in mine + others:
        close(b.out, r["out"])
        got = f64(b.weight_out)
        assert (np.abs(got[:, :pos] - want) <= 4 * WREL * r["weight"][:, :pos] + 4 * 2.0 ** -24 * want).all()
        assert (np.abs(got[:, pos] - r["weight"][:, pos]) <= WREL * r["weight"][:, pos]).all()
        assert torch.equal(b.weight_out[:, pos + 1:], base[:, pos + 1:])


@pytest.mark.parametrize("layers,pos", [(5, 700), (5, 127), (5, 128), (20, 200), (12, 1400), (10, 3327), (40, 640)])
def test_weights_of_a_few_tiles(layers, pos):
    """Units of one CTA and of a cluster, with sums before in place, elsewhere, nowhere, and layers without weights."""
    Smax = (pos // 128 + 1) * 128
    x, h = decode_inputs(31), random_cache(32, Smax, pos)
    base = torch.rand(8, Smax, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    bufs, kinds = [], [("in place", "none", "nowhere", "elsewhere", "elsewhere")[i % 5] for i in range(layers)]
    for kind in kinds:
        wo = {"in place": base.clone(), "none": None}.get(kind, torch.full_like(base, -7.0))
        bufs.append(decode_buffers(x, h.device(), {"in place": wo, "elsewhere": base.clone()}.get(kind), wo))
    ws = ea.alloc_decode_fp8_workspace(layers, Smax, weights=True)
    ea.text_decode_attention_fp8(bufs, pos, Smax, 0, ws)
    check_status(ws)
    r = decode_oracle(x, h, pos, 0)
    for b, kind in zip(bufs, kinds):
        same_cache(b.cache, h, signs=False)
        close(b.out, r["out"])
        if kind != "none":
            weights_close(b.weight_out, None if kind == "nowhere" else base, r["weight"], pos)
            assert torch.equal(b.weight_out[:, pos + 1:], base[:, pos + 1:]) if kind == "in place" else (b.weight_out[:, pos + 1:] == -7.0).all()
