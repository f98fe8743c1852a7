"""The cases on which the operators over an 8-bit KV cache are measured.

A cache of one layer holds K and V rows [8 heads][Smax][128] as e4m3 codes with one fp32 scale for
each head and block of 128 rows, [8][Smax / 128 + 1] (the last column belongs to rows that another
call writes). Four operators work on it:

  write   rows [row0, row0 + n) of K and V appended (the block that row0 falls into gets a larger
          scale where the new rows need one), then the touched blocks' rows read back
  decode  one token's attention of 64 query heads over rows [0, pos], row pos written first
  weigh   the same, which also adds every row's attention weights, summed over the 8 query heads
          of its KV head, to what earlier tokens left there
  evict   of n rows those of most weight kept, in order, beside the first and the latest ones, and
          moved together

``run`` computes them in plain torch, or, where ``own`` is true, by this repository's calls.
"""
import math

import torch

own = False

HQ, HKV, D, BLOCK = 64, 8, 128, 128
THETA, EPS = 5.0e6, 1e-6
E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one layer of the text model early in a conversation: the call's own latency
        {"name": "decode 1 layer pos 300", "op": "decode", "layers": 1, "pos": 300, "Smax": 512, "delta": 0},
        # one layer at the driving prompt's length, called layer by layer by the model
        {"name": "decode 1 layer pos 4700", "op": "decode", "layers": 1, "pos": 4700, "Smax": 8192, "delta": -37},
        # the attention of a whole decode step, all layers' caches at once
        {"name": "decode 64 layers pos 4700", "op": "decode", "layers": 64, "pos": 4700, "Smax": 8192, "delta": 0},
        # a few layers over a very long context, one row short of the cache's end
        {"name": "decode 4 layers pos 131070", "op": "decode", "layers": 4, "pos": 131070, "Smax": 131072, "delta": 0},
        # one layer of a step whose weights decide what is evicted later; the cache has been thinned before
        {"name": "weigh 1 layer pos 4700", "op": "weigh", "layers": 1, "pos": 4700, "Smax": 8192, "delta": 9001},
        # the same step over all layers
        {"name": "weigh 64 layers pos 4700", "op": "weigh", "layers": 64, "pos": 4700, "Smax": 8192, "delta": 0},
        # one new token's rows in every layer, cut out of the fused projection's output
        {"name": "write 64 layers 1 row", "op": "write", "layers": 64, "row0": 4700, "rows": 1, "Smax": 8192,
         "dtype": "bf16", "order": "token"},
        # a prompt's rows after its prefill, behind a short cached prefix
        {"name": "write 16 layers 4700 rows", "op": "write", "layers": 16, "row0": 77, "rows": 4700, "Smax": 8192,
         "dtype": "bf16", "order": "head"},
        # a small cache thinned layer by layer
        {"name": "evict 1 layer 300 to 256", "op": "evict", "layers": 1, "rows": 300, "keep": 256, "first": 4,
         "recent": 64, "Smax": 512},
        # one layer at the driving prompt's length
        {"name": "evict 1 layer 4700 to 4096", "op": "evict", "layers": 1, "rows": 4700, "keep": 4096, "first": 4,
         "recent": 512, "Smax": 8192},
        # all layers at that length, as after a prompt
        {"name": "evict 64 layers 4700 to 4096", "op": "evict", "layers": 64, "rows": 4700, "keep": 4096, "first": 0,
         "recent": 1000, "Smax": 8192},
        # a very long context cut to a quarter
        {"name": "evict 2 layers 131001 to 32769", "op": "evict", "layers": 2, "rows": 131001, "keep": 32769, "first": 16,
         "recent": 4097, "Smax": 131072},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["decode", "weigh", "write", "evict"])
    layers = _log(rng, 1, 64)
    if op in ("decode", "weigh"):
        pos = _log(rng, 1, min(131071, (524288 if op == "decode" else 300000) // layers)) - 1
        return {"op": op, "layers": layers, "pos": pos, "Smax": (pos // BLOCK + 1 + rng.randrange(3)) * BLOCK,
                "delta": rng.randrange(-400, 9000)}
    if op == "write":
        rows, row0 = _log(rng, 1, 52000 // layers), rng.randrange(300)
        return {"op": op, "layers": layers, "row0": row0, "rows": rows, "Smax": ((row0 + rows) // BLOCK + 1 + rng.randrange(2)) * BLOCK,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "order": rng.choice(["head", "token"])}
    rows = _log(rng, 2, min(131000, 262000 // layers))
    keep = rng.randrange(rows // 4 + 1, rows)
    first = rng.choice([0, rng.randrange(keep // 8 + 1)])
    return {"op": op, "layers": layers, "rows": rows, "keep": keep, "first": first, "recent": rng.randrange((keep - first) // 2 + 1),
            "Smax": ((rows - 1) // BLOCK + 1 + rng.randrange(3)) * BLOCK}


# ------------------------------------------------------------------------------------- inputs
def _held(case):
    """Rows that the cache holds before the call."""
    return case["pos"] if case["op"] in ("decode", "weigh") else case["row0"] if case["op"] == "write" else case["rows"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, Smax, bf = case["layers"], case["Smax"], torch.bfloat16
    held, st = _held(case), {"case": case}
    # the cache as a prompt's rows left it: K with the channel gains of a k norm; a block's scale is the largest magnitude
    # of its rows over 448. Made two layers at a time.
    st["cache"] = [torch.zeros(n, HKV, Smax, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    st["scale"] = [torch.ones(n, HKV, Smax // BLOCK + 1, device="cuda") for _ in range(2)]
    for i in range(0, n, 2):
        m = min(2, n - i)
        for j, gain in ((0, torch.exp(0.5 * rand(D))), (1, 1.0)):
            b = (rand(m, HKV, Smax, D) * gain).to(bf).float().unflatten(2, (-1, BLOCK))
            b[:, :, held // BLOCK:].flatten(2, 3)[:, :, held % BLOCK:] = 0
            amax = b.abs().amax((-2, -1))
            s = torch.where(amax > 0, amax / 448, 1.0)
            st["cache"][j][i:i + m] = (b / s[..., None, None]).to(E4M3).view(torch.uint8).flatten(2, 3)
            st["scale"][j][i:i + m, :, :-1] = s
    if case["op"] in ("decode", "weigh"):
        st["q"], st["k"], st["v"] = (rand(n, h, D).to(bf) for h in (HQ, HKV, HKV))
        st["q_gamma"], st["k_gamma"] = ((1 + 0.1 * rand(n, D)).to(bf) for _ in range(2))
        st["out"] = torch.empty(n, HQ, D, dtype=bf, device="cuda")
        st["k_new"], st["v_new"] = (torch.empty(n, HKV, D, dtype=bf, device="cuda") for _ in range(2))
    if case["op"] in ("weigh", "evict"):
        # sums of many tokens' weights: a few rows hold most of it, some rows nothing yet
        st["weight"] = torch.exp(2 * rand(n, HKV, Smax)) * (rand(n, HKV, Smax) > -1.5)
        st["weight_out"] = torch.empty_like(st["weight"])
    if case["op"] == "write":
        rows, dt = case["rows"], DTYPES[case["dtype"]]
        if case["order"] == "head":
            st["k"], st["v"] = (rand(n, HKV, rows, D).to(dt) for _ in range(2))
        else:  # the k and v columns of a fused projection's output [rows][k | v]
            fused = rand(n, rows, 2, HKV, D).to(dt)
            st["k"], st["v"] = (fused[:, :, i].transpose(1, 2) for i in range(2))
        a = case["row0"] // BLOCK * BLOCK  # read back from the first touched block's start
        st["k_back"], st["v_back"] = (torch.empty(n, HKV, case["row0"] + rows - a, D, dtype=dt, device="cuda") for _ in range(2))
    if case["op"] == "evict":
        st["to"] = [torch.zeros_like(c) for c in st["cache"]]
        st["to_scale"] = [torch.ones_like(s) for s in st["scale"]]
        st["kept"] = torch.empty(n, HKV, case["keep"], dtype=torch.int32, device="cuda")
    if own:
        import gqa_attention_long_gb300 as ea
        caches = [ea.Fp8Cache(*(t[i] for t in (*st["cache"], *st["scale"]))) for i in range(n)]
        if case["op"] in ("decode", "weigh"):
            w = case["op"] == "weigh"
            st["args"] = ea.make_decode_fp8_args([ea.DecodeFp8Buffers(
                st["q"][i], st["k"][i], st["v"][i], st["q_gamma"][i], st["k_gamma"][i], caches[i], st["out"][i], st["k_new"][i],
                st["v_new"][i], st["weight"][i] if w else None, st["weight_out"][i] if w else None) for i in range(n)], Smax)
            st["ws"] = ea.alloc_decode_fp8_workspace(n, Smax, weights=w)
            st["got"] = (st["out"], st["k_new"], st["v_new"], *_tail(st))
            st["got"] += (st["weight_out"][..., :case["pos"] + 1],) if w else ()
        elif case["op"] == "write":
            st["args"] = ea.make_fp8_rows_args([ea.Fp8Rows(st["k"][i], st["v"][i], caches[i]) for i in range(n)], Smax)
            st["back"] = ea.make_fp8_rows_args([ea.Fp8Rows(st["k_back"][i], st["v_back"][i], caches[i]) for i in range(n)], Smax)
        else:
            to = [ea.Fp8Cache(*(t[i] for t in (*st["to"], *st["to_scale"]))) for i in range(n)]
            st["args"] = ea.make_evict_fp8_args([ea.EvictFp8Buffers(caches[i], st["weight"][i], st["kept"][i], to[i],
                                                                  st["weight_out"][i]) for i in range(n)], Smax)
            st["ws"] = ea.alloc_evict_fp8_workspace(n, Smax)
            keep = case["keep"]
            k, v = (c[:, :, :keep].view(E4M3) for c in st["to"])
            ks, vs = (s[..., :(keep - 1) // BLOCK + 1] for s in st["to_scale"])
            st["got"] = (st["kept"], st["weight_out"][..., :keep], k, v, ks, vs)
    return st


# ----------------------------------------------------------------------------------- plain forms
def _values(codes, scales, a, b):
    """Rows [a, b) of a cache as fp32 numbers."""
    per_row = scales[..., :-1].repeat_interleave(BLOCK, -1)[..., a:b]
    return codes[:, :, a:b].view(E4M3).float() * per_row[..., None]


def _codes(x):
    return x.clamp(-448, 448).to(E4M3).view(torch.uint8)


def _pow2(e):
    """2^e in fp32, |e| <= 126, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _append(codes, scales, x, row0):
    """Rows x [n, 8, rows, 128] into cache rows [row0, row0 + rows)."""
    x = x.float()
    n, b0, b1 = x.shape[2], row0 // BLOCK, (row0 + x.shape[2] - 1) // BLOCK + 1
    pad = torch.zeros(*x.shape[:2], (b1 - b0) * BLOCK, D, device=x.device)
    pad[:, :, row0 - b0 * BLOCK:row0 - b0 * BLOCK + n] = x
    blocks = pad.unflatten(2, (-1, BLOCK))
    amax = blocks.abs().amax((-2, -1))
    s = torch.full_like(amax, 2.0 ** -100)  # of blocks that begin here
    if row0 % BLOCK:
        s[..., 0] = scales[..., b0]
    (ma, ea), (mt, et) = torch.frexp(amax), torch.frexp(s * 448)
    k = torch.where(amax > 0, ea - et + (ma > mt), 0).clamp(min=0)  # the least with amax <= 448 s 2^k
    s = s * _pow2(k - k // 2) * _pow2(k // 2)
    new = _codes(blocks / s[..., None, None])
    old = codes[:, :, b0 * BLOCK:row0]
    codes[:, :, b0 * BLOCK:row0] = _codes(old.view(E4M3).float() * _pow2(-k[..., 0].clamp(max=60))[..., None, None])
    codes[:, :, row0:row0 + n] = new.flatten(2, 3)[:, :, row0 - b0 * BLOCK:row0 - b0 * BLOCK + n]
    scales[..., b0:b1] = s


def _norm_rope(x, gamma, p):
    """RMS norm and rotate_half RoPE of x [n, heads, 128] at position p, in 64 bits: the angles of far positions and codes
    next to a border need them."""
    x = x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.double()[:, None]
    a = p * THETA ** (-torch.arange(D // 2, dtype=torch.float64, device=x.device) / (D // 2))
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1).float()


def _plain(st):
    case, (kc, vc), (ks, vs) = st["case"], st["cache"], st["scale"]
    if case["op"] == "write":
        a, b = case["row0"] // BLOCK * BLOCK, case["row0"] + case["rows"]
        _append(kc, ks, st["k"], case["row0"])
        _append(vc, vs, st["v"], case["row0"])
        return _values(kc, ks, a, b).to(st["k"].dtype), _values(vc, vs, a, b).to(st["k"].dtype)
    if case["op"] == "evict":
        return _plain_evict(st)
    pos, p = case["pos"], case["pos"] + case["delta"]
    _append(kc, ks, _norm_rope(st["k"], st["k_gamma"], p)[:, :, None], pos)
    _append(vc, vs, st["v"][:, :, None], pos)
    k, v = _values(kc, ks, 0, pos + 1), _values(vc, vs, 0, pos + 1)
    q = _norm_rope(st["q"], st["q_gamma"], p).unflatten(1, (HKV, -1))
    s = q @ k.transpose(-1, -2) / math.sqrt(D)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    w = e / e.sum(-1, keepdim=True)
    got = ((w @ v).flatten(1, 2).to(torch.bfloat16), k[:, :, pos].to(torch.bfloat16), v[:, :, pos].to(torch.bfloat16), *_tail(st))
    if case["op"] == "decode":
        return got
    total = w.sum(2)
    total[..., :pos] += st["weight"][..., :pos]
    return (*got, total)


def _tail(st):
    """The block that the new row went into, as it is now: its codes and its scale, of K and of V."""
    pos = st["case"]["pos"]
    return tuple(x for c, s in zip(st["cache"], st["scale"])
                 for x in (c[:, :, pos // BLOCK * BLOCK:pos + 1].view(E4M3), s[..., pos // BLOCK]))


def _plain_evict(st):
    case, w = st["case"], st["weight"]
    rows, keep, first, recent = (case[x] for x in ("rows", "keep", "first", "recent"))
    among = w[..., first:rows - recent].sort(stable=True, dim=-1, descending=True)[1][..., :keep - first - recent] + first
    ends = torch.cat([torch.arange(first, device=w.device), torch.arange(rows - recent, rows, device=w.device)])
    kept = torch.cat([among, ends.expand(*w.shape[:2], -1)], -1).sort(-1)[0]
    blocks = (keep - 1) // BLOCK + 1
    at = torch.cat([kept, kept[..., -1:].expand(*kept.shape[:2], blocks * BLOCK - keep)], -1)  # (the last one again: its scale is there)
    moved = []
    for codes, scales in zip(st["cache"], st["scale"]):
        src = scales.gather(2, at // BLOCK).unflatten(2, (blocks, BLOCK))
        dst = src.amax(-1)
        x = codes.gather(2, kept[..., None].expand(*kept.shape, D)).view(E4M3).float()
        x = x * (src / dst[..., None]).flatten(2)[..., :keep, None]
        moved += [x.to(E4M3), dst]
    return kept.int(), w.gather(2, kept), moved[0], moved[2], moved[1], moved[3]


def run(st):
    if not own:
        return _plain(st)
    import gqa_attention_long_gb300 as ea
    case, Smax = st["case"], st["case"]["Smax"]
    if case["op"] == "write":
        a, b = case["row0"] // BLOCK * BLOCK, case["row0"] + case["rows"]
        ea.expert_attn_write_fp8(None, case["row0"], case["rows"], Smax, _arr=st["args"])
        ea.expert_attn_read_fp8(None, a, b - a, Smax, _arr=st["back"])
        return st["k_back"], st["v_back"]
    if case["op"] == "evict":
        ea.expert_attn_evict_fp8(None, case["rows"], case["keep"], case["first"], case["recent"], Smax, st["ws"], _arr=st["args"])
        return st["got"]
    ea.text_decode_attention_fp8(None, case["pos"], Smax, case["delta"], st["ws"], _arr=st["args"])
    return st["got"]


def work(case):
    """A row of one head is 128 bytes in K and in V, a block's scale 4 more in each."""
    n = case["layers"]
    if case["op"] in ("decode", "weigh"):
        # q, k, v and the gains in; out and the new row's values out; the new row's codes out; the rows before it in
        small = 2 * D * (HQ + 2 * HKV) + 4 * D + 2 * D * (HQ + 2 * HKV) + HKV * 2 * D
        sums = HKV * 4 * (2 * case["pos"] + 1) if case["op"] == "weigh" else 0
        held = HKV * 2 * (case["pos"] * D + 4 * (case["pos"] // BLOCK + 1))
        return {"bytes": n * (small + held + sums), "flops": n * 4 * HQ * D * (case["pos"] + 1)}
    if case["op"] == "write":
        size, back = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]], case["row0"] % BLOCK + case["rows"]
        return {"bytes": n * 2 * HKV * D * (case["rows"] * (size + 1) + back * (size + 1)), "flops": n * 4 * HKV * D * case["rows"]}
    rows, keep = case["rows"], case["keep"]
    return {"bytes": n * HKV * (4 * rows + keep * (4 * D + 8) + 16 * (keep // BLOCK + 1)), "flops": n * HKV * (rows + 2 * D * keep)}


# ---------------------------------------------------------------------------- 64-bit definition
def _grid():
    """The e4m3 magnitudes in order."""
    i = torch.arange(127, device="cuda")
    e, m = i // 8, (i % 8).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))


def _nearest(x):
    """The nearest e4m3 number of each element of an fp64 tensor, found by distance; of two as near, the even code; 448 at most."""
    grid = _grid()
    a = x.abs().clamp(max=448.0).contiguous()
    i = torch.bucketize(a, grid, right=True).clamp(1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (hi - a < a - lo) | ((hi - a == a - lo) & (i % 2 == 0))
    return torch.where(up, hi, lo) * torch.where(x < 0, -1.0, 1.0)


def _numbers(codes):
    """What e4m3 codes stand for, in fp64."""
    c = codes.long()
    return _grid()[(c % 128).clamp(max=126)] * (1 - 2 * (c // 128))


def _exact_block(old, s, x):
    """A block's numbers after x (fp64, [rows, 128]) is appended to `old` under scale s, and the scale that they are under."""
    amax = float(x.abs().max())
    while amax > 448 * s:
        s, old = s * 2, old / 2
    return torch.cat([_nearest(old), _nearest(x / s)]), s


def _exact_rows(codes, scales, x, row0):
    """One head's touched blocks, from the first one's start, as numbers and scales; codes [Smax, 128], x [rows, 128] in fp64."""
    out, at, r = [], 0, row0
    while at < x.shape[0]:
        b = r // BLOCK
        m = min((b + 1) * BLOCK - r, x.shape[0] - at)
        begun = r % BLOCK > 0
        out.append(_exact_block(_numbers(codes[b * BLOCK:r]), float(scales[b]) if begun else 2.0 ** -100, x[at:at + m]))
        at, r = at + m, r + m
    return out


def exact(case, seed):
    st = prepare(case, seed)
    n, (kc, vc), (ks, vs) = case["layers"], st["cache"], st["scale"]
    if case["op"] == "write":
        if n * (case["rows"] // BLOCK + 2) > 1200:
            return None
        return tuple(torch.stack([torch.stack([
            torch.cat([b * t for b, t in _exact_rows(c[l, h], s[l, h], x[l, h].double(), case["row0"])]) for h in range(HKV)])
                                  for l in range(n)]) for c, s, x in ((kc, ks, st["k"]), (vc, vs, st["v"])))
    if case["op"] == "evict":
        return _exact_evict(st)
    pos, p = case["pos"], case["pos"] + case["delta"]
    b0 = pos // BLOCK * BLOCK
    i = torch.arange(D, device="cuda")
    angle = p * torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), -(2.0 * (i % 64).double()) / D)
    sign = torch.where(i < 64, -1.0, 1.0).double()

    def rot(x, gamma):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * gamma.double()
        return x * torch.cos(angle) + sign * x.roll(64, -1) * torch.sin(angle)

    outs = []
    for l in range(n):
        q, k, v = rot(st["q"][l], st["q_gamma"][l]), rot(st["k"][l], st["k_gamma"][l]).float().double(), st["v"][l].double()
        heads = []
        for h in range(HKV):
            full, tail = [], []
            for c, s, x in ((kc, ks, k), (vc, vs, v)):
                before = _numbers(c[l, h, :b0]) * s[l, h, :b0 // BLOCK].double().repeat_interleave(BLOCK)[:, None]
                (block, scale), = _exact_rows(c[l, h], s[l, h], x[h:h + 1], pos)
                full.append(torch.cat([before, block * scale]))
                tail += [block, torch.tensor(scale, dtype=torch.float64, device="cuda")]
            w = torch.softmax(torch.einsum("rd,sd->rs", q[h * 8:h * 8 + 8], full[0]) / D ** 0.5, -1)
            heads.append((w @ full[1], full[0][pos], full[1][pos], *tail, w.sum(0)))
        out, *rest, w = (torch.stack(t) for t in zip(*heads))
        if case["op"] == "weigh":
            w[:, :pos] += st["weight"][l, :, :pos].double()
        outs.append((out.flatten(0, 1), *rest, w))
    got = tuple(torch.stack(x) for x in zip(*outs))
    return got if case["op"] == "weigh" else got[:-1]


def _exact_evict(st):
    case, w = st["case"], st["weight"]
    rows, keep, first, recent = (case[x] for x in ("rows", "keep", "first", "recent"))
    if case["layers"] * keep > 300000:
        return None
    got = []
    for l in range(case["layers"]):
        for h in range(HKV):
            # a row's rank among the eligible: those above it, and the equal ones before it
            a = w[l, h, first:rows - recent].double()
            order = torch.argsort(-a, stable=True)
            chosen = torch.zeros(rows, dtype=torch.bool, device="cuda")
            chosen[first + order[:keep - first - recent]] = True
            chosen[:first] = True
            chosen[rows - recent:] = True
            at = torch.nonzero(chosen)[:, 0]
            one = [at.int(), w[l, h, at].double()]
            for j in range(2):
                src = st["scale"][j][l, h].double()[at // BLOCK]
                dst = torch.stack([t.max() for t in src.split(BLOCK)])
                one += [_nearest(_numbers(st["cache"][j][l, h, at]) * (src / dst.repeat_interleave(BLOCK)[:keep])[:, None]), dst]
            got.append([one[0], one[1], one[2], one[4], one[3], one[5]])
    return tuple(torch.stack(t).unflatten(0, (case["layers"], HKV)) for t in zip(*got))
