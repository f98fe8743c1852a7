"""The cases on which the operators over a 4-bit KV cache are measured.

A cache of one layer holds K and V rows [8 heads][Smax][128] as MXFP4: E2M1 codes, two to a byte
(the lower channel in the low nibble), and one power-of-two scale byte e + 127 for each 32
channels of a row. Four operators work on it:

  write   rows [row0, row0 + n) of K and V quantised as they are written
  read    the same rows back as numbers
  decode  one token's attention of 64 query heads over rows [0, pos], row pos written first
  expert  64 tokens' attention of 16 query heads over rows [0, S) and their own 64 rows,
          which are written to rows [Smax - 64, Smax) first

``run`` computes them in plain torch, or, where ``own`` is true, by this repository's calls.
"""
import math

import torch

own = False

HKV, D, TOK = 8, 128, 64
THETA, EPS = 5.0e6, 1e-6
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
        # the smallest expert call: a short prompt, one layer
        {"name": "expert 1 layer S 256", "op": "expert", "layers": 1, "S": 256, "Smax": 512, "delta": 0},
        # one layer of the expert at the driving prompt's length
        {"name": "expert 1 layer S 4700", "op": "expert", "layers": 1, "S": 4700, "Smax": 8192, "delta": 0},
        # the attention of one Euler step: 64 layers
        {"name": "expert 64 layers S 4700", "op": "expert", "layers": 64, "S": 4700, "Smax": 8192, "delta": 11},
        # a long video prompt, an odd number of rows
        {"name": "expert 2 layers S 65537", "op": "expert", "layers": 2, "S": 65537, "Smax": 65664, "delta": 0},
        # one new token's rows in every layer, cut out of the fused projection's output
        {"name": "write 64 layers 1 row", "op": "write", "layers": 64, "row0": 4700, "rows": 1, "Smax": 8192,
         "dtype": "bf16", "order": "token"},
        # a prompt's rows after its prefill, head by head
        {"name": "write 16 layers 4700 rows", "op": "write", "layers": 16, "row0": 0, "rows": 4700, "Smax": 8192,
         "dtype": "bf16", "order": "head"},
        # an odd handful of rows looked at in 32 bits
        {"name": "read 1 layer 77 rows", "op": "read", "layers": 1, "row0": 130, "rows": 77, "Smax": 512,
         "dtype": "fp32", "order": "head"},
        # a whole prefix brought back to bf16, for a step that takes a 16-bit cache
        {"name": "read 16 layers 4700 rows", "op": "read", "layers": 16, "row0": 1, "rows": 4700, "Smax": 8192,
         "dtype": "bf16", "order": "head"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["decode", "expert", "write", "read"])
    layers = _log(rng, 1, 64)
    if op == "decode":
        pos = _log(rng, 1, min(131071, 524288 // layers)) - 1
        return {"op": op, "layers": layers, "pos": pos, "Smax": max(128, (pos // 64 + 1 + rng.randrange(4)) * 64),
                "delta": rng.randrange(-400, 400)}
    if op == "expert":
        S = _log(rng, 1, min(65600, 300000 // layers)) - 1
        return {"op": op, "layers": layers, "S": S, "Smax": max(128, (-(-S // 64) + 1 + rng.randrange(4)) * 64),
                "delta": rng.randrange(-400, 400)}
    rows = _log(rng, 1, 75200 // layers)
    row0 = rng.randrange(300)
    return {"op": op, "layers": layers, "row0": row0, "rows": rows, "Smax": (-(-(row0 + rows) // 64) + rng.randrange(4)) * 64,
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "order": rng.choice(["head", "token"])}


# ------------------------------------------------------------------------------------- inputs
def _pow2(e):
    """2^e in fp32, |e| <= 127, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _pack(x):
    """Rows [..., 128] as MXFP4: codes [..., 64] and scale bytes [..., 4]."""
    b = x.float().unflatten(-1, (4, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, 0).clamp(-127, 127)
    a = b.abs() * _pow2(-e)
    c = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = (c + 8 * torch.signbit(b)).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _values(codes, scales):
    """MXFP4 rows as fp32 numbers (exact)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return (table[c].unflatten(-1, (4, 32)) * _pow2(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, Smax, bf = case["layers"], case["Smax"], torch.bfloat16
    st = {"case": case}
    # the cache: K with the channel gains that a k norm leaves behind, so that its blocks' scales
    # differ. The rows hold what earlier calls wrote, made two layers at a time.
    st["cache"] = [torch.empty(n, HKV, Smax, w, dtype=torch.uint8, device="cuda") for w in (64, 4, 64, 4)]
    for i in range(0, n, 2):
        m = min(2, n - i)
        for j, gain in ((0, torch.exp(0.5 * rand(D))), (2, 1.0)):
            st["cache"][j][i:i + m], st["cache"][j + 1][i:i + m] = _pack(rand(m, HKV, Smax, D) * gain)
    if case["op"] in ("decode", "expert"):
        hq, t = (64, 1) if case["op"] == "decode" else (16, TOK)
        st["q"], st["k"], st["v"] = (rand(n, h, t, D).to(bf) for h in (hq, HKV, HKV))
        st["q_gamma"], st["k_gamma"] = ((1 + 0.1 * rand(n, D)).to(bf) for _ in range(2))
        st["out"] = torch.empty(n, hq, t, D, dtype=bf, device="cuda")
        st["k_new"], st["v_new"] = (torch.empty(n, HKV, t, D, dtype=bf, device="cuda") for _ in range(2))
    else:
        rows, dt = case["rows"], DTYPES[case["dtype"]]
        if case["order"] == "head":
            kv = [rand(n, HKV, rows, D).to(dt) for _ in range(2)]
        else:  # the k and v columns of a fused projection's output [rows][k | v]
            fused = rand(n, rows, 2, HKV, D).to(dt)
            kv = [fused[:, :, i].transpose(1, 2) for i in range(2)]
        st["k"], st["v"] = kv
        st["k_back"], st["v_back"] = (torch.empty(n, HKV, rows, D, dtype=dt, device="cuda") for _ in range(2))
    if own:
        import gqa_attention_long_gb300 as ea
        caches = [ea.Mxfp4Cache(*(c[i] for c in st["cache"])) for i in range(n)]
        if case["op"] == "decode":
            bufs = [ea.DecodeMxfp4Buffers(st["q"][i], st["k"][i], st["v"][i], st["q_gamma"][i], st["k_gamma"][i], caches[i],
                                          st["out"][i], st["k_new"][i], st["v_new"][i]) for i in range(n)]
            st["args"] = ea.make_decode_mxfp4_args(bufs, Smax)
            st["ws"] = ea.alloc_decode_mxfp4_workspace(n)
        elif case["op"] == "expert":
            bufs = [ea.LayerMxfp4Buffers(st["q"][i], st["k"][i], st["v"][i], st["q_gamma"][i], st["k_gamma"][i], caches[i],
                                         st["out"][i], st["k_new"][i], st["v_new"][i]) for i in range(n)]
            st["args"] = ea.make_mxfp4_args(bufs, Smax)
            st["ws"] = ea.alloc_mxfp4_workspace(n)
        else:
            st["args"] = ea.make_rows_args([ea.Mxfp4Rows(st["k"][i], st["v"][i], caches[i]) for i in range(n)], Smax)
            st["back"] = ea.make_rows_args([ea.Mxfp4Rows(st["k_back"][i], st["v_back"][i], caches[i]) for i in range(n)], Smax)
    return st


# ----------------------------------------------------------------------------------- plain forms
def _norm_rope(x, gamma, p0):
    """RMS norm and rotate_half RoPE of x [n, heads, t, 128], token t at position p0 + t, in 64 bits:
    the angles of far positions and codes next to a border need them."""
    x = x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.double()[:, None, None]
    inv = THETA ** (-torch.arange(D // 2, dtype=torch.float64, device=x.device) / (D // 2))
    a = (p0 + torch.arange(x.shape[2], dtype=torch.float64, device=x.device))[:, None] * inv
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def _attend(q, k, v):
    """softmax(q k^T / sqrt(128)) v in fp32: q [n, 8, rows, 128], k and v [n, 8, keys, 128]."""
    s = q @ k.transpose(-1, -2) / math.sqrt(D)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p @ v / p.sum(-1, keepdim=True)


def _plain(st):
    case, cache, op = st["case"], st["cache"], st["case"]["op"]
    if op == "write":
        a, b = case["row0"], case["row0"] + case["rows"]
        for c, x in zip(cache, _pack(st["k"]) + _pack(st["v"])):
            c[:, :, a:b] = x
    if op in ("write", "read"):
        a, b = case["row0"], case["row0"] + case["rows"]
        part = [c[:, :, a:b] for c in cache]
        return _values(*part[:2]).to(st["k"].dtype), _values(*part[2:]).to(st["k"].dtype)
    first = case["pos"] if op == "decode" else case["S"]
    q = _norm_rope(st["q"], st["q_gamma"], first + case["delta"]).float()
    k = _norm_rope(st["k"], st["k_gamma"], first + case["delta"]).float()
    new = _pack(k) + _pack(st["v"])
    a = first if op == "decode" else case["Smax"] - TOK
    for c, x in zip(cache, new):
        c[:, :, a:a + x.shape[2]] = x
    keys, vals = (torch.cat([_values(*(c[:, :, :first] for c in cache[j:j + 2])), _values(*new[j:j + 2])], 2) for j in (0, 2))
    out = _attend(q.reshape(q.shape[0], HKV, -1, D), keys, vals).to(torch.bfloat16)
    return out.reshape(q.shape), _values(*new[:2]).to(torch.bfloat16), _values(*new[2:]).to(torch.bfloat16)


def run(st):
    if not own:
        return _plain(st)
    import gqa_attention_long_gb300 as ea
    case = st["case"]
    if case["op"] == "decode":
        ea.text_decode_attention_mxfp4(None, case["pos"], case["Smax"], case["delta"], st["ws"], _arr=st["args"])
        return st["out"], st["k_new"], st["v_new"]
    if case["op"] == "expert":
        ea.expert_attn_layers_mxfp4(None, case["S"], case["Smax"], case["delta"], st["ws"], _arr=st["args"])
        return st["out"], st["k_new"], st["v_new"]
    if case["op"] == "write":
        ea.expert_attn_write_mxfp4(None, case["row0"], case["rows"], case["Smax"], _arr=st["args"])
    ea.expert_attn_read_mxfp4(None, case["row0"], case["rows"], case["Smax"], _arr=st["back"])
    return st["k_back"], st["v_back"]


def work(case):
    """A row of one head is 68 bytes in the cache (64 of codes, 4 of scales), for K and for V."""
    n, row = case["layers"], 2 * HKV * 68
    if case["op"] in ("decode", "expert"):
        hq, t, keys = (64, 1, case["pos"]) if case["op"] == "decode" else (16, TOK, case["S"])
        # q, k, v in; out and the new rows' values out; the new rows' codes out; the rows before them in
        small = 2 * D * t * (hq + 2 * HKV) + 4 * D + 2 * D * t * (hq + 2 * HKV) + t * row
        return {"bytes": n * (small + keys * row), "flops": n * 4 * hq * t * D * (keys + t)}
    values = 2 * HKV * D * {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    once = n * case["rows"] * (values + row)
    return {"bytes": once * (2 if case["op"] == "write" else 1), "flops": n * case["rows"] * 2 * HKV * D}


# ---------------------------------------------------------------------------- 64-bit definition
def _mx(x):
    """The nearest MXFP4 number of each element of fp64 rows (which hold fp32 values), found by
    distance; of two as near, the one with the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    b = x.reshape(*x.shape[:-1], D // 32, 32)
    top = b.abs().amax(-1, keepdim=True)
    power = torch.tensor([2.0 ** j for j in range(-127, 129)], dtype=torch.float64, device=x.device)
    e = torch.bucketize(torch.where(top > 0, top, 4.0).contiguous(), power, right=True) - 3  # power[e] <= top / 4 < power[e + 1]
    two_e = power[e.clamp(min=0)]
    r = (b.abs() / two_e).contiguous()
    i = torch.bucketize(r, grid, right=True).clamp(1, 7)
    lo, hi = grid[i - 1], grid[i]
    up = (hi - r < r - lo) | ((hi - r == r - lo) & (i % 2 == 0))
    return (torch.where(up, hi, lo) * two_e * torch.where(b < 0, -1.0, 1.0)).reshape(x.shape)


def _numbers(codes, scales):
    """What the cache's bytes stand for, in fp64."""
    c = torch.empty(*codes.shape[:-1], D, dtype=torch.int64, device=codes.device)
    c[..., 0::2], c[..., 1::2] = codes % 16, codes // 16
    ee, m = (c // 2) % 4, (c % 2).double()
    mag = torch.where(ee == 0, m / 2, (1 + m / 2) * torch.exp2(ee.double() - 1))
    power = torch.tensor([2.0 ** (j - 127) for j in range(255)], dtype=torch.float64, device=codes.device)
    return mag * (1 - 2 * (c // 8)) * power[scales.long()].repeat_interleave(32, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["cache"]
    if case["op"] == "write":
        return _mx(st["k"].double()), _mx(st["v"].double())
    if case["op"] == "read":
        a, b = case["row0"], case["row0"] + case["rows"]
        return _numbers(c[0][:, :, a:b], c[1][:, :, a:b]), _numbers(c[2][:, :, a:b], c[3][:, :, a:b])
    n, hq, t = st["q"].shape[:3]
    first = case["pos"] if case["op"] == "decode" else case["S"]
    i = torch.arange(D, device="cuda")
    rate = torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), -(2.0 * (i % 64).double()) / D)
    angle = torch.arange(first + case["delta"], first + case["delta"] + t, device="cuda").double()[:, None] * rate
    sign = torch.where(i < 64, -1.0, 1.0).double()
    outs = []
    for l in range(n):
        def rot(x, gamma):
            x = x.double()
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * gamma.double()
            return x * torch.cos(angle) + sign * x.roll(64, -1) * torch.sin(angle)
        q, k = rot(st["q"][l], st["q_gamma"][l]), _mx(rot(st["k"][l], st["k_gamma"][l]).float().double())
        v = _mx(st["v"][l].double())
        heads = []
        for h in range(HKV):
            kk = torch.cat([_numbers(c[0][l, h, :first], c[1][l, h, :first]), k[h]])
            vv = torch.cat([_numbers(c[2][l, h, :first], c[3][l, h, :first]), v[h]])
            s = torch.einsum("rd,sd->rs", q[h * hq // HKV:(h + 1) * hq // HKV].reshape(-1, D), kk) / D ** 0.5
            heads.append(torch.softmax(s, -1) @ vv)
        outs.append((torch.cat(heads).reshape(hq, t, D), k, v))
    return tuple(torch.stack(x) for x in zip(*outs))
