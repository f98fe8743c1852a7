"""Shared helpers of the 8-bit cache's tests: the rule by which rows are appended, the decode step and the eviction, written
out plainly on the host from the oracle's e4m3 table, and device buffers for the library's calls."""
from __future__ import annotations

import numpy as np
import torch

import gqa_attention_long_gb300 as ea
import oracle
from tests._mxfp4_util import bf16_rows, f64, step_inputs  # noqa: F401

DEV = "cuda"
F32 = np.float32


def encode(x: np.ndarray) -> np.ndarray:
    """fp32 -> e4m3 codes: nearest, even on ties, saturating (infinities too); NaN -> 0x7F."""
    nan = np.isnan(x)
    c = oracle.encode_e4m3_rne_sat(np.clip(np.where(nan, 0, x), -1e30, 1e30).astype(F32))
    return np.where(nan, np.uint8(0x7F), c)


def grown(s: F32, amax: F32) -> F32:
    """The scale that a block with scale s has once it holds a value of magnitude amax."""
    with np.errstate(over="ignore"):
        while amax > F32(448) * s and np.frexp(s)[1] - 1 < 118:
            s = F32(s * F32(2))
    return s


class HostCache:
    """One layer's 8-bit caches on the host: [K, V] codes and scales; codes behind the held rows are NaN, or `fill`."""

    def __init__(self, Smax: int, fill: int = 0x7F):
        self.Smax = Smax
        self.codes = [np.full((8, Smax, 128), fill, np.uint8) for _ in range(2)]
        self.scales = [np.full((8, Smax // 128 + 1), np.nan, F32) for _ in range(2)]

    def quantised(self, k, v, n_rows):
        """Filled as expert_attn_quantize_cache fills it (a scale amax / 448)."""
        for i, x in enumerate((k, v)):
            c, s = oracle.quantize_cache_blocks(x, n_rows, max(self.Smax, n_rows + 64 + 127 & -128))
            self.codes[i][:, :n_rows], nb = c[:, :n_rows], -(-n_rows // 128)
            self.scales[i][:, :nb] = s[:, :nb]
        return self

    def append(self, i: int, x: np.ndarray, row0: int) -> None:
        """Rows x (fp32 [8, n, 128]) into cache i (0: K, 1: V), which holds row0 rows."""
        x = np.asarray(x, F32)
        for g in range(8):
            r = row0
            while r < row0 + x.shape[1]:
                b = r // 128
                m = min((b + 1) * 128, row0 + x.shape[1]) - r
                rows = x[g, r - row0:r - row0 + m]
                with np.errstate(invalid="ignore"):
                    amax = F32(np.max(np.abs(np.where(np.isnan(rows), 0, rows))))
                s = self.scales[i][g, b] if r % 128 else F32(2.0 ** -100)
                s1 = grown(s, amax)
                if s1 != s:
                    old = self.codes[i][g, b * 128:r]
                    nan = (old & 0x7F) == 0x7F
                    self.codes[i][g, b * 128:r] = np.where(nan, old, encode((oracle.decode_e4m3(np.where(nan, 0, old)) * float(s) / float(s1)).astype(F32)))
                with np.errstate(over="ignore", invalid="ignore"):
                    self.codes[i][g, r:r + m] = encode(rows / s1)
                self.scales[i][g, b] = s1
                r += m

    def values(self, i: int, n: int) -> np.ndarray:
        """Rows [0, n) as fp64."""
        return oracle.decode_e4m3(self.codes[i][:, :n]) * self.scales[i].astype(np.float64)[:, np.arange(n) // 128][:, :, None]

    def device(self) -> "ea.Fp8Cache":
        return ea.Fp8Cache(*(torch.from_numpy(c.copy()).to(DEV) for c in self.codes), *(torch.from_numpy(s.copy()).to(DEV) for s in self.scales))

    def copy(self) -> "HostCache":
        h = HostCache(1)
        h.Smax, h.codes, h.scales = self.Smax, [c.copy() for c in self.codes], [s.copy() for s in self.scales]
        return h


def same_cache(dev: "ea.Fp8Cache", host: HostCache, what: str = "", signs: bool = True) -> None:
    """Codes bit for bit (any NaN for a NaN), scales too; where the host's scale is NaN nothing was to be written. signs=False: a zero
    of either sign is a zero, as it comes out of a rotation (0 cos - 0 sin has the sign that the formula's order gives it)."""
    for c, s, hc, hs in zip((dev.k_cache, dev.v_cache), (dev.k_scale, dev.v_scale), host.codes, host.scales):
        c, s = c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
        off = (c != hc) & ~(((c & 0x7F) == 0x7F) & ((hc & 0x7F) == 0x7F))
        if not signs:
            off &= ((c | hc) & 0x7F) != 0
        assert not off.any(), f"{what}: {off.sum()} codes, first at {np.argwhere(off)[0]}"
        assert np.array_equal(s, hs, equal_nan=True), f"{what}: scales"


def random_cache(seed: int, Smax: int, valid: int, k_gain=1.0, v_gain=1.0, fill: int = 0x7F) -> HostCache:
    rng = np.random.default_rng(seed)
    x = [torch.from_numpy((rng.standard_normal((8, valid, 128)) * gain).astype(F32)).to(torch.bfloat16).double().numpy()
         for gain in (k_gain, v_gain)]
    return HostCache(Smax, fill).quantised(*x, valid)


def decode_oracle(x: dict, c: HostCache, pos: int, delta: int) -> dict:
    """The decode step in fp64 over the appended caches (c is changed): out, weights [8, pos + 1], the new rows' values."""
    q, k, v = oracle.decode_prologue(*(f64(x[n]) for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")), pos, delta)
    c.append(0, k.astype(F32)[:, None], pos)
    c.append(1, v.astype(F32)[:, None], pos)
    keys, vals = c.values(0, pos + 1), c.values(1, pos + 1)
    out, weights = np.empty((64, 128)), np.empty((8, pos + 1))
    for g in range(8):
        s = q[8 * g:8 * g + 8] @ keys[g].T / np.sqrt(128)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[8 * g:8 * g + 8], weights[g] = w @ vals[g], w.sum(0)
    return {"out": out, "weight": weights, "k": keys[:, pos], "v": vals[:, pos]}


def decode_buffers(x: dict, cache: "ea.Fp8Cache", weight_in=None, weight_out=None) -> "ea.DecodeFp8Buffers":
    d = {n: t.to(DEV) for n, t in x.items()}
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    return ea.DecodeFp8Buffers(**d, cache=cache, out=nan(d["q_raw"]), k_new=nan(d["k_raw"]), v_new=nan(d["v_raw"]),
                               weight_in=weight_in, weight_out=weight_out)


def decode_inputs(seed: int) -> dict:
    return step_inputs(seed, 64, 1)


def evict_oracle(c: HostCache, weight: np.ndarray, n_rows: int, n_keep: int, n_first: int, n_recent: int):
    """Kept rows [8, n_keep], and a cache that holds them and nothing else, with their weights."""
    kept = np.empty((8, n_keep), np.int64)
    for g in range(8):
        mid = np.arange(n_first, n_rows - n_recent)
        w = weight[g, mid].astype(np.float64)
        key = np.where(np.isnan(w), np.inf, w)
        order = np.lexsort((mid, -key, ~np.isnan(w)))  # NaN first, then by weight, then by row
        kept[g] = np.sort(np.concatenate([np.arange(n_first), mid[order[:n_keep - n_first - n_recent]], np.arange(n_rows - n_recent, n_rows)]))
    to = HostCache(c.Smax)
    for i in range(2):
        for g in range(8):
            s = c.scales[i][g, kept[g] // 128]
            for b in range(-(-n_keep // 128)):
                a = slice(128 * b, min(128 * b + 128, n_keep))
                top = s[a].max()
                f = np.where(s[a] == top, F32(1), s[a] / top).astype(F32)
                old = c.codes[i][g, kept[g, a]]
                nan = (old & 0x7F) == 0x7F
                x = oracle.decode_e4m3(np.where(nan, 0, old)).astype(F32) * f[:, None]
                to.codes[i][g, a] = np.where(nan, old, encode(x))
                to.scales[i][g, b] = top
    return kept, to, np.take_along_axis(weight, kept, 1)
