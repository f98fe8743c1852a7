"""Shared helpers of the 4-bit cache tests: caches made by the oracle's quantiser, the oracle's two
attentions over them, and device buffers for the library's calls."""
from __future__ import annotations

import numpy as np
import torch

import gqa_attention_long_gb300 as ea
import oracle

DEV = "cuda"


def quantise(x: np.ndarray):
    """fp32 rows [..., 128] -> (codes [..., 128] in 0..15, exponents [..., 4]); the oracle's rule,
    vectorised (block_exponent is a scalar function)."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], 4, 32)
    amax = np.abs(b).max(-1)
    _, ex = np.frexp(amax)
    e = np.where(amax > 0, np.clip(ex.astype(np.int64) - 3, -127, 127), 0)
    codes = oracle.encode_e2m1_rne_sat((b.astype(np.float64) / np.exp2(e.astype(np.float64))[..., None]).astype(np.float32))
    return codes.reshape(x.shape), e.astype(np.int16)


def packed(codes: np.ndarray, exps: np.ndarray):
    """Codes and exponents as the cache's bytes (CPU tensors)."""
    return (torch.from_numpy((codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)),
            torch.from_numpy((exps.astype(np.int64) + 127).astype(np.uint8)))


def unpacked(codes: torch.Tensor, scales: torch.Tensor):
    """The cache's bytes as codes [..., 128] and exponents [..., 4]."""
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 128), scales.cpu().numpy().astype(np.int16) - 127


class HostCache:
    """Codes and exponents of one layer's K and V caches; rows from `valid` on hold `fill` bytes."""

    def __init__(self, k: np.ndarray, v: np.ndarray, valid: int, fill: int = 0xA7):
        self.k, self.v, self.Smax = quantise(k), quantise(v), k.shape[1]
        self.bytes = [*packed(*self.k), *packed(*self.v)]
        for b in self.bytes:
            b[:, valid:] = fill

    def device(self) -> "ea.Mxfp4Cache":
        return ea.Mxfp4Cache(*(b.to(DEV) for b in self.bytes))


def random_cache(seed: int, Smax: int, valid: int, fill: int = 0xA7, k_gain=1.0, v_gain=1.0) -> HostCache:
    rng = np.random.default_rng(seed)
    return HostCache(rng.standard_normal((8, Smax, 128)) * k_gain, rng.standard_normal((8, Smax, 128)) * v_gain, valid, fill)


def bf16_rows(seed: int, *shape) -> torch.Tensor:
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def decode_oracle(x: dict, c: HostCache, pos: int, delta: int) -> dict:
    q, k, v = oracle.decode_prologue(*(f64(x[n]) for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")), pos, delta)
    kc, ke = quantise(k)
    vc, ve = quantise(v)
    keys, vals = (np.concatenate([oracle.dequantize_rows(a[0][:, :pos], a[1][:, :pos]), oracle.dequantize_rows(*b)[:, None]], 1)
                  for a, b in ((c.k, (kc, ke)), (c.v, (vc, ve))))
    return {"out": oracle.decode_attend(q, keys, vals, pos), "k": (kc, ke), "v": (vc, ve)}


def expert_oracle(x: dict, c: HostCache, S: int, delta: int) -> dict:
    q, k, v = oracle.prologue(*(f64(x[n]) for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")), S, delta)
    new = quantise(k), quantise(v)
    old = [oracle.dequantize_rows(a[0][:, :S], a[1][:, :S]) for a in (c.k, c.v)]
    out = oracle.attention_concat(q, old[0], old[1], S, *(oracle.dequantize_rows(*n) for n in new))
    return {"out": out, "k": new[0], "v": new[1]}


def step_inputs(seed: int, hq: int, tok: int) -> dict:
    t = () if tok == 1 else (tok,)
    return {"q_raw": bf16_rows(seed, hq, *t, 128), "k_raw": bf16_rows(seed + 1, 8, *t, 128),
            "v_raw": bf16_rows(seed + 2, 8, *t, 128),
            "q_gamma": (1 + 0.1 * bf16_rows(seed + 3, 128).float()).to(torch.bfloat16),
            "k_gamma": (1 + 0.1 * bf16_rows(seed + 4, 128).float()).to(torch.bfloat16)}


def device_buffers(x: dict, cache: "ea.Mxfp4Cache", values: bool = True):
    d = {n: t.to(DEV) for n, t in x.items()}
    cls = ea.DecodeMxfp4Buffers if x["q_raw"].shape[0] == 64 else ea.LayerMxfp4Buffers
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    return cls(**d, cache=cache, out=nan(d["q_raw"]), k_new=nan(d["k_raw"]) if values else None,
               v_new=nan(d["v_raw"]) if values else None)
