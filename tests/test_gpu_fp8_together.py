"""The 8-bit cache's calls as a program makes them: a prompt quantised (expert_attn_quantize_cache) or written, tokens generated
with their weights summed, rows evicted, more tokens generated over what is left, and the expert's attention (e4m3) over it;
against the same steps in fp64 on the host."""
import numpy as np
import pytest
import torch

import gqa_attention_long_gb300 as ea
import oracle
from tests._fp8_util import (DEV, F32, HostCache, decode_buffers, decode_inputs, decode_oracle, evict_oracle, f64, same_cache)
from tests._gpu_util import check_status
from tests._mxfp4_util import step_inputs
from tests.test_gpu_fp8_decode import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("producer", ["quantize", "write"])
def test_prompt_tokens_eviction_tokens_expert(producer):
    Smax, prompt, keep = 1024, 700, 500
    rng = np.random.default_rng(1)
    kv = [torch.from_numpy(rng.standard_normal((8, Smax, 128)).astype(F32)).to(torch.bfloat16) for _ in range(2)]
    h, cache = HostCache(Smax), HostCache(Smax).device()
    if producer == "quantize":
        h.quantised(*(f64(x) for x in kv), prompt)
        for x, c, s in zip(kv, (cache.k_cache, cache.v_cache), (cache.k_scale, cache.v_scale)):
            ea.expert_attn_quantize_cache(x.to(DEV), prompt, Smax, c, s)
    else:
        for i, x in enumerate(kv):
            h.append(i, x[:, :prompt].float().numpy(), 0)
        ea.expert_attn_write_fp8([ea.Fp8Rows(*(x[:, :prompt].to(DEV) for x in kv), cache)], 0, prompt, Smax)
    same_cache(cache, h)
    ws, we = ea.alloc_decode_fp8_workspace(1, Smax, weights=True), ea.alloc_evict_fp8_workspace(1, Smax)
    weight = torch.zeros(8, Smax, device=DEV)
    pos, token = prompt, prompt  # the row that comes next, and the token's place in the text
    for part in range(2):
        for i in range(5):
            x = decode_inputs(50 * part + i)
            b = decode_buffers(x, cache, weight, weight)
            ea.text_decode_attention_fp8([b], pos, Smax, token - pos, ws)
            r = decode_oracle(x, h, pos, token - pos)
            same_cache(cache, h, f"token {token}")
            close(b.out, r["out"], f"token {token}")
            pos, token = pos + 1, token + 1
        if part == 0:
            w, kept = weight.cpu().numpy(), torch.empty(8, keep, dtype=torch.int32, device=DEV)
            ea.expert_attn_evict_fp8([ea.EvictFp8Buffers(cache, weight, kept)], pos, keep, 4, 64, Smax, we)
            which, to, wk = evict_oracle(h, w, pos, keep, 4, 64)  # (from the library's own sums: which rows, then, is exact)
            assert np.array_equal(kept.cpu().numpy(), which)
            for i in range(2):
                h.codes[i][:, :keep], h.scales[i][:, :4] = to.codes[i][:, :keep], to.scales[i][:, :4]
            same_cache(cache, h)
            assert np.array_equal(weight.cpu().numpy()[:, :keep], wk)
            pos = keep
    check_status(ws)
    check_status(we)
    # the expert's 64 tokens over what the text model left
    x = {n: t.to(DEV) for n, t in step_inputs(9, 16, 64).items()}
    L = ea.LayerBuffers(**x, k_cache=cache.k_cache, v_cache=cache.v_cache, k_scale=cache.k_scale, v_scale=cache.v_scale,
                        out=torch.full((16, 64, 128), float("nan"), dtype=torch.bfloat16, device=DEV))
    wx = ea.alloc_workspace(1, Smax, ea.EA_KV_FP8_E4M3)
    ea.expert_attn_layers([L], pos, Smax, token - pos, ea.EA_KV_FP8_E4M3, wx)
    check_status(wx)
    want = oracle.expert_attention_layer_fp8(*(f64(x[n]) for n in ("q_raw", "k_raw", "v_raw", "q_gamma", "k_gamma")), h.codes[0], h.scales[0],
                                             h.codes[1], h.scales[1], pos, Smax, token - pos)["out"]
    off = np.abs(f64(L.out) - want)
    assert off.max() <= 2e-2  # the bar of that call's own tests


def test_eight_bits_stay_near_sixteen():
    """One step over a written 8-bit cache against the bf16 step over the rows it was written from. A code is off by at most 2^-4 of
    its value: keys move a score by at most 2^-4 sum |q k| / sqrt(128) and on average by far less; the outputs' distance stays
    under 2^-4 + what the weights change (measured against the fp64 step over the codes in the other tests)."""
    Smax, pos = 1024, 900
    rng = np.random.default_rng(3)
    kv = [torch.from_numpy(rng.standard_normal((8, Smax, 128)).astype(F32)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    x = decode_inputs(4)
    cache = ea.alloc_fp8_cache(Smax)
    ea.expert_attn_write_fp8([ea.Fp8Rows(kv[0][:, :pos], kv[1][:, :pos], cache)], 0, pos, Smax)
    b, ws = decode_buffers(x, cache), ea.alloc_decode_fp8_workspace(1, Smax)
    ea.text_decode_attention_fp8([b], pos, Smax, 0, ws)
    d = {n: t.to(DEV) for n, t in x.items()}
    full = ea.DecodeBuffers(**d, k_cache=kv[0].clone(), v_cache=kv[1].clone(), out=torch.empty(64, 128, dtype=torch.bfloat16, device=DEV))
    wf = ea.alloc_decode_workspace(1)
    ea.text_decode_attention([full], pos, Smax, 0, wf)
    check_status(ws)
    check_status(wf)
    assert torch.linalg.norm(b.out.double() - full.out.double()) <= 0.1 * torch.linalg.norm(full.out.double())
