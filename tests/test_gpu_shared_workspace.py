"""One workspace for calls of different layer counts (and cache types), in turn: each gives what it gives with a workspace of
its own."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300.inputs import decode_inputs_on_device
from tests._gpu_util import check_status
from tests._mxfp4_util import decode_oracle, device_buffers, expert_oracle, random_cache, step_inputs
from tests.test_gpu_mxfp4_attention import close

pytestmark = pytest.mark.gpu


def in_turn(runs, ws, alloc, same):
    """runs: (call(ws), outputs, layers); same(output, the one alone)."""
    alone = []
    for call, outs, n in runs:
        own = alloc(n)
        call(own)
        check_status(own)
        alone.append([o.clone() for o in outs])
    for turn in range(3):
        for i, (call, outs, _) in enumerate(runs):
            for o in outs:
                o.fill_(float("nan"))
            call(ws)
            check_status(ws)
            for l, (o, want) in enumerate(zip(outs, alone[i])):
                assert same(o, want), f"turn {turn}, call {i}, layer {l}"


def test_decode():
    runs = []
    for n, pos, Smax in ((2, 3000, 4096), (64, 700, 768), (1, 2000, 2048), (40, 300, 512)):
        Ls = []
        for l in range(n):
            x = decode_inputs_on_device(900 + 70 * n + l, pos, Smax, "cuda")
            Ls.append(ea.DecodeBuffers(x.q_raw, x.k_raw, x.v_raw, x.q_gamma, x.k_gamma, x.k_cache, x.v_cache,
                                       torch.empty(64, 128, dtype=torch.bfloat16, device="cuda")))
        runs.append((lambda ws, Ls=Ls, pos=pos, Smax=Smax: ea.text_decode_attention(Ls, pos, Smax, 0, ws), [L.out for L in Ls], n))
    in_turn(runs, ea.alloc_decode_workspace(64), ea.alloc_decode_workspace, torch.equal)


def one_rounding(o, want):
    """Of a unit's two parts the one that ends second merges them, with the other's in f16 (2^-12 of a row's largest): which one
    that is may move an output to the next bf16 number, no further."""
    off, w = (o.float() - want.float()).abs(), want.float().abs()
    return bool((off <= 2.0 ** -7 * w + 2.0 ** -11 * w.amax(-1, keepdim=True)).all())


def test_expert_over_both_cache_types():
    from gqa_attention_long_gb300.inputs import layer_inputs_on_device
    from tests.test_gpu_fp8 import quantize_on_gpu
    runs = []
    for n, S, Smax, dtype in ((3, 1000, 1152, ea.EA_KV_FP8_E4M3), (40, 700, 768, ea.EA_KV_BF16), (1, 300, 512, ea.EA_KV_FP8_E4M3),
                              (64, 700, 768, ea.EA_KV_BF16), (18, 300, 512, ea.EA_KV_FP8_E4M3)):
        Ls = []
        for l in range(n):
            x = layer_inputs_on_device(500 + 70 * n + l, S, Smax, "cuda")
            kv = [x.k_cache, x.v_cache, None, None]
            if dtype == ea.EA_KV_FP8_E4M3:
                (kc, ks), (vc, vs) = (quantize_on_gpu(t, S, Smax) for t in kv[:2])
                kv = [kc, vc, ks, vs]
            Ls.append(ea.LayerBuffers(x.q_raw, x.k_raw, x.v_raw, x.q_gamma, x.k_gamma, kv[0], kv[1],
                                      torch.empty(16, 64, 128, dtype=torch.bfloat16, device="cuda"), kv[2], kv[3]))
        runs.append((lambda ws, Ls=Ls, S=S, Smax=Smax, d=dtype: ea.expert_attn_layers(Ls, S, Smax, 0, d, ws), [L.out for L in Ls], n))
    alloc = lambda n: ea.alloc_workspace(n, 1152, ea.EA_KV_FP8_E4M3)  # noqa: E731
    in_turn(runs, alloc(64), alloc, one_rounding)


@pytest.mark.parametrize("form", ["decode", "expert"])
def test_small_calls_between_large_ones_over_a_4_bit_cache(form):
    """What a large call leaves in a workspace does not reach the small one's outputs."""
    call, alloc, ref, hq, tok = {
        "decode": (ea.text_decode_attention_mxfp4, ea.alloc_decode_mxfp4_workspace, decode_oracle, 64, 1),
        "expert": (ea.expert_attn_layers_mxfp4, ea.alloc_mxfp4_workspace, expert_oracle, 16, 64)}[form]
    ws = alloc(64)
    h = random_cache(3, 512, 400)
    many = [device_buffers(step_inputs(l, hq, tok), h.device()) for l in range(64)]
    xs, hs = [step_inputs(100 + l, hq, tok) for l in range(3)], [random_cache(8 + l, 1088, 1000) for l in range(3)]
    few = [device_buffers(a, b.device()) for a, b in zip(xs, hs)]
    want = [ref(a, b, 1000, 0)["out"] for a, b in zip(xs, hs)]
    for turn in range(3):
        call(many, 400, 512, 0, ws)
        for b in few:
            b.out.fill_(float("nan"))
        call(few, 1000, 1088, 0, ws)
        for l in range(3):
            close(few[l].out, want[l], f"turn {turn}, layer {l}")
    check_status(ws)
