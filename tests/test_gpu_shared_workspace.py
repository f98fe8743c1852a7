"""One workspace for calls of different layer counts (and cache types), in turn: each gives, bit for bit, what it gives with
a workspace of its own."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from gqa_attention_long_gb300.inputs import decode_inputs_on_device
from tests._gpu_util import check_status

pytestmark = pytest.mark.gpu


def in_turn(runs, ws, alloc):
    """runs: (call(ws), outputs, layers)."""
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
                assert torch.equal(o, want), f"turn {turn}, call {i}, layer {l}"


def test_decode():
    runs = []
    for n, pos, Smax in ((2, 3000, 4096), (64, 700, 768), (1, 2000, 2048), (40, 300, 512)):
        Ls = []
        for l in range(n):
            x = decode_inputs_on_device(900 + 70 * n + l, pos, Smax, "cuda")
            Ls.append(ea.DecodeBuffers(x.q_raw, x.k_raw, x.v_raw, x.q_gamma, x.k_gamma, x.k_cache, x.v_cache,
                                       torch.empty(64, 128, dtype=torch.bfloat16, device="cuda")))
        runs.append((lambda ws, Ls=Ls, pos=pos, Smax=Smax: ea.text_decode_attention(Ls, pos, Smax, 0, ws), [L.out for L in Ls], n))
    in_turn(runs, ea.alloc_decode_workspace(64), ea.alloc_decode_workspace)
