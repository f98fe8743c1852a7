"""The waits of the kernels over a 4-bit cache, which give up after a number of looks, and the calls that follow one that
gave up (without a fault: see test_gpu_failure)."""
import pytest
import torch

import gqa_attention_long_gb300 as ea
from tests._gpu_util import check_status
from tests._mxfp4_util import decode_oracle, device_buffers, expert_oracle, random_cache, step_inputs
from tests.test_gpu_mxfp4_attention import close

pytestmark = pytest.mark.gpu
WAIT, LOOKS = 1 << 6, 1 << 9


def test_both_kinds_of_waits_give_up_and_report():
    ws = ea.alloc_mxfp4_workspace(1)
    ea.expert_attn_selftest_wait_timeout(1000, ws)
    assert ea.expert_attn_read_status(ws) == (ea._lib.EA_ERR_TIMEOUT, WAIT | LOOKS)


@pytest.mark.parametrize("form", ["decode", "expert"])
def test_a_cleared_workspace_serves_again(form):
    """What a call that gave up leaves: a status, and in a decode step's workspace counts that are not zero."""
    call, alloc, init, ref, hq, tok = {
        "decode": (ea.text_decode_attention_mxfp4, ea.alloc_decode_mxfp4_workspace, ea.text_decode_workspace_init, decode_oracle, 64, 1),
        "expert": (ea.expert_attn_layers_mxfp4, ea.alloc_mxfp4_workspace, ea.expert_attn_workspace_init, expert_oracle, 16, 64)}[form]
    ws = alloc(2)
    ea.expert_attn_selftest_wait_timeout(1000, ws)
    ws[1024:].fill_(3)
    assert ea.expert_attn_read_status(ws)[0] == ea._lib.EA_ERR_TIMEOUT
    init(ws)
    xs, hs = [step_inputs(l, hq, tok) for l in range(2)], [random_cache(5 + l, 2048, 1900) for l in range(2)]
    bufs = [device_buffers(x, h.device()) for x, h in zip(xs, hs)]
    call(bufs, 1900, 2048, 0, ws)
    torch.cuda.synchronize()
    check_status(ws)
    for l in range(2):
        close(bufs[l].out, ref(xs[l], hs[l], 1900, 0)["out"], f"layer {l}")
