"""The library's host side with fake devices (runs without a GPU): what it does once for a device, and where it lays things in
a workspace that calls of different sizes share."""
import pytest

from tests import _host_api as host

OK, UNSUPPORTED = host._lib.EA_OK, host._lib.EA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def h(tmp_path_factory):
    return host.load(str(tmp_path_factory.mktemp("host")))


# a call of one layer, and which of the fake's counts of attributes is its own
CALLS = {"expert": (lambda h: host.expert(h, 1), 0), "decode": (lambda h: host.decode(h, 1), 3), "linear": (host.linear, 2),
         "decode mxfp4": (lambda h: host.decode_mxfp4(h, 1), 4), "expert mxfp4": (lambda h: host.expert_mxfp4(h, 1), 4)}


@pytest.mark.parametrize("name", CALLS)
def test_every_device_gets_its_attributes(h, name):
    """Shared memory beyond 48 KB is granted device by device: the first call on each has to ask for it."""
    call, what = CALLS[name]
    for d in (0, 5, 2):
        h.fake_device(d, -1)
        assert call(h) == OK
        n = h.fake_set(d, what)
        assert n >= 1
        assert call(h) == OK and h.fake_set(d, what) == n  # and only the first


@pytest.mark.parametrize("name", ["decode", "linear", "decode mxfp4", "expert mxfp4"])
def test_a_device_that_refuses_is_asked_again(h, name):
    call, _ = CALLS[name]
    d = 10 + list(CALLS).index(name)
    h.fake_device(d, -1)
    assert h.expert_attn_workspace_size(1, 512, 0) > 0  # (the device's own set-up)
    h.fake_device(d, d)
    assert call(h) == UNSUPPORTED
    h.fake_device(d, -1)
    assert call(h) == OK


def check_one_workspace(spans):
    """spans: by call, the words that it needs at zero (and leaves so) and the scratch that it writes, in one workspace: no
    call's scratch may lie over another's words."""
    for a, (_, (lo, hi)) in spans.items():
        for b, ((z0, z1), _) in spans.items():
            assert hi <= z0 or lo >= z1, f"{a}'s scratch [{lo - host.WS}, {hi - host.WS}) over {b}'s words [{z0 - host.WS}, {z1 - host.WS})"


@pytest.mark.parametrize("call", [host.decode, host.decode_mxfp4])
def test_decode_calls_of_any_layer_count_share_a_workspace(h, call):
    h.fake_device(0, -1)
    spans = {}
    for n in range(1, 65):
        for pos in (0, 300, 511):
            assert call(h, n, pos) == OK
            spans[n, pos] = host.last(h)
    check_one_workspace(spans)
    assert max(s[1][1] for s in spans.values()) - host.WS <= h.text_decode_workspace_size(1)


def test_expert_calls_of_any_layer_count_and_cache_share_a_workspace(h):
    """An e4m3 workspace also serves bf16 calls, which count on words that every call leaves at zero."""
    h.fake_device(0, -1)
    spans = {}
    for n in range(1, 65):
        for dtype in (host._lib.EA_KV_BF16, host._lib.EA_KV_FP8_E4M3):
            assert host.expert(h, n, dtype=dtype) == OK
            spans[n, dtype] = host.last(h)
    check_one_workspace(spans)
    assert max(s[1][1] for s in spans.values()) - host.WS <= h.expert_attn_workspace_size(64, 512, host._lib.EA_KV_FP8_E4M3)


@pytest.mark.parametrize("device,sms", [(30, 152), (31, 148), (32, 132), (33, 77), (34, 8)])
def test_units_of_a_decode_step_have_at_most_32_parts(h, device, sms):
    """A lane of one warp weighs a part, of any number of layers at any length, on GPUs of any size up to this one's."""
    h.fake_device(device, -1)
    h.fake_sms(sms)
    try:
        for n in (1, 2, 3, 4, 5, 6, 9, 18, 19, 20, 33, 64):
            for pos in (0, 31, 400, 1000, 1087, 1100, 2000, 4700, 9999, 20000, 70001, 131071, (1 << 22) - 1):
                assert host.decode_mxfp4(h, n, pos, max(128, -(-(pos + 1) // 64) * 64)) == OK, (n, pos)
                assert 1 <= h.fake_parts() <= 32, (n, pos)
    finally:
        h.fake_sms(152)


def test_a_gpu_with_more_parts_than_that_is_refused(h):
    h.fake_device(40, -1)
    h.fake_sms(400)
    try:
        assert host.decode_mxfp4(h, 1, 131071, 131072) == UNSUPPORTED
    finally:
        h.fake_sms(152)
