"""The host side of the 8-bit cache's calls with fake devices (runs without a GPU): what it does once for a device, which kernel a call
takes, and where it lays things in a workspace that calls of different sizes share."""
import ctypes
import os
import subprocess

import pytest

from gqa_attention_long_gb300 import _lib, build
from tests._host_api import HUGE, WS, fake

OK, UNSUPPORTED, WORKSPACE, INV = _lib.EA_OK, _lib.EA_ERR_UNSUPPORTED, _lib.EA_ERR_WORKSPACE, _lib.EA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def h(tmp_path_factory):
    folder, here = str(tmp_path_factory.mktemp("host")), os.path.dirname(os.path.abspath(__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    objs = [os.path.join(folder, n) for n in ("api.o", "api_fp8.o", "fake_device.o", "fake_fp8.o")]
    cmds = [[build.nvcc(), *build.ARCH, *build.FLAGS, "-c", os.path.join(build.CSRC, s), "-o", o] for s, o in zip(("api.cu", "api_fp8.cu"), objs)]
    cmds += [["g++", "-std=c++17", "-O1", "-fPIC", f"-I{cuda}", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-c", os.path.join(here, s), "-o", o]
             for s, o in zip(("fake_device.cpp", "fake_fp8.cpp"), objs[2:])]
    out = os.path.join(folder, "libhost_fp8.so")
    for cmd in [*cmds, ["g++", "-shared", "-Wl,-Bsymbolic", "-o", out, *objs, "-lpthread"]]:
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(out)
    V, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for name, res, args in (("text_decode_fp8_workspace_size", S, [I, I, I]), ("text_decode_attention_fp8", I, [V, I, I, I, I, V, S, V]),
                            ("expert_attn_evict_fp8_workspace_size", S, [I, I]), ("expert_attn_evict_fp8", I, [V, I, I, I, I, I, I, V, S, V]),
                            ("fake_device", None, [I, I]), ("fake_sms", None, [I]), ("fake_fp8_failing", None, [I]), ("fake_fp8_set", I, [I, I]),
                            ("fake_fp8_last", None, [V]), ("fake_fp8_parts", I, []), ("fake_fp8_kernel", I, []), ("fake_fp8_weights", I, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


def decode(h, n, pos=300, Smax=512, weights=True, size=HUGE):
    a = fake(_lib.EaDecodeFp8Args, n)
    if not weights:
        for x in a:
            x.weight_in = x.weight_out = None
    return h.text_decode_attention_fp8(a, n, pos, Smax, 0, WS, size, None)


def evict(h, n, rows=300, keep=200, Smax=512, size=HUGE):
    a = (_lib.EaEvictFp8Args * n)()
    for i in range(n):
        for j, (name, _) in enumerate(_lib.EaEvictFp8Args._fields_):
            setattr(a[i], name, (1 << 40) * (i + 1) + (1 << 34) * j)
    return h.expert_attn_evict_fp8(a, n, rows, keep, 1, 2, Smax, WS, size, None)


def last(h):
    out = (ctypes.c_uint64 * 4)()
    h.fake_fp8_last(out)
    return (out[0], out[1]), (out[2], out[3])


@pytest.mark.parametrize("call,what", [(decode, 0), (evict, 1)])
def test_every_device_gets_its_attributes(h, call, what):
    for d in (3 + what, 9 + what, 5 + what):
        h.fake_device(d, -1)
        assert call(h, 1) == OK
        n = h.fake_fp8_set(d, what)
        assert n >= 1 and call(h, 1) == OK and h.fake_fp8_set(d, what) == n
    d = 20 + what
    h.fake_device(d, -1)
    h.fake_fp8_failing(d)
    assert call(h, 1) == UNSUPPORTED
    h.fake_fp8_failing(-1)
    assert call(h, 1) == OK


def test_decode_calls_of_any_size_share_a_workspace(h):
    """No call's scratch lies over the counters that another one needs at zero, and all of it within the size that the largest asks for."""
    h.fake_device(0, -1)
    kernels = set()
    for weights in (False, True):
        size = h.text_decode_fp8_workspace_size(64, 4096, weights)
        for n in (1, 2, 5, 8, 9, 20, 33, 64):
            for pos in (0, 127, 300, 600, 1100, 2500, 4095):
                assert decode(h, n, pos, 4096, weights) == OK
                kernels.add(h.fake_fp8_kernel())
                (z0, z1), (lo, hi) = last(h)
                assert WS <= z0 < z1 <= lo < hi <= WS + size, (n, pos, weights)
                own = h.text_decode_fp8_workspace_size(n, 4096, weights)
                assert hi <= WS + own and decode(h, n, pos, 4096, weights, own) == OK and decode(h, n, pos, 4096, weights, own - 1) == WORKSPACE
    assert kernels == {1, 2}


@pytest.mark.parametrize("device,sms", [(30, 152), (31, 148), (32, 132), (33, 77), (34, 9)])
def test_parts_of_little_work(h, device, sms):
    """At most 32 parts to a unit (a lane of one warp weighs one), none without a tile, on GPUs of any size up to this one's."""
    h.fake_device(device, -1)
    h.fake_sms(sms)
    try:
        for n in range(1, 65):
            for pos in (0, 31, 127, 128, 400, 511, 512, 1000, 4700, 9999, 20000, 70001, 131071, (1 << 22) - 1):
                assert decode(h, n, pos, 1 << 22, False) == OK, (n, pos)
                if h.fake_fp8_kernel() == 1:
                    T = pos // 128 + 1
                    assert 1 <= h.fake_fp8_parts() <= min(32, T) and (T <= 2) <= (h.fake_fp8_parts() == 1)
                    assert h.fake_fp8_parts() == 1 or h.fake_fp8_parts() * n * 8 <= sms
    finally:
        h.fake_sms(152)


def test_weights_are_formed_only_if_asked_for(h):
    h.fake_device(0, -1)
    n = h.fake_fp8_weights()
    assert decode(h, 1, 4000, 4096, weights=False) == OK and h.fake_fp8_weights() == n
    # sixteen parts to a unit meet in the workspace, two (three layers, three tiles) in a cluster, which forms the weights itself
    assert decode(h, 1, 4000, 4096) == OK and h.fake_fp8_weights() == n + 1
    assert decode(h, 3) == OK and h.fake_fp8_weights() == n + 1
    # of 68 layers 64 are one launch, which forms them (units of 32 tiles, 3.4 to a CTA), and 4 another (four parts to a unit)
    assert decode(h, 68, 4000, 4096) == OK and h.fake_fp8_weights() == n + 1
    # beyond 39 tiles a unit's scores do not stay where they are
    assert decode(h, 64, 39 * 128 - 1, 8192) == OK and h.fake_fp8_weights() == n + 1
    assert decode(h, 64, 39 * 128, 8192) == OK and h.fake_fp8_weights() == n + 2
    # and fewer than one and a half units to a CTA (28 layers on 152 SMs) are mostly cut
    assert decode(h, 28, 4000, 4096) == OK and h.fake_fp8_weights() == n + 3
    assert decode(h, 29, 4000, 4096) == OK and h.fake_fp8_weights() == n + 3


def test_eviction_stays_in_its_workspace(h):
    h.fake_device(0, -1)
    for n in (1, 7, 64, 70):
        for Smax in (128, 512, 8192, 1 << 22):
            size = h.expert_attn_evict_fp8_workspace_size(n, Smax)
            assert evict(h, n, 100, 50, Smax, size) == OK and evict(h, n, 100, 50, Smax, size - 1) == WORKSPACE
            (z0, z1), (lo, hi) = last(h)
            assert WS <= z0 < z1 <= lo < hi <= WS + size
    assert evict(h, 1, 100, 3, 128) == OK and evict(h, 1, 100, 2, 128) == INV  # (first 1, recent 2)
