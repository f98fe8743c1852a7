"""The library's host side (api.cu) linked with fakes of the CUDA runtime and of the kernels (fake_device.cpp), so that what it
plans and launches can be looked at without a GPU."""
from __future__ import annotations

import ctypes
import os
import subprocess

from gqa_attention_long_gb300 import _lib, build


def load(folder) -> ctypes.CDLL:
    here, out = os.path.dirname(os.path.abspath(__file__)), os.path.join(folder, "libhost_api.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    objs = [os.path.join(folder, n) for n in ("api.o", "fake_device.o")]
    for cmd in ([build.nvcc(), *build.ARCH, *build.FLAGS, "-c", os.path.join(build.CSRC, "api.cu"), "-o", objs[0]],
                ["g++", "-std=c++17", "-O1", "-fPIC", f"-I{cuda}", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-c",
                 os.path.join(here, "fake_device.cpp"), "-o", objs[1]],
                ["g++", "-shared", "-Wl,-Bsymbolic", "-o", out, *objs, "-lpthread"]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
    h = ctypes.CDLL(out)
    V, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for name, res, args in (("text_decode_workspace_size", S, [I]), ("text_decode_mxfp4_workspace_size", S, [I]),
                            ("expert_attn_workspace_size", S, [I, I, I]), ("expert_attn_mxfp4_workspace_size", S, [I]),
                            ("text_decode_attention", I, [V, I, I, I, I, V, S, V]),
                            ("text_decode_attention_mxfp4", I, [V, I, I, I, I, V, S, V]),
                            ("expert_attn_layers", I, [V, I, I, I, I, I, V, S, V]),
                            ("expert_attn_layers_mxfp4", I, [V, I, I, I, I, V, S, V]),
                            ("expert_linear64_workspace_size", S, [I, I]),
                            ("expert_linear64", I, [V, V, V, I, I, V, S, V]),
                            ("fake_device", None, [I, I]), ("fake_set", I, [I, I]), ("fake_sms", None, [I]), ("fake_parts", I, []), ("fake_last", None, [V])):
        f = getattr(h, name)
        f.restype, f.argtypes = res, args
    return h


def fake(struct, n=1):
    """Aligned fake device pointers, all different."""
    a = (struct * n)()
    for i in range(n):
        for j, (name, _) in enumerate(struct._fields_):
            setattr(a[i], name, 0x100000 * (i + 1) + 0x1000 * j)
    return a


def last(h):
    """Of the last launch: [from, to) of the words that it needs at zero, and of the scratch that it writes besides."""
    out = (ctypes.c_uint64 * 4)()
    h.fake_last(out)
    return (out[0], out[1]), (out[2], out[3])


WS, HUGE = 0x40000000, 1 << 40


def decode(h, n, pos=300, Smax=512):
    return h.text_decode_attention(fake(_lib.EaDecodeArgs, n), n, pos, Smax, 0, WS, HUGE, None)


def decode_mxfp4(h, n, pos=300, Smax=512):
    return h.text_decode_attention_mxfp4(fake(_lib.EaAttnMxfp4Args, n), n, pos, Smax, 0, WS, HUGE, None)


def expert(h, n, S=300, Smax=512, dtype=_lib.EA_KV_BF16):
    return h.expert_attn_layers(fake(_lib.EaLayerArgs, n), n, S, Smax, 0, dtype, WS, HUGE, None)


def expert_mxfp4(h, n, S=300, Smax=512):
    return h.expert_attn_layers_mxfp4(fake(_lib.EaAttnMxfp4Args, n), n, S, Smax, 0, WS, HUGE, None)


def linear(h):
    return h.expert_linear64(0x100000, 0x200000, 0x300000, 128, 128, WS, HUGE, None)
