"""CPU checks: addresses that a kernel's vector stores or integer accesses
cannot take are refused on the host, before a device is asked for."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(4096)     # aligned, never dereferenced: validation fails first


def _at(offset):
    return ctypes.c_void_p(4096 + offset)


def test_experts_w4_refuses_a_misaligned_output(lib):
    """The combine stores eight bytes of y a thread."""
    d = dict(x=FAKE, idx=FAKE, bits=64, tw=FAKE, T=4, H=256, I=128, K=2, E=8, w13=FAKE, s13=FAKE,
             w2=FAKE, s2=FAKE, y=FAKE, st=FAKE, ws=FAKE, ws_bytes=0, stream=None)
    assert lib.moe_experts_w4(*d.values()) == -3      # nothing else is wrong but the workspace's size
    for offset in (2, 4, 6, 10):
        assert lib.moe_experts_w4(*dict(d, y=_at(offset)).values()) == -1, offset
    for offset in (8, 16):
        assert lib.moe_experts_w4(*dict(d, y=_at(offset)).values()) == -3, offset
