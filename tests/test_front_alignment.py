"""CPU checks: addresses that a kernel's vector stores or integer accesses
cannot take are refused on the host, before a device is asked for."""
import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("call", ["moe_dispatch_fp8", "moe_dispatch_quant_ex", "moe_dispatch_ex"])
def test_dispatch_refuses_a_workspace_off_its_integers(lib, call):
    """The workspace holds int32 counts; a byte tensor's view may begin anywhere.
    A device is asked for only after the checks: -2 without one."""
    out = [FAKE] * (4 if call == "moe_dispatch_ex" else 5)     # receive buffer(s), counts, source map, status
    head = [FAKE, FAKE, FAKE, 64] if call == "moe_dispatch_fp8" else [FAKE, FAKE, 64, None]
    args = lambda T, ws: [*head, T, 256, 2, 8, 128, 0, *out, ws, 1 << 20, None]
    for offset in (1, 2, 3, 5):
        assert getattr(lib, call)(*args(112, _at(offset))) == -3, offset
    if not torch.cuda.is_available():
        assert getattr(lib, call)(*args(112, _at(4))) in (-2, -4)


def test_ep_offsets_refuse_a_workspace_off_its_integers(lib):
    for offset in (1, 2, 3):
        assert lib.moe_ep_route_offsets(FAKE, 8, 2, FAKE, _at(offset), 1 << 20, None) == -3
