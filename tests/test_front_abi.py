"""CPU checks of the calls around the routed branch: the norm, the router, the
choice of experts, the e4m3 dispatch and the 4-bit experts reject bad arguments
on the host, before a device is asked for."""
import ctypes

import pytest
import torch

from token_dispatch_grouped_topk_gb300 import _lib, api

FAKE = ctypes.c_void_p(4096)     # aligned, never dereferenced: validation fails first
MIS = ctypes.c_void_p(4096 + 4)


def _call(fn, defaults, **changes):
    a = dict(defaults)
    assert set(changes) <= set(a)
    a.update(changes)
    return fn(*a.values())


def test_norm_rejects_on_host(lib):
    d = dict(x=FAKE, residual=FAKE, rbits=16, weight=FAKE, wbits=16, eps=1e-6, T=4, H=256, y=FAKE,
             yq=FAKE, ys=FAKE, ro=FAKE, stream=None)
    for bad in (dict(T=-1), dict(H=200), dict(H=0), dict(H=16512), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(wbits=8), dict(rbits=0),
                dict(residual=None), dict(yq=None), dict(ys=None), dict(x=None),
                dict(weight=None), dict(y=None, yq=None, ys=None), dict(x=MIS), dict(y=MIS),
                dict(yq=MIS), dict(residual=MIS), dict(ro=MIS), dict(weight=MIS)):
        assert _call(lib.moe_add_rms_norm, d, **bad) == -1, bad


def test_logits_reject_on_host(lib):
    d = dict(x=FAKE, w=FAKE, T=4, H=256, E=8, logits=FAKE, st=None, stream=None)
    for bad in (dict(T=-1), dict(H=100), dict(E=0), dict(E=1025), dict(x=None), dict(w=None),
                dict(logits=None), dict(x=MIS), dict(w=MIS)):
        assert _call(lib.moe_router_logits, d, **bad) == -1, bad


def test_topk_rejects_on_host(lib):
    d = dict(logits=FAKE, lbits=32, bias=None, T=4, E=64, K=8, score=0, groups=8, keep=4, top=2,
             renorm=1, scale=1.0, idx=FAKE, ibits=64, w=FAKE, stream=None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=33), dict(K=65),
                dict(lbits=64), dict(ibits=16), dict(score=2), dict(groups=7), dict(groups=0),
                dict(groups=64), dict(keep=0), dict(keep=9), dict(keep=1, K=9), dict(top=0),
                dict(top=3), dict(groups=32, keep=32, E=32, top=2), dict(scale=float("inf")),
                dict(logits=None), dict(idx=None), dict(w=None)):
        assert _call(lib.moe_router_topk, d, **bad) == -1, bad


def test_dispatch_fp8_rejects_on_host(lib):
    d = dict(tq=FAKE, ts=FAKE, idx=FAKE, bits=64, T=112, H=256, K=2, E=8, R=128, rows=0, xq=FAKE,
             xs=FAKE, counts=FAKE, src=FAKE, st=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    for bad in (dict(T=-1), dict(H=200), dict(K=9), dict(bits=8), dict(R=0), dict(rows=223),
                dict(rows=-1), dict(tq=None), dict(ts=None), dict(idx=None), dict(xq=None),
                dict(xs=None), dict(counts=None), dict(src=None), dict(st=None), dict(tq=MIS),
                dict(xq=ctypes.c_void_p(4096 + 8))):
        assert _call(lib.moe_dispatch_fp8, d, **bad) == -1, bad
    assert _call(lib.moe_dispatch_fp8, d, ws=None) == -3
    assert _call(lib.moe_dispatch_fp8, d, ws_bytes=16) == -3


def test_experts_w4_rejects_on_host(lib):
    size = lib.moe_experts_w4_workspace_size
    # at least x and z in two bytes an element and the routes' rows in fp32
    assert size(64, 8, 4096, 1536) >= 64 * 2 * 4096 + 64 * 8 * (1536 * 2 + 4096 * 4)
    assert size(0, 8, 4096, 1536) > 0 and size(1, 8, 4096, 1536) % 256 == 0
    assert size(65, 8, 4096, 1536) == 0 and size(4, 33, 256, 256) == 0 and size(4, 2, 200, 256) == 0
    d = dict(x=FAKE, idx=FAKE, bits=64, tw=FAKE, T=4, H=256, I=128, K=2, E=8, w13=FAKE, s13=FAKE,
             w2=FAKE, s2=FAKE, y=FAKE, st=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    for bad in (dict(T=-1), dict(T=65), dict(H=200), dict(I=100), dict(K=0), dict(K=9), dict(E=0),
                dict(E=1025), dict(bits=16), dict(x=None), dict(idx=None), dict(tw=None),
                dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None), dict(y=None),
                dict(st=None), dict(x=MIS), dict(w13=MIS), dict(w2=MIS),
                dict(s13=MIS), dict(s2=MIS)):
        assert _call(lib.moe_experts_w4, d, **bad) == -1, bad
    assert _call(lib.moe_experts_w4, d, ws=None) == -3
    assert _call(lib.moe_experts_w4, d, ws_bytes=size(4, 2, 256, 128) - 1) == -3
    assert _call(lib.moe_experts_w4, d, ws=ctypes.c_void_p(4096 + 128)) == -3


def test_limits_match_the_header():
    assert api.W4_MAX_TOKENS == _lib.W4_MAX_TOKENS == 64


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.moe_add_rms_norm(x, torch.ones(128))
    with pytest.raises(ValueError):
        api.moe_router_topk(torch.zeros(2, 8), 2)
