"""CPU checks of the 4-bit floating-point calls: the oracle's number format on
its worked values, and bad arguments, refused on the host before a device is
asked for."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_grouped_topk_gb300 import api, build
from test_front_abi import FAKE, MIS, _call

MIS2 = ctypes.c_void_p(4096 + 2)


def test_oracle_codes():
    # every value, the ties between them (to the even code), and beyond six
    v = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, 1e9, .26, 4.99, 5.01, np.nan])
    want = [0, 1, 2, 3, 4, 5, 6, 7, 0, 2, 2, 4, 4, 6, 6, 7, 7, 1, 6, 7, 7]
    assert O.e2m1_encode(v).tolist() == want
    assert O.e2m1_encode(-v[:-1]).tolist() == [c | 8 for c in want[:-1]]


def test_oracle_blocks():
    x = np.zeros((1, 128), np.float32)
    x[0, :16] = 3.0          # nvfp4: 3 / 6 = 0.5, codes 6; mxfp4: 2^(1 - 2), codes 6
    x[0, 32:48] = 7.5        # mxfp4: 2^0, 7.5 -> 6; nvfp4: 1.25, codes 6
    x[0, 64] = np.inf
    q, s = O.fp4_quantize(x, "nvfp4")
    assert s[0].tolist() == [0x30, 0, 0x3A, 0, 0x7F, 0, 0, 0] and q[0, :8].tolist() == [0x77] * 8
    q, s = O.fp4_quantize(x, "mxfp4")
    assert s[0].tolist() == [126, 127, 255, 0] and q[0, 16:24].tolist() == [0x77] * 8
    assert O.fp4_decode(q, s, "mxfp4")[0, [0, 15, 16, 32]].tolist() == [3.0, 3.0, 0.0, 6.0]


def test_quantize_rejects_on_host(lib):
    d = dict(x=FAKE, bits=16, g=FAKE, per=4, rows=4, H=256, fmt=0, xq=FAKE, xs=FAKE, stream=None)
    for bad in (dict(bits=8), dict(per=0), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(H=0), dict(H=192),
                dict(H=16512), dict(fmt=2), dict(fmt=-1), dict(fmt=1), dict(x=None), dict(xq=None),
                dict(xs=None), dict(x=ctypes.c_void_p(4096 + 8)), dict(xq=MIS), dict(xs=MIS2), dict(g=MIS2)):
        assert _call(lib.moe_quantize_fp4, d, **bad) == -1, bad
    d = dict(xq=FAKE, xs=FAKE, g=FAKE, per=4, rows=4, H=256, fmt=0, out=FAKE, bits=16, stream=None)
    for bad in (dict(bits=8), dict(per=0), dict(rows=-1), dict(H=192), dict(fmt=2), dict(fmt=1),
                dict(out=None), dict(xq=None), dict(xs=None), dict(out=ctypes.c_void_p(4096 + 8)),
                dict(xq=MIS), dict(xs=MIS2)):
        assert _call(lib.moe_dequantize_fp4, d, **bad) == -1, bad


def test_dispatch_rejects_on_host(lib):
    d = dict(x=FAKE, idx=FAKE, bits=64, T=112, H=256, K=2, E=8, R=128, rows=0, fmt=0, g=FAKE, xq=FAKE,
             xs=FAKE, counts=FAKE, src=FAKE, st=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    for bad in (dict(T=-1), dict(H=200), dict(K=9), dict(K=0), dict(bits=8), dict(R=0), dict(rows=223),
                dict(rows=-1), dict(fmt=2), dict(fmt=1), dict(x=None), dict(idx=None), dict(xq=None),
                dict(xs=None), dict(counts=None), dict(src=None), dict(st=None), dict(x=MIS), dict(xq=MIS),
                dict(xs=MIS2)):
        assert _call(lib.moe_dispatch_quant_fp4, d, **bad) == -1, bad
    assert _call(lib.moe_dispatch_quant_fp4, d, ws=None) == -3
    assert _call(lib.moe_dispatch_quant_fp4, d, ws=MIS2) == -3
    assert _call(lib.moe_dispatch_quant_fp4, d, ws_bytes=16) == -3


def test_products_reject_on_host(lib):
    d = dict(xq=FAKE, xs=FAKE, xg=FAKE, counts=FAKE, E=8, R=16, rows=0, H=256, I=128, w=FAKE, ws=FAKE,
             wg=FAKE, zg=FAKE, fmt=0, zq=FAKE, zs=FAKE, st=FAKE, flags=0, stream=None)
    for bad in (dict(E=0), dict(E=1025), dict(R=0), dict(R=1 << 30), dict(rows=-1), dict(rows=(1 << 30) + 1),
                dict(H=192), dict(I=64), dict(I=0), dict(fmt=2), dict(fmt=1, xg=None, wg=None),
                dict(fmt=1, zg=None, wg=None), dict(fmt=1, xg=None, zg=None), dict(flags=1), dict(flags=2),
                dict(xq=None), dict(xs=None), dict(counts=None), dict(w=None), dict(ws=None), dict(zq=None),
                dict(zs=None), dict(st=None), dict(xq=MIS), dict(xs=MIS), dict(w=MIS), dict(ws=MIS),
                dict(zq=MIS), dict(zs=MIS), dict(zg=MIS2)):
        assert _call(lib.moe_gemm_gateup_fp4, d, **bad) == -1, bad
    d = dict(a=FAKE, a_s=FAKE, ag=FAKE, counts=FAKE, E=8, R=16, rows=0, K=256, N=128, w=FAKE, ws=FAKE,
             wg=FAKE, fmt=0, out=FAKE, st=FAKE, flags=0, stream=None)
    for bad in (dict(E=0), dict(R=0), dict(rows=-1), dict(K=192), dict(N=100), dict(fmt=3),
                dict(fmt=1, ag=None), dict(fmt=1, wg=None), dict(flags=4), dict(a=None), dict(a_s=None),
                dict(counts=None), dict(w=None), dict(ws=None), dict(out=None), dict(st=None), dict(a=MIS),
                dict(a_s=MIS), dict(w=MIS), dict(ws=MIS), dict(out=MIS)):
        assert _call(lib.moe_grouped_gemm_fp4, d, **bad) == -1, bad


def test_layer_rejects_on_host(lib):
    size = lib.moe_layer_fp4_workspace_size
    assert size(112, 2, 8, 128, 0) >= lib.moe_dispatch_workspace_size(112, 2, 8) + 4 * 9
    assert size(-1, 2, 8, 128, 0) == 0 and size(4, 33, 64, 8, 0) == 0 and size(4, 2, 8, 128, -1) == 0
    d = dict(x=FAKE, idx=FAKE, bits=64, tw=FAKE, T=112, H=256, I=128, K=2, E=8, R=128, rows=0, fmt=0,
             w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, xg=FAKE, g13=FAKE, zg=FAKE, g2=FAKE, xq=FAKE, xs=FAKE,
             zq=FAKE, zs=FAKE, out=FAKE, y=FAKE, counts=FAKE, src=FAKE, st=FAKE, ws=FAKE,
             ws_bytes=1 << 20, flags=0, stream=None)
    pointers = ("x", "idx", "tw", "w13", "s13", "w2", "s2", "xq", "xs", "zq", "zs", "out", "y", "counts",
                "src", "st")
    bad = [dict(T=-1), dict(H=200), dict(I=64), dict(K=0), dict(K=9), dict(E=0), dict(R=0), dict(rows=223),
           dict(rows=-1), dict(bits=8), dict(fmt=2), dict(fmt=1), dict(fmt=1, xg=None, g13=None, zg=None),
           dict(flags=1), dict(flags=6), dict(flags=8), dict(xg=MIS2)]
    bad += [{k: None} for k in pointers]
    bad += [{k: MIS} for k in pointers if k not in ("idx", "tw", "counts", "src", "st")]
    for b in bad:
        assert _call(lib.moe_layer_fp4, d, **b) == -1, b
    assert _call(lib.moe_layer_fp4, d, ws=None) == -3
    assert _call(lib.moe_layer_fp4, d, ws=MIS2) == -3
    assert _call(lib.moe_layer_fp4, d, ws_bytes=size(112, 2, 8, 128, 0) - 1) == -3


def test_what_the_chain_writes_is_read_through_l2():
    """Counts, scales of rows and scales over tensors are written by the launches
    before, which may still run when the products start: no read-only loads."""
    with open(os.path.join(build.PKG_DIR, "csrc", "gemm_fp4.cu")) as f:
        src = f.read()
    assert "__ldg(" not in src and "ld.global.nc" not in src and "ld_stream" not in src
    kernel = src[src.index("grouped_fp4_kernel("):]
    assert kernel.index("pdl_wait()") < kernel.index("tile_prefixes(args, ctl)")
    with open(os.path.join(build.PKG_DIR, "csrc", "combine.cu")) as f:
        src = f.read()
    head = src[src.index("combine_kernel(const uint4* out"):]
    params = head[:head.index("{")]
    assert not re.search(r"(out|src_map)\b[^,]*__restrict__|__restrict__ (out|src_map)", params)


def test_binding_refuses_what_is_not_a_4_bit_lane():
    with pytest.raises(ValueError):
        api.moe_quantize_fp4(torch.zeros(2, 128))                 # host tensor
    with pytest.raises(ValueError):
        api.moe_quantize_fp4(torch.zeros(2, 128), format="int4")
    with pytest.raises(ValueError):
        api.MoeLayerBuffers(4, 4, 2, 256, 128, 8, torch.device("cpu"), fp4="fp4")
    with pytest.raises(ValueError):
        api.MoeLayerBuffers(4, 4, 2, 256, 128, 8, torch.device("cpu"), fp4="nvfp4", fp4_gscales=(None,))
    with pytest.raises(ValueError):
        api.MoeLayerBuffers(4, 4, 2, 256, 128, 8, torch.device("cpu"), fp4="nvfp4", source_slots=2)
