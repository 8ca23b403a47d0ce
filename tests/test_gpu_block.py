"""RoutedBlock: norm, router, choice, and both kinds of experts together.

The FP8 path's expert rows are held to the oracle's bar (2e-2 of a row's
largest value, see tests/helpers.py) on the block's own chosen routes; the 4-bit
path to the bound of tests/test_gpu_experts_w4.py, whose reference is taken on
the block's own normed rows and routes."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import assert_rows_close, f32, u8
from token_dispatch_grouped_topk_gb300 import RoutedBlock, api
from token_dispatch_grouped_topk_gb300 import workloads as W
from test_gpu_experts_w4 import _reference, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _layer(T, E, H, seed, residual=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    r = (2 * torch.randn(T, H, generator=g, device=DEV)).to(residual)
    nw = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    rw = (torch.randn(E, H, generator=g, device=DEV) / H ** 0.5).to(torch.bfloat16)
    return x, r, nw, rw


def _front(block, x, r, nw, rw):
    """The block's norm, logits and choice against 64 bits."""
    s = x.double() + r.double()
    n = s * (s.square().mean(dim=1, keepdim=True) + block.eps).rsqrt() * nw.double()
    assert ((block.h.double() - n).abs() <= 2.0 ** -8 * n.abs() * (1 + 1e-5) + 1e-30).all()
    logits = block.h.double() @ rw.double().t()
    lim = (block.H / 16 + 32) * 2.0 ** -22 * (block.h.double().abs() @ rw.double().abs().t())
    assert ((block.logits.double() - logits).abs() <= lim).all()


@pytest.mark.parametrize("T,E,K,H,I,capacity", [(96, 8, 2, 256, 128, None), (200, 16, 4, 512, 256, 40)])
def test_fp8_block(T, E, K, H, I, capacity):
    x, r, nw, rw = _layer(T, E, H, 3)
    w13, s13, w2, s2 = W.expert_weights(E, H, I, 5, DEV)
    block = RoutedBlock(T, E, K, H, I, nw, rw, capacity=capacity, score="sigmoid", groups=2,
                        topk_groups=2, group_top=2, scale=2.5)
    before = r.clone()
    y = block.forward(x, r, w13, s13, w2, s2)
    assert torch.equal(r, x.float() + before)
    _front(block, x, before, nw, rw)
    idx, tw = block.topk_idx.long(), block.topk_w
    assert (tw.sum(dim=1) - 2.5).abs().max() < 1e-4
    # the oracle's experts on the block's e4m3 rows and routes
    rr = O.route(idx.cpu().numpy(), E, capacity or T)
    assert block.lane.counts.cpu().tolist() == rr.counts.tolist()
    assert block.dev_status.cpu().tolist() == [2 if rr.dropped else 0, rr.dropped]
    hq, hs = u8(block.hq), f32(block.hs)
    want = np.zeros((T, H))
    for t in range(0, T, 7):
        for k in range(K):
            e = int(idx[t, k])
            if rr.src_map[t, k] < 0:
                continue
            o = O.expert_forward(hq[t:t + 1], hs[t:t + 1], u8(w13[e]), f32(s13[e]), u8(w2[e]), f32(s2[e]))[0]
            want[t] += float(tw[t, k]) * o[0]
    rows = [t for t in range(0, T, 7) if np.abs(want[t]).max() > 0]
    assert_rows_close(f32(y)[rows], want[rows])


@pytest.mark.parametrize("T,E,K,H,I", [(1, 16, 4, 512, 256), (20, 8, 2, 256, 384)])
def test_w4_block(T, E, K, H, I):
    x, r, nw, rw = _layer(T, E, H, 4, torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(1)
    weights = (*_weights(g, E, 2 * I, H), *_weights(g, E, H, I))
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    block = RoutedBlock(T, E, K, H, I, nw, rw, w4=True, score="softmax", bias=bias)
    before = r.clone()
    y = block.forward(x, r, *weights)
    _front(block, x, before, nw, rw)
    ref, lim = _reference(block.h, block.topk_idx, block.topk_w, *weights)
    assert ((y.double() - ref).abs() <= lim + 1e-30).all()
    assert block.dev_status.tolist() == [0, 0]


@pytest.mark.parametrize("w4", [False, True])
def test_block_in_a_graph(w4):
    T, E, K, H, I = 32, 8, 2, 256, 128
    x, r, nw, rw = _layer(T, E, H, 9)
    g = torch.Generator(device=DEV).manual_seed(2)
    weights = ((*_weights(g, E, 2 * I, H), *_weights(g, E, H, I)) if w4
               else W.expert_weights(E, H, I, 5, DEV))
    block = RoutedBlock(T, E, K, H, I, nw, rw, w4=w4)
    start = r.clone()
    eager = block.forward(x, r, *weights).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, r, *weights)
    r.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(block.y, eager) and torch.equal(r, x.float() + start)
    # other inputs through the same graph
    x2, r2, _, _ = _layer(T, E, H, 10)
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    torch.cuda.synchronize()
    again = block.y.clone()
    r.copy_(r2)
    assert torch.equal(block.forward(x, r, *weights), again)


def test_refusals():
    x, r, nw, rw = _layer(4, 8, 256, 1)
    with pytest.raises(ValueError):
        RoutedBlock(api.W4_MAX_TOKENS + 1, 8, 2, 256, 128, nw, rw, w4=True)
    lane = api.MoeLayerBuffers(8, 4, 2, 256, 128, 8, torch.device(DEV), source_slots=4, L=2)
    with pytest.raises(ValueError):
        lane.dispatch_fp8(torch.zeros(8, 256, dtype=torch.uint8, device=DEV),
                          torch.zeros(8, 2, device=DEV),
                          torch.zeros(8, 2, dtype=torch.int64, device=DEV))


def test_router_status_is_kept():
    """A forward leaves the projection's status alone: clear if it was, and a
    timeout until the caller has read it."""
    x, r, nw, rw = _layer(4, 8, 256, 9, torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(9)
    w13, s13 = _weights(g, 8, 2 * 128, 256)
    w2, s2 = _weights(g, 8, 256, 128)
    block = RoutedBlock(4, 8, 2, 256, 128, nw, rw, w4=True)
    block.forward(x, r, w13, s13, w2, s2)
    assert block.router_status.tolist() == [0, 0] and block.dev_status.tolist() == [0, 0]
    block.router_status[0] = 4
    block.forward(x, r, w13, s13, w2, s2)
    assert block.router_status.tolist() == [4, 0] and block.dev_status.tolist() == [0, 0]
