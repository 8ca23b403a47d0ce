"""Tensors that are all zero, with the scale over them that the data gives: zero
as well.  Their blocks have scale 0 and zero codes, and products with them are 0."""
import numpy as np
import pytest
import torch

import oracle as O
from token_dispatch_grouped_topk_gb300 import api

DEV = "cuda"


def test_oracle_zero_block_under_a_zero_scale():
    q, s = O.fp4_quantize(np.zeros((2, 128), np.float32), "nvfp4", np.array([0.0, 1.0], np.float32))
    assert not q.any() and not s.any()
    x = np.zeros((1, 128), np.float32)
    x[0, 16] = np.nan
    assert O.fp4_quantize(x, "nvfp4", 0.0)[1][0].tolist() == [0, 0x7F, 0, 0, 0, 0, 0, 0]


def _over(v):
    return (v.float().abs().amax(dim=tuple(range(1, v.dim()))) / 2688.0).contiguous()


def _experts(E, N, K, g, empty):
    w = 0.02 * torch.randn(E, N, K, generator=g, device=DEV)
    w[empty] = 0
    over = _over(w)
    assert over[empty] == 0
    return w, api.moe_quantize_fp4(w, gscale=over), over


@pytest.mark.gpu
@pytest.mark.parametrize("zero_x", (False, True))
@pytest.mark.parametrize("T,packed", [(5, True), (300, False), (1200, True)])
def test_an_all_zero_expert_and_all_zero_rows(T, packed, zero_x):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    E, K, H, I, empty = 6, 4, 256, 128, 2
    g = torch.Generator(device=DEV).manual_seed(T)
    w13, (q13, s13), g13 = _experts(E, 2 * I, H, g, empty)
    w2, (q2, s2), g2 = _experts(E, H, I, g, empty)
    for w, q, s, over in ((w13, q13, s13, g13), (w2, q2, s2, g2)):
        rows = over.repeat_interleave(w.shape[1]).cpu().numpy()
        oq, os_ = O.fp4_quantize(w.reshape(-1, w.shape[2]).cpu().numpy(), "nvfp4", rows)
        assert np.array_equal(q.cpu().numpy().reshape(oq.shape), oq)
        assert np.array_equal(s.cpu().numpy().reshape(os_.shape), os_)
        assert not q[empty].any() and not s[empty].any()
        assert not api.moe_dequantize_fp4(q, s, gscale=over)[empty].any()
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    if not zero_x:
        x.copy_(torch.randn(T, H, generator=g, device=DEV))
    gx = _over(x.reshape(1, -1))
    gz = torch.full((1,), 0.0 if zero_x else 0.004, device=DEV)
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(dim=1)[:, :K].contiguous()
    p = torch.rand(T, K, generator=g, device=DEV)
    lane = api.MoeLayerBuffers(T, E, K, H, I, T, torch.device(DEV), packed=packed, fp4="nvfp4",
                               fp4_gscales=(gx, g13, gz, g2))
    for form in ("one", "two"):
        lane.gemm_launch = form
        y = lane.forward(x, idx, p, q13, s13, q2, s2)
        assert y.isfinite().all() and lane.dev_status.tolist() == [0, 0]
        # routes to the empty expert give zero rows
        at = lane.src_map[idx == empty].long()
        assert len(at) and not lane.out.view(-1, H)[at].any()
        if zero_x:
            assert not y.any()
    # the same y where those routes are left out
    if not zero_x:
        want = y.clone()
        assert torch.equal(lane.forward(x, idx.masked_fill(idx == empty, -1), p, q13, s13, q2, s2), want)
