"""HostPipeline(graph=True): a captured step belongs to everything that its
launches hold of the weights and of the lane, each in its place."""
import types

import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

DEV = "cuda"


def test_key_holds_each_scale_in_its_place():
    pipe = object.__new__(api.HostPipeline)
    w = tuple(torch.zeros(4) for _ in range(4))
    one, per = torch.ones(1), torch.ones(8)
    keys = set()
    lanes = [dict(fp4_gscales=g) for g in (
        (None,) * 4, (one, None, None, None), (None, None, one, None), (one, None, one, None),
        (None, per, None, None), (None, None, None, per), (None, per, None, per))]
    lanes += [dict(gemm_launch="one"), dict(gemm_launch="two"), dict(w13_interleaved=True),
              dict(rank_offsets=per)]
    for kw in lanes:
        base = dict(fp4_gscales=(None,) * 4, gemm_launch=None, w13_interleaved=False, rank_offsets=None)
        pipe.lane = types.SimpleNamespace(**{**base, **kw})
        for k in (0, 1):
            key = pipe._graph_key(k, w)
            assert key == pipe._graph_key(k, w) and key not in keys
            keys.add(key)
            keys.add(pipe._graph_key(k, w[::-1]))
    assert len(keys) == 4 * len(lanes)


@pytest.mark.gpu
def test_a_scale_that_moves_to_another_operand():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, E, K, H, I = 40, 8, 2, 256, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    v, idx = torch.topk(torch.randn(T, E, generator=g, device=DEV), K, dim=1)
    p = torch.softmax(v, 1)
    w = []
    for n, k in ((2 * I, H), (H, I)):
        w += api.moe_quantize_fp4(torch.randn(E, n, k, generator=g, device=DEV) * k ** -0.5)
    one = torch.tensor([0.37], device=DEV)
    per = torch.linspace(0.3, 1.9, E, device=DEV)
    places = [(one, None, None, None), (None, None, one, None),
              (None, per, None, None), (None, None, None, per)]
    lane = lambda gs: api.MoeLayerBuffers(T, E, K, H, I, T, torch.device(DEV), packed=True, fp4="nvfp4",
                                          fp4_gscales=gs)
    want = [lane(gs).forward(x, idx, p, *w).cpu() for gs in places]
    assert all(not torch.equal(want[i], want[j]) for i in range(4) for j in range(i))
    ln = lane(places[0])
    pipe = api.HostPipeline(ln, graph=True)
    host = (x.cpu().pin_memory(), idx.cpu().pin_memory(), p.cpu().pin_memory())
    for i in (0, 1, 0, 2, 3, 2, 1):
        ln.fp4_gscales = places[i]
        out = [torch.empty(T, H, dtype=torch.bfloat16).pin_memory() for _ in range(4)]
        for y in out:
            pipe.submit(*host, y, *w)
        pipe.synchronize()
        assert all(torch.equal(y, want[i]) for y in out), i
