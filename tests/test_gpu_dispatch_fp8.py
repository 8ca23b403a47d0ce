"""moe_dispatch_fp8: rows already in e4m3 reach the same slots, with the same
counts, source map and status, as moe_dispatch_quant gives the BF16 rows they
were quantised from -- bit for bit, and no other row is written."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _routes(T, E, K, seed, pad=0.1, skew=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = torch.randn(T, E, generator=g, device=DEV)
    if skew:
        l -= 1.1 * torch.log(torch.arange(1, E + 1, device=DEV).float())
    idx = torch.topk(l, K, dim=1).indices
    return idx.masked_fill(torch.rand(T, K, generator=g, device=DEV) < pad, -1)


@pytest.mark.parametrize("T,E,K,H,R,packed", [
    (1, 8, 2, 128, 4, False), (1, 4, 1, 7168, 1, True), (5, 3, 3, 384, 2, False),
    (256, 64, 8, 4096, 256, False), (256, 64, 8, 4096, 256, True), (300, 16, 4, 1152, 40, True),
    (2000, 32, 8, 640, 300, False), (3001, 128, 6, 256, 120, True), (700, 256, 32, 128, 90, True),
    (64, 1024, 20, 512, 8, False), (4096, 8, 1, 896, 4096, True)])
def test_same_as_quantising_dispatch(T, E, K, H, R, packed):
    g = torch.Generator(device=DEV).manual_seed(T + H)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    tq, ts = (t[0] for t in api.moe_quantize_fp8(x[None], n))
    rows = api.packed_rows(T, K, E, R) if packed else 0
    lead = (rows,) if packed else (E, R)
    for dt in (torch.int64, torch.int32):
        idx = _routes(T, E, K, T + E, skew=K < E).to(dt)
        if T > 4:
            idx[3, 0] = E + 5                        # reported and ignored
        want = api.moe_dispatch_quant(x, idx, None, E, R, rows=rows)
        xq = torch.full((*lead, H), 0x55, dtype=torch.uint8, device=DEV)
        xs = torch.full((*lead, H // 128), -3.0, device=DEV)
        got = api.moe_dispatch_fp8(tq, ts, idx, E, R, rows=rows, xq=xq, xs=xs)
        for a, b in zip(got[2:], want[2:]):
            assert torch.equal(a, b)
        dest = got[3].view(-1).long()
        dest = dest[dest >= 0]
        assert torch.equal(xq.view(-1, H)[dest], want[0].view(-1, H)[dest])
        assert torch.equal(xs.view(-1, H // 128)[dest], want[1].view(-1, H // 128)[dest])
        free = torch.ones(xq.view(-1, H).shape[0], dtype=torch.bool, device=DEV)
        free[dest] = False
        assert (xq.view(-1, H)[free] == 0x55).all() and (xs.view(-1, H // 128)[free] == -3.0).all()


def test_float8_tensors_no_tokens_and_padding_only():
    tq = torch.randn(6, 256, device=DEV).to(torch.float8_e4m3fn)
    ts = torch.rand(6, 2, device=DEV)
    idx = torch.full((6, 2), -1, device=DEV)
    _, _, counts, src, st = api.moe_dispatch_fp8(tq, ts, idx, 4, 8)
    assert not counts.any() and (src == -1).all() and st.tolist() == [0, 0]
    _, _, counts, _, st = api.moe_dispatch_fp8(tq[:0], ts[:0], idx[:0], 4, 8)
    assert not counts.any() and st.tolist() == [0, 0]
    idx[:] = torch.tensor([1, 3], device=DEV)
    xq, xs, counts, src, _ = api.moe_dispatch_fp8(tq, ts, idx, 4, 8)
    assert torch.equal(xq[1, :6], tq.view(torch.uint8)) and torch.equal(xs[3, :6], ts)
    assert counts.tolist() == [0, 6, 0, 6]


def test_refusals():
    tq, ts = torch.zeros(4, 256, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, device=DEV)
    idx = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    f = api.moe_dispatch_fp8
    with pytest.raises(TypeError):
        f(tq.to(torch.bfloat16), ts, idx, 4, 8)
    with pytest.raises(ValueError):
        f(tq, ts[:, :1].contiguous(), idx, 4, 8)
    with pytest.raises(TypeError):
        f(tq, ts, idx.float(), 4, 8)
    with pytest.raises(ValueError):
        f(tq, ts, idx, 4, 8, xq=torch.empty(4, 7, 256, dtype=torch.uint8, device=DEV))
    with pytest.raises(api.MoeError) as e:
        f(tq, ts, idx, 4, 8, rows=7)                      # fewer than the routes
    assert e.value.status == -1
    with pytest.raises(api.MoeError) as e:
        f(tq, ts, idx, 4, 8, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))
    assert e.value.status == -3
