"""moe_router_logits against the product in 64 bits.

Tolerance: products of BF16 are exact in fp32.  A sum of H of them takes at
most H / 16 steps of the tensor core and a few joins, each off by at most
2^-22 of the running magnitude (a truncated fp32 sum), so |error| <=
(H / 16 + 32) * 2^-22 * sum |x| |w|."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _inputs(T, E, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    # rows after x and w hold NaN: nothing past the matrices may be read in
    xb = torch.full((T + 130, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    wb = torch.full((E + 260, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    xb[:T] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    wb[:E] = (torch.randn(E, H, generator=g, device=DEV) / H ** 0.5).to(torch.bfloat16)
    return xb[:T], wb[:E]


def _assert_close(got, x, w):
    H = x.shape[1]
    want = x.double() @ w.double().t()
    lim = (H / 16 + 32) * 2.0 ** -22 * (x.double().abs() @ w.double().abs().t())
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= lim).all()


@pytest.mark.parametrize("T,E,H", [
    (1, 256, 7168), (1, 1, 128), (2, 7, 256), (17, 60, 4096), (127, 64, 512), (128, 64, 4096),
    (129, 100, 1152), (256, 64, 4096), (300, 160, 2048), (1000, 257, 896), (513, 512, 640),
    (65, 1024, 384), (5000, 256, 1024), (20001, 96, 256), (33, 1000, 16384)])
def test_logits(T, E, H):
    x, w = _inputs(T, E, H, T + E + H)
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    guard = torch.full((T * E + 64,), -7.0, device=DEV)
    out = guard[:T * E].view(T, E)
    got = api.moe_router_logits(x, w, logits=out, dev_status=st)
    _assert_close(got, x, w)
    assert (guard[T * E:] == -7.0).all() and st.tolist() == [0, 0]
    assert torch.equal(api.moe_router_logits(x, w), got)      # the same bits again


def test_one_token_row_with_nan_stays_alone():
    x, w = _inputs(40, 64, 512, 3)
    want = api.moe_router_logits(x, w)
    x[7, 100] = float("nan")
    got = api.moe_router_logits(x, w)
    keep = [t for t in range(40) if t != 7]
    assert torch.equal(got[keep], want[keep]) and got[7].isnan().all()


def test_unaligned_output_and_no_rows():
    x, w = _inputs(37, 64, 256, 5)
    buf = torch.empty(37 * 64 + 1, device=DEV)
    _assert_close(api.moe_router_logits(x, w, logits=buf[1:].view(37, 64)), x, w)
    assert api.moe_router_logits(x[:0], w).shape == (0, 64)


def test_other_stream_and_graph():
    x, w = _inputs(200, 64, 1024, 6)
    want = api.moe_router_logits(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.moe_router_logits(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.moe_router_logits(x, w, logits=out)
    x.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(0))


def test_refusals():
    x, w = _inputs(4, 8, 256, 0)
    f = api.moe_router_logits
    with pytest.raises(TypeError):
        f(x.float(), w)
    with pytest.raises(TypeError):
        f(x, w.float())
    with pytest.raises(ValueError):
        f(x, w[:, :128].contiguous())
    with pytest.raises(ValueError):
        f(x, w, logits=torch.empty(4, 9, device=DEV))
    with pytest.raises(TypeError):
        f(x, w, logits=torch.empty(4, 8, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(api.MoeError):
        f(x, torch.zeros(1025, 256, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(api.MoeError):
        f(x[:, :200].contiguous(), w[:, :200].contiguous())
