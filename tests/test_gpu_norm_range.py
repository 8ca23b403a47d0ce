"""moe_add_rms_norm on rows whose squares leave fp32's range when they are
summed, though their mean does not, and on rows far below 1.

Tolerance: at most 16 terms in sequence per thread and two trees of five steps
put 26 * 2^-24 on the sum of squares, halved by the root; the sum r, the
division, the addition of eps, the root (two last places) and two products add
less than 1.2e-6: 2e-6 in all.  A BF16 result lies between the roundings of the
two ends of that range; e4m3 rounds to nearest within 2^-4 (2^-10 of the scale
below its normal range)."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP32 = 2e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _check(x, r, w, eps):
    y, yq, ys, ro = api.moe_add_rms_norm(x, w, eps, residual=r, quant=True)
    s = x.double() if r is None else x.double() + r.double()
    n = s * (s.square().mean(dim=1, keepdim=True) + eps).rsqrt() * w.double()
    low, high = ((n - d * n.abs()).to(torch.bfloat16) for d in (FP32, -FP32))
    assert ((low <= y) & (y <= high)).all()
    T, H = x.shape
    n = n.view(T, -1, 128)
    top = n.abs().amax(dim=2).clamp_min(float(torch.tensor(1e-4)))
    assert ((ys.double() - top / 448.0).abs() <= 2 * FP32 * top / 448.0).all()
    got = yq.view(torch.float8_e4m3fn).double().view(T, -1, 128) * ys.double()[..., None]
    assert ((got - n).abs() <= (2.0 ** -4 + 4 * FP32) * n.abs() + 2.0 ** -10 * ys.double()[..., None]).all()
    if r is not None:
        assert torch.equal(ro, (x.float() + r.float()).to(r.dtype))


# rows of a warp, of a block with one vector a thread and with two
@pytest.mark.parametrize("H", [128, 256, 384, 4096, 8192, 16384])
@pytest.mark.parametrize("size", [1e19, 1.7e19, 6e18, 3e17, 1e-18])
def test_mean_of_squares_inside_the_range(H, size):
    """Elements around 1e19: each square and their mean are fp32 numbers
    (1.7e19: 2.9e38 at most), the sum of H of them is not."""
    g = torch.Generator(device=DEV).manual_seed(H)
    w = 1 + 0.2 * torch.randn(H, generator=g, device=DEV)
    sign = torch.randint(0, 2, (11, H), generator=g, device=DEV) * 2 - 1
    v = sign * (0.5 + 0.5 * torch.rand(11, H, generator=g, device=DEV)) * size
    x = v.to(torch.bfloat16)
    x[3] = torch.randn(H, generator=g, device=DEV).to(torch.bfloat16)   # an ordinary row beside them
    x[4] = 0
    x[5, 1:] = 0                                                        # one large element
    _check(x, None, w, 1e-6 if size > 1 else 1e-37)
    _check(x, v.neg() * 0.25, w, 1e-6 if size > 1 else 1e-37)


def test_infinite_rows_beside_large_ones():
    """A row with an infinity has a NaN in y, as ever, and changes no other."""
    g = torch.Generator(device=DEV).manual_seed(1)
    for H in (256, 2048):
        w = torch.ones(H, device=DEV)
        x = (1e19 * torch.randn(6, H, generator=g, device=DEV).clamp(-1.5, 1.5)).to(torch.bfloat16)
        want = api.moe_add_rms_norm(x, w)[0]
        x[2, 7], x[4, 9] = float("inf"), float("nan")
        y = api.moe_add_rms_norm(x, w)[0]
        keep = [0, 1, 3, 5]
        assert torch.equal(y[keep], want[keep]) and y[2, 7].isnan() and y[4].isnan().all()
