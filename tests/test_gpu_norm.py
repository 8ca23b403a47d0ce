"""moe_add_rms_norm against the formula in 64 bits.

Tolerances.  The sum of squares of a row is at most 64 terms in sequence per
thread and a tree, (64 + 10) * 2^-24 = 4.4e-6 relative at worst, halved by the
root; the root, the division and two products add a few 2^-24: 4e-6 in all.
A BF16 result has to lie between the roundings of the two ends of that range;
e4m3 rounds to nearest within 2^-4 (2^-10 of the scale below its normal range)."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP32 = 4e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _inputs(T, H, residual, weight, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    r = None if residual is None else (3 * torch.randn(T, H, generator=g, device=DEV)).to(residual)
    w = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(weight)
    return x, r, w


def _reference(x, r, w, eps):
    s = x.double() if r is None else x.double() + r.double()
    return s, s * (s.square().mean(dim=1, keepdim=True) + eps).rsqrt() * w.double()


def _check(x, r, w, eps, y, yq, ys, r_out, r_before):
    s, n = _reference(x, r_before, w, eps)
    if y is not None:
        low, high = ((n - d * n.abs()).to(torch.bfloat16) for d in (FP32, -FP32))
        assert ((low <= y) & (y <= high)).all()
    if r_before is not None:
        assert torch.equal(r_out, (x.float() + r_before.float()).to(r_before.dtype))
    if yq is not None:
        T, H = x.shape
        top = n.view(T, -1, 128).abs().amax(dim=2).clamp_min(float(torch.tensor(1e-4)))
        assert ((ys.double() - top / 448.0).abs() <= 2 * FP32 * top / 448.0).all()
        got = yq.view(torch.float8_e4m3fn).double().view(T, -1, 128) * ys.double()[..., None]
        lim = (2.0 ** -4 + 4 * FP32) * n.view(T, -1, 128).abs() + 2.0 ** -10 * ys.double()[..., None]
        assert ((got - n.view(T, -1, 128)).abs() <= lim).all()


@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 128), (5, 256), (9, 1024), (3, 1152), (1, 7168), (37, 4096),
                                 (700, 2176), (311, 16384), (2, 16384), (1000, 384)])
def test_norm(T, H, residual):
    for weight in (torch.bfloat16, torch.float32):
        x, r, w = _inputs(T, H, residual, weight, T + H)
        y, yq, ys, ro = api.moe_add_rms_norm(x, w, 1e-6, residual=r, quant=True)
        _check(x, r, w, 1e-6, y, yq, ys, ro, r)
        # each output alone gives the same bits
        y2, none_q, none_s, _ = api.moe_add_rms_norm(x, w, 1e-6, residual=r)
        assert none_q is None and none_s is None and torch.equal(y2, y)
        none_y, yq2, ys2, _ = api.moe_add_rms_norm(x, w, 1e-6, residual=r, bf16=False, quant=True)
        assert none_y is None and torch.equal(yq2, yq) and torch.equal(ys2, ys)


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_residual_in_place(residual):
    x, r, w = _inputs(333, 4096, residual, torch.bfloat16, 4)
    y0, _, _, ro = api.moe_add_rms_norm(x, w, residual=r)
    r1 = r.clone()
    y1, _, _, same = api.moe_add_rms_norm(x, w, residual=r1, residual_out=r1)
    assert same is r1 and torch.equal(r1, ro) and torch.equal(y0, y1)


def test_zero_rows_small_rows_and_neighbours():
    """A zero row stays zero; a row far below eps^(1/2) is scaled by eps; a
    row with an infinity or NaN leaves the others alone."""
    x, _, w = _inputs(8, 1152, None, torch.float32, 7)
    clean = api.moe_add_rms_norm(x, w, quant=True)
    x[2] = 0
    x[3] = (x[3].float() * 1e-6).to(torch.bfloat16)
    ref = api.moe_add_rms_norm(x, w, quant=True)
    _check(x, None, w, 1e-6, *ref, None)
    assert not ref[0][2].any() and not ref[1][2].any()
    x[5, 17], x[6, 1000] = float("inf"), float("nan")
    y, yq, ys, _ = api.moe_add_rms_norm(x, w, quant=True)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(y[keep], ref[0][keep]) and torch.equal(yq[keep], ref[1][keep])
    assert torch.equal(ys[keep], ref[2][keep]) and torch.equal(y[0], clean[0][0])
    assert y[6].isnan().all()


def test_rows_past_32_bit_offsets():
    T, H = 140000, 16384       # 2.3e9 elements
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    x[-3:] = _inputs(3, H, None, torch.bfloat16, 1)[0]
    y, yq, ys, _ = api.moe_add_rms_norm(x, w, quant=True)
    want = api.moe_add_rms_norm(x[-3:].clone(), w, quant=True)
    # another number of rows may sum in another order: within the bound
    _check(x[-3:], None, w, 1e-6, y[-3:], yq[-3:], ys[-3:], None, None)
    _check(x[-3:], None, w, 1e-6, *want, None)
    assert not y[:5].any()


def test_no_rows_other_stream_and_graph():
    x, r, w = _inputs(64, 4096, torch.bfloat16, torch.bfloat16, 3)
    assert api.moe_add_rms_norm(x[:0], w)[0].shape == (0, 4096)
    want = api.moe_add_rms_norm(x, w, residual=r, quant=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.moe_add_rms_norm(x, w, residual=r, quant=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = dict(zip(("y", "yq", "ys", "residual_out"), (torch.empty_like(t) for t in want)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.moe_add_rms_norm(x, w, residual=r, **outs)
    x.copy_(x.flip(0))
    want = api.moe_add_rms_norm(x, w, residual=r, quant=True)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs.values(), want))


def test_refusals():
    x, r, w = _inputs(4, 256, torch.bfloat16, torch.bfloat16)
    f = api.moe_add_rms_norm
    with pytest.raises(TypeError):
        f(x.float(), w)
    with pytest.raises(TypeError):
        f(x, w.half())
    with pytest.raises(ValueError):
        f(x, w[:128])
    with pytest.raises(ValueError):
        f(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        f(x, w, residual_out=r)                         # nothing to add
    with pytest.raises(TypeError):
        f(x, w, residual=r, residual_out=r.float())
    with pytest.raises(ValueError):
        f(x, w.cpu())
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        with pytest.raises(api.MoeError):
            f(x, w, eps)
    with pytest.raises(api.MoeError):                   # no output
        f(x, w, bf16=False)
    with pytest.raises(api.MoeError):                   # H % 128
        f(x[:, :200].contiguous(), w[:200].contiguous())
    big = torch.empty(4 * 256 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 256)
    with pytest.raises(api.MoeError):                   # 16-byte alignment
        f(big, w)
