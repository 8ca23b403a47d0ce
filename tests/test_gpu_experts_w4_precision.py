"""The 4-bit experts held to the precision that moe.h states: x enters exactly,
z with eleven significant bits, sums in fp32, at any magnitude of a 128-group.

Tolerance, element by element.  A dot product over n elements takes at most
n / 16 tensor-core steps and joins of a few dozen partial sums, each off by at
most 2^-22 of the magnitudes summed, which are those of code * x and of 8 * x
(the codes' offset is taken off afterwards).  z is rounded within 2^-11 of
itself, or 2^-35 of its group's largest below 2^-24 of that, with SiLU's slope
at most 1.1.  y is the fp32 sum rounded to BF16, so it lies between the
roundings of the two ends of the range."""
import numpy as np
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda" if torch.cuda.is_available() else "cpu"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _pack(q):
    """Codes [..., n] to bytes [..., n / 2], the even element in the low bits."""
    return (q[..., 0::2] + 16 * q[..., 1::2]).to(torch.uint8)


def _codes(g, *shape):
    return torch.randint(0, 16, shape, generator=g, device=DEV)


def _values(q, s):
    """(weights, the magnitudes summed per element): codes and scales per 128."""
    s = s.double().repeat_interleave(128, dim=-1)
    return (q.double() - 8) * s, (q.double() + 8) * s


def _range(x, q13, s13, q2, s2, joins=64):
    """(low, high) of y for x [T, H] on one expert with weight 1."""
    H, I = x.shape[1], q13.shape[0] // 2
    xd = x.double()
    a, a_sum = _values(q13, s13)
    h, dh = xd @ a.t(), (H / 16 + joins) * 2.0 ** -22 * (xd.abs() @ a_sum.t())
    gate, up, dg, du = h[:, :I], h[:, I:], dh[:, :I], dh[:, I:]
    silu = gate * torch.sigmoid(gate)
    z = silu * up
    dz = 1.1 * dg * (up.abs() + du) + silu.abs() * du
    top = (z.abs() + dz).view(len(x), -1, 128).amax(dim=2).repeat_interleave(128, dim=1)
    dz = dz + (2.0 ** -11 + 1e-6) * (z.abs() + dz) + 2.0 ** -35 * top
    b, b_sum = _values(q2, s2)
    y, dy = z @ b.t(), dz @ b.abs().t() + (I / 16 + joins) * 2.0 ** -22 * ((z.abs() + dz) @ b_sum.t())
    dy = dy + 2.0 ** -22 * (y.abs() + dy)
    return (y - dy).float().to(torch.bfloat16), (y + dy).float().to(torch.bfloat16)


def _run(x, q13, s13, q2, s2):
    T = len(x)
    idx = torch.zeros(T, 1, dtype=torch.int64, device=DEV)
    st = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    y = api.moe_experts_w4(x, idx, torch.ones(T, 1, device=DEV), _pack(q13)[None], s13[None],
                           _pack(q2)[None], s2[None], dev_status=st)
    assert st.tolist() == [0, 0] and torch.isfinite(y).all()
    return y


def _check(*args, **kw):
    y = _run(*args)
    low, high = _range(*args, **kw)
    assert ((low <= y) & (y <= high)).all()


def _pairs(seed, T=64, H=128, I=128):
    """Intermediates in pairs that differ in one code of the up row, and down
    rows that take one pair's difference: y is far below the z it comes from,
    so its own rounding hides nothing of z's.  With one group along either
    product nothing is joined: the offset, the scale and the tokens' power of
    two are four roundings more than the products' steps."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    q13 = _codes(g, 2 * I, H)
    q13[1::2] = q13[0::2]
    up = torch.arange(I + 1, 2 * I, 2, device=DEV)
    at = torch.randint(0, H, (I // 2,), generator=g, device=DEV)
    q13[up, at] = (q13[up, at] + 3) % 16
    s13 = torch.full((2 * I, H // 128), 2.0 ** -6, dtype=torch.bfloat16, device=DEV)
    q2 = torch.full((H, I), 8, device=DEV)
    pair = torch.arange(H, device=DEV) % (I // 2)
    q2[torch.arange(H), 2 * pair], q2[torch.arange(H), 2 * pair + 1] = 15, 1
    s2 = torch.ones(H, I // 128, dtype=torch.bfloat16, device=DEV)
    return x, q13, s13, q2, s2


@pytest.mark.parametrize("seed", [1, 2])
def test_z_keeps_eleven_bits(seed):
    _check(*_pairs(seed), joins=4)


def _scales(g, N, G, exponents):
    """Scales [N, G] of 0.004 to 0.008 times a power of two (a number a group, or a row)."""
    base = 0.004 + 0.004 * torch.rand(N, G, generator=g, device=DEV)
    s = (base.double() * 2.0 ** exponents).to(torch.bfloat16)
    assert torch.isfinite(s).all() and (s > 0).all()
    return s


def test_groups_of_x_of_any_magnitude():
    """Groups of x from BF16's subnormals to 2^60 with scales that bring their
    products to one size."""
    g = torch.Generator(device=DEV).manual_seed(3)
    ex = torch.tensor([-127, -100, -20, 0, 60], device=DEV)
    H, I = 128 * len(ex), 256
    x = torch.randn(9, H, generator=g, device=DEV).double() * 2.0 ** ex.repeat_interleave(128)
    _check(x.to(torch.bfloat16), _codes(g, 2 * I, H), _scales(g, 2 * I, len(ex), -ex), _codes(g, H, I),
           _scales(g, H, I // 128, torch.zeros(I // 128, device=DEV)))


def test_groups_of_z_of_any_magnitude():
    """Groups of z from 2^-60 to 2^60, by their up rows' scales, with scales of
    the down product that bring them to one size."""
    g = torch.Generator(device=DEV).manual_seed(6)
    ez = torch.tensor([-60, -20, 0, 25, 60], device=DEV)
    H, I = 256, 128 * len(ez)
    x = torch.randn(9, H, generator=g, device=DEV).to(torch.bfloat16)
    rows = torch.cat((torch.zeros(I, device=DEV), ez.repeat_interleave(128)))
    _check(x, _codes(g, 2 * I, H), _scales(g, 2 * I, H // 128, rows[:, None]), _codes(g, H, I),
           _scales(g, H, len(ez), -ez))


def test_elements_far_below_their_groups_largest():
    """One element of 1 among elements of 2^-8 to 2^-27."""
    g = torch.Generator(device=DEV).manual_seed(4)
    H, I = 384, 128
    x = torch.randn(12, H, generator=g, device=DEV) * 2.0 ** -(8 + torch.arange(12, device=DEV) * 19 / 11)[:, None]
    x[torch.arange(12), torch.arange(12) * 30] = 1.0
    args = (x.to(torch.bfloat16), _codes(g, 2 * I, H),
            torch.full((2 * I, 3), 0.5, dtype=torch.bfloat16, device=DEV), _codes(g, H, I),
            torch.full((H, 1), 0.01, dtype=torch.bfloat16, device=DEV))
    _check(*args)


def test_code_order_and_offset_by_hand():
    """Bytes put together from the header's words and the sums done in numpy."""
    rng = np.random.default_rng(5)
    H, I = 256, 128
    q13, q2 = rng.integers(0, 16, (2 * I, H)), rng.integers(0, 16, (H, I))
    x = np.zeros((64, H))
    k = rng.permutation(H)[:64]
    x[np.arange(64), k] = 4.0
    h = 4.0 * (q13[:, k].T - 8) * 2.0 ** -4
    z = h[:, :I] / (1 + np.exp(-h[:, :I])) * h[:, I:]
    want = z @ ((q2.T - 8) * 2.0 ** -5)
    room = np.abs(z) @ np.abs(q2.T - 8) * 2.0 ** -5 * 2.0 ** -10 + np.abs(want) * 2.0 ** -8 + 1e-6
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    byte = lambda q: t((q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8))[None]
    scale = lambda n, m, v: torch.full((1, n, m), v, dtype=torch.bfloat16, device=DEV)
    y = api.moe_experts_w4(t(x).to(torch.bfloat16), torch.zeros(64, 1, dtype=torch.int64, device=DEV),
                           torch.ones(64, 1, device=DEV), byte(q13), scale(2 * I, 2, 2.0 ** -4), byte(q2),
                           scale(H, 1, 2.0 ** -5))
    assert (np.abs(y.double().cpu().numpy() - want) <= room).all()
