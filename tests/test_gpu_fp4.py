"""Microscaled 4-bit floating point: quantisation bit for bit against the
definition (oracle/fp4.py), products and the layer against 64 bits.

Bounds.  A product's output is bf16(fp32 sum): a rounding of 2^-8 of the value
(half a step), and the sum of K terms in fp32, in whatever order and with each
addition rounded down rather than to nearest, off by at most K * 2^-23 of the
sum of their magnitudes; the scales over the tensors add three roundings of
2^-24.  Z is held in 4 bits: given the scale that was stored, every code has to
be the nearest to z / (s g) but for z's own error, and the scale has to be the
one of some z within that error."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import f32
from token_dispatch_grouped_topk_gb300 import RoutedBlock, api

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = ("nvfp4", "mxfp4")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


_LUT = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def scales64(s, fmt):
    if fmt == "nvfp4":
        return s.view(torch.float8_e4m3fn).double()
    return torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))


def values(codes, scales, fmt):
    """float64 values of codes [..., n / 2] and scales."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    v = _LUT.to(codes.device)[c]
    return v * scales64(scales, fmt).repeat_interleave(O.FP4_BLOCKS[fmt], dim=-1)


def over(x, fmt, dims=None):
    """The scale over a tensor (NVFP4): its largest value to 6 times e4m3's largest."""
    if fmt == "mxfp4":
        return None
    a = x.abs().amax() if dims is None else x.abs().amax(dim=dims)
    return (a.float() / 2688.0).reshape(-1).contiguous()


def weights(E, N, K, seed, fmt):
    g = _gen(seed)
    w = 0.02 * _randn(g, E, N, K)
    wg = over(w, fmt, (1, 2))
    q, s = api.moe_quantize_fp4(w, format=fmt, gscale=wg)
    return q, s, wg


# ------------------------------------------------------------- quantisation

def _special(H, fmt):
    """Rows of edge cases."""
    b = O.FP4_BLOCKS[fmt]
    x = torch.zeros(12, H)
    mids = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.])
    x[0] = mids.repeat(H // 16)                     # ties, scale 1 (nvfp4) or 1 (mxfp4)
    x[1] = mids.repeat(H // 16) * 2.0 ** -20
    x[2] = 1e-30
    x[3] = 3e38 * torch.linspace(-1, 1, H)
    x[4] = torch.linspace(0, 1, H) ** 8
    x[5, ::b] = float("nan")
    x[6, b - 1::b] = float("inf")
    x[7, 3::b] = float("-inf")
    x[8] = 2.0 ** -130                              # below fp32's normal range
    x[9] = -0.0
    x[10] = 7.75 * torch.sign(torch.linspace(-1, 1, H))   # above six of a power of two
    x[11] = 2.0 ** torch.arange(H).remainder(40).sub(20)
    return x


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("rows,H,dtype", [(1, 128, torch.bfloat16), (1, 16384, torch.float32),
                                          (7, 384, torch.float32), (33, 1408, torch.bfloat16),
                                          (300, 4096, torch.bfloat16), (65, 640, torch.float32)])
def test_quantize_bit_exact(fmt, rows, H, dtype):
    g = _gen(rows + H)
    x = _randn(g, rows, H) * torch.exp(2 * _randn(g, rows, 1))
    sp = _special(H, fmt).to(DEV)
    x = torch.cat((x, sp)).to(dtype)
    gs = None if fmt == "mxfp4" else torch.tensor([0.0123], device=DEV)
    for gscale in ((None,) if gs is None else (None, gs)):
        xq, xs = api.moe_quantize_fp4(x, format=fmt, gscale=gscale)
        wq, ws = O.fp4_quantize(f32(x), fmt, None if gscale is None else np.float32(0.0123))
        assert np.array_equal(xs.cpu().numpy(), ws)
        fine = np.repeat(~np.isnan(O.fp4_scale_values(ws, fmt)), O.FP4_BLOCKS[fmt] // 2, axis=1)
        assert np.array_equal(xq.cpu().numpy()[fine], wq[fine])
        # the way back: code * scale is exact, then one rounding by g and one to the type
        for dt in (torch.float32, torch.bfloat16):
            y = api.moe_dequantize_fp4(xq, xs, format=fmt, gscale=gscale, dtype=dt)
            v = torch.from_numpy(O.fp4_decode(xq.cpu().numpy(), ws, fmt)).float()
            v = v if gscale is None else v * gscale.cpu()
            assert torch.equal(y.cpu().nan_to_num(777.0), v.to(dt).nan_to_num(777.0))


def test_quantize_a_scale_per_expert_and_many_rows():
    g = _gen(1)
    x = _randn(g, 5, 37, 256) * torch.arange(1, 6, device=DEV)[:, None, None]
    wg = over(x, "nvfp4", (1, 2))
    xq, xs = api.moe_quantize_fp4(x, gscale=wg)
    for e in range(5):
        q, s = O.fp4_quantize(f32(x[e]), "nvfp4", np.float32(wg[e].item()))
        assert np.array_equal(xq[e].cpu().numpy(), q) and np.array_equal(xs[e].cpu().numpy(), s)
    assert xs.max() == 0x7E and xs.dtype == torch.uint8
    # no rows, and more bytes than 32 bits count
    assert api.moe_quantize_fp4(x[:0, 0])[0].shape == (0, 128)
    big = torch.zeros(70000, 16384, dtype=torch.float32, device=DEV)
    big[-1] = x.flatten()[:16384]
    q, s = api.moe_quantize_fp4(big)
    wq, ws = O.fp4_quantize(f32(big[-1:]), "nvfp4")
    assert np.array_equal(q[-1:].cpu().numpy(), wq) and np.array_equal(s[-1:].cpu().numpy(), ws)
    assert not q[:-1].any()
    y = api.moe_dequantize_fp4(q, s, dtype=torch.float32)
    assert np.array_equal(f32(y[-1:]), O.fp4_decode(wq, ws, "nvfp4").astype(np.float32))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,E,K,H,R,packed", [
    (1, 8, 2, 128, 4, False), (1, 4, 1, 7168, 1, True), (5, 3, 3, 384, 2, False),
    (256, 64, 8, 4096, 256, True), (300, 16, 4, 1152, 40, True), (2000, 32, 8, 640, 300, False),
    (3001, 128, 6, 256, 120, True), (700, 256, 32, 128, 90, True), (64, 1024, 20, 512, 8, False),
    (4096, 8, 1, 896, 4096, True), (90, 8, 3, 16384, 50, False)])
def test_dispatch(fmt, T, E, K, H, R, packed):
    g = _gen(T + H)
    x = _randn(g, T, H).to(torch.bfloat16)
    xg = over(x, fmt)
    tq, ts = api.moe_quantize_fp4(x, format=fmt, gscale=xg)
    rows = api.packed_rows(T, K, E, R) if packed else 0
    lead = (rows,) if packed else (E, R)
    n = H // O.FP4_BLOCKS[fmt]
    for dt in (torch.int64, torch.int32):
        l = _randn(g, T, E) - torch.log(torch.arange(1, E + 1, device=DEV).float())
        idx = torch.topk(l, K, dim=1).indices
        idx = idx.masked_fill(torch.rand(T, K, generator=g, device=DEV) < 0.1, -1).to(dt)
        if T > 4:
            idx[3, 0] = E + 5                        # reported and ignored
        want = api.moe_dispatch(x, idx, None, E, R) if not packed else \
            api.moe_dispatch_packed(x, idx, None, E, R, rows=rows)
        xq = torch.full((*lead, H // 2), 0x55, dtype=torch.uint8, device=DEV)
        xs = torch.full((*lead, n), 0x33, dtype=torch.uint8, device=DEV)
        got = api.moe_dispatch_quant_fp4(x, idx, E, R, format=fmt, x_gscale=xg, rows=rows, xq=xq, xs=xs)
        for a, b in zip(got[2:], want[1:]):
            assert torch.equal(a, b)
        t, k = torch.nonzero(got[3] >= 0, as_tuple=True)
        dest = got[3][t, k].long()
        assert torch.equal(xq.view(-1, H // 2)[dest], tq[t]) and torch.equal(xs.view(-1, n)[dest], ts[t])
        free = torch.ones(xq.view(-1, H // 2).shape[0], dtype=torch.bool, device=DEV)
        free[dest] = False
        assert (xq.view(-1, H // 2)[free] == 0x55).all() and (xs.view(-1, n)[free] == 0x33).all()


def test_dispatch_without_tokens():
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(0, 2, dtype=torch.int64, device=DEV)
    st = torch.ones(2, dtype=torch.int32, device=DEV)
    _, _, counts, _, st = api.moe_dispatch_quant_fp4(x, idx, 4, 8, dev_status=st)
    assert not counts.any() and st.tolist() == [0, 0]


# ----------------------------------------------------------------- products

def _counts(E, R, kind):
    if kind == "full":
        return [R] * E
    if kind == "none":
        return [0] * E
    ends = [0, 1, R, 31, 33, 0, 64, 65, 127, 128, 129, 2, 200, 0, 255, 257]
    return [min(R, ends[(3 * e) % 16]) for e in range(E)]


def _rows(counts, R, packed, rows):
    """(expert, buffer row) of each valid row."""
    e = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    first = torch.cumsum(torch.tensor([0] + counts), 0)[:-1]
    s = torch.arange(len(e)) - first[e]
    return e.to(DEV), (torch.arange(len(e)) if packed else e * R + s).to(DEV)


def _reference(a, a_s, w, w_s, counts, R, packed, fmt, ga, gw):
    """(buffer rows, value, magnitudes' sum) of the valid rows in 64 bits."""
    e, r = _rows(counts, R, packed, a.shape[0])
    av = values(a.view(-1, a.shape[-1]), a_s.view(-1, a_s.shape[-1]), fmt)[r]
    av = av if ga is None else av * ga.double()
    out, mag = [], []
    for i in range(len(counts)):
        wv = values(w[i], w_s[i], fmt)
        wv = wv if gw is None else wv * gw[i].double()
        out.append(av[e == i] @ wv.t())
        mag.append(av[e == i].abs() @ wv.abs().t())
    return r, torch.cat(out), torch.cat(mag)


def _check_product(got, ref, mag, K):
    lim = 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + K * 2.0 ** -23 * mag
    bad = ~((got.double() - ref).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), ((got.double() - ref).abs() / lim).max())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,R,K,N,kind,packed", [
    (1, 1, 128, 128, "full", False), (1, 128, 256, 256, "full", False), (2, 128, 384, 128, "ends", True),
    (3, 40, 128, 384, "full", True), (16, 300, 512, 256, "ends", False), (16, 300, 1408, 640, "ends", True),
    (8, 1, 7168, 512, "full", True), (5, 1000, 896, 1152, "ends", False), (4, 64, 256, 256, "none", True),
    (64, 256, 1536, 1024, "ends", False), (1024, 4, 128, 128, "full", True), (2, 5, 16384, 256, "full", False)])
def test_product(fmt, E, R, K, N, kind, packed):
    g = _gen(E + R + K)
    counts = _counts(E, R, kind)
    rows = max(1, sum(counts)) + 3 if packed else 0
    lead = (rows,) if packed else (E, R)
    a = _randn(g, *lead, K)
    ag = over(a, fmt)
    aq, a_s = api.moe_quantize_fp4(a.view(-1, K), format=fmt, gscale=ag)
    # rows that hold no token hold anything: NaN scales among them
    e, r = _rows(counts, R, packed, rows)
    hole = torch.ones(aq.shape[0], dtype=torch.bool, device=DEV)
    hole[r] = False
    a_s[hole] = 0xFF
    aq, a_s = aq.view(*lead, -1), a_s.view(*lead, -1)
    w, w_s, wg = weights(E, N, K, E + N, fmt)
    out = torch.full((*lead, N), 7.0, dtype=torch.bfloat16, device=DEV)
    n = torch.tensor(counts, dtype=torch.int32, device=DEV)
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    api.moe_grouped_gemm_fp4(aq, a_s, n, w, w_s, format=fmt, a_gscale=ag, w_gscale=wg, R=R, out=out,
                             dev_status=st)
    r, ref, mag = _reference(aq, a_s, w, w_s, counts, R, packed, fmt, ag, wg)
    flat = out.view(-1, N)
    assert st.tolist() == [0, 0] and (flat[hole] == 7.0).all()
    _check_product(flat[r], ref, mag, K)
    # the same bytes on fewer SMs, and without the scales over the tensors
    again = torch.full_like(out, 7.0)
    api.moe_grouped_gemm_fp4(aq, a_s, n, w, w_s, format=fmt, a_gscale=ag, w_gscale=wg, R=R, out=again,
                             max_ctas=3)
    assert torch.equal(again, out)
    plain = api.moe_grouped_gemm_fp4(aq, a_s, n, w, w_s, format=fmt, R=R)
    r, ref, mag = _reference(aq, a_s, w, w_s, counts, R, packed, fmt, None, None)
    _check_product(plain.view(-1, N)[r], ref, mag, K)


@pytest.mark.parametrize("fmt", FMT)
def test_packed_rows_end_with_the_buffer(fmt):
    """Counts that claim more packed rows than there are: those behind the
    buffer are not touched, the ones inside are right."""
    E, R, K, N, rows = 4, 200, 384, 256, 300
    g = _gen(2)
    room = torch.zeros(rows + 200, K, device=DEV)
    room[:rows] = _randn(g, rows, K)
    aq, a_s = api.moe_quantize_fp4(room, format=fmt)
    w, w_s, wg = weights(E, N, K, 3, fmt)
    out = torch.full((rows + 200, N), 7.0, dtype=torch.bfloat16, device=DEV)
    n = torch.tensor([200, 150, 200, 1 << 30], dtype=torch.int32, device=DEV)
    api.moe_grouped_gemm_fp4(aq[:rows], a_s[:rows], n, w, w_s, format=fmt, w_gscale=wg, R=R, out=out[:rows])
    assert (out[rows:] == 7.0).all()
    _, ref, mag = _reference(aq[:rows], a_s[:rows], w, w_s, [200, 100, 0, 0], R, True, fmt, None, wg)
    _check_product(out[:rows], ref, mag, K)


@pytest.mark.parametrize("fmt", FMT)
def test_product_of_every_code_and_scale(fmt):
    """Each pair of codes and each scale byte, exactly: one nonzero element a row."""
    E, K, N = 1, 256, 256
    b = O.FP4_BLOCKS[fmt]
    rows = torch.arange(256, device=DEV)
    a = torch.zeros(256, K // 2, dtype=torch.uint8, device=DEV)
    # row r: code r % 16 at element 5 r % K, scale byte r
    col = (5 * rows) % K
    a[rows, col // 2] = ((rows % 16) << (4 * (col % 2))).to(torch.uint8)
    a_s = rows[:, None].expand(256, K // b).to(torch.uint8).contiguous()
    if fmt == "nvfp4":
        a_s &= 0x7F    # e4m3 without a sign; 0x7F is NaN
    w = torch.full((1, N, K // 2), 0, dtype=torch.uint8, device=DEV)
    nib = (torch.arange(N, device=DEV) % 16).to(torch.uint8)
    w[0] = (nib | (nib << 4))[:, None]
    w_s = torch.full((1, N, K // b), 0x38 if fmt == "nvfp4" else 127, dtype=torch.uint8, device=DEV)   # 1
    n = torch.tensor([256], dtype=torch.int32, device=DEV)
    out = api.moe_grouped_gemm_fp4(a[None], a_s[None], n, w, w_s, format=fmt)[0].float()
    ref = (values(a, a_s, fmt) @ values(w[0], w_s[0], fmt).t()).float().to(torch.bfloat16).float()
    # at the ends of e8m0 the product leaves fp32's normal range
    ok = torch.ones_like(ref, dtype=torch.bool) if fmt == "nvfp4" else \
        ((ref == 0) | (ref.abs() > 2.0 ** -120)) & (ref.abs() < 2.0 ** 126)
    nan = scales64(a_s[:, 0], fmt).isnan()
    assert out[nan].isnan().all()
    keep = ok & ~nan[:, None]
    assert torch.equal(out[keep], ref[keep])


@pytest.mark.parametrize("fmt", FMT)
def test_product_far_into_a_large_buffer(fmt):
    """Row offsets past 32 bits in the rows, the scales and the output."""
    E, R, K, N = 5, 300000, 4096, 2048
    a = torch.zeros(E, R, K // 2, dtype=torch.uint8, device=DEV)
    a_s = torch.zeros(E, R, K // O.FP4_BLOCKS[fmt], dtype=torch.uint8, device=DEV)
    counts = [0, 130, 0, 1, 150]
    g = _gen(4)
    for e, c in enumerate(counts):
        if c:
            a[e, :c], a_s[e, :c] = api.moe_quantize_fp4(_randn(g, c, K), format=fmt)
    w, w_s, wg = weights(E, N, K, 9, fmt)
    n = torch.tensor(counts, dtype=torch.int32, device=DEV)
    out = api.moe_grouped_gemm_fp4(a, a_s, n, w, w_s, format=fmt, w_gscale=wg)
    assert a.numel() > 2 ** 31 and out.numel() > 2 ** 31
    for e, c in enumerate(counts):
        if c:
            av, wv = values(a[e, :c], a_s[e, :c], fmt), values(w[e], w_s[e], fmt)
            wv = wv if wg is None else wv * wg[e].double()
            _check_product(out[e, :c], av @ wv.t(), av.abs() @ wv.abs().t(), K)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,R,H,I,kind,packed", [
    (1, 1, 128, 128, "full", False), (2, 130, 384, 256, "full", True), (16, 300, 1408, 384, "ends", False),
    (16, 270, 512, 640, "ends", True), (8, 1, 7168, 256, "full", True)])
def test_gateup(fmt, E, R, H, I, kind, packed):
    g = _gen(E + R + H)
    counts = _counts(E, R, kind)
    rows = max(1, sum(counts)) if packed else 0
    lead = (rows,) if packed else (E, R)
    x = 2 * _randn(g, *lead, H)
    xg = over(x, fmt)
    xq, xs = (t.view(*lead, -1) for t in api.moe_quantize_fp4(x.view(-1, H), format=fmt, gscale=xg))
    w, w_s, wg = weights(E, 2 * I, H, E + I, fmt)
    b = O.FP4_BLOCKS[fmt]
    zq = torch.full((*lead, I // 2), 0x55, dtype=torch.uint8, device=DEV)
    zs = torch.full((*lead, I // b), 0x33, dtype=torch.uint8, device=DEV)
    zg = torch.tensor([0.004], device=DEV) if fmt == "nvfp4" else None
    n = torch.tensor(counts, dtype=torch.int32, device=DEV)
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    api.moe_gemm_gateup_fp4(xq, xs, n, w, w_s, format=fmt, x_gscale=xg, w13_gscale=wg, z_gscale=zg, R=R,
                            zq=zq, zs=zs, dev_status=st)
    r, ref, mag = _reference(xq, xs, w, w_s, counts, R, packed, fmt, xg, wg)
    fq, fs = zq.view(-1, I // 2), zs.view(-1, I // b)
    hole = torch.ones(fq.shape[0], dtype=torch.bool, device=DEV)
    hole[r] = False
    assert st.tolist() == [0, 0] and (fq[hole] == 0x55).all() and (fs[hole] == 0x33).all()
    gate, up = ref[:, :I], ref[:, I:]
    sig = torch.sigmoid(gate)
    z = gate * sig * up
    # z's error: that of gate and up (|d silu| <= 1.1), and the exponential's,
    # the division's and the products' few units of 2^-23
    dg, du = (K_err * 2.0 ** -23 * m for K_err, m in ((H, mag[:, :I]), (H, mag[:, I:])))
    dz = 1.1 * dg * (up.abs() + du) + (gate * sig).abs() * du + 2.0 ** -19 * z.abs() * (1 + gate.abs()) + 1e-30
    zg64 = 1.0 if zg is None else zg.double()
    s = scales64(fs[r], fmt)
    blk = lambda v: v.unflatten(-1, (-1, b))
    lo = (blk(z).abs() - blk(dz)).clamp_min(0).amax(-1)
    hi = (blk(z).abs() + blk(dz)).amax(-1)

    def scale_of(a):
        if fmt == "nvfp4":
            t = (a / (6 * zg64)).clamp_max(448.0)
            return t.float().to(torch.float8_e4m3fn).double()
        return torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -125))) - 2)
    assert ((s >= scale_of(lo * (1 - 2.0 ** -22))) & (s <= scale_of(hi * (1 + 2.0 ** -22)))).all()
    # the code: nearest to z / (s g), itself off by z's error and two roundings
    sg = s[..., None] * zg64
    v = torch.where(sg > 0, blk(z) / sg.clamp_min(1e-300), 0.0)
    dv = torch.where(sg > 0, blk(dz) / sg.clamp_min(1e-300), 0.0) + 2.0 ** -22 * v.abs()
    code = blk(values(fq[r], torch.full_like(fs[r], 0x38 if fmt == "nvfp4" else 127), fmt))
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    a = code.abs()
    at = torch.searchsorted(grid, a)
    up_mid = (a + grid[(at + 1).clamp_max(7)]) / 2
    lo_mid = (a + grid[(at - 1).clamp_min(0)]) / 2
    va = torch.where(code != 0, v * torch.sign(code), v.abs())
    assert ((va <= up_mid + dv) | (a == 6)).all() and ((va >= lo_mid - dv) | (a == 0)).all()


@pytest.mark.parametrize("fmt", FMT)
def test_nan_and_infinity_stay_in_their_rows(fmt):
    E, R, H, I = 2, 70, 256, 128
    g = _gen(6)
    x = _randn(g, E, R, H)
    x[0, 3, 7], x[1, 69, 255], x[0, 10, 0] = float("nan"), float("inf"), float("-inf")
    xq, xs = api.moe_quantize_fp4(x, format=fmt)
    w, s, wg = weights(E, 2 * I, H, 1, fmt)
    w2, s2, wg2 = weights(E, H, I, 2, fmt)
    n = torch.full((E,), R, dtype=torch.int32, device=DEV)
    zq, zs = api.moe_gemm_gateup_fp4(xq, xs, n, w, s, format=fmt, w13_gscale=wg)
    out = api.moe_grouped_gemm_fp4(zq, zs, n, w2, s2, format=fmt, w_gscale=wg2)
    nan = out.isnan().all(dim=2)
    bad = torch.zeros(E, R, dtype=torch.bool, device=DEV)
    bad[0, 3] = bad[1, 69] = bad[0, 10] = True
    assert torch.equal(nan, bad) and out[~bad].isfinite().all()


# -------------------------------------------------------- the layer together

def _layer(T, E, K, H, I, seed, fmt, pad=0.1):
    g = _gen(seed)
    x = _randn(g, T, H).to(torch.bfloat16)
    v, idx = torch.topk(_randn(g, T, E) + 0.5 * _randn(g, E), K, dim=1)
    idx = idx.masked_fill(torch.rand(T, K, generator=g, device=DEV) < pad, -1)
    w13, s13, g13 = weights(E, 2 * I, H, seed + 1, fmt)
    w2, s2, g2 = weights(E, H, I, seed + 2, fmt)
    gs = (over(x, fmt), g13, torch.tensor([0.004], device=DEV) if fmt == "nvfp4" else None, g2)
    return x, idx.contiguous(), torch.softmax(v, 1).contiguous(), (w13, s13, w2, s2), gs


def _check_layer(lane, x, idx, p, w, gs, fmt):
    """The lane's stages on its own intermediates, and y against the combine's rule."""
    y = lane.forward(x, idx, p, *w)
    rr = O.route(idx.cpu().numpy(), lane.E, lane.R)
    counts = rr.counts.tolist()
    assert lane.counts.tolist() == counts and not (int(lane.dev_status[0]) & 4)
    xq, xs, zq, zs = lane.fp4_rows
    r, ref, mag = _reference(zq, zs, w[2], w[3], counts, lane.R, lane.packed, fmt, gs[2], gs[3])
    _check_product(lane.out.view(-1, lane.H)[r], ref, mag, lane.I)
    want = O.combine_f32_sequential(f32(lane.out.view(-1, lane.H)), lane.src_map.cpu().numpy(),
                                    p.cpu().numpy())
    assert np.array_equal(f32(y), O.f32_to_bf16_rne(want)), "combine"
    return y


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,E,K,H,I,R,packed", [
    (1, 16, 4, 256, 128, 1, True), (9, 8, 2, 384, 128, 4, False), (130, 6, 3, 1408, 640, 60, True),
    (700, 16, 8, 512, 256, 350, False), (2049, 32, 4, 256, 384, 200, True)])
def test_layer(fmt, T, E, K, H, I, R, packed):
    x, idx, p, w, gs = _layer(T, E, K, H, I, T, fmt)
    lane = api.MoeLayerBuffers(T, E, K, H, I, R, torch.device(DEV), packed=packed, fp4=fmt, fp4_gscales=gs)
    y = _check_layer(lane, x, idx, p, w, gs, fmt).clone()
    # the other layout's rows are the same, and so is y
    other = api.MoeLayerBuffers(T, E, K, H, I, R, torch.device(DEV), packed=not packed, fp4=fmt,
                                fp4_gscales=gs)
    assert torch.equal(other.forward(x, idx, p, *w), y)
    # the stages one by one, and both launch forms of the products
    lane.y.zero_()
    lane.dispatch_quant(x, idx, p)
    lane.gemms(*w)
    lane.combine(p, lane.y)
    assert torch.equal(lane.y, y)
    for form in ("one", "two"):
        lane.gemm_launch = form
        for _ in range(3):
            lane.y.zero_()
            assert torch.equal(lane.forward(x, idx, p, *w), y) and lane.dev_status[0].item() & 4 == 0
    lane.gemm_launch = None
    # captured and replayed with other tokens and routes
    x2, idx2, p2, _, _ = _layer(T, E, K, H, I, T + 5, fmt, pad=0.3)
    want = other.forward(x2, idx2, p2, *w).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lane.forward(x, idx, p, *w)
    for a, b in ((x, x2), (idx, idx2), (p, p2)):
        a.copy_(b)
    for _ in range(3):
        lane.y.zero_()
        graph.replay()
        assert torch.equal(lane.y, want)


@pytest.mark.parametrize("fmt", FMT)
def test_layer_from_the_residual_stream_and_from_the_host(fmt):
    T, E, K, H, I = 64, 8, 2, 256, 128
    x, _, _, w, gs = _layer(T, E, K, H, I, 3, fmt)
    g = _gen(8)
    r = _randn(g, T, H)
    nw = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
    rw = (_randn(g, E, H) / H ** 0.5).to(torch.bfloat16)
    block = RoutedBlock(T, E, K, H, I, nw, rw, fp4=fmt, fp4_gscales=gs)
    y = block.forward(x, r, *w).clone()
    lane = api.MoeLayerBuffers(T, E, K, H, I, T, torch.device(DEV), packed=True, fp4=fmt, fp4_gscales=gs)
    want = _check_layer(lane, block.h, block.topk_idx, block.topk_w, w, gs, fmt)
    assert torch.equal(y, want) and block.dev_status.tolist() == [0, 0]
    # pinned host memory in and out
    for graph in (False, True):
        pipe = api.HostPipeline(lane, graph=graph)
        host = [(block.h.cpu().pin_memory(), block.topk_idx.long().cpu().pin_memory(),
                 block.topk_w.cpu().pin_memory(), torch.empty(T, H, dtype=torch.bfloat16).pin_memory())
                for _ in range(5)]
        for h in host:
            pipe.submit(*h, *w)
        pipe.synchronize()
        assert all(torch.equal(h[3], y.cpu()) for h in host)
        if fmt == "nvfp4":   # other scales over the tensors: not the captured ones.
            # Twice W2's doubles out and y, exactly.
            lane.fp4_gscales = (*gs[:3], 2 * gs[3])
            for h in host:
                pipe.submit(*h, *w)
            pipe.synchronize()
            assert all(torch.equal(h[3], 2 * y.cpu()) for h in host)
            lane.fp4_gscales = gs


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,E,K,H,I,R,ids", [(64, 1024, 32, 128, 128, 3, torch.int32),
                                             (3000, 4, 2, 256, 128, 2000, torch.int32),
                                             (33, 8, 1, 1152, 384, 40, torch.int64)])
def test_layer_bad_ids_drops_and_nan(fmt, T, E, K, H, I, R, ids):
    """Ids outside the experts and routes past the capacity are reported and left
    out; a NaN stays in its token; both launch forms and both layouts agree."""
    x, idx, p, w, gs = _layer(T, E, K, H, I, T, fmt, pad=0.02)
    idx = idx.to(ids)
    idx[3, 0], idx[5, 0] = E, -7
    idx[9] = 2                                   # every route of a token to one expert
    x[7, 1] = float("nan")
    got = []
    for packed in (False, True):
        lane = api.MoeLayerBuffers(T, E, K, H, I, R, torch.device(DEV), packed=packed, fp4=fmt, fp4_gscales=gs)
        for form in ("one", "two", None):
            lane.gemm_launch = form
            got.append(lane.forward(x, idx, p, *w).clone())
        rr = O.route(idx.cpu().numpy(), E, R)
        assert lane.counts.tolist() == rr.counts.tolist()
        status, dropped = lane.dev_status.tolist()
        assert status == (1 | (2 if rr.dropped else 0)) and dropped == rr.dropped
    flat = [g.view(torch.int16) for g in got]
    assert all(torch.equal(flat[0], f) for f in flat)
    nan = got[0].isnan().any(dim=1)
    assert not nan[:7].any() and not nan[8:].any()
    assert bool(nan[7]) == bool((lane.src_map[7] >= 0).any())


def test_tokens_without_a_route_and_no_tokens():
    T, E, K, H, I = 20, 4, 2, 256, 128
    x, idx, p, w, gs = _layer(T, E, K, H, I, 1, "nvfp4")
    lane = api.MoeLayerBuffers(T, E, K, H, I, T, torch.device(DEV), fp4="nvfp4", fp4_gscales=gs)
    y = lane.forward(x, torch.full_like(idx, -1), p, *w)
    assert not y.any() and lane.dev_status.tolist() == [0, 0] and not lane.counts.any()
    none = api.MoeLayerBuffers(0, E, K, H, I, 4, torch.device(DEV), fp4="nvfp4", fp4_gscales=gs)
    none.counts.fill_(3)
    assert none.forward(x[:0], idx[:0], p[:0], *w).shape == (0, H) and not none.counts.any()


@pytest.mark.parametrize("fmt", FMT)
def test_scale_types_and_side_streams(fmt):
    """Scales as the 8-bit types that they are, and calls on a stream of their own
    whose outputs are allocated by the call."""
    E, R, H, I = 3, 50, 512, 256
    t8 = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    x = _randn(_gen(3), E, R, H)
    w, s, wg = weights(E, 2 * I, H, 4, fmt)
    n = torch.full((E,), R, dtype=torch.int32, device=DEV)
    xq, xs = api.moe_quantize_fp4(x, format=fmt)
    want = api.moe_grouped_gemm_fp4(xq, xs, n, w, s, format=fmt, w_gscale=wg)
    z = api.moe_gemm_gateup_fp4(xq, xs, n, w, s, format=fmt, w13_gscale=wg)
    assert torch.equal(api.moe_dequantize_fp4(xq, xs.view(t8), format=fmt),
                       api.moe_dequantize_fp4(xq, xs, format=fmt))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        q, sc = api.moe_quantize_fp4(x, format=fmt, stream=side)
        out = api.moe_grouped_gemm_fp4(q, sc.view(t8), n, w, s.view(t8), format=fmt, w_gscale=wg, stream=side)
        zq, zs = api.moe_gemm_gateup_fp4(q, sc, n, w, s, format=fmt, w13_gscale=wg, stream=side, max_ctas=1)
        del q, sc
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(zq, z[0]) and torch.equal(zs, z[1])


def test_two_halves_and_two_streams_at_once():
    T, E, K, H, I, R = 600, 16, 4, 512, 256, 300
    x, idx, p, w, gs = _layer(T, E, K, H, I, 11, "nvfp4")
    two = api.TwoBatchOverlap(T, E, K, H, I, R, torch.device(DEV), gemm_ctas=100, fp4="nvfp4",
                              fp4_gscales=gs)
    a = two.forward(x, idx, p, *w, overlap=False).clone()
    torch.cuda.synchronize()
    for _ in range(5):
        two.y.zero_()
        assert torch.equal(two.forward(x, idx, p, *w), a)
    # two lanes on two streams, and one lane's graph beside the other's eager calls
    lanes = [api.MoeLayerBuffers(T, E, K, H, I, R, torch.device(DEV), packed=True, fp4="nvfp4",
                                 fp4_gscales=gs) for _ in range(2)]
    want = lanes[0].forward(x, idx, p, *w).clone()
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for lane, s in zip(lanes, ss):
            lane.forward(x, idx, p, *w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(lane.y, want) for lane in lanes)


def test_refusals():
    x, idx, p, w, gs = _layer(8, 4, 2, 256, 128, 1, "nvfp4")
    w13, s13, w2, s2 = w
    n = torch.full((4,), 2, dtype=torch.int32, device=DEV)
    xq, xs = api.moe_quantize_fp4(x.view(4, 2, 256))
    with pytest.raises(ValueError):
        api.moe_quantize_fp4(x, format="fp4")
    with pytest.raises(TypeError):
        api.moe_quantize_fp4(x.half())
    with pytest.raises(ValueError):
        api.moe_quantize_fp4(x, gscale=gs[1])            # one for each expert, of rows without experts
    with pytest.raises(api.MoeError):
        api.moe_quantize_fp4(x, format="mxfp4", gscale=gs[0])
    with pytest.raises(api.MoeError):
        api.moe_quantize_fp4(x[:, :192].contiguous())
    with pytest.raises(ValueError):
        api.moe_quantize_fp4(x.t())
    with pytest.raises(ValueError):
        api.moe_dequantize_fp4(xq, xs[..., :-1].contiguous())
    with pytest.raises(ValueError):
        api.moe_grouped_gemm_fp4(xq, xs, n, w13[:, :, :64].contiguous(), s13)
    with pytest.raises(ValueError):
        api.moe_grouped_gemm_fp4(xq, xs, n[:3], w13, s13)
    with pytest.raises(ValueError):
        api.moe_grouped_gemm_fp4(xq.view(8, 128), xs.view(8, 16), n, w13, s13)    # packed without R
    with pytest.raises(ValueError):
        api.moe_grouped_gemm_fp4(xq.cpu(), xs, n, w13, s13)
    with pytest.raises(ValueError):
        api.moe_gemm_gateup_fp4(xq, xs, n, w13, s13, x_gscale=gs[1])
    with pytest.raises(api.MoeError):
        api.moe_grouped_gemm_fp4(xq, xs[..., ::2].contiguous(), n, w13, s13[..., ::2].contiguous(),
                                 format="mxfp4", a_gscale=gs[0])
    with pytest.raises(TypeError):
        api.moe_dispatch_quant_fp4(x.float(), idx, 4, 4)
    kw = dict(fp4="nvfp4", fp4_gscales=gs)
    with pytest.raises(ValueError):
        api.MoeLayerBuffers(8, 4, 2, 256, 128, 8, torch.device(DEV), w13_interleaved=True, **kw)
    lane = api.MoeLayerBuffers(8, 4, 2, 256, 128, 8, torch.device(DEV), **kw)
    for call in (lambda: lane.forward(x, idx, p, *w, fused=False), lambda: lane.recv, lane.workspace_views,
                 lambda: lane.dispatch_fp8(xq, xs, idx), lane.sync_view, lambda: lane.slots_fp8):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        RoutedBlock(8, 4, 2, 256, 128, torch.ones(256, device=DEV), torch.ones(4, 256, device=DEV), w4=True,
                    **kw)
