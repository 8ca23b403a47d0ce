"""moe_experts_w4 against the formula in 64 bits.

Tolerance, element by element, from the roundings: a dot product over n
elements takes at most n / 16 tensor-core steps and joins of a few dozen
partial sums, each off by at most 2^-22 of the magnitudes summed; z is rounded
to BF16 (2^-8), with SiLU's slope at most 1.1; y is rounded to BF16 (2^-8)."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _weights(g, E, N, K):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.int32)
    scales = (0.002 + 0.006 * torch.rand(E, N, K // 128, generator=g, device=DEV))
    return codes.to(torch.uint8), scales.to(torch.bfloat16)


def _wide(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double() - 8
    return (q.unflatten(-1, (-1, 128)) * scales.double()[..., None]).flatten(-2)


def _case(T, E, K, H, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    idx = torch.topk(torch.randn(T, E, generator=g, device=DEV), K, dim=1).indices
    w = torch.softmax(torch.randn(T, K, generator=g, device=DEV), dim=1)
    return (x, idx, w, *_weights(g, E, 2 * I, H), *_weights(g, E, H, I))


def _reference(x, idx, w, w13, s13, w2, s2):
    """(y, bound) in 64 bits."""
    T, H = x.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    lim = torch.zeros_like(y)
    g13, g2 = (H / 16 + 64) * 2.0 ** -22, (I / 16 + 64) * 2.0 ** -22
    for e in torch.unique(idx).tolist():
        if e < 0 or e >= E:
            continue
        t, k = torch.nonzero(idx == e, as_tuple=True)
        a, xd, wt = _wide(w13[e], s13[e]), x[t].double(), w[t, k].double()[:, None]
        h, dh = xd @ a.t(), g13 * (xd.abs() @ a.abs().t())
        silu = h[:, :I] * torch.sigmoid(h[:, :I])
        z = silu * h[:, I:]
        dz = 1.1 * dh[:, :I] * (h[:, I:].abs() + dh[:, I:]) + silu.abs() * dh[:, I:]
        dz += (2.0 ** -8 + 1e-6) * (z.abs() + dz)
        b = _wide(w2[e], s2[e])
        o = z @ b.t()
        do = dz @ b.abs().t() + g2 * ((z.abs() + dz) @ b.abs().t())
        y.index_add_(0, t, wt * o)
        lim.index_add_(0, t, wt.abs() * (do + 2.0 ** -21 * o.abs()))
    return y, lim + 2.0 ** -8 * (y.abs() + lim)


def _check(args, st=(0, 0)):
    status = torch.full((2,), 99, dtype=torch.int32, device=DEV)
    got = api.moe_experts_w4(*args, dev_status=status)
    y, lim = _reference(*args)
    assert torch.isfinite(got).all()
    assert ((got.double() - y).abs() <= lim + 1e-30).all()
    assert status.tolist() == list(st)
    assert torch.equal(api.moe_experts_w4(*args), got)        # the same bits again
    return got


@pytest.mark.parametrize("T,E,K,H,I", [
    (1, 8, 2, 128, 128), (1, 64, 8, 4096, 1536), (2, 4, 1, 256, 384), (7, 16, 4, 640, 256),
    (8, 8, 8, 1152, 128), (9, 3, 2, 384, 640), (33, 256, 8, 512, 256), (64, 40, 6, 256, 512),
    (64, 64, 32, 128, 128), (1, 1024, 32, 256, 128), (5, 5, 5, 16384, 128), (3, 6, 2, 128, 16384)])
def test_experts(T, E, K, H, I):
    args = _case(T, E, K, H, I, T + E + H + I)
    got = _check(args)
    ids32 = (args[0], args[1].to(torch.int32), *args[2:])
    assert torch.equal(api.moe_experts_w4(*ids32), got)


def test_many_tokens_on_one_expert():
    """All 64 tokens on the same two experts: eight passes of eight columns."""
    x, idx, w, *rest = _case(64, 6, 2, 512, 256, 3)
    idx[:] = torch.tensor([4, 1], device=DEV)
    _check((x, idx, w, *rest))


def test_padding_bad_ids_and_repeats():
    x, idx, w, *rest = _case(12, 8, 4, 256, 256, 5)
    idx[0] = -1                        # nothing: zeros
    idx[1, 1:] = -1
    idx[2] = 3                         # one expert four times
    idx[3] = torch.tensor([2, 2, -1, 7], device=DEV)
    got = _check((x, idx, w, *rest))
    assert not got[0].any()
    idx[5, 0], idx[6, 2] = 8, 1 << 40  # reported and ignored
    _check((x, idx, w, *rest), st=(api.DEV_BAD_EXPERT_ID, 0))
    idx[:] = -1
    assert not _check((x, idx, w, *rest)).any()


def test_code_values_and_order():
    """Each code against a token that selects one element: weights come back
    as (code - 8) * scale, the even element in the low four bits."""
    H = I = 128
    g = torch.Generator(device=DEV).manual_seed(1)
    w13, s13 = _weights(g, 1, 2 * I, H)
    w2, s2 = _weights(g, 1, H, I)
    idx = torch.zeros(64, 1, dtype=torch.int64, device=DEV)
    w = torch.ones(64, 1, device=DEV)
    for c0 in (0, 64):
        x = torch.zeros(64, H, dtype=torch.bfloat16, device=DEV)
        x[torch.arange(64), c0 + torch.arange(64)] = 4.0
        _check((x, idx, w, w13, s13, w2, s2))


def test_one_token_with_nan_stays_alone():
    x, idx, w, *rest = _case(6, 4, 2, 256, 128, 8)
    want = api.moe_experts_w4(x, idx, w, *rest)
    x[2, 5] = float("nan")
    got = api.moe_experts_w4(x, idx, w, *rest)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(got[keep], want[keep]) and got[2].isnan().all()


def test_weights_past_32_bit_offsets():
    """The last experts of weight tensors of more than 2^32 bytes."""
    E, H, I = 200, 8192, 2816
    w13 = torch.full((E, 2 * I, H // 2), 0x88, dtype=torch.uint8, device=DEV)   # zeros
    s13 = torch.zeros(E, 2 * I, H // 128, dtype=torch.bfloat16, device=DEV)
    w2 = torch.full((E, H, I // 2), 0x88, dtype=torch.uint8, device=DEV)
    s2 = torch.zeros(E, H, I // 128, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    a, sa = _weights(g, 2, 2 * I, H)
    b, sb = _weights(g, 2, H, I)
    w13[-2:], s13[-2:], w2[-2:], s2[-2:] = a, sa, b, sb
    assert w13.numel() > 2 ** 32
    x = torch.randn(3, H, generator=g, device=DEV).to(torch.bfloat16)
    idx = torch.tensor([[E - 1, 0], [E - 2, E - 1], [1, E - 2]], device=DEV)
    _check((x, idx, torch.rand(3, 2, generator=g, device=DEV), w13, s13, w2, s2))


def test_no_tokens_other_stream_and_graph():
    x, idx, w, *rest = _case(4, 8, 2, 256, 128, 2)
    assert api.moe_experts_w4(x[:0], idx[:0], w[:0], *rest).shape == (0, 256)
    want = api.moe_experts_w4(x, idx, w, *rest)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.moe_experts_w4(x, idx, w, *rest, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    st = torch.empty(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(api.experts_w4_workspace_size(4, 2, 256, 128), dtype=torch.uint8, device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        api.moe_experts_w4(x, idx, w, *rest, y=y, dev_status=st, workspace=ws)
    for t in (x, idx, w):
        t.copy_(t.flip(0))
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want.flip(0))


def test_refusals():
    x, idx, w, w13, s13, w2, s2 = _case(4, 8, 2, 256, 128, 2)
    f = api.moe_experts_w4
    with pytest.raises(TypeError):
        f(x.float(), idx, w, w13, s13, w2, s2)
    with pytest.raises(TypeError):
        f(x, idx, w, w13, s13.float(), w2, s2)
    with pytest.raises(ValueError):
        f(x, idx, w[:, :1].contiguous(), w13, s13, w2, s2)
    with pytest.raises(ValueError):
        f(x, idx, w, w13, s13, w2[:, :, :32].contiguous(), s2)
    with pytest.raises(ValueError):
        f(x, idx, w, w13, s13[:, :, :1].contiguous(), w2, s2)
    with pytest.raises(api.MoeError) as e:      # more tokens than the call takes
        f(x.repeat(17, 1), idx.repeat(17, 1), w.repeat(17, 1), w13, s13, w2, s2)
    assert e.value.status == -1
    with pytest.raises(api.MoeError) as e:
        f(x, idx, w, w13, s13, w2, s2, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == -3


def test_workspace_contents_do_not_matter():
    """Repeated calls on a workspace that is overwritten between them: what a
    call leaves in it is read neither early nor by the next one."""
    args = _case(3, 8, 2, 8192, 2048, 11)
    want = _check(args)
    ws = torch.empty(api.experts_w4_workspace_size(3, 2, 8192, 2048), dtype=torch.uint8, device=DEV)
    for i in range(100):
        ws.fill_(0xFF if i & 1 else 0x7E)
        assert torch.equal(api.moe_experts_w4(*args, workspace=ws), want)


@pytest.mark.parametrize("T,E,K,H,I", [(48, 16, 4, 2048, 1024), (64, 8, 4, 1024, 1408), (20, 64, 2, 4096, 640)])
def test_same_bits_beside_other_work(T, E, K, H, I):
    """Whole and shared tiles, passes of every width: the same bits again and
    again, also while another stream keeps part of the GPU busy."""
    args = _case(T, E, K, H, I, 17)
    want = _check(args)
    other = torch.cuda.Stream()
    a = torch.randn(2048, 2048, device=DEV)
    other.wait_stream(torch.cuda.current_stream())
    for i in range(60):
        if i >= 30:
            with torch.cuda.stream(other):
                a = torch.sin(a)
        assert torch.equal(api.moe_experts_w4(*args), want)
    other.synchronize()


def test_most_experts_tokens_and_routes():
    """1024 experts, 64 tokens, 32 routes each: the largest plan."""
    _check(_case(64, 1024, 32, 128, 128, 23))
