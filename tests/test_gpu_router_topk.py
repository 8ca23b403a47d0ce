"""moe_router_topk against the definition in 64 bits, token after token.

Ids are compared exactly where the choice is not nearer than 1e-5 (scores are
fp32: 2^-23 relative and a few operations, below 1e-6 for scores and biases of
order one); with whole-number logits, ties and all, every id is compared.
Weights: expf, a division, a sum of at most 1024 terms as a tree over 32
partial sums and a product: 1e-5 relative."""
import numpy as np
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _choose(l, K, score, bias, groups, keep, top, renorm, scale):
    """(ids, weights, how near the closest decision was) of one token."""
    E = l.size
    masked = np.isnan(l) | np.isneginf(l)
    lm = np.where(masked, -np.inf, l)
    ids, w = np.full(K, -1), np.zeros(K)
    if masked.all():
        return ids, w, np.inf
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-lm))
    else:
        m = lm.max()
        e = np.exp(np.where(lm == m, 0.0, lm - m) if np.isinf(m) else lm - m)
        if np.isinf(m):
            e = np.where(lm == m, 1.0, 0.0)
        s = e / e.sum()
    s = np.where(masked, 0.0, s)
    c = lm if bias is None else np.where(masked, -np.inf, s + bias)
    near = np.inf
    ok = ~np.isneginf(c)
    if groups > 1:
        gs = []
        for g in range(groups):
            r = slice(g * E // groups, (g + 1) * E // groups)
            v = (c if top == 1 or bias is not None else np.where(masked, -np.inf, s))[r]
            best = np.sort(v)[::-1][:top]
            best = best[~np.isneginf(best)]
            gs.append(best.sum() if best.size else -np.inf)
        gs = np.array(gs)
        order = np.argsort(-gs, kind="stable")
        if keep < groups and np.isfinite(gs[order[keep]]):
            near = min(near, gs[order[keep - 1]] - gs[order[keep]])
        for g in order[keep:]:
            ok[g * E // groups:(g + 1) * E // groups] = False
        for g in order[:keep]:
            if np.isneginf(gs[g]):
                ok[g * E // groups:(g + 1) * E // groups] = False
    c = np.where(ok, c, -np.inf)
    order = np.argsort(-c, kind="stable")
    n = min(K, int(ok.sum()))
    ids[:n] = order[:n]
    w[:n] = s[order[:n]]
    v = c[order[:min(n + 1, int(ok.sum()))]]
    if v.size > 1 and np.isfinite(v).all():
        near = min(near, np.min(v[:-1] - v[1:]))
    if renorm:
        w = w / max(w.sum(), 1e-20)
    return ids, w * scale, near


def _check(logits, K, exact_ids=False, **o):
    opts = dict(score="softmax", bias=None, groups=1, keep=None, top=1, renorm=True, scale=1.0)
    opts.update(o)
    if opts["keep"] is None:
        opts["keep"] = opts["groups"]
    T, E = logits.shape
    both = []
    for dt in (torch.int64, torch.int32):
        idx, w = api.moe_router_topk(
            logits, K, score=opts["score"], bias=opts["bias"], groups=opts["groups"],
            topk_groups=opts["keep"], group_top=opts["top"], renormalize=opts["renorm"],
            scale=opts["scale"], idx_dtype=dt)
        assert idx.dtype == dt
        both.append((idx.long(), w))
    assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1])
    idx, w = both[0][0].cpu().numpy(), both[0][1].double().cpu().numpy()
    l = logits.double().cpu().numpy()
    b = None if opts["bias"] is None else opts["bias"].double().cpu().numpy()
    compared = 0
    with np.errstate(all="ignore"):
        for t in range(T):
            ids, ws, near = _choose(l[t], K, opts["score"], b, opts["groups"], opts["keep"],
                                    opts["top"], opts["renorm"], opts["scale"])
            if not exact_ids and near <= 1e-5:
                continue
            compared += 1
            assert np.array_equal(idx[t], ids), (t, idx[t], ids)
            assert np.all(np.abs(w[t] - ws) <= 1e-5 * np.abs(ws) + 1e-30), t
    assert compared >= 0.8 * T


def _logits(T, E, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, E, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 8, 8), (7, 32, 4), (40, 33, 5), (19, 60, 6),
                                   (300, 64, 8), (33, 100, 3), (700, 128, 8), (64, 160, 32),
                                   (1500, 256, 8), (20, 257, 9), (11, 512, 16), (9, 1000, 32),
                                   (5, 1024, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_plain_choice(T, E, K, score):
    _check(_logits(T, E, T + E), K, score=score)
    _check(_logits(T, E, T + E + 1), K, score=score, renorm=False, scale=2.5)
    bias = 0.05 * _logits(1, E, 5)[0]
    _check(_logits(T, E, T + E + 2), K, score=score, bias=bias)


@pytest.mark.parametrize("E,K,groups,keep", [(256, 8, 8, 4), (60, 6, 6, 3), (160, 6, 8, 3),
                                             (64, 4, 4, 1), (64, 8, 32, 16), (96, 5, 3, 2),
                                             (1024, 8, 8, 2), (10, 2, 5, 1)])
@pytest.mark.parametrize("top", [1, 2])
def test_groups(E, K, groups, keep, top):
    bias = 0.05 * _logits(1, E, 9)[0]
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            _check(_logits(200, E, E + groups), K, score=score, bias=b, groups=groups, keep=keep,
                   top=top)


def test_ties_go_to_the_lowest_id():
    g = torch.Generator(device=DEV).manual_seed(2)
    for dtype in (torch.float32, torch.bfloat16):
        l = torch.randint(-2, 3, (257, 256), generator=g, device=DEV).to(dtype)
        _check(l, 8, exact_ids=True)
        _check(l, 8, exact_ids=True, score="sigmoid")
        _check(l, 8, exact_ids=True, groups=8, keep=4)
    l = torch.zeros(5, 64, device=DEV)
    l[1, ::2] = -0.0                       # minus zero is zero
    idx, w = api.moe_router_topk(l, 8)
    assert torch.equal(idx, torch.arange(8, device=DEV).expand(5, 8))
    assert torch.equal(w, torch.full((5, 8), 0.125, device=DEV))


def test_bf16_logits():
    l = _logits(100, 128, 4, torch.bfloat16)
    a = api.moe_router_topk(l, 8, score="sigmoid")
    b = api.moe_router_topk(l.float(), 8, score="sigmoid")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks(score):
    """-inf and NaN are never chosen; a row may have fewer than K left, or none;
    a whole group, or all but one of its experts, may be masked."""
    l = _logits(64, 64, 8)
    l[0] = float("-inf")
    l[1] = float("nan")
    l[2, 3:] = float("-inf")
    l[3, :60] = float("nan")
    l[4, 5] = float("inf")
    l[5, [7, 9]] = float("inf")
    l[6, 8:16] = float("-inf")
    l[7, 8:15] = float("-inf")
    l[8] = torch.finfo(torch.float32).min
    l[9, ::2] = torch.finfo(torch.float32).min
    l[10] *= 1000                            # scores that leave fp32's range
    l[11:40] = l[11:40].masked_fill(_logits(29, 64, 1) > 0, float("-inf"))
    # equal extremes: every id compared
    _check(l, 8, score=score, exact_ids=score == "softmax")
    _check(l, 8, score=score, groups=8, keep=4)
    bias = 0.1 * _logits(1, 64, 3)[0]
    rows = [r for r in range(64) if r not in (4, 5)]
    _check(l[rows], 8, score=score, bias=bias, groups=8, keep=4, top=2)
    idx, w = api.moe_router_topk(l, 8, score=score)
    assert (idx[:2] == -1).all() and not w[:2].any()
    assert (idx[2, 3:] == -1).all() and (idx[2, :3] >= 0).all()
    bias[:] = float("-inf")                   # nothing can be chosen
    idx, w = api.moe_router_topk(l, 8, score=score, bias=bias)
    assert (idx == -1).all() and not w.any()


def test_chosen_ids_feed_the_dispatch():
    """Padding tokens (all -inf) come out as the dispatch's padding routes."""
    l = _logits(100, 16, 3)
    l[10:20] = float("-inf")
    idx, w = api.moe_router_topk(l, 4)
    x = torch.randn(100, 128, device=DEV).to(torch.bfloat16)
    _, counts, src, st = api.moe_dispatch(x, idx, w, 16, 100)
    assert int(counts.sum()) == 90 * 4 and (src[10:20] == -1).all() and st.tolist() == [0, 0]


def test_no_rows_other_stream_and_graph():
    l = _logits(50, 64, 2)
    assert api.moe_router_topk(l[:0], 4)[0].shape == (0, 4)
    want = api.moe_router_topk(l, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.moe_router_topk(l, 4, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    idx, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.moe_router_topk(l, 4, topk_idx=idx, topk_w=w)
    l.copy_(l.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, want[0].flip(0)) and torch.equal(w, want[1].flip(0))


def test_refusals():
    l = _logits(4, 16, 0)
    f = api.moe_router_topk
    for bad in (dict(K=0), dict(K=17), dict(K=33), dict(K=4, groups=3), dict(K=4, groups=0),
                dict(K=4, groups=4, topk_groups=5), dict(K=4, groups=4, topk_groups=0),
                dict(K=9, groups=4, topk_groups=2), dict(K=4, group_top=3),
                dict(K=2, groups=16, topk_groups=4, group_top=2), dict(K=2, scale=float("nan"))):
        K = bad.pop("K")
        with pytest.raises(api.MoeError):
            f(l, K, topk_idx=torch.empty(4, K, dtype=torch.int64, device=DEV),
              topk_w=torch.empty(4, K, device=DEV), **bad)
    with pytest.raises(api.MoeError):
        f(torch.zeros(2, 1025, device=DEV), 4)
    with pytest.raises(ValueError):
        f(l, 4, score="tanh")
    with pytest.raises(TypeError):
        f(l.double(), 4)
    with pytest.raises(TypeError):
        f(l, 4, bias=torch.zeros(16, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        f(l, 4, bias=torch.zeros(15, device=DEV))
    with pytest.raises(TypeError):
        f(l, 4, idx_dtype=torch.int16)
    with pytest.raises(ValueError):
        f(l.t(), 4)
