"""The operators around the routed branch, as cases to be timed and compared.

Five operators carry a token from the residual stream to its experts:

* ``norm``      -- residual addition, root-mean-square norm, and the normed row as BF16 and as
                   e4m3 codes with one fp32 scale per 128 elements;
* ``logits``    -- the router's projection, fp32 logits of BF16 rows and weights;
* ``topk``      -- the choice of experts from the logits: softmax or sigmoid scores, a bias that
                   enters the choice only, groups of experts, renormalised weights;
* ``dispatch``  -- the scatter of rows that are already in 8 bits to their experts' rows;
* ``experts4``  -- the gated-SiLU experts for a few tokens with 4-bit weights and a scale per
                   128 weights, combined with the router's weights.

``run`` computes them in plain torch operations in fp32, or, where ``own`` is true, by the
package's entry points.  ``exact`` restates them in 64 bits.
"""
import torch

own = False

GROUP = 128
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of the large layer being decoded: the latency of a single row
        dict(name="norm one token", op="norm", T=1, H=7168, residual="bf16", weight="bf16", quant=True),
        # the decode batch, residual stream kept in fp32
        dict(name="norm decode", op="norm", T=256, H=4096, residual="fp32", weight="fp32", quant=True),
        # the large layer's prompt
        dict(name="norm large", op="norm", T=16384, H=7168, residual="bf16", weight="bf16", quant=True),
        # the decode batch's router projection
        dict(name="logits decode", op="logits", T=256, E=64, H=4096),
        # the large layer's router projection
        dict(name="logits large", op="logits", T=16384, E=256, H=7168),
        # the decode batch's choice: softmax scores, no bias, renormalised
        dict(name="topk decode", op="topk", T=256, E=64, K=8, score="softmax", bias=False, groups=1,
             keep=1, top=1, renorm=True, bits=16, ids=64, masked=0.0),
        # an odd number of experts and tokens, groups by their best expert, some padding tokens
        dict(name="topk ragged", op="topk", T=3001, E=60, K=6, score="softmax", bias=False, groups=6,
             keep=3, top=1, renorm=False, bits=32, ids=32, masked=0.05),
        # the large layer's choice: sigmoid scores, balance bias, 4 of 8 groups by their best two
        dict(name="topk large", op="topk", T=16384, E=256, K=8, score="sigmoid", bias=True, groups=8,
             keep=4, top=2, renorm=True, bits=32, ids=64, masked=0.0),
        # the decode batch's rows to their experts, some padding routes
        dict(name="dispatch decode", op="dispatch", T=256, E=64, K=8, H=4096, R=256, skew=0.0, pad=0.02),
        # the skewed prompt of the prefill layer, packed rows, with capacity drops
        dict(name="dispatch prefill", op="dispatch", T=4096, E=128, K=8, H=4096, R=2048, skew=1.1, pad=0.0),
        # one token of the large layer: eight experts' weights are read once
        dict(name="experts4 one token", op="experts4", T=1, E=256, K=8, H=7168, I=2048, pad=0.0),
        # a small decode batch of the decode layer: most experts are active with a few tokens each
        dict(name="experts4 batch", op="experts4", T=48, E=64, K=8, H=4096, I=1536, pad=0.02),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


# hidden sizes in units of 128, about even over the logarithm
_H = (1, 2, 3, 4, 5, 7, 8, 11, 13, 16, 20, 27, 32, 40, 45, 56, 64, 81, 96, 128)


def _hidden(rng, lo, hi):
    return 128 * rng.choice([h for h in _H if lo <= h <= hi])


def draw(rng):
    op = rng.choice(["norm", "logits", "topk", "dispatch", "experts4"])
    if op == "norm":
        # rows up to the largest listed case's bytes (13 bytes an element at most, against its 9)
        H = _hidden(rng, 1, 128)
        T = _log_int(rng, 1, min(65536, 16384 * 7168 * 9 // (13 * H)))
        return dict(op=op, T=T, H=H, residual=rng.choice(["none", "bf16", "fp32"]),
                    weight=rng.choice(["bf16", "fp32"]), quant=rng.random() < 0.7)
    if op == "logits":
        H = _hidden(rng, 1, 64)
        E = _log_int(rng, 8, 512)
        T = _log_int(rng, 1, max(1, min(32768, 16384 * 256 * 7168 // (max(E, 256) * H))))
        return dict(op=op, T=T, E=E, H=H)
    if op == "topk":
        groups = rng.choice([1, 1, 2, 4, 6, 8])
        E = groups * _log_int(rng, 4, 1024 // groups)
        keep = rng.randint(1, groups)
        K = _log_int(rng, 1, min(16, keep * (E // groups)))
        T = _log_int(rng, 1, min(32768, 16384 * 256 // max(E, 256) * 2))
        sig = rng.random() < 0.5
        return dict(op=op, T=T, E=E, K=K, score="sigmoid" if sig else "softmax",
                    bias=sig and rng.random() < 0.7, groups=groups, keep=keep,
                    top=rng.choice([1, 2]), renorm=rng.random() < 0.6, bits=rng.choice([16, 32]),
                    ids=rng.choice([32, 64]), masked=rng.choice([0.0, 0.1]))
    if op == "dispatch":
        H = _hidden(rng, 1, 56)
        E = _log_int(rng, 8, 256)
        K = rng.randint(1, 8)
        T = _log_int(rng, 1, max(1, min(8192, 4096 * 8 * 4096 // (K * H))))
        return dict(op=op, T=T, E=E, K=K, H=H, R=max(1, int(T * K / E * rng.choice([0.7, 2.0, 8.0]))),
                    skew=rng.choice([0.0, 1.1]), pad=rng.choice([0.0, 0.1]))
    E = _log_int(rng, 8, 64)
    return dict(op=op, T=_log_int(rng, 1, 48), E=E, K=rng.randint(1, 8), H=_hidden(rng, 2, 32),
                I=128 * _log_int(rng, 1, 12), pad=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _routes(c, g):
    """Router ids [T, K] (distinct per token, -1 = padding) and weights."""
    logits = _randn(g, c["T"], c["E"])
    if c.get("skew"):
        logits -= c["skew"] * torch.log(torch.arange(1, c["E"] + 1, device=DEV, dtype=torch.float32))
    v, idx = torch.topk(logits, c["K"], dim=1)
    if c["pad"]:
        idx = idx.masked_fill(torch.rand(idx.shape, generator=g, device=DEV) < c["pad"], -1)
    return idx.contiguous(), torch.softmax(v, dim=1).contiguous()


def _weights4(g, E, N, K):
    """Weights ~ N(0, 0.02) [E, N, K] in 4 bits: two's offset codes (value = code - 8) times a
    BF16 scale per 128 along K; two codes a byte, the even element in the low four bits."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // GROUP, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w = _randn(g, N, K // GROUP, GROUP).mul_(0.02)
        s = (w.abs().amax(dim=2) / 7.0).to(torch.bfloat16)
        q = w.div_(s.float()[..., None]).round_().clamp_(-8, 7).add_(8).to(torch.uint8).view(N, K)
        codes[e] = q[:, 0::2] | (q[:, 1::2] << 4)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    if op == "norm":
        T, H = c["T"], c["H"]
        res = None
        if c["residual"] != "none":
            res = (4.0 * _randn(g, T, H)).to(torch.float32 if c["residual"] == "fp32" else torch.bfloat16)
        w = (1.0 + 0.1 * _randn(g, H)).to(torch.float32 if c["weight"] == "fp32" else torch.bfloat16)
        s = dict(x=_randn(g, T, H).to(torch.bfloat16), residual=res, weight=w, eps=1e-6, quant=c["quant"],
                 y=torch.empty(T, H, dtype=torch.bfloat16, device=DEV), yq=None, ys=None,
                 residual_out=None if res is None else torch.empty_like(res))
        if c["quant"]:
            s["yq"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
            s["ys"] = torch.empty(T, H // GROUP, dtype=torch.float32, device=DEV)
    elif op == "logits":
        s = dict(x=_randn(g, c["T"], c["H"]).to(torch.bfloat16),
                 w=(_randn(g, c["E"], c["H"]) * c["H"] ** -0.5).to(torch.bfloat16),
                 out=torch.empty(c["T"], c["E"], dtype=torch.float32, device=DEV))
    elif op == "topk":
        T, E = c["T"], c["E"]
        logits = _randn(g, T, E).to(torch.bfloat16 if c["bits"] == 16 else torch.float32)
        if c["masked"]:   # padding tokens: nothing to choose from
            rows = torch.rand(T, generator=g, device=DEV) < c["masked"]
            logits.masked_fill_(rows[:, None], float("-inf"))
        # the balance bias moves in steps of 0.001 up or down
        bias = (_randn(g, E) * 20).round_() * 0.001 if c["bias"] else None
        s = dict(c=c, logits=logits, bias=bias, scale=2.5 if c["renorm"] else 1.0,
                 idx=torch.empty(T, c["K"], dtype=torch.int64 if c["ids"] == 64 else torch.int32, device=DEV),
                 w=torch.empty(T, c["K"], dtype=torch.float32, device=DEV))
    elif op == "dispatch":
        T, K, E, H, R = c["T"], c["K"], c["E"], c["H"], c["R"]
        x = _randn(g, T, H // GROUP, GROUP)
        sc = x.abs().amax(dim=2) / 448.0
        idx, w = _routes(c, g)
        rows = max(1, min(T * K, E * R))
        s = dict(c=c, xq=(x / sc[..., None]).to(torch.float8_e4m3fn).view(T, H), xs=sc, idx=idx, w=w,
                 rows=rows,   # one row more than is returned: the plain form's place for dropped routes
                 oq=torch.zeros(rows + 1, H, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                 os=torch.zeros(rows + 1, H // GROUP, dtype=torch.float32, device=DEV),
                 counts=torch.empty(E, dtype=torch.int32, device=DEV),
                 src_map=torch.empty(T, K, dtype=torch.int32, device=DEV),
                 status=torch.empty(2, dtype=torch.int32, device=DEV), ws=None)
    else:
        E, H, I = c["E"], c["H"], c["I"]
        w13, s13 = _weights4(g, E, 2 * I, H)
        w2, s2 = _weights4(g, E, H, I)
        idx, w = _routes(c, g)
        s = dict(c=c, x=_randn(g, c["T"], H).to(torch.bfloat16), idx=idx, w=w, w13=w13, s13=s13, w2=w2,
                 s2=s2, y=torch.empty(c["T"], H, dtype=torch.bfloat16, device=DEV),
                 status=torch.zeros(2, dtype=torch.int32, device=DEV), ws=None)
    s["op"] = op
    return s


# ------------------------------------------------------- the plain form, fp32

def _norm(s):
    r = s["x"].float()
    out = {}
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out["residual"] = r.to(s["residual"].dtype)
    n = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"].float()
    out["y"] = n.to(torch.bfloat16)
    if s["quant"]:
        grp = n.view(n.shape[0], -1, GROUP)
        amax = grp.abs().amax(dim=2).clamp_min(1e-4)
        out["yq"] = (grp * (448.0 / amax)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(n.shape)
        out["ys"] = amax / 448.0
    return out


def _scores(logits, score):
    """Scores and, for softmax, the exponentials before the division."""
    if score == "sigmoid":
        e = 1.0 / (1.0 + torch.exp(-logits))
        return e, e
    m = logits.amax(dim=1, keepdim=True)
    e = torch.where(logits == m, 1.0, torch.exp(logits - m))
    e = e.masked_fill(logits == float("-inf"), 0.0)
    return e / e.sum(dim=1, keepdim=True).clamp_min(1e-30), e


def _topk(logits, bias, scale, c):
    ninf = float("-inf")
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    masked = logits == ninf
    s, e = _scores(logits, c["score"])
    # without a bias the scores rise with the logits, which choose exactly
    key = logits if bias is None else (s + bias).masked_fill(masked, ninf)
    if G > 1:
        if c["top"] == 1:
            gs = key.view(T, G, -1).amax(dim=2)
        else:
            val = (e if bias is None else s + bias).masked_fill(masked, ninf).view(T, G, -1)
            best = torch.topk(val, 2, dim=2).values
            gs = torch.where(best[..., 1] == ninf, best[..., 0], best[..., 0] + best[..., 1])
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, order, True)
        key = key.view(T, G, -1).masked_fill(~kept[..., None], ninf).view(T, E)
    v, idx = torch.sort(key, dim=1, descending=True, stable=True)
    v, idx = v[:, :K], idx[:, :K]
    none = v == ninf
    w = s.gather(1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-20)
    return idx.masked_fill(none, -1), w * scale


def _dispatch(s):
    c, rows = s["c"], s["rows"]
    T, K, E, R = c["T"], c["K"], c["E"], c["R"]
    flat = s["idx"].reshape(-1)
    hot = (flat[:, None] == torch.arange(E, device=flat.device)).to(torch.int32)
    slot = (torch.cumsum(hot, 0, dtype=torch.int32) * hot).sum(dim=1) - 1
    total = hot.sum(dim=0)
    counts = total.clamp_max(R)
    base = torch.cumsum(counts, 0) - counts
    kept = (flat >= 0) & (slot < R)
    q = torch.where(kept, base[flat.clamp_min(0)] + slot, -1)
    to = torch.where(kept, q, rows)   # dropped routes go to the spare row
    t = torch.arange(T * K, device=flat.device) // K
    s["oq"].view(torch.uint8)[to] = s["xq"].view(torch.uint8)[t]
    s["os"][to] = s["xs"][t]
    return dict(xq=s["oq"][:rows], xs=s["os"][:rows], counts=counts.to(torch.int32),
                src_map=q.view(T, K).to(torch.int32), dropped=(total - counts).sum().to(torch.int32))


def _wide(codes, scales, dtype):
    """4-bit codes [..., N, K/2] and scales [..., N, K/128] to weights [..., N, K]."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    w = q.to(dtype).sub_(8).unflatten(-1, (-1, GROUP))
    return w.mul_(scales.to(dtype)[..., None]).flatten(-2)


def _experts4(s):
    c = s["c"]
    T, K, E, I = c["T"], c["K"], c["E"], c["I"]
    idx, w, x = s["idx"], s["w"].masked_fill(s["idx"] < 0, 0.0), s["x"].float()
    if T * K < E:   # few routes: the weights of each route's expert
        f = idx.clamp_min(0).reshape(-1)
        h = torch.matmul(_wide(s["w13"][f], s["s13"][f], torch.float32),
                         x.repeat_interleave(K, 0)[..., None])[..., 0]
        z = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
        o = torch.matmul(_wide(s["w2"][f], s["s2"][f], torch.float32), z[..., None])[..., 0]
        return (o.view(T, K, -1) * w[..., None]).sum(dim=1).to(torch.bfloat16)
    h = torch.matmul(x, _wide(s["w13"], s["s13"], torch.float32).transpose(1, 2))   # [E, T, 2I]
    z = h[..., :I] / (1.0 + torch.exp(-h[..., :I])) * h[..., I:]
    o = torch.matmul(z, _wide(s["w2"], s["s2"], torch.float32).transpose(1, 2))
    per = torch.zeros(T, E, device=x.device).scatter_add_(1, idx.clamp_min(0), w)
    return (o * per.t()[..., None]).sum(dim=0).to(torch.bfloat16)


# ------------------------------------------------------------------- passes

def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "norm":
        return _norm(s)
    if op == "logits":
        return torch.matmul(s["x"].float(), s["w"].float().t())
    if op == "topk":
        idx, w = _topk(s["logits"].float(), s["bias"], s["scale"], s["c"])
        return dict(idx=idx.to(s["idx"].dtype), w=w)
    if op == "dispatch":
        return _dispatch(s)
    return _experts4(s)


def _run_own(s):
    from token_dispatch_grouped_topk_gb300 import api
    op = s["op"]
    if op == "norm":
        api.moe_add_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"],
                             residual_out=s["residual_out"], y=s["y"], yq=s["yq"], ys=s["ys"])
        out = dict(y=s["y"])
        if s["residual"] is not None:
            out["residual"] = s["residual_out"]
        if s["quant"]:
            out["yq"], out["ys"] = s["yq"], s["ys"]
        return out
    if op == "logits":
        return api.moe_router_logits(s["x"], s["w"], logits=s["out"])
    c = s["c"]
    if op == "topk":
        idx, w = api.moe_router_topk(s["logits"], c["K"], score=c["score"], bias=s["bias"],
                                     groups=c["groups"], topk_groups=c["keep"], group_top=c["top"],
                                     renormalize=c["renorm"], scale=s["scale"], topk_idx=s["idx"],
                                     topk_w=s["w"])
        return dict(idx=idx, w=w)
    if op == "dispatch":
        if s["ws"] is None:   # a lane's workspace, kept between its calls
            s["ws"] = torch.empty(api.dispatch_workspace_size(c["T"], c["K"], c["E"]),
                                  dtype=torch.uint8, device=DEV)
        rows = s["rows"]
        api.moe_dispatch_fp8(s["xq"], s["xs"], s["idx"], c["E"], c["R"], rows=rows, xq=s["oq"][:rows],
                             xs=s["os"][:rows], counts=s["counts"], src_map=s["src_map"],
                             dev_status=s["status"], workspace=s["ws"])
        return dict(xq=s["oq"][:rows], xs=s["os"][:rows], counts=s["counts"], src_map=s["src_map"],
                    dropped=s["status"][1])
    if s["ws"] is None:
        s["ws"] = torch.empty(api.experts_w4_workspace_size(c["T"], c["K"], c["H"], c["I"]),
                              dtype=torch.uint8, device=DEV)
    return api.moe_experts_w4(s["x"], s["idx"], s["w"], s["w13"], s["s13"], s["w2"], s["s2"],
                              y=s["y"], dev_status=s["status"], workspace=s["ws"])


# --------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    T = c["T"]
    if op == "norm":
        H, res = c["H"], {"none": 0, "bf16": 2, "fp32": 4}[c["residual"]]
        per = 4 + 2 * res + ((1 + 4 / GROUP) if c["quant"] else 0)
        return {"bytes": T * H * per + H * (4 if c["weight"] == "fp32" else 2), "flops": 8 * T * H}
    if op == "logits":
        E, H = c["E"], c["H"]
        return {"bytes": 2 * T * H + 2 * E * H + 4 * T * E, "flops": 2 * T * E * H}
    K = c["K"]
    if op == "topk":
        return {"bytes": T * c["E"] * c["bits"] / 8 + T * K * (4 + c["ids"] / 8) + 4 * c["E"] * c["bias"],
                "flops": 10 * T * c["E"]}
    if op == "dispatch":
        E, R = c["E"], c["R"]
        kept = min(T * K * (1 - c["pad"]), E * R)
        if c["skew"]:   # the popular experts overflow their rows
            p = [(e + 1) ** -c["skew"] for e in range(E)]
            kept = sum(min(R, T, T * K * (1 - c["pad"]) * v / sum(p)) for v in p)
        row = c["H"] + 4 * c["H"] // GROUP
        return {"bytes": T * row + kept * row + T * K * 12 + 4 * E, "flops": 0}
    E, H, I = c["E"], c["H"], c["I"]
    routes = T * K * (1 - c["pad"])
    # the experts that some route takes, each read once
    active = E * (1 - (1 - K * (1 - c["pad"]) / E) ** T)
    return {"bytes": active * 3 * H * I * (0.5 + 2 / GROUP) + 4 * T * H + T * K * 12,
            "flops": 6 * routes * H * I}


# ------------------------------------------------------------- in 64 bits

def _exact_topk(l, bias, scale, c):
    """The chosen experts' weights by the definition, token after token in numpy."""
    import numpy as np
    l = l.double().cpu().numpy()
    b = np.zeros(c["E"]) if bias is None else bias.double().cpu().numpy()
    size = c["E"] // c["groups"]
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max(axis=1, keepdims=True))
            s = s / s.sum(axis=1, keepdims=True)
    key = np.where(np.isneginf(l), -np.inf, s + b)
    w = np.zeros((c["T"], c["K"]))
    for t in range(c["T"]):
        if np.isneginf(l[t]).all():
            continue
        k = key[t]
        if c["groups"] > 1:
            part = -np.sort(-k.reshape(c["groups"], size), axis=1)[:, :c["top"]]
            keep = np.argsort(-part.sum(axis=1), kind="stable")[:c["keep"]]
            only = np.full(c["E"], -np.inf)
            for g in keep:
                only[g * size:(g + 1) * size] = k[g * size:(g + 1) * size]
            k = only
        w[t] = s[t, np.argsort(-k, kind="stable")[:c["K"]]]
    if c["renorm"]:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-20)
    return w * scale


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "dispatch":
        return None   # copies and whole numbers only
    if op == "norm":
        T, H = s["x"].shape
        r = s["x"].double()
        out = {}
        if s["residual"] is not None:
            r += s["residual"]
            out["residual"] = r.clone()
        r *= (r.pow(2).sum(dim=1, keepdim=True) / H + s["eps"]).pow(-0.5)
        r *= s["weight"].double()
        out["y"] = r
        if s["quant"]:
            top = r.view(T, -1, GROUP).abs().amax(dim=2, keepdim=True).clamp_min(1e-4)
            out["yq"] = (r.view(T, -1, GROUP) * 448.0 / top).view(T, H)
            out["ys"] = top[..., 0] / 448.0
        return out
    if op == "logits":
        if 2.0 * case["T"] * case["E"] * case["H"] > 2e12:
            return None
        return torch.nn.functional.linear(s["x"].double(), s["w"].double())
    if op == "topk":
        return dict(idx=None, w=_exact_topk(s["logits"], s["bias"], s["scale"], case))
    y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
    I = case["I"]
    for e in torch.unique(s["idx"]).tolist():
        if e < 0:
            continue
        t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
        h = s["x"][t].double() @ _wide(s["w13"][e], s["s13"][e], torch.float64).t()
        z = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        o = z @ _wide(s["w2"][e], s["s2"][e], torch.float64).t()
        y.index_add_(0, t, o * s["w"][t, k].double()[:, None])
    return y
