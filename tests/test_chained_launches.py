"""The e4m3 dispatch above 4096 routes is a chain of launches that overlap: its
scatter may start while the scan still writes the block bases and the counts.
The read-only path may not be used for them (no const __restrict__, which lets
a compiler take it), and they are read from L2, after the wait."""
import os
import re

import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api, build

DEV = "cuda"


def test_what_the_chain_writes_is_not_read_through_the_read_only_path():
    with open(os.path.join(build.PKG_DIR, "csrc", "dispatch.cu")) as f:
        src = f.read()
    start = src.index("route_scatter_codes_kernel(")
    params, body = src[start:src.index("{", start)], src[src.index("{", start):]
    body = body[:body.index("\n}\n")]
    for name in ("base", "counts"):
        decl = re.search(r"[^,(]*\b%s\b" % name, params).group(0)
        assert "int32_t*" in decl and "__restrict__" not in decl, decl
        # every read goes to L2 (the one-launch form only writes counts)
        assert "__ldcg(%s + " % name in body and not re.search(r"\b%s\[" % name, body)
        assert body.index("chain_wait()") < body.index("__ldcg(%s + " % name)
    assert "expert_prefix(counts" not in body


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,H,packed", [
    (1700, 256, 8, 128, True), (1500, 96, 6, 256, False), (5000, 1024, 2, 128, True), (4097, 8, 1, 384, False)])
def test_changing_routes_on_one_workspace(T, E, K, H, packed):
    """Routes that change from call to call, with rows of block counts that end
    inside a cache line: slots, counts and rows of the quantising dispatch,
    whose launches do not overlap."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    tq, ts = (t[0] for t in api.moe_quantize_fp8(x[None], n))
    R = max(1, T * K // E)
    rows = api.packed_rows(T, K, E, R) if packed else 0
    lead = (rows,) if packed else (E, R)
    ws = torch.empty(api.dispatch_workspace_size(T, K, E), dtype=torch.uint8, device=DEV)
    out = dict(xq=torch.zeros(*lead, H, dtype=torch.uint8, device=DEV), xs=torch.zeros(*lead, H // 128, device=DEV),
               counts=torch.empty(E, dtype=torch.int32, device=DEV),
               src_map=torch.empty(T, K, dtype=torch.int32, device=DEV),
               dev_status=torch.empty(2, dtype=torch.int32, device=DEV), workspace=ws, rows=rows)
    for i in range(12):
        l = torch.randn(T, E, generator=g, device=DEV)
        l[:, i % E] += 2.0
        idx = torch.topk(l, K, dim=1).indices
        ref = {k: torch.zeros_like(v) if torch.is_tensor(v) else v for k, v in out.items()}
        api.moe_dispatch_quant(x, idx, None, E, R, **ref)
        for t in (out["xq"], out["xs"]):
            t.zero_()
        api.moe_dispatch_fp8(tq, ts, idx, E, R, **out)
        for k in ("xq", "xs", "counts", "src_map", "dev_status"):
            assert torch.equal(out[k], ref[k]), (i, k)
