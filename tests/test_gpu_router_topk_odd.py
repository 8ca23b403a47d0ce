"""moe_router_topk on rows that no vector load fits and on groups that do not
end with a lane's experts, BF16 and fp32 logits: both go through the warp's
shared memory.  Ids and weights against the definition in 64 bits, by the
checks of test_gpu_router_topk."""
import os
import re

import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api, build
from test_gpu_router_topk import _check, _logits

DEV = "cuda"


def test_shared_memory_is_read_by_all_before_it_is_written_again():
    """The group pass reads other lanes' values where the keys are then put:
    a warp barrier lies between (a shuffle orders no memory)."""
    with open(os.path.join(build.PKG_DIR, "csrc", "router.cu")) as f:
        src = f.read()
    after = src[src.index("best.add(values["):]
    assert re.match(r"best\.add\(values\[[^;]*;\s*__syncwarp\(\);", after)


@pytest.fixture
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K", [(70, 33, 5), (41, 61, 4), (40, 101, 6), (35, 141, 8), (30, 255, 8), (21, 333, 7),
                                   (17, 599, 16), (12, 1001, 9), (9, 1023, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_odd_rows(cuda, T, E, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(E)
    whole = torch.randint(-3, 4, (T, E), generator=g, device=DEV).to(dtype)   # ties: every id compared
    _check(whole, K, exact_ids=True)
    l = whole + 0.0
    l[::3, ::2] = float("-inf")
    l[1, 3:] = float("nan")
    l[2] = float("-inf")
    _check(l, K, exact_ids=True, renorm=False, scale=1.5)
    bias = 0.05 * _logits(1, E, 5)[0]
    a = api.moe_router_topk(_logits(T, E, E, dtype), K, score="sigmoid", bias=bias)
    b = api.moe_router_topk(_logits(T, E, E, dtype).float(), K, score="sigmoid", bias=bias)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _check(_logits(T, E, E + 1), K, score="sigmoid", bias=bias)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K,groups,keep", [(141, 6, 3, 2), (70, 4, 7, 3), (330, 5, 30, 7), (595, 8, 17, 9),
                                             (1023, 12, 31, 5), (30, 3, 10, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_groups_across_lanes(cuda, E, K, groups, keep, dtype):
    l = _logits(90, E, groups, dtype)
    l[3] = float("-inf")
    l[4, : E // groups] = float("nan")
    for top in (1, 2):
        if dtype == torch.float32:
            _check(l, K, score="sigmoid", bias=0.05 * _logits(1, E, 9)[0], groups=groups, keep=keep, top=top)
            _check(l, K, groups=groups, keep=keep, top=top, renorm=False)
        else:   # BF16 logits tie often: held to the same logits in fp32
            a = api.moe_router_topk(l, K, groups=groups, topk_groups=keep, group_top=top)
            b = api.moe_router_topk(l.float(), K, groups=groups, topk_groups=keep, group_top=top)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    want = api.moe_router_topk(l, K, groups=groups, topk_groups=keep, group_top=2)
    for _ in range(20):
        got = api.moe_router_topk(l, K, groups=groups, topk_groups=keep, group_top=2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
