"""The order of the operators in front of the layer and of the 4-bit experts
within a stream: inputs written by the kernel just before a call, buffers
overwritten just after it, again and again, with the same bits as a call on
inputs at rest.  Their launches overlap, so a wait that is missing shows here."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api
from test_gpu_experts_w4 import _weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _alternate(inputs, call, scratch=()):
    """``call(buffers)`` on two sets of inputs in turn, each copied into the
    same buffers right before it, behind a kernel that keeps the GPU busy."""
    buffers = [t.clone() for t in inputs[0]]
    want = []
    for s in inputs:
        for b, t in zip(buffers, s):
            b.copy_(t)
        torch.cuda.synchronize()
        want.append([o.clone() for o in call(buffers)])
        torch.cuda.synchronize()
    a = torch.randn(1024, 1024, device=DEV)
    results = []
    for i in range(40):
        a = torch.tanh(a @ a)
        for b, t in zip(buffers, inputs[i & 1]):
            b.copy_(t)
        results.append([o.clone() for o in call(buffers)])
        for s in scratch:
            s.fill_(0xFF if i & 2 else 0x7E)
    for i, got in enumerate(results):
        assert all(torch.equal(g, w) for g, w in zip(got, want[i & 1])), i


def _rows(T, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)


def _ids(T, E, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.topk(torch.randn(T, E, generator=g, device=DEV), K, dim=1).indices


@pytest.mark.parametrize("T,E,K,H,I", [(1, 8, 2, 8192, 512), (6, 16, 4, 1024, 256), (48, 16, 4, 2048, 768)])
def test_experts_w4(T, E, K, H, I):
    g = torch.Generator(device=DEV).manual_seed(1)
    weights = (*_weights(g, E, 2 * I, H), *_weights(g, E, H, I))
    ws = torch.empty(api.experts_w4_workspace_size(T, K, H, I), dtype=torch.uint8, device=DEV)
    sets = [(_rows(T, H, s), _ids(T, E, K, s), torch.rand(T, K, generator=g, device=DEV)) for s in (2, 3)]
    _alternate(sets, lambda b: (api.moe_experts_w4(*b, *weights, workspace=ws),), (ws,))


@pytest.mark.parametrize("T,E,K,H", [(1, 8, 2, 256), (200, 64, 8, 2048), (1500, 64, 8, 1024), (3000, 16, 2, 512)])
def test_dispatch_fp8(T, E, K, H):
    ws = torch.empty(api.dispatch_workspace_size(T, K, E), dtype=torch.uint8, device=DEV)
    rows = api.packed_rows(T, K, E, T)
    xq = torch.zeros(rows, H, dtype=torch.uint8, device=DEV)
    xs = torch.zeros(rows, H // 128, device=DEV)
    sets = []
    for s in (4, 5):
        g = torch.Generator(device=DEV).manual_seed(s)
        sets.append((torch.randint(0, 120, (T, H), generator=g, device=DEV).to(torch.uint8),
                     torch.rand(T, H // 128, generator=g, device=DEV), _ids(T, E, K, s)))
    _alternate(sets, lambda b: api.moe_dispatch_fp8(*b, E, T, rows=rows, xq=xq, xs=xs, workspace=ws), (ws,))


@pytest.mark.parametrize("T,E,H", [(1, 64, 4096), (256, 64, 4096), (1024, 64, 2048), (900, 256, 7168), (9000, 96, 512)])
def test_router_logits(T, E, H):
    w = (_rows(E, H, 6).float() / H ** 0.5).to(torch.bfloat16)
    out = torch.empty(T, E, device=DEV)
    _alternate([(_rows(T, H, s),) for s in (7, 8)], lambda b: (api.moe_router_logits(*b, w, logits=out),))


def test_norm_and_choice():
    w = _rows(1, 1024, 9)[0]
    sets = [(_rows(300, 1024, s), torch.randn(300, 60, device=DEV)) for s in (10, 11)]

    def call(b):
        y, yq, ys, _ = api.moe_add_rms_norm(b[0], w, 1e-6, quant=True)
        return (y, yq, ys, *api.moe_router_topk(b[1], 6, score="sigmoid", groups=6, topk_groups=3, group_top=2))

    _alternate(sets, call)
