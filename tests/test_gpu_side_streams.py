"""Calls on a stream that is not the current one, with the tensors that a call
allocates itself: their memory goes to no one before the call's kernels have
ended, nor before the current stream has read the outputs."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import _lib, api
from test_gpu_experts_w4 import _case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class _Recorder:
    """The library, with the arguments of its calls kept."""

    def __init__(self, lib):
        self.lib, self.args = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*a):
            self.args += a
            return fn(*a)
        return call


def _calls():
    """name -> (call(stream) -> its outputs, the inputs' tensors)."""
    g = torch.Generator(device=DEV).manual_seed(1)
    E, K, H, I, T = 8, 2, 1024, 512, 900
    w4 = _case(6, E, K, H, I, 2)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    r = torch.randn(T, H, generator=g, device=DEV)
    nw = torch.ones(H, device=DEV)
    rw = (torch.randn(E, H, generator=g, device=DEV) / 32).to(torch.bfloat16)
    lg = torch.randn(T, 64, generator=g, device=DEV)
    idx = torch.topk(torch.randn(T, 64, generator=g, device=DEV), 8, dim=1).indices
    tw = torch.rand(T, 8, generator=g, device=DEV)
    tw2 = tw[:50, :2].contiguous()
    tq = torch.randint(0, 120, (T, H), generator=g, device=DEV).to(torch.uint8)
    ts = torch.rand(T, H // 128, generator=g, device=DEV)
    recv = torch.randn(4, 64, 256, generator=g, device=DEV).to(torch.bfloat16)
    counts = torch.tensor([64, 0, 3, 30], dtype=torch.int32, device=DEV)
    f8 = lambda *s: torch.randint(0, 100, s, generator=g, device=DEV).to(torch.uint8)
    mlp = (f8(4, 512, 256), torch.rand(4, 4, 2, generator=g, device=DEV),
           f8(4, 256, 256), torch.rand(4, 2, 2, generator=g, device=DEV))
    src = torch.randint(0, 256, (50, 2), generator=g, device=DEV).to(torch.int32)
    return {
        "moe_experts_w4": (lambda s: (api.moe_experts_w4(*w4, stream=s),), w4),
        "moe_dispatch_fp8": (lambda s: api.moe_dispatch_fp8(tq, ts, idx, 64, 120, stream=s), (tq, ts, idx)),
        "moe_add_rms_norm": (lambda s: api.moe_add_rms_norm(x, nw, residual=r, quant=True, stream=s), (x, nw, r)),
        "moe_router_logits": (lambda s: (api.moe_router_logits(x, rw, stream=s),), (x, rw)),
        "moe_router_topk": (lambda s: api.moe_router_topk(lg, 6, stream=s), (lg,)),
        "moe_dispatch_quant": (lambda s: api.moe_dispatch_quant(x, idx, tw, 64, 120, stream=s), (x, idx, tw)),
        "moe_expert_compute": (lambda s: (api.moe_expert_compute(recv, counts, *mlp, stream=s),),
                               (recv, counts, *mlp)),
        "moe_combine": (lambda s: (api.moe_combine(recv, src, tw2, stream=s),), (recv, src, tw2)),
    }


def _spans(tensors):
    return [(t.data_ptr(), t.numel() * t.element_size()) for t in tensors if torch.is_tensor(t)]


@pytest.mark.parametrize("name", ["moe_experts_w4", "moe_dispatch_fp8", "moe_add_rms_norm", "moe_router_logits",
                                  "moe_router_topk", "moe_dispatch_quant", "moe_expert_compute", "moe_combine"])
def test_memory_of_a_call_stays_its_own(name, monkeypatch):
    """While the side stream waits, all that the call allocated is dropped and
    tensors of every size are taken on the current stream: none lies on it."""
    call, inputs = _calls()[name]
    call(None)
    torch.cuda.synchronize()
    rec = _Recorder(_lib.load())
    monkeypatch.setattr(api._lib, "load", lambda *a: rec)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)          # some 20 ms
    del rec.args[:]
    outs = call(s)
    sizes = {n for _, n in _spans(outs)}
    mine = {int(a) for a in rec.args if isinstance(a, int) and a > 1 << 32}
    mine -= {p for p, _ in _spans(inputs)} | {s.cuda_stream}
    assert mine >= {p for p, _ in _spans(outs)}
    del outs
    # sizes of outputs, of workspaces and of everything between
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV)
            for n in sorted(sizes | {1 << k for k in range(8, 25)} | {256 * 3, (1 << 20) + 512}) for _ in range(3)]
    for p in mine:
        for base, n in _spans(junk):
            assert not base <= p < base + n, (name, hex(p), n)
    s.synchronize()


def test_results_while_the_current_stream_fills_new_memory():
    """The 4-bit experts' scratch holds counters and sums: calls on a side
    stream keep their bits while the current stream writes all over memory."""
    args = _case(12, 16, 4, 2048, 512, 7)
    want = api.moe_experts_w4(*args)
    n = api.experts_w4_workspace_size(12, 4, 2048, 512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(40):
        outs.append(api.moe_experts_w4(*args, stream=s))
        for m in (n, 2 * want.numel(), 256):
            torch.empty(m, dtype=torch.uint8, device=DEV).fill_(0x7E if i & 1 else 0xFF)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(y, want) for y in outs)


def test_an_output_dropped_while_the_current_stream_reads_it():
    """A call on the side stream does not write into an output that was dropped
    while the current stream still had it to read."""
    a = _case(12, 16, 4, 2048, 512, 7)
    b = (*_case(12, 16, 4, 2048, 512, 8)[:3], *a[3:])
    want = api.moe_experts_w4(*a)
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    s.wait_stream(cur)
    y = api.moe_experts_w4(*a, stream=s)
    cur.wait_stream(s)
    torch.cuda._sleep(40_000_000)
    got = y.clone()
    at = y.data_ptr()
    del y
    others = [api.moe_experts_w4(*b, stream=s) for _ in range(8)]
    assert at not in {o.data_ptr() for o in others}
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_statuses_start_at_zero_on_the_side_stream():
    """A status that the call makes itself is cleared where its kernels run."""
    g = torch.Generator(device=DEV).manual_seed(3)
    tq, ts = torch.zeros(40, 256, dtype=torch.uint8, device=DEV), torch.zeros(40, 2, device=DEV)
    idx = torch.randint(0, 4, (40, 1), generator=g, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    status = api.moe_dispatch_fp8(tq, ts, idx, 4, 3, stream=s)[4]
    s.synchronize()
    counts = torch.bincount(idx.flatten(), minlength=4)
    assert status.tolist() == [api.DEV_CAPACITY_DROPPED, int((counts - 3).clamp_min(0).sum())]
