"""The launch form that moe_layer_fp4 chooses follows from the work, not from the
room of the buffers: padded and packed lanes of one routing choose the same."""
import pytest
import torch

from token_dispatch_grouped_topk_gb300 import api
from test_gpu_fp4 import _layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _one_launch(lane, *args):
    """Whether the layer runs both products in one launch: only then are the
    launch's counters, behind the dispatch's part of the workspace, written."""
    at = api.dispatch_workspace_size(lane.T, lane.K, lane.E)
    lane.ws_dispatch[at:].fill_(0xFF)
    lane.forward(*args)
    return bool((lane.ws_dispatch[at:at + 4] != 0xFF).any())


@pytest.mark.parametrize("T,E,K,H,I,R,form", [
    (1009, 60, 6, 128, 640, 1009, None), (600, 64, 8, 128, 1536, 600, None), (1, 256, 8, 128, 2048, 1, True),
    (256, 64, 8, 256, 1536, 2048, True), (4096, 64, 8, 128, 2048, 4096, False),
    (256, 1024, 4, 128, 1024, 32, False)])
def test_both_layouts_choose_the_same_form(T, E, K, H, I, R, form):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x, idx, p, w, gs = _layer(T, E, K, H, I, 3, "nvfp4", pad=0.0)
    lanes = [api.MoeLayerBuffers(T, E, K, H, I, R, torch.device(DEV), packed=packed, fp4="nvfp4",
                                 fp4_gscales=gs) for packed in (False, True)]
    got = [_one_launch(lane, x, idx, p, *w) for lane in lanes]
    assert got[0] == got[1]
    assert form is None or got[0] == form
    assert torch.equal(lanes[0].y, lanes[1].y)
    # forced forms are what they say
    for lane in lanes:
        for name, one in (("one", True), ("two", False)):
            lane.gemm_launch = name
            assert _one_launch(lane, x, idx, p, *w) == one
