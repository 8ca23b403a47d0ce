"""The 4-bit products' way out of a wait that runs out, in the kernel itself: a
status, no fault, and a GPU that goes on."""
import ctypes

import pytest
import torch

from token_dispatch_grouped_topk_gb300 import _lib, api
from test_front_abi import FAKE, MIS
from test_gpu_fp4 import _layer

DEV = "cuda"


def test_bad_arguments_are_refused_on_the_host(lib):
    n = lib.moe_selftest_fp4_scratch_size()
    assert n % 16 == 0
    assert lib.moe_selftest_fp4_wait(None, n, FAKE, None) == -1
    assert lib.moe_selftest_fp4_wait(FAKE, n, None, None) == -1
    assert lib.moe_selftest_fp4_wait(MIS, n, FAKE, None) == -1
    assert lib.moe_selftest_fp4_wait(FAKE, n - 1, FAKE, None) == -3


@pytest.mark.gpu
def test_a_count_that_never_fills_ends_the_products_with_a_status():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = _lib.load()
    n = lib.moe_selftest_fp4_scratch_size()
    scratch = torch.empty(n, dtype=torch.uint8, device=DEV)
    st = torch.zeros(2, dtype=torch.int32, device=DEV)
    T, E, K, H, I = 500, 8, 4, 512, 256
    x, idx, p, w, gs = _layer(T, E, K, H, I, 2, "nvfp4")
    lane = api.MoeLayerBuffers(T, E, K, H, I, T, torch.device(DEV), packed=True, fp4="nvfp4", fp4_gscales=gs)
    want = lane.forward(x, idx, p, *w).clone()
    torch.cuda.synchronize()
    rc = lib.moe_selftest_fp4_wait(ctypes.c_void_p(scratch.data_ptr()), n, ctypes.c_void_p(st.data_ptr()),
                                   ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert st.tolist() == [api.DEV_TIMEOUT, 0]
    # what it held is free again: layers that take every SM run on, and report nothing
    for form in ("one", "two"):
        lane.gemm_launch = form
        for _ in range(3):
            lane.y.zero_()
            assert torch.equal(lane.forward(x, idx, p, *w), want) and lane.dev_status.tolist() == [0, 0]
