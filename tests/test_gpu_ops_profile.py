"""What the launch-time profiler calls the kernels of the linear attention, verification and norms."""

import pytest
import torch

import gated_deltanet_03_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def names_of(call):
    gdn.gdn_profile_collect()
    gdn.gdn_profile_enable(True)
    try:
        call()
    finally:
        gdn.gdn_profile_enable(False)
    return {k: n for k, (n, _) in gdn.gdn_profile_collect().items()}


def linear(f, T):
    x = torch.randn(1, T, 1, 64, device=DEV).to(torch.bfloat16)
    return lambda: f(x, x, x, torch.zeros(1, device=DEV))


def test_names():
    assert names_of(linear(gdn.gdn_linear_prefill, 30)) == {"linear_chunk_kernel (whole)": 1}
    assert names_of(linear(gdn.gdn_linear_prefill, 2000)) == {"linear_chunk_kernel (state)": 1,
                                                              "linear_chunk_kernel (outputs)": 1}
    assert names_of(linear(gdn.gdn_linear_step, 2)) == {"linear_step_kernel": 1}
    for V, want in ((500, {"verify_row_kernel": 1}), (70000, {"verify_sum_kernel": 1, "verify_draw_kernel": 1})):
        p = torch.softmax(torch.randn(2, 3, V, device=DEV), -1)
        x, u = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.rand(2, 3, device=DEV)
        assert names_of(lambda: gdn.gdn_verify_drafts(p, None, x, u)) == want
    assert names_of(lambda: gdn.gdn_block_norm(torch.ones(2, 8, device=DEV))) == {"block_norm_kernel": 1}
