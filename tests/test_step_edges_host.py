"""Host side of the operators of include/sbp_step.h and of the paths that use them, at its edges:
nothing here reaches a kernel, so no GPU is needed."""
import pytest
import torch

from memory_efficient_exact_chunk_b200 import build as sbp_build
from memory_efficient_exact_chunk_b200 import sbp, stack


@pytest.fixture(scope="module")
def lib():
    sbp_build.build()
    return sbp.load()


# --------------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("head_dim,dtype", [(64, sbp.SBP_BF16), (128, sbp.SBP_BF16),
                                            (16, sbp.SBP_F32)])
def test_a_stack_of_both_kinds_of_layers_gets_the_larger_workspace(lib, head_dim, dtype):
    """Neither kind needs the larger workspace in every configuration."""
    cfg = sbp.layer_cfg(1, 4096, 128, 4, 2, head_dim, 256, 1e-6, 1e4, dtype, 2)
    normed = {n: torch.ones(head_dim) for n in sbp.QK_NORM_FIELDS}
    sizes = [sbp.layer_workspace_size(cfg), sbp.layer_workspace_size(cfg, True)]
    for layers, need in (([{}, normed], max(sizes)), ([normed, {}, normed], max(sizes)),
                         ([{}], sizes[0]), ([normed, normed], sizes[1])):
        ws = stack.Workspaces("cpu")
        assert stack._layer_ws(cfg, layers, ws).numel() == max(need, 256)
