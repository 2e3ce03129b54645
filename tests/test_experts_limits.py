"""Sizes at and past the limits of the experts' calls (no GPU needed)."""
import pytest
import torch

import means_clustering_gmm_b200 as gmm

WRAP = 1 << 32   # what a 32-bit field drops


@pytest.mark.parametrize("name", ["N", "d", "h", "o", "K", "r"])
@pytest.mark.parametrize("wrap", [WRAP, 1 << 64, -WRAP])
def test_sizes_that_would_wrap_are_invalid(name, wrap):
    """A size whose low bits are a valid size is refused all the same."""
    s = dict(N=100, d=64, h=48, o=32, K=4, r=2, dtype=torch.bfloat16)
    assert gmm.expert_workspace_size(**s) > 0
    s[name] += wrap
    assert gmm.expert_workspace_size(**s) == 0
    assert gmm.expert_workspace_size(**s, backward=True) == 0
    with pytest.raises(ValueError):
        gmm.expert_path(**s)
    with pytest.raises(ValueError):
        gmm.Workspace.for_expert_mlp(**s)
