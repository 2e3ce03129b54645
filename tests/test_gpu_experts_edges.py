"""Calls of the experts' products that their documentation allows and whose
faults depend on timing, on other calls or on unusual values, against the
bounds of test_gpu_experts."""
import pytest
import torch

import means_clustering_gmm_b200 as gmm  # noqa: F401

from .test_gpu_experts import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,gated", [(0, False), (600, True)])
def test_biases_of_the_next_tile(h, gated):
    """Blocks that work through many tiles, experts and columns whose biases
    are far apart, and tiles of which some rows hold no point: a bias read
    from the tile after would be off by whole numbers."""
    N, d, o, K = 9000, 64, 1104, 5
    s = inputs(41, N, d, h, o, K, 1, "f16", gated=gated, cut=0.2, use=[0, 0, 0, 1, 3, 4])
    step = torch.arange(s["b1"].shape[1]) // 32 % 7
    s["b1"] = (s["b1"] + torch.arange(K)[:, None] - step).half()
    check(s, "silu", gated)
