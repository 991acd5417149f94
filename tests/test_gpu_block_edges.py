"""The router at the ends of its range, against its definition in 64 bits."""
import math

import pytest
import torch

import block_ref as ref
import test_gpu_route as routes
from combine_moe_layout_amd import binding as B

pytestmark = pytest.mark.gpu

# groups of 2, 3 and 60 experts meet in LDS, groups of 8, 32 and 256 by lanes of 4, 8 and 16 experts
GROUPS = [(4, 2, 1), (24, 8, 3), (64, 8, 3), (300, 5, 2), (512, 16, 4), (1024, 4, 2)]


@pytest.mark.parametrize("E,groups,topk_groups", GROUPS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_past_fp32(E, groups, topk_groups, score):
    """Biases whose sums by two leave fp32's range, above and below: groups go by the sums in fp64, and a
    group without any usable expert comes after all of them."""
    print("[gpu-edges] group sums", E, groups, topk_groups, score, flush=True)
    T, n = 60, E // groups
    for sign in (1.0, -1.0):
        for seed in range(4):
            g = routes.gen(E + seed)
            logits = torch.randn((T, E), device="cuda", generator=g)
            logits.view(T, groups, n)[1::3, 0] = -math.inf              # the group of the lowest index is dead
            bias = sign * (1.8e38 + 1.6e38 * torch.rand(E, device="cuda", generator=g))
            if E == 4 and seed == 0:
                bias = sign * torch.tensor([3e38, 2e38, 3e38, 3e38], device="cuda")
            router = B.EpRouter(E, 2, routes.SCORES[score], groups, topk_groups, 2)
            idx, _ = routes.route(logits, "fp32", router, bias)
            assert torch.equal(idx, ref.choice(logits, bias, 2, score, groups, topk_groups, 2)), (sign, seed)
