"""Routing within groups whose border 32 bits cannot tell (GPU): each of a group's two best is
rounded at its own size, however small their sum."""
import math

import pytest
import torch

from tests.test_rows import F32, check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,per", [(2, 2), (4, 2), (4, 16), (3, 5)])
def test_biases_of_opposite_sign(score, groups, per):
    """Two best of about +64 and -64: the sum is small, its rounding is not. The groups' sums are
    the same up to differences below that rounding."""
    experts = groups * per
    rand = torch.Generator().manual_seed(groups * per)
    z = torch.zeros(600, groups, per)
    z[:, :, :2] = 2.0 * torch.rand(600, 1, 2, generator=rand) - 1.0
    z[:, :, :2] += 1e-5 * torch.randn(600, groups, 2, generator=rand)
    z = z.reshape(600, experts).cuda()
    bias = torch.full((groups, per), -100.0)
    bias[:, 0], bias[:, 1] = 64.0, -64.0
    bias = bias.reshape(-1).cuda()
    check_route(z, 2, score=score, bias=bias, groups=groups, top_groups=1, grads=False)
    if groups > 2:
        check_route(z, 3, score=score, bias=bias, groups=groups, top_groups=groups - 1, grads=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_set_aside_by_a_large_bias(score):
    """A bias of -1e30 sets an expert or a whole group aside and leaves the others' order alone."""
    g = torch.Generator().manual_seed(9)
    z = torch.randn(500, 64, generator=g).cuda()
    bias = 0.1 * torch.randn(64, generator=g).cuda()
    bias[8:24] = -1e30
    bias[::9] = -1e30
    check_route(z, 4, score=score, bias=bias, groups=8, top_groups=3, grads=False)
    bias[40:48] = -math.inf
    check_route(z, 4, score=score, bias=bias, groups=8, top_groups=3, grads=False)
    check_route(z.to(torch.bfloat16), 4, score=score, bias=bias.to(F32), groups=16, top_groups=5, grads=False)
