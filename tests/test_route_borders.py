"""Routing at borders that 32 bits cannot tell apart (GPU): every expert that is left out is
compared with the last pick, whatever its own error and whatever ties lie between them."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests import rows_util as ru
from tests.test_rows import F32, check_route, rand

pytestmark = pytest.mark.gpu


def column(*values):
    return torch.tensor(values, dtype=F32, device="cuda")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_expert_left_out_with_a_larger_error(score):
    """The first expert left out is all but exact, the second one's score is near 1 and its bias
    takes it back to the border, to within the rounding of its score."""
    g = torch.Generator().manual_seed(3)
    rows = 200
    for trial in range(25):
        z = column(-30.0, -30.5, *(torch.rand(2, generator=g) * 2.0 - 1.0).tolist()).repeat(rows, 1)
        z[:, 2] += torch.arange(rows, device="cuda") * 2.0 ** -25
        s = ru.scores_ref(z, score)[:, 2]
        bias = column(0.001, 0.000999999, 0.001 - float(s[rows // 2]), -10.0)
        # the same in lanes that hold several experts
        wide = torch.full((rows, 70), -30.0, device="cuda")
        wide[:, 40:44] = z
        b = torch.full((70,), -11.0, device="cuda")
        b[40:44] = bias
        for k in (1, 2):
            check_route(z, k, score=score, bias=bias, grads=False)
            check_route(wide, k, score=score, bias=b, grads=False)


def test_the_row_of_the_softmax_example():
    z = column(-30.0, -30.5, 0.3002, -0.4002)[None]
    bias = column(0.001, 0.000999999, -0.66727644, -10.0)
    assert ru.route_ref(z, 1, bias=bias)["ids"].tolist() == [[2]]
    assert fs.route(z, 1, bias=bias).ids.tolist() == [[2]]


@pytest.mark.parametrize("experts", [3, 33, 64, 100, 256, 1000])
@pytest.mark.parametrize("k", [1, 2, 5, 14])
def test_a_better_expert_behind_a_tie(experts, k):
    """Sigmoids that are 1 in 32 bits: the first two are equal in any precision, the third and the
    last are above them in 64 bits alone."""
    k = min(k, experts)
    z = torch.full((40, experts), 17.0, device="cuda")
    z[:, 2] = 18.0
    z[1::2, -1] = 19.0
    z[::3, experts // 2] = 17.5
    check_route(z, k, score="sigmoid", grads=False)
    check_route(z.bfloat16(), k, score="sigmoid", grads=False)
    check_route(z, k, score="sigmoid", bias=torch.full((experts,), 0.25, device="cuda"), grads=False)
    # biases that differ by less than the rounding of the sum
    bias = torch.full((experts,), 4.0, device="cuda")
    bias[1::3] = 4.0 + 2.0 ** -21
    check_route(z, k, score="sigmoid", bias=bias, grads=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_small_biases_below_the_scores_rounding(score):
    """Equal logits and biases that vanish next to the score in 32 bits."""
    for experts, k in ((8, 2), (96, 7), (256, 8), (256, 20)):
        z = torch.zeros(30, experts, device="cuda")
        bias = rand(experts, seed=experts, scale=1e-12)
        check_route(z, k, score=score, bias=bias, grads=False)
        z[:, ::2] = rand(30, (experts + 1) // 2, seed=3, scale=1e-7)
        check_route(z, k, score=score, bias=bias, grads=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_coarse_logits_with_ties_at_the_border(score):
    """Logits of a few values, so that most borders are ties, with and without a bias of few
    values; closed experts among them."""
    g = torch.Generator().manual_seed(5)
    for experts, k in ((6, 2), (60, 6), (256, 8), (384, 31)):
        z = (torch.randint(0, 9, (3000, experts), generator=g) / 4.0).cuda()
        z[torch.rand(3000, experts, generator=g).cuda() < 0.05] = -math.inf
        bias = (torch.randint(0, 3, (experts,), generator=g) / 16.0).cuda()
        check_route(z, k, score=score, grads=False)
        check_route(z, k, score=score, bias=bias, grads=False)
