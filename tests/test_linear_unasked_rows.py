"""linear_logprobs' gradients where rows that nobody asks about hold anything (GPU): the padding
of a batch may be uninitialised, and its infinities and NaN reach no gradient."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests.test_rows import BF, rand, randint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,dim", [(3, 40, 8), (60, 300, 64), (200, 700, 77), (300, 513, 40)])
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, torch.finfo(BF).max])
def test_rows_not_asked_about_reach_no_gradient(rows, cols, dim, fill):
    x, w = rand(rows, dim, seed=1, dtype=BF, scale=1.0), rand(cols, dim, seed=2, dtype=BF, scale=0.3)
    ids = randint(rows, cols)
    unasked = torch.arange(rows, device="cuda") % 3 == 1
    unasked[-1] = rows > 60
    ids[unasked] = -100
    g = rand(rows, seed=3)
    results = []
    for value in (0.0, fill):
        x[unasked] = value
        leaves = [t.detach().clone().requires_grad_(True) for t in (x, w)]
        out = fs.linear_logprobs(*leaves, ids)
        assert all(float(t.detach()[unasked].abs().max()) == 0.0 for t in out)
        results.append(torch.autograd.grad([out.logprobs, out.entropy], leaves, [g, g]))
    for a, b in zip(*results):
        assert torch.isfinite(b).all() and torch.equal(a, b)
    assert float(results[1][0][unasked].abs().max()) == 0.0


@pytest.mark.parametrize("rows", [50, 200])
def test_rows_not_asked_about_get_nothing_from_a_bad_embedding(rows):
    x, w = rand(rows, 64, seed=4, dtype=BF, scale=1.0), rand(300, 64, seed=5, dtype=BF, scale=0.3)
    w[7, 3] = math.inf
    ids = randint(rows, 300)
    ids[::2] = -1
    x.requires_grad_(True)
    (gx,) = torch.autograd.grad(fs.linear_logprobs(x, w, ids).logprobs.sum(), x)
    assert float(gx[::2].abs().max()) == 0.0
