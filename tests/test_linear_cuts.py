"""linear_logprobs (GPU): the tensor cores cut their sums towards 0 after every 16 products, which
makes every score a little too small. Over many rows that would show as a bias of the log-sum-exp
of -(cuts / 8) 2^-23 E[z], E the mean under the row's softmax; less than a third of it may be left."""
import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests.test_rows import BF, rand, randint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [64, 128, 1000])
@pytest.mark.parametrize("dim", [2048, 4096])
def test_scores_are_not_biased(rows, dim):
    cols = 9000
    x, w = rand(rows, dim, seed=1, dtype=BF, scale=1.0), rand(cols, dim, seed=2, dtype=BF, scale=1.5 * dim ** -0.5)
    ids = randint(rows, cols)
    out = fs.linear_logprobs(x, w, ids)
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    mean_z = (p * z).sum(1)
    entropy = lse - mean_z
    accumulators = 2 if rows <= 128 else 1
    cuts = dim / 16 / accumulators
    bias = cuts / 8 * 2.0 ** -23 * float(mean_z.mean())
    # (each row's result is rounded, and its own cuts scatter; the mean over 64 rows and thousands
    # of columns keeps an eighth of one rounding of a number below 16: 2^-24 * 16 / 8)
    room = bias / 3 + 2.0 ** -23
    assert abs(float((out.lse.double() - lse).mean())) <= room
    # the entropy moves by the scores' variance in place of their mean, here the same to a few parts in ten
    assert abs(float((out.entropy.double() - entropy).mean())) <= 2 * room
