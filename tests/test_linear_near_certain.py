"""linear_logprobs' gradients where the given token has nearly all of the probability (GPU): the
scores that the gradient forms again have to be those that the row's sums were made of, bit by bit,
or the difference shows in 1 - p."""
import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests import rows_util as ru
from tests.test_rows import BF, rand, randint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 3, 128, 200])
@pytest.mark.parametrize("dim", [256, 4096])
def test_gradient_of_a_near_certain_token(rows, dim):
    cols = 500
    w = rand(cols, dim, seed=71, dtype=BF, scale=1.0)
    ids = randint(rows, cols)
    x = (16.0 / dim * w[ids].float()).to(BF).requires_grad_(True)
    w.requires_grad_(True)
    out = fs.linear_logprobs(x, w, ids)
    gx, gw = torch.autograd.grad(out.logprobs.sum(), (x, w))
    xd, wd = x.detach().double(), w.detach().double()
    p = torch.softmax(xd @ wd.t(), 1)
    d = -p
    r = torch.arange(rows, device="cuda")
    # (1 - p of the given token without its cancellation)
    rest = p.clone()
    rest[r, ids] = 0.0
    d[r, ids] = rest.sum(1)
    # p: its exponential and the row's sum, as in token_tol for an entropy of nothing; each entry
    # also by twice the error of a score, 2^-23 of sums below 16 after every 16 products
    t = (2.0 * 8.0 + 24.0 + cols / 256.0) * ru.U
    off = 4 * (dim / 16) * 16 * 2.0 ** -23 * d.abs()
    off[r, ids] += t
    # (the entries that are rounded to bf16 as well)
    off += 2.0 ** -8 * d.abs()
    for got, big, e, other in ((gx, d, off, wd), (gw, d.t(), off.t(), xd)):
        ref = big @ other
        tol = 1.01 * (e @ other.abs() + ru.type_tol(ref, BF)) + 1e-37
        over = (got.double() - ref).abs() / tol
        assert float(over.max()) <= 1.0, float(over.max())
