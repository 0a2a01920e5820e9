"""Balancing rows that are open to experts of load 0 alone (GPU): they add nothing to any column but
count among the rows."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests import rows_util as ru
from tests.test_rows import rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,experts", [(50, 12), (30000, 60)])
@pytest.mark.parametrize("eps", [0.2, 0.004])
def test_rows_open_to_no_load_alone(rows, experts, eps):
    z = rand(rows, experts, seed=1, scale=1.0)
    z[7, 2:] = -math.inf
    load = torch.ones(experts, device="cuda")
    load[:2] = 0.0
    f, g = fs.balance(z, score="sigmoid", eps=eps, n_iters=3, load=load)
    assert f[7].item() == 0.0 and torch.isfinite(f).all()
    assert (g[:2] == -math.inf).all()
    # as without that row, each mean over one row more: the shift of an update adds to the last one's
    others = torch.arange(rows) != 7
    fr, gr = ru.balance_ref(z.cpu()[others], "sigmoid", eps, 3, load)
    shift = eps * math.log(rows / (rows - 1))
    tol = 3 * (eps * 64 * ru.U + 8 * ru.U) + 4 * ru.U * 2.0
    ru.assert_near(g[2:], gr[2:] + 3 * shift, tol, "g")
    ru.assert_near(f.cpu()[others], fr - 2 * shift, tol, "f")
