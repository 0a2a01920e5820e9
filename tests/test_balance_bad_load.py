"""A load that is no load (GPU): a negative entry, NaN, an infinity or a sum of 0 makes every
output NaN, those of experts with a load of 0 among them."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests.test_rows import rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,experts", [(40, 12), (30000, 60)])
@pytest.mark.parametrize("bad", [-1.0, -math.inf, math.inf, math.nan])
def test_a_bad_entry_makes_all_outputs_nan(rows, experts, bad):
    z = rand(rows, experts, seed=1, scale=1.0)
    z[3] = -math.inf
    load = torch.ones(experts, device="cuda")
    load[0] = 0.0
    load[5] = bad
    f, g = fs.balance(z, eps=0.1, n_iters=3, load=load)
    assert f.isnan().all() and g.isnan().all()


def test_no_load_at_all():
    f, g = fs.balance(rand(40, 12, seed=1), eps=0.1, n_iters=2, load=torch.zeros(12, device="cuda"))
    assert f.isnan().all() and g.isnan().all()
