"""Balancing with columns whose terms underflow or that no row can take (GPU): the same values as
in 64 bits, and no more time than a few ordinary iterations each."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests.test_rows import check_balance, rand

pytestmark = pytest.mark.gpu


def best_ms(f, tries=5):
    f()
    torch.cuda.synchronize()
    times = []
    for _ in range(tries):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("rows,experts", [(512, 16), (2000, 64), (8000, 256), (30000, 256), (9000, 1000)])
def test_a_closed_expert_costs_next_to_nothing(rows, experts):
    z = rand(rows, experts, seed=rows, scale=1.0)
    run = lambda: fs.balance(z, score="sigmoid", eps=0.1, n_iters=10)  # noqa: E731
    plain = best_ms(run)
    z[:, experts // 3] = -math.inf
    closed = best_ms(run)
    # (one look at the column, which takes about as long as an iteration or two)
    assert closed <= 2.0 * plain + 0.05, (plain, closed)
    check_balance(z, 0.1, 3, "sigmoid")


@pytest.mark.parametrize("rows,experts", [(300, 50), (4000, 64), (30000, 60), (3000, 600)])
def test_sharp_scores_take_a_few_times_as_long(rows, experts):
    z = torch.linspace(-6, 6, experts, device="cuda").repeat(rows, 1) + rand(rows, experts, seed=1, scale=0.01)
    run = lambda eps: fs.balance(z, score="sigmoid", eps=eps, n_iters=10)  # noqa: E731
    plain, sharp = best_ms(lambda: run(0.2)), best_ms(lambda: run(0.003))
    assert sharp <= 10.0 * plain + 0.2, (plain, sharp)
    check_balance(z, 0.003, 3, "sigmoid")


@pytest.mark.parametrize("rows,experts", [(1, 8), (70, 24), (5000, 130), (20011, 250), (2500, 1024)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_closed_and_sharp_columns_match_float64(rows, experts, score):
    z = rand(rows, experts, seed=rows + experts, scale=1.0)
    z[:, 3] = -math.inf
    z[:, experts - 1] = -math.inf
    z[:, 1] -= 3.0
    if rows > 10:
        z[5:9] = -math.inf
        z[10:, 2] = -math.inf  # open to a few rows only
    load = torch.ones(experts, device="cuda")
    load[4] = 0.0
    load[5] = 1e-6
    eps = 0.01 if score == "sigmoid" else 0.5 / experts
    f, g = check_balance(z, eps, 4, score)
    assert g[3].item() == 0.0 and g[experts - 1].item() == 0.0
    f, g = check_balance(z, eps, 4, score, load=load, g_init=rand(experts, seed=3, scale=0.1))
    assert g[3].item() == 0.0 and g[4].item() == -math.inf


@pytest.mark.parametrize("rows,experts", [(700, 24), (20011, 60)])
def test_captured_with_other_closed_columns_at_each_replay(rows, experts):
    z = rand(rows, experts, seed=1, scale=1.0)
    fs.balance(z, score="sigmoid", eps=0.004, n_iters=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fs.balance(z, score="sigmoid", eps=0.004, n_iters=4)
    for seed in (2, 3):
        z.copy_(rand(rows, experts, seed=seed, scale=2.0))
        z[:, seed * 5] = -math.inf
        graph.replay()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(check_balance(z, 0.004, 4, "sigmoid"))
        torch.cuda.synchronize()
        for f, g in got:
            assert torch.equal(f, out[0]) and torch.equal(g, out[1])
