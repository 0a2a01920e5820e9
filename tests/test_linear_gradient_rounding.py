"""linear_logprobs' gradients (GPU): the entries of dL/dz that make up most of a row, the given
token's and that of a token with more than half of the probability, reach both products without a
rounding to bf16. The other entries are made so small here that a rounding of those two shows."""
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from tests import rows_util as ru
from tests.test_rows import BF, rand, randint

pytestmark = pytest.mark.gpu


def check_rounding(x, w, ids, g_logp, g_entropy=None):
    """Against 64 bits: half a bf16 step of the result, half a step of each entry of dL/dz but the
    two of a row that are not rounded (their remainders are to 2^-8: 2^-16), p's own error and
    that of fp32 sums of 16 products a step."""
    x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
    out = fs.linear_logprobs(x, w, ids)
    outs, gs = [out.logprobs], [g_logp]
    if g_entropy is not None:
        outs.append(out.entropy)
        gs.append(g_entropy)
    grads = torch.autograd.grad(outs, (x, w), gs)
    n, v = x.shape[0], w.shape[0]
    xd, wd = x.detach().double(), w.detach().double()
    logp = torch.log_softmax(xd @ wd.t(), 1)
    p = logp.exp()
    known = ids >= 0
    gl = torch.where(known, g_logp.double(), 0.0)
    d = -p * gl[:, None]
    if g_entropy is not None:
        h = -(p * logp).sum(1, keepdim=True)
        d -= p * torch.where(known, g_entropy.double(), 0.0)[:, None] * (logp + h)
    at = ids.clamp(min=0)
    r = torch.arange(n, device=x.device)
    d[r, at] += gl
    main = p > 0.52
    main[r, at] = True
    rounded = torch.where(main, 0.0, d.abs())
    for got, big, k, other, lead in ((grads[0], d, v, wd, rounded), (grads[1], d.t(), n, xd, rounded.t())):
        ref, terms = big @ other, big.abs() @ other.abs()
        acc = (k / 16 + 2) * 2 * ru.U + 128 * ru.U + 2.0 ** -16
        tol = 1.01 * (2.0 ** -8 * (lead @ other.abs()) + acc * terms + ru.type_tol(ref, BF)) + 1e-37
        over = (got.double() - ref).abs() - tol
        assert bool((over <= 0).all()), (float(over.max()), float((over > 0).double().mean()))
    return grads


def few_words(rows, cols, dim, words, seed):
    """An embedding of near-nothing but for its first `words` rows, and tokens among those."""
    w = rand(cols, dim, seed=seed, scale=2.0 ** -12)
    w[:words] = rand(words, dim, seed=seed + 1, scale=1.0)
    return w.to(BF), randint(rows, words, seed=seed + 2)


@pytest.mark.parametrize("rows", [1, 5, 128, 300, 1100])
@pytest.mark.parametrize("dim", [64, 77, 520])
def test_given_token_is_not_rounded(rows, dim):
    w, ids = few_words(rows, 4000, dim, 8, seed=dim)
    x = rand(rows, dim, seed=rows, scale=0.5 / math.sqrt(dim)).to(BF)
    if rows > 4:
        ids[1::5] = -100
    check_rounding(x, w, ids, rand(rows, seed=3, scale=1.0))


@pytest.mark.parametrize("rows", [5, 128, 300])
def test_likely_token_is_not_rounded(rows):
    dim, cols = 64, 4000
    w, likely = few_words(rows, cols, dim, 8, seed=11)
    ids = 8 + randint(rows, cols - 8, seed=12)
    ids[::3] = likely[::3]  # (the two are one)
    ids[::7] = -1
    norm = w[:8].float().pow(2).sum(1)
    x = ((math.log(cols) + 2.0) / norm)[likely][:, None] * w[likely].float()
    check_rounding(x.to(BF), w, ids, rand(rows, seed=13, scale=1.0))
    check_rounding(x.to(BF), w, ids, rand(rows, seed=13, scale=1.0), rand(rows, seed=14, scale=0.1))


def test_one_token_for_all_rows():
    w, ids = few_words(3000, 500, 264, 1, seed=21)
    x = rand(3000, 264, seed=22, scale=0.02).to(BF)
    first = check_rounding(x, w, ids, rand(3000, seed=23, scale=1.0))
    again = check_rounding(x, w, ids, rand(3000, seed=23, scale=1.0))
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_given_token_across_chunks_of_columns():
    # more than 1 GiB of dL/dz: the tokens lie in two chunks of columns
    rows, cols, dim = 8200, 70000, 16
    w, ids = few_words(rows, cols, dim, 8, seed=31)
    w = torch.cat([w[4:], w[:4]])
    ids = torch.where(ids < 4, ids + cols - 4, ids - 4)
    x = rand(rows, dim, seed=32, scale=0.1).to(BF)
    check_rounding(x, w, ids, rand(rows, seed=33, scale=1.0))


def test_sorted_tokens_and_repeated_calls_agree_bit_by_bit():
    w, ids = rand(3001, 96, seed=41, dtype=BF, scale=0.2), randint(700, 40, seed=42)
    x = rand(700, 96, seed=43, dtype=BF, scale=1.0)
    g = rand(700, seed=44)
    leaves = [t.requires_grad_(True) for t in (x, w)]
    want = torch.autograd.grad(fs.linear_logprobs(x, w, ids).logprobs, leaves, g)
    for _ in range(4):
        got = torch.autograd.grad(fs.linear_logprobs(x, w, ids).logprobs, leaves, g)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows", [90, 1500])
def test_captured_with_other_tokens_at_each_replay(rows):
    w, ids = few_words(rows, 3000, 72, 9, seed=51)
    x = rand(rows, 72, seed=52, scale=0.05).to(BF).requires_grad_(True)
    w.requires_grad_(True)
    g = rand(rows, seed=53, scale=1.0)

    def step():
        return torch.autograd.grad(fs.linear_logprobs(x, w, ids).logprobs, (x, w), g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (54, 55):
        ids.copy_(randint(rows, 3000 if seed == 54 else 2, seed=seed))
        ids[::4] = -1
        x.data.copy_(rand(rows, 72, seed=seed, scale=0.05))
        x.data[::4] = math.nan
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        for a, b in zip(out, want):
            assert torch.isfinite(b).all() and torch.equal(a, b)
        torch.cuda.synchronize()


def test_more_rows_than_one_cta_sorts():
    rows, cols, dim = 70001, 2000, 40
    w, ids = few_words(rows, cols, dim, 300, seed=61)
    ids[1::3] = -1
    x = rand(rows, dim, seed=62, scale=0.05).to(BF)
    check_rounding(x, w, ids, rand(rows, seed=63, scale=1.0))
