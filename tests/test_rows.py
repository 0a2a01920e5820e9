"""Log probabilities of given tokens, routing and balancing (GPU) against float64 references at
the sizes, layouts and masks where they can go wrong, and their gradients against the formula
and against differences. The references and tolerances are in rows_util."""
import ctypes
import math

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from streaming_sinkhorn_b200 import _lib, rows
from tests import rows_util as ru

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def rand(*shape, seed=0, dtype=F32, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def randint(n, hi, seed=0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed + 1)
    return torch.randint(0, hi, (n,), generator=g, dtype=dtype).cuda()


def check_tokens(z, ids, eps=1.0, top=0, grads=True, seed=0):
    n, v = z.shape
    z = z.detach().requires_grad_(grads)
    out = fs.token_logprobs(z, ids, eps=eps, top=top)
    g = {}
    if grads:
        g = {"g_logp": rand(n, seed=seed + 2), "g_entropy": rand(n, seed=seed + 3),
             "g_lse": rand(n, seed=seed + 4)}
        outs, gs = [out.logprobs, out.entropy, out.lse], list(g.values())
        if top:
            g["g_top"] = rand(n, top, seed=seed + 5)
            outs.append(out.top_logprobs)
            gs.append(g["g_top"])
        (grad,) = torch.autograd.grad(outs, (z,), gs)
    ref = ru.token_ref(z, ids, eps, top, **g)
    t_lse, t_logp, t_h = ru.token_tol(ref, v, ref["logprobs"])
    ru.assert_near(out.logprobs, ref["logprobs"], t_logp, "logprobs")
    ru.assert_near(out.entropy, ref["entropy"], t_h, "entropy")
    t = t_lse + 3 * ru.U * ref["lse"].abs().nan_to_num(0, 0, 0)
    ru.assert_near(out.lse, ref["lse"], t, "lse")
    if top:
        assert torch.equal(out.top_ids.cpu().long(), ref["top_ids"])
        tt = t_lse[:, None] + 3 * ru.U * ref["top_logprobs"].abs().nan_to_num(0, 0, 0)
        ru.assert_near(out.top_logprobs, ref["top_logprobs"], tt, "top_logprobs")
    if grads:
        assert grad.dtype == z.dtype and grad.shape == z.shape
        # p's own error, and the rounding of the sums that make the coefficient
        rel = t_lse[:, None] + (2 * 24 + 16) * ru.U
        tol = (rel * ref["grad_size"] * 2 + 8 * ru.U * ref["grad"].abs().nan_to_num(0)
               + ru.type_tol(ref["grad"], z.dtype) * 1.01)
        ru.assert_near(grad, ref["grad"], tol, "grad")
    return out


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("rows,cols,top", [(1, 1, 1), (1, 7, 3), (3, 33, 32), (5, 1000, 4),
                                           (2, 4099, 0), (300, 515, 5), (1, 70001, 20),
                                           (9, 20000, 8)])
def test_tokens_match_float64(dtype, rows, cols, top):
    z = rand(rows, cols, seed=cols, dtype=dtype)
    check_tokens(z, randint(rows, cols, seed=rows), top=top, seed=rows)


@pytest.mark.parametrize("eps", [0.25, 1.7])
def test_tokens_temperature_and_int32_ids(eps):
    z = rand(6, 911, seed=3, dtype=BF)
    check_tokens(z, randint(6, 911, dtype=torch.int32), eps=eps, top=3)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_tokens_strided_rows_and_odd_alignment(dtype):
    wide = rand(7, 2050, seed=5, dtype=dtype)
    ids = randint(7, 1000)
    for view in (wide[:, 3:1206], wide[::2, 1:1202][:4], wide[:, :1200], wide.t()[:1200].t()):
        check_tokens(view, ids[: view.shape[0]], top=4)
    one = rand(1, 1003, seed=6, dtype=dtype)
    check_tokens(one.expand(5, 1003), randint(5, 1003), top=2, grads=False)


def test_gradient_of_a_broadcast_row_is_the_sum():
    one = rand(1, 303, seed=8).requires_grad_(True)
    ids = randint(5, 303)
    out = fs.token_logprobs(one.expand(5, 303), ids)
    (g,) = torch.autograd.grad(out.logprobs.sum(), one)
    ref = ru.token_ref(one.expand(5, 303), ids, g_logp=torch.ones(5))["grad"].sum(0, keepdim=True)
    ru.assert_near(g, ref, 5 * 64 * ru.U, "summed gradient")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,top", [(7, 7), (33, 32), (1000, 5), (1000, 20), (5003, 8)])
def test_tokens_alternatives_of_many_rows(dtype, vocab, top):
    """Enough rows for four warps each; rows of ties and of masked scores, and rows that start
    inside a vector."""
    z = rand(2600, vocab + 3, seed=23, dtype=dtype)
    z[::5] = torch.randint(0, 4, z[::5].shape, generator=torch.Generator().manual_seed(2)).to(z)
    z[1::5][torch.rand(z[1::5].shape, generator=torch.Generator().manual_seed(3)).cuda() < 0.98] = -math.inf
    check_tokens(z[:, 3:], randint(2600, vocab), top=top, grads=False)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_tokens_alternatives_of_unkind_rows(dtype):
    """Rows that defeat a bar taken from their beginning: ascending, all equal, a few values only,
    the best at the ends, and long rows with more of them than a warp sets aside at once."""
    v = 30000
    z = rand(7, v, seed=21, dtype=dtype)
    z[0] = torch.linspace(-4, 4, v).to(dtype)
    z[1] = -torch.linspace(-4, 4, v).to(dtype)
    z[2] = 1.5
    z[3] = torch.randint(0, 3, (v,), generator=torch.Generator().manual_seed(1)).to(dtype)
    z[4, 0], z[4, v - 1], z[4, v - 2] = 50.0, 49.0, 50.0
    z[5, ::3] = 9.0
    for top in (1, 20, 32):
        check_tokens(z, randint(7, v), top=top, grads=False)
        check_tokens(z[:, 1:-2], randint(7, v - 3), top=top, grads=False)
    many = rand(700, 5000, seed=22, dtype=dtype)
    many[::5] = 0.25
    check_tokens(many, randint(700, 5000), top=32, grads=False)


def test_tokens_ties_take_the_lowest_index():
    z = torch.zeros(3, 5000, dtype=BF, device="cuda")
    z[1, 4000:] = 1.0
    z[2, ::7] = -0.0  # equal to 0
    out = check_tokens(z, randint(3, 5000), top=8)
    assert out.top_ids[1].tolist() == list(range(4000, 4008))
    assert out.top_ids[2].tolist() == list(range(8))


@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_tokens_masks(dtype):
    low = torch.finfo(dtype).min
    z = rand(8, 1500, seed=11, dtype=dtype)
    z[0, 5:] = -math.inf           # five columns left
    z[1] = -math.inf               # none
    z[2] = low                     # a uniform row at the type's lowest value
    z[3, 100:] = low
    z[4, :] = -math.inf
    z[4, 777] = -3.0               # one
    z[5, 1::2] = -math.inf
    ids = torch.tensor([2, 3, 4, 50, 777, 1, -100, -1], device="cuda")
    out = check_tokens(z, ids, top=7)
    assert out.lse[1].item() == -math.inf and out.entropy[1].item() == 0.0
    assert out.logprobs[5].item() == -math.inf  # the given token is masked
    assert out.entropy[2].item() == pytest.approx(math.log(1500), rel=1e-6)
    assert out.top_ids[6].tolist() == [-1] * 7
    # rows nobody asks about are not read: NaN there changes nothing
    z[6:] = math.nan
    again = check_tokens(z, ids, top=7)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


def test_tokens_nan_inf_and_tokens_out_of_range():
    z = rand(5, 700, seed=12)
    z[0, 13] = math.nan
    z[1, 600] = math.inf
    z[3] = math.nan
    ids = torch.tensor([5, 5, 700, 1, 699], device="cuda")
    z.requires_grad_(True)
    out = fs.token_logprobs(z, ids, top=3)
    assert torch.isnan(out.logprobs[:4]).all() and torch.isfinite(out.logprobs[4])
    assert torch.isnan(out.entropy[[0, 1, 3]]).all() and torch.isfinite(out.entropy[[2, 4]]).all()
    assert torch.isnan(out.top_logprobs[0]).all() and (out.top_ids[0] != 13).all()
    assert out.top_ids[3].tolist() == [-1, -1, -1]
    (g,) = torch.autograd.grad(out.logprobs, z, torch.ones(5, device="cuda"))
    assert torch.isnan(g[:4]).all() and torch.isfinite(g[4]).all()


def test_tokens_no_rows_and_one_column():
    z = torch.zeros(0, 50, device="cuda", requires_grad=True)
    out = fs.token_logprobs(z, torch.zeros(0, dtype=torch.long, device="cuda"), top=2)
    assert out.logprobs.shape == (0,) and out.top_ids.shape == (0, 2)
    (g,) = torch.autograd.grad(out.logprobs.sum(), z)
    assert g.shape == (0, 50)
    out = fs.token_logprobs(torch.full((2, 1), 3.0, device="cuda"), randint(2, 1), top=1)
    assert out.logprobs.tolist() == [0.0, 0.0] and out.top_ids.tolist() == [[0], [0]]


def test_tokens_offsets_past_32_bits():
    # 2^31 elements (2^32 bytes) between the first row and the last
    big = torch.empty(5 << 30, dtype=torch.uint8, device="cuda").view(BF)
    z = big.as_strided((3, 2000), ((1 << 30) + 8, 1))
    vals = rand(3, 2000, seed=13, dtype=BF)
    z.copy_(vals)
    ids = randint(3, 2000)
    a, b = fs.token_logprobs(z, ids, top=2), fs.token_logprobs(vals, ids, top=2)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_tokens_gradient_against_differences():
    z = rand(4, 37, seed=14)
    ids = randint(4, 37)
    zc = z.detach().requires_grad_(True)
    out = fs.token_logprobs(zc, ids, top=3)
    w = [rand(4, seed=s) for s in (15, 16, 17)] + [rand(4, 3, seed=18)]
    (g,) = torch.autograd.grad([out.logprobs, out.entropy, out.lse, out.top_logprobs], zc, w)

    def f(t):
        r = ru.token_ref(t, ids, top=3)
        names = ("logprobs", "entropy", "lse", "top_logprobs")
        return sum(float((r[k] * v.cpu().double()).sum()) for k, v in zip(names, w))

    h = 1e-5
    for s in range(5):
        d = rand(4, 37, seed=20 + s, scale=1.0).cpu().double()
        zd = z.cpu().double()
        num = (f(zd + h * d) - f(zd - h * d)) / (2 * h)
        # central differences: h^2 times a third derivative (at most ~50 here), and 1e-16 / h
        assert float((g.cpu().double() * d).sum()) == pytest.approx(num, abs=1e-4)


# ---- log probabilities from states and an embedding ------------------------------------------

def check_linear(x, w, ids, eps=1.0, seed=0):
    n, v = x.shape[0], w.shape[0]
    x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
    out = fs.linear_logprobs(x, w, ids, eps=eps)
    g = {"g_logp": rand(n, seed=seed + 2), "g_entropy": rand(n, seed=seed + 3),
         "g_lse": rand(n, seed=seed + 4)}
    gx, gw = torch.autograd.grad(list(out), (x, w), list(g.values()))
    ref = ru.linear_ref(x, w, ids, eps, **g)
    t_lse, t_logp, t_h = ru.token_tol(ref, v, ref["logprobs"])
    dz = ref["dz"]
    ru.assert_near(out.logprobs, ref["logprobs"], t_logp + 2 * dz, "logprobs")
    ru.assert_near(out.entropy, ref["entropy"], t_h + 2 * dz * (1 + ref["entropy"]), "entropy")
    ru.assert_near(out.lse, ref["lse"], t_lse + dz + 3 * ru.U * ref["lse"].abs(), "lse")
    # G is rounded to bf16 (half a step, finfo.eps / 2 = 2^-8 of each term), p is off by its argument's error, the sums run in
    # fp32 over the tensor cores' 16-term steps, and the result is rounded once
    rel_p = 2 * (float(t_lse.max()) + 2 * dz + 64 * ru.U)
    for got, name, k in ((gx, "x", v), (gw, "w", n)):
        ref_g, size, terms = ref["grad_" + name], ref["size_" + name], ref["abs_" + name]
        acc = (k / 16 + 2) * 2 * ru.U
        tol = ((2.0 ** -8 + acc) * terms + (rel_p + acc) * size) * 1.01 + \
            ru.type_tol(ref_g, BF) * 1.01 + 1e-37
        assert got.dtype == BF and got.shape == ref_g.shape
        ru.assert_near(got, ref_g, tol, "grad_" + name)
    return out


@pytest.mark.parametrize("rows,cols,dim", [(1, 1, 8), (1, 300, 64), (5, 33, 16), (128, 256, 64),
                                           (129, 257, 72), (300, 1000, 200), (2, 5000, 512),
                                           (257, 3001, 96), (640, 2050, 328)])
def test_linear_matches_float64(rows, cols, dim):
    x, w = rand(rows, dim, seed=rows, dtype=BF, scale=1.0), rand(cols, dim, seed=cols + 1, dtype=BF,
                                                                  scale=2.0 / math.sqrt(dim))
    ids = randint(rows, cols, seed=dim)
    if rows > 4:
        ids[1::5] = -100
    check_linear(x, w, ids, seed=rows)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("dim,cols", [(256, 1000), (264, 77), (512, 20000), (1000, 333), (2048, 5003),
                                      (4096, 1537), (4104, 300)])
def test_linear_few_rows(rows, dim, cols):
    x = rand(rows, dim, seed=rows, dtype=BF, scale=1.0)
    w = rand(cols, dim + 8, seed=dim, dtype=BF, scale=2.0 / math.sqrt(dim))
    ids = randint(rows, cols, seed=dim)
    if rows > 2:
        ids[1] = -1
    for view in (w[:, :dim], w[:, :dim].contiguous()):
        check_linear(x, view, ids, seed=rows)


def test_linear_layouts_and_temperature():
    x, w = rand(40, 130, seed=1, dtype=BF, scale=1.0), rand(70, 130, seed=2, dtype=BF, scale=0.2)
    ids = randint(40, 70, dtype=torch.int32)
    for d0, d in ((0, 128), (2, 64), (8, 100), (1, 77), (0, 1), (0, 130)):
        check_linear(x[:, d0:d0 + d], w[:, d0:d0 + d], ids, eps=0.7)
    check_linear(x[::3], w.t().contiguous().t(), ids[:14])


def test_linear_agrees_with_the_scores_form():
    x, w = rand(200, 64, seed=3, dtype=BF, scale=1.0), rand(900, 64, seed=4, dtype=BF, scale=0.3)
    ids = randint(200, 900)
    a, b = fs.linear_logprobs(x, w, ids), fs.token_logprobs(x.float() @ w.float().t(), ids)
    for s, t in zip(a, b):
        assert float((s - t).abs().max()) < 1e-4  # two orders of fp32 sums of 64 products


def test_linear_one_gradient_only_and_no_rows():
    x, w = rand(30, 32, seed=5, dtype=BF), rand(90, 32, seed=6, dtype=BF)
    ids = randint(30, 90)
    both = [t.clone().requires_grad_(True) for t in (x, w)]
    gx, gw = torch.autograd.grad(fs.linear_logprobs(*both, ids).logprobs.sum(), both)
    only = x.clone().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(fs.linear_logprobs(only, w, ids).logprobs.sum(), only)[0], gx)
    only = w.clone().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(fs.linear_logprobs(x, only, ids).logprobs.sum(), only)[0], gw)
    e = torch.empty(0, 32, dtype=BF, device="cuda").requires_grad_(True)
    out = fs.linear_logprobs(e, both[1], torch.zeros(0, dtype=torch.long, device="cuda"))
    gx, gw = torch.autograd.grad(out.logprobs.sum(), (e, both[1]))
    assert gx.shape == (0, 32) and float(gw.abs().max()) == 0.0


def test_linear_ids_out_of_range_and_nan():
    x, w = rand(150, 32, seed=7, dtype=BF), rand(300, 32, seed=8, dtype=BF)
    ids = randint(150, 300)
    ids[3] = 300
    x[5, 0] = math.nan
    x.requires_grad_(True)
    out = fs.linear_logprobs(x, w, ids)
    bad = torch.isnan(out.logprobs).nonzero().flatten().tolist()
    assert bad == [3, 5] and torch.isnan(out.entropy).nonzero().flatten().tolist() == [5]
    (g,) = torch.autograd.grad(out.logprobs.sum(), x)
    assert torch.isnan(g).any(1).nonzero().flatten().tolist() == [3, 5]


def test_linear_gradient_in_chunks_of_columns():
    # more than 1 GiB of G: two chunks, the states' gradient added over both
    rows, cols, dim = 8200, 70000, 16
    x, w = rand(rows, dim, seed=9, dtype=BF, scale=1.0), rand(cols, dim, seed=10, dtype=BF, scale=0.3)
    ids = randint(rows, cols)
    leaves = [t.requires_grad_(True) for t in (x, w)]
    out = fs.linear_logprobs(x, w, ids)
    gx, gw = torch.autograd.grad(out.logprobs.sum(), leaves)
    xd, wd = x.detach().double(), w.detach().double()
    d = -torch.softmax(xd @ wd.t(), 1)
    d[torch.arange(rows), ids] += 1.0
    for got, ref, terms in ((gx, d @ wd, d.abs() @ wd.abs()), (gw, d.t() @ xd, d.abs().t() @ xd.abs())):
        # 2^-8 from G, 2^-8 from the result, p's own error and the fp32 sums within 2^-10 more
        assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * 1.25 * terms + 2.0 ** -8 * ref.abs()).all())


def test_linear_in_a_graph_and_on_two_streams():
    x, w = rand(70, 64, seed=11, dtype=BF, scale=1.0), rand(4000, 64, seed=12, dtype=BF, scale=0.3)
    ids = randint(70, 4000)
    x.requires_grad_(True)
    w.requires_grad_(True)

    def step():
        out = fs.linear_logprobs(x, w, ids)
        return (*out, *torch.autograd.grad(out.logprobs, (x, w), torch.ones_like(out.logprobs)))

    want = [t.detach().clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    got.append(out)
    for g in got:
        for a, b in zip(want, g):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("dim", [256, 4091])
def test_linear_token_that_has_nearly_all_the_probability(rows, dim):
    """The given token's score is formed apart from the others: it has to take its own place in
    the sum, or a probability near 1 would come out above 1 or with the error of a score."""
    w = rand(500, dim, seed=71, dtype=BF, scale=1.0)
    ids = randint(rows, 500)
    x = (25.0 / dim * w[ids].float()).to(BF)  # the token's score is about 25, the others' 25 / sqrt(dim)
    pad = torch.zeros(rows, 8 * -(-dim // 8), dtype=BF, device="cuda")
    pad[:, :dim] = x
    out = fs.linear_logprobs(pad[:, :dim], w, ids)
    z = x.double().cpu() @ w.double().cpu().t()
    ref = torch.log_softmax(z, 1).gather(1, ids.cpu()[:, None])[:, 0]
    # of the numbers near 1: the sum's rounding (2^-24), two exponentials and a logarithm (2 ulp,
    # 2^-23 each); of the rest of the sum, e to the error of a score, which is below dim / 16 cuts
    # of 2^-23 of sums below 40
    tol = 2.0**-24 + 3 * 2.0**-23 + ref.abs() * (dim / 16 * 40 * 2.0**-23 * 1.5)
    err = (out.logprobs.double().cpu() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()


# ---- routing -----------------------------------------------------------------------------------

def check_route(z, k, grads=True, seed=0, **kw):
    z = z.detach().requires_grad_(grads)
    out = fs.route(z, k, load=True, **kw)
    gw = rand(z.shape[0], k, seed=seed + 9, scale=1.0) if grads else None
    ref = ru.route_ref(z, k, g_weights=gw, **kw)
    assert torch.equal(out.ids.cpu().long(), ref["ids"])
    assert torch.equal(out.load.cpu(), ref["load"])
    # s carries (|x| + 8) u twice (numerator and sum), |x| <= 24 in these tests, and the quotient
    rel = 4 * 34 * ru.U
    ru.assert_near(out.weights, ref["weights"], rel * ref["weights"].abs(), "weights")
    if grads:
        (g,) = torch.autograd.grad(out.weights, z, gw)
        size = ref["grad"].abs().amax(1, keepdim=True) + \
            (gw.cpu().double().abs() * ref["weights"].abs()).amax(1, keepdim=True)
        tol = 4 * rel * size + ru.type_tol(ref["grad"], z.dtype) * 1.01
        assert g.dtype == z.dtype
        ru.assert_near(g, ref["grad"], tol, "grad")
    return out


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rows,experts,k", [(1, 1, 1), (3, 8, 2), (33, 60, 6), (70, 64, 31),
                                            (5, 160, 8), (257, 256, 8), (4, 500, 10),
                                            (6, 1024, 31)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_matches_float64(dtype, score, rows, experts, k, renormalize):
    z = rand(rows, experts, seed=experts + rows, dtype=dtype)
    bias = rand(experts, seed=experts + 1, scale=0.2) if rows % 2 else None
    check_route(z, k, score=score, bias=bias, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,k", [(256, 8, 4, 8), (64, 4, 2, 4), (160, 8, 3, 6),
                                                         (32, 32, 5, 5), (12, 3, 1, 4), (96, 6, 6, 4),
                                                         (21, 7, 2, 6)])
def test_route_groups(score, experts, groups, top_groups, k):
    z = rand(200, experts, seed=experts, dtype=BF)
    bias = rand(experts, seed=2, scale=0.1)
    for b in (bias, None):
        check_route(z, k, score=score, bias=b, groups=groups, top_groups=top_groups)


def test_route_ties_and_close_borders():
    # all equal; pairs one float apart; saturated sigmoids; a bias that makes scores meet
    z = torch.zeros(6, 64, device="cuda")
    z[1] = torch.arange(64, device="cuda") * 2.0 ** -24 + 1.0
    z[2] = 40.0 + torch.arange(64, device="cuda")
    z[3] = -30.0 - torch.arange(64, device="cuda") * 1e-6
    z[4, ::2] = 1e-7
    z[5] = rand(64, seed=1)
    bias = torch.zeros(64, device="cuda")
    for score in ("softmax", "sigmoid"):
        check_route(z, 7, score=score, grads=False)
        check_route(z, 7, score=score, bias=bias, grads=False)
        check_route(z, 6, score=score, groups=8, top_groups=3, grads=False)
    s = ru.scores_ref(z, "sigmoid")
    meet = (0.75 - s[5]).float().cuda()  # s + b is 0.75 up to rounding: only 64 bits tell
    check_route(z[5:], 9, score="sigmoid", bias=meet, grads=False)


def test_route_many_rows_choose_as_in_64_bits():
    # enough rows for some borders to lie within the rounding of 32 bits
    for score, seed in (("softmax", 31), ("sigmoid", 32)):
        z = rand(20000, 128, seed=seed, scale=1.0)
        bias = rand(128, seed=33, scale=0.05)
        check_route(z, 8, score=score, bias=bias, groups=8, top_groups=4, grads=False)
        check_route(z.to(BF), 8, score=score, grads=False)


def test_route_closed_experts_and_empty_rows():
    z = rand(6, 40, seed=41)
    z[0, 3:] = -math.inf
    z[1] = -math.inf
    z[2, ::2] = -math.inf
    bias = torch.zeros(40, device="cuda")
    bias[5] = -math.inf
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for grp in (dict(), dict(groups=4, top_groups=2)):
                out = check_route(z, 6, score=score, bias=b, **grp)
                assert out.ids[1].tolist() == [-1] * 6 and out.weights[1].abs().sum() == 0
    z[3, 7] = math.nan
    out = fs.route(z.requires_grad_(True), 2)
    assert out.ids[3].tolist() == [-1, -1] and torch.isnan(out.weights[3]).all()
    (g,) = torch.autograd.grad(out.weights.sum(), z)
    assert torch.isnan(g[3]).all() and torch.isfinite(g[[0, 1, 2, 4, 5]]).all()


def test_route_underflowing_sigmoids_keep_their_ratio():
    z = torch.full((2, 10), -200.0, device="cuda")
    z[0, 4], z[0, 6] = -120.0, -121.0
    out = check_route(z, 2, score="sigmoid", grads=False)
    assert out.ids[0].tolist() == [4, 6]


def test_route_strides_rows_zero_and_scale():
    wide = rand(9, 130, seed=51, dtype=BF)
    check_route(wide[:, 1:65], 4)
    check_route(wide[::3, 3:], 4, score="sigmoid", scale=0.5)
    out = fs.route(torch.zeros(0, 16, device="cuda"), 2, load=True)
    assert out.ids.shape == (0, 2) and out.load.tolist() == [0] * 16


# ---- balancing ---------------------------------------------------------------------------------

def check_balance(z, eps, n_iters, score="softmax", load=None, g_init=None):
    f, g = fs.balance(z, score=score, eps=eps, n_iters=n_iters, load=load, g_init=g_init)
    fr, gr = ru.balance_ref(z, score, eps, n_iters, load, g_init)
    # an update moves by the rounding of its scores (s / eps in log2 units, |s| <= 1) and of a
    # mean of exponentials; the updates are non-expansive, so errors add up at worst
    tol = n_iters * (eps * 64 * ru.U + 8 * ru.U)
    tol_of = lambda r: tol + 4 * ru.U * r.abs().nan_to_num(0, 0, 0)  # noqa: E731
    ru.assert_near(f, fr, tol_of(fr), "f")
    ru.assert_near(g, gr, tol_of(gr), "g")
    return f, g


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rows,experts", [(1, 1), (5, 3), (100, 8), (257, 16), (1000, 60),
                                          (3001, 64), (513, 256), (300, 300), (700, 1024)])
def test_balance_matches_float64(dtype, score, rows, experts):
    z = rand(rows, experts, seed=rows + experts, dtype=dtype, scale=1.0)
    check_balance(z, 0.1, 5, score)


def test_balance_rows_beyond_shared_memory():
    z = rand(40000, 250, seed=61, scale=1.0)
    check_balance(z, 0.1, 3, "sigmoid")


@pytest.mark.parametrize("rows,experts", [(200003, 60), (70001, 250), (20000, 500), (15500, 1000)])
def test_balance_rows_in_and_beyond_tensor_memory(rows, experts):
    """Rows that fill part of a step of tensor memory, and rows that pass it, for rows of part of
    a warp, of a warp, and of several quads a lane."""
    z = rand(rows, experts, seed=65, scale=1.0)
    check_balance(z, 0.1, 2, "sigmoid")


def test_balance_unkind_rows_across_the_grid():
    z = rand(30011, 64, seed=66, scale=1.0)
    load = torch.arange(64, dtype=F32, device="cuda")
    g0 = rand(64, seed=67, scale=0.1)
    z[:, 5] = -math.inf
    z[7:2000] = -math.inf
    f, g = check_balance(z, 0.2, 3, "sigmoid", load=load, g_init=g0)
    assert g[0].item() == -math.inf and g[5].item() == 0.0 and f[7].item() == 0.0
    z[1:] = -math.inf  # a single row takes part
    check_balance(z, 0.2, 3, "softmax")
    # columns whose terms underflow next to the rows' largest
    z = torch.linspace(-6, 6, 60, device="cuda").repeat(20000, 1) + rand(20000, 60, seed=68, scale=0.01)
    check_balance(z, 0.003, 3, "sigmoid")
    z[19999, 3] = math.nan
    f, g = fs.balance(z, eps=0.1, n_iters=3)
    assert f.isnan().all() and g.isnan().all()


def test_balance_load_start_and_closed():
    z = rand(300, 24, seed=62, scale=1.0)
    z[7] = -math.inf
    z[:, 5] = -math.inf
    z[10:200, 6] = -math.inf
    load = torch.arange(24, dtype=F32, device="cuda")  # expert 0 gets nothing
    g0 = rand(24, seed=63, scale=0.1)
    for score in ("softmax", "sigmoid"):
        f, g = check_balance(z, 0.2, 4, score, load=load, g_init=g0)
        assert g[0].item() == -math.inf and g[5].item() == 0.0 and f[7].item() == 0.0
        check_balance(z, 0.2, 4, score, g_init=g0)


def test_balance_sharp_scores_use_each_columns_own_range():
    # eps so small that a column's terms underflow next to the rows' largest
    z = torch.linspace(-6, 6, 50, device="cuda").repeat(64, 1) + rand(64, 50, seed=64, scale=0.01)
    check_balance(z, 0.003, 4, "sigmoid")


def test_balance_spreads_the_picks_by_the_load():
    """P_i = softmax((s_i + g)/eps) has column sums T b up to the solve's own residual, and
    |[argmax = j] - P_ij| <= 1 - max_j P_ij, so the picks of the best expert are off the load by
    at most sum_i (1 - max_j P_ij) plus that residual."""
    z = rand(4096, 32, seed=65, scale=1.0) + rand(32, seed=66, scale=1.0)
    load = torch.linspace(0.5, 1.5, 32, device="cuda")
    eps = 0.005
    f, g = fs.balance(z, score="sigmoid", eps=eps, n_iters=60, load=load)
    b = (load / load.sum()).cpu().double()
    s = ru.scores_ref(z, "sigmoid")
    plan = torch.exp((s + f.cpu().double()[:, None] + g.cpu().double()) / eps) * b / 4096
    # the columns were made to fit last: exp carries (f, g and s)'s rounding over eps
    assert float((plan.sum(0) / b - 1).abs().max()) <= 64 * ru.U / eps
    p = torch.softmax((s + g.cpu().double()) / eps + torch.log(b), dim=1)
    undecided = float((1 - p.amax(1)).sum())
    # (the choice goes by s + g + eps log b, which is the plan's largest entry)
    bias = g + eps * torch.log(load / load.sum())
    got = fs.route(z, 1, score="sigmoid", bias=bias, load=True).load.cpu().double()
    off = (got - 4096 * b).abs() - 4096 * (p.sum(0) / 4096 - b).abs() - undecided
    assert float(off.max()) <= 1.0
    before = fs.route(z, 1, score="sigmoid", load=True).load.cpu().double()
    assert float((got - 4096 * b).abs().sum()) < 0.5 * float((before - 4096 * b).abs().sum())


# ---- together, streams, graphs ----------------------------------------------------------------

def test_other_streams_and_two_calls_at_once():
    z = rand(64, 5000, seed=71, dtype=BF)
    ids = randint(64, 5000)
    r = rand(3000, 64, seed=72)
    want = (fs.token_logprobs(z, ids, top=5), fs.route(r, 4, load=True),
            fs.balance(r, eps=0.1, n_iters=6))
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for s in (a, b):
            with torch.cuda.stream(s):
                got.append((fs.token_logprobs(z, ids, top=5), fs.route(r, 4, load=True),
                            fs.balance(r, eps=0.1, n_iters=6)))
    torch.cuda.synchronize()
    for g in got:
        for x, y in zip(want, g):
            for t, u in zip(x, y):
                assert (t is None and u is None) or torch.equal(t, u)


def test_balance_over_the_whole_grid_at_once_and_captured():
    """Two calls that each want every SM, on two streams, and one in a graph."""
    z = rand(60000, 250, seed=79, scale=1.0)
    want = fs.balance(z, score="sigmoid", eps=0.1, n_iters=5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fs.balance(z, score="sigmoid", eps=0.1, n_iters=5))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fs.balance(z, score="sigmoid", eps=0.1, n_iters=5)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for f, g in (*got, out):
        assert torch.equal(f, want[0]) and torch.equal(g, want[1])


def test_balance_many_iterations_and_g_in_place():
    z = rand(900, 40, seed=80, scale=1.0)
    check_balance(z, 0.1, 200, "sigmoid")
    g0 = rand(40, seed=85, scale=0.1)
    f, g = check_balance(z, 0.1, 3, g_init=g0)
    lib, m = _lib.load(), rows._matrix(z)
    ws = torch.empty(lib.fs_balance_workspace_bytes(ctypes.byref(m)), dtype=torch.uint8, device="cuda")
    f2 = torch.empty_like(f)
    code = lib.fs_balance(ctypes.byref(m), 0, 0.1, 3, None, g0.data_ptr(), f2.data_ptr(),
                          g0.data_ptr(), ws.data_ptr(), ws.numel(),
                          torch.cuda.current_stream().cuda_stream)
    assert code == 0 and torch.equal(f, f2) and torch.equal(g, g0)


def test_captured_into_a_graph_and_replayed():
    z = rand(8, 3000, seed=73, dtype=BF)
    ids = randint(8, 3000)
    r = rand(500, 32, seed=74)
    bias = torch.zeros(32, device="cuda")

    def step():
        t = fs.token_logprobs(z, ids, top=3)
        _, g = fs.balance(r, score="sigmoid", eps=0.1, n_iters=4)
        return (*t, g, *fs.route(r, 4, score="sigmoid", bias=g, load=True), bias)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (75, 76):
        z.copy_(rand(8, 3000, seed=seed, dtype=BF))
        r.copy_(rand(500, 32, seed=seed + 10))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)


def test_gradients_captured_into_a_graph():
    z = rand(8, 3000, seed=77, dtype=BF).requires_grad_(True)
    r = rand(60, 32, seed=78).requires_grad_(True)
    ids = randint(8, 3000)

    def step():
        t = fs.token_logprobs(z, ids, top=2)
        w = fs.route(r, 4).weights
        return torch.autograd.grad([t.logprobs, t.top_logprobs, w], (z, r),
                                   [torch.ones_like(t.logprobs), torch.ones_like(t.top_logprobs),
                                    torch.ones_like(w)])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    for x, y in zip(out, want):
        assert torch.equal(x, y)


def test_a_training_step_of_a_routed_model():
    """Balanced routing of tokens to experts, logits from the mixture, log probabilities and an
    entropy bonus: gradients reach the router and the head, and agree with float64 autograd at
    the same choice."""
    torch.manual_seed(0)
    t, d, e, v = 96, 16, 8, 301
    x = rand(t, d, seed=81, scale=1.0)
    router = rand(d, e, seed=82, scale=0.5).requires_grad_(True)
    experts = rand(e, d, d, seed=83, scale=0.3).requires_grad_(True)
    head = rand(d, v, seed=84, scale=0.5).requires_grad_(True)
    ids = randint(t, v)
    leaves = (router, experts, head)

    def model(x, router, experts, head, pick=None):
        logits = x @ router
        if pick is None:
            _, g = fs.balance(logits, score="sigmoid", eps=0.05, n_iters=10)
            r = fs.route(logits, 2, score="sigmoid", bias=g)
            w, at = r.weights, r.ids.long()
        else:
            s = torch.sigmoid(logits).gather(1, pick)
            w, at = s / s.sum(1, keepdim=True), pick
        h = (torch.einsum("td,tkdf->tkf", x, experts[at]) * w[:, :, None]).sum(1)
        return h @ head, at

    z, at = model(x, *leaves)
    out = fs.token_logprobs(z, ids)
    loss = -out.logprobs.mean() - 0.01 * out.entropy.mean()
    grads = torch.autograd.grad(loss, leaves)

    ref_leaves = [p.detach().double().requires_grad_(True) for p in leaves]
    zr, _ = model(x.double(), *ref_leaves, pick=at)
    lp = torch.log_softmax(zr, 1)
    ref = -lp.gather(1, ids[:, None]).mean() + 0.01 * (lp.exp() * lp).sum(1).mean()
    want = torch.autograd.grad(ref, ref_leaves)
    assert float(loss.detach()) == pytest.approx(float(ref.detach()), rel=1e-5)
    for a, b in zip(grads, want):
        assert float((a.double() - b).norm()) <= 1e-4 * float(b.norm())
