"""Float64 references of the row-softmax operators and the tolerances of their tests.

Tolerances (float32 arithmetic, u = 2^-24 half a unit in the last place):
  a term 2^((z - m) k): the difference, the product and ex2.approx (2^-22) move it by at most
  (2 |d| + 8) u relative, d = (z - m) log2(e)/eps; a sum of n terms over 256 threads adds at
  most (n / 256 + 16) u. So lse is off by at most (2 dbar + 24 + n / 256) u with dbar the
  p-weighted mean of |d| (at most the entropy in bits plus a few), logp by that plus 3 u |logp|
  (a difference, a product, a sum), the entropy by twice that times (1 + |entropy|).
  A gradient p (c - ge (logp + H)) inherits p's relative error; rounding it to the output's type
  adds half a unit, finfo.eps / 2 relative (or half the spacing of its subnormals).
"""
import math

import torch

U = 2.0 ** -24


def token_ref(z, ids, eps=1.0, top=0, g_logp=None, g_entropy=None, g_lse=None, g_top=None):
    """logp, entropy, lse, top_logp, top_ids, grad of z (T, V) in float64 on the CPU."""
    z = z.detach().cpu().double()
    ids = ids.detach().cpu().long()
    n, v = z.shape
    uz = z / eps
    m = uz.amax(1, keepdim=True)
    empty = (m[:, 0] == -math.inf)
    mm = torch.where(empty[:, None], 0.0, m)
    total = torch.exp(uz - mm).sum(1, keepdim=True)
    lse = (mm + torch.log(total))[:, 0]
    # (the difference first: the logarithm is lost next to a row of the type's lowest value)
    logp_all = (uz - mm) - torch.log(total)
    p = torch.exp(logp_all)
    p[empty] = 0.0
    safe = torch.where(p > 0, logp_all, 0.0)
    h = -(p * safe).sum(1)
    asked = (ids >= 0)
    known = asked & (ids < v)
    r = torch.arange(n)
    logp = torch.where(known, logp_all[r, ids.clamp(0, v - 1)], math.nan)
    logp[known & empty] = -math.inf
    logp[~asked] = 0.0
    h = torch.where(asked & ~empty, h, 0.0)
    out = {"logprobs": logp, "entropy": h,
           "lse": torch.where(asked, lse, 0.0)}
    if top:
        order = torch.sort(z + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
        tl = logp_all.gather(1, order)
        tl[empty] = -math.inf
        out["top_ids"] = torch.where(asked[:, None], order, -1)
        out["top_logprobs"] = torch.where(asked[:, None], tl, -math.inf)
    zero = torch.zeros(n, dtype=torch.float64)
    gl, ge, gs = (zero if g is None else g.detach().cpu().double()
                  for g in (g_logp, g_entropy, g_lse))
    c = gs - gl
    if g_top is not None:
        c = c - g_top.detach().cpu().double().sum(1)
    d = p * (c[:, None] - ge[:, None] * (safe + h[:, None]))
    size = p * (c.abs()[:, None] + ge.abs()[:, None] * (safe.abs() + h[:, None]))
    d[r[known], ids[known]] += gl[known]
    if g_top is not None:
        d.scatter_add_(1, order, g_top.detach().cpu().double())
    d[~asked | empty] = 0.0
    size[~asked | empty] = 0.0
    d[asked & (ids >= v) & ~empty] = math.nan
    out["grad"] = d / eps
    out["grad_size"] = size / eps
    out["p"] = p
    return out


def token_tol(ref, n, logp):
    bits = ref["entropy"].abs() / math.log(2.0) + 8.0
    lse = (2.0 * bits + 24.0 + n / 256.0) * U
    return lse, lse + 3.0 * U * logp.abs().nan_to_num(0.0, 0.0, 0.0), 2.0 * lse * (1 + ref["entropy"])


def assert_near(got, ref, tol, name):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    assert bool((same | fine).all()), f"{name}: infinities or NaN differ"
    err = torch.where(fine, (got - ref).abs(), torch.zeros_like(ref))
    over = err - (tol if torch.is_tensor(tol) else torch.full_like(err, tol))
    if err.numel():
        i = int(over.argmax())
        assert bool((over <= 0).all()), (
            f"{name}: off by {float(err.reshape(-1)[i]):.3g} at {i} "
            f"(got {float(got.reshape(-1)[i])!r}, expected {float(ref.reshape(-1)[i])!r})")


def type_tol(ref, dtype):
    """Half a unit in the last place of each value in ``dtype``."""
    fi = torch.finfo(dtype)
    return ref.abs().nan_to_num(0.0) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def scores_ref(z, score):
    z = z.detach().cpu().double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(z - m)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def route_ref(z, k, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True,
              scale=1.0, g_weights=None):
    """weights, ids, load, grad in float64, row by row."""
    zd = z.detach().cpu().double()
    s = scores_ref(z, score)
    n, e = zd.shape
    b = torch.zeros(e, dtype=torch.float64) if bias is None else bias.detach().cpu().double()
    c = s + b
    c = torch.where((zd == -math.inf) | (b == -math.inf), torch.full_like(c, -math.inf), c)
    if groups > top_groups:
        per = e // groups
        best = c.view(n, groups, per).sort(dim=2, descending=True).values[:, :, :2]
        gs = best[:, :, 0].clone()
        if per > 1:
            two = best[:, :, 1] != -math.inf
            gs[two] += best[:, :, 1][two]
        kept = gs.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        mask = torch.zeros(n, groups, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(per, 1), c, torch.full_like(c, -math.inf))
    order = c.sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :k].clone()
    ids[order.values[:, :k] == -math.inf] = -1
    picked = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), 0.0)
    total = picked.sum(1, keepdim=True) if renormalize else torch.ones(n, 1, dtype=torch.float64)
    w = torch.where(total > 0, scale * picked / total.clamp(min=1e-300), 0.0)
    load = torch.zeros(e, dtype=torch.int32)
    load.scatter_add_(0, ids[ids >= 0], torch.ones(int((ids >= 0).sum()), dtype=torch.int32))
    out = {"weights": w, "ids": ids, "load": load}
    if g_weights is not None:
        gw = g_weights.detach().cpu().double() * scale * (ids >= 0)
        if renormalize:
            ds = torch.where(total > 0, (gw - (gw * picked).sum(1, keepdim=True) /
                                         total.clamp(min=1e-300)) / total.clamp(min=1e-300), 0.0)
        else:
            ds = gw
        d = torch.zeros_like(zd)
        if score == "sigmoid":
            d.scatter_add_(1, ids.clamp(min=0), ds * picked * (1 - picked))
        else:
            d -= s * (ds * picked).sum(1, keepdim=True)
            d.scatter_add_(1, ids.clamp(min=0), ds * picked)
        out["grad"] = d
    return out


def balance_ref(z, score, eps, n_iters, load=None, g_init=None):
    """(f, g) in float64: closed logits, empty rows and columns as the library defines them."""
    zd = z.detach().cpu().double()
    n, e = zd.shape
    u = torch.where(zd == -math.inf, torch.full_like(zd, -math.inf), scores_ref(z, score) / eps)
    rows = (u != -math.inf).any(1)
    cols = (u != -math.inf).any(0)
    b = torch.full((e,), 1.0 / e, dtype=torch.float64) if load is None else (
        load.detach().cpu().double() / load.detach().cpu().double().sum())
    g = torch.zeros(e, dtype=torch.float64) if g_init is None else g_init.cpu().double() / eps
    lb = torch.log(b)
    for _ in range(n_iters):
        f = -torch.logsumexp(u + torch.where(b > 0, g, torch.zeros_like(g)) + lb, dim=1)
        f = torch.where(rows, f, torch.zeros_like(f))
        g = -(torch.logsumexp((u + f[:, None])[rows], dim=0) - math.log(max(int(rows.sum()), 1)))
        g = torch.where(cols, g, torch.zeros_like(g))
        g = torch.where(b > 0, g, torch.full_like(g, -math.inf))
    return eps * f, eps * g


def linear_ref(x, w, ids, eps=1.0, **g):
    """token_ref of z = x w^T with the gradients of x and w, and what bounds their errors: the
    largest error of a score in fp32 accumulation (16 products a step, each sum off by at most
    2^-23 of the absolute sum) and the absolute sums |G| |w|, |G|^T |x|."""
    xd, wd = x.detach().cpu().double(), w.detach().cpu().double()
    ref = token_ref(xd @ wd.t(), ids, eps, **g)
    d = ref["grad"]
    ref["grad_x"], ref["grad_w"] = d @ wd, d.t() @ xd
    ref["abs_x"], ref["abs_w"] = d.abs() @ wd.abs(), d.abs().t() @ xd.abs()
    # |G| with its terms apart: what an error of p alone moves
    ref["size_x"] = ref["grad_size"] @ wd.abs()
    ref["size_w"] = ref["grad_size"].t() @ xd.abs()
    ref["dz"] = (x.shape[1] / 16 + 2) * 2 * U * float((xd.abs() @ wd.abs().t()).max()) / eps
    return ref
