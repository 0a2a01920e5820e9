"""Refusals of the row-softmax operators on the CPU: the C ABI rejects bad arguments before any
device work, and the Python binding names what is wrong. No GPU is needed or used here."""
import ctypes

import pytest
import torch

import streaming_sinkhorn_b200 as fs
from streaming_sinkhorn_b200 import _lib

# A fake, 256-byte aligned "device" address: only ever compared, never dereferenced.
FAKE = 0x7F0000000000
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def mat(data=FAKE, rows=4, cols=64, ld=None, dtype=0):
    return _lib.fs_matrix(data, rows, cols, cols if ld is None else ld, dtype)


BAD_MATRICES = [
    (None, "FS_ERR_NULL"),
    (mat(data=None), "FS_ERR_NULL"),
    (mat(dtype=3), "FS_ERR_DTYPE"),
    (mat(dtype=-1), "FS_ERR_DTYPE"),
    (mat(rows=-1), "FS_ERR_SHAPE"),
    (mat(rows=1 << 31), "FS_ERR_SHAPE"),
    (mat(cols=0), "FS_ERR_SHAPE"),
    (mat(ld=63), "FS_ERR_SHAPE"),
    (mat(ld=1 << 60), "FS_ERR_SHAPE"),
    (mat(data=FAKE + 2), "FS_ERR_ALIGNMENT"),
    (mat(data=FAKE + 1, dtype=2), "FS_ERR_ALIGNMENT"),
]


def st(code):
    return _lib.STATUS[code]


def tokens(z=mat(), eps=1.0, ids=FAKE, ids_64=1, top=0, logp=FAKE, entropy=FAKE, lse=None,
           stats=None, top_logp=FAKE, top_ids=FAKE):
    return st(_lib.load().fs_token_logprobs(None if z is None else ctypes.byref(z), eps, ids,
                                            ids_64, top, logp, entropy, lse, stats, top_logp,
                                            top_ids, None))


def tokens_grad(z=mat(), eps=1.0, ids=FAKE, ids_64=1, top=0, top_ids=None, stats=FAKE,
                entropy=FAKE, g_logp=None, g_entropy=None, g_lse=None, g_top=None, grad=FAKE,
                ld=64):
    return st(_lib.load().fs_token_logprobs_grad(None if z is None else ctypes.byref(z), eps, ids,
                                                 ids_64, top, top_ids, stats, entropy, g_logp,
                                                 g_entropy, g_lse, g_top, grad, ld, None))


def opts(k=2, score=0, groups=1, top_groups=1, renormalize=1, scale=1.0, bias=None):
    return _lib.fs_route_options(k, score, groups, top_groups, renormalize, scale, bias)


def route(z=mat(), o=opts(), weights=FAKE, ids=FAKE, load=None):
    return st(_lib.load().fs_route(None if z is None else ctypes.byref(z),
                                   None if o is None else ctypes.byref(o), weights, ids, load, None))


def route_grad(z=mat(), o=opts(), weights=FAKE, ids=FAKE, g=FAKE, grad=FAKE):
    return st(_lib.load().fs_route_grad(None if z is None else ctypes.byref(z),
                                        None if o is None else ctypes.byref(o), weights, ids, g,
                                        grad, None))


def balance(z=mat(), score=0, eps=0.1, n_iters=3, load=None, g_init=None, f=FAKE, g=FAKE, ws=FAKE,
            ws_bytes=BIG):
    return st(_lib.load().fs_balance(None if z is None else ctypes.byref(z), score, eps, n_iters,
                                     load, g_init, f, g, ws, ws_bytes, None))


@pytest.mark.parametrize("z,expect", BAD_MATRICES)
def test_bad_matrices(z, expect):
    assert tokens(z) == expect
    assert tokens_grad(z) == expect
    assert route(z) == expect
    assert route_grad(z) == expect
    assert balance(z) == expect


def test_token_arguments():
    for eps in (0.0, -1.0, NAN, INF, 1e-45, 3e-39):
        assert tokens(eps=eps) == "FS_ERR_EPS" and tokens_grad(eps=eps) == "FS_ERR_EPS"
    for top in (-1, 33):
        assert tokens(top=top) == "FS_ERR_OPTION" and tokens_grad(top=top) == "FS_ERR_OPTION"
    assert tokens(mat(cols=3), top=4) == "FS_ERR_OPTION"
    assert tokens(ids_64=2) == "FS_ERR_OPTION"
    for name in ("ids", "logp", "entropy"):
        assert tokens(**{name: None}) == "FS_ERR_NULL"
    assert tokens(top=2, top_ids=None) == "FS_ERR_NULL"
    assert tokens(ids=FAKE + 4) == "FS_ERR_ALIGNMENT"
    assert tokens(ids=FAKE + 2, ids_64=0) == "FS_ERR_ALIGNMENT"
    assert tokens(stats=FAKE + 4) == "FS_ERR_ALIGNMENT"
    assert tokens(logp=FAKE + 1) == "FS_ERR_ALIGNMENT"
    assert tokens(mat(data=None, rows=0)) == "FS_OK"
    for name in ("ids", "stats", "entropy", "grad"):
        assert tokens_grad(**{name: None}) == "FS_ERR_NULL"
    assert tokens_grad(top=2, g_top=FAKE) == "FS_ERR_NULL"  # no top_ids
    assert tokens_grad(ld=63) == "FS_ERR_SHAPE"
    assert tokens_grad(grad=FAKE + 2) == "FS_ERR_ALIGNMENT"
    assert tokens_grad(g_logp=FAKE + 2) == "FS_ERR_ALIGNMENT"


def test_route_arguments():
    assert route(o=None) == "FS_ERR_NULL" and route_grad(o=None) == "FS_ERR_NULL"
    assert route(mat(cols=1025)) == "FS_ERR_SHAPE"
    for o in (opts(k=0), opts(k=32), opts(score=2), opts(groups=0), opts(groups=3), opts(groups=64),
              opts(groups=4, top_groups=0), opts(groups=4, top_groups=5),
              opts(k=17, groups=4, top_groups=1), opts(renormalize=2), opts(scale=NAN),
              opts(scale=INF)):
        assert route(o=o) == "FS_ERR_OPTION" and route_grad(o=o) == "FS_ERR_OPTION"
    assert route(o=opts(bias=FAKE + 2)) == "FS_ERR_ALIGNMENT"
    assert route(weights=None) == "FS_ERR_NULL" and route(ids=None) == "FS_ERR_NULL"
    assert route(load=FAKE + 2) == "FS_ERR_ALIGNMENT"
    assert route_grad(g=None) == "FS_ERR_NULL" and route_grad(grad=FAKE + 2) == "FS_ERR_ALIGNMENT"
    assert route(mat(data=None, rows=0), weights=None, ids=None) == "FS_OK"


def test_balance_arguments():
    lib = _lib.load()
    need = lib.fs_balance_workspace_bytes(ctypes.byref(mat()))
    assert need > 0 and need % 256 == 0
    assert lib.fs_balance_workspace_bytes(ctypes.byref(mat(cols=1025))) == 0
    assert lib.fs_balance_workspace_bytes(None) == 0
    # rows beyond shared memory need room in the workspace
    big = lib.fs_balance_workspace_bytes(ctypes.byref(mat(rows=1 << 20, cols=256)))
    assert big > (1 << 20) * 256 * 4 * 3 // 4
    assert balance(mat(cols=1025)) == "FS_ERR_SHAPE"
    assert balance(eps=0.0) == "FS_ERR_EPS" and balance(eps=NAN) == "FS_ERR_EPS"
    assert balance(n_iters=0) == "FS_ERR_ITERS" and balance(n_iters=1000001) == "FS_ERR_ITERS"
    assert balance(score=2) == "FS_ERR_OPTION"
    assert balance(f=None) == "FS_ERR_NULL" and balance(g=None) == "FS_ERR_NULL"
    assert balance(load=FAKE + 2) == "FS_ERR_ALIGNMENT"
    assert balance(ws=None) == "FS_ERR_WORKSPACE" and balance(ws=FAKE + 8) == "FS_ERR_WORKSPACE"
    assert balance(ws_bytes=need - 1) == "FS_ERR_WORKSPACE"


def linear(x=mat(dtype=2), w=mat(dtype=2, rows=100), eps=1.0, ids=FAKE, ids_64=1, logp=FAKE,
           entropy=FAKE, lse=None, stats=None, ws=FAKE, ws_bytes=BIG):
    ref = lambda m: None if m is None else ctypes.byref(m)  # noqa: E731
    return st(_lib.load().fs_linear_logprobs(ref(x), ref(w), eps, ids, ids_64, logp, entropy, lse,
                                             stats, ws, ws_bytes, None))


def linear_grad(x=mat(dtype=2), w=mat(dtype=2, rows=100), eps=1.0, ids=FAKE, ids_64=1, stats=FAKE,
                entropy=FAKE, g=None, gx=FAKE, gw=FAKE, ws=FAKE, ws_bytes=BIG):
    ref = lambda m: None if m is None else ctypes.byref(m)  # noqa: E731
    return st(_lib.load().fs_linear_logprobs_grad(ref(x), ref(w), eps, ids, ids_64, stats, entropy,
                                                  g, None, None, gx, gw, ws, ws_bytes, None))


@pytest.mark.parametrize("z,expect", [
    (None, "FS_ERR_NULL"), (mat(data=None, dtype=2), "FS_ERR_NULL"), (mat(dtype=0), "FS_ERR_DTYPE"),
    (mat(dtype=1), "FS_ERR_DTYPE"), (mat(rows=-1, dtype=2), "FS_ERR_SHAPE"),
    (mat(cols=0, dtype=2), "FS_ERR_SHAPE"), (mat(ld=60, dtype=2), "FS_ERR_SHAPE"),
    (mat(ld=68, dtype=2), "FS_ERR_ALIGNMENT"), (mat(data=FAKE + 8, dtype=2), "FS_ERR_ALIGNMENT"),
    (mat(cols=72, dtype=2), "FS_ERR_SHAPE"),  # not the other's dim
])
def test_bad_operands_of_the_linear_form(z, expect):
    for call in (linear, linear_grad):
        assert call(x=z) == expect
        assert call(w=z) == expect


def test_linear_arguments():
    lib = _lib.load()
    x, w = mat(dtype=2), mat(dtype=2, rows=100)
    need = lib.fs_linear_logprobs_workspace_bytes(ctypes.byref(x), ctypes.byref(w))
    need_g = lib.fs_linear_logprobs_grad_workspace_bytes(ctypes.byref(x), ctypes.byref(w))
    assert need > 0 and need % 256 == 0 and need_g > 4 * 100 * 2 and need_g % 256 == 0
    other = mat(cols=72, dtype=2)
    assert lib.fs_linear_logprobs_workspace_bytes(ctypes.byref(x), ctypes.byref(other)) == 0
    assert lib.fs_linear_logprobs_grad_workspace_bytes(None, ctypes.byref(w)) == 0
    # the gradient keeps at most 1 GiB of G, plus the sums of dx
    big = [mat(rows=r, cols=1024, dtype=2) for r in (8192, 262144)]
    assert lib.fs_linear_logprobs_grad_workspace_bytes(*map(ctypes.byref, big)) < 2 << 30
    assert linear(w=mat(dtype=2, rows=0)) == "FS_ERR_SHAPE"
    for eps in (0.0, NAN, INF, -2.0):
        assert linear(eps=eps) == "FS_ERR_EPS" and linear_grad(eps=eps) == "FS_ERR_EPS"
    assert linear(ids_64=2) == "FS_ERR_OPTION" and linear_grad(ids_64=-1) == "FS_ERR_OPTION"
    for name in ("ids", "logp", "entropy"):
        assert linear(**{name: None}) == "FS_ERR_NULL"
    for name in ("ids", "stats", "entropy"):
        assert linear_grad(**{name: None}) == "FS_ERR_NULL"
    assert linear(stats=FAKE + 4) == "FS_ERR_ALIGNMENT"
    assert linear_grad(g=FAKE + 2) == "FS_ERR_ALIGNMENT"
    assert linear_grad(gx=FAKE + 1) == "FS_ERR_ALIGNMENT"
    assert linear_grad(gx=None, gw=None) == "FS_OK"
    for call, size in ((linear, need), (linear_grad, need_g)):
        assert call(ws=None) == "FS_ERR_WORKSPACE" and call(ws=FAKE + 64) == "FS_ERR_WORKSPACE"
        assert call(ws_bytes=size - 1) == "FS_ERR_WORKSPACE"


def test_python_binding_refuses():
    z = torch.zeros(4, 16)
    ids = torch.zeros(4, dtype=torch.long)
    for call in (lambda t: fs.token_logprobs(t, ids), lambda t: fs.route(t, 2),
                 lambda t: fs.balance(t, eps=0.1, n_iters=1)):
        with pytest.raises(ValueError, match="CUDA"):
            call(z)
        with pytest.raises(ValueError, match="float64"):
            call(z.double())
        with pytest.raises(TypeError, match="int32"):
            call(z.int())
        with pytest.raises(ValueError, match="2-D"):
            call(z[0])
        with pytest.raises(TypeError, match="Tensor"):
            call(z.numpy())
    for bad in (z, z.half()):
        with pytest.raises(ValueError, match="CUDA"):
            fs.linear_logprobs(bad, bad, ids)
