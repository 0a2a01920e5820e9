"""Optional vectors of the row-softmax operators that are no tensors are refused by name (GPU: the
matrix before them has to be a CUDA tensor)."""
import pytest
import torch

import streaming_sinkhorn_b200 as fs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [[0.0] * 16, 0.5, torch.zeros(16).numpy()])
def test_vectors_that_are_no_tensors(bad):
    z = torch.zeros(4, 16, device="cuda")
    for name, call in (("bias", lambda: fs.route(z, 2, bias=bad)),
                       ("load", lambda: fs.balance(z, eps=0.1, n_iters=1, load=bad)),
                       ("g_init", lambda: fs.balance(z, eps=0.1, n_iters=1, g_init=bad))):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            call()


def test_vectors_that_require_grad_take_no_part_in_the_gradient():
    z = torch.randn(4, 16, device="cuda", requires_grad=True)
    b = torch.zeros(32, device="cuda", requires_grad=True)
    out = fs.route(z, 2, bias=b[::2])
    (g,) = torch.autograd.grad(out.weights[:, 0].sum(), z)
    assert torch.isfinite(g).all()
    f, _ = fs.balance(z, eps=0.1, n_iters=2, load=(b + 1.0)[::2], g_init=b[:16])
    assert not f.requires_grad
