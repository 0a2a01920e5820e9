"""Forward-mode derivatives of the row-softmax operators are refused, not dropped: a result
without a tangent would read as a derivative of 0."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import streaming_sinkhorn_b200 as fs


def calls(z, x, w, ids):
    return (lambda: fs.token_logprobs(z, ids), lambda: fs.route(z, 2), lambda: fs.linear_logprobs(x, w, ids))


def test_refused_before_anything_else():
    # (on the CPU: the refusal comes before the operand's device is looked at)
    z, ids = torch.zeros(4, 16), torch.zeros(4, dtype=torch.long)
    w = torch.zeros(5, 16).bfloat16()
    with fwad.dual_level():
        dual = fwad.make_dual(z, torch.ones_like(z))
        dual_w = fwad.make_dual(w, torch.ones_like(w))
        for call in calls(dual, dual_w, dual_w, ids):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        for call in calls(z, w, w, ids):  # no tangent: refused for the device alone
            with pytest.raises(ValueError, match="CUDA"):
                call()


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [False, True])
def test_refused_on_the_gpu(grad):
    z = torch.randn(4, 16, device="cuda", requires_grad=grad)
    x = torch.randn(4, 16, device="cuda", dtype=torch.bfloat16, requires_grad=grad)
    ids = torch.zeros(4, dtype=torch.long, device="cuda")
    with fwad.dual_level():
        dz, dx = (fwad.make_dual(t, torch.ones_like(t)) for t in (z, x))
        for call in (*calls(dz, dx, x, ids), lambda: fs.linear_logprobs(x, dx, ids)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        fs.token_logprobs(z, ids), fs.route(z, 2), fs.linear_logprobs(x, x, ids)
