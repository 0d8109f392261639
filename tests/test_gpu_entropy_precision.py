"""How exactly the cross entropy's gradient holds probabilities far below the largest,
against the formula in 64 bits, every product exact by construction."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def test_float32_probabilities_far_below_the_largest(gpu_lib):
    """D = exp(z - lse) for z - lse from 0 down to -86, all of it exact before the
    exponential: lse is given as 0, X is one, so z is W's first column. The exponential
    is one instruction of at most 2^-23 with its argument's roundings put back: three float32
    roundings beside it, 2^-22 + 2^-24 in all. D's planes and dW keep every bit down to 2^-110;
    below, the second and third plane (2^-8 and 2^-16 of D) pass bfloat16's smallest
    normal number, 2^-126, and may lose that much each: 2^-125."""
    gen = torch.Generator().manual_seed(2)
    for V in (999, 40000):
        z = -86.0 * torch.rand(V, generator=gen)
        z[:4] = torch.tensor([0.0, -1e-6, -86.0, float("-inf")])
        W = torch.zeros(V, 8)
        W[:, 0] = z
        W[3, 0] = -3e38
        X = torch.zeros(1, 8)
        X[0, 0] = 1.0
        X, W = X.cuda(), W.cuda()
        y = torch.tensor([0], device="cuda")
        one, zero = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
        _, dW = gpu_lib.cross_entropy_grad(X, W, y, zero, one, need_dX=False)
        want = torch.exp(W[:, 0].double())
        err = (dW[1:, 0].double() - want[1:]).abs()
        tol = (2.0 ** -22 + E) * want[1:] + 2.0 ** -125
        assert (err <= tol).all(), (err / tol).max()
        assert dW[3, 0] == 0 and (dW[:, 1:] == 0).all()
