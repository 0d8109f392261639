"""The cross entropy's gradient with respect to W where tokens differ widely in weight,
against the formula in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ratio", [1.0, 0.7 * 2.0 ** -6, 0.7 * 2.0 ** -16, 1.3 * 2.0 ** -22, -0.9 * 2.0 ** -24])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -8, 40.0])
def test_tokens_of_little_weight_in_float16(gpu_lib, ratio, size):
    """dW where a token of small g stands alone: the token of the largest g holds
    one column, the small one all others. W is zero, so p is 1 / 5 (lse off by
    at most 2^-21, its exponential by 2^-22). D is rounded to 11 bits, (g / max g) X to 11
    bits, and to 2^-39 of its largest below 2^-28 of that (float16's last place under the power
    of two that brings the largest to 2^14), dW to float16: 2^-11 relative each, 2^-25 below its
    normal range."""
    gen = torch.Generator().manual_seed(4)
    X = torch.randn(2, 200, generator=gen) * size
    X[0, 1:], X[1, 0] = 0, 0
    X = X.half().cuda()
    W = torch.zeros(5, 200, dtype=torch.float16, device="cuda")
    y = torch.tensor([1, 3], device="cuda")
    big = 2.0 ** -4 / abs(ratio) / size
    g = torch.tensor([big, big * ratio], device="cuda")
    _, lse = gpu_lib.cross_entropy(X, W, y)
    dX, dW = gpu_lib.cross_entropy_grad(X, W, y, lse, g)
    assert (dX == 0).all()
    D = torch.full((2, 5), 0.2, dtype=torch.float64, device="cuda")
    D[0, 1] -= 1
    D[1, 3] -= 1
    gX = g.double()[:, None] * X.double()
    want = D.T @ gX
    S = D.abs().T @ gX.abs()
    last = 2.0 ** -39 * gX.abs().max()
    tol = S * (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -20) + D.abs().sum(0)[:, None] * last + 2.0 ** -11 * want.abs() + 2.0 ** -25
    # float16 ends at 65504 and rounds from 65520 on to infinity: the large token's own column
    # reaches that where its g does, and may be infinite there
    over = torch.isinf(dW) & (dW.sign() == want.sign()) & (want.abs() + tol >= 65520)
    assert not over[:, 1:].any()
    err = torch.where(over, 0.0, (dW.double() - want).abs())
    assert (want[:, 1:].abs().amax() >= 2.0 ** -6) and (err <= tol).all(), (err / tol).max()


def test_captured_with_weights_that_change(gpu_lib):
    """The float16 gradient in a HIP graph: the power of two comes from each replay's own tokens."""
    bk = gpu_lib
    gen = torch.Generator(device="cuda").manual_seed(8)

    def inputs():
        X = torch.randn(90, 136, device="cuda", generator=gen) * 2.0 ** torch.randint(-6, 6, (90, 1), device="cuda", generator=gen)
        W = torch.randn(500, 136, device="cuda", generator=gen) * 0.05
        y = torch.randint(0, 500, (90,), device="cuda", generator=gen)
        y[::7] = -100
        g = torch.randn(90, device="cuda", generator=gen) * 2.0 ** torch.randint(-20, 6, (90,), device="cuda", generator=gen)
        X, W = X.half(), W.half()
        return X, W, y, bk.cross_entropy(X, W, y)[1], g

    static = inputs()
    bk.cross_entropy_grad(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bk.cross_entropy_grad(*static)
    for _ in range(4):
        new = inputs()
        for t, v in zip(static, new):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, bk.cross_entropy_grad(*new)):
            assert torch.equal(u, v)
