"""Gradients of 8-bit floating point and of a layer of experts against differences of the forward computation in 64
bits, with bounds that a zero, a missing term or a wrong sign cannot meet.

The products are linear in the tokens' values x, so the difference of sum(G Y) between x + d and x - d is twice the
gradient's product with d but for 64-bit rounding. With the direction d chosen as the sign of the exact gradient
every term of that product is positive, so it is as large as the gradient's absolute sum; the gradient's own
tolerance, element by element, then adds up to a small part of it, which each test asserts.

Tolerances (E = 2^-24): a gradient of m terms in three planes 3 m 2^-23 of the terms' absolute sum S and 3 E for the scale and
the blocks; a sum of k rows (k - 1) E of their absolute sum; each result half a step of its type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
E = 2.0 ** -24


def values(q, s, rows):
    """What codes and scales stand for, in 64 bits."""
    a, n = q.shape[-2:]
    s = s.double().repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(128, -1)[..., :n]
    return q.float().double() * s


def grad_tolerance(u, v, ref, t):
    """Of u @ v as the gradient's products take it."""
    S = u.abs() @ v.abs()
    return S * (3 * v.size(0) * 2.0 ** -23 + 3 * E) + ref.abs() * torch.finfo(t).eps / 2 * (1 + 2.0 ** -8) + torch.finfo(t).tiny


def holds(D, want, f, x, tol, part=2.0 ** -6):
    """D against the exact gradient `want` element by element, and its product with a direction against f's differences."""
    assert ((D.double() - want).abs() <= tol).all(), ((D.double() - want).abs() / tol).max()
    d = want.sign()
    change = (f(x + d) - f(x - d)) / 2
    bound = tol.sum() + 1e-9 * change.abs()
    assert bound < part * change.abs()  # zero or a sign the other way round would not pass
    assert ((D.double() * d).sum() - change).abs() <= bound


@pytest.mark.parametrize("T,m,n", [(6, 150, 200), (1, 1000, 300), (300, 260, 500), (130, 40, 1003)])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
def test_product(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + m)
    Wq, sw = gpu_lib.quantize_fp8(torch.randn(m, n, generator=g).cuda(), 128)
    V = values(Wq, sw, 128)
    G = torch.randn(T, m, generator=g).to(t).cuda()
    x = torch.randn(T, n, generator=g).double().cuda()
    D = gpu_lib.matmul_fp8_grad(G, Wq, sw)
    want = G.double() @ V
    holds(D, want, lambda x: (G.double() * (x @ V.T)).sum(), x, grad_tolerance(G.double(), V, want, t))


def layer(T, k, n_experts, n, h, seed):
    g = torch.Generator().manual_seed(seed)
    W1 = torch.randn(n_experts, h, n, generator=g) * n ** -0.5
    W2 = torch.randn(n_experts, n, h, generator=g) * h ** -0.5
    w, ids = torch.randn(T, n_experts, generator=g).softmax(1).topk(k, 1)
    ids[::17] = -1  # padding
    G = torch.randn(T, n, generator=g)
    return [t.cuda() for t in (W1, W2, w.contiguous(), ids, G, torch.randn(T, n, generator=g))]


@pytest.mark.parametrize("T,k,n_experts,n,h", [(200, 2, 6, 384, 260), (33, 3, 9, 130, 128), (500, 1, 4, 257, 300)])
def test_layer_of_experts(gpu_lib, T, k, n_experts, n, h):
    """Back through both products and both ends of the routes, each step on its own inputs; and the whole of it: the
    tokens' gradient and the routes' weights' against differences of the layer."""
    bk = gpu_lib
    W1, W2, w, ids, G, X = layer(T, k, n_experts, n, h, seed=T + n)
    W1q, W2q = bk.quantize_fp8(W1, 128), bk.quantize_fp8(W2, 128)
    V1, V2 = values(*W1q, 128), values(*W2q, 128)
    order, slots, offsets = bk.sort_tokens(ids, n_experts)
    off, has, at = offsets.tolist(), slots >= 0, slots.long().clamp(min=0)
    zeros = lambda c: torch.zeros(order.numel(), c, device="cuda")
    # a forward of the values, in 64 bits: the products' rounding of tokens is passed straight through
    Xs = torch.where((order >= 0)[:, None], X.double()[order.long().clamp(min=0) // k], 0.0)
    H, Ys = zeros(h).double(), zeros(n).double()
    for e in range(n_experts):
        H[off[e]:off[e + 1]] = Xs[off[e]:off[e + 1]] @ V1[e].T
        Ys[off[e]:off[e + 1]] = H[off[e]:off[e + 1]] @ V2[e].T
    Ysf = Ys.float()
    dYs, dw = bk.combine_tokens_grad(G, Ysf, slots, w)
    dH = bk.matmul_fp8_grad(dYs, *W2q, offsets=offsets, out=zeros(h))
    dXs = bk.matmul_fp8_grad(dH, *W1q, offsets=offsets, out=zeros(n))
    dX = bk.combine_tokens(dXs, slots)
    # the first and last steps, element by element
    rows = at[has]
    want = (w[:, :, None].double() * G.double()[:, None])[has]
    assert ((dYs.double()[rows] - want).abs() <= want.abs() * E * (1 + 2.0 ** -20)).all()
    terms = torch.where(has[:, :, None], Ysf.double()[at] * G.double()[:, None], 0.0)
    assert ((dw.double() - terms.sum(2)).abs() <= terms.abs().sum(2) * (n + 1) * E + 2.0 ** -149).all()
    terms = torch.where(has[:, :, None], dXs.double()[at], 0.0)
    assert ((dX.double() - terms.sum(1)).abs() <= terms.abs().sum(1) * k * E).all()
    assert (dX[::17] == 0).all() and (dX.abs().sum(1) > 0).sum() == T - len(range(0, T, 17))

    # the whole: each element's tolerance is that of the last step and what the steps before left, passed on
    def whole(x, w):
        out = torch.zeros(T, n, dtype=torch.float64, device="cuda")
        for j in range(k):
            for e in range(n_experts):
                t = (ids[:, j] == e).nonzero().squeeze(1)
                out[t] += w[t, j, None] * (x[t] @ V1[e].T @ V2[e].T)
        return (out * G.double()).sum()
    want, tol = torch.zeros(T, n, dtype=torch.float64, device="cuda"), torch.zeros(T, n, dtype=torch.float64, device="cuda")
    S = torch.zeros(T, n, dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(n_experts):
            t = (ids[:, j] == e).nonzero().squeeze(1)
            u = w[t, j, None].double() * G.double()[t]
            a = u.abs() * E * 1.001  # dYs
            b = a @ V2[e].abs() + (u.abs() + a) @ V2[e].abs() * (3 * n * 2.0 ** -23 + 4 * E)  # dH
            p = u.abs() @ V2[e].abs() + b
            want[t] += u @ V2[e] @ V1[e]
            tol[t] += b @ V1[e].abs() + p @ V1[e].abs() * (3 * h * 2.0 ** -23 + 4 * E)  # dXs
            S[t] += p @ V1[e].abs() * 1.001
    tol = tol + S * k * E
    holds(dX, want, lambda x: whole(x, w.double()), X.double(), tol, part=0.25)
    # linear in the routes' weights too
    d = torch.where(has, 1.0, 0.0).double() * torch.where(has[:, :, None], Ys[at] * G.double()[:, None], 0.0).sum(2).sign()
    change = (whole(X.double(), w.double() + d) - whole(X.double(), w.double() - d)) / 2
    bound = (torch.where(has[:, :, None], Ys[at] * G.double()[:, None], 0.0).abs().sum(2) * (n + 3) * E).sum() + 1e-9 * change.abs()
    assert bound < 2.0 ** -6 * change.abs() and ((dw.double() * d).sum() - change).abs() <= bound
