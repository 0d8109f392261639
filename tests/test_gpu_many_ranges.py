"""Products of few outputs over a long sum, whose k is divided over many workgroups and
joined: against 64 bits, the same twice, and the rows' other columns as they were."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24


@pytest.mark.parametrize("T,m,n", [(1, 40000, 64), (1, 100003, 3), (70, 9000, 60), (3, 30011, 129), (130, 14336, 260)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_input_gradient(gpu_lib, T, m, n, t):
    """Terms rounded to 11 bits for the 16-bit types (2^-11 each, and 2^-39 of the token's
    largest), m float32 additions of at most three planes' terms (6 sqrt(3 m) 2^-24 of their absolute sum:
    roundings are independent), the output half a step."""
    g = torch.Generator().manual_seed(T + m + n)
    G = torch.randn(T, m, generator=g).to(TYPES[t]).cuda()
    V = torch.randint(-8, 8, (m, n), generator=g, dtype=torch.int8).cuda()
    sv = (0.01 * (torch.rand(m, generator=g) + 0.5)).cuda()
    wide = torch.full((T, n + 5), 7.0, dtype=TYPES[t], device="cuda")
    out = wide[:, 2:2 + n]
    gpu_lib.matmul_int8_grad(G, V, sv, out=out)
    x = G.double() * sv.double()
    ref, S = x @ V.double(), x.abs() @ V.double().abs()
    tol = S * (6 * math.sqrt(3 * m) * E + E + (0.0 if t == "f32" else 2.0 ** -11)) + ref.abs() * torch.finfo(TYPES[t]).eps / 2
    tol += 0.0 if t == "f32" else 2.0 ** -39 * x.abs().amax(1, keepdim=True) * V.double().abs().sum(0) + 2.0 ** -25
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + n:] == 7).all()
    assert torch.equal(gpu_lib.matmul_int8_grad(G, V, sv), out)


@pytest.mark.parametrize("T,m,n", [(70, 70, 131071), (66, 3, 100000), (100, 130, 40000), (200, 64, 20011)])
def test_product(gpu_lib, T, m, n):
    """Exact sums, three float32 roundings."""
    g = torch.Generator().manual_seed(T + m + n)
    X = torch.randint(-127, 128, (T, n), generator=g, dtype=torch.int16).to(torch.int8).cuda()
    V = torch.randint(-128, 128, (m, n), generator=g, dtype=torch.int16).to(torch.int8).cuda()
    sx, sv = torch.rand(T, generator=g).cuda() + 0.5, torch.rand(m, generator=g).cuda() + 0.5
    ref = X.double() @ V.double().T * sx.double()[:, None] * sv.double()
    err = (gpu_lib.matmul_int8(X, sx, V, sv).double() - ref).abs()
    assert (err <= 3 * E * (1 + 4 * E) * ref.abs()).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_hidden_gradient_of_one_token(gpu_lib, t):
    """dX of one token with a narrow hidden state and a large vocabulary. D is rounded
    to its planes (2^-8, 2^-11 and 2^-39, 2^-24), p off by its logit (6 sqrt(6 d) 2^-24 and 2^-21 of
    the terms' absolute sum), its argument and its exponential (2^-22 + 2^-23 of at most 32)."""
    d, V = 48, 100003
    g = torch.Generator().manual_seed(9)
    X = torch.randn(1, d, generator=g).to(TYPES[t]).cuda()
    W = (torch.randn(V, d, generator=g) * (2.0 / math.sqrt(d))).to(TYPES[t]).cuda()
    y, one = torch.tensor([77777], device="cuda"), torch.ones(1, device="cuda")
    _, lse = gpu_lib.cross_entropy(X, W, y)
    dX, _ = gpu_lib.cross_entropy_grad(X, W, y, lse, one, need_dW=False)
    z, Sz = X.double() @ W.double().T, X.double().abs() @ W.double().abs().T
    p = torch.exp(z - lse.double())
    D = p.clone()
    D[0, 77777] -= 1
    kept = {"f32": E, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[t]
    dD = p * ((6 * math.sqrt(6 * d) * E + 2.0 ** -21) * Sz + 32 * E + 2.0 ** -22 + 2.0 ** -23) + kept * D.abs()
    dD += 2.0 ** -39 if t == "f16" else 0.0
    S = D.abs() @ W.double().abs()
    tol = dD @ W.double().abs() * 1.01 + (6 * math.sqrt(6 * V) * E + (2.0 ** -21 if t == "f32" else 0.0)) * S
    ref = D @ W.double()
    tol += torch.finfo(TYPES[t]).eps / 2 * ref.abs() + 2.0 ** -25
    err = (dX.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()
