"""The cross entropy's workspaces where the vocabulary goes by in pieces that differ with the
operands' alignment: exactly as large as asked for, whatever they held before."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24


@pytest.mark.parametrize("T,d,V", [(5, 2048, 70001), (70, 1000, 140000)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_aligned_and_misaligned(gpu_lib, T, d, V, t):
    """The same call on aligned rows (one piece) and on misaligned ones (three, laid out), against the
    gradient in 64 bits. D is rounded to 2^-8 or 2^-11 (and 2^-39) of itself and is off by its logit (6 sqrt(d)
    2^-24 of the terms' absolute sum), its argument (2^-24 of at most 64) and its exponential (2^-22);
    the sums over at most V terms by 6 sqrt(V) 2^-24 of their absolute sum, the output by half a step."""
    bk, L = gpu_lib, gpu_lib.lib()
    code = bk.BF16 if t == "bf16" else bk.F16
    g = torch.Generator(device="cuda").manual_seed(T)
    W0 = torch.full((V, d + 9), float("nan"), dtype=TYPES[t], device="cuda")
    W0[:, 1:1 + d] = torch.randn(V, d, device="cuda", generator=g) * (2.0 / math.sqrt(d))
    X = torch.randn(T, d, device="cuda", generator=g).to(TYPES[t])
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    one = torch.ones(T, device="cuda")
    slant, W = W0[:, 1:1 + d], W0[:, 1:1 + d].contiguous()
    n = L.bakron_cross_entropy_grad_workspace_bytes(code, T, d, V)
    lse = bk.cross_entropy(X, W, y)[1]
    Wd, Xd = W.double(), X.double()
    z = Xd @ Wd.T
    p = torch.exp(z - lse.double()[:, None])
    del z
    D = p.clone()
    D[torch.arange(T, device="cuda"), y] -= 1
    kept = 2.0 ** -8 if t == "bf16" else 2.0 ** -11
    dD = p * (6 * math.sqrt(d) * E * (Xd.abs() @ Wd.abs().T) + 64 * E + 2.0 ** -22) + kept * D.abs()
    dD += 2.0 ** -39 if t == "f16" else 0.0
    half = torch.finfo(TYPES[t]).eps / 2
    tiny = 2.0 ** -25 if t == "f16" else 1e-37
    wantX, wantW = D @ Wd, D.T @ Xd
    tolX = 1.01 * (dD @ Wd.abs() + 6 * math.sqrt(V) * E * (D.abs() @ Wd.abs())) + half * wantX.abs() + tiny
    tolW = 1.01 * (dD.T @ Xd.abs() + 6 * math.sqrt(T) * E * (D.abs().T @ Xd.abs())) + half * wantW.abs() + tiny
    for w in (W, slant):
        for fill in (0, 255):
            buf = torch.full((n + 4096,), fill, dtype=torch.uint8, device="cuda")
            dX, dW = bk.cross_entropy_grad(X, w, y, lse, one, workspace=buf[:n])
            assert (buf[n:] == fill).all()
            del buf
            for got, want, tol in ((dX, wantX, tolX), (dW, wantW, tolW)):
                err = (got.double() - want).abs()
                assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("T,d,V", [(300, 64, 65000), (2000, 40, 33000), (65, 4096, 700), (130, 2056, 4000)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_forward(gpu_lib, T, d, V, t):
    """Loss and lse from workspaces of exactly the queried size, aligned rows and not: guards stay,
    and what a workspace held before makes no difference."""
    bk = gpu_lib
    dtype = dict(TYPES, f32=torch.float32)[t]
    code = {"f32": bk.F32, "bf16": bk.BF16, "f16": bk.F16}[t]
    g = torch.Generator(device="cuda").manual_seed(T)
    W0 = (torch.randn(V, d + 3, device="cuda", generator=g) * (2.0 / math.sqrt(d))).to(dtype)
    X = torch.randn(T, d, device="cuda", generator=g).to(dtype)
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    n = bk.lib().bakron_cross_entropy_workspace_bytes(code, T, d, V)
    for w in (W0[:, 3:], W0[:, 3:].contiguous()):
        ref = torch.logsumexp(X.double() @ w.double().T, 1)
        results = []
        for fill in (0, 255):
            buf = torch.full((n + 4096,), fill, dtype=torch.uint8, device="cuda")
            results.append(bk.cross_entropy(X, w, y, workspace=buf[:n]))
            assert (buf[n:] == fill).all()
        assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
        # logits' sums 6 sqrt(6 d) 2^-24 (+ 2^-21) of at most 8 sqrt(d) in absolute terms; lse's own 2^-15
        tol = (6 * math.sqrt(6 * d) * E + 2.0 ** -21) * 8 * math.sqrt(d) + 2.0 ** -15
        assert ((results[0][1].double() - ref).abs() <= tol).all()
