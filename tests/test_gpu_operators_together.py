"""The 8-bit product and the cross entropy as a program uses them: from a loss
to Kronecker factors to codes to the quantised layer, on other streams, in HIP
graphs, beyond 32-bit offsets, and the same twice.

The pipeline's steps are each held to 64-bit arithmetic on that step's own inputs,
with the roundings of its definition (e = 2^-24, a float32's half step): a product
of int8 codes rounds 3 times and once to its output; a gradient's sums of n
terms err by at most 6 sqrt(6 n) e (independent roundings, three planes) plus 2^-21
of the terms' absolute sum."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def problem(T=300, n=96, m=64, V=500, seed=3):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, n, generator=g) * torch.exp(0.5 * torch.randn(n, generator=g))
    W = torch.randn(m, n, generator=g) * (1.0 / math.sqrt(n))
    out = torch.randn(V, m, generator=g) * (2.0 / math.sqrt(m))
    y = torch.randint(0, V, (T,), generator=g)
    y[::9] = -100
    return X.cuda(), W.cuda(), out.cuda(), y.cuda()


@pytest.mark.parametrize("columns", [False, True])
def test_from_loss_to_quantised_layer(gpu_lib, columns):
    bk = gpu_lib
    X, W, out, y = problem()
    T, n = X.shape
    m, V = W.size(0), out.size(0)
    hidden = X @ W.t()
    # the loss of the unquantised layer, and its output gradients as samples
    loss, lse = bk.cross_entropy(hidden, out, y)
    g = torch.where(y >= 0, 1.0, 0.0).float()
    dY, none = bk.cross_entropy_grad(hidden, out, y, lse, g, need_dW=False)
    p = torch.softmax(hidden.double() @ out.double().T, 1)
    p[torch.arange(T, device="cuda"), y.clamp(min=0)] -= 1
    ref = (p * g.double()[:, None]) @ out.double()
    S = (p.abs() * g.double()[:, None]) @ out.double().abs()
    # p itself is off by the logits' and exponentials' roundings: below 2^-16 of it here
    assert ((dY.double() - ref).abs() <= (2.0 ** -16 + 6 * math.sqrt(6 * V) * E + 2.0 ** -21) * (S + out.double().abs().sum(0) * 2.0 ** -20)).all()
    A, B = bk.kfac_factors(X, dY, damp_rel=0.01)
    LA, LB, _, _ = bk.factor(A, B)
    if columns:
        s = (W.abs().amax(0) / 7).contiguous()
        codes = bk.solve(W, LA, LB, (-8, 7, 0), s, scale_mode=bk.SCALE_COL, check=True)
        Wq, rows, cols = codes.double() * s.double(), None, s
    else:
        s = bk.row_scales(W, 7)
        codes = bk.solve(W, LA, LB, (-8, 7, 0), s, check=True)
        Wq, rows, cols = codes.double() * s.double()[:, None], s, None
    assert codes.min() >= -8 and codes.max() <= 7
    Vq = codes.to(torch.int8)
    # the quantised layer on the same tokens
    Xq, sx = bk.quantize_tokens(X, cols)
    Y = bk.matmul_int8(Xq, sx, Vq, rows)
    ref = (Xq.double() @ codes.double().T) * sx.double()[:, None] * (1.0 if rows is None else rows.double())
    assert ((Y.double() - ref).abs() <= 4 * E * ref.abs()).all()
    # which is X Wq^T but for the tokens' rounding: half a step sx of each entry
    exact = X.double() @ Wq.T
    step = 0.5 * sx.double()[:, None] * (1 + 2.0 ** -10)
    bound = step * (codes.double().abs().sum(1) * (1.0 if rows is None else rows.double()))
    assert ((Y.double() - exact).abs() <= bound + 1e-5 * exact.abs()).all()
    # the loss through it, and its gradient back to the tokens
    loss_q, lse_q = bk.cross_entropy(Y, out, y)
    assert torch.isfinite(loss_q).all() and (loss_q[y < 0] == 0).all()
    dYq, _ = bk.cross_entropy_grad(Y, out, y, lse_q, g, need_dW=False)
    dX = bk.matmul_int8_grad(dYq, Vq, rows, cols)
    ref, S = dYq.double() @ Wq, dYq.double().abs() @ Wq.abs()
    assert ((dX.double() - ref).abs() <= (6 * math.sqrt(3 * m) + 6) * E * S).all()


def calls(bk, X, W, out, y, Vq, sv, g):
    """Every operator once; all outputs."""
    Xq, sx = bk.quantize_tokens(X)
    Y = bk.matmul_int8(Xq, sx, Vq, sv, out_dtype=torch.bfloat16)
    one = bk.matmul_int8(Xq[:1], sx[:1], Vq, sv, out_dtype=torch.bfloat16)
    O = out.bfloat16()
    loss, lse = bk.cross_entropy(Y, O, y)
    few, _ = bk.cross_entropy(Y[:3], O, y[:3])
    dY, dO = bk.cross_entropy_grad(Y, O, y, lse, g)
    dX = bk.matmul_int8_grad(dY, Vq, sv)
    f32 = bk.cross_entropy_grad(Y.float(), out, y, lse, g)
    return [Xq.clone(), sx, Y, one, loss, lse, few, dY, dO, dX, *f32]


def setup(seed=5, T=200, n=1024, m=256, V=3000):
    X, W, out, y = problem(T, n, m, V, seed)
    s = (W.abs().amax(1) / 7).contiguous()
    Vq = (W / s[:, None]).round().clamp(-8, 7).to(torch.int8)
    g = torch.where(y >= 0, 1.0 / T, 0.0).float()
    return X, W, out, y, Vq, s, g


def test_the_same_twice(gpu_lib):
    a = setup()
    first, second = calls(gpu_lib, *a), calls(gpu_lib, *a)
    assert all(torch.equal(u, v) for u, v in zip(first, second))


def test_two_streams_at_once(gpu_lib):
    """Two chains of calls on two streams, each with its own inputs, beside each
    other, against the same chains alone."""
    a, b = setup(5), setup(6)
    want = calls(gpu_lib, *a), calls(gpu_lib, *b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(calls(gpu_lib, *x))
        torch.cuda.synchronize()
        for w, r in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(w, r))


def test_captured_and_replayed(gpu_lib):
    """The whole chain in a HIP graph, replayed on new inputs with eager work in
    between, and beside it a second graph that was given the same workspace."""
    bk = gpu_lib
    static = setup(7)
    X, W, out, y, Vq, s, g = static
    calls(bk, *static)  # loads the kernels
    n = bk.lib().bakron_cross_entropy_grad_workspace_bytes(bk.F32, X.size(0), W.size(0), out.size(0))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    hidden = X @ W.t()
    lse0 = bk.cross_entropy(hidden, out, y)[1]
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got = calls(bk, *static)
        shared = bk.cross_entropy_grad(hidden, out, y, lse0, g, workspace=ws)
    with torch.cuda.graph(second):
        other = bk.cross_entropy_grad(hidden, out, y, lse0, 2 * g, workspace=ws)
    for seed in (8, 9, 10, 11):
        new = setup(seed)
        for t, v in zip(static, new):
            t.copy_(v)
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, calls(bk, *new)):
            assert torch.equal(u, v)
        for u, v in zip(shared, bk.cross_entropy_grad(hidden, out, y, lse0, g)):
            assert torch.equal(u, v)
        for u, v in zip(other, bk.cross_entropy_grad(hidden, out, y, lse0, 2 * g)):
            assert torch.equal(u, v)


def test_workspaces_are_enough(gpu_lib):
    """Workspaces of exactly the queried size, with guards behind them, and of any
    content before: a call writes nothing past them and reads nothing it has
    not written."""
    bk, L = gpu_lib, gpu_lib.lib()
    X, W, out, y, Vq, s, g = setup(12, T=150, n=1000, m=300, V=2001)
    hidden = X @ W.t()
    lse = bk.cross_entropy(hidden, out, y)[1]
    Xq, sx = bk.quantize_tokens(X)
    m, n, T, V = 300, 1000, 150, 2001
    for t, code in ((torch.float32, bk.F32), (torch.bfloat16, bk.BF16), (torch.float16, bk.F16)):
        h, o = hidden.to(t), out.to(t)
        for size, f in (
                (L.bakron_matmul_int8_workspace_bytes(T, m, n),
                 lambda w: (bk.matmul_int8(Xq, sx, Vq, s, t, workspace=w),)),
                (L.bakron_matmul_int8_grad_workspace_bytes(code, T, m, n),
                 lambda w: (bk.matmul_int8_grad(h, Vq, s, workspace=w),)),
                (L.bakron_cross_entropy_workspace_bytes(code, T, m, V), lambda w: bk.cross_entropy(h, o, y, workspace=w)),
                (L.bakron_cross_entropy_workspace_bytes(code, 9, m, V),
                 lambda w: bk.cross_entropy(h[:9], o, y[:9], workspace=w)),
                (L.bakron_cross_entropy_grad_workspace_bytes(code, T, m, V),
                 lambda w: bk.cross_entropy_grad(h, o, y, lse, g, workspace=w))):
            results = []
            for fill in (0, 255, 127):
                buf = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
                results.append([r.clone() for r in f(buf[:size])])
                assert (buf[size:] == fill).all()
            for r in results[1:]:
                assert all(torch.equal(a, b) for a, b in zip(results[0], r))


@pytest.mark.parametrize("T", [2, 70])
def test_codes_beyond_32_bits(gpu_lib, T):
    """5.2 GB of codes: the last channels, and a few others."""
    m, n = 40000, 131056
    V = torch.randint(-8, 8, (m, n), dtype=torch.int8, device="cuda")
    X = torch.randint(-127, 128, (T, n), dtype=torch.int8, device="cuda")
    sx, sv = torch.rand(T, device="cuda") + 0.5, torch.rand(m, device="cuda") + 0.5
    Y = gpu_lib.matmul_int8(X, sx, V, sv)
    at = torch.cat([torch.arange(m - 40, m), torch.tensor([0, 127, 16384, 32767, 32768])]).cuda()
    ref = X.double() @ V[at].double().T * sx.double()[:, None] * sv.double()[at]
    assert ((Y[:, at].double() - ref).abs() <= 4 * E * ref.abs()).all()


def test_vocabulary_beyond_32_bits(gpu_lib):
    """4.6 GB of output layer, and as much of its gradient."""
    bk = gpu_lib
    V, d = 1100000, 2048
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 100000):
        W[a:a + 100000] = torch.randn(min(100000, V - a), d, device="cuda") * (2.0 / math.sqrt(d))
    for T in (3, 70):
        X = torch.randn(T, d, device="cuda").bfloat16()
        y = torch.randint(V - 1000, V, (T,), device="cuda")
        y[0] = 1 << 20
        loss, lse = bk.cross_entropy(X, W, y)
        z = torch.cat([X.double() @ W[a:a + 100000].double().T for a in range(0, V, 100000)], 1)
        ref = torch.logsumexp(z, 1)
        # 2048 products of float32 sums, |terms| summing to about 60: 6 sqrt(2048) e 60 < 2^-10
        assert ((lse.double() - ref).abs() <= 2.0 ** -10).all()
        assert ((loss.double() - (ref - z.gather(1, y[:, None])[:, 0])).abs() <= 2.0 ** -9).all()
        if T == 70:
            continue
        g = torch.ones(T, device="cuda")
        dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
        D = torch.exp(z - lse.double()[:, None])
        D[torch.arange(T, device="cuda"), y] -= 1
        rows = torch.cat([torch.arange(V - 1000, V), torch.arange((1 << 20) - 5, (1 << 20) + 5)]).cuda()
        want, S = D[:, rows].T @ X.double(), D[:, rows].T.abs() @ X.double().abs()
        # D to bfloat16 2^-8 and off by its logits (2^-10), dW to bfloat16 2^-8
        assert ((dW[rows].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -9) * S + 2.0 ** -8 * want.abs()).all()
        want = sum(D[:, a:a + 100000] @ W[a:a + 100000].double() for a in range(0, V, 100000))
        S = sum(D[:, a:a + 100000].abs() @ W[a:a + 100000].double().abs() for a in range(0, V, 100000))
        assert ((dX.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -9) * S + 2.0 ** -8 * want.abs()).all()
