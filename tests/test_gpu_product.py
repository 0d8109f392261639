"""The 8-bit product (bakron_quantize_tokens, bakron_matmul_int8) and its input
gradient (bakron_matmul_int8_grad) against plain 64-bit arithmetic.

Tolerances, counted in the roundings of the definitions. Quantisation: the
scale is one float32 division, the codes are whole numbers and equal. Product:
the int32 sum is exact; its conversion to float32 and the two scale products
round once each, and the output once, so |Y - Y64| <= (3 eps32 (1 + 2 eps32) +
eps_out) |Y64| with eps half a step (2^-24; bf16 2^-8, fp16 2^-11 relative to
the value), plus the smallest subnormal of a float16 output. Gradient: with S
the sum of the terms' absolute values, each term carries the rounding of G sv
(2^-24) and what its planes drop (bf16 and fp16: half a step of 11 bits, 2^-11
of the term, or of float16's last place under the token's power of two, 2^-39 of
the token's largest; nothing for float32, whose 24 bits are all kept), the at most 3 m float32 additions 2^-24 of S each,
the channel factor 2^-24 and the output half a step of its type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E32 = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def tokens64(X, c=None):
    """The definition in float32 steps on the CPU (numpy divides correctly
    rounded): scales and codes."""
    x = X.float().cpu().numpy()
    if c is not None:
        x = (x * c.cpu().numpy()).astype(np.float32)
    a = np.abs(x).max(axis=1, initial=0.0).astype(np.float32)
    s = np.where(a == 0, np.float32(1), (a / np.float32(127)).astype(np.float32)).astype(np.float32)
    q = np.clip(np.rint((x / s[:, None]).astype(np.float32)), -127, 127)
    return q.astype(np.int64), s


@pytest.mark.parametrize("T,n", [(1, 1), (1, 4096), (3, 17), (37, 1000), (5, 4099), (130, 256), (2, 20011),
                                 (1, 70000), (9, 64)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("channel", [False, True])
def test_quantize_tokens(gpu_lib, T, n, t, channel):
    g = torch.Generator().manual_seed(T * 31 + n)
    X = (torch.randn(T, n, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(TYPES[t])
    if T > 2:
        X[1] = 0
    c = torch.exp(0.3 * torch.randn(n, generator=g)) if channel else None
    q, s = gpu_lib.quantize_tokens(X.cuda(), None if c is None else c.cuda())
    qr, sr = tokens64(X, c)
    assert q.dtype == torch.int8 and q.shape == (T, n) and (n == 1 or q.stride(1) == 1)
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), qr)


def test_quantize_tokens_edge_values(gpu_lib):
    """Ties, the smallest values, rows with infinities and NaN, strided rows, no
    rows, no columns, and what lies around the codes."""
    bk = gpu_lib
    # ties: scale 1 exactly, halves round to even
    X = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0, 126.5]])
    q, s = bk.quantize_tokens(X.cuda())
    assert s.item() == 1.0 and q.cpu().tolist() == [[127, 0, 2, 2, 0, -2, -127, 126]]
    # subnormal rows, and the largest floats
    X = torch.tensor([[1e-44, -1e-42, 3e-43, 0.0], [1e-38, -5e-39, 2e-40, 1e-45], [3.4e38, -1e38, 1.0, 0.0]])
    q, s = bk.quantize_tokens(X.cuda())
    qr, sr = tokens64(X)
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    # a row with an infinity or a NaN, alone among its neighbours
    for bad in (float("inf"), float("-inf"), float("nan")):
        X = torch.randn(3, 70)
        X[1, 69] = bad
        q, s = bk.quantize_tokens(X.cuda())
        assert not torch.isfinite(s[1]) and torch.isfinite(s[[0, 2]]).all()
        Y = bk.matmul_int8(q, s, torch.ones(5, 70, dtype=torch.int8, device="cuda"))
        assert torch.isnan(Y[1]).all() and torch.isfinite(Y[[0, 2]]).all()
    # a slice of a wider buffer, its rows not aligned
    base = torch.randn(40, 133)
    q, s = bk.quantize_tokens(base.cuda()[:, 3:90])
    qr, sr = tokens64(base[:, 3:90])
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    # through the C ABI into a buffer wider than the codes: the rest stays
    L, buf = bk.lib(), torch.full((40, 100), 77, dtype=torch.int8, device="cuda")
    X = base[:, 3:90].contiguous().cuda()
    assert L.bakron_quantize_tokens(bk.F32, 40, 87, bk._p(X), 87, None, bk._p(buf), 100, bk._p(s),
                                    bk._stream(X.device)) == bk.OK
    assert np.array_equal(buf[:, :87].cpu().numpy(), qr) and (buf[:, 87:] == 77).all()
    q, s = bk.quantize_tokens(torch.empty(0, 8, device="cuda"))
    assert q.shape == (0, 8) and s.shape == (0,)
    q, s = bk.quantize_tokens(torch.empty(4, 0, device="cuda"))
    assert q.shape == (4, 0) and (s == 1).all()


def int8(rows, cols, g, lo=-128, hi=127, pad=0):
    """int8 values in [lo, hi] in a buffer whose rows are `pad` bytes longer,
    filled with others."""
    buf = torch.randint(-128, 128, (rows, cols + pad), generator=g, dtype=torch.int16).to(torch.int8)
    buf[:, :cols] = torch.randint(lo, hi + 1, (rows, cols), generator=g, dtype=torch.int16).to(torch.int8)
    return buf


def check_product(bk, Xb, Vb, n, sx, sv, t, out=None):
    X, V = Xb.cuda()[:, :n], Vb.cuda()[:, :n]
    Y = bk.matmul_int8(X, sx.cuda(), V, None if sv is None else sv.cuda(), out_dtype=TYPES[t], out=out)
    ref = Xb[:, :n].double() @ Vb[:, :n].double().T * sx.double()[:, None]
    if sv is not None:
        ref = ref * sv.double()
    assert Y.dtype == TYPES[t]
    err = (Y.cpu().double() - ref).abs()
    tol = ref.abs() * (3 * E32 * (1 + 2 * E32) + half_step(TYPES[t])) * (1 + E32)
    tol += {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}[t]
    assert (err <= tol).all(), (err / tol.clamp(min=1e-300)).max()
    return Y


@pytest.mark.parametrize("T,m,n", [
    (1, 1, 1), (1, 4096, 4096), (1, 1000, 1536), (2, 70, 48), (5, 33, 17), (16, 256, 512), (17, 300, 1040),
    (37, 1003, 768), (64, 512, 64), (65, 129, 4096), (130, 260, 128), (200, 1003, 1531), (128, 128, 112),
    (257, 500, 2064), (600, 1500, 96), (4, 7, 40000), (3000, 4100, 160),
])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_matmul_int8(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + 3 * m + 7 * n)
    sx = torch.exp(torch.randn(T, generator=g)) * 0.02
    sv = torch.exp(torch.randn(m, generator=g)) * 0.01
    check_product(gpu_lib, int8(T, n, g), int8(m, n, g, -8, 7), n, sx, sv, t)


@pytest.mark.parametrize("T,m,n", [
    (20, 15000, 2560), (9, 13001, 5216), (70, 9000, 2700), (128, 14000, 2689), (900, 4000, 2570), (1000, 3900, 5200),
])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_matmul_int8_few_tiles_long_rows(gpu_lib, T, m, n, t):
    """Tiles that have a CU almost to themselves and many steps of n."""
    g = torch.Generator().manual_seed(T + 3 * m + 7 * n)
    sx, sv = torch.rand(T, generator=g) + 0.5, torch.rand(m, generator=g) + 0.5
    check_product(gpu_lib, int8(T, n, g), int8(m, n, g, -8, 7), n, sx, sv, t)


@pytest.mark.parametrize("T", [5, 150])
def test_matmul_int8_rows_far_apart(gpu_lib, T):
    """Rows of codes more than 4 MB apart, all aligned; the gradient through them."""
    g = torch.Generator().manual_seed(T)
    X, V, sx, sv = int8(T, 160, g), int8(90, 160, g), torch.rand(T, generator=g) + 0.5, torch.rand(90, generator=g) + 0.5
    far = torch.full((90, 4400000), 99, dtype=torch.int8, device="cuda")
    far[:, :160] = V.cuda()
    a = gpu_lib.matmul_int8(X.cuda(), sx.cuda(), far[:, :160], sv.cuda())
    assert torch.equal(a, check_product(gpu_lib, X, V, 160, sx, sv, "f32"))
    G = torch.randn(T, 90, generator=g).cuda()
    assert torch.equal(gpu_lib.matmul_int8_grad(G, far[:, :160], sv.cuda()), gpu_lib.matmul_int8_grad(G, V.cuda(), sv.cuda()))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_matmul_int8_empty_sums_of_many_tokens(gpu_lib, t):
    e = dict(dtype=torch.int8, device="cuda")
    Y = gpu_lib.matmul_int8(torch.empty(200, 0, **e), torch.ones(200, device="cuda"), torch.empty(333, 0, **e), out_dtype=TYPES[t])
    assert Y.shape == (200, 333) and (Y == 0).all()
    D = gpu_lib.matmul_int8_grad(torch.empty(200, 0, dtype=TYPES[t], device="cuda"), torch.empty(0, 333, **e))
    assert D.shape == (200, 333) and (D == 0).all()


@pytest.mark.parametrize("T", [1, 13, 40, 150, 2500])
@pytest.mark.parametrize("n,pad", [(512, 16), (512, 3), (500, 12), (499, 0), (1, 15), (31, 1)])
def test_matmul_int8_strides(gpu_lib, T, n, pad):
    """Rows inside wider buffers whose other bytes are not zero, aligned to 16
    bytes or not, with and without row scales, into a strided output whose other
    columns stay."""
    g = torch.Generator().manual_seed(T + n + pad)
    m = 2100 if T == 2500 else 301
    sx, sv = torch.rand(T, generator=g) + 0.5, torch.rand(m, generator=g) + 0.5
    X, V = int8(T, n, g, pad=pad), int8(m, n, g, pad=pad)
    check_product(gpu_lib, X, V, n, sx, None, "f32")
    wide = torch.full((T, m + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    check_product(gpu_lib, X, V, n, sx, sv, "bf16", out=wide[:, 2:2 + m])
    assert (wide[:, :2] == 5).all() and (wide[:, 2 + m:] == 5).all()


def test_matmul_int8_largest_sums(gpu_lib):
    """Every product at its largest, at the longest rows: the int32 sum of
    131071 times 128 * 128 is 2^31 - 2^14, exact."""
    n = 131071
    X = torch.full((2, n), -128, dtype=torch.int8, device="cuda")
    V = torch.full((3, n), -128, dtype=torch.int8, device="cuda")
    V[1] = 127
    one = torch.ones(2, device="cuda")
    Y = gpu_lib.matmul_int8(X, one, V).cpu()
    for i, want in enumerate((n * 16384, -n * 16256, n * 16384)):
        assert (Y[:, i] == torch.tensor(float(want), dtype=torch.float64).float()).all()
    with pytest.raises(gpu_lib.BakronError) as e:
        gpu_lib.matmul_int8(torch.zeros(1, n + 1, dtype=torch.int8, device="cuda"), one[:1],
                            torch.zeros(1, n + 1, dtype=torch.int8, device="cuda"))
    assert e.value.status == gpu_lib.EINVAL


def test_matmul_int8_empty(gpu_lib):
    bk, e = gpu_lib, dict(dtype=torch.int8, device="cuda")
    assert bk.matmul_int8(torch.empty(0, 8, **e), torch.empty(0, device="cuda"), torch.empty(4, 8, **e)).shape == (0, 4)
    assert bk.matmul_int8(torch.empty(3, 8, **e), torch.ones(3, device="cuda"), torch.empty(0, 8, **e)).shape == (3, 0)
    Y = bk.matmul_int8(torch.empty(3, 0, **e), torch.ones(3, device="cuda"), torch.empty(5, 0, **e))
    assert Y.shape == (3, 5) and (Y == 0).all()


KEPT = {"f32": 0.0, "bf16": 2.0 ** -11, "f16": 2.0 ** -11}


def check_grad(bk, G, V, sv, c, t, out=None):
    D = bk.matmul_int8_grad(G.cuda(), V.cuda(), None if sv is None else sv.cuda(),
                            None if c is None else c.cuda(), out=out)
    m = G.shape[1]
    g = G.double() if sv is None else G.double() * sv.double()
    f = 1.0 if c is None else c.double()
    ref, S = (g @ V.double()) * f, (g.abs() @ V.double().abs()) * f
    assert D.dtype == TYPES[t]
    tol = S * (KEPT[t] + (3 * m + 4) * E32) * (1 + 2.0 ** -6) + ref.abs() * half_step(TYPES[t])
    tol += {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}[t] + 1e-40
    if t != "f32":
        tol += 2.0 ** -39 * g.abs().amax(1, keepdim=True) * V.double().abs().sum(0) * f if m else 0.0
    got = D.cpu().double()
    # float16 ends at 65504 = 2^16 - 2^5 and the rounding of anything from 2^16 - 2^4 on is infinity: a
    # result may be infinite where its value, moved by its tolerance, reaches that (float32 and bfloat16
    # end at 2^128, out of these inputs' reach)
    over = torch.isinf(got) & (got.sign() == ref.sign()) & (ref.abs() + tol >= 65520) & (t == "f16")
    err = torch.where(over, 0.0, (got - ref).abs())
    assert (err <= tol).all(), (err / tol).max()
    return D


@pytest.mark.parametrize("T,m,n", [(1, 1, 1), (1, 4096, 300), (3, 17, 65), (33, 200, 1000), (129, 64, 130),
                                   (300, 1003, 511), (1, 70, 4096), (2600, 300, 2100)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_matmul_int8_grad(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + 3 * m + 7 * n)
    G = torch.randn(T, m, generator=g).to(TYPES[t])
    sv, c = torch.exp(torch.randn(m, generator=g)), torch.exp(torch.randn(n, generator=g))
    V = int8(m, n, g)
    check_grad(gpu_lib, G, V, sv, c, t)
    check_grad(gpu_lib, G, V, None, None, t)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_matmul_int8_grad_strides(gpu_lib, t):
    """Slices of wider buffers, unaligned; a strided output whose other columns
    stay; gradients of very different sizes in one row."""
    g = torch.Generator().manual_seed(7)
    base = torch.randn(40, 101, generator=g) * 10.0 ** torch.randint(-3, 3, (40, 101), generator=g)
    G, V = base.to(TYPES[t])[:, 3:80], int8(77, 133, g)[:, 1:121]
    sv = torch.rand(77, generator=g) + 0.5
    wide = torch.full((40, 131), 9.0, dtype=TYPES[t], device="cuda")
    check_grad(gpu_lib, G, V, sv, None, t, out=wide[:, 5:125])
    assert (wide[:, :5] == 9).all() and (wide[:, 125:] == 9).all()


def test_matmul_int8_grad_edge_values(gpu_lib):
    """No rows, no outputs, no inputs; infinities and NaN stay in their rows."""
    bk, e = gpu_lib, dict(dtype=torch.int8, device="cuda")
    assert bk.matmul_int8_grad(torch.empty(0, 4, device="cuda"), torch.empty(4, 6, **e)).shape == (0, 6)
    assert bk.matmul_int8_grad(torch.empty(3, 4, device="cuda"), torch.empty(4, 0, **e)).shape == (3, 0)
    D = bk.matmul_int8_grad(torch.empty(3, 0, device="cuda"), torch.empty(0, 6, **e))
    assert D.shape == (3, 6) and (D == 0).all()
    for t in TYPES.values():
        G = torch.ones(4, 9, device="cuda", dtype=t)
        G[1, 3], G[2, 8] = float("inf"), float("nan")
        D = bk.matmul_int8_grad(G, torch.ones(9, 20, **e))
        assert (D[1] == float("inf")).all() and torch.isnan(D[2]).all() and (D[[0, 3]] == 9).all()
    # the largest floats are kept, not rounded up to infinity
    G = torch.full((1, 1), 3.4e38, device="cuda")
    assert bk.matmul_int8_grad(G, torch.ones(1, 1, **e)).item() == G.item()


def test_grad_is_the_products_derivative(gpu_lib):
    """Differences of the layer's outputs: where the tokens are whole numbers of
    steps the rounding is exact, and one step h of x[t][j] moves sum(G Y) by
    h dX[t][j]."""
    bk = gpu_lib
    g = torch.Generator().manual_seed(11)
    T, m, n = 3, 50, 40
    X = torch.randint(-100, 101, (T, n), generator=g).float() / 64
    X[:, 0] = 127.0 / 64  # fixes every token's scale at 1/64
    V, sv = int8(m, n, g, -8, 7), torch.rand(m, generator=g) + 0.5
    c = 2.0 ** torch.randint(-1, 2, (n,), generator=g).float()
    c[0] = 1.0
    X[:, 1:] = X[:, 1:] / 2  # stays below the first column under the channel factors
    X = torch.round(X * 64 * c) / 64 / c
    G = torch.randn(T, m, generator=g)

    def value(x):
        q, s = bk.quantize_tokens(x.cuda(), c.cuda())
        assert (s == 1.0 / 64).all()
        return (G.double() * bk.matmul_int8(q, s, V.cuda(), sv.cuda()).cpu().double()).sum()

    D = bk.matmul_int8_grad(G.cuda(), V.cuda(), sv.cuda(), c.cuda()).cpu().double()
    for t, j in ((0, 1), (1, 17), (2, 39), (0, 20)):
        h = 1.0 / 64 / float(c[j])
        up, down = X.clone(), X.clone()
        up[t, j] += h
        down[t, j] -= h
        slope = (value(up) - value(down)) / (2 * h)
        # each Y is off by 3 roundings of 2^-24 of itself, the slope by their sum over 2 h
        size = 2 * 3 * E32 * (G[t].abs().double() * (V.double().abs() @ (X[t].double() * c.double()).abs())
                              * sv.double()).sum()
        scale = size * 1.1 / h + 1e-6 * D[t, j].abs() + 200 * E32 * (G[t].abs().double() * sv.double()
                                                                      * V[:, j].abs().double()).sum() * float(c[j])
        assert abs(slope - D[t, j]) <= scale, (t, j)
