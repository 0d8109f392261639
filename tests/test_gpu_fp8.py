"""8-bit floating point with block scales (bakron_quantize_fp8, bakron_matmul_fp8,
bakron_matmul_fp8_grad) against plain 64-bit arithmetic.

Tolerances, counted in the roundings of the definitions. Quantisation: one float32
division for the scale and one for each code, then the nearest code: equal. Product: with
p_b a block's sum, S_b the sum of its terms' absolute values and f_b the two scales'
product, the at most 129 float32 additions of a block cut 2^-23 of S_b each, f_b
and its product with p_b round to 2^-24, and the nb additions of blocks to 2^-24 of the
sum of |f_b| S_b: 131 2^-23 + nb 2^-24 of that sum in all, plus half a step of Y's type.
Below float32 the 8-bit instructions cut, of eight neighbouring products, seven below
2^-13 of the largest: 7 2^-13 of S_b, and nothing for codes whose exponents lie within
[3, 6], whose products' bits lie within 2^13. Gradient: float32 products are exact in
three planes, each of 3 m additions rounds to 2^-23 of S, and the scales and blocks as
above; below float32 G is kept to 2^-39 of its row's largest (11 bits hold the rest)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
E32 = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def smallest(t):
    return 2.0 ** -25 if t == torch.float16 else 2.0 ** -134 if t == torch.bfloat16 else 2.0 ** -150


def blocks(n):
    return -(-n // 128)


def spread(s, rows, a, n):
    """Each block's scale at its elements."""
    return s.repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(128, -1)[..., :n]


def quantized(X, rows):
    """The definition in float32 steps on the CPU: codes (as bytes) and scales."""
    x = X.float().cpu()
    a, n = x.shape
    p = torch.zeros(-(-a // rows) * rows, blocks(n) * 128)
    p[:a, :n] = x.abs()
    top = p.view(-1, rows, blocks(n), 128).amax((1, 3)).numpy()
    s = np.where(top == 0, np.float32(1), np.maximum((top / np.float32(448)).astype(np.float32), np.float32(2.0 ** -126)))
    s = torch.from_numpy(s.astype(np.float32))
    q = torch.from_numpy((x.numpy() / spread(s, rows, a, n).numpy()).astype(np.float32))
    return q.to(F8).view(torch.uint8), s


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_any_scale(gpu_lib, rows):
    """Blocks of every size from the smallest to the largest floats, with quotients at, and one step to
    either side of, the middle between two codes."""
    g = torch.Generator().manual_seed(7)
    n = 128 * 254
    e = torch.arange(254).repeat_interleave(128)
    X = torch.ldexp(torch.rand(256, n, generator=g) + 1, (e - 126).expand(256, n).to(torch.int32))
    X = X * torch.where(torch.rand(256, n, generator=g) < 0.5, -1.0, 1.0) * torch.rand(256, n, generator=g)
    top = torch.zeros(256, 254)
    top[:] = X.view(256, 254, 128).abs().amax(2) if rows == 1 else X.view(2, 128, 254, 128).abs().amax((1, 3)).repeat_interleave(128, 0)
    s = torch.where(top == 0, torch.ones(()), (top / torch.full((), 448.0)).clamp(min=2.0 ** -126)).repeat_interleave(128, 1)
    # middles: 1 + 1/16 and so on, times the scale, and its neighbours
    mid = torch.ldexp(1 + (2 * torch.randint(0, 8, (256, n), generator=g) + 1) / 16.0, torch.randint(-9, 8, (256, n), generator=g, dtype=torch.int32)) * s
    step = torch.randint(-2, 3, (256, n), generator=g).to(torch.int32)
    near = (mid.view(torch.int32) + step).view(torch.float32)
    X = torch.where((torch.rand(256, n, generator=g) < 0.7) & (near < top.repeat_interleave(128, 1)), near, X)
    q, sc = gpu_lib.quantize_fp8(X.cuda(), rows)
    qr, sr = quantized(X, rows)
    assert torch.equal(sc.cpu(), sr)
    assert torch.equal(q.cpu().contiguous().view(torch.uint8), qr)


@pytest.mark.parametrize("a,n", [(1, 1), (1, 4096), (3, 17), (37, 1000), (5, 4099), (130, 256), (129, 385), (2, 20011),
                                 (256, 640), (300, 129)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(gpu_lib, a, n, t, rows):
    g = torch.Generator().manual_seed(a * 31 + n)
    X = (torch.randn(a, n, generator=g) * torch.exp(2 * torch.randn(a, 1, generator=g))).to(TYPES[t])
    if a > 2:
        X[1] = 0
    if n > 300:
        X[:, 128:256] = 0  # blocks of zeros, and of 128 rows too
    q, s = gpu_lib.quantize_fp8(X.cuda(), rows)
    qr, sr = quantized(X, rows)
    assert q.dtype == F8 and q.shape == (a, n) and s.shape == sr.shape
    assert torch.equal(s.cpu(), sr)
    assert torch.equal(q.cpu().contiguous().view(torch.uint8), qr)


def test_quantize_edge_values(gpu_lib):
    """Ties, subnormal and the largest values, infinities and NaN, strided rows, batches,
    no rows, no columns, and what lies around the codes."""
    bk = gpu_lib
    X = torch.tensor([[448.0, 17.0, 19.0, 18.0, -21.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -(2.0 ** -10), 0.0, 1.0625]])
    q, s = bk.quantize_fp8(X.cuda())
    assert s.item() == 1.0
    assert q.float().cpu().tolist() == [[448.0, 16.0, 20.0, 18.0, -20.0, 2.0 ** -9, 0.0, 2.0 ** -8, 0.0, 0.0, 1.0]]
    X = torch.tensor([[0.0, -0.0, -1e-9, 1.0], [-0.0, -0.0, 0.0, -0.0]])  # the sign of zero, as the division's
    q, s = bk.quantize_fp8(X.cuda())
    assert q.cpu().view(torch.uint8).tolist() == [[0, 128, 128, 126], [128, 128, 0, 128]] and s[1].item() == 1.0
    X = torch.tensor([[1e-44, -1e-42, 3e-43, 0.0], [1e-38, -5e-39, 2e-40, 1e-45], [3.4e38, -1e38, 1.0, 0.0],
                      [6e-36, 5e-37, 0.0, -1e-45]])
    for rows in (1, 128):
        q, s = bk.quantize_fp8(X.cuda(), rows)
        qr, sr = quantized(X, rows)
        assert torch.equal(s.cpu(), sr) and torch.equal(q.cpu().contiguous().view(torch.uint8), qr)
    W = torch.full((5, 300), 0x38, dtype=torch.uint8, device="cuda").view(F8)  # 1.0
    for bad in (float("inf"), float("-inf"), float("nan")):
        X = torch.randn(3, 300)
        X[1, 299] = bad
        q, s = bk.quantize_fp8(X.cuda())
        assert not torch.isfinite(s[1, 2]) and torch.isfinite(s[1, :2]).all() and torch.isfinite(s[[0, 2]]).all()
        for t in TYPES.values():
            Y = bk.matmul_fp8(q, s, W, torch.ones(1, 3, device="cuda"), out_dtype=t)
            assert torch.isnan(Y[1]).all() and torch.isfinite(Y[[0, 2]]).all()
    base = torch.randn(40, 533)
    qr, sr = quantized(base[:, 3:390], 1)
    q, s = bk.quantize_fp8(base.cuda()[:, 3:390])
    assert torch.equal(s.cpu(), sr) and torch.equal(q.cpu().contiguous().view(torch.uint8), qr)
    # into a buffer wider than the codes, scales row by row: the rest stays
    buf = torch.full((40, 500), 77, dtype=torch.uint8, device="cuda")
    sc = torch.full((40, 9), -1.0, device="cuda")
    X = base[:, 3:390].contiguous().cuda()
    assert bk.lib().bakron_quantize_fp8(bk.F32, 1, 40, 387, bk._p(X), 387, 0, 1, bk._p(buf), 500, 0, bk._p(sc), 9, 1,
                                        0, bk._stream(X.device)) == bk.OK
    assert torch.equal(buf[:, :387].cpu(), qr) and (buf[:, 387:] == 77).all()
    assert torch.equal(sc[:, :4].cpu(), sr) and (sc[:, 4:] == -1).all()
    # a batch, as one by one
    B = torch.randn(3, 130, 200, device="cuda")
    for rows in (1, 128):
        q, s = bk.quantize_fp8(B[:, :, 7:], rows)
        assert q.shape == (3, 130, 193) and s.shape == (3, 130 if rows == 1 else 2, 2)
        for z in range(3):
            qz, sz = bk.quantize_fp8(B[z, :, 7:], rows)
            assert torch.equal(q[z].view(torch.uint8), qz.view(torch.uint8)) and torch.equal(s[z], sz)
    assert bk.quantize_fp8(torch.empty(0, 8, device="cuda"))[0].shape == (0, 8)
    assert bk.quantize_fp8(torch.empty(4, 0, device="cuda"))[1].shape == (4, 0)
    assert bk.quantize_fp8(torch.empty(0, 4, 8, device="cuda"), 128)[1].shape == (0, 1, 1)


def codes(rows, cols, g, narrow, pad=0):
    """Codes in a buffer whose rows are `pad` bytes longer: any finite one, or zeros and those with
    exponents 3 to 6 (all eight fractions, both signs)."""
    if narrow:
        e = torch.randint(10, 14, (rows, cols + pad), generator=g)
        b = e * 8 + torch.randint(0, 8, (rows, cols + pad), generator=g)
        b = torch.where(torch.rand(b.shape, generator=g) < 0.1, 0, b) + 128 * torch.randint(0, 2, b.shape, generator=g)
    else:
        b = torch.randint(0, 256, (rows, cols + pad), generator=g)
        b = torch.where((b & 127) == 127, 5, b)
    return b.to(torch.uint8)


def scales(a, n, g):
    return 0.02 * torch.exp(torch.randn(a, n, generator=g))


def values(b, n):
    return b[..., :n].contiguous().view(F8).double()


def expected(x, sx, w, sw):
    """Y in 64 bits and the sum of |f_b| S_b: x T x n, w m x n values, scales by block."""
    n, m = x.size(1), w.size(0)
    X, W = x * spread(sx, 1, x.size(0), n).double(), w * spread(sw, 128, m, n).double()
    return X @ W.T, X.abs() @ W.abs().T


def tolerance(ref, S, n, t, narrow):
    tol = S * (131 * 2.0 ** -23 + blocks(n) * E32) + ref.abs() * half_step(t) * (1 + 2.0 ** -8) + smallest(t)
    if t != torch.float32 and not narrow:
        tol = tol + S * 7 * 2.0 ** -13
    return tol


def check(bk, xb, wb, n, sx, sw, t, narrow, out=None, scales_by_token=False):
    tx = sx.cuda() if scales_by_token else sx.t().contiguous().t().cuda()
    Y = bk.matmul_fp8(xb.cuda().view(F8)[:, :n], tx, wb.cuda().view(F8)[:, :n], sw.cuda(), out_dtype=TYPES[t], out=out)
    ref, S = expected(values(xb, n), sx, values(wb, n), sw)
    assert Y.dtype == TYPES[t] and Y.shape == ref.shape
    err, tol = (Y.cpu().double() - ref).abs(), tolerance(ref, S, n, TYPES[t], narrow)
    assert (err <= tol).all(), (err / tol.clamp(min=1e-300)).max()
    return Y


SIZES = [(1, 1, 1), (1, 4096, 4096), (1, 1000, 1536), (2, 70, 48), (5, 33, 17), (16, 256, 512), (17, 300, 1040),
         (37, 1003, 768), (64, 512, 64), (65, 129, 4096), (130, 260, 128), (200, 1003, 1531), (128, 128, 112),
         (257, 500, 2064), (600, 1500, 96), (4, 7, 40000), (1000, 1300, 272), (300, 384, 129), (33, 900, 255)]


@pytest.mark.parametrize("T,m,n", SIZES)
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_matmul(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + 3 * m + 7 * n)
    for narrow in (True, False):
        check(gpu_lib, codes(T, n, g, narrow), codes(m, n, g, narrow), n, scales(T, blocks(n), g) * 0.05,
              scales(blocks(m), blocks(n), g) * 0.05, t, narrow)


@pytest.mark.parametrize("pad,first", [(16, 0), (3, 0), (16, 5), (0, 1)])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_matmul_strides(gpu_lib, pad, first, T):
    """Rows longer than n, at any alignment; scales with a token's side by side; an output
    with rows further apart, what lies between them as it was."""
    g = torch.Generator().manual_seed(pad * 5 + first + T)
    n, m = 400, 210
    xb, wb = codes(T, n + first, g, True, pad)[:, first:], codes(m, n + first, g, True, pad)[:, first:]
    sx, sw = scales(T, 4, g), scales(2, 4, g)
    buf = torch.full((T, m + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    check(gpu_lib, xb, wb, n, sx, sw, "bf16", True, out=buf[:, 3:m + 3], scales_by_token=True)
    assert (buf[:, :3] == 7).all() and (buf[:, m + 3:] == 7).all()
    # slices of larger tensors, offsets off 16 bytes on the GPU too
    X, W = xb.cuda().view(F8), wb.cuda().view(F8)
    big = torch.zeros(T, n + 40, dtype=torch.uint8, device="cuda").view(F8)
    big.view(torch.uint8)[:, 7:7 + n] = X.view(torch.uint8)[:, :n]
    a = gpu_lib.matmul_fp8(big[:, 7:7 + n], sx.cuda(), W[:, :n], sw.cuda())
    b = gpu_lib.matmul_fp8(X[:, :n].contiguous(), sx.cuda(), W[:, :n].contiguous(), sw.cuda())
    assert (a - b).abs().max() <= 1e-5 * b.abs().max()


@pytest.mark.parametrize("T,m,n", [(1, 70, 129), (40, 300, 255), (300, 200, 407), (90, 500, 1531), (700, 900, 130), (257, 140, 113),
                                   (130, 260, 4097), (3600, 3600, 143), (3500, 3700, 17)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_rows_end_inside_a_group_of_16(gpu_lib, T, m, n, t):
    """Codes with rows on 16 bytes and of any length, as quantize_fp8 lays them out, NaN codes behind
    each row: the product, by experts too, and the gradient."""
    bk = gpu_lib
    g = torch.Generator().manual_seed(T + m + n)
    ld = (n + 15) // 16 * 16 + 16 * (T % 3)
    xb, wb = codes(T, n, g, True), codes(m, n, g, True)
    X, W = torch.full((T, ld), 0x7f, dtype=torch.uint8, device="cuda"), torch.full((m, ld), 0xff, dtype=torch.uint8, device="cuda")
    X[:, :n], W[:, :n] = xb.cuda(), wb.cuda()
    sx, sw = scales(T, blocks(n), g) * 0.05, scales(blocks(m), blocks(n), g) * 0.05
    big = T * m > 1 << 22  # the reference on the GPU
    u, v = (values(b, n).cuda() if big else values(b, n) for b in (xb, wb))
    a, b = (s.cuda() if big else s for s in (sx, sw))
    ref, S = expected(u, a, v, b)
    Xv, Wv = X.view(F8)[:, :n], W.view(F8)[:, :n]
    off = torch.tensor([0, T // 3, T], dtype=torch.int32).cuda()
    both, scale2 = torch.stack([W, W])[:, :, :n].view(F8), torch.stack([sw, sw]).cuda()
    assert both.stride(1) == ld
    tol = tolerance(ref, S, n, TYPES[t], True)
    for Y in (bk.matmul_fp8(Xv, sx.cuda(), Wv, sw.cuda(), out_dtype=TYPES[t]),
              bk.matmul_fp8(Xv, sx.cuda(), both, scale2, offsets=off, order=torch.arange(T, dtype=torch.int32).cuda(), out_dtype=TYPES[t])):
        assert ((Y.to(ref.device).double() - ref).abs() <= tol).all()
    G = torch.randn(T, m, generator=g).to(TYPES[t])
    V = (v.cpu() if big else v) * spread(sw, 128, m, n).double()
    H, V = (G.double().cuda(), V.cuda()) if big else (G.double(), V)
    ref, S = H @ V, H.abs() @ V.abs()
    tol = S * (3 * m * 2.0 ** -23 + 3 * E32) + ref.abs() * half_step(TYPES[t]) * (1 + 2.0 ** -8) + smallest(TYPES[t])
    for D in (bk.matmul_fp8_grad(G.cuda(), Wv, sw.cuda()), bk.matmul_fp8_grad(G.cuda(), both, scale2, offsets=off)):
        assert ((D.to(ref.device).double() - ref).abs() <= tol).all()


def test_matmul_empty(gpu_lib):
    bk = gpu_lib
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda").view(F8)
    o = lambda *s: torch.ones(*s, device="cuda")
    assert bk.matmul_fp8(z(0, 8), o(0, 1), z(5, 8), o(1, 1)).shape == (0, 5)
    assert bk.matmul_fp8(z(4, 8), o(4, 1), z(0, 8), o(0, 1)).shape == (4, 0)
    for T in (4, 200):
        Y = bk.matmul_fp8(z(T, 0), o(T, 0), z(150, 0), o(2, 0), out=torch.full((T, 150), 3.0, device="cuda"))
        assert (Y == 0).all()
        D = bk.matmul_fp8_grad(o(T, 0), z(0, 150), o(0, 2), out=torch.full((T, 150), 3.0, device="cuda"))
        assert (D == 0).all()
    for T, R in ((0, 3), (0, 300), (1, 300)):  # an order that names no token, of none
        order = torch.full((R,), T, dtype=torch.int32, device="cuda")
        for n in (400, 401):
            Y = bk.matmul_fp8(z(T, n), o(T, 4), z(130, n), torch.full((2, 4), float("nan"), device="cuda"), order=order)
            assert Y.shape == (R, 130) and (Y == 0).all()
    assert bk.matmul_fp8_grad(o(0, 5), z(5, 8), o(1, 1)).shape == (0, 8)
    assert bk.matmul_fp8_grad(o(4, 5), z(5, 0), o(1, 0)).shape == (4, 0)


def routed(T, k, E, g, drop=0.1, skew=1.0):
    """Experts of each token (distinct), some routes dropped, and the sorted order."""
    score = torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    ids = score.topk(k, 1).indices
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids


GROUPS = [(1, 1, 1, 5, 7), (1, 8, 64, 300, 400), (5, 2, 7, 130, 129), (40, 4, 16, 260, 1000), (200, 2, 3, 513, 257),
          (700, 3, 5, 200, 640), (64, 8, 130, 96, 272), (900, 1, 2, 300, 128)]


@pytest.mark.parametrize("T,k,E,m,n", GROUPS)
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ordered", [True, False])
def test_matmul_by_experts(gpu_lib, T, k, E, m, n, t, ordered):
    bk = gpu_lib
    g = torch.Generator().manual_seed(T + k + E + m + n)
    ids = routed(T, k, E, g)
    order, slots, offsets = bk.sort_tokens(ids.cuda(), E)
    off, o = offsets.tolist(), order.cpu().long()
    xb, wb = codes(T, n, g, True), codes(E * m, n, g, True).view(E, m, n)
    sx, sw = scales(T, blocks(n), g), scales(E * blocks(m), blocks(n), g).view(E, blocks(m), blocks(n))
    rows = torch.where(o >= 0, o // k, 0)
    X, S = xb.cuda().view(F8), sx.cuda()
    out = torch.full((T * k, m), 7.0, dtype=TYPES[t], device="cuda")
    if ordered:
        Y = bk.matmul_fp8(X, S, wb.cuda().view(F8), sw.cuda(), offsets=offsets, order=order, per_token=k, out=out)
    else:
        r = rows.cuda()
        Y = bk.matmul_fp8(X.view(torch.uint8)[r].view(F8), S[r], wb.cuda().view(F8), sw.cuda(), offsets=offsets, out=out)
    Y = Y.cpu().double()
    assert (Y[off[-1]:] == 7).all()
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        ref, A = expected(values(xb, n)[rows[a:b]], sx[rows[a:b]], values(wb[e], n), sw[e])
        err, tol = (Y[a:b] - ref).abs(), tolerance(ref, A, n, TYPES[t], True)
        assert (err <= tol).all(), (e, (err / tol).max())


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_odd_groups(gpu_lib, t):
    """One group with everything, all but one empty, rows outside every group before, between
    nothing and after, offsets past the rows, an order that names no token, weights of one
    layer for all groups."""
    bk = gpu_lib
    g = torch.Generator().manual_seed(5)
    R, m, n, E = 150, 140, 200, 4
    xb, wb = codes(R, n, g, True), codes(E * m, n, g, True).view(E, m, n)
    sx, sw = scales(R, 2, g), scales(E * 2, 2, g).view(E, 2, 2)
    X, S, W, SW = xb.cuda().view(F8), sx.cuda(), wb.cuda().view(F8), sw.cuda()
    each = [expected(values(xb, n), sx, values(wb[e], n), sw[e]) for e in range(E)]
    for off in ([0, 150, 150, 150, 150], [0, 0, 0, 0, 150], [0, 0, 150, 150, 150], [10, 20, 20, 90, 130],
                [0, 1, 2, 3, 4], [0, 64, 128, 150, 400], [0, 50, 40, 60, 60], [-5, 3, 3, 149, 150]):
        out = torch.full((R, m), 7.0, dtype=TYPES[t], device="cuda")
        Y = bk.matmul_fp8(X, S, W, SW, offsets=torch.tensor(off, dtype=torch.int32).cuda(), out=out).cpu().double()
        own, a = torch.full((R,), -1), 0
        for e in range(E):  # an offset below an earlier one counts as it
            a, b = max(a, min(R, off[e])), min(R, off[e + 1])
            own[a:max(a, b)] = e
        for e in range(E):
            i = own == e
            err = (Y[i] - each[e][0][i]).abs()
            assert (err <= tolerance(each[e][0][i], each[e][1][i], n, TYPES[t], True)).all(), (off, e)
        assert (Y[own < 0] == 7).all(), off
    order = torch.arange(R, dtype=torch.int32)
    order[[3, 70, 149]] = torch.tensor([-1, R, 1 << 30], dtype=torch.int32)
    off = torch.tensor([0, 40, 80, 100, 150], dtype=torch.int32).cuda()
    Y = bk.matmul_fp8(X, S, W, SW, offsets=off, order=order.cuda(), out_dtype=TYPES[t])
    plain = bk.matmul_fp8(X, S, W, SW, offsets=off, out_dtype=TYPES[t])
    plain[[3, 70, 149]] = 0
    assert torch.equal(Y, plain)
    # one layer's weights for all groups, and as one group (sums may be ordered otherwise: the definition's
    # tolerance for each)
    for w, v, o in ((W[:1].expand(E, m, n), SW[:1].expand(E, 2, 2), off),
                    (W[:1].contiguous(), SW[:1].contiguous(), off[[0, 4]].contiguous())):
        err = (bk.matmul_fp8(X, S, w, v, offsets=o, out_dtype=TYPES[t]).cpu().double() - each[0][0]).abs()
        assert (err <= tolerance(each[0][0], each[0][1], n, TYPES[t], True)).all()


def check_grad(bk, G, wb, n, sw, out=None):
    t, m = G.dtype, G.size(1)
    D = bk.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8)[:, :n], sw.cuda(), out=out)
    W = values(wb, n) * spread(sw, 128, m, n).double()
    ref, S = G.double() @ W, G.double().abs() @ W.abs()
    assert D.dtype == t and D.shape == ref.shape
    tol = S * (3 * m * 2.0 ** -23 + 3 * E32) + ref.abs() * half_step(t) * (1 + 2.0 ** -8) + smallest(t)
    if t != torch.float32 and m:
        tol = tol + G.double().abs().amax(1, keepdim=True) * 2.0 ** -39 * W.abs().sum(0)
    err = (D.cpu().double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()
    return D


@pytest.mark.parametrize("T,m,n", SIZES[:15] + [(257, 1500, 500), (700, 300, 400)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_grad(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + 3 * m + 7 * n)
    G = (torch.randn(T, m, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(TYPES[t])
    if T > 2:
        G[1] = 0
    check_grad(gpu_lib, G, codes(m, n, g, False), n, scales(blocks(m), blocks(n), g))


@pytest.mark.parametrize("pad,first", [(16, 0), (3, 0), (0, 5)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_grad_strides(gpu_lib, pad, first, t):
    g = torch.Generator().manual_seed(pad + first)
    G = torch.randn(70, 190, generator=g).to(TYPES[t])
    wb = codes(180, 300 + first, g, False, pad)[:, first:]
    buf = torch.full((70, 311), 7.0, dtype=TYPES[t], device="cuda")
    check_grad(gpu_lib, G[:, 5:185], wb, 300, scales(2, 3, g), out=buf[:, 3:303])
    assert (buf[:, :3] == 7).all() and (buf[:, 303:] == 7).all()
    # rows of whole groups of 16 that do not start on 16 bytes, of the codes, of G, of both
    wb, sw = codes(184, 304 + 7, g, False), scales(2, 3, g)
    for a, b in ((0, 0), (0, 7), (3, 0), (3, 7)):
        W, H = torch.empty(184, 320 + 7, dtype=torch.uint8), torch.empty(70, 192 + 3, dtype=TYPES[t])
        W[:, b:b + 304], H[:, a:a + 184] = wb[:, :304], G[:, 1:185]
        W, H = W.cuda()[:, b:b + 304].view(F8), H.cuda()[:, a:a + 184]
        D = gpu_lib.matmul_fp8_grad(H, W, sw.cuda())
        E = gpu_lib.matmul_fp8_grad(H.contiguous(), W.contiguous(), sw.cuda())
        V = values(wb, 304) * spread(sw, 128, 184, 304).double()
        ref, S = G[:, 1:185].double() @ V, G[:, 1:185].double().abs() @ V.abs()
        tol = S * (3 * 184 * 2.0 ** -23 + 3 * E32) + ref.abs() * half_step(TYPES[t]) * (1 + 2.0 ** -8) + smallest(TYPES[t])
        assert ((D.cpu().double() - ref).abs() <= tol).all() and ((E.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_grad_small_values(gpu_lib, t):
    """Subnormal and small gradients count as they are."""
    g = torch.Generator().manual_seed(2)
    least = 2.0 ** -24 if t == "f16" else 2.0 ** -133
    G = (torch.randint(-40, 41, (20, 256), generator=g) * least).to(TYPES[t])
    wb = torch.full((256, 64), 0x78, dtype=torch.uint8)  # 256
    wb[:, 1::2] = 0xf8
    sw = torch.full((2, 1), 2.0 ** 16 if t == "f16" else 2.0 ** 100)
    D = gpu_lib.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8), sw.cuda()).cpu().double()
    ref = G.double() @ (values(wb, 64) * sw[0, 0].double())
    assert (ref != 0).any()
    assert ((D - ref).abs() <= ref.abs() * half_step(TYPES[t])).all()  # sums of few whole multiples: exact


@pytest.mark.parametrize("T,k,E,m,n", GROUPS)
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_grad_by_experts(gpu_lib, T, k, E, m, n, t):
    bk = gpu_lib
    g = torch.Generator().manual_seed(T + k + E + m + n + 1)
    order, slots, offsets = bk.sort_tokens(routed(T, k, E, g).cuda(), E)
    off, R = offsets.tolist(), T * k
    G = torch.randn(R, m, generator=g).to(TYPES[t])
    wb = codes(E * m, n, g, False).view(E, m, n)
    sw = scales(E * blocks(m), blocks(n), g).view(E, blocks(m), blocks(n))
    out = torch.full((R, n), 7.0, dtype=TYPES[t], device="cuda")
    D = bk.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8), sw.cuda(), offsets=offsets, out=out).cpu().double()
    assert (D[off[-1]:] == 7).all()
    for e in range(E):
        a, b = off[e], off[e + 1]
        W = values(wb[e], n) * spread(sw[e], 128, m, n).double()
        ref, S = G[a:b].double() @ W, G[a:b].double().abs() @ W.abs()
        tol = S * (3 * m * 2.0 ** -23 + 3 * E32) + ref.abs() * half_step(TYPES[t]) * (1 + 2.0 ** -8) + smallest(TYPES[t])
        if t != "f32":
            tol = tol + G[a:b].double().abs().amax(1, keepdim=True) * 2.0 ** -39 * W.abs().sum(0)
        assert ((D[a:b] - ref).abs() <= tol).all(), e


def test_grad_is_the_gradient(gpu_lib):
    """Against differences of the product in 64 bits: sum(G Y) changes with each token's value as
    the gradient says (the product is linear in the tokens' values)."""
    g = torch.Generator().manual_seed(1)
    T, m, n = 6, 150, 200
    wb, sw = codes(m, n, g, False), scales(2, 2, g)
    G = torch.randn(T, m, generator=g)
    D = gpu_lib.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8), sw.cuda()).cpu().double()
    W = values(wb, n) * spread(sw, 128, m, n).double()
    X, d = torch.randn(T, n, generator=g).double(), torch.randn(T, n, generator=g).double()
    step = 2.0 ** -10
    change = ((G.double() * ((X + step * d) @ W.T)).sum() - (G.double() * ((X - step * d) @ W.T)).sum()) / (2 * step)
    bound = ((G.double().abs() @ W.abs()) * d.abs()).sum() * (3 * m + 8) * 2.0 ** -23 + 1e-9 * change.abs()
    assert ((D * d).sum() - change).abs() <= bound


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_not_finite(gpu_lib, t):
    """An infinite or NaN scale, code or gradient reaches the results it enters, and no others."""
    bk = gpu_lib
    g = torch.Generator().manual_seed(3)
    for T in (3, 90):
        xb, wb = codes(T, 300, g, True), codes(200, 300, g, True)
        xb[:, 130], wb[:, 130] = 0x40, 0x40
        sx, sw = scales(T, 3, g), scales(2, 3, g)
        xb[1, 130] = 0x7f
        Y = bk.matmul_fp8(xb.cuda().view(F8), sx.cuda(), wb.cuda().view(F8), sw.cuda(), out_dtype=TYPES[t])
        assert torch.isnan(Y[1]).all() and torch.isfinite(Y[[0, 2]]).all()
        xb[1, 130] = 0x40
        sw[1, 1] = float("nan")
        Y = bk.matmul_fp8(xb.cuda().view(F8), sx.cuda(), wb.cuda().view(F8), sw.cuda(), out_dtype=TYPES[t])
        assert torch.isnan(Y[:, 128:]).all() and torch.isfinite(Y[:, :128]).all()
        G = torch.randn(T, 200, generator=g).to(TYPES[t])
        D = bk.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8), sw.cuda())
        assert torch.isnan(D[:, 128:256]).all() and torch.isfinite(D[:, :128]).all() and torch.isfinite(D[:, 256:]).all()
        sw[1, 1] = 1.0
        for bad in (float("inf"), float("nan")):
            G[1, 150] = bad
            D = bk.matmul_fp8_grad(G.cuda(), wb.cuda().view(F8), sw.cuda())
            assert not torch.isfinite(D[1][values(wb, 300)[150].cuda() != 0]).any()
            assert torch.isfinite(D[[0, 2]]).all()
