"""The cross entropy (bakron_cross_entropy, bakron_cross_entropy_grad) against
plain 64-bit arithmetic on the same inputs.

Tolerances. With e = 2^-24 and S the sum of a product's absolute terms, n float32
additions err by at most 6 sqrt(n) e S (roundings are independent and each at
most e of a partial sum, itself at most S: six standard deviations of their
sum). A float32 product drops the plane pairs below 2^-21 of each term, and adds
6 terms for each. Logits: dz = 6 sqrt(n) e S_z (+ 2^-21 S_z for float32). lse: dz,
then each exponential's relative error (its argument a is rounded twice and log2 e once, 3 e |a|,
and the instruction is off by at most 2^-22), the additions (no more than 200
in a row at these sizes, 2^-16 at most), the logarithm and the last addition
(2^-22 of their size). loss: that and the target's dz. D: p times (dz + the
exponential's error, its lse being given), then what its planes drop: 2^-8 of D for
bf16, 2^-11 (and 2^-39, float16's last place under the scale 2^14) for fp16, 2^-24 for
float32. dX, dW: D's errors through the product, its additions, the factor g
(and for dW g relative to its largest, rounded to the type with X: 2^-8,
2^-11, 2^-24 where g varies), and half a step of the output's type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24
KEPT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
DROPPED = {"f32": 2.0 ** -21, "bf16": 0.0, "f16": 0.0}


def adds(n, t):
    return 6 * math.sqrt(6 * n if t == "f32" else n) * E + DROPPED[t]


class Ref:
    """Everything in 64 bits, with the tolerances above, on the inputs' device."""

    def __init__(self, X, W, y, g, t, lse=None):
        X, W = X.double(), W.double()
        T, V, d = X.shape[0], W.shape[0], X.shape[1]
        z, Sz = X @ W.T, X.abs() @ W.abs().T
        self.lse = torch.logsumexp(z, 1)
        has = (y >= 0) & (y < V)
        zy = z.gather(1, torch.where(has, y, 0)[:, None]).squeeze(1)
        self.loss = torch.where(has, self.lse - zy, 0.0)
        dz = adds(d, t) * Sz + 1e-37
        dzm = dz.amax(1)
        spread = (z - z.amax(1, keepdim=True)).abs().amax(1)
        self.lse_tol = dzm + 3 * E * spread + 2.0 ** -22 + 2.0 ** -16 + 2.0 ** -22 * (self.lse.abs() + math.log(V))
        self.loss_tol = torch.where(has, self.lse_tol + dzm + 2 * E * self.loss.abs(), 0.0)
        l = self.lse if lse is None else lse.double()
        a = z - l[:, None]
        p = torch.exp(a)
        D = p.clone()
        D[has.nonzero().squeeze(1), y[has]] -= 1
        D[~has] = 0
        w = torch.where(has, g.double(), 0.0)
        dD = p * (dz + 3 * E * a.abs() + E * z.abs() + 2.0 ** -22) + E * D.abs()
        dD = dD + (KEPT[t] * D.abs() + (2.0 ** -39 if t == "f16" else 0.0))
        dD[~has] = 0
        out = torch.finfo(TYPES[t]).eps / 2
        tiny = 2.0 ** -25 if t == "f16" else 1e-37
        self.dX = w[:, None] * (D @ W)
        self.dX_tol = (w.abs()[:, None] * (dD @ W.abs() + (adds(V, t) + 2 * E) * (D.abs() @ W.abs())) * 1.01
                       + out * self.dX.abs() + tiny)
        Xh = torch.where(has[:, None], X, 0.0)
        self.dW = D.T @ (w[:, None] * Xh)
        even = w[has].unique().numel() <= 1
        wX = (w[:, None] * Xh).abs()
        # below float16's normal range g relative to its largest, times X, errs by 2^-25 of the largest
        low = 2.0 ** -25 * w.abs().max() * D.abs().sum(0)[:, None] if t == "f16" and not even else 0.0
        self.dW_tol = ((dD.T @ wX + (adds(max(T, 1), t) + 3 * E + (0.0 if even else 1.01 * KEPT[t]))
                        * (D.abs().T @ wX) + low) * 1.01 + out * self.dW.abs() + tiny)


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, (err / tol).max().item())


def check(bk, X, W, y, g, t):
    loss, lse = bk.cross_entropy(X, W, y)
    r = Ref(X, W, y, g, t, lse)
    assert loss.dtype == lse.dtype == torch.float32
    within(lse, r.lse, r.lse_tol, "lse")
    within(loss, r.loss, r.loss_tol, "loss")
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
    assert dX.dtype == dW.dtype == X.dtype
    within(dX, r.dX, r.dX_tol, "dX")
    within(dW, r.dW, r.dW_tol, "dW")
    return loss, lse, dX, dW


def inputs(T, d, V, t, seed, masked=0.2, even=True):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, d, generator=g).to(TYPES[t])
    W = (torch.randn(V, d, generator=g) * (2.0 / math.sqrt(d))).to(TYPES[t])
    y = torch.randint(0, V, (T,), generator=g)
    off = torch.rand(T, generator=g) < masked
    y = torch.where(off, torch.where(torch.rand(T, generator=g) < 0.5, -100, V + 7), y)
    w = torch.full((T,), 1.0 / max(T, 1)) if even else torch.randn(T, generator=g) * 2.0 ** torch.randint(-6, 6, (T,), generator=g)
    return X.cuda(), W.cuda(), y.cuda(), w.float().cuda()


@pytest.mark.parametrize("T,d,V", [(1, 1, 1), (1, 64, 1000), (3, 17, 5), (37, 40, 1003), (130, 128, 300),
                                   (257, 100, 515), (64, 256, 4100), (5, 512, 20000), (700, 72, 257), (2, 8, 2),
                                   (1, 2048, 3001), (16, 999, 640), (17, 130, 4097), (48, 520, 1000), (33, 96, 31),
                                   (64, 2056, 2000), (65, 64, 1023)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("even", [True, False])
def test_cross_entropy(gpu_lib, T, d, V, t, even):
    check(gpu_lib, *inputs(T, d, V, t, T + d + V, even=even), t)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_pieces_of_the_vocabulary(gpu_lib, t):
    """More than one piece in the gradient (and large tiles)."""
    check(gpu_lib, *inputs(4096, 48, 33001, t, 5), t)


def test_pieces_of_float32_planes(gpu_lib):
    """More than one piece of W's planes in the forward call."""
    X, W, y, g = inputs(65, 4096, 30001, "f32", 6, masked=0.0)
    loss, lse = gpu_lib.cross_entropy(X, W, y)
    r = Ref(X, W, y, g, "f32")
    within(lse, r.lse, r.lse_tol, "lse")
    within(loss, r.loss, r.loss_tol, "loss")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_strides(gpu_lib, t):
    """Rows of wider buffers (the rest NaN), aligned to 16 bytes or not."""
    for first, extra in ((0, 8), (8, 16), (3, 2), (0, 1)):
        X, W, y, g = inputs(70, 96, 310, t, 9)
        wide = lambda m: torch.full((m.size(0), first + 96 + extra), float("nan"), dtype=m.dtype, device="cuda")
        Xw, Ww = wide(X), wide(W)
        Xw[:, first:first + 96], Ww[:, first:first + 96] = X, W
        check(gpu_lib, Xw[:, first:first + 96], Ww[:, first:first + 96], y, g, t)


def test_strided_outputs_through_the_abi(gpu_lib):
    """dX and dW inside wider buffers whose other columns stay."""
    bk, L = gpu_lib, gpu_lib.lib()
    for t, code in (("f32", bk.F32), ("bf16", bk.BF16), ("f16", bk.F16)):
        X, W, y, g = inputs(33, 50, 130, t, 4)
        loss, lse = bk.cross_entropy(X, W, y)
        dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
        wx = torch.full((33, 57), 3.0, dtype=X.dtype, device="cuda")
        ww = torch.full((130, 53), 3.0, dtype=X.dtype, device="cuda")
        n = L.bakron_cross_entropy_grad_workspace_bytes(code, 33, 50, 130)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        vx, vw = wx[:, 4:54], ww[:, 1:51]
        assert L.bakron_cross_entropy_grad(code, 33, 50, 130, bk._p(X), 50, bk._p(W), 50, bk._p(y), bk._p(lse),
                                           bk._p(g), bk._p(vx), 57, bk._p(vw), 53, bk._p(ws), n,
                                           bk._stream(X.device)) == bk.OK
        assert torch.equal(vx, dX) and torch.equal(vw, dW)
        assert (wx[:, :4] == 3).all() and (wx[:, 54:] == 3).all()
        assert (ww[:, :1] == 3).all() and (ww[:, 51:] == 3).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_tokens_without_targets(gpu_lib, t):
    """They take no part, whatever they hold: NaN hidden states, g and lse."""
    bk = gpu_lib
    X, W, y, g = inputs(50, 64, 200, t, 3, masked=0.0)
    y[::5] = torch.tensor([-100, -1, 200, 1 << 40, -(1 << 62)] * 2, device="cuda")
    keep = (y >= 0) & (y < 200)
    loss, lse = bk.cross_entropy(X, W, y)
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
    X2, g2 = X.clone(), g.clone()
    X2[~keep], g2[~keep] = float("nan"), float("nan")
    X2[5], g2[5] = float("inf"), float("inf")
    loss2, lse2 = bk.cross_entropy(X2, W, y)
    dX2, dW2 = bk.cross_entropy_grad(X2, W, y, lse2, g2)
    assert (loss2[~keep] == 0).all() and torch.equal(loss, loss2) and torch.equal(lse[keep], lse2[keep])
    assert (dX2[~keep] == 0).all() and torch.equal(dX[keep], dX2[keep]) and torch.equal(dW, dW2)
    # no token has a target
    none = torch.full((50,), -100, device="cuda")
    loss, lse = bk.cross_entropy(X, W, none)
    dX, dW = bk.cross_entropy_grad(X, W, none, lse, g)
    assert (loss == 0).all() and (dX == 0).all() and (dW == 0).all() and torch.isfinite(lse).all()
    # every g zero
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, torch.zeros_like(g))
    assert (dX == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_large_and_infinite_logits(gpu_lib, t):
    """Logits far apart (no overflow; a certain target has loss 0), logits of
    -inf, and tokens with a NaN."""
    bk = gpu_lib
    X = torch.zeros(6, 8, dtype=TYPES[t], device="cuda")
    W = torch.zeros(300, 8, dtype=TYPES[t], device="cuda")
    X[:, 0] = torch.tensor([1.0, 100.0, -100.0, 1.0, 0.0, 1.0])
    W[7, 0], W[290, 0] = 200.0, -200.0
    y = torch.tensor([7, 7, 290, 290, 5, 0], device="cuda")
    loss, lse = bk.cross_entropy(X, W, y)
    want = torch.tensor([0.0, 0.0, 0.0, 400.0, math.log(300), 200.0], dtype=torch.float64)
    assert ((loss.cpu().double() - want).abs() <= 2.0 ** -15 + 2.0 ** -21 * want).all()
    check(bk, X, W, y, torch.ones(6, device="cuda"), t)
    X[:, 1] = 1.0
    W[:, 1] = float("-inf")  # all but two entries
    W[3, 1], W[299, 1] = 0.0, 0.0
    loss, lse = bk.cross_entropy(X, W, torch.full((6,), 3, device="cuda"))
    if t == "f32":  # an infinity in an operand may give NaN
        loss = torch.where(torch.isnan(loss), math.log(2), loss)
    want = torch.full((6,), math.log(2), dtype=torch.float64)
    assert ((loss.cpu().double() - want).abs() <= 2.0 ** -16).all()
    X[2, 5] = float("nan")
    loss, lse = bk.cross_entropy(X, W, torch.full((6,), 3, device="cuda"))
    assert torch.isnan(loss[2]) and torch.isnan(lse[2]) and torch.isfinite(loss[[0, 1, 3, 4, 5]]).all()


def test_one_gradient_at_a_time(gpu_lib):
    bk = gpu_lib
    X, W, y, g = inputs(40, 64, 500, "bf16", 8)
    _, lse = bk.cross_entropy(X, W, y)
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
    a, none = bk.cross_entropy_grad(X, W, y, lse, g, need_dW=False)
    assert none is None and torch.equal(a, dX)
    none, b = bk.cross_entropy_grad(X, W, y, lse, g, need_dX=False)
    assert none is None and torch.equal(b, dW)
    assert bk.cross_entropy_grad(X, W, y, lse, g, False, False) == (None, None)


def test_empty(gpu_lib):
    bk = gpu_lib
    X, W = torch.empty(0, 6, device="cuda"), torch.randn(9, 6, device="cuda")
    y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = bk.cross_entropy(X, W, y)
    assert loss.shape == lse.shape == (0,)
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, f)
    assert dX.shape == (0, 6) and dW.shape == (9, 6) and (dW == 0).all()
    loss, lse = bk.cross_entropy(torch.empty(3, 0, device="cuda"), torch.empty(9, 0, device="cuda"),
                                 torch.tensor([0, 8, -100], device="cuda"))
    assert (lse.cpu().double() - math.log(9)).abs().max() <= 2.0 ** -15 and loss[2] == 0


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_no_hidden_size_and_many_tokens(gpu_lib, t):
    X, W = torch.empty(150, 0, dtype=TYPES[t], device="cuda"), torch.empty(300, 0, dtype=TYPES[t], device="cuda")
    loss, lse = gpu_lib.cross_entropy(X, W, torch.arange(150, device="cuda"))
    for v in (loss, lse):  # every logit is 0
        assert (v.cpu().double() - math.log(300)).abs().max() <= 2.0 ** -15
    dX, dW = gpu_lib.cross_entropy_grad(X, W, torch.arange(150, device="cuda"), lse, torch.ones(150, device="cuda"))
    assert dX.shape == (150, 0) and dW.shape == (300, 0)


@pytest.mark.parametrize("T", [9, 90])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_rows_far_apart(gpu_lib, T, t):
    """Rows of W more than 4 MB apart, all aligned."""
    X, W, y, g = inputs(T, 72, 130, t, T)
    far = torch.full((130, 2200000), float("nan"), dtype=TYPES[t], device="cuda")
    far[:, :72] = W
    check(gpu_lib, X, far[:, :72], y, g, t)


@pytest.mark.parametrize("T,V", [(5, 700), (140, 300)])
def test_gradient_is_the_losses_derivative(gpu_lib, T, V):
    """Differences of the 64-bit loss along random directions against the float32
    gradient: central, so off by h^2 / 6 times a third derivative of at most
    |v|^3 of the logits' changes."""
    X, W, y, g = inputs(T, 32, V, "f32", 12)
    _, lse = gpu_lib.cross_entropy(X, W, y)
    dX, dW = gpu_lib.cross_entropy_grad(X, W, y, lse, g)
    gen = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randn(X.shape, dtype=torch.float64, device="cuda", generator=gen)
    B = torch.randn(W.shape, dtype=torch.float64, device="cuda", generator=gen) * 0.1
    h = 1e-4

    def value(s):
        r = Ref(X.double() + s * A, W.double() + s * B, y, g, "f32")
        return (r.loss * g.double()).sum()

    slope = (value(h) - value(-h)) / (2 * h)
    got = (dX.double() * A).sum() + (dW.double() * B).sum()
    r = Ref(X, W, y, g, "f32", lse)
    change = (A @ W.double().T + X.double() @ B.T).abs().amax(1) + h * (A @ B.T).abs().amax(1)
    cubic = (g.abs().double() * (2 * change) ** 3).sum() * h * h
    cross = (g.abs().double() * 6 * (2 * change) * (A @ B.T).abs().amax(1)).sum() * h * h
    tol = (r.dX_tol * A.abs()).sum() + (r.dW_tol * B.abs()).sum() + cubic + cross + 1e-9
    assert abs(slope - got) <= tol
