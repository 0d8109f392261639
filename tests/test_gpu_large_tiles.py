"""The 256 x 256 tiles of every product over many steps of k, ragged in rows, columns and k,
each against 64 bits; and the tiled forward's infinities and NaN. That a size takes these tiles
is asserted, so that a change of the plan cannot move it elsewhere unseen."""
import math

import pytest
import torch

from test_gpu_entropy import Ref, inputs, within
from test_gpu_product import KEPT, TYPES

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def up(a, b):
    return -(-a // b)


def large(bk, M, N, steps, pairs=1, kmajor=False, may_split=True):
    assert steps * pairs >= 9 and bk.debug_plan(M, N, steps, pairs, kmajor, may_split)[:2] == (256, 1)


@pytest.mark.parametrize("T,m,n", [(3300, 3900, 1104), (3203, 3901, 2063), (3585, 3585, 4096)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_int8_product(gpu_lib, T, m, n, t):
    """Exact sums; the sum and two scales round to float32, then once to the output."""
    large(gpu_lib, m, T, up(n, 128))
    g = torch.Generator(device="cuda").manual_seed(T)
    X = torch.randint(-128, 128, (T, n), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    V = torch.randint(-128, 128, (m, n), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    sx = 0.01 * (torch.rand(T, generator=g, device="cuda") + 0.5)
    sv = 0.01 * (torch.rand(m, generator=g, device="cuda") + 0.5)
    ref = X.double() @ V.double().T * sx.double()[:, None] * sv.double()
    wide = torch.full((T, m + 3), 5.0, dtype=TYPES[t], device="cuda")
    for out in (None, wide[:, 1:1 + m]):  # by whole groups where aligned, and one by one
        Y = gpu_lib.matmul_int8(X, sx, V, sv, out_dtype=TYPES[t], out=out)
        tol = ref.abs() * (3 * E * (1 + 4 * E) + torch.finfo(TYPES[t]).eps / 2) * (1 + E) + (2.0 ** -25 if t == "f16" else 0.0)
        err = (Y.double() - ref).abs()
        assert (err <= tol).all(), (err / tol.clamp(min=1e-300)).max()
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + m:] == 5).all()


@pytest.mark.parametrize("T,m,n", [(3601, 907, 3999), (3588, 1024, 3588)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_input_gradient(gpu_lib, T, m, n, t):
    """Terms of 11 bits for the 16-bit types (and 2^-39 of the token's largest), 3 m float32 additions (6
    sqrt(3 m) 2^-24 of their absolute sum), the channel factor, the output half a step."""
    large(gpu_lib, n, T, up(m, 64), 3 if t == "f32" else 1, True)
    g = torch.Generator(device="cuda").manual_seed(T)
    G = torch.randn(T, m, generator=g, device="cuda").to(TYPES[t])
    V = torch.randint(-8, 8, (m, n), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    sv = torch.exp(torch.randn(m, generator=g, device="cuda")) * 0.01
    c = torch.rand(n, generator=g, device="cuda") + 0.5
    D = gpu_lib.matmul_int8_grad(G, V, sv, c)
    x = G.double() * sv.double()
    ref, S = x @ V.double() * c.double(), x.abs() @ V.double().abs() * c.double()
    tol = S * (KEPT[t] + (6 * math.sqrt(3 * m) + 4) * E) * 1.01 + ref.abs() * torch.finfo(TYPES[t]).eps / 2
    if t != "f32":
        tol += 2.0 ** -39 * x.abs().amax(1, keepdim=True) * (V.double().abs().sum(0) * c.double()) + 2.0 ** -25
    err = (D.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()


def check(bk, X, W, y, g, t):
    loss, lse = bk.cross_entropy(X, W, y)
    dX, dW = bk.cross_entropy_grad(X, W, y, lse, g)
    torch.cuda.empty_cache()
    r = Ref(X, W, y, g, t, lse)
    for got, ref, tol, what in ((lse, r.lse, r.lse_tol, "lse"), (loss, r.loss, r.loss_tol, "loss"),
                                (dX, r.dX, r.dX_tol, "dX"), (dW, r.dW, r.dW_tol, "dW")):
        within(got, ref, tol, what)


@pytest.mark.parametrize("d", [1000, 1003])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_logits(gpu_lib, d, t):
    """The forward and D (in 16 bit with odd d: as planes)."""
    T, V = 3300, 4100
    large(gpu_lib, V, T, up(d, 64), 6 if t == "f32" else 1, may_split=False)
    check(gpu_lib, *inputs(T, d, V, t, 1), t)


@pytest.mark.parametrize("T,d,V", [(4100, 3300, 1001), (3588, 3592, 1024)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_hidden_gradient(gpu_lib, T, d, V, t):
    large(gpu_lib, d, T, up(V, 64), 6 if t == "f32" else 1, True)
    check(gpu_lib, *inputs(T, d, V, t, 2, even=False), t)


@pytest.mark.parametrize("T,d,V", [(1101, 3300, 4001), (1088, 3592, 3588)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_output_layer_gradient(gpu_lib, T, d, V, t):
    large(gpu_lib, d, V, up(T, 64), 6 if t == "f32" else 1, True)
    check(gpu_lib, *inputs(T, d, V, t, 3, even=False), t)


@pytest.mark.parametrize("t,V", [("f32", 11901), ("bf16", 33403), ("f16", 33403)])
def test_hidden_gradient_over_pieces(gpu_lib, t, V):
    """dX summed over two pieces of the vocabulary: a piece holds 256 MiB of D's planes, 32768 words
    of 4100 tokens in 16 bits and a third in float32."""
    T, d, pairs = 4100, 3304, 6 if t == "f32" else 1
    piece = (256 << 20) // (2 * T * (3 if t == "f32" else 1)) // 256 * 256
    assert piece < V < 2 * piece
    large(gpu_lib, d, T, up(V - piece, 64), pairs, True)
    large(gpu_lib, d, T, up(piece, 64), pairs, True)
    check(gpu_lib, *inputs(T, d, V, t, 4), t)


@pytest.mark.parametrize("T", [6, 70, 300, 3500])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_infinite_logits(gpu_lib, T, t):
    """Logits of -inf add nothing, a logit of +inf or NaN makes its token NaN and no other, at every
    kind of forward kernel. Above 64 tokens a float32 infinity may make the logits it enters NaN."""
    V = 4100 if T == 3500 else 300
    if T == 3500:
        large(gpu_lib, V, T, 9, 1, may_split=False)
    X = torch.zeros(T, 576, dtype=TYPES[t], device="cuda")
    W = torch.zeros(V, 576, dtype=TYPES[t], device="cuda")
    X[:, 1] = 1.0
    W[:, 1] = float("-inf")  # all but two entries
    W[3, 1], W[V - 1, 1] = 0.0, 0.0
    y = torch.full((T,), 3, device="cuda")
    split = t == "f32" and T > 64
    loss, lse = gpu_lib.cross_entropy(X, W, y)
    ok = (loss.double() - math.log(2)).abs() <= 2.0 ** -20
    assert (ok | torch.isnan(loss)).all() if split else ok.all()
    # one token of NaN, one whose logit V - 1 is +inf
    W[:, 1] = 0.0
    X[2, 5] = float("nan")
    X[4, 7], W[V - 1, 7] = float("inf"), 1.0
    loss, lse = gpu_lib.cross_entropy(X, W, y)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[2] = bad[4] = True
    assert torch.isnan(loss[bad]).all() and torch.isnan(lse[bad]).all()
    # 0 times that infinity is NaN too, in every row of W; else only log V is left
    assert ((loss[~bad].double() - math.log(V)).abs() <= 2.0 ** -15).all()
    # without a target its loss is 0 all the same
    y[2] = y[4] = -100
    loss, lse = gpu_lib.cross_entropy(X, W, y)
    assert (loss[bad] == 0).all() and torch.isnan(lse[bad]).all()
