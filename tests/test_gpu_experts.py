"""The tokens of experts: bakron_sort_tokens, bakron_gather_tokens,
bakron_combine_tokens and its gradient, against plain arithmetic.

Sorting and gathering are exact. The weighted sum of k rows rounds to 2^-24 of the
terms' absolute sum for each of its k terms, and once to the output's type; a gradient
row is one product, rounded twice; a weight's gradient has n terms and float32 sums: n 2^-24
of their absolute sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E32 = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def smallest(t):
    return 2.0 ** -25 if t == torch.float16 else 2.0 ** -134 if t == torch.bfloat16 else 2.0 ** -150


def sorted_routes(ids, E):
    """order, slots, offsets by a stable sort."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    key, order = key.sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1))
    slots = torch.full_like(order, -1)
    slots[order] = torch.where(key < E, torch.arange(order.numel()), -1)
    return torch.where(key < E, order, -1).int(), slots.view(ids.shape).int(), offsets.int()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (2, 3, 5), (100, 4, 16), (255, 8, 256), (256, 8, 1024),
                                   (257, 8, 1000), (1000, 6, 60), (4096, 1, 3), (8192, 8, 128), (5, 7, 1024),
                                   (100003, 6, 37), (0, 4, 9), (3, 1, 63), (3000, 2, 64)])
def test_sort(gpu_lib, T, k, E):
    g = torch.Generator().manual_seed(T * 3 + k + E)
    ids = torch.randint(0, E, (T, k), generator=g)
    drop = torch.rand(T, k, generator=g)
    ids = torch.where(drop < 0.05, -1, torch.where(drop < 0.08, E, torch.where(drop < 0.1, 1 << 40, ids)))
    got = gpu_lib.sort_tokens(ids.cuda(), E)
    for a, b in zip(got, sorted_routes(ids, E)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b)


@pytest.mark.parametrize("value", [0, 6, -1, 7, -(1 << 62)])
def test_sort_one_expert(gpu_lib, value):
    """All routes to one expert, or all dropped."""
    for T in (3, 3000):
        ids = torch.full((T, 2), value, dtype=torch.int64)
        for a, b in zip(gpu_lib.sort_tokens(ids.cuda(), 7), sorted_routes(ids, 7)):
            assert torch.equal(a.cpu(), b)


def test_sort_strided(gpu_lib):
    ids = torch.randint(-1, 20, (700, 9), generator=torch.Generator().manual_seed(1))
    for a, b in zip(gpu_lib.sort_tokens(ids.cuda()[:, 2:7], 20), sorted_routes(ids[:, 2:7], 20)):
        assert torch.equal(a.cpu(), b)


def problem(T, k, E, n, t, seed, drop=0.2):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices
    ids[torch.rand(T, k, generator=g) < drop] = -1
    order, slots, offsets = sorted_routes(ids, E)
    X = torch.randn(T, n, generator=g).to(t)
    Ys = torch.randn(T * k, n, generator=g).to(t)
    w = torch.rand(T, k, generator=g)
    return order, slots, offsets, X, Ys, w


SIZES = [(1, 1, 1, 1), (1, 8, 64, 2048), (3, 2, 4, 7), (50, 6, 10, 1531), (33, 5, 9, 2056), (20, 9, 16, 4100),
         (7, 3, 3, 20000), (300, 8, 32, 64), (129, 1, 5, 513), (2, 17, 40, 100)]


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("t", list(TYPES))
def test_gather(gpu_lib, T, k, E, n, t):
    order, slots, _, X, _, _ = problem(T, k, E, n, TYPES[t], T + n)
    Xs = gpu_lib.gather_tokens(X.cuda(), order.cuda(), k)
    assert torch.equal(Xs.cpu(), torch.where((order >= 0)[:, None], X[(order.long() // k).clamp(min=0)], 0))
    # strided, unaligned rows, into a wider buffer, fewer rows than routes
    if n > 4:
        buf = torch.full((order.numel(), n + 3), 7.0, dtype=TYPES[t], device="cuda")
        gpu_lib.gather_tokens(X.cuda()[:, 1:n - 1], order.cuda(), k, out=buf[:, 2:n])
        assert torch.equal(buf[:, 2:n].cpu(), Xs.cpu()[:, 1:n - 1]) and (buf[:, :2] == 7).all() and (buf[:, n:] == 7).all()
    part = order[:order.numel() // 2].contiguous()
    assert torch.equal(gpu_lib.gather_tokens(X.cuda(), part.cuda(), k), Xs[:part.numel()])


def test_gather_names_no_token(gpu_lib):
    order = torch.tensor([0, -1, 5, 6, 1 << 30, -(1 << 31), 3], dtype=torch.int32).cuda()
    X = torch.randn(3, 40, device="cuda")
    Xs = gpu_lib.gather_tokens(X, order, 2)
    zero = torch.zeros(40, device="cuda")
    assert torch.equal(Xs, torch.stack([X[0], zero, X[2], zero, zero, zero, X[1]]))
    assert (gpu_lib.gather_tokens(X[:0], order) == 0).all()
    assert gpu_lib.gather_tokens(X, order[:0]).shape == (0, 40)
    assert gpu_lib.gather_tokens(X[:, :0], order).shape == (7, 0)


def combined(Ys, slots, w):
    has = (slots >= 0) & (slots < Ys.size(0))
    y = torch.where(has[:, :, None], Ys.double()[slots.long().clamp(0, max(Ys.size(0) - 1, 0))], 0.0)
    terms = y * (1.0 if w is None else w.double()[:, :, None])
    return terms.sum(1), terms.abs().sum(1)


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(gpu_lib, T, k, E, n, t, weighted):
    _, slots, _, _, Ys, w = problem(T, k, E, n, TYPES[t], T + n)
    w = w if weighted else None
    for a in (0, 1) if n > 4 else (0,):
        y = Ys[:, a:]
        Y = gpu_lib.combine_tokens(Ys.cuda()[:, a:], slots.cuda(), None if w is None else w.cuda())
        ref, S = combined(y, slots, w)
        assert Y.dtype == TYPES[t] and Y.shape == ref.shape
        tol = S * k * E32 + ref.abs() * half_step(TYPES[t]) * (1 + 2.0 ** -8) + smallest(TYPES[t])
        assert ((Y.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(gpu_lib, T, k, E, n, t, weighted):
    _, slots, offsets, X, Ys, w = problem(T, k, E, n, TYPES[t], T + n)
    w, G, t = w if weighted else None, X, TYPES[t]
    R = int(offsets[-1])
    for a in (0, 1) if n > 4 else (0,):
        dYs, dw = gpu_lib.combine_tokens_grad(G.cuda()[:, a:], Ys.cuda()[:, a:], slots.cuda(),
                                              None if w is None else w.cuda())
        g, y = G[:, a:].double(), Ys[:, a:].double()
        has = slots >= 0
        terms = torch.where(has[:, :, None], y[slots.long().clamp(min=0)], 0.0) * g[:, None]
        assert dw.dtype == torch.float32
        assert ((dw.cpu().double() - terms.sum(2)).abs() <= terms.abs().sum(2) * n * E32 + 2.0 ** -149).all()
        assert (dw.cpu()[~has] == 0).all()
        ref = torch.zeros(T * k, g.size(1), dtype=torch.float64)
        ref[slots[has].long()] = (g[:, None] * (torch.ones(T, k) if w is None else w).double()[:, :, None])[has]
        err = (dYs.cpu().double() - ref).abs()[:R]
        assert (err <= ref[:R].abs() * (E32 + half_step(t)) * (1 + 2.0 ** -8) + smallest(t)).all()
        only, none = gpu_lib.combine_tokens_grad(G.cuda()[:, a:], Ys.cuda()[:, a:], slots.cuda(),
                                                 None if w is None else w.cuda(), need_dweights=False)
        assert none is None and torch.equal(only[:R], dYs[:R])
        none, only = gpu_lib.combine_tokens_grad(G.cuda()[:, a:], Ys.cuda()[:, a:], slots.cuda(),
                                                 None if w is None else w.cuda(), need_dYs=False)
        assert none is None and torch.equal(only, dw)


def test_combine_grad_against_differences(gpu_lib):
    """sum(G Y) changes with Ys and with the weights as the gradients say."""
    _, slots, offsets, G, Ys, w = problem(20, 4, 6, 90, torch.float32, 3)
    R = int(offsets[-1])
    dYs, dw = (x.cpu().double() for x in gpu_lib.combine_tokens_grad(G.cuda(), Ys.cuda(), slots.cuda(), w.cuda()))
    f = lambda y, v: (G.double() * combined(y, slots, v)[0]).sum()
    g = torch.Generator().manual_seed(4)
    dy, dv = torch.randn(Ys.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
    h = 2.0 ** -8
    a = (f(Ys.double() + h * dy, w) - f(Ys.double() - h * dy, w)) / (2 * h)
    b = (f(Ys, w.double() + h * dv) - f(Ys, w.double() - h * dv)) / (2 * h)
    assert ((dYs[:R] * dy[:R]).sum() - a).abs() <= (dYs[:R] * dy[:R]).abs().sum() * 2 * E32 + 1e-9
    assert ((dw * dv).sum() - b).abs() <= (G.double().abs().sum() * Ys.double().abs().max() * dv.abs().max()) * 90 * E32


def test_combine_takes_no_part(gpu_lib):
    """Slots outside the rows are not read, whatever their weights are; what lies in rows that no
    slot names does not matter, and their gradient is not written; infinities stay in their token."""
    bk = gpu_lib
    Ys = torch.randn(4, 50, device="cuda")
    Ys[2] = float("nan")
    Ys[3, 7] = float("inf")
    slots = torch.tensor([[0, -1], [1, 4], [-5, 1 << 30], [3, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [2.0, float("inf")], [1.0, 1.0], [1.0, 1.0]], device="cuda")
    Y = bk.combine_tokens(Ys, slots, w)
    assert torch.equal(Y[0], Ys[0] * 0.5) and torch.equal(Y[1], Ys[1] * 2) and (Y[2] == 0).all()
    assert torch.isinf(Y[3, 7]) and torch.isfinite(Y[3, :7]).all()
    G = torch.randn(4, 50, device="cuda")
    out, dw = torch.full((4, 50), 7.0, device="cuda"), torch.full((4, 2), 7.0, device="cuda")
    slots[3, 1] = -1
    assert bk.lib().bakron_combine_tokens_grad(bk.F32, 4, 2, 50, 4, bk._p(G), 50, bk._p(Ys), 50, bk._p(slots), bk._p(w),
                                               bk._p(out), 50, bk._p(dw), bk._stream(G.device)) == bk.OK
    assert (out[2] == 7).all() and torch.equal(out[0], G[0] * 0.5) and torch.equal(out[1], 2 * G[1])
    assert (dw[[0, 1, 2, 2, 3], [1, 1, 0, 1, 1]] == 0).all()
    assert (bk.combine_tokens(Ys[:0], slots, w) == 0).all()
    assert (bk.combine_tokens(Ys, slots[:, :0].contiguous()) == 0).all()
    assert bk.combine_tokens(Ys, slots[:0], w[:0]).shape == (0, 50)
    assert bk.combine_tokens_grad(G[:, :0], Ys[:, :0], slots, w)[1].eq(0).all()
