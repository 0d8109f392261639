"""Calls of 8-bit floating point and of the tokens of experts that their documentation allows, each against the same
work done another way: operands with strides of 0, an order with several routes a token and no experts, k split and at
any alignment, one expert with offsets, tokens or experts named again and again, one column, and all of it captured in
a HIP graph and replayed on other data."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def layer(bk, T, m, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(T, n, generator=g).cuda(), torch.randn(m, n, generator=g).cuda()
    return *bk.quantize_fp8(x), *bk.quantize_fp8(w, 128)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_quantize_one_matrix_for_a_batch(gpu_lib, rows, t):
    """A batch with stride 0, and one of a single matrix; of matrices that interleave."""
    bk = gpu_lib
    x = torch.randn(70, 300, device="cuda").to(t)
    q, s = bk.quantize_fp8(x, rows)
    for batch in (1, 3):
        b, c = bk.quantize_fp8(x.expand(batch, 70, 300), rows)
        assert all(same(b[z], q) and torch.equal(c[z], s) for z in range(batch))
    y = torch.randn(70, 2, 300, device="cuda").to(t).transpose(0, 1)  # rows of two matrices in turn
    b, c = bk.quantize_fp8(y, rows)
    for z in range(2):
        q, s = bk.quantize_fp8(y[z].contiguous(), rows)
        assert same(b[z], q) and torch.equal(c[z], s)


@pytest.mark.parametrize("T,m,n", [(5, 300, 400), (300, 300, 401), (200, 1000, 4096), (1, 1, 1), (300, 1, 1), (1, 300, 1)])
def test_scales_with_strides_of_0(gpu_lib, T, m, n):
    bk = gpu_lib
    Xq, _, Wq, _ = layer(bk, T, m, n)
    nb, mb = -(-n // 128), -(-m // 128)
    one, two = torch.full((1, 1), 0.25, device="cuda"), torch.full((1, nb), 0.5, device="cuda")
    for t in (torch.float32, torch.float16):
        a = bk.matmul_fp8(Xq, one.expand(T, nb), Wq, two.expand(mb, nb).contiguous(), out_dtype=t)
        b = bk.matmul_fp8(Xq, one.expand(T, nb).contiguous(), Wq, two.expand(mb, nb).contiguous(), out_dtype=t)
        c = bk.matmul_fp8(Xq, one.expand(T, nb).t().contiguous().t(), Wq, two.expand(mb, nb).contiguous(), out_dtype=t)
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("T,k,m,n", [(3, 2, 130, 400), (100, 3, 1000, 4096), (100, 3, 130, 4097), (100, 4, 2000, 272), (700, 4, 1500, 400)])
@pytest.mark.parametrize("first", [0, 5])
def test_an_order_without_experts(gpu_lib, T, k, m, n, first):
    """Routes of one layer, some named twice: as the product of the tokens copied into that order."""
    bk = gpu_lib
    Xq, sx, Wq, sw = layer(bk, T, m, n)
    if first:
        buf = torch.zeros(T, n + 16, dtype=torch.uint8, device="cuda")
        buf[:, first:first + n] = Xq.view(torch.uint8)
        Xq = buf.view(F8)[:, first:first + n]
    g = torch.Generator().manual_seed(n)
    order = torch.randint(0, T * k, (T * k,), generator=g, dtype=torch.int32).cuda()
    order[1] = order[0]
    at = order.long() // k
    rows = torch.zeros(T * k, (n + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    rows[:, :n] = Xq.view(torch.uint8)[at]
    for t in (torch.float32, torch.bfloat16):
        Y = bk.matmul_fp8(Xq, sx, Wq, sw, order=order, per_token=k, out_dtype=t)
        Z = bk.matmul_fp8(rows.view(F8)[:, :n], sx[at], Wq, sw, out_dtype=t)
        # one expert's offsets around all of them
        V = bk.matmul_fp8(Xq, sx, Wq[None], sw[None], offsets=torch.tensor([0, T * k], dtype=torch.int32).cuda(), order=order,
                          per_token=k, out_dtype=t)
        x, w = rows.view(F8)[:, :n].float().double(), Wq.float().double()
        x = x * sx[at].double().repeat_interleave(128, 1)[:, :n]
        w = w * sw.double().repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :n]
        ref, S = x @ w.T, x.abs() @ w.abs().T
        # as tests/test_gpu_fp8.py counts: any codes
        tol = S * (131 * 2.0 ** -23 + sx.size(1) * 2.0 ** -24) + ref.abs() * torch.finfo(t).eps / 2 * (1 + 2.0 ** -8)
        if t != torch.float32:
            tol = tol + S * 7 * 2.0 ** -13
        for got in (Y, Z, V):
            assert ((got.double() - ref).abs() <= tol).all()
        assert torch.equal(Y[0], Y[1])


def test_one_expert_and_its_gradient(gpu_lib):
    """Offsets of one expert that leave rows out on both sides, at sizes where a layer's k would be split."""
    bk = gpu_lib
    R, m, n = 300, 1000, 4096
    Xq, sx, Wq, sw = layer(bk, R, m, n)
    off = torch.tensor([40, 250], dtype=torch.int32).cuda()
    out = torch.full((R, m), 7.0, device="cuda")
    bk.matmul_fp8(Xq, sx, Wq[None], sw[None], offsets=off, out=out)
    want = bk.matmul_fp8(Xq, sx, Wq, sw)
    assert (out[:40] == 7).all() and (out[250:] == 7).all()
    assert (out[40:250] - want[40:250]).norm() <= 1e-5 * want.norm()  # float32 sums in two orders: 2^-24 sqrt(n) and less
    G = torch.randn(R, m, device="cuda")
    out = torch.full((R, n), 7.0, device="cuda")
    bk.matmul_fp8_grad(G, Wq[None], sw[None], offsets=off, out=out)
    want = bk.matmul_fp8_grad(G, Wq, sw)
    assert (out[:40] == 7).all() and (out[250:] == 7).all() and (out[40:250] - want[40:250]).norm() <= 1e-5 * want.norm()


def test_every_route_to_one_expert(gpu_lib):
    """The same expert several times for one token, and one expert for all: stable, and added up as often."""
    bk = gpu_lib
    T, k, n = 500, 4, 300
    ids = torch.full((T, k), 3, device="cuda")
    order, slots, offsets = bk.sort_tokens(ids, 7)
    assert torch.equal(order, torch.arange(T * k, device="cuda").int()) and torch.equal(slots.flatten(), order)
    assert offsets.tolist() == [0, 0, 0, 0, T * k, T * k, T * k, T * k]
    X = torch.randn(T, n, device="cuda")
    assert torch.equal(bk.combine_tokens(bk.gather_tokens(X, order, k), slots), 4 * X)
    # only dropped routes
    order, slots, offsets = bk.sort_tokens(torch.full((T, k), 7, device="cuda"), 7)
    assert (order == -1).all() and (slots == -1).all() and (offsets == 0).all()
    assert (bk.combine_tokens(X, slots) == 0).all() and (bk.gather_tokens(X, order, k) == 0).all()
    dYs, dw = bk.combine_tokens_grad(X, X, slots, need_dYs=False)
    assert dYs is None and (dw == 0).all()
    assert bk.combine_tokens_grad(X[:, :0], X[:, :0], slots)[1].eq(0).all()


def test_rows_without_a_token_in_a_graph(gpu_lib):
    """Few rows, k split and odd lengths under an order that changes from replay to replay, NaN scales beside it."""
    bk = gpu_lib
    T, n = 100, 4095
    static = [layer(bk, T, m, n, seed=m) for m in (200, 1000)]
    for _, _, _, sw in static:
        sw[-1, 3] = float("nan")
    order = torch.zeros(300, dtype=torch.int32, device="cuda")
    few = torch.zeros(9, dtype=torch.int32, device="cuda")
    def calls():
        return [bk.matmul_fp8(*a, order=o, out_dtype=t) for a in static for o in (order, few) for t in (torch.float32, torch.bfloat16)]
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    g = torch.Generator().manual_seed(1)
    for _ in range(4):
        order.copy_(torch.randint(-T // 2, 2 * T, (300,), generator=g, dtype=torch.int32))
        few.copy_(torch.randint(-T // 2, 2 * T, (9,), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for u, v, o in zip(got, calls(), [order, order, few, few] * 2):
            missing = (o < 0) | (o >= T)
            assert (u[missing] == 0).all() and torch.isnan(u[~missing]).any()
            assert torch.equal(u.nan_to_num(), v.nan_to_num()) and torch.equal(u.isnan(), v.isnan())
