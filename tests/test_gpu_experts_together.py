"""8-bit floating point and the tokens of experts as a program uses them together: a layer of
experts forward and back, an expert's Kronecker factor, beside the solve's own codes; the
same twice, on other streams, in HIP graphs, with a shared workspace, beyond 32-bit offsets.

A step of the chain is held to 64-bit arithmetic on that step's own inputs, with the
roundings of its definition (E = 2^-24, a float32's half step): a float32 product of codes rounds as
tests/test_gpu_fp8.py counts, 131 2^-23 + blocks 2^-24 of the terms' absolute sum; a gradient's sums of m terms in
three planes 3 m 2^-23; a weighted sum of k rows k 2^-24."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
E = 2.0 ** -24


def blocks(n):
    return -(-n // 128)


def values(q, s, rows):
    """What codes and scales stand for, in 64 bits."""
    a, n = q.shape[-2:]
    s = s.double().repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(128, -1)[..., :n]
    return q.float().double() * s


def layer(T=200, k=2, E_=6, n=384, h=260, seed=3, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, n, generator=g) * torch.exp(0.5 * torch.randn(n, generator=g))
    W1 = torch.randn(E_, h, n, generator=g) * n ** -0.5
    W2 = torch.randn(E_, n, h, generator=g) * h ** -0.5
    score = torch.randn(T, E_, generator=g)
    w, ids = score.softmax(1).topk(k, 1)
    ids[::17] = -1  # padding
    G = torch.randn(T, n, generator=g)
    return [t.to(device) for t in (X, W1, W2, w.contiguous(), ids, G)]


def forward(bk, X, W1q, W2q, w, ids, dtype=torch.float32):
    E_, k = W1q[0].size(0), ids.size(1)
    order, slots, offsets = bk.sort_tokens(ids, E_)
    Xq, sx = bk.quantize_fp8(X)
    H = bk.matmul_fp8(Xq, sx, *W1q, offsets=offsets, order=order, per_token=k,
                      out=torch.zeros(order.numel(), W1q[0].size(1), dtype=dtype, device=X.device))
    Hq, sh = bk.quantize_fp8(H)
    Ys = bk.matmul_fp8(Hq, sh, *W2q, offsets=offsets, out=torch.zeros(order.numel(), X.size(1), dtype=dtype, device=X.device))
    return order, slots, offsets, Xq, sx, H, Hq, sh, Ys, bk.combine_tokens(Ys, slots, w)


def backward(bk, G, Ys, W1q, W2q, slots, offsets, w):
    dYs, dw = bk.combine_tokens_grad(G, Ys, slots, w)
    dH = bk.matmul_fp8_grad(dYs, *W2q, offsets=offsets)
    dXs = bk.matmul_fp8_grad(dH, *W1q, offsets=offsets)
    return dYs, dw, dH, dXs, bk.combine_tokens(dXs, slots)


def test_layer_of_experts(gpu_lib):
    bk = gpu_lib
    X, W1, W2, w, ids, G = layer()
    T, k, E_, n, h = X.size(0), ids.size(1), W1.size(0), X.size(1), W1.size(1)
    W1q, W2q = bk.quantize_fp8(W1, 128), bk.quantize_fp8(W2, 128)
    order, slots, offsets, Xq, sx, H, Hq, sh, Ys, Y = forward(bk, X, W1q, W2q, w, ids)
    off, tok = offsets.tolist(), (order.long() // k)
    V1, V2 = values(*W1q, 128), values(*W2q, 128)
    # quantisation: half a step of 4 bits, and of the smallest code under the block's scale
    x = values(Xq, sx, 1)
    step = sx.double().repeat_interleave(128, 1)[:, :n] * 2.0 ** -10
    assert ((x - X.double()).abs() <= X.double().abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + step).all()
    for e in range(E_):
        a, b = off[e], off[e + 1]
        for got, u, v in ((H, x[tok[a:b]], V1[e]), (Ys, values(Hq, sh, 1)[a:b], V2[e])):
            ref, S = u @ v.T, u.abs() @ v.abs().T
            assert ((got[a:b].double() - ref).abs() <= S * (131 * 2.0 ** -23 + blocks(u.size(1)) * E) + ref.abs() * E).all()
    has = slots >= 0
    y = torch.where(has[:, :, None], Ys.double()[slots.long().clamp(min=0)], 0.0) * w.double()[:, :, None]
    assert ((Y.double() - y.sum(1)).abs() <= y.abs().sum(1) * (k + 1) * E).all()
    assert (Y[::17] == 0).all()
    # back: the gradient with respect to the tokens, their rounding passed straight through
    dYs, dw, dH, dXs, dX = backward(bk, G, Ys, W1q, W2q, slots, offsets, w)
    assert ((dw.double() - torch.where(has[:, :, None], Ys.double()[slots.long().clamp(min=0)] * G.double()[:, None], 0.0).sum(2)).abs()
            <= 2 * n * E * (Ys.double().abs().max() * G.double().abs().sum(1, keepdim=True))).all()
    for e in range(E_):
        a, b = off[e], off[e + 1]
        for got, u, v in ((dH, dYs, V2[e]), (dXs, dH, V1[e])):
            ref, S = u[a:b].double() @ v, u[a:b].double().abs() @ v.abs()
            assert ((got[a:b].double() - ref).abs() <= S * (3 * v.size(0) * 2.0 ** -23 + 3 * E) + ref.abs() * E).all()
    # and as a whole, against differences of the layer on the tokens' and weights' values in 64 bits
    def whole(x, w):
        out = torch.zeros(T, n, dtype=torch.float64, device="cuda")
        for j in range(k):
            for e in range(E_):
                t = (ids[:, j] == e).nonzero().squeeze(1)
                out[t] += w[t, j, None] * (x[t] @ V1[e].T @ V2[e].T)
        return (out * G.double()).sum()
    g = torch.Generator().manual_seed(9)
    d = torch.randn(T, n, generator=g).double().cuda()
    change = (whole(X.double() + 2.0 ** -8 * d, w.double()) - whole(X.double() - 2.0 ** -8 * d, w.double())) * 2.0 ** 7
    S = (G.double().abs() @ V2.abs().sum(0)) @ V1.abs().sum(0)  # more than the terms' absolute sum
    bound = (S * d.abs()).sum() * (3 * (n + h) * 2.0 ** -23 + (k + 8) * E)
    assert ((dX.double() * d).sum() - change).abs() <= bound


def test_an_experts_factor_and_codes(gpu_lib):
    """The samples routed to an expert make its Kronecker factor; the solve's codes of that
    expert take its tokens beside the 8-bit floating point ones."""
    bk = gpu_lib
    X, W1, _, w, ids, G = layer(T=400, n=96, h=64, seed=5)
    k, E_, n, m = ids.size(1), W1.size(0), X.size(1), W1.size(1)
    order, slots, offsets = bk.sort_tokens(ids, E_)
    Xs, off, e = bk.gather_tokens(X, order, k), offsets.tolist(), 2
    mine = Xs[off[e]:off[e + 1]]
    assert torch.equal(mine, X[(ids == e).any(1)]) and (Xs[off[-1]:] == 0).all()
    A = bk.gram(mine, damp_rel=0.01)
    ref = mine.double().T @ mine.double() / mine.size(0)
    ref += 0.01 * ref.diagonal().mean() * torch.eye(n, dtype=torch.float64, device="cuda")
    S = mine.double().abs().T @ mine.double().abs() / mine.size(0)
    assert ((A.double() - ref).abs() <= (mine.size(0) + 8) * E * (S + 0.01 * S.diagonal().mean())).all()
    B = torch.eye(m, device="cuda")
    LA, LB, _, _ = bk.factor(A, B)
    s = bk.row_scales(W1[e], 7)
    V = bk.solve(W1[e], LA, LB, (-8, 7, 0), s, check=True)
    Xq, sx = bk.quantize_tokens(mine)
    Y4 = bk.matmul_int8(Xq, sx, V.to(torch.int8), s)
    Y8 = bk.matmul_fp8(*bk.quantize_fp8(mine), *bk.quantize_fp8(W1[e], 128))
    # each is X W^T but for the roundings of its two operands: half a step of the codes; and 2^-4 of each, half the
    # smallest code's step
    exact = mine.double() @ W1[e].double().T
    Wq = V.double() * s.double()[:, None]
    step = 0.5 * sx.double()[:, None] * (1 + 2.0 ** -10)
    assert ((Y4.double() - mine.double() @ Wq.T).abs() <= step * Wq.abs().sum(1) + 1e-5 * (mine.double().abs() @ Wq.abs().T)).all()
    S = mine.double().abs() @ W1[e].double().abs().T
    tiny = mine.abs().amax(1, keepdim=True).double() / 448 * 2.0 ** -10
    bound = S * (2 * 2.0 ** -4 + 2.0 ** -8 + 1e-4) + 2 * tiny * W1[e].double().abs().sum(1) + 2 * mine.double().abs().sum(1, keepdim=True) * (W1[e].abs().max().double() / 448 * 2.0 ** -10)
    assert ((Y8.double() - exact).abs() <= bound).all()


def calls(bk, X, W1, W2, w, ids, G):
    """Every operator once, in float32 and bfloat16; all outputs."""
    got = []
    for t in (torch.float32, torch.bfloat16):
        W1q, W2q = bk.quantize_fp8(W1.to(t), 128), bk.quantize_fp8(W2.to(t), 128)
        f = forward(bk, X.to(t), W1q, W2q, w, ids, t)
        order, slots, offsets, Xq, sx, H, Hq, sh, Ys, Y = f
        b = backward(bk, G.to(t), Ys, W1q, W2q, slots, offsets, w)
        Xs = bk.gather_tokens(X.to(t), order, ids.size(1))
        dense = bk.matmul_fp8(Xq, sx, W1q[0][0], W1q[1][0], out_dtype=t)
        one = bk.matmul_fp8(Xq[:1], sx[:1], W1q[0][0], W1q[1][0], out_dtype=t)
        R = int(ids.numel() - (ids < 0).sum())
        got += [order, slots, offsets, Xq.view(torch.uint8).clone(), sx, H, Hq.view(torch.uint8).clone()[:R], Ys, Y, b[0][:R], b[1],
                b[2][:R], b[3][:R], b[4], Xs, dense, one, bk.matmul_fp8_grad(dense, W1q[0][0], W1q[1][0])]
    return got


@pytest.mark.parametrize("T,n,h", [(150, 384, 260), (700, 1024, 512)])
def test_the_same_twice(gpu_lib, T, n, h):
    a = layer(T=T, n=n, h=h, seed=7)
    assert all(torch.equal(u, v) for u, v in zip(calls(gpu_lib, *a), calls(gpu_lib, *a)))


def test_two_streams_at_once(gpu_lib):
    a, b = layer(T=3000, n=512, h=300, seed=5), layer(T=2500, n=512, h=300, seed=6)
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


def graph_calls(bk, X, W1q, W2q, w, ids, G, ws):
    f = forward(bk, X, W1q, W2q, w, ids, torch.bfloat16)
    order, slots, offsets, Xq, sx, H, Hq, sh, Ys, Y = f
    b = backward(bk, G, Ys, W1q, W2q, slots, offsets, w)
    split = bk.matmul_fp8(Xq, sx, W1q[0][0], W1q[1][0], workspace=ws)  # k split: sums in the workspace
    back = bk.matmul_fp8_grad(split, W1q[0][0], W1q[1][0], workspace=ws)
    return [order, slots, offsets, H, Ys, Y, b[1], b[4], split, back]


def test_captured_and_replayed(gpu_lib):
    """Forward and backward in a HIP graph, replayed on other tokens and routes with eager
    work in between, and beside it a second graph that was given the same workspace."""
    bk = gpu_lib
    make = lambda seed: layer(T=1500, n=2048, h=130, E_=5, seed=seed)
    X, W1, W2, w, ids, G = make(1)
    W1q, W2q = bk.quantize_fp8(W1, 128), bk.quantize_fp8(W2, 128)
    static = [X.bfloat16(), W1q, W2q, w, ids, G.bfloat16()]
    L = bk.lib()
    need = max(L.bakron_matmul_fp8_workspace_bytes(bk.F32, 1500, 1500, 1, 130, 2048),
               L.bakron_matmul_fp8_grad_workspace_bytes(bk.F32, 1500, 1, 130, 2048))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    graph_calls(bk, *static, ws)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        got = graph_calls(bk, *static, ws)
    with torch.cuda.graph(second):
        other = graph_calls(bk, *static, ws)
    for seed in (2, 3, 4, 5):
        new = make(seed)
        for t, v in zip((static[0], static[3], static[4], static[5]), (new[0].bfloat16(), new[3], new[4], new[5].bfloat16())):
            t.copy_(v)
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        want = graph_calls(bk, *static, torch.empty_like(ws))
        for u, v, x in zip(got, other, want):
            assert torch.equal(u, x) and torch.equal(v, x)


def test_workspace_of_exactly_the_size(gpu_lib):
    """Every path that takes a workspace keeps to the size its query names: what lies behind stays."""
    bk = gpu_lib
    L, g = bk.lib(), torch.Generator().manual_seed(4)
    def buffer(nbytes):
        buf = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
        at = -buf.data_ptr() % 256
        return buf, buf[at:at + nbytes], at + nbytes
    for T, m, n in ((100, 200, 5001), (300, 130, 4096), (64, 700, 1003)):
        x, wt = torch.randn(T, n, generator=g).cuda(), torch.randn(m, n, generator=g).cuda()
        Xq, sx = bk.quantize_fp8(x)
        Wq, sw = bk.quantize_fp8(wt, 128)
        for t, c in ((torch.float32, bk.F32), (torch.bfloat16, bk.BF16)):
            buf, ws, end = buffer(max(L.bakron_matmul_fp8_workspace_bytes(c, T, T, 1, m, n) - 256, 0))
            Y = torch.empty(T, m, dtype=t, device="cuda")
            assert L.bakron_matmul_fp8(c, T, T, 1, m, n, bk._p(Xq), Xq.stride(0), bk._p(sx), 1, T, bk._p(Wq), Wq.stride(0), 0,
                                       bk._p(sw), sw.stride(0), 0, None, None, 1, bk._p(Y), m, ws.data_ptr() if ws.numel() else None,
                                       ws.numel(), bk._stream(Y.device)) == bk.OK
            assert torch.equal(Y, bk.matmul_fp8(Xq, sx, Wq, sw, out_dtype=t)) and (buf[end:] == 171).all()
            G = torch.randn(T, m, generator=g).to(t).cuda()
            buf, ws, end = buffer(max(L.bakron_matmul_fp8_grad_workspace_bytes(c, T, 1, m, n) - 256, 0))
            D = torch.empty(T, n, dtype=t, device="cuda")
            assert L.bakron_matmul_fp8_grad(c, T, 1, m, n, bk._p(G), m, bk._p(Wq), Wq.stride(0), 0, bk._p(sw), sw.stride(0), 0,
                                            None, bk._p(D), n, ws.data_ptr() if ws.numel() else None, ws.numel(),
                                            bk._stream(D.device)) == bk.OK
            assert torch.equal(D, bk.matmul_fp8_grad(G, Wq, sw)) and (buf[end:] == 171).all()
    ids = torch.randint(-1, 50, (9000, 3), generator=g).cuda()
    buf, ws, end = buffer(L.bakron_sort_tokens_workspace_bytes(9000, 3, 50) - 256)
    out = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (27000, 27000, 51)]
    assert L.bakron_sort_tokens(9000, 3, 50, bk._p(ids), 3, *[bk._p(t) for t in out], ws.data_ptr(), ws.numel(),
                                bk._stream(ids.device)) == bk.OK
    for u, v in zip(out, bk.sort_tokens(ids, 50)):
        assert torch.equal(u, v.flatten())
    assert (buf[end:] == 171).all()


def test_beyond_32_bit_offsets(gpu_lib):
    """Operands of more than 2^31 bytes, and of more than 2^32: the last rows as they are alone."""
    bk = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    n, T = 16384, 270000  # 4.4e9 codes
    X = torch.randint(0, 120, (T, n), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    sx = torch.rand(blocks(n), T, device="cuda", generator=g).t()
    W = torch.randint(0, 120, (3, 128, n), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    sw = torch.rand(3, 1, blocks(n), device="cuda", generator=g)
    Y = bk.matmul_fp8(X, sx, W[0], sw[0], out_dtype=torch.bfloat16)
    part = bk.matmul_fp8(X[-300:], sx[-300:], W[0], sw[0])
    assert ((Y[-300:].float() - part).abs() <= part.abs() * (2.0 ** -8 + 2.0 ** -9)).all()  # positive terms: 7 2^-13 at most
    # by an order that reaches all of them, on the tiles and on the few rows' kernel
    for R in (300, 9):
        order = torch.randint(T - 2000, T, (R,), device="cuda", generator=g).int()
        off = torch.tensor([0, R // 3, R // 3, R], dtype=torch.int32, device="cuda")
        Z = bk.matmul_fp8(X, sx, W, sw, offsets=off, order=order)
        ref = torch.cat([bk.matmul_fp8(X.view(torch.uint8)[order[a:b].long()].view(F8), sx[order[a:b].long()], W[e], sw[e])
                         for e, a, b in ((0, 0, R // 3), (2, R // 3, R))])
        assert ((Z - ref).abs() <= ref.abs() * 2.0 ** -15).all()  # positive terms, two orders of 2^14 float32 sums
    del X, Y
    torch.cuda.empty_cache()
    # experts' weights of more than 4 GiB: the last one's
    E_, m, n = 70, 8192, 8192
    W = torch.randint(0, 120, (E_, m, n), dtype=torch.uint8, device="cuda", generator=g).view(F8)
    sw = torch.rand(E_, blocks(m), blocks(n), device="cuda", generator=g)
    for R in (40, 1500):
        x = torch.randn(R, n, device="cuda", generator=g)
        Xq, sx = bk.quantize_fp8(x)
        off = torch.full((E_ + 1,), R, dtype=torch.int32, device="cuda")
        off[:-1] = R // 4
        off[0] = 0
        Z = bk.matmul_fp8(Xq, sx, W, sw, offsets=off)
        D = bk.matmul_fp8_grad(x, Wq := W, sw, offsets=off)
        for e, a, b in ((0, 0, R // 4), (E_ - 1, R // 4, R)):
            u, v = bk.matmul_fp8(Xq[a:b], sx[a:b], W[e], sw[e]), bk.matmul_fp8_grad(x[a:b].contiguous(), W[e], sw[e])
            assert (Z[a:b] - u).norm() <= 1e-5 * u.norm() and (D[a:b] - v).norm() <= 1e-5 * v.norm()
    del W, Wq
    torch.cuda.empty_cache()
    # rows moved beyond 4 GiB
    X = torch.randn(300, 4096, device="cuda", generator=g)
    ids = torch.randint(0, 9, (300, 1), device="cuda", generator=g)
    order, slots, _ = bk.sort_tokens(ids, 9)
    wide = torch.zeros(300, 4 << 20, device="cuda")  # 5 GiB
    bk.gather_tokens(X, order, 1, out=wide[:, 5:4101])
    assert torch.equal(wide[:, 5:4101], X[order.long()]) and (wide[:, 4101:4200] == 0).all()
    assert torch.equal(bk.combine_tokens(wide[:, 5:4101], slots), X)


def test_beside_another_device_or_stream(gpu_lib):
    """The calls run on the current stream of their tensors' device, whatever device is current."""
    bk = gpu_lib
    a = layer(T=50, n=256, h=128, seed=8)
    want = calls(bk, *a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.device(0), torch.cuda.stream(s):
        got = calls(bk, *a)
        done = s.record_event()
    done.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
