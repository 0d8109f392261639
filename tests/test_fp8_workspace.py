"""Workspaces of the products with block scales: rows of codes that start on 16 bytes are read as they lie,
so their calls need no room for copies, and take none; others are copied, and refused without the room."""
import ctypes

import pytest
import torch

import kronecker_factored_gptq_amd as bk

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": bk.F32, "bf16": bk.BF16, "f16": bk.F16}


def blocks(n):
    return -(-n // 128)


def queries():
    L = bk.lib()
    return (L.bakron_matmul_fp8_workspace_bytes, L.bakron_matmul_fp8_aligned_workspace_bytes,
            L.bakron_matmul_fp8_grad_workspace_bytes, L.bakron_matmul_fp8_grad_aligned_workspace_bytes)


@pytest.mark.parametrize("T,R,E,m,n", [(4096, 16384, 64, 2048, 4095), (300, 300, 3, 200, 401), (300, 300, 1, 1000, 4097),
                                       (77, 900, 1, 5000, 129), (1, 300, 5, 200, 33)])
@pytest.mark.parametrize("t", CODES.values())
def test_queries(T, R, E, m, n, t):
    any_, aligned, any_grad, aligned_grad = queries()
    line = (n + 127) // 128 * 128
    up = lambda x: (x + 255) // 256 * 256
    a, b = any_(t, T, R, E, m, n), aligned(t, T, R, E, m, n)
    assert a - b == up(T * line) + up(E * m * line) + (256 if b == 0 else 0)  # the copies and nothing else
    if E > 1:
        assert b == 0  # nothing is split by experts
    a, b = any_grad(t, R, E, m, n), aligned_grad(t, R, E, m, n)
    assert a - b == up(E * m * line) + (256 if b == 0 else 0)
    # whole groups of 16: no copies either way
    n = n // 16 * 16
    assert any_(t, T, R, E, m, n) == aligned(t, T, R, E, m, n)
    assert any_grad(t, R, E, m, n) == aligned_grad(t, R, E, m, n)


def test_queries_of_refused_sizes():
    _, aligned, _, aligned_grad = queries()
    assert aligned(bk.F64, 3, 12, 4, 140, 301) == aligned(bk.F32, -1, 12, 4, 140, 301) == aligned(bk.F32, 3, 12, 0, 140, 301) == 0
    assert aligned_grad(bk.F64, 12, 4, 140, 301) == aligned_grad(bk.F32, -1, 4, 140, 301) == aligned_grad(bk.F32, 12, 1025, 140, 301) == 0


def at(k, more=0):
    """An address that is never dereferenced."""
    return ctypes.c_void_p(0x1000000 * k + more)


@pytest.mark.parametrize("off", [dict(X=at(1, 8)), dict(W=at(3, 1)), dict(ldx=401), dict(ldw=408), dict(sW=56000 + 8)])
def test_copies_without_room_are_refused(off):
    """Codes off 16 bytes, with the room that those on 16 bytes need."""
    a = dict(X=at(1), ldx=416, W=at(3), ldw=416, sW=83200)
    a.update(off)
    need = bk.lib().bakron_matmul_fp8_aligned_workspace_bytes(bk.F32, 300, 300, 3, 200, 401)
    assert bk.lib().bakron_matmul_fp8(bk.F32, 300, 300, 3, 200, 401, a["X"], a["ldx"], at(4), 1, 300, a["W"], a["ldw"],
                                      a["sW"], at(5), 4, 8, at(6), None, 1, at(7), 200, at(8), need, None) == bk.EINVAL
    if "X" in off or "ldx" in off:
        return
    # of the gradient the planes of G alone
    need = bk.lib().bakron_matmul_fp8_grad_aligned_workspace_bytes(bk.F32, 300, 3, 200, 401)
    assert bk.lib().bakron_matmul_fp8_grad(bk.F32, 300, 3, 200, 401, at(1), 200, a["W"], a["ldw"], a["sW"], at(5), 4, 8,
                                           at(6), at(7), 401, at(8), need, None) == bk.EINVAL


def buffer(nbytes):
    """nbytes of workspace, aligned, and the buffer it lies in, filled with 171."""
    buf = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
    first = -buf.data_ptr() % 256
    return buf, buf[first:first + nbytes] if nbytes else None, first + nbytes


def layer(T, E, m, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(T, n, generator=g).cuda(), torch.randn(E, m, n, generator=g).cuda()
    return *bk.quantize_fp8(x), *bk.quantize_fp8(w, 128)


def off_16(q):
    """The same codes in rows of n + 1, one byte off."""
    buf = torch.zeros(*q.shape[:-1], q.size(-1) + 1, dtype=torch.uint8, device="cuda")
    buf[..., 1:] = q.view(torch.uint8)
    return buf.view(F8)[..., 1:]


# many rows, few rows (nothing is copied at any alignment), k split, one row of tokens or of weights
CASES = [(300, 900, 3, 200, 401), (100, 100, 1, 200, 5001), (300, 300, 1, 1000, 4097), (9, 9, 1, 300, 401), (1, 300, 2, 200, 401),
         (300, 300, 3, 1, 401)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,R,E,m,n", CASES)
@pytest.mark.parametrize("t", TYPES)
def test_only_what_is_needed(gpu_lib, T, R, E, m, n, t):
    """With exactly the room that the aligned query names, or none, and nothing written behind it; the
    unaligned codes with the other query's give the same."""
    L, c, dt = bk.lib(), CODES[t], TYPES[t]
    Xq, sx, Wq, sw = layer(T, E, m, n)
    assert Xq.stride(0) % 16 == Wq.stride(1) % 16 == 0
    g = torch.Generator().manual_seed(3)
    off = None if E == 1 else torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32).cuda()
    order = None if R == T else torch.randint(0, T, (R,), generator=g, dtype=torch.int32).cuda()
    G = torch.randn(R, m, generator=g).to(dt).cuda()

    def product(X, W, nbytes, ldx, ldw, sW):
        buf, ws, end = buffer(nbytes)
        Y = torch.empty(R, m, dtype=dt, device="cuda")
        assert L.bakron_matmul_fp8(c, T, R, E, m, n, bk._p(X), ldx, bk._p(sx), 1, T, bk._p(W), ldw, sW, bk._p(sw), sw.stride(1),
                                   sw.stride(0), None if off is None else bk._p(off), None if order is None else bk._p(order), 1,
                                   bk._p(Y), m, None if ws is None else ws.data_ptr(), nbytes, bk._stream(Y.device)) == bk.OK
        assert (buf[end:] == 171).all()
        return Y

    def gradient(W, nbytes, ldw, sW):
        buf, ws, end = buffer(nbytes)
        D = torch.empty(R, n, dtype=dt, device="cuda")
        assert L.bakron_matmul_fp8_grad(c, R, E, m, n, bk._p(G), m, bk._p(W), ldw, sW, bk._p(sw), sw.stride(1), sw.stride(0),
                                        None if off is None else bk._p(off), bk._p(D), n, None if ws is None else ws.data_ptr(),
                                        nbytes, bk._stream(D.device)) == bk.OK
        assert (buf[end:] == 171).all()
        return D

    any_, aligned, any_grad, aligned_grad = queries()
    room = lambda q: max(q - 256, 0)
    # a single row's leading dimension and a single expert's stride say nothing
    ldx, ldw = (Xq.stride(0) if T > 1 else n), (Wq.stride(1) if m > 1 else n)
    sW = Wq.stride(0) if E > 1 else 3
    Y = product(Xq, Wq, room(aligned(c, T, R, E, m, n)), ldx, ldw, sW)
    D = gradient(Wq, room(aligned_grad(c, R, E, m, n)), ldw, sW)
    Xo, Wo = off_16(Xq), off_16(Wq)
    Z = product(Xo, Wo, room(any_(c, T, R, E, m, n)), Xo.stride(0), Wo.stride(1), Wo.stride(0))
    H = gradient(Wo, room(any_grad(c, R, E, m, n)), Wo.stride(1), Wo.stride(0))
    # the same tiles over the same codes: the same bits
    assert torch.equal(Y, Z) and torch.equal(D, H)
    w = (Wq, sw) if E > 1 else (Wq[0], sw[0])
    assert torch.equal(Y, bk.matmul_fp8(Xq, sx, *w, offsets=off, order=order, out_dtype=dt))
    assert torch.equal(D, bk.matmul_fp8_grad(G, *w, offsets=off))


@pytest.mark.gpu
@pytest.mark.parametrize("T,R,E,m,n", [(512, 2048, 32, 1024, 1531), (1, 300, 32, 1024, 1531), (700, 700, 1, 4096, 4095)])
def test_the_binding_takes_no_copies(gpu_lib, T, R, E, m, n):
    """Memory that a call takes: its result, and less than a copy of the codes."""
    Xq, sx, Wq, sw = layer(T, E, m, n)
    off = None if E == 1 else torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32).cuda()
    order = None if R == T else (torch.arange(R) % T).int().cuda()
    w = (Wq, sw) if E > 1 else (Wq[0], sw[0])
    G = torch.randn(R, m, device="cuda").bfloat16()
    for call, own in ((lambda: bk.matmul_fp8(Xq, sx, *w, offsets=off, order=order, out_dtype=torch.bfloat16), R * m * 2),
                      (lambda: bk.matmul_fp8_grad(G, *w, offsets=off), R * n * 2)):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        call()
        torch.cuda.synchronize()
        split = bk.lib().bakron_matmul_fp8_aligned_workspace_bytes(bk.BF16, T, R, E, m, n)
        grad = bk.lib().bakron_matmul_fp8_grad_aligned_workspace_bytes(bk.BF16, R, E, m, n)
        # the allocator counts whole blocks: two of them, each up to 1 MiB larger than asked for, since what is left of a
        # block beyond that is split off; a copy of the codes is 16 MiB (4096 rows of 4096 bytes) or more in every case here
        assert E * m * (n // 128 * 128) >= 15 << 20
        assert torch.cuda.max_memory_allocated() - before <= own + max(split, grad) + (2 << 20)
        if E > 1:
            assert max(split, grad) == 0
