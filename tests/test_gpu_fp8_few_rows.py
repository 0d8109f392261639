"""Few rows times weights in 8-bit floating point: sums are float32 for every result type, so that small products
beside large ones that cancel keep all their bits.

Of each 8 neighbouring products one is 448 * 448, another -448 * 448 and six are whole multiples of 1/4 up to 36. In
a block of 128 every sum, in any order, is a multiple of 1/4 below 16 * 448 * 448 + 96 * 36 < 2^22: 24 bits, exact in
float32. Blocks add up to at most 96 * 36 each, and scales are powers of two: the result is the exact sum
rounded once to its type, whatever the order."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def blocks(n):
    return -(-n // 128)


def operands(T, m, n, g):
    """Tokens and weights as values, exact in e4m3."""
    few = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 6.0])
    x = few[torch.randint(0, 6, (T, n), generator=g)] * (2.0 * torch.randint(0, 2, (T, n), generator=g) - 1)
    w = few[torch.randint(0, 6, (m, n), generator=g)] * (2.0 * torch.randint(0, 2, (m, n), generator=g) - 1)
    whole = n // 8 * 8
    place = torch.rand(whole // 8, 8, generator=g).argsort(1)
    plus, minus = (8 * torch.arange(whole // 8) + place[:, i] for i in (0, 1))
    x[:, plus], w[:, plus], x[:, minus], w[:, minus] = 448.0, 448.0, 448.0, -448.0
    return x, w


def power(*shape, g):
    return 2.0 ** torch.randint(-3, 1, shape, generator=g)


def spread(s, rows, a, n):
    return s.repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(128, -1)[..., :n]


def nearest(ref, t):
    """Sums in 64 bits, rounded once (the sums have at most 24 bits, so by way of float32 it is one rounding)."""
    assert torch.equal(ref.float().double(), ref)
    return ref.float().to(t)


@pytest.mark.parametrize("T,m,n", [(1, 1, 8), (1, 4096, 4096), (1, 70, 1003), (3, 130, 400), (16, 300, 2048), (17, 513, 1024),
                                   (33, 256, 512), (64, 1000, 1024), (64, 40, 4099), (16, 14336, 1024), (8, 8192, 8704)])
@pytest.mark.parametrize("t", TYPES)
def test_one_layer(gpu_lib, T, m, n, t):
    g = torch.Generator().manual_seed(T + m + n)
    x, w = operands(T, m, n, g)
    sx, sw = power(T, 1, g=g).expand(T, blocks(n)).contiguous(), power(blocks(m), 1, g=g).expand(blocks(m), blocks(n)).contiguous()
    Y = gpu_lib.matmul_fp8(x.to(F8).cuda(), sx.cuda(), w.to(F8).cuda(), sw.cuda(), out_dtype=TYPES[t])
    ref = (x.double().cuda() @ w.double().cuda().T).cpu() * sx[:, :1].double() * sw[:, :1].repeat_interleave(128, 0)[:m].T.double()
    assert torch.equal(Y.cpu(), nearest(ref, TYPES[t]))


@pytest.mark.parametrize("R,E,m,n", [(1, 8, 300, 2048), (20, 5, 130, 2064), (64, 8, 2048, 4096), (250, 40, 257, 2049)])
@pytest.mark.parametrize("t", TYPES)
def test_by_experts(gpu_lib, R, E, m, n, t):
    g = torch.Generator().manual_seed(R + E + m)
    x, w = operands(R, E * m, n, g)
    w = w.view(E, m, n)
    sx, sw = torch.ones(R, blocks(n)), torch.ones(E, blocks(m), blocks(n))
    off = torch.cat([torch.zeros(1), torch.rand(E - 1, generator=g).sort().values * R, torch.full((1,), R)]).int()
    order = torch.randperm(R, generator=g).int()
    Y = gpu_lib.matmul_fp8(x.to(F8).cuda(), sx.cuda(), w.to(F8).cuda(), sw.cuda(), offsets=off.cuda(), order=order.cuda(),
                           out_dtype=TYPES[t]).cpu()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        ref = x[order[a:b].long()].double() @ w[e].double().T
        assert torch.equal(Y[a:b], nearest(ref, TYPES[t])), e
