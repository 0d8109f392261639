"""Scales at the ends of float32 in the product with block scales: a block's factor is the float32 product of its
two scales, on every path (few rows, tiles, k split, operands of any alignment). All codes are powers of two or
zero, so that a block's sum is exact, and every result one block's: factor times sum, rounded to float32 (no
rounding: the sum is a power of two and the result a normal float)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn

# rows, channels, k, first byte of a row: few rows, tiles, tiles over ranges of k, through registers
PATHS = [(5, 130, 400, 0), (300, 5000, 128, 0), (300, 130, 16384, 0), (300, 200, 400, 5)]


def call(bk, T, m, n, first, sx, sw, zero=()):
    """Y, where only column 3 of both operands is not zero: 2^8 * 2^8; none in the tokens `zero`."""
    x, w = torch.zeros(T, n + first), torch.zeros(m, n + first)
    x[:, first + 3] = w[:, first + 3] = 256.0
    x[list(zero)] = 0.0
    X, W = x.to(F8).cuda()[:, first:], w.to(F8).cuda()[:, first:]
    nb = -(-n // 128)
    a, b = torch.ones(T, nb), torch.ones(-(-m // 128), nb)
    a[:, 0], b[:, 0] = sx, sw
    return bk.matmul_fp8(X, a.cuda(), W, b.cuda()).cpu()


@pytest.mark.parametrize("T,m,n,first", PATHS)
def test_small_products_of_scales(gpu_lib, T, m, n, first):
    g = torch.Generator().manual_seed(T + m)
    # factors from 2^-148 to 2^-126: with 1 to 23 bits
    sx = torch.ldexp(1 + torch.rand(T, generator=g), torch.randint(-100, -90, (T,), generator=g, dtype=torch.int32))
    sw = torch.ldexp(1 + torch.rand(-(-m // 128), generator=g), torch.randint(-48, -35, (-(-m // 128),), generator=g, dtype=torch.int32))
    f = sx[:, None] * sw[None, :]
    assert (f < 2.0 ** -126).any() and (f > 0).all()
    assert torch.equal(call(gpu_lib, T, m, n, first, sx, sw), (f * 2.0 ** 16).repeat_interleave(128, 1)[:, :m])


@pytest.mark.parametrize("T,m,n,first", PATHS)
def test_large_products_of_scales(gpu_lib, T, m, n, first):
    """Finite up to 2^128, whatever the two are; beyond that infinite, NaN where the sum is 0."""
    sw = torch.full((-(-m // 128),), 2.0 ** -60)
    assert torch.equal(call(gpu_lib, T, m, n, first, torch.full((T,), 2.0 ** 127), sw), torch.full((T, m), 2.0 ** 83))
    Y = call(gpu_lib, T, m, n, first, torch.full((T,), 2.0 ** 100), torch.full_like(sw, 2.0 ** 30), zero=[1])
    assert torch.isnan(Y[1]).all() and torch.isinf(Y[[0, 2]]).all()
