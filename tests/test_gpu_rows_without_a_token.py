"""Rows whose order names no token are 0 whatever the weights hold (bakron_matmul_fp8), on every
path of the product: few rows, tiles, k split over workgroups, copies of unaligned rows, operands
of any alignment, and by experts. The weights have a NaN scale, an infinite scale and a NaN code, so that
0 times any of them shows. Rows with a token are held to the same call on their own tokens' codes, bit by
bit: the same tiles and order of sums, NaN in the same places."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def blocks(n):
    return -(-n // 128)


def operands(T, m, n, g, first=0, pad=0):
    """Codes with exponents 3 to 6 in rows `pad` bytes longer than n, `first` bytes off; and scales."""
    def codes(rows):
        b = torch.randint(80, 112, (rows, n), generator=g) + 128 * torch.randint(0, 2, (rows, n), generator=g)
        buf = torch.zeros(rows, n + pad + first, dtype=torch.uint8, device="cuda")
        buf[:, first:first + n] = b.to(torch.uint8).cuda()
        return buf[:, first:first + n]
    sx = torch.rand(T, blocks(n), generator=g) + 0.5
    sw = torch.rand(blocks(m), blocks(n), generator=g) + 0.5
    return codes(T), sx.cuda(), codes(m), sw.cuda()


def spoil(W, sw):
    """A NaN code in row 2, and in the second 128 rows a NaN and an infinite scale."""
    W[2, W.size(1) // 2] = 0x7f
    if sw.size(0) > 1:
        sw[1, sw.size(1) // 2] = float("nan")
        sw[1, 0] = float("inf")


def some_missing(R, T, g):
    """An order of R rows of T tokens, a third of which name none: below 0, T and beyond."""
    order = torch.randint(0, T, (R,), generator=g, dtype=torch.int32)
    at = torch.arange(R) % 3 == 1
    order[at] = torch.tensor([-1, T, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.arange(int(at.sum())) % 4]
    return order, at


def check(bk, X, sx, W, sw, order, missing, t, offsets=None):
    call = lambda x, s, o: bk.matmul_fp8(x.view(F8), s, W.view(F8), sw, offsets=offsets, order=o, out_dtype=TYPES[t])
    Y = call(X, sx, order.cuda())
    assert (Y[missing] == 0).all(), Y[missing].isnan().sum()
    # the same rows, their missing tokens replaced by the first one's
    full = torch.where(missing, 0, order).cuda()
    Z = call(X, sx, full)
    assert torch.isnan(Z).any() and not torch.isnan(Z).all()
    keep = ~missing
    assert torch.equal(Y[keep].isnan(), Z[keep].isnan()) and torch.equal(Y[keep].nan_to_num(), Z[keep].nan_to_num())


# few rows; tiles over all of k; k split (the workspace holds the ranges' sums); odd lengths in place
@pytest.mark.parametrize("R,m,n,splits", [(5, 130, 400, False), (16, 300, 4096, False), (300, 5000, 128, False),
                                          (300, 1000, 4096, True), (300, 130, 16384, True), (100, 130, 4097, True),
                                          (2000, 2100, 400, False)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_one_layer(gpu_lib, R, m, n, splits, t):
    bk = gpu_lib
    g = torch.Generator().manual_seed(R + m + n)
    T = 70
    code = {"f32": bk.F32, "bf16": bk.BF16, "f16": bk.F16}[t]
    need = bk.lib().bakron_matmul_fp8_workspace_bytes(code, T, R, 1, m, n // 16 * 16)
    assert (need >= 2 * 4 * m * R) == splits  # sums of at least two ranges
    X, sx, W, sw = operands(T, m, n, g, pad=-n % 16)
    spoil(W, sw)
    order, missing = some_missing(R, T, g)
    check(bk, X, sx, W, sw, order, missing, t)


# rows that do not start on 16 bytes: of whole groups of 16 (read through registers) and not (copied first)
@pytest.mark.parametrize("R,m,n,first,pad", [(300, 200, 400, 5, 0), (300, 1000, 4096, 1, 15), (100, 130, 4096, 0, 3),
                                             (300, 200, 401, 0, 0), (9, 200, 400, 5, 0)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_any_alignment(gpu_lib, R, m, n, first, pad, t):
    g = torch.Generator().manual_seed(R + m + n + first)
    X, sx, W, sw = operands(70, m, n, g, first, pad)
    spoil(W, sw)
    order, missing = some_missing(R, 70, g)
    check(gpu_lib, X, sx, W, sw, order, missing, t)


@pytest.mark.parametrize("first", [0, 5])
@pytest.mark.parametrize("R", [20, 900])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_by_experts(gpu_lib, first, R, t):
    """Rows without a token inside the groups, on tiles, on the few rows' kernel and at any alignment."""
    g = torch.Generator().manual_seed(R + first)
    E, m, n = 3, 200, 2048
    X, sx, W, sw = operands(70, E * m, n, g, first, 16 - first)
    sw = (torch.rand(E, blocks(m), blocks(n), generator=g) + 0.5).cuda()
    W = W.view(torch.uint8).as_strided((E, m, n), (m * W.stride(0), W.stride(0), 1), W.storage_offset())
    for e in (0, 2):
        spoil(W[e], sw[e])
    order, missing = some_missing(R, 70, g)
    off = torch.tensor([0, R // 2, R // 2 + R // 5, R], dtype=torch.int32).cuda()
    check(gpu_lib, X, sx, W, sw, order, missing, t, offsets=off)


@pytest.mark.parametrize("T", [0, 1])
@pytest.mark.parametrize("m,n", [(130, 16384), (1000, 4096)])
def test_no_token_at_all(gpu_lib, T, m, n):
    """k split, and every row of the order names none."""
    g = torch.Generator().manual_seed(m)
    X, sx, W, sw = operands(T, m, n, g)
    spoil(W, sw)
    order = torch.full((300,), T, dtype=torch.int32).cuda()
    for t in TYPES.values():
        Y = gpu_lib.matmul_fp8(X.view(F8), sx, W.view(F8), sw, order=order, out_dtype=t)
        assert Y.shape == (300, m) and (Y == 0).all()
