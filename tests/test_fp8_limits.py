"""Sizes that 8-bit floating point and the tokens of experts take and refuse: the largest accepted and the
smallest refused, and a call beyond what was refused once."""
import ctypes

import pytest
import torch

import kronecker_factored_gptq_amd as bk


def at(k):
    """An address that is never dereferenced."""
    return ctypes.c_void_p(0x1000000 * k)


def test_the_largest_gather():
    """R <= 2^26 - 4: a wave to a row, four to a workgroup, fewer than 2^24 workgroups. No columns: nothing is launched."""
    gather = lambda R: bk.lib().bakron_gather_tokens(bk.F32, 5, 0, at(1), 1, 1, R, at(2), at(3), 1, None)
    assert gather((1 << 26) - 4) == bk.OK
    assert gather((1 << 26) - 3) == gather(1 << 26) == bk.EINVAL


@pytest.mark.parametrize("rows,n,block_rows", [(((1 << 24) - 1), 8 * 1024 * 128, 1), (1 << 23, 128 * 128 + 1, 1),
                                               ((1 << 24) - 1, 1 << 24, 128), (1 << 24, 1, 1)])
def test_quantize_beyond_one_launch(rows, n, block_rows):
    nb, na = (n + 127) // 128, -(-rows // block_rows)
    assert bk.lib().bakron_quantize_fp8(bk.F32, 1, rows, n, at(1), n, 0, block_rows, ctypes.c_void_p(1 << 56), n, 0,
                                        ctypes.c_void_p(1 << 52), nb, 1, na * nb, None) == bk.EINVAL


@pytest.mark.gpu
def test_quantize_more_than_2_33_elements(gpu_lib):
    """16 GiB of bfloat16 tokens: rows at both ends and in between as they are alone."""
    rows, n = (1 << 23) + 37, 1024
    X = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(4099, n, device="cuda", generator=g).bfloat16()
    for a in range(0, rows, 4099):  # every row some row of base
        b = min(rows, a + 4099)
        X[a:b] = base[:b - a]
    q, s = bk.quantize_fp8(X)
    q, want = q.view(torch.uint8), bk.quantize_fp8(base)
    for a in (0, 4099 * 1000, (rows // 4099 - 1) * 4099):
        assert torch.equal(q[a:a + 4099], want[0].view(torch.uint8)) and torch.equal(s[a:a + 4099], want[1])
    a = rows // 4099 * 4099
    assert torch.equal(q[a:], want[0].view(torch.uint8)[:rows - a]) and torch.equal(s[a:], want[1][:rows - a])
