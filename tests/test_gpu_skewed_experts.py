"""Products with block scales by experts whose rows are far from even: all of them, or all but a few, to one of many
experts, on the few rows' kernel and on tiles, each result held to 64 bits (tolerances as in
tests/test_gpu_fp8.py: 131 2^-23 + blocks 2^-24 of the terms' absolute sum for codes with exponents 3 to 6, 3 m 2^-23 +
3 2^-24 for the gradient, and half a step of the type)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def codes(*shape, g):
    b = torch.randint(80, 112, shape, generator=g, device="cuda") + 128 * torch.randint(0, 2, shape, generator=g, device="cuda")
    return b.to(torch.uint8).view(F8)


def spread(s, rows, a, n):
    return s.double().repeat_interleave(rows, -2)[..., :a, :].repeat_interleave(128, -1)[..., :n]


def layouts(R, E):
    """Offsets: everything to one expert in the middle; one row to each of the first and last experts and the rest to one;
    half to one, the other half even; the last expert alone."""
    one = torch.full((E + 1,), R)
    one[:E // 3] = 0
    few = torch.arange(E + 1).clamp(max=E // 2)
    few[E // 2 + 1:] = R - (E - 1 - E // 2) + torch.arange(E - E // 2)
    half = torch.arange(E + 1) * (R // 2) // E
    half[E // 4:] += R - R // 2
    last = torch.full((E + 1,), 0)
    last[E] = R
    for o in (one, few, half, last):
        assert o[0] == 0 and o[-1] == R and (o[1:] >= o[:-1]).all()
        yield o


# few rows by the average (R <= 8 E and n >= 2048), and more
@pytest.mark.parametrize("R,E,m,n", [(256, 64, 200, 2048), (511, 64, 130, 2064), (2000, 250, 130, 2049), (1000, 64, 200, 400),
                                     (5000, 64, 300, 384), (9000, 16, 260, 272)])
@pytest.mark.parametrize("t", TYPES)
def test_skewed(gpu_lib, R, E, m, n, t):
    bk = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(R + E)
    X, W = codes(R, n, g=g), codes(E, m, n, g=g)
    nb, mb = -(-n // 128), -(-m // 128)
    sx = torch.rand(R, nb, device="cuda", generator=g) + 0.5
    sw = (torch.rand(E, mb, nb, device="cuda", generator=g) + 0.5) * 2.0 ** -9
    G = torch.randn(R, m, device="cuda", generator=g).to(TYPES[t])
    x = X.float().double() * spread(sx, 1, R, n)
    half = torch.finfo(TYPES[t]).eps / 2 * (1 + 2.0 ** -8)
    for off in layouts(R, E):
        Y = bk.matmul_fp8(X, sx, W, sw, offsets=off.int().cuda(), out_dtype=TYPES[t]).double()
        D = bk.matmul_fp8_grad(G, W, sw, offsets=off.int().cuda()).double()
        for e in range(E):
            a, b = int(off[e]), int(off[e + 1])
            if a == b:
                continue
            v = W[e].float().double() * spread(sw[e], 128, m, n)
            for got, u, v, k in ((Y, x, v.T, 131 * 2.0 ** -23 + nb * 2.0 ** -24), (D, G.double(), v, 3 * m * 2.0 ** -23 + 3 * 2.0 ** -24)):
                ref, S = u[a:b] @ v, u[a:b].abs() @ v.abs()
                assert ((got[a:b] - ref).abs() <= S * k + ref.abs() * half + torch.finfo(TYPES[t]).tiny).all(), (off.tolist(), e)
