"""Refusals of the 8-bit product, through the C ABI and the binding (no GPU:
every call here fails its checks or has nothing to do)."""
import ctypes

import pytest
import torch

import kronecker_factored_gptq_amd as bk


def at(k):
    """An address that is never dereferenced."""
    return ctypes.c_void_p(0x100000 * k)


def _quantize(**kw):
    a = dict(t=bk.F32, T=3, n=4, X=at(1), ldx=4, c=None, q=at(2), ldq=4, s=at(3))
    a.update(kw)
    return bk.lib().bakron_quantize_tokens(a["t"], a["T"], a["n"], a["X"], a["ldx"], a["c"], a["q"], a["ldq"],
                                           a["s"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=9), dict(t=-1), dict(T=-1), dict(n=-1), dict(T=1 << 31), dict(X=None), dict(q=None),
    dict(s=None), dict(ldx=3), dict(ldq=3), dict(ldx=1 << 62), dict(X=ctypes.c_void_p(0x100002)),
    dict(s=ctypes.c_void_p(0x300002)), dict(c=ctypes.c_void_p(0x400001)),
    # outputs over inputs, or over each other
    dict(q=at(1)), dict(s=at(1)), dict(s=at(2)), dict(c=at(3)),
])
def test_quantize_tokens_rejects_bad_arguments(bad):
    assert _quantize(**bad) == bk.EINVAL


def test_quantize_tokens_empty():
    assert _quantize(T=0, X=None, q=None, s=None) == bk.OK


def _matmul(**kw):
    a = dict(t=bk.F32, T=3, m=5, n=4, X=at(1), ldx=4, sx=at(2), V=at(3), ldv=4, sv=at(4), Y=at(5), ldy=5, ws=at(9),
             wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_matmul_int8(a["t"], a["T"], a["m"], a["n"], a["X"], a["ldx"], a["sx"], a["V"], a["ldv"],
                                       a["sv"], a["Y"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=4), dict(T=-1), dict(m=-1), dict(n=-1), dict(T=1 << 31), dict(m=1 << 31),
    dict(n=131072, ldx=131072, ldv=131072), dict(X=None), dict(V=None), dict(Y=None), dict(sx=None),
    dict(ldx=3), dict(ldv=3), dict(ldy=4), dict(ldv=1 << 62), dict(Y=ctypes.c_void_p(0x500002)),
    dict(sx=ctypes.c_void_p(0x200001)), dict(sv=ctypes.c_void_p(0x400002)),
    dict(t=bk.BF16, Y=ctypes.c_void_p(0x500001)),
    # more tiles than a launch holds
    dict(T=(1 << 31) - 1, m=(1 << 31) - 1, ldy=(1 << 31) - 1),
    # the output over an input
    dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3)), dict(Y=at(4)),
    # a call that needs a workspace
    dict(T=100, n=8192, ldx=8192, ldv=8192, ws=None), dict(T=100, n=8192, ldx=8192, ldv=8192, wsb=100),
    dict(T=100, n=8192, ldx=8192, ldv=8192, ws=ctypes.c_void_p(0x900008)),
])
def test_matmul_int8_rejects_bad_arguments(bad):
    assert _matmul(**bad) == bk.EINVAL


def test_matmul_int8_empty():
    assert _matmul(T=0, X=None, sx=None, Y=None) == bk.OK
    assert _matmul(m=0, V=None, sv=None, Y=None) == bk.OK
    q = bk.lib().bakron_matmul_int8_workspace_bytes
    assert q(1, 4096, 4096) == q(8192, 14336, 4096) == q(0, 5, 5) == q(5, 0, 5) == q(-1, 5, 5) == 0
    assert 0 < q(100, 4096, 8192) <= 512 * 128 * 128 * 4 + 256


def _grad(**kw):
    a = dict(t=bk.F32, T=3, m=5, n=4, G=at(1), ldg=5, V=at(2), ldv=4, sv=at(3), c=at(4), D=at(5), ldx=4, ws=at(6),
             wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_matmul_int8_grad(a["t"], a["T"], a["m"], a["n"], a["G"], a["ldg"], a["V"], a["ldv"],
                                            a["sv"], a["c"], a["D"], a["ldx"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=4), dict(T=-1), dict(m=-1), dict(n=-1), dict(T=1 << 31), dict(G=None), dict(V=None),
    dict(D=None), dict(ldg=4), dict(ldv=3), dict(ldx=3), dict(m=(1 << 20) + 1, ldg=1 << 21),
    dict(n=(1 << 20) + 1, ldv=1 << 21, ldx=1 << 21), dict(G=ctypes.c_void_p(0x100002)),
    dict(D=ctypes.c_void_p(0x500002)), dict(sv=ctypes.c_void_p(0x300002)), dict(c=ctypes.c_void_p(0x400002)),
    dict(ws=None), dict(wsb=1000), dict(ws=ctypes.c_void_p(0x600008)),
    dict(D=at(1)), dict(D=at(2)), dict(D=at(3)), dict(D=at(4)),
])
def test_matmul_int8_grad_rejects_bad_arguments(bad):
    assert _grad(**bad) == bk.EINVAL


def test_matmul_int8_grad_empty_and_workspace():
    assert _grad(T=0, G=None, D=None, ws=None) == bk.OK
    assert _grad(n=0, V=None, c=None, D=None, ws=None) == bk.OK
    q = bk.lib().bakron_matmul_int8_grad_workspace_bytes
    assert 0 < q(bk.BF16, 64, 64, 64) == q(bk.F16, 64, 64, 64) < q(bk.F32, 64, 64, 64) < q(bk.F32, 64, 200, 64)
    assert q(bk.F64, 64, 64, 64) == q(bk.F32, -1, 64, 64) == q(bk.F32, 64, 1 << 21, 64) == 0


def test_sizes_past_a_launch_are_refused():
    big = 1 << 24
    assert _quantize(T=big) == bk.EINVAL
    for kw in (dict(T=big), dict(m=big, ldy=big), dict(T=1 << 20, m=1 << 19, ldy=1 << 19),
               dict(T=1 << 20, n=100001, ldx=100001, ldv=100001)):
        assert _matmul(**kw) == bk.EINVAL
    for kw in (dict(T=big), dict(T=1 << 18, m=1 << 18, ldg=1 << 18),
               dict(m=1 << 18, n=1 << 18, ldg=1 << 18, ldv=1 << 18, ldx=1 << 18)):
        assert _grad(**kw) == bk.EINVAL


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4)
    q = torch.zeros(2, 4, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        bk.quantize_tokens(x)
    with pytest.raises(ValueError, match="GPU"):
        bk.matmul_int8(q, x[:, 0].contiguous(), q)


@pytest.fixture
def as_if_gpu(monkeypatch):
    """The binding's own checks, on CPU tensors (nothing is launched: each call
    raises before it reaches the library)."""
    monkeypatch.setattr(bk, "_check_device", lambda *ts: torch.device("cpu"))


def test_binding_checks(as_if_gpu):
    x, q = torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.int8)
    s = torch.ones(3)
    for bad in (lambda: bk.quantize_tokens(x.double()), lambda: bk.quantize_tokens(x, torch.ones(4).double()),
                lambda: bk.matmul_int8(x, s, q), lambda: bk.matmul_int8(q, s, q.to(torch.int32)),
                lambda: bk.matmul_int8(q, s.double(), q), lambda: bk.matmul_int8(q, s, q, s.half()),
                lambda: bk.matmul_int8(q, s, q, out_dtype=torch.float64),
                lambda: bk.matmul_int8_grad(x.double(), q), lambda: bk.matmul_int8_grad(x[:, :3], x),
                lambda: bk.matmul_int8_grad(x[:, :3], q, s.double()),
                lambda: bk.matmul_int8_grad(x[:, :3], q, out=torch.zeros(3, 4).half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bk.quantize_tokens(x[0]), lambda: bk.quantize_tokens(x.t()),
                lambda: bk.quantize_tokens(x, torch.ones(3)), lambda: bk.quantize_tokens(x, torch.ones(8)[::2]),
                lambda: bk.quantize_tokens(torch.zeros(1, 4).expand(3, 4)),
                lambda: bk.matmul_int8(q.t(), s, q), lambda: bk.matmul_int8(q, s[:2], q),
                lambda: bk.matmul_int8(q, s, q[:, :3]), lambda: bk.matmul_int8(q, s, q, torch.ones(4)),
                lambda: bk.matmul_int8(q, s, q, out=torch.zeros(3, 4)),
                lambda: bk.matmul_int8_grad(x, q), lambda: bk.matmul_int8_grad(x[:, :3], q, torch.ones(4)),
                lambda: bk.matmul_int8_grad(x[:, :3], q, s, torch.ones(3)),
                lambda: bk.matmul_int8_grad(x[:, :3], q, s, out=torch.zeros(3, 3)),
                lambda: bk.matmul_int8_grad(x[:, :3], q, workspace=torch.zeros(9, dtype=torch.uint8)),
                lambda: bk.matmul_int8(q, s, q, out=torch.zeros(3, 6)[:, ::2])):
        with pytest.raises(ValueError):
            bad()
