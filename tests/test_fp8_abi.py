"""Refusals of 8-bit floating point and of the tokens of experts, through the C ABI and
the binding (no GPU: every call here fails its checks or has nothing to do)."""
import ctypes

import pytest
import torch

import kronecker_factored_gptq_amd as bk

F8 = torch.float8_e4m3fn


def at(k, more=0):
    """An address that is never dereferenced."""
    return ctypes.c_void_p(0x1000000 * k + more)


def _quantize(**kw):
    a = dict(t=bk.F32, batch=2, rows=5, n=300, X=at(1), ldx=300, sX=1500, br=1, q=at(2), ldq=304, sQ=1520, s=at(3),
             srow=1, sblock=5, sS=15)
    a.update(kw)
    return bk.lib().bakron_quantize_fp8(a["t"], a["batch"], a["rows"], a["n"], a["X"], a["ldx"], a["sX"], a["br"],
                                        a["q"], a["ldq"], a["sQ"], a["s"], a["srow"], a["sblock"], a["sS"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=7), dict(batch=-1), dict(rows=-1), dict(n=-1), dict(br=0), dict(br=64), dict(batch=65536),
    dict(rows=1 << 24), dict(X=None), dict(q=None), dict(s=None), dict(ldx=299), dict(ldq=299), dict(ldx=1 << 62),
    dict(X=at(1, 2)), dict(s=at(3, 2)), dict(sX=-1), dict(sQ=-1), dict(sS=-1), dict(srow=-1), dict(sblock=-1),
    # outputs over each other, or over the input
    dict(sQ=1519 - 4), dict(sS=14), dict(srow=0), dict(sblock=0), dict(srow=2, sblock=5, sS=100), dict(q=at(1)),
    dict(s=at(1)), dict(s=at(2)), dict(q=at(1, 4 * 2999)), dict(rows=1 << 23, n=1 << 20, batch=1, ldx=1 << 20, ldq=1 << 20),
])
def test_quantize_fp8_rejects_bad_arguments(bad):
    assert _quantize(**bad) == bk.EINVAL


def test_quantize_fp8_empty():
    for kw in (dict(batch=0), dict(rows=0), dict(n=0)):
        assert _quantize(X=None, q=None, s=None, **kw) == bk.OK


def _matmul(**kw):
    a = dict(t=bk.F32, T=3, R=12, E=4, m=140, n=300, X=at(1), ldx=300, sx=at(2), st=1, sb=3, W=at(3), ldw=300,
             sW=42000, sw=at(4), ldsw=3, sS=6, off=at(5), order=at(6), per=4, Y=at(7), ldy=140, ws=at(9), wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_matmul_fp8(a["t"], a["T"], a["R"], a["E"], a["m"], a["n"], a["X"], a["ldx"], a["sx"],
                                      a["st"], a["sb"], a["W"], a["ldw"], a["sW"], a["sw"], a["ldsw"], a["sS"],
                                      a["off"], a["order"], a["per"], a["Y"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=-1), dict(T=-1), dict(R=-1), dict(E=0), dict(E=1025), dict(m=-1), dict(n=-1),
    dict(T=1 << 24), dict(R=1 << 24), dict(m=(1 << 20) + 1, ldy=1 << 21), dict(n=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21),
    dict(X=None), dict(sx=None), dict(W=None), dict(sw=None), dict(Y=None), dict(ldx=299), dict(ldw=299), dict(ldsw=2),
    dict(ldy=139), dict(sW=-1), dict(sS=-1), dict(st=-1), dict(sb=-1), dict(ldw=1 << 62), dict(sW=1 << 62),
    dict(Y=at(7, 2)), dict(sx=at(2, 1)), dict(sw=at(4, 2)), dict(off=at(5, 2)), dict(order=at(6, 3)),
    dict(t=bk.F16, Y=at(7, 1)), dict(off=None), dict(order=None), dict(per=0), dict(per=1 << 31),
    # the output over an input
    dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3)), dict(Y=at(4)), dict(Y=at(5)), dict(Y=at(6)),
    dict(Y=at(3, 4 * 41996)),
    # more than a launch holds
    dict(R=(1 << 24) - 1, m=1 << 20, ldy=1 << 20),
])
def test_matmul_fp8_rejects_bad_arguments(bad):
    assert _matmul(**bad) == bk.EINVAL


def test_matmul_fp8_empty():
    assert _matmul(R=0, order=at(6), Y=None) == bk.OK
    assert _matmul(m=0, W=None, sw=None, Y=None) == bk.OK
    q = bk.lib().bakron_matmul_fp8_workspace_bytes
    assert q(bk.F64, 3, 12, 4, 140, 300) == q(bk.F32, -1, 12, 4, 140, 300) == q(bk.F32, 3, 12, 0, 140, 300) == 0


def _grad(**kw):
    a = dict(t=bk.F32, R=12, E=4, m=140, n=300, G=at(1), ldg=140, W=at(3), ldw=300, sW=42000, sw=at(4), ldsw=3, sS=6,
             off=at(5), D=at(7), ldx=300, ws=at(9), wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_matmul_fp8_grad(a["t"], a["R"], a["E"], a["m"], a["n"], a["G"], a["ldg"], a["W"], a["ldw"],
                                           a["sW"], a["sw"], a["ldsw"], a["sS"], a["off"], a["D"], a["ldx"], a["ws"],
                                           a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=4), dict(R=-1), dict(E=0), dict(E=1025), dict(m=-1), dict(n=-1), dict(R=1 << 24),
    dict(m=(1 << 20) + 1, ldg=1 << 21), dict(n=(1 << 20) + 1, ldw=1 << 21, ldx=1 << 21), dict(G=None), dict(W=None),
    dict(sw=None), dict(D=None), dict(ldg=139), dict(ldw=299), dict(ldsw=2), dict(ldx=299), dict(sW=-1), dict(sS=-1),
    dict(G=at(1, 2)), dict(D=at(7, 2)), dict(sw=at(4, 1)), dict(off=at(5, 1)), dict(off=None),
    dict(D=at(1)), dict(D=at(3)), dict(D=at(4)), dict(D=at(5)), dict(R=(1 << 24) - 1, n=1 << 19, ldw=1 << 19, ldx=1 << 19),
])
def test_matmul_fp8_grad_rejects_bad_arguments(bad):
    assert _grad(**bad) == bk.EINVAL


def test_matmul_fp8_grad_empty():
    assert _grad(R=0, G=None, D=None) == bk.OK
    assert _grad(n=0, W=None, sw=None, D=None) == bk.OK
    q = bk.lib().bakron_matmul_fp8_grad_workspace_bytes
    assert q(bk.F64, 12, 4, 140, 300) == q(bk.F32, -1, 4, 140, 300) == q(bk.F32, 12, 1025, 140, 300) == 0


def _sort(**kw):
    a = dict(T=1000, k=3, E=7, ids=at(1), ld=3, order=at(2), slots=at(3), off=at(4), ws=at(5), wsb=1 << 30)
    a.update(kw)
    return bk.lib().bakron_sort_tokens(a["T"], a["k"], a["E"], a["ids"], a["ld"], a["order"], a["slots"], a["off"],
                                       a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(T=1 << 30), dict(ids=None), dict(order=None), dict(slots=None),
    dict(off=None), dict(ld=2), dict(ids=at(1, 4)), dict(order=at(2, 2)), dict(slots=at(3, 1)), dict(off=at(4, 2)),
    dict(ws=None), dict(wsb=8), dict(ws=at(5, 8)), dict(order=at(1)), dict(slots=at(1)), dict(off=at(1)),
    dict(slots=at(2)), dict(off=at(2)), dict(off=at(3)),
])
def test_sort_tokens_rejects_bad_arguments(bad):
    assert _sort(**bad) == bk.EINVAL


def test_sort_tokens_workspace():
    q = bk.lib().bakron_sort_tokens_workspace_bytes
    assert q(1, 8, 64) == q(0, 8, 64) == q(-1, 8, 64) == q(8, 0, 64) == q(8, 1, 1025) == 0
    assert q(8192, 8, 128) > 0


def _gather(**kw):
    a = dict(t=bk.F32, T=5, n=20, X=at(1), ldx=20, per=2, R=10, order=at(2), Xs=at(3), ldxs=20)
    a.update(kw)
    return bk.lib().bakron_gather_tokens(a["t"], a["T"], a["n"], a["X"], a["ldx"], a["per"], a["R"], a["order"],
                                         a["Xs"], a["ldxs"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(T=-1), dict(n=-1), dict(R=-1), dict(per=0), dict(R=1 << 27), dict(X=None), dict(order=None),
    dict(Xs=None), dict(ldx=19), dict(ldxs=19), dict(X=at(1, 2)), dict(Xs=at(3, 1)), dict(order=at(2, 2)),
    dict(Xs=at(1)), dict(Xs=at(2)),
])
def test_gather_tokens_rejects_bad_arguments(bad):
    assert _gather(**bad) == bk.EINVAL


def _combine(**kw):
    a = dict(t=bk.F32, T=5, k=2, n=20, R=10, Ys=at(1), ldys=20, slots=at(2), w=at(3), Y=at(4), ldy=20)
    a.update(kw)
    return bk.lib().bakron_combine_tokens(a["t"], a["T"], a["k"], a["n"], a["R"], a["Ys"], a["ldys"], a["slots"],
                                          a["w"], a["Y"], a["ldy"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(T=-1), dict(k=-1), dict(n=-1), dict(R=-1), dict(T=1 << 24), dict(k=1 << 30), dict(Ys=None),
    dict(slots=None), dict(Y=None), dict(ldys=19), dict(ldy=19), dict(Ys=at(1, 2)), dict(w=at(3, 2)),
    dict(slots=at(2, 1)), dict(Y=at(4, 2)), dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3)),
    dict(T=(1 << 24) - 1, k=1, n=1 << 20, ldys=1 << 20, ldy=1 << 20),
])
def test_combine_tokens_rejects_bad_arguments(bad):
    assert _combine(**bad) == bk.EINVAL


def _combine_grad(**kw):
    a = dict(t=bk.F32, T=5, k=2, n=20, R=10, G=at(1), ldg=20, Ys=at(2), ldys=20, slots=at(3), w=at(4), D=at(5), ldd=20,
             dw=at(6))
    a.update(kw)
    return bk.lib().bakron_combine_tokens_grad(a["t"], a["T"], a["k"], a["n"], a["R"], a["G"], a["ldg"], a["Ys"],
                                               a["ldys"], a["slots"], a["w"], a["D"], a["ldd"], a["dw"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(T=-1), dict(k=-1), dict(n=-1), dict(R=-1), dict(T=1 << 24), dict(k=1 << 30), dict(G=None),
    dict(Ys=None), dict(slots=None), dict(ldg=19), dict(ldys=19), dict(ldd=19), dict(G=at(1, 2)), dict(dw=at(6, 1)),
    dict(w=at(4, 1)), dict(D=at(5, 2)), dict(D=at(1)), dict(D=at(2)), dict(D=at(3)), dict(D=at(4)), dict(dw=at(5)),
    dict(dw=at(1)), dict(dw=at(2)), dict(dw=at(3)), dict(dw=at(4)),
    dict(T=(1 << 24) - 1, k=100),
])
def test_combine_tokens_grad_rejects_bad_arguments(bad):
    assert _combine_grad(**bad) == bk.EINVAL


def test_nothing_to_move():
    assert _gather(R=0, order=None, Xs=None) == _gather(n=0, X=None, Xs=None) == bk.OK
    assert _combine(T=0, slots=None, Y=None) == _combine(n=0, Ys=None, Y=None) == bk.OK
    assert _combine_grad(T=0, G=None) == _combine_grad(D=None, dw=None) == _combine_grad(k=0, slots=None) == bk.OK


@pytest.fixture
def as_if_gpu(monkeypatch):
    """The binding's own checks, on CPU tensors (nothing is launched: each call
    raises before it reaches the library)."""
    monkeypatch.setattr(bk, "_check_device", lambda *ts: torch.device("cpu"))


def test_binding_refuses_cpu_tensors():
    x, q, s = torch.zeros(2, 4), torch.zeros(2, 4, dtype=F8), torch.zeros(2, 1)
    i = torch.zeros(2, 4, dtype=torch.int64)
    for call in (lambda: bk.quantize_fp8(x), lambda: bk.matmul_fp8(q, s, q, s[:1]), lambda: bk.matmul_fp8_grad(x, q, s),
                 lambda: bk.sort_tokens(i, 3), lambda: bk.gather_tokens(x, i[0].int()),
                 lambda: bk.combine_tokens(x, i.int()), lambda: bk.combine_tokens_grad(x, x, i.int())):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_checks(as_if_gpu):
    x, q = torch.zeros(3, 4), torch.zeros(3, 4, dtype=F8)
    sx, sw, off = torch.ones(3, 1), torch.ones(1, 1), torch.zeros(3, dtype=torch.int32)
    q3, s3, i = torch.zeros(2, 3, 4, dtype=F8), torch.ones(2, 1, 1), torch.zeros(3, 2, dtype=torch.int64)
    y, w = torch.zeros(6, 4), torch.ones(3, 2)
    for bad in (lambda: bk.quantize_fp8(x.double()), lambda: bk.matmul_fp8(x, sx, q, sw),
                lambda: bk.matmul_fp8(q, sx.double(), q, sw), lambda: bk.matmul_fp8(q, sx, q.view(torch.int8), sw),
                lambda: bk.matmul_fp8(q, sx, q, sw.double()), lambda: bk.matmul_fp8(q, sx, q, sw, out_dtype=torch.float64),
                lambda: bk.matmul_fp8(q, sx, q3, s3, offsets=off.long()),
                lambda: bk.matmul_fp8(q, sx, q, sw, order=off.long()),
                lambda: bk.matmul_fp8_grad(x[:, :3].double(), q, sw), lambda: bk.matmul_fp8_grad(x[:, :3], x, sw),
                lambda: bk.matmul_fp8_grad(x[:, :3], q, sw, out=torch.zeros(3, 4).half()),
                lambda: bk.sort_tokens(i.int(), 4), lambda: bk.gather_tokens(x.double(), off),
                lambda: bk.gather_tokens(x, off.long()), lambda: bk.combine_tokens(y.double(), i.int()),
                lambda: bk.combine_tokens(y, i), lambda: bk.combine_tokens(y, i.int(), w.double()),
                lambda: bk.combine_tokens_grad(x.half(), y, i.int())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bk.quantize_fp8(x[0]), lambda: bk.quantize_fp8(x.t()), lambda: bk.quantize_fp8(x, 64),
                lambda: bk.quantize_fp8(torch.zeros(1, 4).expand(3, 4)), lambda: bk.quantize_fp8(torch.zeros(2, 2, 3, 4)),
                lambda: bk.matmul_fp8(q.t(), sx, q, sw), lambda: bk.matmul_fp8(q, sx[:2], q, sw),
                lambda: bk.matmul_fp8(q, sx, q[:, :3], sw), lambda: bk.matmul_fp8(q, sx, q, sx),
                lambda: bk.matmul_fp8(q, sx, q3, s3), lambda: bk.matmul_fp8(q, sx, q, sw, offsets=off),
                lambda: bk.matmul_fp8(q, sx, q3, s3, offsets=off[:2]),
                lambda: bk.matmul_fp8(q, sx, q3[:0], s3[:0], offsets=off[:1]),
                lambda: bk.matmul_fp8(q, sx, q, sw, order=i.int()), lambda: bk.matmul_fp8(q, sx, q, sw, per_token=0),
                lambda: bk.matmul_fp8(q, sx, q, sw, out=torch.zeros(3, 4)),
                lambda: bk.matmul_fp8_grad(x, q, sw), lambda: bk.matmul_fp8_grad(x[:, :3], q3, s3),
                lambda: bk.matmul_fp8_grad(x[:, :3], q, sw, out=torch.zeros(3, 3)),
                lambda: bk.sort_tokens(i[0], 4), lambda: bk.sort_tokens(i, 0), lambda: bk.sort_tokens(i[:, :0], 3),
                lambda: bk.gather_tokens(x, off[None]), lambda: bk.gather_tokens(x, off, 0),
                lambda: bk.gather_tokens(x, off, out=torch.zeros(2, 4)), lambda: bk.combine_tokens(y, off),
                lambda: bk.combine_tokens(y, i.int().t()), lambda: bk.combine_tokens(y, i.int(), w[:2]),
                lambda: bk.combine_tokens(y, i.int(), out=torch.zeros(2, 4)),
                lambda: bk.combine_tokens_grad(x[:2], y, i.int()), lambda: bk.combine_tokens_grad(x[:, :3], y, i.int())):
        with pytest.raises(ValueError):
            bad()
