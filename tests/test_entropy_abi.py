"""Refusals of the cross entropy, through the C ABI and the binding (no GPU:
every call here fails its checks or has nothing to do)."""
import ctypes

import pytest
import torch

import kronecker_factored_gptq_amd as bk


def at(k):
    """An address that is never dereferenced."""
    return ctypes.c_void_p(0x100000 * k)


def _forward(**kw):
    a = dict(t=bk.F32, T=3, d=4, V=6, X=at(1), ldx=4, W=at(2), ldw=4, y=at(3), loss=at(4), lse=at(5), ws=at(6),
             wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_cross_entropy(a["t"], a["T"], a["d"], a["V"], a["X"], a["ldx"], a["W"], a["ldw"], a["y"],
                                         a["loss"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=4), dict(T=-1), dict(d=-1), dict(V=0), dict(V=-1), dict(T=(1 << 20) + 1),
    dict(d=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), dict(V=1 << 31), dict(X=None), dict(W=None), dict(y=None),
    dict(loss=None), dict(lse=None), dict(ldx=3), dict(ldw=3), dict(ldw=1 << 62), dict(X=ctypes.c_void_p(0x100002)),
    dict(t=bk.F16, W=ctypes.c_void_p(0x200001)), dict(y=ctypes.c_void_p(0x300004)),
    dict(loss=ctypes.c_void_p(0x400002)), dict(lse=ctypes.c_void_p(0x500001)),
    dict(ws=None), dict(wsb=100), dict(ws=ctypes.c_void_p(0x600010)),
    dict(T=1 << 20, V=(1 << 31) - 1),  # more tiles than a launch holds
    dict(loss=at(1)), dict(loss=at(2)), dict(loss=at(3)), dict(lse=at(1)), dict(lse=at(2)), dict(lse=at(3)),
    dict(lse=at(4)),
])
def test_cross_entropy_rejects_bad_arguments(bad):
    assert _forward(**bad) == bk.EINVAL


def _grad(**kw):
    a = dict(t=bk.F32, T=3, d=4, V=6, X=at(1), ldx=4, W=at(2), ldw=4, y=at(3), lse=at(4), g=at(5), dX=at(6), lddx=4,
             dW=at(7), lddw=4, ws=at(8), wsb=1 << 40)
    a.update(kw)
    return bk.lib().bakron_cross_entropy_grad(a["t"], a["T"], a["d"], a["V"], a["X"], a["ldx"], a["W"], a["ldw"],
                                              a["y"], a["lse"], a["g"], a["dX"], a["lddx"], a["dW"], a["lddw"],
                                              a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [
    dict(V=1 << 24), dict(T=1 << 20, V=1 << 18), dict(T=1 << 18, d=1 << 18, ldx=1 << 18, ldw=1 << 18, lddx=1 << 18, lddw=1 << 18),
    dict(V=1 << 18, d=1 << 18, ldx=1 << 18, ldw=1 << 18, lddx=1 << 18, lddw=1 << 18),
])
def test_sizes_past_a_launch_are_refused(kw):
    assert _grad(**kw) == bk.EINVAL
    assert _forward(**{k: v for k, v in kw.items() if k not in ("lddx", "lddw")}) == bk.EINVAL


@pytest.mark.parametrize("bad", [
    dict(t=bk.F64), dict(t=-1), dict(T=-1), dict(d=-1), dict(V=0), dict(T=(1 << 20) + 1), dict(V=1 << 31),
    dict(X=None), dict(W=None), dict(y=None), dict(lse=None), dict(g=None), dict(ldx=3), dict(ldw=3), dict(lddx=3),
    dict(lddw=3), dict(y=ctypes.c_void_p(0x300004)), dict(lse=ctypes.c_void_p(0x400002)),
    dict(g=ctypes.c_void_p(0x500002)), dict(dX=ctypes.c_void_p(0x600001)), dict(dW=ctypes.c_void_p(0x700002)),
    dict(ws=None), dict(wsb=100), dict(ws=ctypes.c_void_p(0x800010)),
    dict(dX=at(1)), dict(dX=at(2)), dict(dX=at(3)), dict(dX=at(4)), dict(dX=at(5)),
    dict(dW=at(1)), dict(dW=at(2)), dict(dW=at(3)), dict(dW=at(4)), dict(dW=at(5)), dict(dW=at(6)),
])
def test_cross_entropy_grad_rejects_bad_arguments(bad):
    assert _grad(**bad) == bk.EINVAL


def test_empty_and_workspaces():
    assert _forward(T=0, X=None, y=None, loss=None, lse=None, ws=None) == bk.OK
    assert _grad(T=0, X=None, y=None, lse=None, g=None, dX=None, dW=None, ws=None) == bk.OK
    assert _grad(d=0, X=None, W=None, dX=None, dW=None, ws=None) == bk.OK
    assert _grad(dX=None, dW=None, ws=None) == bk.OK
    for q in (bk.lib().bakron_cross_entropy_workspace_bytes, bk.lib().bakron_cross_entropy_grad_workspace_bytes):
        assert 0 < q(bk.BF16, 128, 64, 64) < q(bk.F32, 128, 64, 64) < q(bk.F32, 128, 64, 6400)
        assert q(bk.F64, 64, 64, 64) == q(bk.F32, -1, 64, 64) == q(bk.F32, 64, 64, 0) == 0
    # pieces, not the logits: 16384 tokens of 131072 words hold 4 GiB of bfloat16 logits
    assert bk.lib().bakron_cross_entropy_grad_workspace_bytes(bk.BF16, 16384, 4096, 131072) < (3 << 30) // 2


def test_binding_checks(monkeypatch):
    X, W, y = torch.zeros(3, 4), torch.zeros(6, 4), torch.zeros(3, dtype=torch.int64)
    f = torch.zeros(3)
    with pytest.raises(ValueError, match="GPU"):
        bk.cross_entropy(X, W, y)
    # the binding's own checks, on CPU tensors: each call raises before it reaches the library
    monkeypatch.setattr(bk, "_check_device", lambda *ts: torch.device("cpu"))
    for bad in (lambda: bk.cross_entropy(X.double(), W.double(), y), lambda: bk.cross_entropy(X, W.half(), y),
                lambda: bk.cross_entropy(X, W, y.int()), lambda: bk.cross_entropy_grad(X, W, y, f.double(), f),
                lambda: bk.cross_entropy_grad(X, W, y, f, f.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bk.cross_entropy(X[0], W, y), lambda: bk.cross_entropy(X, W[:, :3], y),
                lambda: bk.cross_entropy(X, W[:0], y), lambda: bk.cross_entropy(X, W, y[:2]),
                lambda: bk.cross_entropy(X, torch.zeros(4, 6).t(), y),
                lambda: bk.cross_entropy(X, torch.zeros(1, 4).expand(6, 4), y),
                lambda: bk.cross_entropy(X, W, torch.zeros(6, dtype=torch.int64)[::2]),
                lambda: bk.cross_entropy(X, W, y, workspace=torch.zeros(8, dtype=torch.uint8)),
                lambda: bk.cross_entropy_grad(X, W, y, f[:2], f), lambda: bk.cross_entropy_grad(X, W, y, f, f[:2])):
        with pytest.raises(ValueError):
            bad()


def test_gradient_workspaces_of_few_tokens():
    """Pieces of W, 256 MiB with D's, not W: one bfloat16 token of 4096 on 128256 words (1002 MiB
    of output layer), and three of 2048 on 1.1 million (4.2 GiB); and the planes of operands that are
    read as they are take no room beside D's 256 MiB."""
    q = bk.lib().bakron_cross_entropy_grad_workspace_bytes
    for t in (bk.BF16, bk.F16):
        assert q(t, 1, 4096, 128256) < 264 << 20 and q(t, 3, 2048, 1100000) < 264 << 20
        assert q(t, 4096, 4096, 128256) < 400 << 20
    # the forward's maxima and sums: 8 bytes a token for every 64 words at most of these sizes
    f = bk.lib().bakron_cross_entropy_workspace_bytes
    assert f(bk.BF16, 4096, 4096, 128256) <= 4096 * 8 * (128256 // 64 + 2)
