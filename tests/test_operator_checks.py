"""The pre-norm, its gradient and the few-token layer without a GPU: the
oracle's formulas are pinned, and bad arguments are refused on the host."""
import ctypes

import numpy as np
import pytest
import torch

from fine_grained_fp8_sigmoid_b200 import _lib
from fine_grained_fp8_sigmoid_b200 import binding as B
from oracle import moe as O


def test_rmsnorm_oracle():
    s = np.array([[3.0, 4.0], [0.0, 0.0]])
    y = O.rmsnorm(s, np.array([1.0, 2.0]), 0.5)
    r = 1.0 / np.sqrt(13.0)
    assert np.allclose(y, [[3 * r, 8 * r], [0, 0]], rtol=1e-15)


@pytest.mark.parametrize("with_dres", [False, True])
def test_rmsnorm_backward_oracle(with_dres):
    g = torch.Generator().manual_seed(0)
    h = torch.randn(5, 24, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(24, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 24, generator=g, dtype=torch.float64)
    dres = torch.randn(5, 24, generator=g, dtype=torch.float64) if with_dres else None
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-3) * w
    loss = (y * dy).sum() + (0 if dres is None else (h * dres).sum())
    loss.backward()
    a = [t.detach().numpy() for t in (dy, h, w)]
    dh, dw = O.rmsnorm_backward(*a, 1e-3, None if dres is None else dres.numpy())
    assert np.allclose(dh, h.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-12, atol=1e-13)
    # and against differences of the forward
    f = lambda hh: (O.rmsnorm(hh, a[2], 1e-3) * a[0]).sum() + (0 if dres is None else (hh * dres.numpy()).sum())
    for i, j in ((0, 0), (3, 17)):
        e = np.zeros_like(a[1])
        e[i, j] = 1e-5
        assert abs((f(a[1] + e) - f(a[1] - e)) / 2e-5 - dh[i, j]) < 1e-8


def _codes(*statuses):
    return [getattr(_lib, "MOE_" + s) for s in statuses]


def test_norm_refusals():
    lib = _lib.load()
    N, s, f = None, ctypes.c_void_p(0), ctypes.c_float
    A = ctypes.c_void_p(1 << 20)             # an aligned address that is never read
    bad = ctypes.c_void_p((1 << 20) + 2)
    INV, UNS = _codes("ERR_INVALID_ARG", "ERR_UNSUPPORTED")
    call = lambda x=A, ldx=256, res=N, w=A, eps=1e-6, rows=4, d=256, h=N, y=A, q=N, sc=N: lib.moe_rmsnorm_quant(
        x, ldx, res, 0, w, 0, f(eps), rows, d, h, y, q, sc, s)
    assert call(rows=0) == 0
    assert call(rows=-1) == INV and call(eps=-1.0) == INV and call(eps=float("nan")) == INV
    assert call(ldx=128) == INV                      # rows would overlap
    assert call(ldx=260) == UNS
    assert call(d=260, ldx=264) == UNS               # no multiple of 8
    assert call(d=264, ldx=264, q=A, sc=A) == UNS    # no whole tiles
    assert call(d=32776, ldx=32776) == UNS
    assert call(x=N) == INV and call(w=N) == INV and call(y=N) == INV
    assert call(q=A) == INV and call(sc=A) == INV    # one without the other
    assert call(x=bad) == INV and call(y=bad) == INV and call(res=bad) == INV
    assert lib.moe_rmsnorm_backward_workspace(0, 256) == 0
    assert lib.moe_rmsnorm_backward_workspace(3, 256) == 3 * 256 * 4
    size = lib.moe_rmsnorm_backward_workspace(100000, 256)
    assert 0 < size <= 1024 * 256 * 4
    back = lambda dy=A, h=A, w=A, eps=1e-6, rows=4, d=256, dh=A, dw=A, ws=A, n=1 << 20: lib.moe_rmsnorm_backward(
        dy, h, 0, w, 0, f(eps), N, rows, d, dh, dw, ws, n, s)
    assert back(d=260) == UNS and back(d=16392) == UNS
    assert back(n=16) == INV and back(ws=N) == INV and back(dw=N) == INV and back(dh=bad) == INV
    assert back(rows=-2) == INV and back(eps=-1.0) == INV


def test_norm_backward_refuses_rows_past_2_to_the_30():
    lib = _lib.load()
    A, N = ctypes.c_void_p(1 << 20), None    # an address that is never read
    size = lib.moe_rmsnorm_backward_workspace(2**31 - 1, 8)
    assert size == lib.moe_rmsnorm_backward_workspace(1 << 30, 8)
    for rows in ((1 << 30) + 1, 2**31 - 1):
        assert lib.moe_rmsnorm_backward(A, A, 0, A, 0, ctypes.c_float(1e-6), N, rows, 8, A, A, A, size,
                                        ctypes.c_void_p(0)) == _lib.MOE_ERR_UNSUPPORTED


def test_few_tokens_refusals():
    lib = _lib.load()
    N, s = None, ctypes.c_void_p(0)
    A = ctypes.c_void_p(1 << 20)
    bad = ctypes.c_void_p((1 << 20) + 2)
    INV, UNS = _codes("ERR_INVALID_ARG", "ERR_UNSUPPORTED")

    def call(u=A, xq=N, xs=N, e=A, T=4, d=256, N_r=8, K=2, w=A, sc=A, I=128, out=A, idx=A, ws=A, n=1 << 30):
        return lib.moe_few_tokens(u, xq, xs, N, e, A, T, d, N_r, K, w, A, A, sc, A, A, I, out, idx, A, N, ws, n, s)

    assert call(T=0) == 0
    assert call(T=-1) == INV and call(T=17) == UNS
    assert call(K=9) == UNS and call(K=0) == UNS and call(K=17, N_r=64) == UNS
    assert call(N_r=257) == UNS and call(N_r=0) == INV
    assert call(d=128) == UNS and call(d=8448) == UNS and call(d=0) == INV
    assert call(I=192) == UNS and call(I=8320) == UNS and call(I=0) == INV
    assert call(u=N) == INV and call(e=N) == INV and call(w=N) == INV and call(sc=N) == INV
    assert call(out=N) == INV and call(idx=N) == INV and call(ws=N) == INV
    assert call(xq=A) == INV and call(xs=A) == INV       # one without the other
    assert call(u=bad) == INV and call(w=bad) == INV and call(ws=bad) == INV
    need = lib.moe_few_tokens_workspace(4, 256, 8, 2, 128)
    assert need > 0 and call(n=need - 1) == INV
    assert lib.moe_few_tokens_workspace(17, 256, 8, 2, 128) == 0
    assert lib.moe_few_tokens_workspace(0, 256, 8, 2, 128) == 0
    assert lib.moe_few_tokens_workspace(4, 256, 8, 9, 128) == 0


class _OnDevice:
    """A host tensor that says it lives on CUDA device `dev`."""

    def __init__(self, t, dev):
        self._t, self._dev, self.is_cuda, self.device = t, dev, True, f"cuda:{dev}"

    def get_device(self):
        return self._dev

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_binding_names_what_is_wrong():
    bf = torch.bfloat16
    x = torch.zeros(4, 128, dtype=bf)
    with pytest.raises(ValueError, match="y must be a CUDA tensor"):
        B._p(x, bf, (4, 128), 0, "y")
    with pytest.raises(ValueError, match="y: dtype"):
        B._p(_OnDevice(x, 0), torch.float32, (4, 128), 0, "y")
    with pytest.raises(ValueError, match="y: shape"):
        B._p(_OnDevice(x, 0), bf, (4, 256), 0, "y")
    with pytest.raises(ValueError, match="y must be contiguous"):
        B._p(_OnDevice(x.t(), 0), bf, (128, 4), 0, "y")
    with pytest.raises(ValueError, match="y is on cuda:1, but the current device is cuda:0"):
        B._p(_OnDevice(x, 1), bf, (4, 128), 0, "y")
    with pytest.raises(ValueError, match="y is required"):
        B._p(None, bf, (4, 128), 0, "y")
    assert B._p(_OnDevice(x, 0), bf, (4, 128), 0, "y") == x.data_ptr()
    assert B._popt(None, bf, (4, 128), 0, "y") is None
    for bad in (None, x, _OnDevice(x, 1), _OnDevice(x.t(), 0)):
        with pytest.raises(ValueError, match="workspace"):
            B._ws(bad, 0)
    with pytest.raises(ValueError, match="CUDA matrix"):
        B.moe_rmsnorm_quant(x, torch.ones(128), 1e-6, y=x)
