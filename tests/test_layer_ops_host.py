"""The operators in front of, between and beside the experts' products refuse what they cannot do
before anything is launched (no GPU needed: no call here passes its checks)."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_fp4_top_amd as moe
from tests import layer_ops_ref as ref

L = moe._lib
A, B, C, D, F, G, P, Q, R = (ctypes.c_void_p((i + 1) << 36) for i in range(9))  # far apart, never read
ODD = ctypes.c_void_p((1 << 44) + 1)


def err():
    return L.moe_last_error().decode()


def route(x=A, ld=64, dt=2, bias=B, T=4, E=64, K=8, score=0, groups=8, top=4, best=2, renorm=1, scale=1.0, ids=C, w=D):
    return L.moe_route(x, ld, dt, bias, T, E, K, score, groups, top, best, renorm, scale, ids, w, None)


def test_route_refuses():
    assert route(dt=3) == 1 and route(score=2) == 1 and route(T=-1) == 1
    assert route(E=0, groups=1, top=1) == 1 and route(E=1025, groups=1, top=1) == 1
    assert route(K=0) == 1 and route(K=65) == 1 and route(E=8, K=9) == 1
    assert route(groups=0) == 1 and route(groups=7) == 1 and route(groups=128) == 1 and "divide" in err()
    assert route(top=0) == 1 and route(top=9) == 1 and route(best=0) == 1 and route(best=3) == 1 and route(renorm=2) == 1
    assert route(scale=float("inf")) == 1 and route(scale=float("nan")) == 1
    assert route(T=1 << 21) == 2 and "routes" in err()
    assert route(x=None) == 1 and route(ids=None) == 1 and route(w=None) == 1
    assert route(ld=-1) == 1 and route(ld=1 << 33) == 1
    assert route(x=ODD) == 1 and route(bias=ODD) == 1 and route(ids=ODD) == 1 and route(w=ODD) == 1
    assert route(ids=A) == 1 and route(w=B) == 1 and route(w=C) == 1 and "overlap" in err()


def route_grad(dw=A, x=B, ld=64, dt=2, ids=C, T=4, E=64, K=8, score=0, renorm=1, scale=1.0, out=D, ldo=64):
    return L.moe_route_grad(dw, x, ld, dt, ids, T, E, K, score, renorm, scale, out, ldo, None)


def test_route_grad_refuses():
    assert route_grad(dt=-1) == 1 and route_grad(score=-1) == 1 and route_grad(K=65) == 1 and route_grad(renorm=-1) == 1
    assert route_grad(dw=None) == 1 and route_grad(x=None) == 1 and route_grad(ids=None) == 1 and route_grad(out=None) == 1
    assert route_grad(ldo=63) == 1 and route_grad(ld=-1) == 1 and route_grad(ldo=1 << 33) == 1
    assert route_grad(out=A) == 1 and route_grad(out=B) == 1 and route_grad(out=C) == 1 and route_grad(out=ODD) == 1


def norm(x=A, ldx=64, res=B, ldr=64, dt=0, w=C, wdt=0, rows=4, cols=64, eps=1e-6, total=D, ldt=64, y=F, ldy=64, codes=G,
         ldc=64, scales=P):
    return L.moe_rms_norm(x, ldx, res, ldr, dt, w, wdt, rows, cols, eps, total, ldt, y, ldy, codes, ldc, scales, None)


def test_norm_refuses():
    assert norm(dt=3) == 1 and norm(wdt=1) == 1 and norm(rows=-1) == 1 and norm(rows=(1 << 23) + 1) == 2
    assert norm(cols=0) == 2 and norm(cols=32769, ldx=1 << 16) == 2
    assert norm(eps=-1.0) == 1 and norm(eps=float("nan")) == 1 and norm(eps=float("inf")) == 1
    assert norm(res=None) == 1 and norm(total=None) == 1 and "together" in err()
    assert norm(codes=None) == 1 and norm(scales=None) == 1 and norm(x=None) == 1
    assert norm(y=None, codes=None, scales=None) == 1
    assert norm(ldx=-1) == 1 and norm(ldt=63) == 1 and norm(ldy=63) == 1 and norm(ldc=63) == 1 and norm(ldr=-1) == 1
    assert norm(x=ODD) == 1 and norm(w=ODD) == 1 and norm(total=ODD) == 1 and norm(y=ODD) == 1 and norm(scales=ODD) == 1
    assert norm(total=A) == 1 and norm(y=A) == 1 and norm(y=B) == 1 and norm(codes=C) == 1 and norm(scales=D) == 1
    # total may be the residual, row by row only
    assert norm(total=B, ldt=128) == 1 and norm(total=ctypes.c_void_p(B.value + 2)) == 1
    assert norm(total=B, y=B) == 1 and "overlap" in err()


def norm_grad(dy=A, lddy=64, h=B, ldh=64, dt=0, w=C, wdt=2, dt2=D, ldt=64, rows=4, cols=64, eps=1e-6, ws=F, n=1 << 20, dx=G,
              lddx=64, dw=P):
    return L.moe_rms_norm_grad(dy, lddy, h, ldh, dt, w, wdt, dt2, ldt, rows, cols, eps, ws, n, dx, lddx, dw, None)


def test_norm_grad_refuses():
    assert norm_grad(dt=5) == 1 and norm_grad(wdt=1) == 1 and norm_grad(cols=40000) == 2 and norm_grad(eps=-1.0) == 1
    assert norm_grad(dy=None) == 1 and norm_grad(h=None) == 1 and norm_grad(dx=None) == 1 and norm_grad(ws=None) == 1
    assert norm_grad(n=64 * 4 * 4 - 1) == 3 and "workspace" in err()
    assert norm_grad(lddx=63) == 1 and norm_grad(lddy=-1) == 1 and norm_grad(ldh=-1) == 1 and norm_grad(ldt=-1) == 1
    assert norm_grad(dy=ODD) == 1 and norm_grad(dw=ODD) == 1 and norm_grad(ws=ODD) == 1
    assert norm_grad(dx=A) == 1 and norm_grad(dx=D) == 1 and norm_grad(dw=C) == 1 and norm_grad(ws=B) == 1 and norm_grad(dw=G) == 1
    assert L.moe_rms_norm_grad_workspace_bytes(4, 0) == 0 and L.moe_rms_norm_grad_workspace_bytes(0, 8) > 0
    last = 0
    for rows in (0, 1, 100, 512, 513, 1 << 20):
        now = L.moe_rms_norm_grad_workspace_bytes(rows, 1000)
        assert now >= last
        last = now


def act(h=A, ld=128, dt=0, a=0, rows=8, I=64, off=B, E=4, r2r=C, w=D, out=F, ldo=64):
    return L.moe_activate(h, ld, dt, a, rows, I, off, E, r2r, w, out, ldo, None)


def act_int(h=A, ld=128, dt=0, a=0, rows=8, I=64, off=B, E=4, r2r=C, w=D, codes=F, ldc=64, scales=G):
    return L.moe_activate_int(h, ld, dt, a, rows, I, off, E, r2r, w, codes, ldc, scales, None)


def act_grad(da=P, ldda=64, h=A, ld=128, dt=0, a=0, rows=8, I=64, off=B, E=4, r2r=C, rt2=Q, w=D, dh=F, lddh=128, dw=G):
    return L.moe_activate_grad(da, ldda, h, ld, dt, a, rows, I, off, E, r2r, rt2, w, dh, lddh, dw, None)


@pytest.mark.parametrize("call", [act, act_int, act_grad])
def test_activate_refuses(call):
    assert call(dt=3) == 1 and call(a=2) == 1 and call(rows=-1) == 1 and call(rows=(1 << 23) + 1) == 2
    assert call(I=0) == 2 and call(I=32769) == 2 and call(E=0) == 1 and call(E=1025) == 1
    assert call(off=None) == 1 and call(r2r=None) == 1 and call(h=None) == 1
    assert call(h=ODD) == 1 and call(w=ODD) == 1 and call(off=ODD) == 1 and call(r2r=ODD) == 1 and call(ld=-1) == 1


def test_activate_refuses_outputs():
    assert act(out=None) == 1 and act(ldo=63) == 1 and act(out=ODD) == 1 and act(out=A) == 1 and act(out=D) == 1
    assert act(out=ctypes.c_void_p(A.value + 64 * 2), ldo=127) == 1  # (columns of h's rows, at another stride)
    assert act_int(codes=None) == 1 and act_int(scales=None) == 1 and act_int(ldc=63) == 1 and act_int(scales=ODD) == 1
    assert act_int(codes=A) == 1 and act_int(scales=D) == 1 and act_int(scales=F) == 1
    assert act_grad(da=None) == 1 and act_grad(dh=None) == 1 and act_grad(lddh=127) == 1 and act_grad(ldda=-1) == 1
    assert act_grad(rt2=None) == 1 and act_grad(w=None) == 1 and act_grad(dw=ODD) == 1 and act_grad(dh=P) == 1
    assert act_grad(dw=D) == 1 and act_grad(dw=F) == 1 and act_grad(dh=Q) == 1


def adapt(base=A, ldb=96, x=B, ldx=64, dt=0, r2t=C, t2r=D, off=F, a=G, ae=64 * 16, lda=64, b=P, be=96 * 16, ldbb=16, s=None,
          T=4, n=3, H=64, r=16, N=96, ws=Q, size=1 << 20, out=R, ldo=96):
    return L.moe_adapt(base, ldb, x, ldx, dt, r2t, t2r, off, a, ae, lda, b, be, ldbb, s, T, n, H, r, N, ws, size, out, ldo, None)


def test_adapt_refuses():
    assert adapt(dt=2) == 1 and adapt(T=-1) == 1 and adapt(T=(1 << 22) + 1) == 2 and adapt(n=0) == 1 and adapt(n=1025) == 1
    assert adapt(H=0) == 1 and adapt(r=0) == 1 and adapt(N=0) == 1
    assert adapt(H=72) == 2 and adapt(r=12) == 2 and adapt(r=264) == 2 and adapt(H=1 << 21) == 2 and adapt(N=(1 << 20) + 1) == 2
    for name in ("base", "x", "r2t", "t2r", "off", "a", "b", "ws", "out"):
        assert adapt(**{name: None}) == 1, name
        assert adapt(**{name: ODD}) == 1, name
    assert adapt(s=ODD) == 1 and adapt(ldo=95) == 1 and adapt(ldx=-1) == 1 and adapt(ae=-1) == 1 and adapt(be=1 << 49) == 1
    assert adapt(size=16) == 3 and "workspace" in err()
    assert adapt(out=B) == 1 and adapt(out=C) == 1 and adapt(out=G) == 1 and adapt(out=P) == 1 and adapt(ws=A) == 1
    assert adapt(out=A, ldo=97) == 1 and adapt(out=Q) == 1 and adapt(out=ctypes.c_void_p(A.value + 2)) == 1
    assert L.moe_adapt_workspace_bytes(4, 3, 63, 16) == 0 and L.moe_adapt_workspace_bytes(0, 3, 64, 16) > 0


def test_binding_refuses_without_a_gpu():
    x = torch.zeros(4, 16)
    i = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: moe.route(x, 2), lambda: moe.route_grad(x, x, i), lambda: moe.rms_norm(x), lambda: moe.rms_norm_int8(x),
                 lambda: moe.rms_norm_grad(x, x), lambda: moe.activate(x), lambda: moe.activate_int8(x),
                 lambda: moe.activate_grad(x, x), lambda: moe.adapt(x, x, None, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: moe.route(None, 2), lambda: moe.rms_norm(None), lambda: moe.activate(None), lambda: moe.adapt(None, x, None, x, x)):
        with pytest.raises(TypeError):
            call()


def test_reference_route_by_hand():
    """The 64-bit reference itself."""
    x = np.log([[1.0, 2.0, 4.0, 1.0], [3.0, 3.0, 1.0, 1.0]])
    ids, w = ref.route(x, 2, "softmax", None, 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[2, 1], [0, 1]] and np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]])
    ids, w = ref.route(x, 2, "softmax", None, 1, 1, 1, False, 2.0)
    assert np.allclose(w, [[1.0, 0.5], [0.75, 0.75]])
    # two groups by their two best: 3 against 5 of 8; then only the second group's experts
    ids, _ = ref.route(x[:1], 2, "softmax", None, 2, 1, 2, True, 1.0)
    assert ids.tolist() == [[2, 3]]
    ids, w = ref.route(x[:1], 2, "sigmoid", np.array([1.0, 0, 0, 0]), 1, 1, 1, False, 1.0)  # s: 1/2, 2/3, 4/5, 1/2
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[0.5, 0.8]])
    x = np.full((1, 4), -np.inf)
    x[0, 2] = 0.0
    ids, w = ref.route(x, 2, "softmax", None, 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[2, -1]] and w.tolist() == [[1.0, 0.0]]


def test_reference_norm_by_hand():
    h = np.array([[3.0, 4.0], [1e200, 1e200], [0.0, 0.0]])
    r = ref.inverse_rms(h, 0.0)
    assert np.allclose(r[:2, 0], [12.5 ** -0.5, 1e-200])
    assert np.allclose(ref.inverse_rms(h, 4.0)[2], 0.5)
    # y is homogeneous of degree 0 in h where eps = 0: dx is orthogonal to h
    dx, _, dw, _ = ref.norm_grad(np.array([[1.0, -2.0]]), h[:1], np.array([2.0, 1.0]), 0.0, None)
    assert abs((dx * h[:1]).sum()) < 1e-12 and np.allclose(dw, [3 / 12.5 ** 0.5, -8 / 12.5 ** 0.5])


def test_reference_activation_by_hand():
    assert ref.activation(np.array([[0.0, np.log(3.0), 5.0, 4.0]]), "swiglu").tolist() == [[0.0, np.log(3.0) * 0.75 * 4.0]]
    assert ref.activation(np.array([[-1.0, 3.0]]), "relu2").tolist() == [[0.0, 9.0]]
