"""The operators around the experts refuse what they cannot do before anything is
launched (no GPU needed: no call here passes its checks)."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_fp4_top_amd as moe
from tests import expert_ops_ref as ref

L = moe._lib
A, B, C, D, F, G = (ctypes.c_void_p((i + 1) << 32) for i in range(6))  # far apart, never read
ODD = ctypes.c_void_p((1 << 40) + 1)


def err():
    return L.moe_last_error().decode()


def sort(ids=A, wide=0, T=4, K=2, E=8, ws=B, n=1 << 20, r2r=C, rt2=D, off=F):
    return L.moe_sort_routes(ids, wide, T, K, E, ws, n, r2r, rt2, off, None)


def test_sort_refuses():
    assert sort(E=0) == 1 and sort(E=1025) == 1 and sort(K=0) == 1 and sort(K=65) == 1 and sort(T=-1) == 1
    assert sort(T=1 << 26, K=2) == 2 and "routes" in err()
    assert sort(wide=2) == 1
    assert sort(ids=None) == 1 and sort(r2r=None) == 1 and sort(rt2=None) == 1 and sort(off=None) == 1 and sort(ws=None) == 1
    assert sort(ids=ODD) == 1 and sort(off=ODD) == 1 and sort(ws=ODD) == 1
    assert sort(n=1) == 3 and "workspace" in err()
    assert sort(r2r=A) == 1 and "overlap" in err()
    assert sort(rt2=ctypes.c_void_p(C.value + 4 * 7)) == 1
    assert L.moe_sort_workspace_bytes(4, 2, 0) == 0 and L.moe_sort_workspace_bytes(4, 2, 8) > 0


def test_sort_workspace_never_shrinks():
    last = 0
    for T in (0, 1, 100, 2048, 2049, 5000, 100000, 131072, 131073, 1 << 18, (1 << 18) + 1, 1 << 20, 1 << 22):
        n = L.moe_sort_workspace_bytes(T, 2, 64)
        assert n >= last and n > 0
        last = n
    assert L.moe_sort_workspace_bytes((1 << 22) + 1, 2, 64) == 0


def test_columns_of_one_matrix_do_not_overlap():
    """Buffers are compared row by row where their strides agree: only here the checks
    after it are reached (K too large), else the call is refused as overlapping."""
    def at(out, ld_out=128, H=64):
        return L.moe_dispatch(A, 128, 2, B, C, 4, 1, H, out, ld_out, None), err()
    # rows of 128 floats: x in columns 0..63; out in columns 32..95 overlaps
    assert at(ctypes.c_void_p(A.value + 32 * 4)) == (1, "an output overlaps an input")
    assert at(ctypes.c_void_p(A.value - 32 * 4)) == (1, "an output overlaps an input")
    assert at(ctypes.c_void_p(A.value + 64 * 4), ld_out=127)[0] == 1  # other strides: refused
    assert at(ctypes.c_void_p(A.value + 65 * 4))[0] == 1              # runs over into the next row's x


def rows_call(name, src=A, ld=64, dt=0, r2=B, w=C, other=D, ldo=64, T=4, K=2, H=64, out=F, ld_out=64, dw=G):
    if name == "dispatch":
        return L.moe_dispatch(src, ld, dt, r2, w, T, K, H, out, ld_out, None)
    if name == "combine":
        return L.moe_combine(src, ld, dt, r2, w, T, K, H, out, ld_out, None)
    return getattr(L, "moe_" + name)(src, ld, dt, r2, w, other, ldo, T, K, H, out, ld_out, dw, None)


@pytest.mark.parametrize("name", ["dispatch", "dispatch_grad", "combine", "combine_grad"])
def test_rows_refuse(name):
    def bad(code=1, **kw):
        return rows_call(name, **kw) == code
    assert bad(dt=3) and bad(dt=-1) and bad(T=-1) and bad(K=0) and bad(K=65)
    assert bad(2, H=0) and bad(2, H=(1 << 20) + 1) and bad(2, T=1 << 26)
    assert bad(src=None) and bad(r2=None) and bad(out=None)
    assert bad(ld=-1) and bad(ld_out=63) and bad(2, ld=1 << 33, ld_out=1 << 33)
    assert bad(src=ODD) and bad(out=ODD) and bad(w=ODD) and bad(r2=ODD)
    assert bad(out=A) and bad(out=B) and bad(out=C) and "overlaps" in err()
    if name.endswith("grad"):
        assert bad(w=None) and bad(other=None) and bad(dw=ODD) and bad(dw=A) and bad(dw=F) and bad(out=D) and bad(ldo=-1)


def quant(x=A, ld=64, dt=0, rows=4, cols=64, codes=B, ldc=64, scales=C):
    return L.moe_int_quantize(x, ld, dt, rows, cols, codes, ldc, scales, None)


def test_quantize_refuses():
    assert quant(dt=7) == 1 and quant(rows=-1) == 1 and quant(cols=0) == 2 and quant(cols=(1 << 20) + 1) == 2
    assert quant(x=None) == 1 and quant(codes=None) == 1 and quant(scales=None) == 1
    assert quant(ld=-1) == 1 and quant(ldc=63) == 1
    assert quant(x=ODD) == 1 and quant(scales=ODD) == 1
    assert quant(codes=A) == 1 and quant(scales=A) == 1 and quant(scales=B) == 1


def mm(a=A, lda=64, sa=B, b=C, ldb=64, sb=D, bias=None, M=4, N=8, K=64, dt=0, y=F, ldy=8):
    return L.moe_int_matmul(a, lda, sa, b, ldb, sb, bias, M, N, K, dt, y, ldy, None)


def test_matmul_refuses():
    assert mm(dt=3) == 1 and mm(M=-1) == 1 and mm(N=0) == 1 and mm(K=0) == 1
    assert mm(K=40, lda=48, ldb=48) == 2 and "multiple of 16" in err()
    assert mm(K=131072, lda=131072, ldb=131072) == 2
    assert mm(N=(1 << 20) + 1, ldy=1 << 21) == 2 and mm(M=(1 << 26) + 1) == 2
    assert mm(a=None) == 1 and mm(sa=None) == 1 and mm(b=None) == 1 and mm(sb=None) == 1 and mm(y=None) == 1
    assert mm(lda=48) == 1 and mm(ldb=48) == 1 and mm(ldy=7) == 1
    assert mm(lda=72) == 2 and mm(ldb=72) == 2
    assert mm(a=ctypes.c_void_p(A.value + 8)) == 1 and mm(b=ctypes.c_void_p(C.value + 8)) == 1
    assert mm(y=ODD) == 1 and mm(sa=ODD) == 1 and mm(sb=ODD) == 1 and mm(bias=ODD) == 1
    assert mm(y=A) == 1 and mm(y=C) == 1 and mm(y=B) == 1 and mm(bias=F) == 1 and "overlaps" in err()


def gmm(a=A, lda=64, sa=B, a_rows=4, b=C, ldb=64, be=64 * 8, sb=D, bias=None, off=F, r2r=None, topk=1, M=4, N=8,
        K=64, E=2, dt=0, y=G, ldy=8):
    return L.moe_int_grouped_matmul(a, lda, sa, a_rows, b, ldb, be, sb, bias, off, r2r, topk, M, N, K, E, dt, y,
                                    ldy, None)


def test_grouped_matmul_refuses():
    R = ctypes.c_void_p(1 << 44)
    assert gmm(a_rows=3) == 1 and gmm(a_rows=-1) == 1
    assert gmm(E=0) == 1 and gmm(E=1025) == 1 and gmm(off=None) == 1 and gmm(off=ODD) == 1
    assert gmm(r2r=R, topk=0) == 1 and gmm(r2r=R, topk=65) == 1 and gmm(r2r=R, topk=2, a_rows=3) == 1
    assert gmm(be=-16) == 1 and gmm(be=520) == 2
    assert gmm(y=F) == 1 and gmm(y=R, r2r=R, topk=2, a_rows=2) == 1


def test_binding_refuses_without_a_gpu():
    x = torch.zeros(4, 16)
    for call in (lambda: moe.sort_routes(torch.zeros(4, 2, dtype=torch.int32), 4), lambda: moe.quantize_int8(x),
                 lambda: moe.dispatch(x, None), lambda: moe.combine(x, None),
                 lambda: moe.int8_matmul(x, None, None, None)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        moe.dispatch(None, None)
    with pytest.raises(ValueError):
        moe.RouteOrder(torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                       torch.zeros(3, dtype=torch.int32), 2, 2, 2)


def test_reference_quantizer_ties_and_edges():
    """The 64-bit reference itself: exact ties go to even, -0 and zero rows give 0, a
    row with an infinity or a NaN gives codes 0."""
    c, s = ref.quantize(np.array([[127.0, 0.5, 1.5, -2.5, -0.0], [0, 0, 0, 0, 0], [np.inf, 1, 2, 3, 4],
                                  [np.nan, 1, 2, 3, 4]]))
    assert c[0].tolist() == [127, 0, 2, -2, 0] and s[0] == 1.0
    assert not c[1:].any() and s[1] == 0 and np.isinf(s[2]) and np.isnan(s[3])


def test_reference_sort_by_hand():
    r2r, rt2, off = ref.sort_routes([[1, 0], [5, 1], [-1, 0]], 2)
    assert r2r.tolist() == [1, 5, 0, 3, -1, -1] and rt2.tolist() == [2, 0, -1, 3, -1, 1] and off.tolist() == [0, 2, 4]
