"""The binding of the operators around the experts refuses sizes that its int32
arguments cannot hold, instead of taking them modulo 2^32 (no GPU needed; on one, the
public calls)."""
import ctypes

import pytest
import torch

import block_scaled_fp4_top_amd as moe

FAR = (1 << 32) + 4  # 4 modulo 2^32
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")


@pytest.mark.parametrize("shape", [(FAR, 1), (1, FAR), (1 << 31, 1), (1, 1 << 31)])
def test_matrices(shape):
    t = torch.empty(1, 1).expand(shape)
    with pytest.raises(ValueError, match="32 bits"):
        moe._matrix(t, "x", torch.float32, -1)


def test_orders():
    empty = torch.empty(0, dtype=torch.int32)
    for T, K, E in ((FAR, 1, 8), (1, FAR, 8), (0, FAR, 8), (4, 2, FAR), (1 << 20, 1 << 12, 8)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.RouteOrder(empty, empty, empty, T, K, E)


def test_experts_far_apart():
    """A stride whose product with the experts wraps 64 bits hid an output that overlaps
    the weights, and every other check behind it."""
    a, sa, b, sb, off, y = (ctypes.c_void_p((i + 1) << 32) for i in range(6))  # far apart, never read
    def call(E, stride, y=y):
        return moe._lib.moe_int_grouped_matmul(a, 64, sa, 4, b, 64, stride, sb, None, off, None, 1, 4, 8, 64, E, 0, y, 8, None)
    for stride in (1 << 62, (1 << 48) + 16):
        assert call(3, stride) == 2 and b"apart" in moe._lib.moe_last_error()
    assert call(3, 1 << 48, y=b) == 1 and call(1, 1 << 62, y=b) == 1 and b"overlaps" in moe._lib.moe_last_error()


def test_layer_calls(monkeypatch):
    """finalize and quantize, past the checks of the device."""
    monkeypatch.setattr(moe, "_need", lambda *a, **k: None)
    with pytest.raises(ValueError, match="32 bits"):
        moe.quantize(torch.empty(1, 1).expand(1, (1 << 32) + 16), "nvfp4_tensor")
    with pytest.raises(ValueError, match="32 bits"):
        moe.finalize(torch.empty(1, 1).expand(FAR, 8), None, None, FAR, 1)


@pytest.mark.gpu
@needs_gpu
def test_public_calls():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    order = moe.sort_routes(ids, 8)
    c, s = torch.ones(4, 16, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    for call in (lambda: moe.sort_routes(ids, FAR), lambda: moe.sort_routes(ids, 8 - (1 << 32)),
                 lambda: moe.quantize_int8(one.expand(FAR, 1)), lambda: moe.quantize_int8(one.expand(1, FAR)),
                 lambda: moe.dispatch(one.expand(4, FAR), order), lambda: moe.combine(one.expand(8, FAR), order),
                 lambda: moe.int8_matmul(c, s, c[:1].expand(FAR, 16), s),
                 lambda: moe.int8_grouped_matmul(c, s, c[:1].expand(8, FAR, 16), s, order, gather=True)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
