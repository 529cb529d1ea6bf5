"""When buffers of the row operators share bytes, decided on the host (no GPU needed: no
call here passes its checks).

combine_grad compares its inputs with both outputs first ("an output overlaps an input")
and then the outputs with each other ("the outputs overlap"). Here dweights always lies
inside drows, so the second message says that every input was found to lie apart."""
import ctypes

import pytest

import block_scaled_fp4_top_amd as moe

BASE = 1 << 40
H, T = 64, 4  # fp32 rows of 256 bytes
APART, SHARED = b"the outputs overlap", b"an output overlaps an input"


def at(offset):
    return ctypes.c_void_p(BASE + offset)


FAR = {"token": 1 << 32, "rows": 2 << 32, "route": 3 << 32, "w": 4 << 32}


def message(out, ld_out=128, token=FAR["token"], ld_token=64, rows=FAR["rows"], ld_rows=64, route=FAR["route"], w=FAR["w"], T=T):
    rc = moe._lib.moe_combine_grad(at(token), ld_token, 2, at(route), at(w), at(rows), ld_rows, T, 1, H, at(out), ld_out,
                                   at(out), None)
    assert rc == 1
    return moe._lib.moe_last_error()


def test_columns_apart():
    """Rows of 512 bytes shared by an input and an output, 256 bytes each, on either side,
    the output beginning in an earlier or in a later row."""
    for name in ("token", "rows"):
        for shift in (0, 512, -512, 3 * 512, -3 * 512):
            assert message(256 + shift, **{name: 0, "ld_" + name: 128}) == APART
            assert message(shift, **{name: 256, "ld_" + name: 128}) == APART


def test_columns_that_share_bytes():
    for name in ("token", "rows"):
        for shift in (0, 4, 252, 260, 508, 512, -4, -252, -260, -508, -512):
            # (512 and its multiples: the same columns; 252 .. 260: into the next piece on one side)
            want = APART if shift % 512 == 256 else SHARED
            assert message(shift, **{name: 0, "ld_" + name: 128}) == want, shift


def test_one_row_in_the_gap():
    """16 bytes (the map, the weights) between an output's columns, and next to them."""
    for name in ("route", "w"):
        for offset in (256, 300, 496, 512 + 256, 3 * 512 - 16):
            assert message(0, **{name: offset}) == APART, offset
        for offset in (0, 240, 252, 500, 512, 3 * 512):
            assert message(0, **{name: offset}) == SHARED, offset
        # behind the last row's columns, before the first one's
        assert message(0, **{name: 3 * 512 + 256}) == APART and message(0, **{name: -16}) == APART
        assert message(0, **{name: -12}) == SHARED


def test_one_token():
    """One row against one row: no stride decides."""
    for offset, want in ((0, SHARED), (252, SHARED), (256, APART), (-256, APART), (-252, SHARED)):
        assert message(0, ld_out=64, token=offset, T=1) == want, offset


@pytest.mark.parametrize("ld", [0, 127, 64, 63, 256])
def test_other_strides_are_taken_to_share(ld):
    """Rows of another stride whose extents cross, one row for all tokens among them."""
    assert message(256, token=0 if ld else 512, ld_token=ld) == SHARED


@pytest.mark.parametrize("ld", [0, 127, 256])
def test_other_strides_behind(ld):
    assert message(0, token=3 * 512 + 256, ld_token=ld) == APART
    assert message(3 * ld * 4 + 256, token=0, ld_token=ld) == APART
