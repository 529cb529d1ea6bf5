"""Values and strides at which the operators in front of, between and beside the experts'
products once went wrong, against plain 64-bit references."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_top_amd as moe  # noqa: E402
from tests import layer_ops_ref as ref  # noqa: E402
from tests.expert_ops_ref import U32, assert_within, f64, stored  # noqa: E402

DT = [torch.bfloat16, torch.float16, torch.float32]
NAME = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
DEV = "cuda"


def rng(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def over(rows, T):
    """The rows over and over, T in all."""
    if isinstance(rows, torch.Tensor):
        return rows.repeat(-(-T // len(rows)), 1)[:T]
    return np.resize(rows, (T,) + rows.shape[1:])


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 33, 2048])  # (from 2048 on the wide kernels)
@pytest.mark.parametrize("r", [8, 16, 64, 104, 256])
@pytest.mark.parametrize("dtype", DT[:2], ids=NAME.get)
def test_adapt_keeps_every_bit_between_the_products(T, r, dtype):
    """Two ranks whose a x differ in the last bits that fp32 holds beside their first, and b of 1
    and -1: what is left is that difference, exactly (each sum here has at most 24 bits)."""
    say("adapt bits", T, r, NAME[dtype])
    H, N, k = 16, 130, 10 if dtype == torch.bfloat16 else 12
    last = 2.0 ** -20 if dtype == torch.bfloat16 else 2.0 ** -23
    for at in ((0, 1), (r - 1, 2), (r // 2, r // 2 - 1)):
        x, a, b = np.zeros((T, H)), np.zeros((1, r, H)), np.zeros((1, N, r))
        x[:, 0] = x[:, 1] = 1.0
        x[:, 2] = last * 2.0 ** k
        size = np.resize([1.0, -2.0, 4.0, -0.5, 16.0], T)  # of a token
        a[0, at[0], :3] = a[0, at[1], :2] = 1.0
        a[0, at[0], 1:3] = a[0, at[1], 1] = 2.0 ** -k  # 1 + 2^-k + last, and 1 + 2^-k
        b[0, :, at[0]], b[0, :, at[1]] = 1.0, -1.0
        order = moe.sort_routes(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1)
        got = moe.adapt(torch.zeros(T, N, dtype=dtype, device=DEV), dev(x * size[:, None], dtype), order, dev(a, dtype),
                        dev(b, dtype), torch.full((1,), 1024.0, device=DEV))
        assert np.array_equal(f64(got), np.repeat((1024.0 * last * size)[:, None], N, axis=1)), at


@pytest.mark.parametrize("T,r,N", [(40, 16, 300), (2048, 16, 300), (2100, 64, 130), (2050, 104, 257), (2048, 256, 128)])
@pytest.mark.parametrize("dtype", DT[:2], ids=NAME.get)
def test_adapt_rows_of_b_that_share_memory(T, r, N, dtype):
    """Row strides of b (and of a) below the rank: one row for all columns, rows that overlap,
    on both sides of where the wide kernels begin."""
    say("adapt strides", T, r, N, NAME[dtype])
    n, H = 2, 64
    g = rng(T + r)
    ids = g.integers(0, n, T)
    base, x = dev(g.standard_normal((T, N)), dtype), dev(g.standard_normal((T, H)), dtype)
    pool = dev(g.standard_normal(2 * (N + 1) * r + r * H) / r ** 0.5, dtype)
    a = dev(g.standard_normal((n, r, H)) / H ** 0.5, dtype)
    order = moe.sort_routes(dev(ids.astype(np.int32)[:, None]), n)
    for ld in (0, 1, 4, 8, r - 1):
        b = pool.as_strided((n, N, r), (N * ld + r, ld, 1))
        for a_t in (a, a[:, :1].expand(n, r, H), pool.as_strided((n, r, H), (r * 8, 8, 1))):
            got = moe.adapt(base, x, order, a_t, b)
            assert torch.equal(got, moe.adapt(base, x, order, a_t.contiguous(), b.contiguous())), ld
            want, bound = ref.adapt(f64(base), f64(x), ids, f64(a_t), f64(b), np.ones(n), 0.0 if dtype == torch.bfloat16 else 2.0 ** -23)
            assert_within(got, want, stored(bound, want, dtype), ld)


@pytest.mark.parametrize("T", [64, 2048])
@pytest.mark.parametrize("dtype", DT[:2], ids=NAME.get)
def test_adapt_one_column(T, dtype):
    """N = 1: b as a transposed view, whose row stride is 1 (no row follows)."""
    n, r, H = 3, 256, 64
    g = rng(T)
    base, x, a = dev(g.standard_normal((T, 1)), dtype), dev(g.standard_normal((T, H)), dtype), dev(g.standard_normal((n, r, H)), dtype)
    w = dev(g.standard_normal((n, r)) / 64, dtype)
    order = moe.sort_routes(dev(g.integers(0, n, (T, 1)).astype(np.int32)), n)
    b = w.view(n, r, 1).transpose(1, 2)
    assert b.stride(1) == 1
    got = moe.adapt(base, x, order, a, b)
    assert torch.equal(got, moe.adapt(base, x, order, a, w.clone().view(n, 1, r))) and not torch.equal(got, base)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
BORDERS = [([0.0, -50.0, -50.0, -40.0], 2), ([0.0, -1e4, -1e4, -40.0], 2), ([1.0, 1.0, 1.0 + 2.0 ** -21, -3.0], 1),
           ([16.0, 16.0, 16.125, -3.0], 1), ([20.0, 0.0, 0.0, 3.0], 2), ([5.0] * 9 + [5.0 + 2.0 ** -20] + [5.0] * 3, 4)]


@pytest.mark.parametrize("E", [16, 64, 128, 256, 300, 1024])
@pytest.mark.parametrize("T", [6, 1100])  # (lanes of a token: 64, and 16 up to 256 experts)
def test_route_equal_choices_across_the_last_place(E, T):
    """Equal experts on both sides of the last place, and a better one behind them that the fast
    comparison cannot tell from them."""
    say("route borders", E, T)
    g = rng(E + T)
    for dtype in DT:
        for row, K in BORDERS:
            x = np.full((min(T, 60), E), -np.inf)
            for t in range(len(x)):  # spread over the experts, in this order; the rest masked or far below
                at = np.arange(len(row)) if t < 2 else np.sort(g.permutation(E)[:len(row)])
                x[t] = -np.inf if t % 2 else -1e5 if dtype != torch.float16 else -6e4
                x[t, at] = row
            xt = over(dev(x, dtype), T)
            for score in ("softmax", "sigmoid"):
                for bias in (None, np.zeros(E), np.full(E, 0.25)):
                    ids, w = moe.route(xt, K, score=score, bias=None if bias is None else dev(bias, torch.float32))
                    want_ids, want = ref.route(f64(xt[:len(x)]), K, score, bias, 1, 1, 1, True, 1.0)
                    want_ids, want = over(want_ids, T), over(want, T)
                    assert np.array_equal(ids.cpu().numpy(), want_ids), (dtype, row, score, bias is None)
                    # (what is not 0 lies less than 104 below the top: 104 half steps of the difference, 50
                    # of the exponent, the sum and a dozen operations)
                    assert_within(w, want, 200 * U32 * want + 2.0 ** -126, (dtype, row, score))


@pytest.mark.parametrize("E,G", [(16, 4), (64, 8), (128, 8), (256, 16), (160, 5), (300, 50), (1024, 16)])
def test_route_few_values(E, G):
    """Rows of a few values only, some next to each other, with and without equal biases and
    groups: every border lies in a run of equal experts."""
    say("route few values", E, G)
    g = rng(E)
    for T in (37, 1100):
        sets = [[0.0, -50.0, -40.0, -1e4], [1.0, 1.0 + 2.0 ** -21, 0.5], [16.0, 16.125, -3.0], [20.0, 0.0, 3.0, -np.inf]]
        x = np.stack([g.choice(sets[t % 4], E) for t in range(min(T, 60))])
        xt = over(dev(x, torch.float32), T)
        for score in ("softmax", "sigmoid"):
            for bias in (None, np.zeros(E), np.full(E, 0.25), g.choice([0.0, 0.25], E)):
                for groups, best in ((1, 1), (G, 1), (G, 2)):
                    if best == 2 and bias is not None and len(set(bias)) > 1:
                        continue  # (sums of the same scores and biases in another order: equal but for roundings)
                    K = int(g.integers(1, 9))
                    top = min(3, groups)
                    ids, _ = moe.route(xt, K, score=score, bias=None if bias is None else dev(bias, torch.float32), groups=groups,
                                       top_groups=top, group_top=best)
                    want_ids, _ = ref.route(f64(xt[:len(x)]), K, score, bias, groups, top, best, True, 1.0)
                    assert np.array_equal(ids.cpu().numpy(), over(want_ids, T)), (T, score, bias is None, groups, best, K)


@pytest.mark.parametrize("E,G", [(8, 4), (64, 8), (128, 8), (256, 16), (160, 5), (300, 50), (1024, 16)])
@pytest.mark.parametrize("T", [5, 1100])
def test_route_groups_of_lowest_choices(E, G, T):
    """Groups whose best two choices count as the lowest value, or are biases near it: their sum
    lies below fp32's range, and yet above a group with nothing to choose."""
    say("route lowest groups", E, G, T)
    S = E // G
    bias = np.zeros(E)
    bias[-S:] = -3e38
    x = np.full((T, E), -np.inf)
    x[0::2, S:2 * S] = np.nan      # groups 0 and 2 on: nothing to choose
    x[1::2, -S:] = 1.0             # the last group alone, by its bias
    for score in ("softmax", "sigmoid"):
        ids, w = moe.route(dev(x, torch.float32), 2, score=score, bias=dev(bias, torch.float32), groups=G, top_groups=1, group_top=2)
        want = np.where((np.arange(T) % 2 == 0)[:, None], [[S, S + 1]], [[E - S, E - S + 1]])
        assert np.array_equal(ids.cpu().numpy(), want), score
        w = f64(w)
        assert np.isnan(w[0::2]).all() and np.array_equal(w[1::2], np.full(w[1::2].shape, 0.5))


# ---------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("I", [7, 300, 2048, 5000])
def test_activate_codes_of_subnormal_gates(I):
    """Gates below fp32's normal range (silu there is half of a few steps) times large ups: the
    codes are those of the product in 64 bits."""
    say("subnormal gates", I)
    g = rng(I)
    for dtype in (torch.float32, torch.bfloat16):
        step = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
        for rows in (6, 4100 if I == 300 else 6):
            h = np.concatenate([g.integers(-9, 10, (rows, I)) * step, g.standard_normal((rows, I)) * 2.0 ** 100], axis=1)
            h[1, I:] *= 2.0 ** 27 / np.abs(h[1, I:]).max() * 2.0 ** 100
            h[2, I // 2] = 2.0 ** -100  # among others
            h[3, :I] = step             # 0 after one rounding of silu
            h[4, :I] = g.standard_normal(I) * 2.0 ** -128
            h[5, I:] = 1.0              # too small for a scale
            ht = dev(h, dtype)
            codes, scales = moe.activate_int8(ht)
            codes64, s64 = ref.quantize(ref.activation(f64(ht), "swiglu"))
            assert np.array_equal(f64(scales), s64), dtype
            assert np.array_equal(codes.cpu().numpy(), codes64), dtype


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H", [33, 2000, 5000])
def test_norm_small_values_beside_large_ones(H):
    """Rows whose squares leave fp32's range keep the bits of their small values."""
    say("norm small beside large", H)
    g = rng(H)
    h = g.standard_normal((6, H)) * 2.0 ** np.array([-45, -48, -40, -30, 0, -50])[:, None]
    h[:, H // 3] = [2.0 ** 70, 2.0 ** 65, 2.0 ** 100, 2.0 ** 126, 2.0 ** 90, -2.0 ** 75]
    w = g.standard_normal(H)
    ht, wt = dev(h, torch.float32), dev(w, torch.float32)
    h64, w64 = f64(ht), f64(wt)
    want = h64 * ref.inverse_rms(h64, 1e-6) * w64
    # r is off by 50 half steps, and there are three products; two of them may be subnormal
    y, _ = moe.rms_norm(ht, wt)
    assert_within(y, want, 55 * U32 * np.abs(want) + 2.0 ** -150 * (1 + np.abs(w64)), "y")
    small = dev(np.full(H, 2.0 ** -120), torch.float32)
    codes, scales, _ = moe.rms_norm_int8(ht, small)
    codes64, s64 = ref.quantize(h64 * 2.0 ** -120)
    want_s = s64 * ref.inverse_rms(h64, 1e-6)[:, 0]
    assert np.array_equal(codes.cpu().numpy(), codes64)
    assert_within(scales, want_s, 55 * U32 * want_s + 2.0 ** -150, "scales")
    dy = dev(g.standard_normal((6, H)), torch.float32)
    dx, dw = moe.rms_norm_grad(dy, ht, wt)
    want, bound, want_w, bound_w = ref.norm_grad(f64(dy), h64, w64, 1e-6, None)
    assert_within(dx, want, bound + U32 * np.abs(want) + 2.0 ** -148, "dx")
    # (h / rms below 2^-126 is off by 2^-150, and so is each of six additions there)
    assert_within(dw, want_w, bound_w + 2.0 ** -150 * (np.abs(f64(dy)).sum(axis=0) + 6), "dweight")
