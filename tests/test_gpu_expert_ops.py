"""The operators around the experts on the GPU against plain 64-bit references:
routes sorted by expert, dispatch, combine, their gradients, the 8-bit integer
quantizer and products, and runs of them together."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_top_amd as moe  # noqa: E402
from tests import expert_ops_ref as ref  # noqa: E402
from tests.expert_ops_ref import HALF, U32, assert_within, f64, stored  # noqa: E402

DT = [torch.bfloat16, torch.float16, torch.float32]
NAME = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
DEV = "cuda"


def rng(seed):
    return np.random.default_rng(seed)



def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def order_of(ids, E):
    o = moe.sort_routes(dev(ids.astype(np.int32)), E)
    return o, [v.cpu().numpy() for v in o.tensors()]


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------
SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 256), (3, 5, 2), (64, 8, 256), (63, 1, 64), (65, 1, 65), (513, 8, 7),
         (512, 8, 256), (513, 8, 256), (1024, 4, 1), (4097, 1, 300), (2048, 8, 1024), (5000, 3, 1024),
         (16384, 8, 256), (40000, 8, 1023), (100000, 5, 33), (70000, 16, 5), (300000, 8, 200)]


@pytest.mark.parametrize("T,K,E", SORTS)
@pytest.mark.parametrize("wide", [False, True], ids=["int32", "int64"])
def test_sort_routes(T, K, E, wide):
    say("sort", T, K, E, wide)
    g = rng(T * 31 + K * 7 + E)
    for kind in ("even", "dropped", "skewed"):
        if kind == "even":
            ids = g.integers(0, E, (T, K))
        elif kind == "dropped":  # experts of other GPUs on both sides
            ids = g.integers(-E, 2 * E, (T, K))
        else:  # nearly all on one expert, also twice in one token
            ids = np.where(g.random((T, K)) < 0.9, E // 2, g.integers(0, E, (T, K)))
        if wide and kind == "dropped" and T:
            ids[0, 0] = 1 << 40
            ids[-1, -1] = -(1 << 40) + 1
        o = moe.sort_routes(dev(ids.astype(np.int64 if wide else np.int32)), E)
        for got, want, name in zip(o.tensors(), ref.sort_routes(ids, E), ("row_to_route", "route_to_row", "offsets")):
            assert np.array_equal(got.cpu().numpy(), want), (kind, name)


def test_sort_all_dropped():
    ids = np.full((700, 8), -1)
    o, (r2r, rt2, off) = order_of(ids, 16)
    assert (r2r == -1).all() and (rt2 == -1).all() and not off.any()


# ---------------------------------------------------------------------------
# dispatch, combine and their gradients
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 1, 1), (1, 8, 64, 256), (2, 3, 7, 4), (5, 2, 8, 3), (37, 6, 129, 16), (64, 8, 256, 64), (9, 64, 40, 80),
          (33, 9, 1000, 12), (3, 17, 2049, 20), (17, 2, 4100, 8), (300, 8, 520, 32), (6, 4, 9001, 5)]


def routes(seed, T, K, E, drop):
    """K expert ids for each token (repeats where K > E), some out of range; the first
    token loses all its routes when any are dropped."""
    g = rng(seed)
    ids = g.integers(0, E, (T, K))
    if drop:
        ids = np.where(g.random((T, K)) < 0.3, E + 5, ids)
        ids[0] = -1
    return ids


def strided(a, pad, dtype):
    """The matrix as a view with `pad` more elements between its rows (NaN there)."""
    full = np.full((a.shape[0], a.shape[1] + pad), np.nan)
    full[:, :a.shape[1]] = a
    return dev(full, dtype)[:, :a.shape[1]]


@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
@pytest.mark.parametrize("T,K,H,E", SHAPES)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_dispatch_and_combine(T, K, H, E, dtype, pad):
    say("rows", T, K, H, E, NAME[dtype], pad)
    R = T * K
    for drop in (False, True):
        ids = routes(T + K + H, T, K, E, drop)
        o, (r2r, rt2, off) = order_of(ids, E)
        kept = off[-1]
        route = r2r[:kept]
        g = rng(H + drop)
        w = g.standard_normal((T, K)).astype(np.float32)
        tok = strided(g.standard_normal((T, H)), pad, dtype)
        rows_np = g.standard_normal((R, H))
        rows_np[kept:] = np.nan  # behind the last row: never read
        rows = strided(rows_np, pad, dtype)
        x64, r64, w64 = f64(tok), f64(rows), w.astype(np.float64)
        wd = dev(w)
        for weights in (None, wd):
            wv = np.ones(kept) if weights is None else w64.reshape(-1)[route]
            # to the experts' rows
            want = np.full((R, H), 7.0)
            want[:kept] = x64[route // K] * wv[:, None]
            bound = np.where(np.arange(R)[:, None] < kept, 0.0 if weights is None else stored(U32 * np.abs(want), want, dtype), 0.0)
            out = torch.full((R, H + pad), 7.0, dtype=dtype, device=DEV)
            got = moe.dispatch(tok, o, weights, out=out[:, :H])
            assert_within(got, want, bound, "dispatch")
            assert (out[:, H:] == 7).all(), "dispatch wrote between the rows"
            out = torch.full((R, H), 7.0, dtype=dtype, device=DEV)
            got, dw = moe.combine_grad(tok, o, rows if weights is not None else None, weights, out=out)
            assert_within(got, want, bound, "combine_grad rows")
            # back
            terms = np.zeros((T, K, H))
            terms.reshape(R, H)[route] = r64[:kept] * wv[:, None]
            want = terms.sum(1)
            bound = stored((K + 1) * U32 * np.abs(terms).sum(1), want, dtype)
            got = moe.combine(rows, o, weights)
            assert_within(got, want, bound, "combine")
            got, dw2 = moe.dispatch_grad(rows, o, tok if weights is not None else None, weights)
            assert_within(got, want, bound, "dispatch_grad tokens")
            if weights is None:
                assert dw is None and dw2 is None
                continue
            want, mag = np.zeros(R), np.zeros(R)
            prod = r64[:kept] * x64[route // K]
            want[route], mag[route] = prod.sum(1), np.abs(prod).sum(1)
            bound = ((H + 1) * U32 * mag).reshape(T, K)
            assert_within(dw, want.reshape(T, K), bound, "combine_grad weights")
            assert_within(dw2, want.reshape(T, K), bound, "dispatch_grad weights")


@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
@pytest.mark.parametrize("T,K,H,E", [(4200, 4, 1032, 9), (2100, 8, 2056, 20), (2100, 10, 2056, 20), (5000, 3, 1544, 6)])
def test_large_rows(T, K, H, E, dtype):
    """Outputs of 32 MB and more (stored past the caches), rows of a wave and of a block
    per token, against 64 bits on the GPU; some routes dropped."""
    say("large rows", T, K, H, E, NAME[dtype])
    g = torch.Generator(device=DEV).manual_seed(K)
    ids = torch.randint(0, E + 2, (T, K), device=DEV, generator=g)
    o = moe.sort_routes(ids, E)
    kept = int(o.offsets[-1])
    tok, rows = (torch.randn(n, H, device=DEV, generator=g).to(dtype) for n in (T, T * K))
    rows[kept:] = float("nan")
    w = torch.randn(T, K, device=DEV, generator=g)
    route = o.row_to_route[:kept].long()
    token, wr = route // K, w.double().view(-1)[route][:, None]
    out = torch.full((T * K, H), 7.0, dtype=dtype, device=DEV)
    moe.dispatch(tok, o, out=out)
    assert torch.equal(out[:kept], tok[token]) and (out[kept:] == 7).all()
    want = tok.double()[token] * wr
    def within(got, want, mag, n):
        b = n * U32 * mag
        return bool(((got.double() - want).abs() <= b + (want.abs() + b) * HALF[dtype] + ref.TINY[dtype]).all())
    drows, dw = moe.combine_grad(tok, o, rows, w, out=out)
    assert within(drows[:kept], want, want.abs(), 1) and (out[kept:] == 7).all()
    prod = rows[:kept].double() * tok.double()[token]
    dots, dmag = (torch.zeros(T * K, dtype=torch.float64, device=DEV) for _ in range(2))
    dots[route], dmag[route] = prod.sum(1), prod.abs().sum(1)
    bound = (H + 1) * U32 * dmag.view(T, K)
    assert bool(((dw.double() - dots.view(T, K)).abs() <= bound).all())
    term = rows[:kept].double() * wr
    y, mag = (torch.zeros(T, H, dtype=torch.float64, device=DEV).index_add_(0, token, v) for v in (term, term.abs()))
    assert within(moe.combine(rows, o, w), y, mag, K + 1)
    dx, dw = moe.dispatch_grad(rows, o, tok, w)
    assert within(dx, y, mag, K + 1) and bool(((dw.double() - dots.view(T, K)).abs() <= bound).all())


def test_offsets_beyond_32_bits():
    """More than 2^31 elements and 4 GiB in every matrix: the last rows arrive right."""
    T, K, H, E = 36000, 8, 8192, 5
    R = T * K
    g = torch.Generator(device=DEV).manual_seed(1)
    o = moe.sort_routes(torch.randint(0, E, (T, K), device=DEV, generator=g), E)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    rows = moe.dispatch(x, o)
    token = o.row_to_route.long() // K
    for at in (slice(0, 64), slice(R // 2, R // 2 + 64), slice(R - 64, R)):
        assert torch.equal(rows[at], x[token[at]])
    w = torch.rand(T, K, device=DEV, generator=g)
    y = moe.combine(rows, o, w)
    at = slice(T - 64, T)
    want = x[at].double() * w[at].double().sum(1, keepdim=True)
    mag = x[at].double().abs() * w[at].double().sum(1, keepdim=True)
    assert bool(((y[at].double() - want).abs() <= (K + 1) * U32 * mag + (want.abs() + 1e-6 * mag) * HALF[x.dtype] + 1e-38).all())
    c, s = moe.quantize_int8(rows)
    want_c, want_s = ref.quantize(f64(rows[R - 8:]))
    assert np.array_equal(c[R - 8:].cpu().numpy(), want_c) and np.array_equal(f64(s[R - 8:]), want_s)
    del rows
    b, sb = torch.randint(-127, 128, (48, H), dtype=torch.int8, device=DEV, generator=g), torch.rand(48, device=DEV, generator=g)
    y = moe.int8_matmul(c[-280000:], s[-280000:], b, sb, out_dtype=torch.float32)
    want, bound = ref.matmul(c[-16:].cpu().numpy(), f64(s[-16:]), b.cpu().numpy(), f64(sb))
    assert_within(y[-16:], want, stored(bound, want, torch.float32), "far rows of a")
    del y
    b, sb = torch.randint(-127, 128, (H, 32), dtype=torch.int8, device=DEV, generator=g), torch.rand(H, device=DEV, generator=g)
    a = c[:, :32].contiguous()
    y = moe.int8_matmul(a, s, b, sb)
    want, bound = ref.matmul(a[-16:].cpu().numpy(), f64(s[-16:]), b.cpu().numpy(), f64(sb))
    assert_within(y[-16:], want, stored(bound, want, torch.bfloat16), "far rows of y")
    with pytest.raises(moe.MoeError) as e:  # 560000 x 8192 gathered: 4.6 GB
        big = torch.empty(560000, H, dtype=torch.int8, device=DEV)
        oo = moe.sort_routes(torch.zeros(560000, 1, dtype=torch.int32, device=DEV), 1)
        moe.int8_grouped_matmul(big, torch.ones(560000, device=DEV), b.new_zeros(1, 16, H), torch.ones(1, 16, device=DEV),
                                oo, gather=True)
    assert e.value.code == 2


def test_most_routes():
    """2^23 routes, a third of them on one expert, some dropped."""
    ids = rng(1).integers(-1, 7, (1 << 20, 8))
    ids[: 1 << 18] = 3
    o = moe.sort_routes(dev(ids.astype(np.int32)), 6)
    for got, want in zip(o.tensors(), ref.sort_routes(ids, 6)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
def test_columns_that_begin_anywhere(dtype):
    """Matrices whose first element and whose rows are aligned to their element only."""
    T, K, H, E = 33, 3, 600, 4
    o, (r2r, rt2, off) = order_of(routes(6, T, K, E, False), E)
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(T, H + 5, device=DEV, generator=g).to(dtype)[:, 1:H + 1]
    rows = torch.full((T * K, H + 3), 2.0, device=DEV, dtype=dtype)
    moe.dispatch(x, o, out=rows[:, 3:])
    want = x[torch.as_tensor(r2r // K, device=DEV)]
    assert torch.equal(rows[:, 3:], want) and (rows[:, :3] == 2).all()
    w = torch.rand(T, K, device=DEV, generator=g)
    y, dw = moe.dispatch_grad(rows[:, 3:], o, x, w)
    z, dw2 = moe.dispatch_grad(want.contiguous(), o, x.contiguous(), w)
    assert torch.equal(y, z) and torch.equal(dw, dw2) and torch.equal(y, moe.combine(want.contiguous(), o, w))
    out = torch.zeros(T, H + 7, dtype=torch.int8, device=DEV)
    c, s = moe.quantize_int8(x, out=out[:, 7:])
    c2, s2 = moe.quantize_int8(x.contiguous())
    assert torch.equal(c, c2) and torch.equal(s, s2) and not out[:, :7].any()


def test_one_matrix_for_all_experts():
    T, K, E, N, D = 30, 2, 6, 72, 64
    o, _ = order_of(routes(6, T, K, E, False), E)
    g = rng(2)
    a, b, sa, sb = dev(codes(g, T, D)), dev(codes(g, N, D)), dev(scale(g, T)), dev(scale(g, N))
    y = moe.int8_grouped_matmul(a, sa, b.expand(E, N, D), sb.expand(E, N).contiguous(), o, gather=True)
    z = moe.dispatch(moe.int8_matmul(a, sa, b, sb), o)
    assert torch.equal(y, z)


def test_output_in_other_columns_of_the_input():
    T, K, H, E = 6, 1, 40, 3
    o, (r2r, rt2, off) = order_of(routes(2, T, K, E, False), E)
    both = torch.randn(T, 2 * H, device=DEV)
    x = both[:, :H].clone()
    got = moe.dispatch(both[:, :H], o, out=both[:, H:])
    assert torch.equal(got, x[torch.as_tensor(r2r, device=DEV).long()]) and torch.equal(both[:, :H], x)


def test_rows_without_tokens():
    o = moe.sort_routes(torch.empty(0, 4, dtype=torch.int32, device=DEV), 8)
    x = torch.empty(0, 16, device=DEV)
    w = torch.empty(0, 4, device=DEV)
    assert moe.dispatch(x, o, w).shape == (0, 16) and moe.combine(x, o, w).shape == (0, 16)
    assert moe.combine_grad(x, o, x, w)[1].shape == (0, 4) and not o.offsets.any()
    c, s = moe.quantize_int8(x)
    assert c.shape == (0, 16) and s.shape == (0,)
    b, sb = torch.ones(8, 16, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    assert moe.int8_matmul(c, s, b, sb).shape == (0, 8)


def test_broadcast_token_and_nan():
    """One row for all tokens (stride 0), and values that are not finite: they arrive
    where they belong and nowhere else, a NaN of any payload as a NaN."""
    T, K, H, E = 5, 2, 72, 4
    o, (r2r, rt2, off) = order_of(routes(3, T, K, E, False), E)
    for dtype in DT:
        x = torch.randn(1, H, device=DEV, dtype=dtype)
        got = moe.dispatch(x.expand(T, H), o)
        assert torch.equal(got, x.expand(T * K, H))
        rows = torch.randn(T * K, H, device=DEV, dtype=dtype)
        rows[rt2[2 * K], 7] = float("nan")
        rows[rt2[4 * K], 9] = float("inf")
        y = moe.combine(rows, o, torch.ones(T, K, device=DEV))
        bad = ~torch.isfinite(y)
        assert bad.sum() == 2 and torch.isnan(y[2, 7]) and torch.isinf(y[4, 9])
    x = torch.full((T, H), -1, dtype=torch.int16, device=DEV).view(torch.bfloat16)  # NaN, all bits set
    assert torch.isnan(moe.dispatch(x, o, torch.ones(T, K, device=DEV))).all()


@pytest.mark.parametrize("T,K,H,E", [(5, 3, 70, 4), (40, 8, 264, 16)])
def test_gradients_against_differences(T, K, H, E):
    """combine and dispatch are linear in rows and in weights, so a difference over a
    step of 1 is the derivative; fp32, each value within its rounding bound."""
    o, (r2r, rt2, off) = order_of(routes(11, T, K, E, True), E)
    g = torch.Generator(device=DEV).manual_seed(5)
    kept = int(off[-1])
    rows, drow = (torch.randn(T * K, H, device=DEV, generator=g) for _ in range(2))
    rows[kept:] = 0
    drow[kept:] = 0
    tok, w, dw_dir = torch.randn(T, H, device=DEV, generator=g), torch.randn(T, K, device=DEV, generator=g), \
        torch.randn(T, K, device=DEV, generator=g)

    def check(lo, hi, seed, grad, direction, what):
        diff = ((f64(hi) - f64(lo)) * f64(seed)).sum()
        want = (f64(grad) * f64(direction)).sum()
        # every value of lo and hi is within (K + 2) roundings of sums of at most
        # K terms of magnitude |w||rows| (fp32 steps w + 1, rows + 1 count one more)
        mag = ((f64(hi).__abs__() + f64(lo).__abs__() + 4 * K * 16) * np.abs(f64(seed))).sum()
        grad_mag = (np.abs(f64(grad)) * np.abs(f64(direction))).sum() + H * 16 * np.abs(f64(direction)).sum()
        bound = (K + 4) * U32 * mag + (H + 4) * U32 * grad_mag
        assert abs(diff - want) <= bound, (what, diff, want, bound)

    dy = torch.randn(T, H, device=DEV, generator=g)
    drows = torch.zeros(T * K, H, device=DEV)
    _, dw = moe.combine_grad(dy, o, rows, w, out=drows)
    check(moe.combine(rows, o, w), moe.combine(rows + drow, o, w), dy, drows, drow, "combine rows")
    check(moe.combine(rows, o, w), moe.combine(rows, o, w + dw_dir), dy, dw, dw_dir, "combine weights")
    gx, gw = moe.dispatch_grad(drow, o, tok, w)
    z = lambda: torch.zeros(T * K, H, device=DEV)  # noqa: E731
    dtok = torch.randn(T, H, device=DEV, generator=g)
    check(moe.dispatch(tok, o, w, out=z()), moe.dispatch(tok + dtok, o, w, out=z()), drow, gx, dtok, "dispatch tokens")
    check(moe.dispatch(tok, o, w, out=z()), moe.dispatch(tok, o, w + dw_dir, out=z()), drow, gw, dw_dir, "dispatch weights")


def test_damaged_map_stays_in_range():
    """Entries of the maps that name no row, route or group count as dropped."""
    T, K, H, E = 6, 2, 48, 3
    o, _ = order_of(routes(2, T, K, E, False), E)
    rt2 = o.route_to_row.clone()
    rt2[3], rt2[5] = T * K, -7
    bad = moe.RouteOrder(o.row_to_route, rt2, o.offsets, T, K, E)
    rows = torch.randn(T * K, H, device=DEV)
    want = torch.zeros(T, H, device=DEV)
    for r in range(T * K):
        if r not in (3, 5):
            want[r // K] += rows[rt2[r]]
    assert torch.allclose(moe.combine(rows, bad), want, rtol=1e-6, atol=1e-6)
    off = torch.tensor([-5, 4, 2, 1 << 30], dtype=torch.int32, device=DEV)
    r2r = o.row_to_route.clone()
    r2r[0] = 1 << 30
    bad = moe.RouteOrder(r2r, rt2, off, T, K, E)
    a = torch.ones(T, 16, dtype=torch.int8, device=DEV)
    b = torch.ones(E, 8, 16, dtype=torch.int8, device=DEV)
    out = torch.full((T * K, 8), -1.0, device=DEV)
    moe.int8_grouped_matmul(a, torch.ones(T, device=DEV), b, torch.ones(E, 8, device=DEV), bad, gather=True, out=out)
    assert (out[0] == -1).all() and (out[1:] == 16).all()


@pytest.mark.parametrize("N", [8, 4000])  # narrow and wide tiles
def test_routes_that_name_no_token(N):
    T, K, E = 60, 2, 20
    o, _ = order_of(routes(5, T, K, E, False), E)
    r2r = o.row_to_route.clone()
    r2r[3], r2r[50], r2r[-1] = -1, T * K, -(1 << 31)
    bad = moe.RouteOrder(r2r, o.route_to_row, o.offsets, T, K, E)
    a, b = torch.ones(T, 32, dtype=torch.int8, device=DEV), torch.ones(E, N, 32, dtype=torch.int8, device=DEV)
    out = torch.full((T * K, N), -1.0, device=DEV)
    moe.int8_grouped_matmul(a, torch.ones(T, device=DEV), b, torch.ones(E, N, device=DEV), bad, gather=True, out=out)
    want = torch.full((T * K, N), 32.0, device=DEV)
    want[[3, 50, T * K - 1]] = -1
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# quantizer
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (2, 64), (5, 129), (70, 512), (33, 2048), (9, 2056), (4, 7168),
                                 (3, 8200), (2, 20001), (1, 70000),
                                 (4100, 1023), (4097, 2000), (4096, 513)])
def test_quantize_int8(M, N, dtype):
    say("quantize", M, N, NAME[dtype])
    g = rng(M * 7 + N)
    x = g.standard_normal((M, N)) * np.exp(g.standard_normal((M, 1)) * 3)
    if M > 2:
        x[0] = 0.0
        x[1] = np.round(x[1] * 8) / 2  # many exact halves once the largest is 127
        x[1, 0] = 127.0
        x[1] = np.clip(x[1], -127, 127)
    if M > 8:
        x[2, N // 2] = np.inf
        x[3, N - 1] = np.nan
        x[4] *= 1e-7 if dtype == torch.float16 else 1e-38
        x[5] = -0.0
        x[6] = 6e-8 if dtype == torch.float16 else 1e-40
        x[7] *= 1e4 if dtype == torch.float16 else 1e37
    for pad in (0, 5):
        t = strided(x, pad, dtype)
        out = torch.full((M, N + pad), 99, dtype=torch.int8, device=DEV)
        codes, scales = moe.quantize_int8(t, out=out[:, :N])
        want_c, want_s = ref.quantize(f64(t))
        assert np.array_equal(f64(scales), want_s, equal_nan=True)
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert (out[:, N:] == 99).all()


def test_quantize_next_to_ties():
    """fp32 quotients next to a half: x one step around (n + 1/2) s for scales s with
    many bits."""
    g = rng(8)
    x = np.zeros((64, 3 * 126 + 1), np.float32)
    for m in range(64):
        top = np.float32(np.exp(g.standard_normal()))
        s = np.float32(np.float64(top) / 127)
        h = ((np.arange(126) + 0.5) * np.float64(s)).astype(np.float32)
        x[m] = np.concatenate([[top], h, np.nextafter(h, np.float32(9e9)), np.nextafter(h, np.float32(0))])
        x[m, 1::2] *= -1
    codes, scales = moe.quantize_int8(dev(x))
    want_c, want_s = ref.quantize(x.astype(np.float64))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(f64(scales), want_s)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def codes(g, *shape):
    return g.integers(-128, 128, shape).astype(np.int8)


def scale(g, *shape):
    return np.exp(g.standard_normal(shape) * 0.5).astype(np.float32) * np.float32(0.01)


def pad_codes(a, pad):
    """The codes as a view with `pad` more bytes between the rows (of value 77)."""
    full = np.full((*a.shape[:-1], a.shape[-1] + pad), 77, np.int8)
    full[..., :a.shape[-1]] = a
    return dev(full)[..., :a.shape[-1]]


MATMULS = [(1, 1, 16), (1, 17, 32), (1, 4096, 512), (2, 16, 48), (3, 300, 64), (15, 64, 80), (16, 256, 128), (17, 130, 144),
           (31, 33, 2064), (33, 512, 256), (64, 100, 1008), (65, 257, 272), (128, 128, 128), (129, 255, 512), (200, 640, 2048),
           (257, 513, 400), (300, 1024, 1024), (513, 777, 176), (1000, 520, 640), (1025, 1100, 336),
           # every tile shape on a chip of 256 CUs, with ragged edges: 16x32, 32x32, 64x32, 64x128, 128x128, 128x256
           # and 256x256, depths of one step, of several and with a cut last step
           (1, 28690, 80), (16, 7200, 272), (30, 7190, 656), (60, 7201, 144), (300, 2601, 304), (301, 2602, 1296), (1000, 3603, 16),
           (999, 3601, 400), (1801, 4002, 128), (1799, 4001, 272), (4000, 3702, 176), (3851, 3841, 256), (3999, 3701, 528)]


@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
@pytest.mark.parametrize("M,N,K", MATMULS)
def test_int8_matmul(M, N, K, dtype):
    say("matmul", M, N, K, NAME[dtype])
    g = rng(M + 3 * N + 5 * K)
    a, b, sa, sb = codes(g, M, K), codes(g, N, K), scale(g, M), scale(g, N)
    bias = (g.standard_normal(N) * 30).astype(np.float32)
    for pad, with_bias in ((0, False), (0, True), (16, True)):
        want, bound = ref.matmul(a, sa.astype(np.float64), b, sb.astype(np.float64),
                                 bias.astype(np.float64) if with_bias else None)
        out = torch.full((M, N + pad), 5.0, dtype=dtype, device=DEV)
        got = moe.int8_matmul(pad_codes(a, pad), dev(sa), pad_codes(b, pad), dev(sb), dev(bias) if with_bias else None,
                              out=out[:, :N])
        assert_within(got, want, stored(bound, want, dtype), f"pad={pad} bias={with_bias}")
        assert (out[:, N:] == 5).all(), "wrote between the rows"


def test_int8_matmul_largest_sums():
    """Every product 2^14 over the greatest depth: the 32-bit sums do not overflow."""
    K = 131056
    a = torch.full((17, K), -128, dtype=torch.int8, device=DEV)
    b = torch.full((40, K), -128, dtype=torch.int8, device=DEV)
    y = moe.int8_matmul(a, torch.ones(17, device=DEV), b, torch.ones(40, device=DEV), out_dtype=torch.float32)
    assert (f64(y) == float(np.float32(K * 16384))).all()


def test_int8_matmul_scales_that_are_not_finite():
    a, b = torch.ones(3, 32, dtype=torch.int8, device=DEV), torch.ones(20, 32, dtype=torch.int8, device=DEV)
    a[1] = 0
    sa = torch.tensor([1.0, float("inf"), float("nan")], device=DEV)
    y = moe.int8_matmul(a, sa, b, torch.ones(20, device=DEV))
    assert (y[0] == 32).all() and torch.isnan(y[1:]).all()


GROUPED = [  # T, K, N, depth, E, drop, skew
    (1, 1, 16, 16, 1, False, False), (1, 8, 96, 64, 32, False, False), (7, 2, 33, 48, 5, True, False),
    (64, 8, 256, 512, 64, False, False), (40, 3, 130, 144, 16, True, True), (100, 8, 512, 256, 4, False, False),
    (300, 4, 260, 208, 8, True, False), (513, 2, 192, 128, 3, False, True), (600, 8, 640, 384, 12, True, False),
    (128, 1, 64, 2048, 100, False, False), (9, 64, 48, 32, 7, True, False), (700, 6, 257, 1040, 2, False, False),
    # the wide tiles: 64x128, 128x128, 128x256 (many and few rows), 256x256, with empty and ragged groups
    (90, 6, 1301, 208, 10, True, False), (160, 6, 1902, 336, 16, True, True), (300, 4, 3003, 144, 20, False, False),
    (1, 8, 1000, 64, 1024, False, False), (3, 8, 70, 32, 1000, True, False), (40, 8, 2050, 272, 60, False, True), (1200, 4, 2403, 208, 12, False, False), (1100, 4, 2302, 400, 12, True, True)]


@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
@pytest.mark.parametrize("T,K,N,D,E,drop,skew", GROUPED)
def test_int8_grouped_matmul(T, K, N, D, E, drop, skew, dtype):
    say("grouped", T, K, N, D, E, drop, skew, NAME[dtype])
    ids = routes(T + N, T, K, E, drop)
    if skew:
        ids = np.where((ids >= 0) & (ids < E) & (rng(1).random(ids.shape) < 0.8), E - 1, ids)
    o, (r2r, rt2, off) = order_of(ids, E)
    R, kept = T * K, off[-1]
    g = rng(D + E)
    b, sb, bias = codes(g, E, N, D), scale(g, E, N), g.standard_normal((E, N)).astype(np.float32)
    expert = np.searchsorted(off, np.arange(kept), side="right") - 1
    for gather in (False, True):
        n = T if gather else R
        a, sa = codes(g, n, D), scale(g, n)
        src = r2r[:kept] // K if gather else np.arange(kept)
        for pad, with_bias in ((0, False), (16, True)):
            want, bound = np.full((R, N), 5.0), np.zeros((R, N))
            for e in range(E):
                at = np.nonzero(expert == e)[0]
                y, bd = ref.matmul(a[src[at]], sa[src[at]].astype(np.float64), b[e], sb[e].astype(np.float64),
                                   bias[e].astype(np.float64) if with_bias else None)
                want[at], bound[at] = y, stored(bd, y, dtype)
            out = torch.full((R, N + pad), 5.0, dtype=dtype, device=DEV)
            got = moe.int8_grouped_matmul(pad_codes(a, pad), dev(sa), pad_codes(b, pad), dev(sb), o, gather=gather,
                                          bias=dev(bias) if with_bias else None, out=out[:, :N])
            assert_within(got, want, bound, f"gather={gather} pad={pad} bias={with_bias}")
            assert (out[:, N:] == 5).all(), "wrote between the rows"


def test_grouped_weights_as_a_part_of_a_larger_tensor():
    """b as every expert's upper half, experts further apart than their rows."""
    T, K, N, D, E = 20, 2, 32, 64, 4
    o, (r2r, rt2, off) = order_of(routes(4, T, K, E, False), E)
    g = rng(0)
    b, sb = codes(g, E, 2 * N, D), scale(g, E, N)
    a, sa = codes(g, T, D), scale(g, T)
    bt = dev(b)
    y = moe.int8_grouped_matmul(dev(a), dev(sa), bt[:, N:], dev(sb), o, gather=True, out_dtype=torch.float32)
    z = moe.int8_grouped_matmul(dev(a), dev(sa), bt[:, N:].contiguous(), dev(sb), o, gather=True, out_dtype=torch.float32)
    assert torch.equal(y, z)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,K,E,H,I", [(1, 2, 8, 128, 64), (37, 4, 16, 256, 128), (300, 8, 12, 384, 256)])
def test_int8_layer(T, K, E, H, I):
    """An 8-bit MoE layer as it is served: sort, FC1 gathering the tokens' rows, SwiGLU,
    quantize, FC2, combine; the end against the 64-bit evaluation from the GPU's own
    FC2 input."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, H, device=DEV, generator=g, dtype=torch.bfloat16)
    top, ids = torch.randn(T, 2 * E, device=DEV, generator=g).topk(K)  # half of the experts are elsewhere
    w = torch.softmax(top, 1).contiguous()
    w1, s1 = moe.quantize_int8(torch.randn(E * 2 * I, H, device=DEV, generator=g) * H ** -0.5)
    w2, s2 = moe.quantize_int8(torch.randn(E * H, I, device=DEV, generator=g) * I ** -0.5)
    o = moe.sort_routes(ids, E)
    kept = int(o.offsets[-1])
    xq, xs = moe.quantize_int8(x)
    h = torch.zeros(T * K, 2 * I, dtype=torch.bfloat16, device=DEV)
    moe.int8_grouped_matmul(xq, xs, w1.view(E, 2 * I, H), s1.view(E, 2 * I), o, gather=True, out=h)
    gate, up = h.float().chunk(2, dim=1)
    aq, a_s = moe.quantize_int8(torch.nn.functional.silu(gate) * up)
    fc2 = moe.int8_grouped_matmul(aq, a_s, w2.view(E, H, I), s2.view(E, H), o, out_dtype=torch.float32)
    y = moe.combine(fc2, o, w)
    r2r, _, off = (v.cpu().numpy() for v in o.tensors())
    expert = np.searchsorted(off, np.arange(kept), side="right") - 1
    route = r2r[:kept]
    xd, w1d = f64(xq) * f64(xs)[:, None], (f64(w1) * f64(s1)[:, None]).reshape(E, 2 * I, H)
    ad, w2d = f64(aq) * f64(a_s)[:, None], (f64(w2) * f64(s2)[:, None]).reshape(E, H, I)
    want_h = np.stack([w1d[e] @ xd[r // K] for e, r in zip(expert, route)]) if kept else np.zeros((0, 2 * I))
    assert_within(h[:kept], want_h, stored(3.01 * U32 * np.abs(want_h) + 1e-12, want_h, torch.bfloat16), "FC1")
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    for row in range(kept):
        term = f64(w).reshape(-1)[route[row]] * (w2d[expert[row]] @ ad[row])
        want[route[row] // K] += term
        mag[route[row] // K] += np.abs(term)
    # each term: 3 roundings of the product and 1 of its storage, then K + 1 of the sum; 1e-12: the reference's own
    assert_within(y, want, (K + 6) * U32 * mag + 1e-12, "layer")


@pytest.mark.parametrize("on_input", [False, True])
def test_training_step(on_input):
    """One training step's expert part, dispatch -> linear experts -> combine and back,
    against autograd in 64 bits. The router weight is applied on either side."""
    T, K, E, H, D = 50, 3, 6, 72, 40
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, H, device=DEV, generator=g)
    w = torch.rand(T, K, device=DEV, generator=g)
    ids = torch.randint(0, E + 2, (T, K), device=DEV, generator=g)
    W = torch.randn(E, D, H, device=DEV, generator=g)
    dy = torch.randn(T, D, device=DEV, generator=g)
    o = moe.sort_routes(ids, E)
    off = o.offsets.tolist()
    w_in, w_out = (w, None) if on_input else (None, w)
    xs = moe.dispatch(x, o, w_in, out=torch.zeros(T * K, H, device=DEV))
    rows = torch.zeros(T * K, D, device=DEV)
    for e in range(E):
        rows[off[e]:off[e + 1]] = (xs[off[e]:off[e + 1]].double() @ W[e].double().t().contiguous()).float()
    y = moe.combine(rows, o, w_out)
    drows, dw = moe.combine_grad(dy, o, None if on_input else rows, w_out, out=torch.zeros(T * K, D, device=DEV))
    dxs = torch.zeros(T * K, H, device=DEV)
    for e in range(E):
        dxs[off[e]:off[e + 1]] = (drows[off[e]:off[e + 1]].double() @ W[e].double()).float()
    dx, dw_in = moe.dispatch_grad(dxs, o, x if on_input else None, w_in)
    dw = dw_in if on_input else dw
    X, Wt = x.cpu().double().requires_grad_(), w.cpu().double().requires_grad_()
    idc, Wc = ids.cpu(), W.cpu().double()
    Y = torch.zeros(T, D, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            if idc[t, k] < E:
                Y[t] = Y[t] + Wt[t, k] * (Wc[idc[t, k]] @ X[t])
    (Y * dy.cpu().double()).sum().backward()
    # each value is a sum of products of fp32 values that passed at most 3 roundings
    # each (dispatch, experts, storage) and K + 1 or H + 1 in its own sum
    aW, ax, aw, ady = (v.cpu().double().abs().numpy() for v in (W, x, w, dy))
    my, mx, mw = np.zeros((T, D)), np.zeros((T, H)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            e = int(idc[t, k])
            if e < E:
                my[t] += aw[t, k] * (aW[e] @ ax[t])
                mx[t] += aw[t, k] * (ady[t] @ aW[e])
                mw[t, k] = ady[t] @ aW[e] @ ax[t]
    n = K + 8
    assert_within(y, Y.detach().numpy(), n * U32 * my, "y")
    assert_within(dx, X.grad.numpy(), n * U32 * mx, "dx")
    assert_within(dw, Wt.grad.numpy(), (max(H, D) + 8) * U32 * mw, "dw")


def chain(x, ids, w, b, sb, E):
    o = moe.sort_routes(ids, E)
    q, s = moe.quantize_int8(x)
    rows = moe.int8_grouped_matmul(q, s, b, sb, o, gather=True)
    y = moe.combine(rows, o, w)
    drows, dw = moe.combine_grad(y, o, rows, w)
    dx, dw2 = moe.dispatch_grad(drows, o, y, w)
    return y, dw, dx, dw2


def chain_inputs(seed, T=70, K=4, E=9, H=192, N=160):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, device=DEV, generator=g, dtype=torch.bfloat16)
    ids = torch.randint(0, E, (T, K), device=DEV, generator=g)
    w = torch.rand(T, K, device=DEV, generator=g)
    b, sb = moe.quantize_int8(torch.randn(E * N, H, device=DEV, generator=g))
    return x, ids, w, b.view(E, N, H), sb.view(E, N), E


def test_two_streams_at_once():
    ins = [chain_inputs(i, T=200 + 100 * i) for i in range(2)]
    want = [chain(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        got = []
        for i, s in zip(ins, streams):
            with torch.cuda.stream(s):
                got.append(chain(*i))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_stream_argument():
    """A call on another stream than the current one: its results and temporaries belong
    to that stream."""
    x, ids, w, b, sb, E = chain_inputs(4)
    want = chain(x, ids, w, b, sb, E)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = moe.sort_routes(ids, E, stream=s)
    q, qs = moe.quantize_int8(x, stream=s)
    rows = moe.int8_grouped_matmul(q, qs, b, sb, o, gather=True, stream=s)
    y = moe.combine(rows=rows, order=o, weights=w, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_graph_replay():
    """Captured once, replayed on new inputs with eager work of the same operators in
    between; two graphs at once. Each replay equals the eager result."""
    a, b = chain_inputs(1), chain_inputs(2, T=330, K=2, E=5)
    for i in (a, b):
        chain(*i)
    torch.cuda.synchronize()
    graphs = []
    for i in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(*i)
        graphs.append((g, out))
    for n in range(4):
        for k, i in enumerate((a, b)):
            i[0].copy_(chain_inputs(10 * n + k, T=i[0].shape[0], K=i[1].shape[1], E=i[5])[0])
            i[1].copy_((i[1] + n + 1) % i[5])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, (g, out) in zip((a, b), graphs):
            want = chain(*i)
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(out, want)), n


def test_binding_refuses():
    x, ids, w, b, sb, E = chain_inputs(1)
    o = moe.sort_routes(ids, E)
    T, K = ids.shape
    bad = [
        lambda: moe.sort_routes(ids.float(), E), lambda: moe.sort_routes(ids[0], E), lambda: moe.sort_routes(ids.t(), E),
        lambda: moe.dispatch(x[:-1], o), lambda: moe.dispatch(x.double(), o), lambda: moe.dispatch(x.t(), o),
        lambda: moe.dispatch(x, o, w.double()), lambda: moe.dispatch(x, o, w[:, :1]), lambda: moe.dispatch(x, o, w.cpu()),
        lambda: moe.dispatch(x, o, out=x), lambda: moe.dispatch(x, (o,)),
        lambda: moe.combine(x, o), lambda: moe.combine(torch.zeros(T * K, 8, device=DEV), o, out=torch.zeros(T, 9, device=DEV)),
        lambda: moe.combine_grad(x, o, rows=torch.zeros(T * K, x.shape[1], device=DEV, dtype=x.dtype)),
        lambda: moe.dispatch_grad(torch.zeros(T * K, 8, device=DEV), o, x=torch.zeros(T, 8, device=DEV)),
        lambda: moe.quantize_int8(x.int()), lambda: moe.quantize_int8(x[0]), lambda: moe.quantize_int8(x, out=x),
        lambda: moe.int8_matmul(x, w, b[0], sb[0]), lambda: moe.int8_matmul(b[0], sb[0], b[0][:, :64], sb[0]),
        lambda: moe.int8_matmul(b[0], sb[0][:-1], b[1], sb[1]), lambda: moe.int8_matmul(b[0], sb[0], b[1], sb[1], bias=sb),
        lambda: moe.int8_matmul(b[0], sb[0], b[1], sb[1], out_dtype=torch.float64),
        lambda: moe.int8_matmul(b[0], sb[0], b[1], sb[1], out_dtype=torch.float16, out=torch.zeros(160, 160, device=DEV)),
        lambda: moe.int8_grouped_matmul(b[0], sb[0], b, sb, o), lambda: moe.int8_grouped_matmul(b[0], sb[0], b[0], sb, o),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, moe.MoeError)):
            f()
            say("accepted", i)
    y = torch.zeros(T, T * K * 8, device=DEV)
    with pytest.raises(moe.MoeError):  # an output that shares memory with an input
        moe.combine(y.view(-1)[:T * K * 8].view(T * K, 8), o, out=y.view(-1)[:T * 8].view(T, 8))
