"""The operators in front of, between and beside the experts' products on the GPU, against plain
64-bit references: routing, RMS norm, activation (with their gradients) and low-rank
adapters, and runs of them together with the operators around the experts."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_top_amd as moe  # noqa: E402
from tests import expert_ops_ref as eref  # noqa: E402
from tests import layer_ops_ref as ref  # noqa: E402
from tests.expert_ops_ref import HALF, TINY, U32, assert_within, f64, stored  # noqa: E402

DT = [torch.bfloat16, torch.float16, torch.float32]
NAME = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
DEV = "cuda"


def rng(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def strided(a, pad, dtype):
    """The matrix as a view with `pad` more elements between its rows (NaN there)."""
    full = np.full((a.shape[0], a.shape[1] + pad), np.nan)
    full[:, :a.shape[1]] = a
    return dev(full, dtype)[:, :a.shape[1]]


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
#          T, E, K, groups, top_groups, group_top
ROUTES = [(1, 1, 1, 1, 1, 1), (5, 8, 2, 1, 1, 1), (3, 7, 7, 1, 1, 1), (64, 256, 8, 8, 4, 2), (63, 256, 8, 8, 3, 1),
          (33, 128, 6, 1, 1, 1), (17, 160, 6, 5, 2, 2), (9, 100, 20, 10, 3, 1), (6, 1024, 64, 1, 1, 1), (7, 300, 9, 3, 2, 2),
          (5, 1023, 5, 1, 1, 1), (11, 512, 8, 64, 7, 2), (130, 16, 4, 16, 5, 2), (4, 64, 64, 2, 2, 2), (2, 96, 3, 48, 2, 2)]


def logits_of(seed, T, E, dtype, mask):
    g = rng(seed)
    x = g.standard_normal((T, E)) * 2
    if mask == "ties":  # many equal logits
        x = np.round(x)
    if mask == "masked":  # experts left out, a token without any, one with the type's lowest values
        x[g.random((T, E)) < 0.3] = -np.inf
        x[0] = -np.inf
        if T > 1:
            x[1] = float(torch.finfo(dtype).min)
    return x


@pytest.mark.parametrize("T,E,K,G,top_groups,group_top", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, K, G, top_groups, group_top, score):
    say("route", T, E, K, G, top_groups, group_top, score)
    for n, (dtype, mask, renorm, with_bias) in enumerate([(torch.float32, "", True, True), (torch.bfloat16, "ties", True, False),
                                                          (torch.float16, "masked", False, False), (torch.float32, "masked", True, True),
                                                          (torch.bfloat16, "", False, True)]):
        g = rng(n + T + E)
        x = strided(logits_of(n + E, T, E, dtype, mask), n % 3, dtype)
        bias = (g.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
        if with_bias and mask and E > 8:
            bias[E // 2] = -np.inf
        x64 = f64(x)
        ids, w = moe.route(x, K, score=score, bias=None if bias is None else dev(bias), groups=G, top_groups=top_groups,
                           group_top=group_top, renormalize=renorm, scale=2.5)
        want_ids, want = ref.route(x64, K, score, None if bias is None else bias.astype(np.float64), G, top_groups, group_top,
                                   renorm, 2.5)
        assert ids.dtype == torch.int32 and w.dtype == torch.float32
        assert np.array_equal(ids.cpu().numpy(), want_ids), (dtype, mask, renorm)
        low = x64 > -1e30  # (the row of lowest values: distances are 0 there)
        slack = ref.route_slack(np.where(low, x64, -np.inf), score, K, renorm)
        assert_within(w, want, slack * want + 2.0 ** -149, (dtype, mask, renorm))


def test_route_infinities_and_nans():
    inf, nan = np.inf, np.nan
    x = np.array([[inf, 0.0, inf, -inf], [nan, 1.0, 0.0, 2.0], [nan, nan, nan, nan], [inf, nan, -inf, -inf], [0.0, 0.0, 0.0, 0.0]])
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(4, device=DEV)):
            ids, w = moe.route(dev(x, torch.float32), 3, score=score, bias=bias, renormalize=True)
            assert ids.tolist() == [[0, 2, 1], [3, 1, 2], [0, 1, 2], [0, 1, -1], [0, 1, 2]], score
            w = f64(w)
            assert np.isnan(w[1:4]).all() and np.allclose(w[4], 1 / 3, atol=1e-7)
            assert np.allclose(w[0], [0.5, 0.5, 0.0] if score == "softmax" else [0.4, 0.4, 0.2], atol=1e-7)
    # a bias decides where scores do not; +inf always chooses; NaN spoils every token
    x = torch.zeros(2, 4, device=DEV)
    assert moe.route(x, 2, bias=dev(np.array([0.0, 0.1, inf, -inf]), torch.float32))[0].tolist() == [[2, 1]] * 2
    assert moe.route(x, 2, bias=dev(np.array([0.0, nan, 0, 0]), torch.float32))[1].isnan().all()


def test_route_close_choices():
    """Scores that an fp32 score cannot tell apart: sigmoids of 20 + k / 2^19 differ by 4e-15."""
    x = 20 + np.arange(64)[rng(1).permutation(64)] / 2.0 ** 19
    x = np.stack([x, x[::-1]])
    for bias in (None, torch.full((64,), 0.25, device=DEV)):
        for score in ("sigmoid", "softmax"):
            ids, _ = moe.route(dev(x, torch.float32), 64, score=score, bias=bias)
            assert np.array_equal(ids.cpu().numpy(), np.argsort(-x, axis=1))


def test_route_equal_logits():
    """Rows of one value, of the type's lowest, of two values, alone and among others: the lower
    expert first, also where choices are compared in 64 bits."""
    for E, K in ((64, 8), (256, 8), (300, 64), (16, 16)):
        x = rng(E).standard_normal((13, E))
        x[1], x[2], x[4] = 0.0, -1e9, np.finfo(np.float32).min
        x[6] = np.where(np.arange(E) % 3 == 0, 1.0, 0.25)
        x[7, E // 2:] = -1e9
        for score, bias, G in (("softmax", None, 1), ("sigmoid", np.zeros(E), 1), ("softmax", np.full(E, 0.25), 1),
                               ("sigmoid", np.tile([0.25, 0.0], E // 2), 4)):
            for rows in (slice(None), slice(1, 3)):
                ids, w = moe.route(dev(x[rows], torch.float32), K, score=score, bias=None if bias is None else dev(bias, torch.float32),
                                   groups=G, top_groups=3 if G > 1 else 1, group_top=2)
                want_ids, want = ref.route(ref.f32(x[rows]), ids.shape[1], score, bias, G, 3 if G > 1 else 1, 2, True, 1.0)
                assert np.array_equal(ids.cpu().numpy(), want_ids), (E, score, G)
                # (distances below 16, up to 64 terms, a dozen operations: below 128 half steps)
                assert_within(w, want, 128 * U32 * want + 2.0 ** -149, (E, score, G))


def test_route_many_tokens():
    """Odd numbers of tokens over many blocks, a broadcast row, no tokens."""
    T, E, K = 5003, 64, 6
    x = rng(3).standard_normal((T, E)).astype(np.float32)
    ids, w = moe.route(dev(x), K, score="sigmoid", bias=torch.zeros(E, device=DEV), groups=8, top_groups=3, group_top=2)
    want_ids, want = ref.route(x.astype(np.float64), K, "sigmoid", np.zeros(E), 8, 3, 2, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert_within(w, want, ref.route_slack(x, "sigmoid", K, True) * want, "weights")
    one = dev(x[:1]).expand(100, E)
    ids, _ = moe.route(one, K)
    assert (ids == ids[0]).all()
    ids, w = moe.route(dev(x[:0]), K)
    assert ids.shape == (0, K) and w.shape == (0, K)
    assert moe.route_grad(w, dev(x[:0]), ids).shape == (0, E)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (5, 8, 2), (33, 128, 8), (7, 256, 8), (6, 1024, 64), (9, 300, 9), (130, 31, 3), (3, 60, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad(T, E, K, score, renorm):
    say("route_grad", T, E, K, score, renorm)
    for dtype in DT:
        g = rng(T + E)
        x = strided(g.standard_normal((T, E)) * 2, 3, dtype)
        x64 = f64(x)
        ids = np.argsort(-x64, axis=1, kind="stable")[:, :K].astype(np.int32)
        ids[g.random((T, K)) < 0.1] = -1
        dw = g.standard_normal((T, K)).astype(np.float32)
        out = torch.full((T, E + 5), 7.0, dtype=dtype, device=DEV)
        got = moe.route_grad(dev(dw), x, dev(ids), score=score, renormalize=renorm, scale=1.5, out=out[:, :E])
        want, mag = ref.route_grad(dw.astype(np.float64), x64, ids, score, renorm, 1.5)
        bound = 2 * (ref.route_slack(x64, score, K, renorm) + 8 * U32) * mag
        assert_within(got, want, stored(bound, want, dtype), NAME[dtype])
        assert (out[:, E:] == 7).all()


def test_route_grad_against_differences():
    """Central differences of the 64-bit weights; -inf logits, repeated and missing ids."""
    x = rng(5).standard_normal((4, 12))
    x[1, 3] = -np.inf
    ids = np.array([[0, 5, 7], [3, 2, -1], [4, 4, 9], [-1, -1, 100]], np.int32)
    dw = rng(6).standard_normal((4, 3)).astype(np.float32)

    def loss(x, score, renorm):
        total = 0.0
        for t in range(4):
            s = ref.scores(x[t:t + 1], score)[0]
            at = [(i, q) for i, q in zip(ids[t], dw[t]) if 0 <= i < 12 and x[t, i] > -np.inf]
            norm = sum(s[i] for i, _ in at) if renorm else 1.0
            total += sum(s[i] * q / norm for i, q in at)
        return total

    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = f64(moe.route_grad(dev(dw), dev(x, torch.float32), dev(ids), score=score, renormalize=renorm))
            x32 = ref.f32(x)
            h = 1e-5
            for t in range(4):
                for j in range(12):
                    if x32[t, j] == -np.inf:
                        assert got[t, j] == 0
                        continue
                    up, down = x32.copy(), x32.copy()
                    up[t, j] += h
                    down[t, j] -= h
                    slope = (loss(up, score, renorm) - loss(down, score, renorm)) / (2 * h)
                    # third derivatives of these are below 10, the terms below 4 in magnitude
                    assert abs(slope - got[t, j]) <= 10 * h * h + 1e-10 + 100 * U32 * 4, (score, renorm, t, j)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORMS = [(1, 1), (3, 7), (2, 8), (5, 64), (4, 129), (9, 520), (3, 1000), (2, 2049), (3, 4100), (64, 7168), (2, 9001),
         (3, 16392), (2, 32768), (600, 40), (4100, 264), (4097, 1500)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
def test_norm(T, H, dtype):
    say("norm", T, H, NAME[dtype])
    for n, (residual, wdt) in enumerate([(True, dtype), (False, torch.float32), (True, None)]):
        g = rng(T + H + n)
        pad = (0, 3, 8)[n]
        x = strided(g.standard_normal((T, H)), pad, dtype)
        res = strided(g.standard_normal((T, H)) * 3, 5 * n, dtype) if residual else None
        w = None if wdt is None else dev(g.standard_normal(H), wdt)
        w64 = np.ones(H) if w is None else f64(w)
        want_h = (x.float() + res.float()).to(dtype) if residual else x
        h64 = f64(want_h)
        r = ref.inverse_rms(h64, 1e-5)
        y64 = h64 * r * w64
        out = torch.full((T, H + pad), 7.0, dtype=dtype, device=DEV)
        y, h = moe.rms_norm(x, w, 1e-5, residual=res, out=out[:, :H])
        assert torch.equal(h, want_h) and (out[:, H:] == 7).all() and (residual or h is x)
        bound = 55 * U32 * np.abs(y64)
        assert_within(y, y64, stored(bound, y64, dtype), "y")
        # 8 bits: the codes of fl32(h w)
        p = ref.f32(np.float32(h64) * np.float32(w64))
        codes64, s64 = ref.quantize(p)
        both = torch.full((T, H), 7.0, dtype=dtype, device=DEV)
        codes, scales, h = moe.rms_norm_int8(x, w, 1e-5, residual=res, y=both)
        assert np.array_equal(codes.cpu().numpy(), codes64) and torch.equal(both, y) and torch.equal(h, want_h)
        s64 = s64 * r[:, 0]
        assert_within(scales, s64, 55 * U32 * s64 + 2.0 ** -149, "scales")
        alone = moe.rms_norm_int8(x, w, 1e-5, residual=res)
        assert torch.equal(alone[0], codes) and torch.equal(alone[1], scales)


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 64), (4, 129), (9, 520), (7, 2049), (3, 4100), (70, 7168), (2, 9001),
                                 (3, 16392), (2, 32768), (1500, 40), (1100, 1032)])
@pytest.mark.parametrize("dtype", DT, ids=NAME.get)
def test_norm_grad(T, H, dtype):
    say("norm_grad", T, H, NAME[dtype])
    for n, (more, wdt) in enumerate([(True, torch.float32), (False, dtype), (True, None)]):
        g = rng(T + H + n)
        dy, h = strided(g.standard_normal((T, H)), n, dtype), strided(g.standard_normal((T, H)), 2 * n, dtype)
        dtotal = strided(g.standard_normal((T, H)), 8 * n, dtype) if more else None
        w = None if wdt is None else dev(g.standard_normal(H), wdt)
        want, bound, dw64, dw_bound = ref.norm_grad(f64(dy), f64(h), np.ones(H) if w is None else f64(w), 1e-5,
                                                    None if dtotal is None else f64(dtotal))
        out = torch.full((T, H + n), 7.0, dtype=dtype, device=DEV)
        dx, dw = moe.rms_norm_grad(dy, h, w, 1e-5, dtotal=dtotal, out=out[:, :H])
        assert_within(dx, want, stored(bound, want, dtype), "dx")
        assert (out[:, H:] == 7).all()
        assert (dw is None) == (w is None)
        if w is not None:
            assert_within(dw, dw64, dw_bound, "dweight")
            again = moe.rms_norm_grad(dy, h, w, 1e-5, dtotal=dtotal)
            assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_norm_grad_against_differences():
    g = rng(9)
    x, w, dy = g.standard_normal((3, 20)), g.standard_normal(20), g.standard_normal((3, 20))
    xt, wt, dyt = dev(x, torch.float32), dev(w, torch.float32), dev(dy, torch.float32)
    x, w, dy = f64(xt), f64(wt), f64(dyt)
    dx, dw = (f64(v) for v in moe.rms_norm_grad(dyt, xt, wt, 1e-2))

    def loss(x, w):
        return (dy * (x / np.sqrt((x * x).mean(axis=1, keepdims=True) + 1e-2) * w)).sum()

    h = 1e-5
    for t in range(3):
        for j in range(20):
            step = np.zeros_like(x)
            step[t, j] = h
            # (third derivatives below 100; 300 roundings of terms below 20)
            assert abs((loss(x + step, w) - loss(x - step, w)) / (2 * h) - dx[t, j]) <= 100 * h * h + 1e-9 + 300 * U32 * 20
    for j in range(20):
        step = np.zeros_like(w)
        step[j] = h
        assert abs((loss(x, w + step) - loss(x, w - step)) / (2 * h) - dw[j]) <= 1e-9 + 300 * U32 * 20


@pytest.mark.parametrize("H", [33, 2000, 5000])
def test_norm_extremes(H):
    """Rows whose squares leave fp32's range both ways, zero rows, infinities and NaN."""
    g = rng(H)
    x = g.standard_normal((8, H))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0.0
    x[3] *= 2.0 ** -140  # subnormal
    x[4, 1] = np.inf
    x[5, 2] = np.nan
    x[6, :] = 1e-22
    x[7, 0] = 3e38
    for eps in (1e-6, 0.0, 1e-30):
        xt = dev(x, torch.float32)
        x64 = f64(xt)
        y, _ = moe.rms_norm(xt, None, eps)
        codes, scales, _ = moe.rms_norm_int8(xt, None, eps)
        rows = [r for r in (0, 1, 2, 3, 6, 7) if r != 2 or eps > 0]
        want = x64[rows] * ref.inverse_rms(x64[rows], eps)
        # (results below 2^-126 are subnormal: half of the smallest step)
        assert_within(y[rows], want, 55 * U32 * np.abs(want) + 2.0 ** -149, eps)
        codes64, s64 = ref.quantize(x64[rows])
        assert np.array_equal(codes[rows].cpu().numpy(), codes64)
        want = s64 * ref.inverse_rms(x64[rows], eps)[:, 0]
        assert_within(scales[rows], want, 55 * U32 * want + 2.0 ** -149, eps)
        y, codes, scales = f64(y), codes.cpu().numpy(), f64(scales)
        assert np.isnan(y[4, 1]) and (np.delete(y[4], 1) == 0).all() and np.isnan(y[5]).all()
        assert not codes[4:6].any() and not np.isfinite(scales[4:6]).any()
        if eps == 0:
            assert np.isnan(y[2]).all() and not codes[2].any()
        # the gradient of the rows in range
        dy = dev(g.standard_normal((8, H)), torch.float32)
        dx, _ = moe.rms_norm_grad(dy, xt, None, eps)
        rows = [0, 7] + ([2] if eps > 0 else []) + ([1, 6] if eps != 1e-30 else [])
        want, bound, _, _ = ref.norm_grad(f64(dy)[rows], x64[rows], np.ones(H), eps, None)
        ok = np.abs(want) < 1e38
        assert_within(dx[rows][torch.as_tensor(ok).to(DEV)], want[ok], (bound + U32 * np.abs(want) + 2.0 ** -148)[ok], eps)


def test_norm_in_place_total():
    for T, H in ((5, 1000), (4100, 264)):
        x, res = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T, H, device=DEV).bfloat16()
        y, h = moe.rms_norm(x, None, residual=res)
        kept = res.clone()
        y2, h2 = moe.rms_norm(x, None, residual=kept, total=kept)
        assert h2 is kept and torch.equal(h, kept) and torch.equal(y, y2)
    # one row of residual for all tokens, one row of x for all
    y, h = moe.rms_norm(x[:1].expand(T, H), None, residual=res[:1].expand(T, H))
    assert (h == h[0]).all() and (y == y[0]).all()
    y, h = moe.rms_norm(x[:0], None, residual=res[:0])
    assert y.shape == (0, H)
    dx, dw = moe.rms_norm_grad(x[:0], x[:0], torch.ones(H, device=DEV))
    assert dx.shape == (0, H) and not dw.any()


# ---------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------
ACTS = [(1, 1, 1, 1), (2, 3, 7, 4), (5, 2, 8, 3), (37, 6, 129, 16), (64, 8, 256, 64), (33, 9, 1000, 12), (3, 17, 2049, 20),
        (5, 2, 4100, 8), (2, 2, 9001, 5), (1, 3, 32768, 4), (600, 8, 520, 32)]


def sorted_routes(seed, T, K, E, drop):
    g = rng(seed)
    ids = g.integers(0, E, (T, K))
    if drop:
        ids = np.where(g.random((T, K)) < 0.4, E + 3, ids)
        ids[0] = -1
    order = moe.sort_routes(dev(ids.astype(np.int32)), E)
    r2r, rt2, off = (v.cpu().numpy() for v in order.tensors())
    return order, r2r, rt2, off[-1]


@pytest.mark.parametrize("T,K,I,E", ACTS)
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_activate(T, K, I, E, act):
    say("activate", T, K, I, E, act)
    wide = 2 * I if act == "swiglu" else I
    for n, dtype in enumerate(DT):
        for drop in (False, True):
            order, r2r, rt2, kept = sorted_routes(T + K + n, T, K, E, drop)
            R = T * K
            g = rng(I + n + drop)
            h_np = g.standard_normal((R, wide)) * 2
            h_np[kept:] = np.nan  # never read
            pad = (0, 3, 8)[n]
            h = strided(h_np, pad, dtype)
            h64 = f64(h)[:kept]
            a64 = ref.activation(h64, act)
            w = g.standard_normal((T, K)).astype(np.float32)
            for weights in (None, dev(w)):
                wv = np.ones(kept) if weights is None else w.reshape(-1)[r2r[:kept]].astype(np.float64)
                want = np.full((R, I), 7.0)
                want[:kept] = a64 * wv[:, None]
                bound = stored(12 * U32 * np.abs(want), want, dtype)
                bound[kept:] = 0
                out = torch.full((R, I + pad), 7.0, dtype=dtype, device=DEV)
                got = moe.activate(h, act, order, weights, out=out[:, :I])
                assert_within(got, want, bound, "activate")
                assert (out[:, I:] == 7).all()
                # 8 bits
                codes64, s64 = ref.quantize(a64)
                out = torch.full((R, I + pad), 7, dtype=torch.int8, device=DEV)
                scales = torch.full((R,), 7.0, device=DEV)
                codes, got_s = moe.activate_int8(h, act, order, weights, out=out[:, :I], scales=scales)
                want_c = np.full((R, I), 7)
                want_c[:kept] = codes64
                assert np.array_equal(codes.cpu().numpy(), want_c) and (out[:, I:] == 7).all() and got_s is scales
                want_s = np.full(R, 7.0)
                want_s[:kept] = np.float32(s64) * np.float32(wv)
                assert np.array_equal(f64(scales), want_s)
                # gradient
                da_np = g.standard_normal((R, I))
                da_np[kept:] = np.nan
                da = strided(da_np, 8 - pad, dtype)
                da64 = f64(da)[:kept]
                want = np.full((R, wide), 7.0)
                grad, gb = ref.activation_grad(da64, h64, act, wv)
                want[:kept] = grad
                bound = np.zeros((R, wide))
                bound[:kept] = stored(gb, grad, dtype)
                out = torch.full((R, wide + pad), 7.0, dtype=dtype, device=DEV)
                dh, dw = moe.activate_grad(da, h, act, order, weights, out=out[:, :wide])
                assert_within(dh, want, bound, "dh")
                assert (out[:, wide:] == 7).all() and (dw is None) == (weights is None)
                if weights is not None:
                    terms = da64 * a64
                    want_w, bound_w = np.zeros(R), np.zeros(R)
                    want_w[r2r[:kept]] = terms.sum(axis=1)
                    bound_w[r2r[:kept]] = (ref.DEPTH + 12) * U32 * np.abs(terms).sum(axis=1)
                    assert_within(dw.reshape(-1), want_w, bound_w, "dweights")
    # all rows, without an order
    got = moe.activate(h[:kept], act)
    assert_within(got, a64, stored(12 * U32 * np.abs(a64), a64, dtype), "all rows")


def test_activate_wave_rows():
    """Rows of a wave each, several a block and many blocks; the activation alone."""
    for dtype, R, I in ((torch.bfloat16, 9001, 1032), (torch.float32, 4100, 200), (torch.float16, 4099, 2048)):
        h = dev(rng(R).standard_normal((R, 2 * I)), dtype)
        h64 = f64(h)
        a64 = ref.activation(h64, "swiglu")
        assert_within(moe.activate(h), a64, stored(12 * U32 * np.abs(a64), a64, dtype), "activate")
        codes, scales = moe.activate_int8(h)
        codes64, s64 = ref.quantize(a64)
        assert np.array_equal(codes.cpu().numpy(), codes64) and np.array_equal(f64(scales), s64)


def test_activate_blocks_walk_over_rows():
    """More rows than a launch has blocks, a block's barriers in between: the bits of the same rows
    alone (codes are exact in any case, gradients sum in an order that the rows do not change)."""
    g = rng(12)
    for dtype, R, I in ((torch.bfloat16, 8700, 2064), (torch.float32, 8500, 1029)):
        h, da = dev(g.standard_normal((R, 2 * I)), dtype), dev(g.standard_normal((R, I)), dtype)
        h[5, :I] = -40.0  # (by the exact way)
        weights = dev(g.standard_normal((R, 1)).astype(np.float32))
        one = lambda n: moe.sort_routes(torch.zeros(n, 1, dtype=torch.int32, device=DEV), 1)
        order = one(R)
        codes, scales = moe.activate_int8(h, order=order, weights=weights)
        out = moe.activate(h, order=order, weights=weights)
        dh, dw = moe.activate_grad(da, h, order=order, weights=weights)
        for lo in (0, 4000, R - 600):
            s, part = slice(lo, lo + 600), one(600)
            c, sc = moe.activate_int8(h[s], order=part, weights=weights[s])
            assert torch.equal(c, codes[s]) and torch.equal(sc, scales[s])
            assert torch.equal(moe.activate(h[s], order=part, weights=weights[s]), out[s])
            d, w = moe.activate_grad(da[s], h[s], order=part, weights=weights[s])
            assert torch.equal(d, dh[s]) and torch.equal(w, dw[s])


def test_activate_codes_next_to_a_half():
    """relu2 of integers: many exact halves (ties to even), and values that fp32 rounds onto
    the wrong side: rows whose largest square is 127 * 2^k."""
    g = rng(4)
    h = np.zeros((40, 300))
    for m in range(40):
        h[m] = np.sqrt((g.integers(0, 254, 300) + g.choice([0.0, 1e-6, -1e-6], 300)) / 2 * 2.0 ** (m - 20)).clip(0)
        h[m, 0] = np.sqrt(127 * 2.0 ** (m - 20))
    ht = dev(np.nan_to_num(h), torch.float32)
    codes, scales = moe.activate_int8(ht, "relu2")
    codes64, s64 = ref.quantize(ref.activation(f64(ht), "relu2"))
    assert np.array_equal(codes.cpu().numpy(), codes64) and np.array_equal(f64(scales), s64)
    h = dev(np.tile(np.concatenate([[127.0], np.arange(0, 127, 0.5)]) ** 0.5, (3, 1)), torch.float64)
    ht = h.float()
    codes, _ = moe.activate_int8(ht, "relu2")
    assert np.array_equal(codes.cpu().numpy(), ref.quantize(ref.activation(f64(ht), "relu2"))[0])


def test_activate_extremes():
    """Gates far out on both sides, subnormal and zero rows, infinities and NaN."""
    I = 300
    g = rng(8)
    h = g.standard_normal((9, 2 * I))
    h[0, :I] = -np.linspace(70, 130, I)  # exp below fp32's normal range
    h[0, I:] = 1e30
    h[1, :I] = np.linspace(-700, 700, I)
    h[2] *= 1e-20                        # activations of 1e-40
    h[3] = 0.0
    h[4, :I] *= 1e-30
    h[5, 3] = np.nan
    h[6, I + 5] = np.inf
    h[7, :I] = -90.0
    h[8, 0] = -np.inf                    # silu(-inf) is 0 * inf: NaN, as the formula in fp32 gives it
    ht = dev(h, torch.float32)
    a64 = ref.activation(f64(ht)[:8], "swiglu")
    codes, scales = moe.activate_int8(ht)
    fine = [0, 1, 2, 3, 4, 7]
    codes64, s64 = ref.quantize(a64[fine])
    assert np.array_equal(codes[fine].cpu().numpy(), codes64) and np.array_equal(f64(scales[fine]), s64)
    bad = [5, 6, 8]
    assert not codes[bad].any() and not torch.isfinite(scales[bad]).any()
    got = f64(moe.activate(ht))
    # exp below 2^-126 is subnormal: off by half of 2^-149 times |g u|
    mag = np.abs(f64(ht)[:8, :I] * f64(ht)[:8, I:])
    with np.errstate(invalid="ignore"):
        bound = 12 * U32 * np.abs(a64) + 2.0 ** -148 * mag + 2.0 ** -149
    assert (np.abs(got[fine] - a64[fine]) <= bound[fine]).all()
    assert np.isnan(got[5, 3]) and np.isinf(got[6, 5]) and np.isnan(got[8, 0])
    z = dev(np.array([[np.nan, -1.0, 2.0], [-np.inf, np.inf, 1.0]]), torch.float32)
    assert torch.equal(torch.nan_to_num(moe.activate(z, "relu2"), nan=5.0), dev(np.array([[5.0, 0, 4], [0, np.inf, 1]]), torch.float32).nan_to_num(nan=5.0))


def test_activate_grad_against_differences():
    g = rng(10)
    h, da = dev(g.standard_normal((3, 24)) * 2, torch.float32), dev(g.standard_normal((3, 12)), torch.float32)
    dh, _ = moe.activate_grad(da, h)
    h64, da64, dh = f64(h), f64(da), f64(dh)
    e = 1e-5
    for t in range(3):
        for j in range(24):
            step = np.zeros_like(h64)
            step[t, j] = e
            slope = ((ref.activation(h64 + step, "swiglu") - ref.activation(h64 - step, "swiglu")) * da64).sum() / (2 * e)
            assert abs(slope - dh[t, j]) <= 20 * e * e + 1e-9 + 40 * U32 * 30


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------
#          T, n, r, H, N
ADAPTS = [(1, 1, 8, 16, 1), (1, 8, 16, 7168, 4096), (3, 2, 8, 48, 17), (64, 32, 16, 1024, 520), (17, 1024, 8, 64, 100),
          (70, 3, 40, 208, 300), (33, 4, 256, 320, 257), (200, 2, 64, 512, 130), (300, 1, 16, 2048, 64), (129, 1, 104, 272, 96),
          # many tokens an adapter
          (2100, 3, 64, 208, 300), (2048, 2, 256, 64, 200), (2300, 70, 16, 144, 130), (2200, 1, 104, 272, 96),
          (2050, 5, 128, 80, 257), (2100, 2, 8, 400, 128), (2049, 4, 40, 2064, 137), (2060, 1, 32, 96, 1000), (2048, 1, 16, 16, 5)]


def adapter_case(seed, T, n, r, H, N, dtype, none):
    g = rng(seed)
    ids = g.integers(0, n, T)
    ids[g.random(T) < none] = -1
    return (ids, g.standard_normal((T, N)), g.standard_normal((T, H)), g.standard_normal((n, r, H)) / H ** 0.5,
            g.standard_normal((n, N, r)) / r ** 0.5, (g.random(n) + 0.5).astype(np.float32))


@pytest.mark.parametrize("T,n,r,H,N", ADAPTS)
@pytest.mark.parametrize("dtype", DT[:2], ids=NAME.get)
def test_adapt(T, n, r, H, N, dtype):
    say("adapt", T, n, r, H, N, NAME[dtype])
    part = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -21
    for none, pad in ((0.0, 0), (0.4, 3)):
        ids, base, x, a, b, scales = adapter_case(T + r + H, T, n, r, H, N, dtype, none)
        base, x = strided(base, pad, dtype), strided(x, 2 * pad, dtype)
        pool_a = torch.full((n, r + pad, H + pad), float("nan"), dtype=dtype, device=DEV)  # (a pool's slices)
        pool_b = torch.full((n, N, r + 5 * pad), float("nan"), dtype=dtype, device=DEV)
        a_t, b_t = pool_a[:, :r, :H], pool_b[:, :, :r]
        a_t.copy_(dev(a, dtype))
        b_t.copy_(dev(b, dtype))
        order = moe.sort_routes(dev(ids.astype(np.int32)[:, None]), n)
        out = torch.full((T, N + pad), 7.0, dtype=dtype, device=DEV)
        got = moe.adapt(base, x, order, a_t, b_t, dev(scales), out=out[:, :N])
        want, bound = ref.adapt(f64(base), f64(x), ids, f64(a_t), f64(b_t), scales.astype(np.float64), part)
        assert_within(got, want, np.where((ids >= 0)[:, None], stored(bound, want, dtype), 0.0), "adapt")
        assert (out[:, N:] == 7).all()
        fresh = moe.adapt(base, x, order, a_t, b_t, dev(scales))
        assert torch.equal(fresh, got)
        here = base.clone() if pad == 0 else base
        moe.adapt(here, x, order, a_t, b_t, dev(scales), out=here)  # in place
        assert torch.equal(here, got)


#                 T, n, r, H, N: blocks that walk over several pieces of the columns
WALKS = [(4100, 3, 24, 64, 4100), (9000, 5, 72, 64, 2600), (6000, 4, 256, 48, 3333), (16000, 2, 16, 16, 2000),
         (1500, 200, 72, 64, 2000), (1900, 300, 16, 64, 4000)]


@pytest.mark.parametrize("T,n,r,H,N", WALKS)
@pytest.mark.parametrize("dtype", DT[:2], ids=NAME.get)
def test_adapt_many_columns(T, n, r, H, N, dtype):
    say("adapt", T, n, r, H, N, NAME[dtype])
    part = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -21
    ids, base, x, a, b, scales = adapter_case(T + r, T, n, r, H, N, dtype, 0.1)
    base, x, a, b = dev(base, dtype), dev(x, dtype), dev(a, dtype), dev(b, dtype)
    order = moe.sort_routes(dev(ids.astype(np.int32)[:, None]), n)
    got = moe.adapt(base, x, order, a, b, dev(scales))
    some = np.unique(np.concatenate([np.arange(200), rng(1).integers(0, T, 300), [T - 1]]))
    want, bound = ref.adapt(f64(base)[some], f64(x)[some], ids[some], f64(a), f64(b), scales.astype(np.float64), part)
    assert_within(got[torch.from_numpy(some).to(DEV)], want,
                  np.where((ids[some] >= 0)[:, None], stored(bound, want, dtype), 0.0), "adapt")
    for _ in range(3):
        here = base.clone()
        moe.adapt(here, x, order, a, b, dev(scales), out=here)
        assert torch.equal(here, got)


def test_adapt_edges():
    """No tokens, no token with an adapter, one adapter for all by stride 0, scales missing, a
    token with an infinity, values beyond the type's range between the products."""
    T, n, r, H, N = 40, 3, 16, 64, 80
    for dtype in DT[:2]:
        ids, base, x, a, b, _ = adapter_case(1, T, n, r, H, N, dtype, 0.2)
        base, x, a, b = dev(base, dtype), dev(x, dtype), dev(a, dtype), dev(b, dtype)
        nobody = moe.sort_routes(torch.full((T, 1), -1, device=DEV), n)
        assert torch.equal(moe.adapt(base, x, nobody, a, b), base)
        empty = moe.sort_routes(torch.zeros((0, 1), dtype=torch.int32, device=DEV), n)
        assert moe.adapt(base[:0], x[:0], empty, a, b).shape == (0, N)
        order = moe.sort_routes(dev(ids.astype(np.int32)[:, None]), n)
        one = moe.adapt(base, x, order, a[:1].expand(n, r, H), b[:1].expand(n, N, r))
        same = moe.sort_routes(dev(np.where(ids >= 0, 0, -1).astype(np.int32)[:, None]), 1)
        assert torch.equal(one, moe.adapt(base, x, same, a[:1], b[:1], torch.ones(1, device=DEV)))
        ref_out = moe.adapt(base, x, order, a, b)
        t = int(np.nonzero(ids >= 0)[0][0])
        x2 = x.clone()
        x2[t, 3] = float("inf")
        got = moe.adapt(base, x2, order, a, b)
        assert not torch.isfinite(got[t]).any() and torch.equal(got[torch.arange(T) != t], ref_out[torch.arange(T) != t])
        # v up to 1e6 and more (fp16 ends at 65504), brought back by b; and v of 1e-9
        for up in (2.0 ** 15, 2.0 ** -22):
            big = dev(f64(x) * 16, dtype) if up > 1 else dev(f64(x) * 2.0 ** -10, dtype)
            a3 = dev(f64(a) * 2.0 ** 11, dtype) if up > 1 else dev(f64(a) * 2.0 ** -8, dtype)
            b3 = dev(f64(b) * 2.0 ** -13, dtype) if up > 1 else dev(f64(b) * 2.0 ** 12, dtype)
            got = moe.adapt(base, big, order, a3, b3)
            part = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -21
            want, bound = ref.adapt(f64(base), f64(big), ids, f64(a3), f64(b3), np.ones(n), part)
            assert_within(got, want, stored(bound, want, dtype), up)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_serving_run():
    """norm -> route -> sort -> experts in 8 bits -> combine, beside a shared projection with
    adapters, each step against its reference on what the GPU had."""
    T, H, I, E, K, n = 37, 256, 128, 16, 4, 3
    g = rng(20)
    dtype = torch.bfloat16
    x, stream = dev(g.standard_normal((T, H)), dtype), dev(g.standard_normal((T, H)), dtype)
    weight, bias = dev(g.random(H) + 0.5, dtype), dev(g.standard_normal(E) * 0.1, torch.float32)
    y = torch.empty_like(x)
    codes, scales, total = moe.rms_norm_int8(x, weight, residual=stream, y=y)
    logits = y.float() @ dev(g.standard_normal((H, E)) / 16, torch.float32)
    ids, w = moe.route(logits, K, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2, scale=2.5)
    want_ids, want_w = ref.route(f64(logits), K, "sigmoid", f64(bias), 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    here = E // 2  # the other experts are elsewhere
    order = moe.sort_routes(ids, here)
    w1, s1 = moe.quantize_int8(dev(g.standard_normal((here * 2 * I, H)), torch.float32))
    w2, s2 = moe.quantize_int8(dev(g.standard_normal((here * H, I)), torch.float32))
    h = moe.int8_grouped_matmul(codes, scales, w1.view(here, 2 * I, H), s1.view(here, -1), order, gather=True)
    aq, a_s = moe.activate_int8(h, "swiglu", order)
    rows = moe.int8_grouped_matmul(aq, a_s, w2.view(here, H, I), s2.view(here, -1), order)
    out = moe.combine(rows, order, w)
    kept = int(order.offsets[-1])
    r2r = order.row_to_route.cpu().numpy()[:kept]
    want_c, want_s = ref.quantize(ref.activation(f64(h)[:kept], "swiglu"))
    assert np.array_equal(aq[:kept].cpu().numpy(), want_c) and np.array_equal(f64(a_s)[:kept], want_s)
    experts = np.searchsorted(order.offsets.cpu().numpy(), np.arange(kept), side="right") - 1
    deq2 = f64(w2).reshape(here, H, I) * f64(s2).reshape(here, H)[:, :, None]
    full = np.einsum("rij,rj->ri", deq2[experts], want_c * want_s[:, None])
    terms = np.zeros((T * K, H))
    terms[r2r] = full * f64(w).reshape(-1)[r2r][:, None]
    want = terms.reshape(T, K, H).sum(1)
    mag = np.abs(terms).reshape(T, K, H).sum(1)
    # rows of bf16 (2^-8 each), then the sum
    assert_within(out, want, stored((HALF[dtype] + 10 * U32) * mag, want, dtype), "layer")
    # the shared projection, and its adapters
    ws, ss = moe.quantize_int8(dev(g.standard_normal((96, H)), torch.float32))
    shared = moe.int8_matmul(codes, scales, ws, ss)
    who = g.integers(-1, n, (T, 1)).astype(np.int32)
    a, b = dev(g.standard_normal((n, 16, H)) / 16, dtype), dev(g.standard_normal((n, 96, 16)) / 4, dtype)
    want, bound = ref.adapt(f64(shared), f64(y), who[:, 0], f64(a), f64(b), np.ones(n), 2.0 ** -16)
    got = moe.adapt(shared, y, moe.sort_routes(dev(who), n), a, b, out=shared)
    assert_within(got, want, stored(bound, want, dtype), "adapters")


class Layer(torch.autograd.Function):
    """norm -> route -> dispatch -> products -> activation with the router's weights -> products
    -> combine, and back, as a training program would wrap the calls."""
    @staticmethod
    def forward(ctx, x, res, wn, wr, w1, w2, K):
        y, h = moe.rms_norm(x, wn, residual=res)
        logits = y @ wr
        ids, w = moe.route(logits, K)
        order = moe.sort_routes(ids, w1.shape[0])
        ctx.order, ctx.off = order, order.offsets.tolist()
        xs = moe.dispatch(y, order)
        h1 = torch.cat([xs[a:b] @ w1[e] for e, (a, b) in enumerate(zip(ctx.off, ctx.off[1:]))])
        a = moe.activate(h1, "swiglu", order, w)
        rows = torch.cat([a[i:j] @ w2[e] for e, (i, j) in enumerate(zip(ctx.off, ctx.off[1:]))])
        ctx.save_for_backward(h, y, wn, wr, logits, ids, w, xs, h1, a, w1, w2)
        return moe.combine(rows, order), h

    @staticmethod
    def backward(ctx, dout, dh):
        h, y, wn, wr, logits, ids, w, xs, h1, a, w1, w2 = ctx.saved_tensors
        spans = list(enumerate(zip(ctx.off, ctx.off[1:])))
        drows, _ = moe.combine_grad(dout.contiguous(), ctx.order)
        da = torch.cat([drows[i:j] @ w2[e].t().contiguous() for e, (i, j) in spans])
        dw2 = torch.stack([a[i:j].t().contiguous() @ drows[i:j] for _, (i, j) in spans])
        dh1, dw = moe.activate_grad(da, h1, "swiglu", ctx.order, w)
        dxs = torch.cat([dh1[i:j] @ w1[e].t().contiguous() for e, (i, j) in spans])
        dw1 = torch.stack([xs[i:j].t().contiguous() @ dh1[i:j] for _, (i, j) in spans])
        dy, _ = moe.dispatch_grad(dxs, ctx.order)
        dlogits = moe.route_grad(dw, logits, ids)
        dy = dy + dlogits @ wr.t().contiguous()
        dx, dwn = moe.rms_norm_grad(dy, h, wn, dtotal=dh.contiguous())
        return dx, dx, dwn, y.t().contiguous() @ dlogits, dw1, dw2, None


def test_training_run():
    """The gradients of a layer made of the calls, in fp32, against autograd in 64 bits on the
    CPU with the GPU's choice of experts."""
    T, H, I, E, K = 24, 32, 16, 6, 2
    g = rng(30)
    make = [g.standard_normal((T, H)), g.standard_normal((T, H)), g.random(H) + 0.5, g.standard_normal((H, E)) / 4,
            g.standard_normal((E, H, 2 * I)) / 5, g.standard_normal((E, I, H)) / 4]
    mine = [dev(v, torch.float32).requires_grad_(True) for v in make]
    out, h = Layer.apply(*mine, K)
    d_out, d_h = dev(g.standard_normal((T, H)), torch.float32), dev(g.standard_normal((T, H)), torch.float32)
    torch.autograd.backward([out, h], [d_out, d_h])
    x, res, wn, wr, w1, w2 = plain = [v.detach().cpu().double().requires_grad_(True) for v in mine]
    hp = x + res
    y = hp / torch.sqrt((hp * hp).mean(dim=1, keepdim=True) + 1e-6) * wn
    logits = y @ wr
    ids = logits.topk(K, dim=1)[1]
    w = torch.softmax(logits.gather(1, ids), dim=1)
    want = torch.zeros(T, H, dtype=torch.float64)
    for k in range(K):
        z = torch.bmm(y[:, None], w1[ids[:, k]])[:, 0]
        a = torch.nn.functional.silu(z[:, :I]) * z[:, I:] * w[:, k:k + 1]
        want = want + torch.bmm(a[:, None], w2[ids[:, k]])[:, 0]
    torch.autograd.backward([want, hp], [d_out.cpu().double(), d_h.cpu().double()])
    # chains of a few hundred roundings of terms that are at most 100 times the largest result
    for got, right, name in [(out, want, "out")] + [(m.grad, p.grad, i) for i, (m, p) in enumerate(zip(mine, plain))]:
        right = right.detach().numpy()
        assert np.abs(f64(got) - right).max() <= 300 * 100 * U32 * np.abs(right).max(), name


# ---------------------------------------------------------------------------
# streams, graphs, repeated calls
# ---------------------------------------------------------------------------
def every_call(seed):
    """One call of each operator on its own inputs: a list of (function, inputs)."""
    g = rng(seed)
    T, H, E, K, I, n, r, N = 45, 520, 24, 3, 136, 5, 24, 200
    f = lambda *s: dev(g.standard_normal(s), torch.bfloat16)  # noqa: E731
    logits, bias = dev(g.standard_normal((T, E)), torch.float32), dev(g.standard_normal(E) * 0.1, torch.float32)
    ids, w = moe.route(logits, K)
    order = moe.sort_routes(ids, E)
    wn = dev(g.random(H), torch.float32)
    tokens = moe.sort_routes(dev(g.integers(-1, n, (T, 1)).astype(np.int32)), n)
    return [lambda: moe.route(logits, K, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2),
            lambda: [moe.route_grad(w, logits, ids)],
            lambda x=f(T, H), s=f(T, H): moe.rms_norm(x, wn, residual=s),
            lambda x=f(T, H): moe.rms_norm_int8(x, wn)[:2],
            lambda d=f(T, H), h=f(T, H): moe.rms_norm_grad(d, h, wn),
            lambda h=f(T * K, 2 * I): [moe.activate(h, "swiglu", order, w)],
            lambda h=f(T * K, 2 * I): moe.activate_int8(h, "swiglu", order),
            lambda d=f(T * K, I), h=f(T * K, 2 * I): moe.activate_grad(d, h, "swiglu", order, w),
            lambda y=f(T, N), x=f(T, H - 8), a=f(n, r, H - 8), b=f(n, N, r): [moe.adapt(y, x, tokens, a, b)]]


def test_graph_replays():
    calls = every_call(1)
    want = [[v.clone() for v in c()] for c in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls]
    for _ in range(3):
        for vs in got:
            for v in vs:
                v.fill_(0) if v.dtype != torch.int8 else v.zero_()
        graph.replay()
        eager = [c() for c in calls]  # between the replays, on workspaces of their own
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, eager):
            for x, y, z in zip(a, b, c):
                assert torch.equal(x, y) and torch.equal(z, y)


def test_two_streams_at_once():
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    left, right = every_call(2), every_call(3)
    want = [[[v.clone() for v in c()] for c in side] for side in (left, right)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for a, b in zip(left, right):
            with torch.cuda.stream(one):
                got[0].append(a())
            with torch.cuda.stream(two):
                got[1].append(b())
    torch.cuda.synchronize()
    for side in (0, 1):
        for i, vs in enumerate(got[side]):
            assert all(torch.equal(x, y) for x, y in zip(vs, want[side][i % len(left)]))


def test_stream_argument():
    s = torch.cuda.Stream()
    x = torch.randn(33, 264, device=DEV)
    torch.cuda.synchronize()
    y, _ = moe.rms_norm(x, stream=s)
    ids, w = moe.route(x, 4, stream=s)
    a = moe.activate(x, stream=s)
    d = moe.route_grad(w, x, ids, stream=s)
    s.synchronize()
    assert torch.equal(y, moe.rms_norm(x)[0]) and torch.equal(a, moe.activate(x))
    assert torch.equal(ids, moe.route(x, 4)[0]) and torch.equal(d, moe.route_grad(w, x, ids))


def test_damaged_maps_stay_in_range():
    """Entries that name no route, token or row, and offsets that go back or beyond: nothing
    outside the buffers is written (guards on both sides)."""
    T, K, E, I, H, N = 50, 2, 6, 72, 64, 90
    R = T * K
    order, r2r, _, kept = sorted_routes(7, T, K, E, True)
    h, w = torch.randn(R, 2 * I, device=DEV), torch.rand(T, K, device=DEV)
    bad = order.row_to_route.clone()
    bad[3], bad[5] = 1 << 30, -7
    rt2 = order.route_to_row.clone()
    rt2[0] = 1 << 30
    for off in (order.offsets, torch.tensor([0, 40, 10, 1 << 30, -5, 20, 1 << 20], dtype=torch.int32, device=DEV)):
        o = moe.RouteOrder(bad, rt2, off, T, K, E)
        guard = torch.full((R + 2, I), 7.0, device=DEV)
        moe.activate(h, "swiglu", o, w, out=guard[1:-1])
        assert (guard[0] == 7).all() and (guard[-1] == 7).all() and (guard[4] == 7).all() and (guard[6] == 7).all()
        moe.activate_int8(h, "swiglu", o, w)
        moe.activate_grad(guard[1:-1].clone(), h, "swiglu", o, w)
    ids = dev((np.arange(T) % E)[:, None].astype(np.int32))
    order = moe.sort_routes(ids, E)
    bad, rt2 = order.row_to_route.clone(), order.route_to_row.clone()
    bad[4], bad[9], rt2[6] = 1 << 30, -1, 1 << 30
    x, base = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T, N, device=DEV).bfloat16()
    a, b = torch.randn(E, 8, H, device=DEV).bfloat16(), torch.randn(E, N, 8, device=DEV).bfloat16()
    for off in (order.offsets, torch.tensor([0, 40, 10, 1 << 30, -5, 20, 1 << 20], dtype=torch.int32, device=DEV)):
        guard = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
        moe.adapt(base, x, moe.RouteOrder(bad, rt2, off, T, 1, E), a, b, out=guard[1:-1])
        assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    torch.cuda.synchronize()


def test_far_rows():
    """Rows more than 2^31 elements apart."""
    big = torch.empty((1 << 31) + (1 << 22), dtype=torch.bfloat16, device=DEV)
    far = big.as_strided((2, 520), ((1 << 31) + 8, 1))
    far.copy_(torch.randn(2, 520, device=DEV))
    near = far.contiguous()
    assert torch.equal(moe.rms_norm(far)[0], moe.rms_norm(near)[0])
    assert torch.equal(moe.activate(far), moe.activate(near))
    assert torch.equal(moe.route(far, 4)[0], moe.route(near, 4)[0])
    out = big.as_strided((2, 520), ((1 << 31) + 8, 1), 1024)
    moe.rms_norm_grad(near, near, out=out)
    assert torch.equal(out.contiguous(), moe.rms_norm_grad(near, near)[0])
    a, b = torch.randn(1, 8, 512, device=DEV).bfloat16(), torch.randn(1, 520, 8, device=DEV).bfloat16()
    one = moe.sort_routes(torch.zeros(2, 1, dtype=torch.int32, device=DEV), 1)
    assert torch.equal(moe.adapt(far, far[:, :512], one, a, b), moe.adapt(near, near[:, :512], one, a, b))
    # tokens' rows just below and above 4 GiB in all
    x, base = torch.randn(2048, 64, device=DEV).bfloat16(), torch.randn(2048, 40, device=DEV).bfloat16()
    a, b = torch.randn(1, 8, 64, device=DEV).bfloat16(), torch.randn(1, 40, 8, device=DEV).bfloat16()
    one = moe.sort_routes(torch.zeros(2048, 1, dtype=torch.int32, device=DEV), 1)
    for stride in (1 << 20, (1 << 20) + 1024):
        far = big.as_strided((2048, 64), (stride, 1))
        far.copy_(x)
        # (the two kernels sum in different orders: each within its bound of the other's middle)
        got, want = moe.adapt(base, far, one, a, b), moe.adapt(base, x, one, a, b)
        assert torch.equal(got, want) if stride == 1 << 20 else ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -10).all()
