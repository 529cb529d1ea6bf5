"""The operators around the experts at their edges, on the GPU: scales near the ends
of fp32, offsets that go back, blocks that walk several tiles, rows far apart, calls
from several host threads, gradients joined to autograd's."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_top_amd as moe  # noqa: E402
from tests import expert_ops_ref as ref  # noqa: E402
from tests.expert_ops_ref import HALF, TINY, U32, assert_within, f64, stored  # noqa: E402

DEV = "cuda"
MAX32 = float(np.finfo(np.float32).max)


def say(*a):
    print(*a, flush=True)


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------------------
# scales near the ends of fp32
# ---------------------------------------------------------------------------
# powers of two, so that a product is either far below the largest fp32 or far above
SCALES = np.array([2.0 ** -149, -5 * 2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 2.0 ** -100, -2.0 ** -60, 2.0 ** -20, 1.0, -2.0 ** 20,
                   2.0 ** 60, 2.0 ** 96, -2.0 ** 97, 2.0 ** 97 * 1.5, 2.0 ** 110, 2.0 ** 127, 0.0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,E", [(5, 70, 80, 0), (300, 2601, 144, 0), (999, 3601, 80, 0), (4000, 3702, 16, 0),
                                     (37, 96, 64, 5), (500, 2050, 80, 7)])
def test_scales_at_the_ends_of_fp32(M, N, K, E, dtype):
    """Where one scale alone takes the sum out of fp32 and the other brings it back, the
    result is the finite value; infinite only where it is. The roundings are the ones of
    ordinary scales: the sum to fp32, the first product, the fma (and the subnormals'
    half step, which `stored` counts)."""
    say("scales", M, N, K, E, dtype)
    g = np.random.default_rng(M + N)
    a = g.integers(-128, 128, (M, K)).astype(np.int8)
    b = g.integers(-128, 128, (max(E, 1), N, K)).astype(np.int8)
    a[::7] = 0  # sums of 0 and of 1: 0 times anything finite is 0
    a[1::7], b[:, ::5] = 0, np.sign(b[:, ::5])
    a[1::7, 3] = 1
    sa = g.choice(SCALES, M).astype(np.float32)
    sb = g.choice(SCALES, (max(E, 1), N)).astype(np.float32)
    bias = (g.standard_normal((max(E, 1), N)) * 2.0 ** g.integers(-120, 120, (max(E, 1), N))).astype(np.float32)
    if E:
        o = moe.sort_routes(dev(g.integers(0, E, (M, 1)).astype(np.int32)), E)
        off, route = o.offsets.cpu().numpy(), o.row_to_route.cpu().numpy()
        expert = np.searchsorted(off, np.arange(M), side="right") - 1
    for with_bias in (False, True):
        if E:
            got = moe.int8_grouped_matmul(dev(a), dev(sa), dev(b), dev(sb), o, gather=True,
                                          bias=dev(bias) if with_bias else None, out_dtype=dtype)
            want, bound = np.zeros((M, N)), np.zeros((M, N))
            for e in range(E):
                at = np.nonzero(expert == e)[0]
                want[at], bound[at] = ref.matmul(a[route[at]], f64(dev(sa))[route[at]], b[e], sb[e].astype(np.float64),
                                                 bias[e].astype(np.float64) if with_bias else None)
        else:
            got = moe.int8_matmul(dev(a), dev(sa), dev(b[0]), dev(sb[0]), dev(bias[0]) if with_bias else None, out_dtype=dtype)
            want, bound = ref.matmul(a, sa.astype(np.float64), b[0], sb[0].astype(np.float64),
                                     bias[0].astype(np.float64) if with_bias else None)
        got = f64(got)
        over = np.abs(want) > MAX32 * (1 + 2.0 ** -7)
        sure = np.abs(want) < MAX32 * (1 - 2.0 ** -7)  # between the two the rounding decides
        assert bool((over | sure).mean() > 0.99) and (bool(over.any()) or M < 37)
        assert np.array_equal(got[over], np.copysign(np.inf, want[over])), "overflow"
        assert_within(torch.as_tensor(got[sure]), want[sure], stored(bound, want, dtype)[sure], f"bias={with_bias}")


# ---------------------------------------------------------------------------
# offsets that go back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N", [8, 1300, 2050, 9000])  # narrow tiles, 64x128, 128x256 twice
def test_offsets_that_go_back(N, gather):
    """Every second expert claims all rows, which makes more tiles than an ascending list
    can have. All experts hold the same matrix, so whichever writes a row, it is right;
    nothing outside the rows is touched."""
    say("offsets that go back", N, gather)
    M, E, D = 600, 40, 80
    g = torch.Generator(device=DEV).manual_seed(N)
    a = torch.randint(-127, 128, (M, D), dtype=torch.int8, device=DEV, generator=g)
    b = torch.randint(-127, 128, (N, D), dtype=torch.int8, device=DEV, generator=g)
    off = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    rows = torch.arange(M, dtype=torch.int32, device=DEV)
    order = moe.RouteOrder(rows, rows, off, M, 1, E)
    around = torch.full((M + 2, N + 4), 5.0, device=DEV)
    one = torch.ones(1, device=DEV)
    moe.int8_grouped_matmul(a, one.expand(M).contiguous(), b.expand(E, N, D), one.expand(E, N).contiguous(), order,
                            gather=gather, out=around[1:-1, 2:-2])
    want = (a.double() @ b.double().t().contiguous()).float()
    assert torch.equal(around[1:-1, 2:-2], want)
    around[1:-1, 2:-2] = 5
    assert bool((around == 5).all())


# ---------------------------------------------------------------------------
# blocks that walk several tiles
# ---------------------------------------------------------------------------
def gpu_rand(g, *shape):
    return torch.randint(-128, 128, shape, dtype=torch.int8, device=DEV, generator=g)


def gpu_scale(g, *shape):
    return torch.rand(shape, device=DEV, generator=g) * 0.02 + 0.005


def product(a, sa, b, sb, bias):
    """(y, bound) in 64 bits on the GPU: three roundings of the scaled sum, one of the bias."""
    y = a.double() @ b.double().t().contiguous() * sa.double()[:, None] * sb.double()
    bound = 3.01 * U32 * y.abs()
    y = y + bias.double()
    return y, bound + U32 * y.abs()


def within(got, y, bound, dtype):
    return bool(((got.double() - y).abs() <= bound + (y.abs() + bound) * HALF[dtype] + TINY[dtype]).all())


# On 256 CUs: 3 x 110 tiles of 64x128, 3 x 140 of 128x128, 2 x 301 of 128x256, 20 x 31 of
# 256x256, each with ragged rows and columns; depths with a cut last step, shorter than
# the buffers and longer.
WALKS = [(190, 14001, 80), (190, 14001, 1104), (299, 17900, 400), (299, 17900, 1040), (150, 77003, 48), (150, 77003, 656),
         (4999, 7901, 80), (4999, 7901, 528)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", WALKS)
def test_dense_blocks_that_walk_several_tiles(M, N, K, dtype):
    """Every block takes the next tile's rows, scales and bias over while it stores."""
    say("walk", M, N, K, dtype)
    g = torch.Generator(device=DEV).manual_seed(M + K)
    a, b, sa, sb = gpu_rand(g, M, K), gpu_rand(g, N, K), gpu_scale(g, M), gpu_scale(g, N)
    bias = torch.randn(N, device=DEV, generator=g) * 30
    y, bound = product(a, sa, b, sb, bias)
    assert within(moe.int8_matmul(a, sa, b, sb, bias, out_dtype=dtype), y, bound, dtype)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,K,N,D,E", [(3000, 4, 3411, 272, 24), (3000, 4, 3411, 1040, 24), (1500, 4, 4101, 144, 40),
                                       (470, 1, 1601, 208, 16)])  # 256x256, 128x256, 64x128
def test_grouped_blocks_that_walk_several_tiles(T, K, N, D, E, gather):
    """Experts of very unequal sizes, some empty, a fifth of the routes dropped: from tile
    to tile a block's expert and the number of its rows change."""
    say("grouped walk", T, K, N, D, E, gather)
    g = torch.Generator(device=DEV).manual_seed(T + D)
    share = torch.rand(E + 1, device=DEV, generator=g) ** 3
    share[3], share[E] = 0, share[:E].sum() / 4
    ids = torch.multinomial(share, T * K, replacement=True, generator=g).view(T, K)
    o = moe.sort_routes(ids, E)
    off = o.offsets.tolist()
    n = T if gather else T * K
    a, sa, b, sb = gpu_rand(g, n, D), gpu_scale(g, n), gpu_rand(g, E, N, D), gpu_scale(g, E, N)
    bias = torch.randn(E, N, device=DEV, generator=g) * 30
    out = torch.full((T * K, N), 7.0, device=DEV)
    moe.int8_grouped_matmul(a, sa, b, sb, o, gather=gather, bias=bias, out=out)
    for e in range(E):
        at = slice(off[e], off[e + 1])
        src = o.row_to_route[at].long() // K if gather else at
        y, bound = product(a[src], sa[src], b[e], sb[e], bias[e])
        assert within(out[at], y, bound, torch.float32), e
    assert bool((out[off[E]:] == 7).all())


# ---------------------------------------------------------------------------
# rows far apart
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N", [(5, 70), (300, 2601), (3999, 3701)])  # narrow, 128x128 and 256x256 tiles
def test_rows_at_the_greatest_stride(M, N):
    """Rows of A and of B 2^23 bytes apart: offsets inside a tile of 256 rows reach 2^31."""
    say("far rows", M, N)
    K, far = 272, 1 << 23
    g = torch.Generator(device=DEV).manual_seed(N)
    a, b = (torch.empty(n, far, dtype=torch.int8, device=DEV)[:, :K] for n in (M, N))
    a.copy_(gpu_rand(g, M, K))
    b.copy_(gpu_rand(g, N, K))
    sa, sb = gpu_scale(g, M), gpu_scale(g, N)
    near = moe.int8_matmul(a.contiguous(), sa, b.contiguous(), sb, out_dtype=torch.float32)
    assert torch.equal(moe.int8_matmul(a, sa, b, sb, out_dtype=torch.float32), near)
    y, bound = product(a, sa, b, sb, torch.zeros(N, device=DEV))
    assert within(near, y, bound, torch.float32)


@pytest.mark.parametrize("N", [40, 2600])
def test_gathered_rows_at_the_greatest_stride(N):
    """511 gathered tokens 2^23 bytes apart: just below the 4 GiB of one buffer."""
    say("far gathered rows", N)
    T, K, E, D, far = 511, 2, 6, 96, 1 << 23
    g = torch.Generator(device=DEV).manual_seed(N)
    a = torch.empty(T, far, dtype=torch.int8, device=DEV)[:, :D]
    a.copy_(gpu_rand(g, T, D))
    sa, b, sb = gpu_scale(g, T), gpu_rand(g, E, N, D), gpu_scale(g, E, N)
    o = moe.sort_routes(torch.randint(0, E, (T, K), device=DEV, generator=g), E)
    got = moe.int8_grouped_matmul(a, sa, b, sb, o, gather=True)
    assert torch.equal(got, moe.int8_grouped_matmul(a.contiguous(), sa, b, sb, o, gather=True))
    off = o.offsets.tolist()
    for e in range(E):
        src = o.row_to_route[off[e]:off[e + 1]].long() // K
        y, bound = product(a[src], sa[src], b[e], sb[e], torch.zeros(N, device=DEV))
        assert within(got[off[e]:off[e + 1]], y, bound, torch.bfloat16)


# ---------------------------------------------------------------------------
# several host threads
# ---------------------------------------------------------------------------
def test_host_threads():
    """Four threads on streams of their own, each with its own sizes; every result equals
    the one of a single thread, and a refusal's message is its own thread's."""
    def chain(i):
        T, K, E, H, N = 60 + 40 * i, 1 + i, 5 + i, 128 + 16 * i, 200 + 300 * i
        g = torch.Generator(device=DEV).manual_seed(i)
        x = torch.randn(T, H, device=DEV, generator=g, dtype=torch.bfloat16)
        ids = torch.randint(0, E + 1, (T, K), device=DEV, generator=g)
        w = torch.rand(T, K, device=DEV, generator=g)
        o = moe.sort_routes(ids, E)
        q, s = moe.quantize_int8(x)
        b, sb = gpu_rand(g, E, N, H), gpu_scale(g, E, N)
        rows = torch.zeros(T * K, N, dtype=torch.bfloat16, device=DEV)
        moe.int8_grouped_matmul(q, s, b, sb, o, gather=True, out=rows)
        y = moe.combine(rows, o, w)
        drows, dw = moe.combine_grad(y, o, rows, w, out=torch.zeros_like(rows))
        with pytest.raises(moe.MoeError, match=f"K={8 * (2 * i + 1)} must be a multiple of 16"):
            odd = 8 * (2 * i + 1)
            one = torch.ones(2, 16 * (2 * i + 1), dtype=torch.int8, device=DEV)[:, :odd]
            moe.int8_matmul(one, torch.ones(2, device=DEV), one, torch.ones(2, device=DEV))
        return [v.cpu() for v in (y, drows, dw)]
    want = [chain(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    if not all(torch.equal(u, v) for u, v in zip(chain(i), want[i])):
                        wrong.append(i)
        except BaseException as e:  # (an assertion in a thread is not the test's otherwise)
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---------------------------------------------------------------------------
# gradients joined to autograd's
# ---------------------------------------------------------------------------
class Experts(torch.autograd.Function):
    """dispatch, experts that scale their rows, combine, as a user wraps them."""
    @staticmethod
    def forward(ctx, x, w, factor, order):
        rows = moe.dispatch(x, order) * factor
        ctx.save_for_backward(rows, w, factor)
        ctx.order = order
        return moe.combine(rows, order, w)

    @staticmethod
    def backward(ctx, dy):
        rows, w, factor = ctx.saved_tensors
        drows, dw = moe.combine_grad(dy.contiguous(), ctx.order, rows, w)
        dx, _ = moe.dispatch_grad(drows * factor, ctx.order)
        return dx, dw, None, None


@pytest.mark.parametrize("wrapped", [False, True])
def test_gradients_joined_to_autograd(wrapped):
    """Results carry no gradient by themselves. Their gradients go back into autograd's
    graph by torch.autograd.backward, or by a Function around the calls."""
    T, K, E, H = 40, 3, 7, 24
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(T, H, device=DEV, generator=g, requires_grad=True)
    logits = torch.randn(T, E, device=DEV, generator=g, requires_grad=True)
    dy = torch.randn(T, H, device=DEV, generator=g)
    ids = logits.detach().topk(K, dim=1).indices
    w = torch.softmax(logits.gather(1, ids), dim=1)
    o = moe.sort_routes(ids, E)  # no route is dropped: every row is written
    expert = torch.searchsorted(o.offsets, torch.arange(T * K, device=DEV, dtype=torch.int32), right=True) - 1
    factor = (1.0 + expert.float())[:, None]  # 1 .. 7: exact
    if wrapped:
        y = Experts.apply(x, w, factor, o)
        y.backward(dy)
    else:
        rows = moe.dispatch(x, o) * factor
        y = moe.combine(rows, o, w)
        assert not rows.requires_grad and not y.requires_grad
        drows, dw = moe.combine_grad(dy, o, rows, w)
        dx, _ = moe.dispatch_grad(drows * factor, o)
        torch.autograd.backward([x, w], [dx, dw])
    X, L, I = x.detach().cpu().double().requires_grad_(), logits.detach().cpu().double().requires_grad_(), ids.cpu()
    W = torch.softmax(L.gather(1, I), dim=1)
    c = W * (1 + I.double())
    Y = c.sum(1, keepdim=True) * X
    Y.backward(dy.cpu().double())
    aX, aD, aW = X.detach().abs(), dy.cpu().double().abs(), W.detach()
    mag_w = (1 + I.double()) * (aX * aD).sum(1, keepdim=True)          # of dw
    mag_l = torch.zeros(T, E, dtype=torch.float64).scatter_(1, I, aW * (mag_w + (aW * mag_w).sum(1, keepdim=True)))
    # w itself is within 16 roundings (the difference to the largest logit of up to 8
    # magnitudes, exp, sum, quotient); then the products and sums of K, H or E terms
    assert_within(y.detach(), Y.detach().numpy(), (K + 24) * U32 * (c.detach().sum(1, keepdim=True) * aX).numpy(), "y")
    assert_within(x.grad, X.grad.numpy(), (K + 24) * U32 * (c.detach().sum(1, keepdim=True) * aD).numpy(), "dx")
    assert_within(logits.grad, L.grad.numpy(), (H + 2 * K + 48) * U32 * mag_l.numpy(), "dlogits")
