"""The operators around the experts at their edges, on the GPU: scales near the ends
of fp32, and offsets that go back."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_top_amd as moe  # noqa: E402
from tests import expert_ops_ref as ref  # noqa: E402
from tests.expert_ops_ref import assert_within, f64, stored  # noqa: E402

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
