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
