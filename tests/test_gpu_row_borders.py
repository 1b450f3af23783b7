"""top_logits and distill_loss on rows around the border of the running sum's
reference (logits times log2(e) / T at -2^31, where a float32's steps are 128 and
256) and on rows with logits as far above 0."""
import numpy as np
import pytest

from tests.harness import log
from tests.test_gpu_distill import check as check_loss
from tests.test_gpu_distill import teacher
from tests.test_gpu_top import _t, check

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def border_rows(V, T, dtype, g):
    """Rows of values on both sides of the border, a few steps of their type apart; one of each alone; ordinary ones
    among them."""
    import torch

    at = -2.0 ** 31 * T / LOG2E
    eps = torch.finfo(_t(dtype)).eps
    steps = torch.randint(-3, 4, (8, V), device="cuda", generator=g).double()
    x = (at * (1 + eps * steps)).to(_t(dtype))
    for r, s in ((1, -3), (2, -1), (3, 0), (4, 1), (5, 3)):
        x[r] = at * (1 + eps * s)
    x[6, V // 2:] = (torch.randn((V - V // 2,), device="cuda", generator=g) * T).to(_t(dtype))
    x[7, V // 3] = 0.5 * T
    return x


@pytest.mark.parametrize("T", [1e-9, 0.37, 1.0, 2.9, 1e9])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(5, 3), (513, 20), (5001, 64), (128256, 300)])
def test_rows_at_the_border(V, k, dtype, T):
    import torch

    log(f"[borders] V={V} k={k} {dtype} T={T}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = border_rows(V, T, dtype, g)
    check(x, k, float(np.float32(T)))
    _, index, values, lse = teacher(8, V, k, dtype, 1.0, g)
    values = values * T
    check_loss(x, index, values, lse, T)
    check_loss(x, index, values, None, T)


@pytest.mark.parametrize("large", [1e9, 1e10, 1e20, 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(66, 16), (5001, 64), (128256, 64), (200000, 1000)])
def test_large_logits(V, k, dtype, large):
    import torch

    log(f"[borders] large={large} V={V} k={k} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x, index, values, lse = teacher(5, V, k, dtype, 1.0, g)
    x[0, V // 2] = large
    x[1, ::3] = large
    x[2] = x[2] * (large / 20)
    x[3, :9] = large
    x[3, -9:] = -large
    x[4] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, large, -large)
    for T in (1.0, 2.0):
        check(x, k, T)
        check_loss(x, index, values * 2 ** -7, None, T, weight=torch.full((5,), 2.0 ** -7, device="cuda"))
