"""distill_loss where the teacher or the student holds NaN: the loss and all of
the row's gradient are NaN, and the other rows are as without it."""
import math

import pytest

from tests.harness import log
from tests.test_gpu_distill import teacher
from tests.test_gpu_top import _t

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), math.inf


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(5, 3), (70, 12), (5001, 64), (128256, 130), (300001, 33)])
def test_nan_is_not_swallowed(V, k, dtype, rest):
    import torch

    from rejection_sampling_verify_09_amd import distill_loss

    log(f"[distill] NaN V={V} k={k} {dtype} rest={rest}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    rows = 16
    x, index, values, lse = teacher(rows, V, k, dtype, 1.0, g)
    listed = torch.zeros((rows, V), device="cuda", dtype=torch.bool).scatter_(1, index.long(), True)
    want = distill_loss(x, index, values, top_lse=lse if rest else None, with_grad=True)
    bad = [0, 2, 4, 6, 8, 10]
    values[0, k // 2] = NAN
    values[2, 1] = INF
    lse[2] = INF
    values[4, 0] = -torch.tensor(NAN)
    values[4, 1:] = -INF
    x[6] = torch.where(listed[6], x[6], -INF)      # nothing but the list, and NaN there
    x[6, index[6, 1].long()] = NAN
    x[8] = torch.where(listed[8], x[8], -INF)
    x[8, index[8, 0].long()] = INF
    x[10] = NAN
    if rest:
        bad += [12, 14]
        lse[12] = NAN
        lse[14] = NAN                              # and a list without tokens
        index[14] = -1
    for kw in (dict(), dict(with_loss=False)):
        loss, grad = distill_loss(x, index, values, top_lse=lse if rest else None, with_grad=True, **kw)
        assert torch.isnan(grad[bad]).all()
        assert loss is None or torch.isnan(loss[bad]).all()
        assert torch.equal(grad[1::2], want[1][1::2]) and (loss is None or torch.equal(loss[1::2], want[0][1::2]))
    loss, _ = distill_loss(x, index, values, top_lse=lse if rest else None)
    assert torch.isnan(loss[bad]).all() and torch.equal(loss[1::2], want[0][1::2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_target_with_nan_gives_a_teacher_with_nan(dtype):
    """top_logits puts NaN first and its log-sum-exp is NaN: distill_loss of that is NaN throughout."""
    import torch

    from rejection_sampling_verify_09_amd import distill_loss, top_logits

    t = torch.randn((2, 3000), device="cuda").to(_t(dtype))
    t[1, 77] = NAN
    values, index, lse = top_logits(t, 9)
    x = torch.randn((2, 3000), device="cuda").to(_t(dtype))
    for rest in (lse, None):
        loss, grad = distill_loss(x, index, values, top_lse=rest, with_grad=True)
        assert torch.isnan(loss[1]) and torch.isnan(grad[1]).all() and torch.isfinite(loss[0]) and torch.isfinite(grad[0]).all()
