"""distill_loss with teachers that have nothing on their list."""
import math

import pytest

from tests.harness import log
from tests.test_gpu_distill import HALF, check, teacher
from tests.test_gpu_top import _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 300, 5001, 128256, 300001])
def test_a_list_without_tokens_teaches_nothing(V, dtype):
    """The rest is all of the vocabulary: R = r = 1, whatever the log-sum-exp."""
    import torch

    from rejection_sampling_verify_09_amd import distill_loss

    log(f"[distill] no tokens V={V} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    rows, k = 60, 7
    x = (torch.randn((rows, V), device="cuda", generator=g) * 3).to(_t(dtype))
    x[3, 1:] = -1e20
    x[4] = torch.finfo(x.dtype).min
    index = torch.full((rows, k), -1, device="cuda", dtype=torch.int32)
    index[1::2] = V
    values = torch.randn((rows, k), device="cuda", generator=g)
    lse = torch.randn((rows,), device="cuda", generator=g) * 5
    weight = torch.rand((rows,), device="cuda", generator=g) + 0.1
    for T in (1.0, 0.7, 3.0):
        loss, grad = distill_loss(x, index, values, top_lse=lse, temperature=T, weight=weight, with_grad=True)
        assert (loss == 0).all() and (grad == 0).all()
        loss, grad = distill_loss(x, index, values, temperature=T, weight=weight, with_grad=True)
        assert (loss == 0).all() and (grad == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(70, 12), (5001, 64), (128256, 130)])
def test_a_list_of_minus_infinity(V, k, dtype):
    """With a finite log-sum-exp: the rest has all of the mass; without it, or with one of -inf: no teacher."""
    import torch

    log(f"[distill] values of -inf V={V} k={k} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x, index, values, lse = teacher(4, V, k, dtype, 1.0, g)
    values[:2] = -math.inf
    values[2, 1:] = -math.inf
    index[1, ::2] = -1
    loss, grad = check(x, index, values, lse)
    assert (loss[:2] > 0).all()
    loss, grad = check(x, index, values, None)
    assert (loss[:2] == 0).all() and not grad[:2].any()
    loss, grad = check(x, index, values, torch.full_like(lse, -math.inf))
    assert (loss == 0).all() and not grad.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_closed_form(dtype):
    """Three equal logits, one listed without mass: the loss is -log(2/3), the gradient [-1/6, 1/3, -1/6].  Within the
    roundings: of the sum of three exponentials (4 of 2^-24) and of the result (half a step of its type)."""
    import torch

    from rejection_sampling_verify_09_amd import distill_loss

    x = torch.zeros((1, 3), device="cuda", dtype=_t(dtype))
    loss, grad = distill_loss(x, torch.tensor([[1]], device="cuda", dtype=torch.int32),
                              torch.tensor([[-math.inf]], device="cuda"), top_lse=torch.zeros(1, device="cuda"), with_grad=True)
    assert abs(loss.item() - math.log(1.5)) <= 5 * 2.0 ** -24
    want = torch.tensor([-1 / 6, 1 / 3, -1 / 6], dtype=torch.float64)
    assert ((grad[0].double().cpu() - want).abs() <= want.abs() * (HALF[dtype] + 8 * 2.0 ** -24)).all()
