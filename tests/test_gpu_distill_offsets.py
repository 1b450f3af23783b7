"""distill_loss where all of a row's logits are large and close to each other,
relative to their magnitude: the divergence is of the order of 1, and what the
logits have in common, 10^20 and more, takes none of its digits."""
import pytest

from tests.harness import log
from tests.test_gpu_distill import check, teacher
from tests.test_gpu_top import _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(5, 5), (70, 12), (5001, 64), (128256, 130)])
def test_one_value(V, k, dtype, rest):
    import torch

    log(f"[distill] one value V={V} k={k} {dtype} rest={rest}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    fi = torch.finfo(_t(dtype))
    at = (-1e9, -1e13, -1e20, 1e20, -1e30, fi.min, fi.max)
    x, index, values, lse = teacher(len(at), V, k, dtype, 1.0, g)
    for r, v in enumerate(at):
        x[r] = v
    loss, _ = check(x, index, values, lse if rest else None)
    # q is 1 / V everywhere: the same loss in all rows of one teacher
    same = lambda t: t[:1].expand(t.shape).contiguous()  # noqa: E731
    loss, _ = check(x, same(index), same(values), same(lse) if rest else None)
    assert (loss > 0).all() and (loss - loss[0]).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("base,T", [(-1e30, 1e28), (2.0 ** 40, 2.0 ** 35), (-2.0 ** 60, 2.0 ** 55)])
def test_large_logits_at_large_temperatures(base, T, dtype):
    import torch

    log(f"[distill] base={base} T={T} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    _, index, values, lse = teacher(4, 3001, 32, dtype, 1.0, g)
    x = (base * (1 + 0.05 * torch.rand((4, 3001), device="cuda", generator=g))).to(_t(dtype))
    values = values * T
    check(x, index, values, lse, T)
    check(x, index, values, None, T)
