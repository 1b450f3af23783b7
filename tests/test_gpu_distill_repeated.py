"""distill_loss on lists with tokens listed many times: which entry stands for
the token's q goes by the list, so that every call gives the same bits."""
import pytest

from tests.harness import log
from tests.test_gpu_distill import check, teacher
from tests.test_gpu_top import _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k,of", [(70, 60, 9), (5001, 1024, 100), (128256, 300, 3)])
def test_every_call_gives_the_same_bits(V, k, of, dtype):
    import torch

    from rejection_sampling_verify_09_amd import distill_loss

    log(f"[distill] repeated V={V} k={k} of {of} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x, index, values, lse = teacher(40, V, k, dtype, 1.0, g)
    at = torch.randint(0, of, (40, k), device="cuda", generator=g)
    index = index.gather(1, at).contiguous()
    values = (values.gather(1, at) - torch.rand((40, k), device="cuda", generator=g) * 4).contiguous()
    want = check(x, index, values, None)
    for _ in range(20):
        got = distill_loss(x, index, values, with_grad=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
