"""distill_loss on students masked by large finite values: here and there, at
the front (a thread's first run, which its sums are relative to), at the end,
but for a few tokens, but for the list, and altogether."""
import numpy as np
import pytest

from oracle import fine_tune as ref
from tests.harness import log
from tests.test_gpu_distill import check, teacher
from tests.test_gpu_top import _t

pytestmark = pytest.mark.gpu


def check_range(x, index, values, lse, T):
    """check, where a loss may lie past float32: what is at or above 2^128 - 2^103 rounds to infinity.  Such rows are
    checked with 1 / 16 of the weight, which takes no digits."""
    import torch

    from rejection_sampling_verify_09_amd import distill_loss

    idx, val = index.cpu().numpy(), values.cpu().numpy().astype(np.float64)
    xs, ls = x.float().cpu().numpy().astype(np.float64), [None] * len(idx) if lse is None else lse.cpu().numpy()
    want = np.array([ref.distill_row(xs[r], idx[r], val[r], ls[r], T)[0] for r in range(len(idx))])
    past = np.isfinite(want) & (np.abs(want) >= 2.0 ** 128 - 2.0 ** 103)
    check(x, index, values, lse, T, rows=np.flatnonzero(~past))
    if past.any():
        loss = distill_loss(x, index, values, top_lse=lse, temperature=T)[0].cpu().numpy()
        assert np.array_equal(loss[past], np.sign(want[past]) * np.inf)
        check(x, index, values, lse, T, weight=torch.full((len(idx),), 2.0 ** -4, device="cuda"))


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e20, -1e30, "lowest"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(66, 16), (5001, 64), (128256, 64), (300001, 100)])
def test_masked_tokens(V, k, dtype, mask):
    import torch

    log(f"[distill] masked V={V} k={k} {dtype} mask={mask}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V + k)
    m = torch.finfo(_t(dtype)).min if mask == "lowest" else mask
    x, index, values, lse = teacher(8, V, k, dtype, 1.0, g)
    listed = torch.zeros((8, V), device="cuda", dtype=torch.bool).scatter_(1, index.long(), True)
    x[0] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, x[0], m)
    x[1, :V // 2] = m
    x[2, V // 2:] = m
    x[3] = torch.where(torch.rand(V, device="cuda", generator=g) < 20 / V, x[3], m)
    x[4] = torch.where(listed[4], x[4], m)
    x[5] = m
    x[6] = torch.where(torch.arange(V, device="cuda") // 64 % 2 == 0, m, x[6])
    x[7, :9] = m
    for T in (1.0, 2.0):
        check_range(x, index, values, None, T)
        check_range(x, index, values, (lse / T).contiguous(), T)
