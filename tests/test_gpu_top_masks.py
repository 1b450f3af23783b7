"""top_logits on rows masked by large finite values, whose product with log2(e)
/ T has no digits left for a difference: an exponential of a thread that reads
such a run ahead of ordinary ones overflows, and the thread's maxima are taken
for unknown, as with NaN.  Where many threads are so and the others have few
large logits, no bound from the others' maxima is reached by k logits."""
import numpy as np
import pytest

from tests.harness import log
from tests.test_gpu_top import _t, check

pytestmark = pytest.mark.gpu


def rows(V, run, threads, mask, share, large):
    """Of each `share` threads one has a few `large` logits, and the others a
    run of masked ones ahead of ordinary ones."""
    x = np.full(V, 0.5, np.float32)
    t = np.arange(V) // run % threads
    low = t % share != 0
    x[low] = 1.0
    first = np.arange(V) < threads * run
    x[first & low] = mask
    x[first & ~low & (np.arange(V) % run == run // 2)] = large
    return x


@pytest.mark.parametrize("T", [0.7, 1.0, 1.5, 2.0, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [600, 1000, 1024])
def test_few_large_logits_beside_masked_runs(k, dtype, T):
    import torch

    log(f"[top] masked runs k={k} {dtype} T={T}")
    run = 4 if dtype == "f32" else 8
    lowest = torch.finfo(_t(dtype)).min
    for V in (25000 * run, 25000 * run - 3, 300 * 1024 * run // 8):
        x = np.stack([rows(V, run, 1024, mask, share, large)
                      for mask in (-1e20, -1e30, lowest) for share in (2, 4) for large in (1.5, 10.0)])
        check(torch.from_numpy(x).cuda().to(_t(dtype)), k, T)


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e20, -1e30, "lowest"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(1000, 64), (5000, 300), (24979, 33), (128256, 64), (200000, 1000)])
def test_masked_tokens(V, k, dtype, mask):
    """Masked here and there, at the front, at the end, but for a few tokens, and altogether."""
    import torch

    log(f"[top] masked V={V} k={k} {dtype} mask={mask}")
    g = torch.Generator(device="cuda")
    g.manual_seed(V + k)
    m = torch.finfo(_t(dtype)).min if mask == "lowest" else mask
    x = torch.randn((6, V), device="cuda", generator=g) * 2
    x[0] = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, x[0], m)
    x[1, :V // 2] = m
    x[2, V // 2:] = m
    x[3] = torch.where(torch.rand(V, device="cuda", generator=g) < 20 / V, x[3], m)
    x[4] = m
    x[5] = torch.where(torch.arange(V, device="cuda") // 64 % 2 == 0, m, x[5])
    for T in (1.0, 2.0):
        check(x.to(_t(dtype)), k, T)
