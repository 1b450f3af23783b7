"""linear sums in float32 whatever its operands' and its output's types:
products that differ by all that e4m3 can hold, in one run of k, where large
ones cancel and the small ones are the result.

Exact sums: the elements are small multiples of 2^-3, but for one pair of
448 x 448 and 448 x -448.  Products are then multiples of 2^-6 and any partial
sum, in any order, is below 448^2 + K 49 / 64 < 2^18 for K <= 4096: 24 bits
hold each of them, so that the result is the exact sum, rounded once.  Others
are held to the bound of K float32 additions in any order, gamma_K sum |x w|
with u = 2^-24, and the output's half step."""
import numpy as np
import pytest

from oracle import last_layer as ref
from tests.harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SHAPES = [(1, 300, 64), (1, 700, 4096), (7, 9000, 128), (16, 500, 4096), (40, 300, 192), (64, 1024, 576),
          (130, 1000, 4096), (200, 6000, 64), (300, 700, 320), (440, 30001, 64), (448, 2100, 1024)]


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def scales(dtype, M, N):
    import torch

    return {} if dtype == "bf16" else dict(x_scale=torch.ones(M, device="cuda"), weight_scale=torch.ones(N, device="cuda"))


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_what_large_products_leave_when_they_cancel(M, N, K, dtype, odt):
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    log(f"[linear sums] M={M} N={N} K={K} {dtype} -> {odt}")
    x = torch.randint(-7, 8, (M, K), device="cuda", generator=g).float() / 8
    w = torch.randint(-7, 8, (N, K), device="cuda", generator=g).float() / 8
    at = K // 2 + 2  # the pair: two neighbours of one run of eight
    x[:, at:at + 2] = 0
    want = (x.cpu() @ w.cpu().T).to(_t(odt))  # exact before the rounding
    x[:, at:at + 2] = 448.0
    w[:, at], w[:, at + 1] = 448.0, -448.0
    got = linear(x.to(_t(dtype)), w.to(_t(dtype)), out_dtype=_t(odt), **scales(dtype, M, N)).cpu()
    bad = (got != want).nonzero()
    assert bad.numel() == 0, (len(bad), got[tuple(bad[0])].item(), want[tuple(bad[0])].item())


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (40, 700, 512), (130, 1000, 4096), (448, 2100, 1024)])
@pytest.mark.parametrize("kind", ["outliers", "halves that cancel"])
def test_unlike_magnitudes_stay_within_the_float32_bound(kind, M, N, K, dtype, odt):
    """Columns of x 60 times the others; then a second half of x that is the first, under weights that nearly cancel it."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M * 3 + N + K)
    log(f"[linear sums] {kind} M={M} N={N} K={K} {dtype} -> {odt}")
    x = torch.randn((M, K), device="cuda", generator=g)
    w = torch.randn((N, K), device="cuda", generator=g)
    if kind == "outliers":
        x[:, ::97] *= 60
    else:
        x[:, K // 2:] = x[:, :K // 2]
        w[:, K // 2:] = w[:, K // 2:] / 8 - w[:, :K // 2]
    x = (x / x.abs().amax(1, keepdim=True) * 448).clamp(-448, 448).to(_t(dtype))
    w = (w / w.abs().amax(1, keepdim=True) * 448).clamp(-448, 448).to(_t(dtype))
    want = ref.linear(np64(x), np64(w))
    bound = ((K + 4) * U / (1 - K * U)) * (np.abs(np64(x)) @ np.abs(np64(w)).T)
    got = np64(linear(x, w, out_dtype=_t(odt), **scales(dtype, M, N)))
    err = np.abs(got - want)
    log(f"   relative {np.linalg.norm(err) / np.linalg.norm(want):.3g}, worst err / bound {np.max(err / bound):.3g}")
    assert np.all(err <= bound + (2.0 ** -8 * (np.abs(want) + bound) if odt == "bf16" else 0.0))
