"""GPU parity of linear with the float64 oracle.

Grid inputs (small multiples of powers of two) make every partial sum an
exact float32 number, so the product, the bias and the residual must come out
bit for bit in float32 and correctly rounded in bfloat16.  Other inputs are
held to the bound of K float32 additions in any order, gamma_K sum |x w| with
u = 2^-24.  e4m3 operands with a bfloat16 output go through the 8-bit matrix
instructions, whose inner sums keep fewer bits: they are allowed 2^-10 of sum
|x w| besides the output's half step, and 2^-8 in the 2-norm.  Activations on exact sums: relative
errors of expf (1 ulp), erfcf (16 ulp) and of their rounded arguments, which
an argument z magnifies by |z| (exp) and 2 z^2 + 1 (erfc)."""
import numpy as np
import pytest

from oracle import last_layer as ref
from tests.harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ULP = 2.0 ** -23


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def grid(g, shape, dtype, lim=7):
    """Integers of magnitude at most lim over 8: exact in bfloat16 and e4m3; sums of K <= 65536 products of
    magnitude at most 49 / 64 are multiples of 1 / 64 below 2^22."""
    import torch

    return (torch.randint(-lim, lim + 1, shape, device="cuda", generator=g).float() / 8).to(_t(dtype))


SHAPES = [
    # M, N, K
    (1, 1, 64), (1, 4096, 4096), (2, 33, 128), (3, 1000, 192), (7, 257, 64), (15, 48, 320), (16, 16, 4096),
    (17, 129, 576), (31, 640, 1024), (32, 2000, 256), (33, 65, 448), (48, 515, 2112), (63, 100, 64), (64, 1024, 512),
    (65, 300, 704), (96, 2049, 128), (127, 127, 192), (128, 256, 1088), (129, 513, 64), (200, 1500, 448),
    (256, 511, 320), (257, 1025, 192), (384, 2050, 256), (448, 5001, 128), (1000, 300, 64), (1, 70001, 64),
    (5, 12, 65536), (300, 20, 8192),
]


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_on_the_grid(M, N, K, dtype, odt):
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M * 7 + N * 3 + K)
    log(f"[linear grid] M={M} N={N} K={K} {dtype} -> {odt}")
    x, w = grid(g, (M, K), dtype), grid(g, (N, K), dtype)
    sx = sw = None
    if dtype == "e4m3":
        sx = torch.exp2(torch.randint(-3, 4, (M,), device="cuda", generator=g).float())
        sw = torch.exp2(torch.randint(-3, 4, (N,), device="cuda", generator=g).float())
    heads = 3 if N % 3 == 0 else 1
    for bias, res in ((None, None), (grid(g, (N,), odt), grid(g, (M, N // heads), odt))):
        out = linear(x, w, bias=bias, residual=res, x_scale=sx, weight_scale=sw, out_dtype=_t(odt))
        want = ref.linear(np64(x), np64(w), None if bias is None else np64(bias), None if res is None else np64(res),
                          "none", None if sx is None else np64(sx), None if sw is None else np64(sw))
        want = torch.from_numpy(want).to(_t(odt))
        got = out.cpu()
        bad = (got != want).nonzero()
        assert bad.numel() == 0, (len(bad), bad[:3].tolist(), got[tuple(bad[0])].item(), want[tuple(bad[0])].item())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (40, 700, 8192), (130, 1000, 4096), (300, 400, 2112)])
def test_within_the_float32_bound(M, N, K, dtype):
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    x = torch.randn((M, K), device="cuda", generator=g)
    w = torch.randn((N, K), device="cuda", generator=g)
    sx = sw = None
    a = 1.0
    if dtype == "e4m3":
        sx, sw = torch.rand((M,), device="cuda") + 0.01, torch.rand((N,), device="cuda") + 0.01
        x, w = x * 100, w * 100
        a = np64(sx)[:, None] * np64(sw)[None, :]
    x, w = x.to(_t(dtype)), w.to(_t(dtype))
    got = np64(linear(x, w, x_scale=sx, weight_scale=sw, out_dtype=torch.float32))
    want = ref.linear(np64(x), np64(w), x_scale=None if sx is None else np64(sx),
                      weight_scale=None if sw is None else np64(sw))
    bound = ((K + 4) * U / (1 - K * U)) * a * (np.abs(np64(x)) @ np.abs(np64(w)).T)
    # normals past 448 became NaN in the conversion to e4m3: their rows and columns are NaN on both sides
    fine = ~np.isnan(want)
    assert np.array_equal(fine, ~np.isnan(got)) and fine.any()
    err = np.abs(got - want)[fine]
    log(f"[linear normal] M={M} N={N} K={K} {dtype}: worst err / bound {np.max(err / bound[fine]):.3g}, "
        f"relative {np.linalg.norm(err) / np.linalg.norm(want[fine]):.3g}")
    assert np.all(err <= bound[fine])
    low = np64(linear(x, w, x_scale=sx, weight_scale=sw))
    assert np.array_equal(fine, ~np.isnan(low))
    err = np.abs(low - want)[fine]
    unit = a * (np.abs(np64(x)) @ np.abs(np64(w)).T) * 2.0 ** -10 if dtype == "e4m3" else bound
    assert np.all(err <= (2.0 ** -8 * np.abs(want) * (1 + U) + unit)[fine])
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want[fine])


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", [(1, 500, 128), (40, 300, 64), (150, 260, 192), (300, 700, 64)])
def test_activations(M, N, K, act, odt):
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    log(f"[linear {act}] M={M} N={N} K={K} -> {odt}")
    x, w = grid(g, (M, K), "bf16"), grid(g, (N, K), "bf16")
    bias, res = grid(g, (N,), odt), grid(g, (M, N // 5), odt)
    v = ref.linear(np64(x), np64(w), np64(bias))
    got = np64(linear(x, w, bias=bias, residual=res, activation=act, out_dtype=_t(odt)))
    y = ref.activate(v, act)
    want = y + np.tile(np64(res), (1, 5))
    if act == "gelu":
        z = np.abs(v) / np.sqrt(2)
        rel = (2 * z * z + 1) * 2 * ULP + 20 * ULP
    elif act == "gelu_tanh":
        z = np.abs(2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3))
        rel = (8 + 4 * z) * ULP
    else:
        rel = 8 * ULP
    # below FLT_MIN an activation may come out as zero; the addition of the residual rounds once
    tol = rel * np.abs(y) + 2.0 ** -120 + ULP * np.abs(want) + (2.0 ** -8 if odt == "bf16" else 0.0) * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= tol), (np.max(err / tol), v[np.unravel_index(np.argmax(err / tol), v.shape)])


def test_the_output_over_the_residual_and_inside_a_larger_buffer():
    import torch

    from rejection_sampling_verify_09_amd import linear

    log("[linear] in place over the residual; margins")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for M, N, K in [(5, 300, 128), (70, 301, 192), (300, 260, 64)]:
        x, w = grid(g, (M, K), "bf16"), grid(g, (N, K), "bf16")
        res = grid(g, (M, N), "bf16")
        want = linear(x, w, residual=res, activation="silu")
        buf = torch.full((M * N + 66,), 7.0, device="cuda", dtype=torch.bfloat16)
        mine = buf[33:33 + M * N].view(M, N)
        mine.copy_(res)
        out = linear(x, w, residual=mine, activation="silu", out=mine)
        assert out.data_ptr() == mine.data_ptr() and torch.equal(out, want)
        assert (buf[:33] == 7).all() and (buf[33 + M * N:] == 7).all()


def test_stacked_heads_equal_the_heads_one_by_one():
    import torch

    from rejection_sampling_verify_09_amd import linear

    log("[linear] stacked heads")
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    H, d = 4, 256
    for lead in [(1,), (3, 7), (64,), (200,)]:
        x = grid(g, lead + (d,), "bf16")
        w = grid(g, (H * d, d), "bf16")
        b = grid(g, (H * d,), "bf16")
        y = linear(x, w, bias=b, residual=x, activation="silu")
        assert y.shape == lead + (H * d,)
        for k in range(H):
            s = slice(k * d, (k + 1) * d)
            assert torch.equal(y[..., s], linear(x, w[s], bias=b[s], residual=x, activation="silu"))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 20, 130, 300])
def test_non_finite_rows_stay_in_their_rows(M, dtype):
    """A NaN in a row of x makes that row NaN and no other; one in a row of the weight, that column."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    log(f"[linear] NaN M={M} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    N, K = 333, 320
    x, w = grid(g, (M, K), dtype), grid(g, (N, K), dtype)
    sc = {}
    if dtype == "e4m3":
        sc = dict(x_scale=torch.ones(M, device="cuda"), weight_scale=torch.ones(N, device="cuda"))
    clean = linear(x, w, out_dtype=torch.float32, **sc)
    xb = x.float()
    xb[M // 2, K - 1] = float("nan")
    wb = w.float()
    wb[N - 1, 0] = float("nan")
    got = linear(xb.to(_t(dtype)), wb.to(_t(dtype)), out_dtype=torch.float32, **sc)
    assert torch.isnan(got[M // 2]).all() and torch.isnan(got[:, N - 1]).all()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[keep][:, :N - 1], clean[keep][:, :N - 1])


def test_offsets_past_32_bits():
    """An output and a weight whose byte offsets pass 2^32: the last rows and columns come out as in a small call."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    log("[linear] large output and weight")
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for M, N, K in [(2049, 600000, 64), (3, 40000, 65536)]:
        x = grid(g, (M, K), "bf16")
        w = torch.empty((N, K), device="cuda", dtype=torch.bfloat16)
        for i in range(0, N, 10000):
            w[i:i + 10000] = grid(g, (min(10000, N - i), K), "bf16")
        out = linear(x, w, out_dtype=torch.float32)
        part = linear(x[-2:].clone(), w[-77:].clone(), out_dtype=torch.float32)
        assert torch.equal(out[-2:, -77:], part)
        first = linear(x[:2].clone(), w[:77].clone(), out_dtype=torch.float32)
        assert torch.equal(out[:2, :77], first)
        del out, w


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(440, 30001, 64), (1001, 8190, 128), (192, 32003, 64), (130, 20007, 576)])
def test_wide_tiles_between_margins(M, N, K, dtype, odt):
    """Products of many tiles, rows of an odd length from any element on: the
    sums are exact, and nothing around the output is written."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    log(f"[linear wide] M={M} N={N} K={K} {dtype} -> {odt}")
    x, w = grid(g, (M, K), dtype), grid(g, (N, K), dtype)
    sx = sw = None
    if dtype == "e4m3":
        sx = torch.exp2(torch.randint(-3, 4, (M,), device="cuda", generator=g).float())
        sw = torch.exp2(torch.randint(-3, 4, (N,), device="cuda", generator=g).float())
    want = x.float().cpu() @ w.float().cpu().T  # exact
    if sx is not None:
        want = want * sx.cpu()[:, None] * sw.cpu()
    for off in (1, 5):
        buf = torch.full((M * N + 16,), 7.0, device="cuda", dtype=_t(odt))
        out = buf[off:off + M * N].view(M, N)
        linear(x, w, x_scale=sx, weight_scale=sw, out_dtype=_t(odt), out=out)
        assert torch.equal(out.cpu(), want.to(_t(odt)))
        assert (buf[:off] == 7).all() and (buf[off + M * N:] == 7).all()


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 40])
def test_activations_of_extreme_values(M, act, odt):
    """Signed zeros, the smallest and largest values, infinities and NaN,
    brought in by the bias of a product of zeros."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    log(f"[linear extremes] M={M} {act} -> {odt}")
    v = [0.0, -0.0, 1e-45, -1e-45, 1.2e-38, -1.2e-38, 1e-20, -1e-20, 1e4, -1e4, 1e10, -1e10, 1e20, -1e20, 3e38, -3e38,
         float("inf"), -float("inf"), float("nan")]
    v += [s * k for k in (0.5, 1.0, 5.0, 9.0, 13.0, 14.5, 20.0, 86.0, 87.5, 88.5, 100.0, 103.5, 127.0, 128.0, 129.0)
          for s in (1.0, -1.0)]
    bias = torch.tensor(v, device="cuda").to(_t(odt))
    x = torch.zeros((M, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.zeros((len(v), 64), device="cuda", dtype=torch.bfloat16)
    got = np64(linear(x, w, bias=bias, activation=act, out_dtype=_t(odt)))
    b = np64(bias)
    with np.errstate(all="ignore"):
        want = np.tile(ref.activate(b, act), (M, 1))
        z = np.minimum(np.abs(2 * np.sqrt(2 / np.pi) * (b + 0.044715 * b ** 3)) if act == "gelu_tanh" else np.abs(b), 200.0)
        rel = (2 * (z * z / 2) + 1) * 2 * ULP + 20 * ULP if act == "gelu" else (8 + 4 * z) * ULP
        tol = rel * np.abs(want) + 2.0 ** -120 + (2.0 ** -8 if odt == "bf16" else 0.0) * np.abs(want)
    nan, inf = np.isnan(want), np.isinf(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[inf], want[inf])
    ok = ~nan & ~inf
    assert np.all(np.abs(got[ok] - want[ok]) <= tol[ok])


@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,R", [(440, 30030, 30030), (440, 30030, 10010), (130, 30030, 7), (1001, 6006, 1), (190, 30030, 143)])
def test_wide_tiles_with_residuals(M, N, R, dtype, odt):
    """Residuals that repeat inside a tile's columns, of an odd width, and the
    output's own memory; sums, bias and residual are exact before the one
    rounding."""
    import torch

    from rejection_sampling_verify_09_amd import linear

    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + R)
    log(f"[linear wide residual] M={M} N={N} R={R} {dtype} -> {odt}")
    x, w = grid(g, (M, 128), dtype), grid(g, (N, 128), dtype)
    sx = sw = None
    if dtype == "e4m3":
        sx = torch.exp2(torch.randint(-3, 4, (M,), device="cuda", generator=g).float())
        sw = torch.exp2(torch.randint(-3, 4, (N,), device="cuda", generator=g).float())
    bias, res = grid(g, (N,), odt), grid(g, (M, R), odt)
    want = x.float().cpu() @ w.float().cpu().T
    if sx is not None:
        want = want * sx.cpu()[:, None] * sw.cpu()
    want = (want + bias.float().cpu() + res.float().cpu().repeat(1, N // R)).to(_t(odt))
    out = linear(x, w, bias=bias, residual=res, x_scale=sx, weight_scale=sw, out_dtype=_t(odt))
    assert torch.equal(out.cpu(), want)
    if R == N:
        linear(x, w, bias=bias, residual=res, x_scale=sx, weight_scale=sw, out_dtype=_t(odt), out=res)
        assert torch.equal(res, out)
