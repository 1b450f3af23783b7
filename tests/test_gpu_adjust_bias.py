"""The biases of adjust_logits where their order and number matter: added to
each other in the order they are listed, in float32, and then to the logit."""
import numpy as np
import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def cuda(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def summed(tok, val, V):
    """float32 sums of each token's biases in their order, and which tokens have any."""
    out, has = np.zeros(V, dtype=np.float32), np.zeros(V, dtype=bool)
    for t in np.unique(tok):
        out[t] = np.add.accumulate(val[tok == t], dtype=np.float32)[-1]
        has[t] = True
    return out, has


@pytest.mark.parametrize("n", [2, 16, 17, 40, 900, 1500])
def test_biases_are_added_to_each_other_before_the_logit(n):
    """1e8, whose neighbours are 8 away, and n biases of 3: one by one they would not move it."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log(f"[adjust] {n} small biases of a large logit")
    V = 700
    tok, val = np.full(n, 123, dtype=np.int32), np.full(n, 3.0, dtype=np.float32)
    total = np.float32(3 * n)
    lg = torch.full((2, V), 1e8, device="cuda")
    bias = (cuda(np.array([0, n, n], dtype=np.int32)), cuda(tok), cuda(val))
    for out in (None, lg):
        got = adjust_logits(lg, bias=bias, out=out).cpu().numpy()
        want = np.full((2, V), 1e8, dtype=np.float32)
        want[0, 123] = np.float32(1e8) + total
        assert want[0, 123] >= np.float32(1e8) + 8 and np.array_equal(got, want)


def test_biases_at_the_end_of_the_longest_list():
    """Offsets next to 2^31, where positions a few past the last bias do not fit a signed number; all but the last
    60 entries of the list are in no sequence."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    n, V, m = (1 << 31) - 1, 3000, 60
    log(f"[adjust] the last {m} of {n} biases")
    tok = torch.empty((n,), device="cuda", dtype=torch.int32)
    val = torch.empty((n,), device="cuda", dtype=torch.float32)
    g = np.random.default_rng(3)
    t, v = g.integers(-1, 40, m).astype(np.int32) * 71, g.standard_normal(m).astype(np.float32)
    tok[-m:], val[-m:] = cuda(t), cuda(v)
    cu = torch.tensor([n - m, n - m + 20, n], device="cuda", dtype=torch.int32)
    lg = torch.zeros((2, V), device="cuda")
    for out in (None, lg):
        got = adjust_logits(lg, bias=(cu, tok, val), out=out).cpu().numpy()
        for b, s in enumerate((slice(0, 20), slice(20, m))):
            ok = t[s] >= 0
            assert np.array_equal(got[b], summed(t[s][ok], v[s][ok], V)[0]), b


def many(kind, n, V, g):
    """Token lists of n biases of one sequence."""
    if kind == "two tokens, one behind the other":
        return np.repeat(np.array([5, 900], dtype=np.int32), n // 2)
    if kind == "every token twice, far apart":
        one = g.permutation(V)[:n // 2].astype(np.int32)
        return np.concatenate([one, one[::-1]])
    if kind == "one long chain among others":
        tok = g.integers(0, V, n).astype(np.int32)
        tok[g.permutation(n)[:40]] = 77
        return tok
    return g.integers(0, 300, n).astype(np.int32)


@pytest.mark.parametrize("kind,n,V", [
    ("two tokens, one behind the other", 200_000, 1000), ("every token twice, far apart", 150_000, 100_000),
    ("one long chain among others", 60_000, 128_256), ("a few tokens over and over", 200_000, 2049),
    ("a few tokens over and over", 1_025, 2049), ("a few tokens over and over", 5_000, 1)])
def test_long_lists_of_repeated_biases(kind, n, V):
    """The walk through the list, whose time is the list's length times a constant: a search for each bias of a
    repeated token would take n^2 / 4 steps here."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log(f"[adjust] {n} biases, V={V}: {kind}")
    g = np.random.default_rng(n + V)
    tok = many(kind, n, V, g)
    val = (g.standard_normal(len(tok)) * 10.0 ** g.integers(-3, 4, len(tok))).astype(np.float32)
    few = g.integers(0, V, 9).astype(np.int32)  # and an ordinary sequence next to it
    fval = g.standard_normal(9).astype(np.float32)
    cu = cuda(np.array([0, len(tok), len(tok) + 9], dtype=np.int32))
    bias = (cu, cuda(np.concatenate([tok, few])), cuda(np.concatenate([val, fval])))
    keep = tok < V
    want = np.stack([summed(tok[keep], val[keep], V)[0], summed(few, fval, V)[0]])
    lg = torch.zeros((2, 3, V), device="cuda")
    for out in (None, None, lg):
        got = adjust_logits(lg, bias=bias, out=out).cpu().numpy()
        for r in range(3):
            assert np.array_equal(got[:, r], want)


def test_long_histories_beside_long_lists_of_biases():
    """The widest slices, whose workgroups have more threads than the walk's pieces have room."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    V, n = 20_003, 30_000
    log(f"[adjust] {n} biases beside a history of 20,000")
    g = np.random.default_rng(11)
    tok = np.where(g.random(n) < 0.5, g.integers(0, 50, n), g.integers(0, V, n)).astype(np.int32)
    val = g.standard_normal(n).astype(np.float32)
    hist = torch.zeros((40, 20_000), device="cuda", dtype=torch.int32)
    cu = np.zeros(41, dtype=np.int32)
    cu[1:] = n  # the first sequence has them all, so that the slices' room is the least
    want = np.zeros((40, V), dtype=np.float32)
    want[0] = summed(tok, val, V)[0]
    pres = torch.full((40,), 2.0, device="cuda")
    lg = torch.zeros((40, V), device="cuda")
    want[:, 0] = np.float32(-2.0) + want[:, 0]
    for out in (None, lg):
        got = adjust_logits(lg, history=hist, presence_penalty=pres, bias=(cuda(cu), cuda(tok), cuda(val)), out=out)
        assert np.array_equal(got.cpu().numpy(), want)


def test_offsets_outside_the_list_are_taken_as_its_ends():
    """Negative and large offsets, and ones that run backwards, of a list inside a longer buffer."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log("[adjust] bias offsets past the list's ends")
    V, n = 50, 6
    tok = torch.arange(100, device="cuda", dtype=torch.int32) % V
    val = torch.arange(1, 101, device="cuda").float()
    lo, hi = -(1 << 31), (1 << 31) - 1
    for cu, ranges in (((-5, 3, 100), ((0, 3), (3, 6))), ((2, hi, hi), ((2, 6), (6, 6))), ((4, 1, 5), ((4, 4), (1, 5))),
                       ((lo, lo, lo), ((0, 0), (0, 0))), ((3, lo, hi), ((3, 3), (0, 6))), ((7, lo, 6), ((6, 6), (0, 6)))):
        want = np.zeros((2, V), dtype=np.float32)
        for b, (i, k) in enumerate(ranges):
            want[b, i:k] = np.arange(i + 1, k + 1)
        lg = torch.zeros((2, V), device="cuda")
        offsets = torch.tensor(cu, device="cuda", dtype=torch.int64).to(torch.int32)
        for out in (None, lg):
            got = adjust_logits(lg, bias=(offsets, tok[:n], val[:n]), out=out).cpu().numpy()
            assert np.array_equal(got, want), cu
