"""GPU parity of adjust_logits with the float64 oracle.  Each step is one
float32 rounding (u = 2^-24) of a value whose magnitude the oracle sums up;
bfloat16 rounds once more (2^-8).  Logits that nothing touches keep their
bits."""
import numpy as np
import pytest

from oracle import last_layer as ref
from tests.harness import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _t(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def cuda(a, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def pack_mask(allowed):
    rows, V = allowed.shape
    W = (V + 31) // 32
    bits = np.zeros((rows, W * 32), dtype=np.uint64)
    bits[:, :V] = allowed
    bits[:, V:] = np.random.default_rng(1).integers(0, 2, (rows, W * 32 - V))  # bits past V mean nothing
    words = (bits.reshape(rows, W, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return words.astype(np.uint32).view(np.int32)


def make(seed, B, R, K, V, cap, dtype, seen=0, penalties=True, nbias=0, mask="none", ks=None, bonus=1):
    """A batch; ks: draft lengths of a ragged one."""
    g = np.random.default_rng(seed)
    rows = B * R if ks is None else int(sum(ks)) + B * bonus
    c = dict(B=B, R=R, K=K, V=V, cap=cap, dtype=dtype, seen=seen, ks=ks, bonus=bonus, rows=rows)
    lg = (g.standard_normal((rows, V)) * 2).astype(np.float32)
    lg[g.random((rows, V)) < 0.01] = -np.inf
    lg[g.random((rows, V)) < 0.01] = 0.0
    c["logits"] = cuda(lg, _t(dtype)).view((B, R, V) if ks is None else (rows, V))
    hot = g.integers(0, V, 40)  # tokens that come up often
    tok = lambda n: np.where(g.random(n) < 0.5, g.choice(hot, n), g.integers(-2, V + 2, n)).astype(np.int32)  # noqa: E731
    c["hist"] = tok((B, cap))
    c["hlen"] = g.integers(-1, cap + 3, B).astype(np.int32)
    c["plen"] = g.integers(-1, cap + 3, B).astype(np.int32)
    nd = B * K if ks is None else int(sum(ks))
    c["drafts"] = tok((B, K) if ks is None else (nd,))
    c["rep"] = (0.5 + 1.5 * g.random(B)).astype(np.float32) if penalties else None
    c["freq"] = (g.random(B) - 0.3).astype(np.float32) if penalties else None
    c["pres"] = (g.random(B) - 0.3).astype(np.float32) if penalties else None
    c["cub"] = None
    if nbias:
        n = g.integers(0, nbias + 1, B)
        c["cub"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["btok"] = tok(int(c["cub"][-1]))
        c["bval"] = g.standard_normal(int(c["cub"][-1])).astype(np.float32)
        c["bval"][g.random(c["bval"].shape) < 0.05] = -np.inf
    c["allowed"] = c["midx"] = None
    if mask != "none":
        n = rows if mask == "rows" else 5
        share = g.choice([0.0, 0.01, 0.5, 0.99, 1.0], n)
        c["allowed"] = g.random((n, V)) < share[:, None]
        if mask == "index":
            c["midx"] = g.integers(-1, n + 1, rows).astype(np.int32)
    return c


def call(c, out=None, logits=None, **more):
    from rejection_sampling_verify_09_amd import adjust_logits

    kw = dict(history=cuda(c["hist"]), history_len=cuda(c["hlen"]), prompt_len=cuda(c["plen"]),
              draft_tokens=cuda(c["drafts"]))
    for k, n in (("rep", "repetition_penalty"), ("freq", "frequency_penalty"), ("pres", "presence_penalty")):
        if c[k] is not None:
            kw[n] = cuda(c[k])
    if c["cub"] is not None:
        kw["bias"] = (cuda(c["cub"]), cuda(c["btok"]), cuda(c["bval"]))
    if c["allowed"] is not None:
        kw["mask"] = cuda(pack_mask(c["allowed"]))
    if c["midx"] is not None:
        kw["mask_index"] = cuda(c["midx"])
    if c["ks"] is not None:
        kw.update(cu_num_draft=cuda(np.concatenate([[0], np.cumsum(c["ks"])]).astype(np.int32)), max_k=c["K"])
    else:
        kw["drafts_seen"] = c["seen"]
    kw.update(more)
    return adjust_logits(c["logits"] if logits is None else logits, out=out, **kw)


def check(c, got):
    lg = c["logits"].float().cpu().numpy().astype(np.float64).reshape(c["rows"], c["V"])
    gb = got.cpu().reshape(c["rows"], c["V"])
    g64 = gb.float().numpy().astype(np.float64)
    raw = c["logits"].cpu().reshape(c["rows"], c["V"])
    row = 0
    d0 = 0
    for b in range(c["B"]):
        nr = c["R"] if c["ks"] is None else int(c["ks"][b]) + c["bonus"]
        n = min(max(int(c["hlen"][b]), 0), c["cap"])
        p = min(max(int(c["plen"][b]), 0), n)
        x = c["drafts"][b] if c["ks"] is None else c["drafts"][d0:d0 + int(c["ks"][b])]
        d0 += 0 if c["ks"] is None else int(c["ks"][b])
        pen = c["rep"] is not None
        bi = () if c["cub"] is None else list(zip(c["btok"], c["bval"]))[c["cub"][b]:c["cub"][b + 1]]
        for i in range(nr):
            allowed = None
            if c["allowed"] is not None:
                k = row if c["midx"] is None else int(c["midx"][row])
                allowed = c["allowed"][k] if 0 <= k < len(c["allowed"]) else None
            said = list(c["hist"][b, p:n]) + list(x[:c["seen"] + i])
            want, mag, touched = ref.adjust_row(
                lg[row], c["hist"][b, :p] if pen else (), said if pen else (), float(c["rep"][b]) if pen else 1.0,
                float(c["freq"][b]) if pen else 0.0, float(c["pres"][b]) if pen else 0.0, bi, allowed)
            inf = np.isinf(want)
            assert np.array_equal(g64[row][inf], want[inf]), (b, i)
            tol = 2 * U * np.where(inf, 0, mag) + (2.0 ** -8 if c["dtype"] == "bf16" else 0) * np.where(inf, 0, np.abs(want))
            err = np.abs(np.where(inf, 0, g64[row]) - np.where(inf, 0, want))
            keep = ~touched if allowed is None else ~touched & allowed
            assert np.all(err[touched] <= tol[touched] + 2.0 ** -140), (b, i, np.argwhere(err > tol)[:3])
            idx = np.flatnonzero(keep)
            assert np.array_equal(gb[row][idx].view(_bits(c)).numpy(), raw[row][idx].view(_bits(c)).numpy()), (b, i)
            row += 1
    assert row == c["rows"]


def _bits(c):
    import torch

    return torch.int32 if c["dtype"] == "f32" else torch.int16


CASES = {
    "one row": dict(B=1, R=1, K=0, V=1000, cap=50),
    "one token": dict(B=3, R=2, K=1, V=1, cap=4),
    "no history": dict(B=2, R=3, K=2, V=77, cap=0),
    "target rows": dict(B=4, R=6, K=5, V=5000, cap=300),
    "draft rows": dict(B=3, R=4, K=4, V=4097, cap=100),
    "one row behind drafts": dict(B=5, R=1, K=7, V=2048, cap=20, seen=5),
    "rows from the third draft": dict(B=2, R=3, K=6, V=999, cap=20, seen=3),
    "slices": dict(B=2, R=3, K=2, V=20003, cap=1000),
    "aligned slices": dict(B=2, R=3, K=2, V=32768, cap=1000),
    "many rows": dict(B=1, R=65, K=64, V=10008, cap=64),
    "biases": dict(B=4, R=3, K=2, V=3000, cap=100, nbias=200),
    "biases alone": dict(B=3, R=2, K=1, V=9000, cap=0, penalties=False, nbias=100),
    "masks": dict(B=3, R=4, K=3, V=9001, cap=60, mask="rows"),
    "masks alone": dict(B=3, R=4, K=3, V=8320, cap=0, penalties=False, mask="rows"),
    "mask table": dict(B=4, R=5, K=4, V=17000, cap=60, nbias=40, mask="index"),
    "mask table alone": dict(B=4, R=2, K=1, V=333, cap=0, penalties=False, mask="index"),
    "ragged targets": dict(B=6, R=0, K=5, V=6008, cap=80, ks=(0, 5, 2, 0, 1, 4), nbias=9, mask="rows"),
    "ragged drafts": dict(B=5, R=0, K=6, V=2500, cap=80, ks=(3, 0, 6, 0, 2), bonus=0),
    "ragged without drafts": dict(B=3, R=0, K=4, V=700, cap=9, ks=(0, 0, 0)),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_oracle(name, dtype):
    log(f"[adjust] {name} {dtype}")
    c = make(len(name) * 7 + 1, dtype=dtype, **CASES[name])
    got = call(c)
    check(c, got)
    # in place, and in place between margins that stay as they were
    import torch

    mine = c["logits"].clone()
    assert call(c, out=mine, logits=mine).data_ptr() == mine.data_ptr()
    assert torch.equal(mine.view(_bits(c)), got.view(_bits(c)))
    n = c["logits"].numel()
    buf = torch.full((n + 18,), 7.0, device="cuda", dtype=_t(dtype))
    off = buf[9:9 + n].view(c["logits"].shape)  # bases that are not 16-byte aligned
    off.copy_(c["logits"])
    call(c, out=off, logits=off)
    assert torch.equal(off.view(_bits(c)), got.view(_bits(c)))
    off2 = torch.full_like(buf, 7.0)
    call(c, out=off2[9:9 + n].view(c["logits"].shape))
    assert torch.equal(off2[9:9 + n].view(c["logits"].shape).view(_bits(c)), got.view(_bits(c)))
    for b in (buf, off2):
        assert (b[:9] == 7).all() and (b[9 + n:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_non_finite_logits(dtype):
    """NaN and infinities where the mask forbids are -inf; where nothing touches them they stay; -inf stays -inf
    under every penalty."""
    import torch

    log(f"[adjust] non-finite {dtype}")
    c = make(5, B=2, R=2, K=1, V=4104, cap=64, dtype=dtype, mask="rows")
    c["allowed"][:] = np.random.default_rng(2).random(c["allowed"].shape) < 0.5
    lg = c["logits"].view(4, -1)
    lg[:, 0:64] = float("nan")
    lg[:, 64:128] = float("inf")
    lg[:, 128:192] = -float("inf")
    for out in (None, lg.clone()):
        src = c["logits"] if out is None else out.view(c["logits"].shape)
        got = call(c, out=None if out is None else src, logits=src).view(4, -1).float().cpu()
        al = torch.from_numpy(c["allowed"])
        assert (got[~al] == -float("inf")).all()
        assert torch.isnan(got[:, 0:64][al[:, 0:64]]).all()
        assert (got[:, 64:128][al[:, 64:128]] == float("inf")).all()
        assert (got[:, 128:192] == -float("inf")).all()


def test_a_mask_that_allows_nothing_gives_a_row_without_a_distribution():
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits, sample

    log("[adjust] empty rows, then sample")
    V = 5000
    lg = torch.randn((4, V), device="cuda")
    mask = torch.full((4, (V + 31) // 32), -1, device="cuda", dtype=torch.int32)
    mask[1] = 0
    mask[3] = 0
    mask[3, 70] = 1 << 5  # one token
    out = adjust_logits(lg, mask=mask)
    tok, p = sample(out, torch.full((4,), 0.5, device="cuda"), 0.8, 0, 0.9)
    tok, p = tok.cpu(), p.cpu()
    assert tok[1] == -1 and torch.isnan(p[1]) and tok[3] == 70 * 32 + 5 and p[3] == 1.0
    assert (tok[[0, 2]] >= 0).all()


def test_ragged_offsets_that_describe_no_packing_write_nothing():
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log("[adjust] bad offsets")
    lg = torch.randn((8, 300), device="cuda")
    rep = torch.full((3,), 1.5, device="cuda")
    hist = torch.randint(0, 300, (3, 40), device="cuda", dtype=torch.int32)
    x = torch.zeros(5, device="cuda", dtype=torch.int32)
    for cu in ([1, 2, 3, 5], [0, 2, 3, 4], [0, 3, 2, 5], [0, 5, 5, 5], [0, -1, 4, 5]):
        out = torch.full_like(lg, 7.0)
        adjust_logits(lg, history=hist, repetition_penalty=rep, draft_tokens=x, max_k=4, out=out,
                      cu_num_draft=torch.tensor(cu, device="cuda", dtype=torch.int32))
        assert (out == 7).all(), cu
    adjust_logits(lg, history=hist, repetition_penalty=rep, draft_tokens=x, max_k=4, out=out,
                  cu_num_draft=torch.tensor([0, 4, 4, 5], device="cuda", dtype=torch.int32))
    assert not (out == 7).any()


def test_long_histories_and_counts():
    """A token that fills a history of 100,000, next to ordinary ones."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log("[adjust] long history")
    V, n = 40000, 100_000
    lg = torch.zeros((2, V), device="cuda")
    hist = torch.full((2, n), 123, device="cuda", dtype=torch.int32)
    hist[1] = torch.arange(n, device="cuda", dtype=torch.int32) % V
    freq = torch.tensor([2.0 ** -10, 1.0], device="cuda")
    out = adjust_logits(lg, history=hist, frequency_penalty=freq).cpu()
    assert out[0, 123] == -n * 2.0 ** -10 and (out[0].nonzero().numel() == 1)
    want = -(torch.arange(V) < n % V).float() - n // V
    assert torch.equal(out[1], want)


def test_many_biases_of_one_token_add_up_in_their_order():
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log("[adjust] duplicate biases")
    g = np.random.default_rng(8)
    V = 3000
    tok = g.integers(0, 6, 500).astype(np.int32) * 499
    val = (g.standard_normal(500) * 10.0 ** g.integers(-4, 5, 500)).astype(np.float32)
    want = np.zeros(V, dtype=np.float32)
    for j in range(0, 2995, 499):
        s = None
        for t, v in zip(tok, val):
            if t == j:
                s = v if s is None else np.float32(s + v)
        want[j] = 0.0 if s is None else s
    # and more of them than the kernel holds on chip
    more = np.concatenate([tok, np.full(1500, 499, dtype=np.int32), tok])
    mval = np.concatenate([val, np.full(1500, 2.0 ** -3, dtype=np.float32), val])
    mw = np.zeros(V, dtype=np.float32)
    for t, v in zip(more, mval):
        mw[t] = np.float32(mw[t] + v)
    out = adjust_logits(torch.zeros((1, V), device="cuda"),
                        bias=(cuda(np.array([0, 2500], dtype=np.int32)), cuda(more), cuda(mval))).cpu().numpy()
    assert np.array_equal(out[0], mw)
    cu = cuda(np.array([0, 500], dtype=np.int32))
    for _ in range(3):
        out = adjust_logits(torch.zeros((1, V), device="cuda"), bias=(cu, cuda(tok), cuda(val))).cpu().numpy()
        assert np.array_equal(out[0], want)


def test_offsets_past_32_bits():
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log("[adjust] large batch")
    B, R, V = 600, 9, 400_000  # 8.6 GB of float32 logits
    lg = torch.zeros((B, R, V), device="cuda")
    hist = torch.full((B, 3), V - 1, device="cuda", dtype=torch.int32)
    pres = torch.full((B,), 1.0, device="cuda")
    mask = torch.full((1, (V + 31) // 32), -1, device="cuda", dtype=torch.int32)
    mask[0, 0] = -2
    idx = torch.zeros((B * R,), device="cuda", dtype=torch.int32)
    out = adjust_logits(lg, history=hist, presence_penalty=pres, mask=mask, mask_index=idx)
    for o in (out, adjust_logits(lg, history=hist, presence_penalty=pres, mask=mask, mask_index=idx, out=lg)):
        v = o.view(-1, V)
        assert (v[:, -1] == -1).all() and (v[:, 0] == -float("inf")).all()
        assert int(torch.count_nonzero(v[-1])) == 2 and int(torch.count_nonzero(v[0])) == 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nbias", [60, 3000])
def test_the_widest_slices(nbias, dtype):
    """Long histories take the widest slices: with biases, and in place, the
    tables fill more than 64 KB of LDS."""
    import torch

    log(f"[adjust] widest slices {nbias} {dtype}")
    c = make(40 + nbias, B=2, R=3, K=2, V=20003, cap=20000, dtype=dtype, nbias=nbias, mask="index")
    got = call(c)
    check(c, got)
    mine = c["logits"].clone()
    call(c, out=mine, logits=mine)
    assert torch.equal(mine.view(_bits(c)), got.view(_bits(c)))


@pytest.mark.parametrize("n,tokens", [(200, 3), (200, 40), (250, 1), (256, 256), (257, 30), (17, 1), (18, 1)])
def test_chains_of_biases_add_up_in_their_order(n, tokens):
    """Few and many biases of one token, in one slice and on both sides of
    what it holds on chip; the float32 sums are those of the listed order."""
    import torch

    from rejection_sampling_verify_09_amd import adjust_logits

    log(f"[adjust] {n} biases of {tokens} tokens")
    g = np.random.default_rng(n * 1000 + tokens)
    V = 900
    tok = (g.permutation(n) % tokens * 3 + 1).astype(np.int32)
    val = (g.standard_normal(n) * 10.0 ** g.integers(-4, 5, n)).astype(np.float32)
    want = np.zeros(V, dtype=np.float32)
    seen = set()
    for t, v in zip(tok, val):
        want[t] = np.float32(want[t] + v) if t in seen else v
        seen.add(int(t))
    # a second sequence without any, and a third with the same in another place of the list
    cu = cuda(np.array([0, n, n, 2 * n], dtype=np.int32))
    b = (cu, cuda(np.concatenate([tok, tok])), cuda(np.concatenate([val, val])))
    lg = torch.zeros((3, V), device="cuda")
    for _ in range(2):
        out = adjust_logits(lg, bias=b).cpu().numpy()
        assert np.array_equal(out[0], want) and np.array_equal(out[2], want) and not out[1].any()
    adjust_logits(lg, bias=b, out=lg)
    assert np.array_equal(lg.cpu().numpy(), out)
