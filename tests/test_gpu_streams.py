"""Calls with ``stream=``: their new outputs are written on that stream, whose
work the current stream's is not ordered with, so they must not lie in memory
that the current stream has freed and still reads, nor be handed out again
while the current stream reads them."""
import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def calls():
    """name -> (call of the stream argument, bytes of its first output)."""
    import torch

    import rejection_sampling_verify_09_amd as sv

    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn((2048, 1024), device="cuda", generator=g).bfloat16()
    w = torch.randn((1024,), device="cuda", generator=g).bfloat16()
    wide = torch.randn((2048, 1024), device="cuda", generator=g).bfloat16()
    pres = torch.full((2048,), 0.5, device="cuda")
    return {
        "rms_norm": (lambda s: sv.rms_norm(x, w, stream=s)[0], 2048 * 1024 * 2),
        "linear": (lambda s: sv.linear(x, wide, stream=s), 2048 * 2048 * 2),
        "adjust_logits": (lambda s: sv.adjust_logits(x, presence_penalty=pres, stream=s), 2048 * 1024 * 2),
        **verification(g),
    }


def verification(g):
    import torch

    import rejection_sampling_verify_09_amd as sv

    B, K, V, d = 640, 3, 1000, 128
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    tl, dl = rnd(B, K + 1, V), rnd(B, K, V)
    x = torch.randint(0, V, (B, K), device="cuda", generator=g, dtype=torch.int32)
    u = torch.rand((B, K + 1), device="cuda", generator=g)
    q = torch.softmax(dl, 2)
    cu = torch.arange(0, (B + 1) * K, K, device="cuda", dtype=torch.int32)
    h, hd, w = rnd(B, K + 1, d).bfloat16(), rnd(B, K, d).bfloat16(), rnd(V, d).bfloat16()
    rows, words = tl.view(-1, V), torch.arange(1 << 20, device="cuda", dtype=torch.int32)
    tokens = B * (K + 1) * 4
    return {
        "spec_verify": (lambda s: sv.spec_verify(tl, dl, x, u, stream=s)[0], tokens),
        "spec_verify debug": (lambda s: sv.spec_verify(tl, dl, x, u, stream=s, debug=True)[2]["p"], B * K * 8),
        "spec_verify_noalloc": (lambda s: sv.spec_verify_noalloc(tl[:64], dl[:64], x[:64], u[:64], stream=s)[0], 1024),
        "spec_verify_ragged": (lambda s: sv.spec_verify_ragged(rows, dl.view(-1, V), x.view(-1), u.view(-1), cu, K,
                                                               stream=s)[0], tokens),
        "spec_verify_probs": (lambda s: sv.spec_verify_probs(tl, q, x, u, stream=s)[0], tokens),
        "spec_verify_lmhead": (lambda s: sv.spec_verify_lmhead(h, w, hd, w, x, u, stream=s)[0], tokens),
        "lm_logits": (lambda s: sv.lm_logits(h, w, stream=s), B * (K + 1) * V * 4),
        "filtered_probs": (lambda s: sv.filtered_probs(rows, 0.8, stream=s), B * (K + 1) * V * 4),
        "sample": (lambda s: sv.sample(rows, u.view(-1), stream=s)[0], tokens),
        "read_floor": (lambda s: sv.read_floor(words, stream=s), 1024),
    }


NAMES = ["rms_norm", "linear", "adjust_logits", "spec_verify", "spec_verify debug", "spec_verify_noalloc",
         "spec_verify_ragged", "spec_verify_probs", "spec_verify_lmhead", "lm_logits", "filtered_probs", "sample",
         "read_floor"]


def busy(a, n=12):
    """Some milliseconds of work on the current stream."""
    for _ in range(n):
        a = a @ a
    return a


@pytest.mark.parametrize("kind", ["stream", "handle", "default stream's handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_leave_memory_alone_that_the_current_stream_still_reads(name, kind):
    import torch

    log(f"[streams] {name}, {kind}")
    call, nbytes = calls()[name]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    # the stream the program works on, and the one the call is queued on
    here = other if kind == "default stream's handle" else torch.cuda.current_stream()
    there = {"stream": side, "handle": side.cuda_stream, "default stream's handle": 0}[kind]
    want = call(None).clone()
    mat = torch.eye(4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        for _ in range(2):
            held = torch.arange(nbytes // 4, device="cuda", dtype=torch.int32)
            saved = held.clone()
            here.synchronize()
            at = held.data_ptr()
            busy(mat)
            copy = held.clone()  # queued behind the work
            del held  # free again in this stream's memory, and not read yet
            out = call(there)
            assert out.data_ptr() != at
            torch.cuda.synchronize()
            assert torch.equal(copy, saved)
            assert torch.equal(out, want)
            del out


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_until_the_current_stream_has_read_them(name):
    import torch

    log(f"[streams] {name}, read on the current stream")
    call, nbytes = calls()[name]
    side = torch.cuda.Stream()
    want = call(None).clone()
    mat = torch.eye(4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        out = call(handle)
        torch.cuda.current_stream().wait_stream(side)
        busy(mat)
        copy = out.clone()  # queued behind the work
        del out
        with torch.cuda.stream(side):  # would take the freed memory and write it at once
            junk = [torch.full((nbytes // 4,), 7, device="cuda", dtype=torch.int32) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del junk


def test_a_round_given_a_stream():
    """Every call of a round queued on a stream that is not the current one, the program's own tensor work as well."""
    import torch

    from tests.test_gpu_last_layer import Round, _flat, _same

    log("[streams] a round on a given stream")
    r = Round(seed=6)
    want = _flat(r.run())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            got = r.run(stream=handle)
        torch.cuda.synchronize()
        assert _same(_flat(got), want)


def test_a_captured_fork_onto_a_given_stream():
    """A capture whose calls are queued on a second stream that it has forked, replayed between eager calls."""
    import torch

    import rejection_sampling_verify_09_amd as sv

    log("[streams] captured fork")
    x = torch.randn((300, 512), device="cuda").bfloat16()
    w = torch.randn((512,), device="cuda").bfloat16()
    wide = torch.randn((1000, 512), device="cuda").bfloat16()
    pres = torch.full((300,), 0.5, device="cuda")
    side = torch.cuda.Stream()

    def chain(stream):
        here = torch.cuda.current_stream()
        if stream is not None:
            side.wait_stream(here)
        y, _, _ = sv.rms_norm(x, w, stream=stream)
        logits = sv.linear(y, wide, stream=stream)
        out = sv.adjust_logits(logits, history=hist, presence_penalty=pres, stream=stream)
        if stream is not None:
            here.wait_stream(side)
        return y + 0, logits + 0, out + 0

    hist = torch.randint(0, 1000, (300, 40), device="cuda", dtype=torch.int32)
    chain(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(side)
    for rep in range(4):
        x.copy_(torch.randn((300, 512), device="cuda"))
        hist.random_(0, 1000)
        g.replay()
        want = chain(side if rep % 2 else None)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep


def test_a_stream_of_another_device_is_refused():
    import torch

    import rejection_sampling_verify_09_amd as sv

    class Elsewhere(torch.cuda.Stream):
        device = torch.device("cuda:1")

    log("[streams] another device's stream")
    x = torch.zeros((2, 64), device="cuda", dtype=torch.bfloat16)
    s = Elsewhere()
    for f in (lambda: sv.rms_norm(x, x[0], stream=s), lambda: sv.linear(x, x, stream=s),
              lambda: sv.adjust_logits(x, stream=s)):
        with pytest.raises(ValueError, match="stream on cuda:1"):
            f()
