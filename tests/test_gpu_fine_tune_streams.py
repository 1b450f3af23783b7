"""The operators for fine-tuning a draft as a program may call them: with
``stream=``, on two streams at once, in captured graphs (the largest
vocabularies included, whose kernels need more LDS than a launch has by
default), replayed several times over new inputs."""
import pytest

from tests.harness import log

pytestmark = pytest.mark.gpu


def calls(V=1000, k=40, rows=2048, d=1024, dtype=None, seed=0):
    """name -> (call of the stream argument, its input tensors, bytes of its first output)."""
    import torch

    import rejection_sampling_verify_09_amd as sv

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = dtype or torch.bfloat16
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g).to(dtype)  # noqa: E731
    x, h, w, logits = rnd(rows, d), rnd(rows, d), rnd(d), rnd(rows, V)
    target = rnd(rows, V)
    values, index, lse = sv.top_logits(target, k)
    es = x.element_size()
    return {
        "layer_norm": (lambda s: sv.layer_norm(x, w, w, residual=h, stream=s), (x, h), rows * d * es),
        "layer_norm_backward": (lambda s: sv.layer_norm_backward(x, h, w, stream=s), (x, h), rows * d * es),
        "rms_norm_backward": (lambda s: sv.rms_norm_backward(x, h, w, stream=s), (x, h), rows * d * es),
        "top_logits": (lambda s: sv.top_logits(logits, k, stream=s), (logits,), rows * k * 4),
        "distill_loss": (lambda s: sv.distill_loss(logits, index, values, top_lse=lse, with_grad=True, stream=s)[::-1],
                         (logits,), rows * V * es),
    }


NAMES = ["layer_norm", "layer_norm_backward", "rms_norm_backward", "top_logits", "distill_loss"]


def same(a, b):
    import torch

    return all(x is y is None or torch.equal(x, y) for x, y in zip(a, b))


def copies(a):
    return [None if v is None else v.clone() for v in a]


def busy(a, n=12):
    """Some milliseconds of work on the current stream."""
    for _ in range(n):
        a = a @ a
    return a


@pytest.mark.parametrize("kind", ["stream", "handle", "default stream's handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_leave_memory_alone_that_the_current_stream_still_reads(name, kind):
    import torch

    log(f"[fine-tune streams] {name}, {kind}")
    call, _, nbytes = calls()[name]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    here = other if kind == "default stream's handle" else torch.cuda.current_stream()
    there = {"stream": side, "handle": side.cuda_stream, "default stream's handle": 0}[kind]
    want = copies(call(None))
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
            assert out[0].data_ptr() != at
            torch.cuda.synchronize()
            assert torch.equal(copy, saved) and same(out, want)
            del out


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_until_the_current_stream_has_read_them(name):
    import torch

    log(f"[fine-tune streams] {name}, read on the current stream")
    call, _, nbytes = calls()[name]
    side = torch.cuda.Stream()
    want = copies(call(None))
    mat = torch.eye(4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        out = call(handle)
        torch.cuda.current_stream().wait_stream(side)
        busy(mat)
        copy = copies(out)  # queued behind the work
        del out
        with torch.cuda.stream(side):
            junk = [torch.full((nbytes // 4,), 3, device="cuda", dtype=torch.int32) for _ in range(3)]
        torch.cuda.synchronize()
        assert same(copy, want)
        del junk


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    import torch

    log(f"[fine-tune streams] {name}, two streams at once")
    a, b = calls(seed=1)[name], calls(seed=2)[name]
    want = [copies(c[0](None)) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(6):
        for i, (c, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                outs[i].append(c[0](None))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert same(o, want[i])


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("big", [False, True])
def test_captured_and_replayed(name, big):
    import torch

    if big and "norm" in name:
        shape = dict(rows=300, d=20000)
    else:
        shape = dict(V=1000001, rows=3, k=300, d=64, dtype=torch.float32) if big else dict(rows=300)
    log(f"[fine-tune streams] {name}, captured, {shape}")
    call, ins, _ = calls(**shape)[name]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = call(None)
    for turn in range(3):
        for v in ins:
            v.copy_(torch.randn(v.shape, device="cuda") * (turn + 1))
        want = copies(call(None))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, want)
        for o in outs:
            if o is not None:
                o.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, want)


def test_a_stream_of_another_device_and_tensors_on_the_host_are_refused():
    import torch

    import rejection_sampling_verify_09_amd as sv

    x = torch.zeros((2, 64), device="cuda")
    i, v = torch.zeros((2, 4), device="cuda", dtype=torch.int32), torch.zeros((2, 4), device="cuda")
    for call in (lambda: sv.distill_loss(x, i.cpu(), v), lambda: sv.distill_loss(x, i, v.cpu()),
                 lambda: sv.distill_loss(x, i, v, weight=torch.zeros(2)),
                 lambda: sv.layer_norm(x, torch.zeros(64)), lambda: sv.layer_norm_backward(x, x.cpu()),
                 lambda: sv.top_logits(x, 2, out_lse=torch.zeros(2))):
        with pytest.raises(ValueError):
            call()
    if torch.cuda.device_count() > 1:
        other = torch.cuda.Stream(device=1)
        for call in (lambda: sv.layer_norm(x, stream=other), lambda: sv.layer_norm_backward(x, x, stream=other),
                     lambda: sv.top_logits(x, 2, stream=other), lambda: sv.distill_loss(x, i, v, stream=other)):
            with pytest.raises(ValueError):
                call()


def test_element_offsets_past_32_bits():
    """More than 2^31 elements: the last rows come out as in a batch of their own."""
    import torch

    import rejection_sampling_verify_09_amd as sv

    log("[fine-tune] offsets past 32 bits")
    b = torch.bfloat16
    rows, d = (1 << 20) + 3000, 2048
    x, dy = torch.empty((rows, d), device="cuda", dtype=b).normal_(), torch.empty((rows, d), device="cuda", dtype=b).normal_()
    w = torch.randn((d,), device="cuda").to(b)
    last = slice(rows - 5, rows)
    y, _, _ = sv.layer_norm(x, w, w)
    assert torch.equal(y[last], sv.layer_norm(x[last], w, w)[0])
    for back in (sv.layer_norm_backward, sv.rms_norm_backward):
        got = back(dy, x, w, out=y)
        assert torch.equal(got[0][last], back(dy[last], x[last], w)[0]) and torch.isfinite(got[1]).all()
    del x, dy, y, got
    rows, V, k = 17000, 128256, 8
    x = torch.empty((rows, V), device="cuda", dtype=b).normal_()
    index = torch.randint(0, V, (rows, k), device="cuda", dtype=torch.int32)
    values = torch.randn((rows, k), device="cuda")
    last = slice(rows - 4, rows)
    want = sv.distill_loss(x[last].clone(), index[last], values[last], with_grad=True)
    loss, grad = sv.distill_loss(x, index, values, with_grad=True, out_grad=x)
    assert torch.equal(loss[last], want[0]) and torch.equal(grad[last], want[1]) and torch.isfinite(loss).all()
