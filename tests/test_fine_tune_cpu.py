"""The operators for fine-tuning a draft, without a GPU: refusals of the C ABI
(answered before any HIP call), refusals of the binding, and the oracle's own
pins: closed forms, and gradients against differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rejection_sampling_verify_09_amd as sv
from oracle import fine_tune as ref
from rejection_sampling_verify_09_amd import _lib as L


def P(i, off=0):
    """Addresses a terabyte apart, never dereferenced."""
    return ctypes.c_void_p(((i + 1) << 40) + off)


def layer(x=P(0), res=P(1), w=P(2), b=P(6), eps=1e-6, out=P(3), scale=P(4), hres=P(5), rows=3, d=64, dt=L.SV_BF16,
          odt=L.SV_BF16):
    return L.lib().sv_layer_norm(x, res, w, b, eps, out, scale, hres, rows, d, dt, odt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SV_ERR_SHAPE), (dict(d=0), L.SV_ERR_SHAPE), (dict(d=65537), L.SV_ERR_SHAPE),
    (dict(rows=1 << 23, d=8192), L.SV_ERR_SHAPE), (dict(rows=2 ** 31 - 1, d=1), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(dt=-1), L.SV_ERR_DTYPE), (dict(odt=3), L.SV_ERR_DTYPE),
    (dict(eps=0.0), L.SV_ERR_PARAM), (dict(eps=-1.0), L.SV_ERR_PARAM), (dict(eps=math.nan), L.SV_ERR_PARAM),
    (dict(eps=math.inf), L.SV_ERR_PARAM),
    (dict(x=None), L.SV_ERR_NULL), (dict(out=None), L.SV_ERR_NULL), (dict(res=None), L.SV_ERR_NULL),
    (dict(odt=L.SV_E4M3, scale=None), L.SV_ERR_NULL),
    (dict(x=P(0, 1)), L.SV_ERR_SHAPE), (dict(b=P(6, 1)), L.SV_ERR_SHAPE), (dict(out=P(3, 2), odt=L.SV_F32), L.SV_ERR_SHAPE),
    (dict(out=P(0), odt=L.SV_F32), L.SV_ERR_PARAM), (dict(out=P(0, 2)), L.SV_ERR_PARAM),
    (dict(hres=P(3)), L.SV_ERR_PARAM), (dict(out=P(2)), L.SV_ERR_PARAM), (dict(out=P(6)), L.SV_ERR_PARAM),
    (dict(hres=P(6)), L.SV_ERR_PARAM), (dict(odt=L.SV_E4M3, scale=P(6)), L.SV_ERR_PARAM),
    (dict(odt=L.SV_E4M3, scale=P(3)), L.SV_ERR_PARAM), (dict(odt=L.SV_E4M3, out=P(1)), L.SV_ERR_PARAM),
    (dict(rows=0, x=None, res=None, w=None, b=None, out=None, scale=None, hres=None), L.SV_OK),
])
def test_layer_norm_refusals(kw, code):
    assert layer(**kw) == code


def back(center=True, dy=P(0), h=P(1), w=P(2), dres=P(3), eps=1e-6, dh=P(4), dw=P(5), db=P(6), ws=P(7), nbytes=None,
         rows=300, d=64, dt=L.SV_BF16):
    if nbytes is None:
        nbytes = max(0, L.lib().sv_norm_backward_workspace(rows, d))
    if center:
        return L.lib().sv_layer_norm_backward(dy, h, w, dres, eps, dh, dw, db, ws, nbytes, rows, d, dt, None)
    return L.lib().sv_rms_norm_backward(dy, h, w, dres, eps, dh, dw, ws, nbytes, rows, d, dt, None)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SV_ERR_SHAPE), (dict(d=0), L.SV_ERR_SHAPE), (dict(d=65537), L.SV_ERR_SHAPE),
    (dict(rows=2 ** 30 + 1, d=1), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(eps=0.0), L.SV_ERR_PARAM), (dict(eps=math.nan), L.SV_ERR_PARAM),
    (dict(dy=None), L.SV_ERR_NULL), (dict(h=None), L.SV_ERR_NULL), (dict(dh=None), L.SV_ERR_NULL),
    (dict(ws=None), L.SV_ERR_NULL), (dict(nbytes=16), L.SV_ERR_WORKSPACE), (dict(nbytes=-1), L.SV_ERR_WORKSPACE),
    (dict(dy=P(0, 1)), L.SV_ERR_SHAPE), (dict(dw=P(5, 2)), L.SV_ERR_SHAPE), (dict(ws=P(7, 4)), L.SV_ERR_SHAPE),
    (dict(dh=P(0, 2)), L.SV_ERR_PARAM), (dict(dh=P(2)), L.SV_ERR_PARAM), (dict(dw=P(0)), L.SV_ERR_PARAM),
    (dict(dw=P(2)), L.SV_ERR_PARAM), (dict(dw=P(4)), L.SV_ERR_PARAM), (dict(ws=P(1)), L.SV_ERR_PARAM),
    (dict(ws=P(4)), L.SV_ERR_PARAM), (dict(ws=P(5)), L.SV_ERR_PARAM), (dict(h=P(0), dh=P(0, 128)), L.SV_ERR_PARAM),
])
def test_norm_backward_refusals(center, kw, code):
    assert back(center=center, **kw) == code


def test_the_bias_gradient_has_its_own_memory():
    assert back(db=P(5)) == L.SV_ERR_PARAM and back(db=P(4)) == L.SV_ERR_PARAM and back(db=P(7)) == L.SV_ERR_PARAM
    assert back(db=P(6, 1)) == L.SV_ERR_SHAPE


def test_workspace_sizes():
    f = L.lib().sv_norm_backward_workspace
    assert f(0, 64) == 0 and f(1, 65536) == 0
    assert f(2 ** 30 + 1, 1) == L.SV_ERR_SHAPE and f(-1, 64) == L.SV_ERR_SHAPE and f(4, 0) == L.SV_ERR_SHAPE and f(4, 65537) == L.SV_ERR_SHAPE
    for rows, d in ((2, 1), (448, 4096), (2 ** 30, 65536)):
        assert 0 <= f(rows, d) <= 2048 * 8 * d and f(rows, d) % 16 == 0


def top(x=P(0), k=5, T=1.0, v=P(1), i=P(2), s=P(3), rows=3, V=100, dt=L.SV_F32):
    return L.lib().sv_top_logits(x, k, T, v, i, s, rows, V, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SV_ERR_SHAPE), (dict(V=0), L.SV_ERR_SHAPE), (dict(V=2097153), L.SV_ERR_SHAPE),
    (dict(k=0), L.SV_ERR_SHAPE), (dict(k=-1), L.SV_ERR_SHAPE), (dict(k=101), L.SV_ERR_SHAPE),
    (dict(k=1025, V=5000), L.SV_ERR_SHAPE), (dict(rows=1 << 22, V=128256), L.SV_ERR_SHAPE),
    (dict(rows=2 ** 31 - 1), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(dt=9), L.SV_ERR_DTYPE),
    (dict(T=0.0), L.SV_ERR_PARAM), (dict(T=-1.0), L.SV_ERR_PARAM), (dict(T=math.inf), L.SV_ERR_PARAM),
    (dict(T=math.nan), L.SV_ERR_PARAM), (dict(T=1e-39), L.SV_ERR_PARAM),
    (dict(x=None), L.SV_ERR_NULL), (dict(v=None), L.SV_ERR_NULL), (dict(i=None), L.SV_ERR_NULL),
    (dict(x=P(0, 2)), L.SV_ERR_SHAPE), (dict(v=P(1, 2)), L.SV_ERR_SHAPE), (dict(s=P(3, 1)), L.SV_ERR_SHAPE),
    (dict(v=P(0)), L.SV_ERR_PARAM), (dict(i=P(0, 1196)), L.SV_ERR_PARAM), (dict(s=P(0)), L.SV_ERR_PARAM),
    (dict(i=P(1, 56)), L.SV_ERR_PARAM), (dict(s=P(1)), L.SV_ERR_PARAM), (dict(s=P(2, 56)), L.SV_ERR_PARAM),
    (dict(rows=0, x=None, v=None, i=None, s=None), L.SV_OK),
])
def test_top_logits_refusals(kw, code):
    assert top(**kw) == code


def distill(x=P(0), i=P(1), v=P(2), s=P(3), w=P(4), T=1.0, loss=P(5), grad=P(6), rows=3, V=100, k=5, dt=L.SV_BF16):
    return L.lib().sv_distill_loss(x, i, v, s, w, T, loss, grad, rows, V, k, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SV_ERR_SHAPE), (dict(V=0), L.SV_ERR_SHAPE), (dict(V=1048577), L.SV_ERR_SHAPE),
    (dict(k=0), L.SV_ERR_SHAPE), (dict(k=1025), L.SV_ERR_SHAPE), (dict(rows=1 << 22, V=128256), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(T=0.0), L.SV_ERR_PARAM), (dict(T=math.nan), L.SV_ERR_PARAM),
    (dict(T=math.inf), L.SV_ERR_PARAM), (dict(T=1e-39), L.SV_ERR_PARAM),
    (dict(x=None), L.SV_ERR_NULL), (dict(i=None), L.SV_ERR_NULL), (dict(v=None), L.SV_ERR_NULL),
    (dict(loss=None, grad=None), L.SV_ERR_NULL),
    (dict(x=P(0, 1)), L.SV_ERR_SHAPE), (dict(grad=P(6, 1)), L.SV_ERR_SHAPE), (dict(i=P(1, 2)), L.SV_ERR_SHAPE),
    (dict(v=P(2, 2)), L.SV_ERR_SHAPE), (dict(s=P(3, 2)), L.SV_ERR_SHAPE), (dict(w=P(4, 2)), L.SV_ERR_SHAPE),
    (dict(loss=P(5, 2)), L.SV_ERR_SHAPE),
    (dict(grad=P(0, 2)), L.SV_ERR_PARAM), (dict(grad=P(1)), L.SV_ERR_PARAM), (dict(grad=P(2)), L.SV_ERR_PARAM),
    (dict(grad=P(3)), L.SV_ERR_PARAM), (dict(grad=P(4)), L.SV_ERR_PARAM), (dict(grad=P(5)), L.SV_ERR_PARAM),
    (dict(loss=P(0)), L.SV_ERR_PARAM), (dict(loss=P(2)), L.SV_ERR_PARAM), (dict(loss=P(4)), L.SV_ERR_PARAM),
    (dict(x=P(1), grad=P(1)), L.SV_ERR_PARAM),  # in place, over the list as well
    (dict(rows=0, x=None, i=None, v=None, s=None, w=None, loss=None, grad=None), L.SV_OK),
])
def test_distill_loss_refusals(kw, code):
    assert distill(**kw) == code


def test_the_binding_checks_its_arguments_before_any_call():
    b, f, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w = torch.zeros((3, 64), dtype=b), torch.zeros((64,), dtype=b)
    idx, val, one = torch.zeros((3, 4), dtype=i32), torch.zeros((3, 4)), torch.zeros((3,))
    z, odd = torch.zeros((3, 65), dtype=b), torch.zeros((3, 128), dtype=b)[:, ::2]
    typed = [
        lambda: sv.layer_norm(x.half()), lambda: sv.layer_norm(x, w.float()), lambda: sv.layer_norm(x, bias=w.float()),
        lambda: sv.layer_norm(x, residual=x.float()), lambda: sv.layer_norm(x, out_dtype=torch.float16),
        lambda: sv.layer_norm_backward(x.float(), x), lambda: sv.layer_norm_backward(x, x, w.float()),
        lambda: sv.layer_norm_backward(x, x, out_weight=w), lambda: sv.rms_norm_backward(x, x, grad_residual=x.float()),
        lambda: sv.top_logits(x.half(), 2), lambda: sv.top_logits(x, 2, out_index=torch.zeros((3, 2), dtype=torch.int64)),
        lambda: sv.distill_loss(x.half(), idx, val), lambda: sv.distill_loss(x, idx.long(), val),
        lambda: sv.distill_loss(x, idx, val.to(b)), lambda: sv.distill_loss(x, idx, val, top_lse=one.double()),
        lambda: sv.distill_loss(x, idx, val, with_grad=True, out_grad=x.float()),
    ]
    for call in typed:
        with pytest.raises((TypeError, ValueError)):  # whichever argument is looked at first: these are host tensors too
            call()
    shaped = [
        lambda: sv.layer_norm(x, w[:63]), lambda: sv.layer_norm(x, bias=w[:63]), lambda: sv.layer_norm(x, residual=z),
        lambda: sv.layer_norm(x, out_residual=x), lambda: sv.layer_norm(x, out_scale=one),
        lambda: sv.layer_norm(torch.zeros((3, 0))), lambda: sv.layer_norm(torch.zeros(())),
        lambda: sv.layer_norm_backward(z, x), lambda: sv.layer_norm_backward(x, x, w[:63]),
        lambda: sv.layer_norm_backward(x, x, with_weight=False, out_weight=torch.zeros(64)),
        lambda: sv.layer_norm_backward(x, x, with_bias=False, out_bias=torch.zeros(64)),
        lambda: sv.rms_norm_backward(x, x, out_weight=torch.zeros(63)), lambda: sv.rms_norm_backward(x, x, grad_residual=z),
        lambda: sv.top_logits(x, 0), lambda: sv.top_logits(x, 2, out_values=torch.zeros((3, 3))),
        lambda: sv.top_logits(x, 2, with_lse=False, out_lse=one), lambda: sv.top_logits(torch.zeros((3, 0)), 1),
        lambda: sv.top_logits(x, 2 ** 32 + 2),
        lambda: sv.distill_loss(x, idx[:2], val), lambda: sv.distill_loss(x, idx, val[:, :3]),
        lambda: sv.distill_loss(x, idx, val, top_lse=val), lambda: sv.distill_loss(x, idx, val, weight=one[:2]),
        lambda: sv.distill_loss(x, idx, val, with_loss=False), lambda: sv.distill_loss(x, idx, val, out_grad=x),
        lambda: sv.distill_loss(x, idx, val, with_loss=False, with_grad=True, out_loss=one),
        lambda: sv.distill_loss(x, idx[:, :0], val[:, :0]),
        # host tensors
        lambda: sv.layer_norm(x), lambda: sv.layer_norm_backward(x, x), lambda: sv.rms_norm_backward(x, x),
        lambda: sv.top_logits(x, 2), lambda: sv.distill_loss(x, idx, val),
        # strides
        lambda: sv.layer_norm(odd), lambda: sv.layer_norm_backward(odd, odd), lambda: sv.top_logits(odd, 2),
        lambda: sv.distill_loss(odd, idx, val),
    ]
    for call in shaped:
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ oracle's pins

def test_top_logits_oracle():
    v, i, lse = ref.top_logits([1.0, 3.0, -0.0, 3.0, 0.0, -np.inf], 5)
    assert i.tolist() == [1, 3, 0, 2, 4] and v.tolist() == [3.0, 3.0, 1.0, 0.0, 0.0]
    assert abs(lse - math.log(2 * math.exp(3) + math.e + 2)) < 1e-14
    v, i, lse = ref.top_logits([1.0, np.nan, np.inf, np.nan], 4)
    assert i.tolist() == [1, 3, 2, 0] and math.isnan(lse)
    assert ref.top_logits([-np.inf] * 3, 2)[1:] [0].tolist() == [0, 1] and ref.top_logits([-np.inf] * 3, 2)[2] == -np.inf


def test_distill_oracle_in_closed_form():
    # two tokens, the list is both: a plain divergence of two distributions
    loss, g, _ = ref.distill_row([0.0, 0.0], [0, 1], [math.log(3.0), 0.0])
    assert abs(loss - (0.75 * math.log(1.5) + 0.25 * math.log(0.5))) < 1e-15
    assert np.allclose(g, [0.5 - 0.75, 0.5 - 0.25], atol=1e-15)
    # three tokens, one listed with half of the mass, the rest as one outcome of mass 1/2 against 2/3
    loss, g, d = ref.distill_row([0.0, 0.0, 0.0], [1], [0.0], lse=math.log(2.0))
    assert abs(d["r"] - 0.5) < 1e-15 and abs(d["R"] - 2 / 3) < 1e-15
    assert abs(loss - (0.5 * math.log(1.5) + 0.5 * math.log(0.75))) < 1e-15
    assert np.allclose(g, [(2 / 3 - 0.5) / 2, 1 / 3 - 0.5, (2 / 3 - 0.5) / 2], atol=1e-15)
    # the teacher itself: nothing to learn, whatever the list leaves
    s = np.random.default_rng(0).normal(size=50) * 3
    v, i, lse = ref.top_logits(s, 7, 2.0)
    loss, g, _ = ref.distill_row(s, i, v, lse, 2.0)
    assert abs(loss) < 1e-14 and np.max(np.abs(g)) < 1e-14
    for kw in (dict(weight=0.0), dict(lse=-np.inf)):
        loss, g, _ = ref.distill_row(s, i, v, **kw)
        assert loss == 0.0 and not g.any()
    assert ref.distill_row(s, [-1, 50], [1.0, 2.0])[0] == 0.0
    assert ref.distill_row(s, [3], [-np.inf])[0] == 0.0


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T", [0.7, 1.0, 3.0])
def test_distill_oracle_against_differences(rest, T):
    rng = np.random.default_rng(5)
    s, t = rng.normal(size=12) * 2, rng.normal(size=12) * 2
    index = [4, 1, -1, 7, 4, 99]  # a token twice, absent entries
    values = t[[4, 1, 0, 7, 4, 0]].copy()
    values[4] -= 1.0
    lse = ref.log_sum_exp(t / T) if rest else None
    f = lambda z: ref.distill_row(z, index, values, lse, T, 0.3)[0]  # noqa: E731
    _, g, _ = ref.distill_row(s, index, values, lse, T, 0.3)
    for j in range(12):
        e = np.zeros(12)
        e[j] = 1e-5
        assert abs((f(s + e) - f(s - e)) / 2e-5 - g[j]) < 1e-9


@pytest.mark.parametrize("center", [True, False])
def test_norm_backward_oracle_against_differences(center):
    from oracle import last_layer

    rng = np.random.default_rng(6)
    h, dy, w = rng.normal(size=(3, 9)) + 0.5, rng.normal(size=(3, 9)), rng.normal(size=9)
    b, dres = rng.normal(size=9), rng.normal(size=(3, 9))

    def f(h, w, b):
        y = ref.layer_norm(h, w, b, eps=0.01)[0] if center else last_layer.rms_norm(h, w, eps=0.01)[0]
        return np.sum(y * dy) + np.sum(h * dres)

    dh, dw, db = ref.norm_backward(center, dy, h, w, dres, 0.01)
    for j in range(9):
        e = np.zeros(9)
        e[j] = 1e-5
        for i in range(3):
            z = np.zeros((3, 9))
            z[i, j] = 1e-5
            assert abs((f(h + z, w, b) - f(h - z, w, b)) / 2e-5 - dh[i, j]) < 1e-8
        assert abs((f(h, w + e, b) - f(h, w - e, b)) / 2e-5 - dw[j]) < 1e-8
        if center:
            assert abs((f(h, w, b + e) - f(h, w, b - e)) / 2e-5 - db[j]) < 1e-8
