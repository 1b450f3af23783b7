"""The operators between a model's last layer and the verification, without a
GPU: refusals of the C ABI (answered before any HIP call), refusals of the
binding, and the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rejection_sampling_verify_09_amd as sv
from oracle import last_layer as ref
from rejection_sampling_verify_09_amd import _lib as L


def P(i):
    """Addresses a terabyte apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) << 40)


def norm(x=P(0), res=P(1), w=P(2), eps=1e-6, out=P(3), scale=P(4), hres=P(5), rows=3, d=64, dt=L.SV_BF16, odt=L.SV_BF16):
    return L.lib().sv_rms_norm(x, res, w, eps, out, scale, hres, rows, d, dt, odt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), L.SV_ERR_SHAPE), (dict(d=0), L.SV_ERR_SHAPE), (dict(d=65537), L.SV_ERR_SHAPE),
    (dict(rows=1 << 23, d=8192), L.SV_ERR_SHAPE),  # more threads than one launch holds
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(dt=7), L.SV_ERR_DTYPE), (dict(odt=3), L.SV_ERR_DTYPE),
    (dict(eps=0.0), L.SV_ERR_PARAM), (dict(eps=-1.0), L.SV_ERR_PARAM), (dict(eps=math.nan), L.SV_ERR_PARAM),
    (dict(eps=math.inf), L.SV_ERR_PARAM),
    (dict(x=None), L.SV_ERR_NULL), (dict(w=None), L.SV_ERR_NULL), (dict(out=None), L.SV_ERR_NULL),
    (dict(res=None), L.SV_ERR_NULL),  # out_residual without a residual
    (dict(odt=L.SV_E4M3, scale=None), L.SV_ERR_NULL),
    (dict(x=ctypes.c_void_p((1 << 40) + 1)), L.SV_ERR_SHAPE),
    (dict(out=ctypes.c_void_p((4 << 40) + 2), odt=L.SV_F32), L.SV_ERR_SHAPE),
    (dict(out=P(0), odt=L.SV_F32), L.SV_ERR_PARAM),            # in place, but of another type
    (dict(out=ctypes.c_void_p((1 << 40) + 2)), L.SV_ERR_PARAM),  # shifted over x
    (dict(hres=P(3)), L.SV_ERR_PARAM), (dict(out=P(2)), L.SV_ERR_PARAM), (dict(hres=P(2)), L.SV_ERR_PARAM),
    (dict(odt=L.SV_E4M3, scale=P(0)), L.SV_ERR_PARAM), (dict(odt=L.SV_E4M3, scale=P(3)), L.SV_ERR_PARAM),
    (dict(odt=L.SV_E4M3, out=P(1)), L.SV_ERR_PARAM),
    (dict(rows=0, x=None, res=None, w=None, out=None, scale=None, hres=None), L.SV_OK),
])
def test_rms_norm_refusals(kw, code):
    assert norm(**kw) == code


def lin(x=P(0), w=P(1), sx=P(2), sw=P(3), bias=P(4), res=P(5), out=P(6), M=3, N=12, K=64, R=4, act=0, dt=L.SV_E4M3,
        odt=L.SV_F32):
    return L.lib().sv_linear(x, w, sx, sw, bias, res, out, M, N, K, R, act, dt, odt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), L.SV_ERR_SHAPE), (dict(N=0), L.SV_ERR_SHAPE), (dict(K=0), L.SV_ERR_SHAPE), (dict(K=96), L.SV_ERR_SHAPE),
    (dict(K=65536 + 64), L.SV_ERR_SHAPE), (dict(R=5), L.SV_ERR_SHAPE), (dict(R=0), L.SV_ERR_SHAPE),
    (dict(M=2 ** 31 - 1, N=2 ** 31 - 1), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_F32), L.SV_ERR_DTYPE), (dict(odt=L.SV_E4M3), L.SV_ERR_DTYPE), (dict(odt=9), L.SV_ERR_DTYPE),
    (dict(act=-1), L.SV_ERR_PARAM), (dict(act=5), L.SV_ERR_PARAM),
    (dict(x=None), L.SV_ERR_NULL), (dict(w=None), L.SV_ERR_NULL), (dict(out=None), L.SV_ERR_NULL),
    (dict(sx=None), L.SV_ERR_NULL), (dict(sw=None), L.SV_ERR_NULL),
    (dict(x=ctypes.c_void_p((1 << 40) + 8)), L.SV_ERR_SHAPE), (dict(w=ctypes.c_void_p((2 << 40) + 4)), L.SV_ERR_SHAPE),
    (dict(out=ctypes.c_void_p((7 << 40) + 2)), L.SV_ERR_SHAPE), (dict(bias=ctypes.c_void_p((5 << 40) + 1)), L.SV_ERR_SHAPE),
    (dict(out=P(0)), L.SV_ERR_PARAM), (dict(out=P(1)), L.SV_ERR_PARAM), (dict(out=P(2)), L.SV_ERR_PARAM),
    (dict(out=P(3)), L.SV_ERR_PARAM), (dict(out=P(4)), L.SV_ERR_PARAM),
    (dict(out=P(5)), L.SV_ERR_PARAM),                                    # over a shared residual
    (dict(out=ctypes.c_void_p((6 << 40) + 4), R=12), L.SV_ERR_PARAM),    # shifted over the residual
    (dict(M=0, x=None, w=None, sx=None, sw=None, out=None), L.SV_OK),
])
def test_linear_refusals(kw, code):
    assert lin(**kw) == code


ADJ = ["logits", "out", "hist", "hlen", "plen", "x", "rep", "freq", "pres", "cub", "btok", "bval", "mask", "midx"]


def adj(B=2, R=3, K=2, seen=0, cap=5, nb=4, mrows=6, V=100, dt=L.SV_F32, **kw):
    p = [kw.get(n, P(i)) for i, n in enumerate(ADJ)]
    return L.lib().sv_adjust_logits(*p, B, R, K, seen, cap, nb, mrows, V, dt, None)


def adjr(B=2, N=3, max_k=2, bonus=1, cap=5, nb=4, mrows=5, V=100, dt=L.SV_F32, cu=P(30), **kw):
    p = [kw.get(n, P(i)) for i, n in enumerate(ADJ)]
    return L.lib().sv_adjust_logits_ragged(*p[:6], cu, *p[6:], B, N, max_k, bonus, cap, nb, mrows, V, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), L.SV_ERR_SHAPE), (dict(R=-1), L.SV_ERR_SHAPE), (dict(K=-1), L.SV_ERR_SHAPE),
    (dict(K=65, R=1), L.SV_ERR_SHAPE), (dict(seen=-1), L.SV_ERR_SHAPE), (dict(seen=1), L.SV_ERR_SHAPE),
    (dict(cap=-1), L.SV_ERR_SHAPE), (dict(cap=(1 << 27) + 1), L.SV_ERR_SHAPE), (dict(nb=-1), L.SV_ERR_SHAPE),
    (dict(mrows=-1), L.SV_ERR_SHAPE), (dict(V=0), L.SV_ERR_SHAPE), (dict(V=2097153), L.SV_ERR_SHAPE),
    (dict(B=1 << 30, V=1 << 20), L.SV_ERR_SHAPE), (dict(mrows=5, midx=None), L.SV_ERR_SHAPE),
    (dict(dt=L.SV_E4M3), L.SV_ERR_DTYPE),
    (dict(logits=None), L.SV_ERR_NULL), (dict(out=None), L.SV_ERR_NULL), (dict(hist=None), L.SV_ERR_NULL),
    (dict(x=None), L.SV_ERR_NULL), (dict(btok=None), L.SV_ERR_NULL), (dict(bval=None), L.SV_ERR_NULL),
    (dict(out=ctypes.c_void_p((1 << 40) + 400)), L.SV_ERR_PARAM),  # shifted over the logits
    (dict(out=P(2)), L.SV_ERR_PARAM), (dict(out=P(6)), L.SV_ERR_PARAM), (dict(out=P(12)), L.SV_ERR_PARAM),
    (dict(logits=ctypes.c_void_p((1 << 40) + 2)), L.SV_ERR_SHAPE),
    (dict(B=0, logits=None, out=None), L.SV_OK), (dict(R=0, mrows=0, logits=None, out=None), L.SV_OK),
])
def test_adjust_refusals(kw, code):
    assert adj(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), L.SV_ERR_SHAPE), (dict(N=5), L.SV_ERR_SHAPE), (dict(max_k=65), L.SV_ERR_SHAPE),
    (dict(bonus=2), L.SV_ERR_PARAM), (dict(cu=None), L.SV_ERR_NULL), (dict(x=None), L.SV_ERR_NULL),
    (dict(out=P(30)), L.SV_ERR_PARAM), (dict(B=0, N=0, cu=None), L.SV_OK),
    (dict(N=0, bonus=0, mrows=0, logits=None, out=None, x=None), L.SV_OK),
])
def test_adjust_ragged_refusals(kw, code):
    assert adjr(**kw) == code


def test_the_binding_checks_its_arguments_before_any_call():
    b, f = torch.bfloat16, torch.float32
    x, w = torch.zeros((3, 64), dtype=b), torch.zeros((10, 64), dtype=b)
    with pytest.raises(TypeError):
        sv.rms_norm(x.half(), w[0])
    with pytest.raises(TypeError):
        sv.rms_norm(x, w[0].float())
    with pytest.raises(TypeError):
        sv.rms_norm(x, w[0], out_dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.rms_norm(x, w[0, :32])
    with pytest.raises(ValueError):
        sv.rms_norm(x, w[0], out_residual=x)
    with pytest.raises(ValueError):
        sv.rms_norm(x, w[0], out_scale=torch.zeros(3))
    with pytest.raises(ValueError):
        sv.rms_norm(x, w[0])  # not on a device
    with pytest.raises(TypeError):
        sv.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        sv.linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        sv.linear(x, w[:, :32])
    with pytest.raises(ValueError):
        sv.linear(x, w, x_scale=torch.zeros(3), weight_scale=torch.zeros(10))
    with pytest.raises(ValueError):
        sv.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        sv.linear(x, w, residual=torch.zeros((3, 3), dtype=b))
    with pytest.raises(ValueError):
        sv.linear(x, w)
    lg = torch.zeros((2, 3, 100))
    with pytest.raises(TypeError):
        sv.adjust_logits(lg.half())
    with pytest.raises(ValueError):
        sv.adjust_logits(lg[0, 0])
    with pytest.raises(ValueError):
        sv.adjust_logits(lg, mask=torch.zeros((5, 4), dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.adjust_logits(lg, mask_index=torch.zeros(6, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.adjust_logits(lg, history_len=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.adjust_logits(lg, cu_num_draft=torch.zeros(3, dtype=torch.int32), max_k=2)
    with pytest.raises(ValueError):
        sv.adjust_logits(lg[:, 0], cu_num_draft=torch.zeros(3, dtype=torch.int32), max_k=2,
                         draft_tokens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        sv.adjust_logits(lg.to(f), bias=(torch.zeros(3, dtype=torch.int64),) * 3)
    with pytest.raises(ValueError):
        sv.adjust_logits(lg)


def test_e4m3_values_agree_with_torch():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(t)) and np.array_equal(v[~np.isnan(v)], t[~np.isnan(t)])
    assert np.nanmax(v) == ref.E4M3_MAX


def test_oracle_norm_and_linear_pins():
    y, h = ref.rms_norm([[3.0, 4.0]], [1.0, 2.0], [[0.0, 0.0]], 0.0 + 12.5 * 3)
    # mean of squares 12.5, plus 37.5: the root of 50
    assert np.allclose(y, [[3 / math.sqrt(50), 8 / math.sqrt(50)]]) and np.array_equal(h, [[3.0, 4.0]])
    assert ref.e4m3_scale(np.array([[0.0, -896.0]]))[0] == 2.0 and ref.e4m3_scale(np.zeros((1, 2)))[0] == ref.FLT_MIN
    out = ref.linear([[1.0, 2.0]], [[1.0, 0.0], [0.0, 1.0], [1.0, 1.0], [-1.0, -1.0]], [0.0, 0.5, 0.0, 0.0],
                     [[10.0, 20.0]], "relu")
    assert np.array_equal(out, [[11.0, 22.5, 13.0, 20.0]])
    v = np.linspace(-6, 6, 41)
    t = torch.from_numpy(v)
    assert np.allclose(ref.activate(v, "silu"), torch.nn.functional.silu(t).numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(ref.activate(v, "gelu"), torch.nn.functional.gelu(t).numpy(), rtol=1e-9, atol=1e-14)
    assert np.allclose(ref.activate(v, "gelu_tanh"), torch.nn.functional.gelu(t, approximate="tanh").numpy(), rtol=1e-9,
                       atol=1e-14)


def test_oracle_adjust_pins():
    row, _, touched = ref.adjust_row([2.0, -2.0, 2.0, 1.0, 0.0], prompt=[0, 1], said=[2, 2, 7], repetition=2.0,
                                     frequency=0.25, presence=0.5, biases=[(3, 1.0), (3, 2.0), (-1, 9.0)],
                                     allowed=np.array([True, True, True, True, False]))
    assert row[:4].tolist() == [1.0, -4.0, 0.0, 4.0] and row[4] == -np.inf
    assert touched.tolist() == [True, True, True, True, False]


def test_sizes_past_32_bits_are_refused_not_cut_off():
    """The C ABI counts in 32 bits; ctypes would pass 2^32 + 3 on as 3."""
    big, b, i32 = (1 << 32) + 3, torch.bfloat16, torch.int32
    x = torch.zeros((1, 64), dtype=b).expand(big, 64)
    with pytest.raises(ValueError, match="32 bits"):
        sv.rms_norm(x, x[0])
    with pytest.raises(ValueError, match="32 bits"):
        sv.linear(x, torch.zeros((10, 64), dtype=b))
    with pytest.raises(ValueError, match="32 bits"):
        sv.linear(torch.zeros((2, 64), dtype=b), x)
    wide = torch.zeros((1, 1)).expand(2, big)
    with pytest.raises(ValueError, match="32 bits"):
        sv.rms_norm(wide, wide[0])
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(wide)
    lg, many = torch.zeros((2, 3, 100)), torch.zeros((1,), dtype=i32).expand(big)
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(lg[:, 0], draft_tokens=torch.zeros((2, 1), dtype=i32), drafts_seen=1 << 32)
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(lg, history=many.expand(2, big), presence_penalty=torch.zeros(2))
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(lg, bias=(torch.zeros(3, dtype=i32), many, many.float()))
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(lg, mask=many[:, None].expand(big, 4), mask_index=torch.zeros(6, dtype=i32))
    with pytest.raises(ValueError, match="32 bits"):
        sv.adjust_logits(lg[:, 0], cu_num_draft=torch.zeros(3, dtype=i32), max_k=1 << 32)


def test_rows_that_the_grid_cannot_count_are_refused():
    assert adj(B=1, R=(1 << 31) - 1, K=0, V=1, midx=P(20), dt=L.SV_BF16) == L.SV_ERR_SHAPE
    assert adj(B=1, R=(1 << 30) + 1, K=0, V=1, midx=P(20), dt=L.SV_BF16) == L.SV_ERR_SHAPE
