"""Streaming-block operators, host side: the packed INT4 layout, what the calls
refuse before they touch a device, and pins of their oracle against closed forms."""
import ctypes
import struct

import numpy as np
import pytest

import oracle
from conformer_speech_recognition_b200 import gam

P = 1 << 20  # stands for a device address: every call here is refused before it is used


@pytest.fixture(scope="module")
def L():
    from conformer_speech_recognition_b200 import build
    build.build()
    return gam.lib()


def _refused(status, name, text=""):
    assert gam.STATUS[status] == name
    assert text in gam.lib().gam_last_error(None).decode()


# ---- packing -------------------------------------------------------------------

@pytest.mark.parametrize("n,k", [(1, 64), (3, 128), (17, 192)])
def test_pack_round_trip(L, n, k):
    q = np.random.default_rng(n * k).integers(-7, 8, size=(n, k)).astype(np.int8)
    packed = gam.gam_quant_linear_pack(q)
    assert packed.shape == (n, k // 2)
    assert np.array_equal(oracle.unpack_int4(packed), q)


def test_pack_hand_word(L):
    q = np.zeros((1, 64), np.int8)
    q[0, :8] = [-7, -6, -5, -4, 1, 2, 3, 7]          # stored 1 2 3 4 9 10 11 15
    assert bytes(gam.gam_quant_linear_pack(q)[0, :4]) == bytes([0x31, 0xB9, 0x42, 0xFA])
    assert bytes(gam.gam_quant_linear_pack(q)[0, 4:8]) == bytes([0x88] * 4)


def test_pack_refusals(L):
    for bad, name in ((np.full((1, 64), 8, np.int8), "GAM_ERR_WEIGHTS"), (np.full((1, 64), -8, np.int8), "GAM_ERR_WEIGHTS"),
                      (np.zeros((1, 63), np.int8), "GAM_ERR_SHAPE"), (np.zeros((0, 64), np.int8), "GAM_ERR_INVALID_ARG"),
                      (np.zeros((1, 64), np.int32), "GAM_ERR_INVALID_ARG")):
        with pytest.raises(gam.GamError) as e:
            gam.gam_quant_linear_pack(bad)
        assert e.value.name == name


# ---- refusals of the device calls ------------------------------------------------

LINEAR = dict(x=P, dtype=1, ldx=128, packed=P, scale=P, bias=None, act=0, rows=2, n=32, k=128, y=2 * P, ldy=32)


@pytest.mark.parametrize("change,name", [
    (dict(dtype=2), "GAM_ERR_INVALID_ARG"), (dict(dtype=9), "GAM_ERR_INVALID_ARG"), (dict(act=2), "GAM_ERR_INVALID_ARG"),
    (dict(rows=-1), "GAM_ERR_INVALID_ARG"), (dict(rows=65), "GAM_ERR_CAPACITY"), (dict(n=0), "GAM_ERR_INVALID_ARG"),
    (dict(k=100), "GAM_ERR_SHAPE"), (dict(k=0), "GAM_ERR_INVALID_ARG"), (dict(x=None), "GAM_ERR_INVALID_ARG"),
    (dict(packed=None), "GAM_ERR_INVALID_ARG"), (dict(scale=None), "GAM_ERR_INVALID_ARG"),
    (dict(y=None), "GAM_ERR_INVALID_ARG"), (dict(packed=P + 8), "GAM_ERR_INVALID_ARG"), (dict(x=P + 1), "GAM_ERR_INVALID_ARG"),
    (dict(bias=P + 2), "GAM_ERR_INVALID_ARG"), (dict(ldx=127), "GAM_ERR_SHAPE"), (dict(ldy=31), "GAM_ERR_SHAPE"),
    (dict(y=P), "GAM_ERR_INVALID_ARG"), (dict(n=2 ** 30 + 1, ldy=2 ** 31), "GAM_ERR_CAPACITY")])
def test_linear_refusals(L, change, name):
    a = dict(LINEAR, **change)
    _refused(L.gam_quant_linear(*a.values(), None), name)


def test_linear_no_rows(L):
    assert L.gam_quant_linear(*dict(LINEAR, rows=0, x=None, y=None).values(), None) == 0


CONV = dict(x=P, dtype=1, xb=320, xr=32, w=P, bias=None, taps=4, act=1, batch=2, t=10, d=32, lengths=None, si=None,
            so=None, y=2 * P, yb=320, yr=32)


@pytest.mark.parametrize("change,name", [
    (dict(dtype=2), "GAM_ERR_INVALID_ARG"), (dict(act=3), "GAM_ERR_INVALID_ARG"), (dict(taps=1), "GAM_ERR_SHAPE"),
    (dict(taps=9), "GAM_ERR_SHAPE"), (dict(batch=-1), "GAM_ERR_INVALID_ARG"), (dict(t=-1), "GAM_ERR_INVALID_ARG"),
    (dict(d=0), "GAM_ERR_INVALID_ARG"), (dict(x=None), "GAM_ERR_INVALID_ARG"), (dict(w=None), "GAM_ERR_INVALID_ARG"),
    (dict(y=None), "GAM_ERR_INVALID_ARG"), (dict(y=P), "GAM_ERR_INVALID_ARG"), (dict(x=P + 1), "GAM_ERR_INVALID_ARG"),
    (dict(si=P + 1), "GAM_ERR_INVALID_ARG"), (dict(lengths=P + 2), "GAM_ERR_INVALID_ARG"),
    (dict(yr=31), "GAM_ERR_SHAPE"), (dict(yb=319), "GAM_ERR_SHAPE"),
    (dict(t=2 ** 30 + 1), "GAM_ERR_CAPACITY"), (dict(d=2 ** 30 + 1), "GAM_ERR_CAPACITY")])
def test_conv_refusals(L, change, name):
    a = dict(CONV, **change)
    _refused(L.gam_short_conv(*a.values(), None), name)


def test_conv_no_sequences(L):
    assert L.gam_short_conv(*dict(CONV, batch=0).values(), None) == 0


SCAN = dict(x=P, dt=P, a=P, b=P, c=P, d_skip=0, z=0, dt_bias=0, lengths=0, state_in=0, state_out=0, y=2 * P,
            xb=320, xr=32, db=320, dr=32, bb=160, br=16, cb=160, cr=16, zb=0, zr=0, yb=320, yr=32,
            dtype=1, batch=2, t=10, d=32, n=16, softplus=1)


def _scan(L, **change):
    return L.gam_selective_scan(struct.pack("12Q12q6i", *dict(SCAN, **change).values()), None)


@pytest.mark.parametrize("change,name", [
    (dict(dtype=2), "GAM_ERR_INVALID_ARG"), (dict(batch=-1), "GAM_ERR_INVALID_ARG"), (dict(t=-1), "GAM_ERR_INVALID_ARG"),
    (dict(d=0), "GAM_ERR_INVALID_ARG"), (dict(n=0), "GAM_ERR_SHAPE"), (dict(n=65), "GAM_ERR_SHAPE"),
    (dict(x=0), "GAM_ERR_INVALID_ARG"), (dict(dt=0), "GAM_ERR_INVALID_ARG"), (dict(a=0), "GAM_ERR_INVALID_ARG"),
    (dict(b=0), "GAM_ERR_INVALID_ARG"), (dict(c=0), "GAM_ERR_INVALID_ARG"), (dict(y=0), "GAM_ERR_INVALID_ARG"),
    (dict(y=P), "GAM_ERR_INVALID_ARG"), (dict(b=P + 1), "GAM_ERR_INVALID_ARG"), (dict(a=P + 2), "GAM_ERR_INVALID_ARG"),
    (dict(state_in=P + 2), "GAM_ERR_INVALID_ARG"), (dict(yr=31), "GAM_ERR_SHAPE"), (dict(yb=319), "GAM_ERR_SHAPE"),
    (dict(t=2 ** 30 + 1), "GAM_ERR_CAPACITY"), (dict(d=2 ** 30 + 1), "GAM_ERR_CAPACITY")])
def test_scan_refusals(L, change, name):
    _refused(_scan(L, **change), name)


def test_scan_null_and_empty(L):
    _refused(L.gam_selective_scan(None, None), "GAM_ERR_INVALID_ARG")
    assert _scan(L, batch=0) == 0


NORM = dict(x=P, y=2 * P, gate=0, ls=0, pw=0, pb=0, rw=0, rb=0, x_out=P, u=3 * P, xs=64, ys=64, gs=0, xos=64, us=64,
            rows=6, gate_rows=1, x_dtype=0, dtype=1, d=64, gate_act=0, post=1, pre=1, alpha=0.5, eps=1e-5)


def _norm(L, **change):
    return L.gam_residual_norm(struct.pack("10Q7q6i2f", *dict(NORM, **change).values()), None)


@pytest.mark.parametrize("change,name", [
    (dict(dtype=2), "GAM_ERR_INVALID_ARG"), (dict(x_dtype=3), "GAM_ERR_INVALID_ARG"), (dict(post=3), "GAM_ERR_INVALID_ARG"),
    (dict(pre=-1), "GAM_ERR_INVALID_ARG"), (dict(gate_act=4), "GAM_ERR_INVALID_ARG"), (dict(rows=-1), "GAM_ERR_INVALID_ARG"),
    (dict(d=0), "GAM_ERR_INVALID_ARG"), (dict(d=16385, xs=20000, ys=20000, xos=20000, us=20000), "GAM_ERR_CAPACITY"),
    (dict(eps=-1.0), "GAM_ERR_INVALID_ARG"), (dict(eps=float("nan")), "GAM_ERR_INVALID_ARG"), (dict(x=0), "GAM_ERR_INVALID_ARG"),
    (dict(y=0), "GAM_ERR_INVALID_ARG"), (dict(x_out=0, u=0), "GAM_ERR_INVALID_ARG"),
    (dict(gate=4 * P, gate_rows=4, gs=64), "GAM_ERR_SHAPE"), (dict(gate=4 * P, gate_rows=0, gs=64), "GAM_ERR_SHAPE"),
    (dict(gate=4 * P, gate_rows=6, gs=63), "GAM_ERR_SHAPE"), (dict(xs=63), "GAM_ERR_SHAPE"), (dict(us=63), "GAM_ERR_SHAPE"),
    (dict(xos=128), "GAM_ERR_INVALID_ARG"), (dict(u=2 * P, us=128), "GAM_ERR_INVALID_ARG"), (dict(u=P), "GAM_ERR_INVALID_ARG"),
    (dict(x_out=2 * P), "GAM_ERR_INVALID_ARG"), (dict(gate=3 * P, gs=64), "GAM_ERR_INVALID_ARG"),
    (dict(x=P + 2), "GAM_ERR_INVALID_ARG"), (dict(pw=P + 1), "GAM_ERR_INVALID_ARG")])
def test_norm_refusals(L, change, name):
    _refused(_norm(L, **change), name)


def test_norm_null_and_empty(L):
    _refused(L.gam_residual_norm(None, None), "GAM_ERR_INVALID_ARG")
    assert _norm(L, rows=0) == 0


def test_valid_calls_without_a_gpu_report_the_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the addresses here are not memory")
    for status in (L.gam_quant_linear(*LINEAR.values(), None), L.gam_short_conv(*CONV.values(), None), _scan(L), _norm(L)):
        _refused(status, "GAM_ERR_UNSUPPORTED_DEVICE")


def test_binding_refuses_cpu_tensors(L):
    import torch
    x = torch.zeros(2, 64)
    for call in (lambda: gam.gam_quant_linear(x, x, x), lambda: gam.gam_short_conv(x[None], x),
                 lambda: gam.gam_selective_scan(x[None], x, x, x, x), lambda: gam.gam_residual_norm(x, x)):
        with pytest.raises(gam.GamError) as e:
            call()
        assert e.value.name == "GAM_ERR_INVALID_ARG"


# ---- oracle pins ---------------------------------------------------------------

def test_oracle_conv_is_a_causal_correlation():
    rng = np.random.default_rng(3)
    x, w, state = rng.normal(size=(20, 3)), rng.normal(size=(3, 4)), rng.normal(size=(3, 3))
    y, new = oracle.causal_conv(x, w, state=state)
    for c in range(3):
        full = np.convolve(np.concatenate([state[:, c], x[:, c]]), w[c][::-1], "valid")
        assert np.allclose(y[:, c], full, atol=1e-12)
    assert np.array_equal(new, x[-3:])
    # an impulse comes out as the reversed kernel, after it and never before
    e = np.zeros((6, 1))
    e[2] = 1
    y, _ = oracle.causal_conv(e, np.array([[1.0, 2.0, 3.0]]))
    assert np.array_equal(y[:, 0], [0, 0, 3, 2, 1, 0])


def test_oracle_conv_state_carries_over():
    rng = np.random.default_rng(4)
    x, w = rng.normal(size=(11, 2)), rng.normal(size=(2, 5))
    whole, end = oracle.causal_conv(x, w)
    state, parts = None, []
    for lo, hi in ((0, 1), (1, 2), (2, 2), (2, 9), (9, 11)):
        y, state = oracle.causal_conv(x[lo:hi], w, state=state)
        parts.append(y)
    assert np.allclose(np.concatenate(parts), whole, atol=1e-13) and np.array_equal(state, end)


def test_oracle_scan_closed_forms():
    # step 1 (no softplus), a = log 1/2, x = b = c = 1: h_t = 2 - 2^-t
    t = 12
    one = np.ones((t, 1))
    y, h, _, _ = oracle.scan_clip(one, one, np.full((1, 1), np.log(0.5)), one, one, softplus=False)
    assert np.allclose(y[:, 0], 2 - 0.5 ** np.arange(t), atol=1e-14) and np.allclose(h, 2 - 0.5 ** (t - 1))
    # a = 0 sums; the skip term adds x; the gate multiplies by swish(z)
    y, _, _, _ = oracle.scan_clip(one, one, np.zeros((1, 1)), one, one, d_skip=[3.0], z=np.full((t, 1), 2.0), softplus=False)
    assert np.allclose(y[:, 0], (np.arange(1, t + 1) + 3) * 2 / (1 + np.exp(-2)))
    # softplus(0) = log 2 on dt = 1 with bias -1
    _, h, _, _ = oracle.scan_clip(one[:1], one[:1], np.zeros((1, 1)), one[:1], one[:1], dt_bias=[-1.0])
    assert np.allclose(h, np.log(2))


def test_oracle_norms_and_residual():
    rng = np.random.default_rng(5)
    v = rng.normal(size=50) * 3 + 2
    n = oracle.op_norm(v, "layer", eps=0.0)
    assert abs(n.mean()) < 1e-12 and np.isclose((n ** 2).mean(), 1)
    assert np.isclose((oracle.op_norm(v, "rms", eps=0.0) ** 2).mean(), 1)
    assert np.allclose(oracle.op_norm(v, "layer"), oracle.layer_norm(v[None], np.ones(50), np.zeros(50), 1e-5)[0])
    x, u = oracle.residual_norm(v, v, alpha=0.5, pre="none")
    assert np.allclose(x, 1.5 * v) and np.array_equal(x, u)
