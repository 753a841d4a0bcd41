"""Streaming-block operators on the GPU: ends of the ranges, host threads, autograd and the kernel forms of large calls.

Tolerances are derived as in test_gpu_stream_ops, with u = 2^-24 and an output's rounding of half a step."""
import ctypes
import threading

import numpy as np
import pytest

import oracle
from conformer_speech_recognition_b200 import gam
from test_gpu_stream_ops import (U, _dt, _torch, conv_check, dev, host, inside, linear_check, linear_inputs, norm_check,
                                 normal, scan_call, scan_check, scan_inputs)

pytestmark = pytest.mark.gpu


def test_linear_calls_of_several_threads():
    """The C entry called by host threads with different numbers of rows, each on a stream of its own."""
    torch = _torch()
    n, k, calls = 4104, 6208, 6000                     # just enough weights for the form that sizes its shared memory by the call
    _, _, q, scale, _ = linear_inputs(1, 1, n, k, "bf16", False)
    w, s = dev(gam.gam_quant_linear_pack(q)), dev(scale)
    entry = gam.lib().gam_quant_linear
    jobs = []
    for rows in (1, 8, 1, 8):
        x, _ = normal(np.random.default_rng(rows), rows, k, dtype="bf16")
        jobs.append((x, gam.gam_quant_linear(x, w, s), torch.zeros(rows, n, dtype=x.dtype, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(jobs))

    def work(x, want, y, stream):
        args = (x.data_ptr(), gam.DTYPE_BF16, k, w.data_ptr(), s.data_ptr(), None, 0, len(x), n, k, y.data_ptr(), n,
                ctypes.c_void_p(stream.cuda_stream))
        start.wait()
        for i in range(calls):
            st = entry(*args)
            if st:
                bad.append(st)
            if i % 100 == 99:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, f"{len(bad)} of {len(jobs) * calls} calls failed: {gam.STATUS[bad[0]]}"
    for _, want, y, _ in jobs:
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,n", [(3, 16), (40, 16), (1500, 16), (40, 5)])
def test_scan_nan_rate_reaches_its_channel_only(dtype, T, n):
    """A rate that is NaN makes its channel's outputs NaN from the first valid frame on."""
    torch = _torch()
    t, _ = scan_inputs(31 + T, 2, T, 48, n, dtype)
    ln = dev(np.array([T, T - 1], np.int32))
    clean, end = scan_call(t, ln)
    t["a"] = t["a"].clone()
    t["a"][5, 2] = float("nan")
    y, new = scan_call(t, ln)
    assert bool(torch.isnan(y[0, :, 5]).all()) and bool(torch.isnan(y[1, :T - 1, 5]).all())
    assert bool(torch.isnan(new[:, 5, 2]).all())
    keep = torch.arange(48, device="cuda") != 5
    assert torch.equal(y[..., keep], clean[..., keep]) and torch.equal(new[:, keep], end[:, keep])
    others = torch.arange(n, device="cuda") != 2
    assert torch.equal(new[:, 5, others], end[:, 5, others])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("T", [1, 2, 40, 1500])
def test_scan_infinite_rates_clear_large_states(dtype, T):
    """exp(-inf) and exp(-1e4) are 0: nothing of a state of 1e30 is left."""
    torch = _torch()
    t, _ = scan_inputs(32, 2, T, 24, 16, dtype)
    t["state"] = torch.full_like(t["state"], 1e30)
    t["x"] = torch.zeros_like(t["x"])
    t["a"][:, 1], t["a"][:, 2] = float("-inf"), -1e8
    _, new = scan_call(t)
    assert bool((new[..., 1:3] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 1500])
def test_scan_sequences_without_frames_keep_their_states(dtype, T):
    """Whatever the rates are: NaN here, and 0 times infinity where a step of 0 meets an infinite one."""
    torch = _torch()
    t, _ = scan_inputs(39 + T, 3, T, 48, 16, dtype)
    t["a"] = t["a"].clone()
    t["a"][5, 2], t["a"][6, 3] = float("nan"), float("-inf")
    _, new = scan_call(t, dev(np.array([T, 0, -1], np.int32)))
    assert torch.equal(new[1:], t["state"][1:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 4, 5, 40, 1500])
def test_scan_steps_of_zero_keep_states_of_infinite_rates(dtype, T):
    """An infinite rate stands for the largest finite one, so a step of 0 keeps the state, in prompts and frames alike."""
    torch = _torch()
    t, _ = scan_inputs(33 + T, 2, T, 24, 16, dtype)
    t["a"] = t["a"].clone()
    t["a"][:, 1], t["a"][:, 3] = float("-inf"), float("inf")
    t["dt"], t["dt_bias"] = torch.zeros_like(t["dt"]), None
    y, new = scan_call(t, dt_softplus=False)
    assert torch.equal(new, t["state"]) and bool(torch.isfinite(y).all())
    t["a"][:, 3] = -1.0
    t["dt"] = torch.full_like(t["dt"], -200.0)         # its softplus is below the smallest fp32 number
    y, new = scan_call(t)
    assert torch.equal(new, t["state"]) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,n", [(2, 3, 24, 1), (2, 3, 33, 5), (2, 4, 24, 12), (2, 40, 24, 1), (2, 40, 33, 5), (2, 40, 24, 12),
                                     (1, 700, 24, 5), (1, 700, 24, 12), (2, 40, 24, 16), (2, 40, 24, 33), (64, 20, 1272, 7),
                                     (64, 20, 640, 12)])
def test_scan_infinite_inputs_do_not_depend_on_the_padding_of_n(dtype, B, T, d, n):
    """An infinite x makes its channel's states and outputs infinite from its frame on, whatever n is."""
    torch = _torch()
    t, _ = scan_inputs(34 + T + n, B, T, d, n, dtype, z=False)
    t["b"], t["c"] = t["b"].abs() + 0.25, t["c"].abs() + 0.25
    t["d_skip"] = t["d_skip"].abs() + 0.25
    t["a"] = t["a"].clamp(min=-2.0)                    # no decay is 0
    clean, end = scan_call(t)
    t["x"] = t["x"].clone()
    at = T // 2
    t["x"][0, at, 3] = float("inf")
    y, new = scan_call(t)
    hurt = torch.zeros_like(y, dtype=torch.bool)
    hurt[0, at:, 3] = True
    assert bool((y[hurt] == float("inf")).all()) and torch.equal(y[~hurt], clean[~hurt])
    assert bool((new[0, 3] == float("inf")).all())
    new[0, 3] = end[0, 3]
    assert torch.equal(new, end)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scan_growing_states_of_long_prompts(dtype):
    """Rates above 0: a product of decays may pass fp32's range where the states do not."""
    torch = _torch()
    # states that grow, but are 0 until the last frames
    t, f = scan_inputs(35, 1, 1500, 16, 16, dtype, state=False)
    for name in ("x", "dt", "dt_bias", "a"):
        t[name] = t[name].clone()
    t["x"][:, :-5] = 0
    t["dt"][:], t["dt_bias"][:] = 0.5, 0
    t["a"][:, :3] = 1.0
    f.update({name: host(t[name]) for name in ("x", "dt", "dt_bias", "a")})
    y, new = scan_call(t, dt_softplus=False)
    scan_check(y, new, f, [1500], dtype, softplus=False)
    # a state of 1e-37 that grows by e^93 within 64 frames
    t, f = scan_inputs(36, 1, 512, 16, 16, dtype)
    for name in ("x", "dt", "dt_bias", "a", "state"):
        t[name] = t[name].clone()
    t["x"][:], t["dt"][:], t["dt_bias"][:] = 0, 0, 0
    t["dt"][:, 64:128] = 1.453125
    t["a"][:, 0], t["state"][:] = 1.0, 1e-37
    f.update({name: host(t[name]) for name in ("x", "dt", "dt_bias", "a", "state")})
    y, new = scan_call(t, dt_softplus=False)
    scan_check(y, new, f, [512], dtype, softplus=False)
    assert bool((new[..., 0] > 100).all())
    # an infinite state stays infinite under decays whose product is too small for fp32
    t, _ = scan_inputs(37, 1, 1500, 16, 16, dtype)
    t["x"] = t["x"].clone()
    t["x"][0, 2, 3] = float("inf")
    t["dt"], t["dt_bias"] = torch.full_like(t["dt"], 0.5), None
    _, new = scan_call(t, dt_softplus=False)
    assert bool(torch.isinf(new[0, 3]).all())


# ---- activations in fp32 -------------------------------------------------------------

# v / (1 + e^-v): the hardware's 2^x is within 2^-22 (4 u), the factor that corrects its argument and the product
# with it add u each, the sum u, the hardware's reciprocal 2^-23 (2 u), the last product u: 10 u
GATE = 10 * U


def _swept(dtype, rows, d, lo=-86.0, hi=30.0):
    t = dev(np.linspace(lo, hi, rows * d, dtype=np.float32).reshape(rows, d), _dt(dtype))
    return t, host(t)


def test_conv_swish_keeps_fp32():
    v, f = _swept("f32", 96, 40)
    w = dev(np.tile(np.array([0, 0, 1], np.float32), (40, 1)))
    y, _ = gam.gam_short_conv(v[None], w, act="swish")
    ref = oracle.op_activation(f, "swish")
    inside(y[0], ref, GATE * np.abs(ref))


def test_linear_swish_keeps_fp32():
    """The identity as weights: each product is x or 0."""
    torch = _torch()
    v, f = _swept("f32", 7, 64)
    w, s = dev(gam.gam_quant_linear_pack(np.eye(64, dtype=np.int8))), torch.ones(64, 1, dtype=torch.float16, device="cuda")
    y = gam.gam_quant_linear(v, w, s, act="swish")
    ref = oracle.op_activation(f, "swish")
    inside(y, ref, GATE * np.abs(ref))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["swish", "sigmoid"])
@pytest.mark.parametrize("rows,d", [(5, 64), (7, 201), (3, 1024)])
def test_norm_gate_keeps_fp32(dtype, act, rows, d):
    """x' = 0 + gate: fp32 whatever the gate's type."""
    torch = _torch()
    g, f = _swept(dtype, rows, d)
    x, y = torch.zeros(rows, d, device="cuda"), torch.ones(rows, d, dtype=_dt(dtype), device="cuda")
    xo, _ = gam.gam_residual_norm(x, y, gate=g, gate_act=act)
    ref = oracle.op_activation(f, act)
    inside(xo, ref, GATE * np.abs(ref))


@pytest.mark.parametrize("T,d", [(3, 40), (70, 40), (70, 33)])
def test_scan_gate_keeps_fp32(T, d):
    """No state and a skip of 1: the outputs are swish(z)."""
    torch = _torch()
    z, f = _swept("f32", T, d)
    one, zero = torch.ones(1, T, d, device="cuda"), torch.zeros(1, T, 4, device="cuda")
    y, _ = gam.gam_selective_scan(one, one, -torch.ones(d, 4, device="cuda"), zero, zero, d_skip=torch.ones(d, device="cuda"),
                                  z=z[None])
    ref = oracle.op_activation(f, "swish")
    inside(y[0], ref, GATE * np.abs(ref))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,d", [(2, 2048), (40, 2048), (40, 2047)])
def test_scan_step_sizes_keep_fp32(dtype, T, d):
    """The state after one input of 1 is softplus(dt), fp32 in every type: e^-|v| within 2 steps (4 u), the
    polynomial 3 u with its evaluation, the last product u, and u to spare: 9 u."""
    torch = _torch()
    dt, f = _swept(dtype, 1, d, -80.0, 30.0)
    x = torch.zeros(1, T, d, dtype=dt.dtype, device="cuda")
    x[:, T - 2] = 1
    one = torch.ones(1, T, 1, dtype=dt.dtype, device="cuda")
    _, new = gam.gam_selective_scan(x, dt.expand(1, T, d).contiguous(), torch.zeros(d, 1, device="cuda"), one, one)
    ref = np.logaddexp(0, f[0])
    inside(new[0, :, 0], ref, 9 * U * ref)


# ---- what autograd sees --------------------------------------------------------------

def test_forward_mode_tangents_are_refused():
    torch = _torch()
    import torch.autograd.forward_ad as fwd
    x, y = torch.randn(3, 64, device="cuda"), torch.randn(3, 64, device="cuda")
    w, s = torch.full((8, 32), 0x99, dtype=torch.uint8, device="cuda"), torch.ones(8, 1, dtype=torch.float16, device="cuda")
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: gam.gam_residual_norm(dual, y), lambda: gam.gam_residual_norm(x, dual),
                     lambda: gam.gam_quant_linear(dual, w, s)):
            with pytest.raises(gam.GamError, match="gradient"):
                call()
        gam.gam_residual_norm(fwd.unpack_dual(dual).primal.detach(), y)


def test_lazily_negated_views_are_refused():
    """Such a tensor's memory holds the negated values."""
    torch = _torch()
    z = torch.randn(6, 1, dtype=torch.complex64, device="cuda")
    x = z.conj().imag
    assert x.is_neg()
    with pytest.raises(gam.GamError) as e:
        gam.gam_residual_norm(x, torch.zeros(6, 1, device="cuda"))
    assert e.value.name == "GAM_ERR_INVALID_ARG"
    xo, _ = gam.gam_residual_norm(x.resolve_neg(), torch.zeros(6, 1, device="cuda"))
    assert torch.equal(xo, x)


def test_outputs_count_as_changed():
    """A tensor that a call writes counts one change, so that a backward pass which saved it notices."""
    torch = _torch()
    w = torch.ones(4, 32, device="cuda", requires_grad=True)
    x, y = torch.randn(4, 32, device="cuda"), torch.randn(4, 32, device="cuda")
    loss = (w * x).sum()                               # saves x
    with torch.no_grad():
        gam.gam_residual_norm(x, y, x_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    v = torch.randn(2, 3, 8, device="cuda")
    out, st = torch.empty_like(v), torch.zeros(2, 3, 8, device="cuda")
    before = out._version, st._version, v._version
    gam.gam_short_conv(v, torch.ones(8, 4, device="cuda"), state=st, out=out, state_out=st)
    assert (out._version, st._version, v._version) == (before[0] + 1, before[1] + 1, before[2])
    with torch.inference_mode():                       # these keep no count
        a = torch.randn(4, 32, device="cuda")
        gam.gam_residual_norm(a, torch.randn(4, 32, device="cuda"), x_out=a)


def test_scan_softplus_flag_without_a_truth_value():
    torch = _torch()
    t, _ = scan_inputs(38, 1, 2, 8, 4, "f32")
    with pytest.raises(ValueError):
        scan_call(t, dt_softplus=np.array([True, False]))
    torch.cuda.synchronize()


def test_norm_scale_that_requires_a_gradient_is_refused():
    torch = _torch()
    x, y = torch.randn(3, 32, device="cuda"), torch.randn(3, 32, device="cuda")
    alpha = torch.tensor(0.5, device="cuda", requires_grad=True)
    with pytest.raises(gam.GamError, match="alpha requires a gradient"):
        gam.gam_residual_norm(x, y, alpha=alpha)
    want = gam.gam_residual_norm(x, y, alpha=0.5)
    with torch.no_grad():
        got = gam.gam_residual_norm(x, y, alpha=alpha)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(TypeError):
        gam.gam_residual_norm(x, y, alpha="half")


def test_errors_of_other_calls_are_not_reported():
    """An error that the caller's own CUDA call left behind is not this call's."""
    torch = _torch()
    cudart = ctypes.CDLL("libcudart.so.12")
    x, y, w = torch.randn(3, 64, device="cuda"), torch.randn(3, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    t, _ = scan_inputs(40, 1, 2, 8, 4, "f32")
    t40, _ = scan_inputs(41, 1, 40, 8, 4, "f32")
    q = dev(gam.gam_quant_linear_pack(np.ones((131072, 128), np.int8)))
    s = torch.ones(131072, 2, dtype=torch.float16, device="cuda")
    xq = torch.randn(4, 128, device="cuda")
    calls = (lambda: gam.gam_residual_norm(x, y), lambda: gam.gam_short_conv(x[None], w), lambda: scan_call(t), lambda: scan_call(t40),
             lambda: gam.gam_quant_linear(xq, q, s), lambda: gam.gam_quant_linear(xq, q[:64], s[:64]))
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in calls:
        assert cudart.cudaSetDevice(4096) != 0         # refused on the host, and remembered
        try:
            call()
        finally:
            cudart.cudaGetLastError()
    torch.cuda.synchronize()


# ---- the forms of large calls ---------------------------------------------------------

@pytest.mark.parametrize("xdtype,dtype", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("d,extra,per,gate_act", [
    (64, 0, 1, "swish"), (256, 0, 0, "none"), (512, 0, 7, "tanh"), (500, 0, 1, "sigmoid"), (1000, 0, 0, "none"), (1024, 0, 1, "swish"),
    (62, 0, 1, "sigmoid"), (201, 0, 1, "swish"), (250, 0, 5000, "none"), (201, 2, 0, "none"), (257, 0, 1, "tanh"), (61, 1, 7, "swish"),
    (1024, 8, 1, "sigmoid"), (1040, 0, 0, "none")])
def test_norm_many_rows(xdtype, dtype, d, extra, per, gate_act):
    """Rows enough for warps to walk over several of them: aligned rows, odd ones, rows further apart than d; in place too."""
    torch = _torch()
    rng = np.random.default_rng(d + extra)
    rows = 4998 if per == 7 else 5000

    def make(name, std):
        base = torch.full((rows, d + extra), float("nan"), dtype=_dt(name), device="cuda")
        base[:, :d] = dev((rng.normal(size=(rows, d)) * std).astype(np.float32))
        return base, base[:, :d]
    (bx, x), (by, y) = make(xdtype, 2.0), make(dtype, 1.0)
    kt = {k: dev(rng.normal(size=d).astype(np.float32)) for k in ("post_weight", "post_bias", "pre_weight", "pre_bias", "layer_scale")}
    if per:
        kt["gate"] = dev(rng.normal(size=(rows // per, d)).astype(np.float32), _dt(dtype))
    kw = dict(post="layer", pre="layer", gate_act=gate_act, alpha=0.5)
    xf, yf = x.clone(), y.clone()
    xo, u = gam.gam_residual_norm(x, y, **kw, **kt)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # the first and last rows, some between, and where warps come to their second row
    pick = np.unique(np.r_[0:6, rng.integers(0, rows, 16), [v for v in (k * sms * 4 + i for k in (3, 5, 8) for i in (-1, 0, 1)) if v < rows], rows - 6:rows])
    some = dev(pick.astype(np.int64))
    ref = dict(kw, **{k: host(v) for k, v in kt.items() if k != "gate"})
    if per:
        ref["gate"] = host(kt["gate"].index_select(0, some // per))
    norm_check(xo.index_select(0, some), u.index_select(0, some), host(xf.index_select(0, some)), host(yf.index_select(0, some)),
               xdtype, dtype, ref)
    gam.gam_residual_norm(x, y, x_out=x, out=y, **kw, **kt)
    assert torch.equal(x, xo) and torch.equal(y, u)
    if extra:
        assert bool(torch.isnan(bx[:, d:]).all()) and bool(torch.isnan(by[:, d:]).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,n,z", [
    (64, 40, 1272, 7, True), (64, 40, 1273, 8, False), (64, 50, 640, 16, True), (64, 45, 601, 11, True), (40, 70, 512, 32, False),
    (40, 66, 497, 30, True), (40, 70, 256, 64, True), (40, 67, 243, 50, False)])
def test_scan_many_channels(dtype, B, T, d, n, z):
    """Two channels to a lane, over four tiles of frames and more; ragged."""
    torch = _torch()
    t, f = scan_inputs(B + T + d + n, B, T, d, n, dtype, z=z)
    lens = [T - (i * 5) % (T + 1) for i in range(B)]
    lens[1], lens[2] = 0, 1
    for i, m in enumerate(lens):
        for name in ("x", "dt", "b", "c") + (("z",) if z else ()):
            t[name][i, m:] = float("nan")
    ln = dev(np.array(lens, np.int32))
    y, new = scan_call(t, ln)
    some = [0, 1, 2, 7, B - 1]
    pick = dev(np.array(some, np.int64))
    part = {k: (None if v is None else v[some] if k in ("x", "dt", "b", "c", "z", "state") else v) for k, v in f.items()}
    scan_check(y.index_select(0, pick), new.index_select(0, pick), part, [lens[i] for i in some], dtype)
    # the other sequences: as in a call of their own, which another form serves
    for i in (3, B // 2):
        one = {k: (v if v is None or k in ("a", "d_skip", "dt_bias") else v[i:i + 1]) for k, v in t.items()}
        y1, s1 = scan_call(one, ln[i:i + 1])
        alone = {k: (None if v is None else v[i:i + 1] if k in ("x", "dt", "b", "c", "z", "state") else v) for k, v in f.items()}
        scan_check(y1, s1, alone, [lens[i]], dtype)
        scan_check(y[i:i + 1], new[i:i + 1], alone, [lens[i]], dtype)
    y2, s2 = scan_call(t, ln, state_out=t["state"])
    assert torch.equal(y2, y) and torch.equal(s2, new)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,taps", [(32, 90, 2048, 2), (32, 95, 2048, 3), (32, 90, 2048, 5), (32, 97, 2048, 7), (32, 90, 2048, 8),
                                        (40, 21, 2047, 4), (40, 30, 2047, 6)])
def test_conv_many_rows(dtype, B, T, d, taps):
    """Eight rows of a segment on their way at a time; ragged."""
    torch = _torch()
    rng = np.random.default_rng(T + d + taps)
    x, xf = normal(rng, B, T, d, dtype=dtype)
    s, sf = normal(rng, B, taps - 1, d, dtype=dtype)
    w, b = rng.normal(size=(d, taps)).astype(np.float32), rng.normal(size=d).astype(np.float32)
    lens = [T - (i * 7) % (T + 1) for i in range(B)]
    lens[1], lens[2] = 0, 1
    for i, m in enumerate(lens):
        x[i, m:] = float("nan")
    y, new = gam.gam_short_conv(x, dev(w), bias=dev(b), act="swish", lengths=dev(np.array(lens, np.int32)), state=s)
    some = [0, 1, 2, 9, B - 1]
    pick = dev(np.array(some, np.int64))
    conv_check(y.index_select(0, pick), new.index_select(0, pick), xf[some], w, b, [lens[i] for i in some], sf[some], "swish", dtype,
               True)
    for i in (3, B // 2, B - 2):                       # the other forms give the same bits
        y1, s1 = gam.gam_short_conv(x[i:i + 1], dev(w), bias=dev(b), act="swish", lengths=dev(np.array(lens[i:i + 1], np.int32)),
                                    state=s[i:i + 1])
        assert torch.equal(y1[0], y[i]) and torch.equal(s1[0], new[i])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [24, 40, 64])
def test_linear_many_rows_and_weights(dtype, rows):
    x, xf, q, scale, b = linear_inputs(rows, rows, 4101, 2112, dtype, True)
    y = gam.gam_quant_linear(x, dev(gam.gam_quant_linear_pack(q)), dev(scale), bias=dev(b), act="swish")
    linear_check(y, xf, q, scale, b, "swish", dtype)
