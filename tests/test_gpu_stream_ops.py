"""Streaming-block operators on the GPU against their fp64 oracle.

Tolerances are bounds derived from the arithmetic, per element, with u = 2^-24:
an output is rounded once to its type (half a step: eps / 2 of its size), sums are
fp32.  `half_step` is that rounding; the other terms stand at each test."""
import numpy as np
import pytest

import oracle
from conformer_speech_recognition_b200 import gam

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch
    return torch


def _dt(name):
    torch = _torch()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def half_step(ref, dtype):
    """Half a step of `dtype` at the size of ref (of its smallest normal below that)."""
    info = _torch().finfo(dtype)
    return info.eps / 2 * np.maximum(np.abs(ref), info.tiny)


def dev(a, dtype=None):
    t = _torch().from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def normal(rng, *shape, dtype="f32", std=1.0):
    """(CUDA tensor of the type, the same values in fp64)"""
    t = dev((rng.normal(size=shape) * std).astype(np.float32), _dt(dtype))
    return t, host(t)


def inside(got, ref, tol, what=""):
    got, ref, tol = np.broadcast_arrays(host(got) if hasattr(got, "is_cuda") else got, ref, tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"got {got[tuple(np.argwhere(bad)[0])]}, want {ref[tuple(np.argwhere(bad)[0])]}"


# ---- quantised linear ------------------------------------------------------------

def linear_inputs(seed, rows, n, k, dtype, bias):
    rng = np.random.default_rng(seed)
    q = rng.integers(-7, 8, size=(n, k)).astype(np.int8)
    scale = (rng.uniform(0.5, 1.5, size=(n, k // 64)) * 0.25 / k ** 0.5).astype(np.float16)
    b = rng.normal(size=n).astype(np.float32) * 0.1 if bias else None
    x, xf = normal(rng, rows, k, dtype=dtype)
    return x, xf, q, scale, b


def linear_check(y, xf, q, scale, b, act, dtype):
    """The products q x are exact or rounded once; at most 64 + k / 64 + 16 fp32 additions
    follow one another, each off by 2 u (tensor cores may truncate) of the sum of
    magnitudes S; swish has slope at most 1.1 and adds 8 u of its value."""
    k = q.shape[1]
    pre = oracle.quant_linear(xf, q, scale, b)
    S = np.abs(xf) @ np.abs(q * np.repeat(scale.astype(np.float64), 64, axis=1)).T + (0 if b is None else np.abs(b))
    ref = oracle.op_activation(pre, act)
    tol = 1.1 * (80 + k / 64) * 2 * U * S + 8 * U * np.abs(ref)
    inside(y, ref, tol + half_step(np.abs(ref) + tol, _dt(dtype)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,n,k,act,bias", [
    (1, 1, 64, "none", False), (1, 768, 768, "none", True), (2, 17, 192, "swish", True), (5, 1025, 1024, "none", True),
    (7, 31, 64, "none", False), (8, 256, 512, "swish", False), (9, 100, 320, "none", True), (16, 512, 2048, "swish", True),
    (17, 48, 128, "none", False), (33, 130, 448, "swish", True), (64, 257, 4096, "none", True), (1, 4100, 4160, "none", False),
    (3, 16, 16384, "none", True), (11, 2100, 4160, "none", False), (16, 600, 16384, "swish", True),
    (20, 2101, 4160, "none", True), (17, 4801, 128, "swish", True), (9, 33, 8192, "none", False)])
def test_linear(dtype, rows, n, k, act, bias):
    x, xf, q, scale, b = linear_inputs(rows * 1000 + n + k, rows, n, k, dtype, bias)
    y = gam.gam_quant_linear(x, dev(gam.gam_quant_linear_pack(q)), dev(scale), bias=None if b is None else dev(b), act=act)
    assert y.dtype == x.dtype and tuple(y.shape) == (rows, n)
    linear_check(y, xf, q, scale, b, act, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,n,k,act,bias", [
    (1, 16385, 1536, "none", True), (3, 4100, 6208, "swish", True), (8, 4097, 24064, "none", False),
    (7, 37890, 704, "none", True)])
def test_linear_many_weights_few_rows(dtype, rows, n, k, act, bias):
    """Ends of tiles, of runs of groups and of what is held of x; aligned rows, and strided ones at an odd offset."""
    torch = _torch()
    x, xf, q, scale, b = linear_inputs(rows + n + k, rows, n, k, dtype, bias)
    w, s, bd = dev(gam.gam_quant_linear_pack(q)), dev(scale), None if b is None else dev(b)
    y = gam.gam_quant_linear(x, w, s, bias=bd, act=act)
    some = np.r_[0:40, n // 2:n // 2 + 40, n - 300:n]
    linear_check(y[:, dev(some)], xf, q[some], scale[some], None if b is None else b[some], act, dtype)
    xb = torch.full((rows, k + 9), float("nan"), dtype=x.dtype, device="cuda")
    xb[:, 3:3 + k] = x
    yb = torch.full((rows + 2, n + 5), 77.0, dtype=x.dtype, device="cuda")
    yv = yb[1:1 + rows, 1:1 + n]
    gam.gam_quant_linear(xb[:, 3:3 + k], w, s, bias=bd, act=act, out=yv)
    assert torch.equal(yv, y)
    yv.fill_(77.0)
    assert bool((yb == 77.0).all())
    if rows > 1:
        x[1, 5] = float("nan")
        got = gam.gam_quant_linear(x, w, s, bias=bd, act=act)
        assert bool(torch.isnan(got[1]).all()) and torch.equal(got[2:], y[2:]) and torch.equal(got[0], y[0])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_strided_rows_and_untouched_memory(dtype):
    """x and out inside larger buffers at an odd offset: nothing beside out's rows changes."""
    torch = _torch()
    linear_strided(torch, 6, 37, 192, dtype)
    linear_strided(torch, 10, 2051, 4160, dtype)   # weights enough for every form


def linear_strided(torch, rows, n, k, dtype):
    x, xf, q, scale, b = linear_inputs(11, rows, n, k, dtype, True)
    xb = torch.full((rows, k + 9), float("nan"), dtype=x.dtype, device="cuda")
    xv = xb[:, 3:3 + k]
    xv.copy_(x)
    yb = torch.full((rows + 2, n + 5), 77.0, dtype=x.dtype, device="cuda")
    yv = yb[1:1 + rows, 1:1 + n]
    gam.gam_quant_linear(xv, dev(gam.gam_quant_linear_pack(q)), dev(scale), bias=dev(b), out=yv)
    linear_check(yv, xf, q, scale, b, "none", dtype)
    yv.fill_(77.0)
    assert bool((yb == 77.0).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_linear_rows_do_not_touch_one_another(dtype):
    """Infinities and NaN in some rows stay in them; a row of the largest finite values is exact to its scale."""
    torch = _torch()
    rows, n, k = 10, 40, 256
    x, xf, q, scale, b = linear_inputs(12, rows, n, k, dtype, False)
    w, s = dev(gam.gam_quant_linear_pack(q)), dev(scale)
    clean = gam.gam_quant_linear(x, w, s)
    dirty = x.clone()
    dirty[2, 5], dirty[4, 100], dirty[9, 255] = float("inf"), float("nan"), float("-inf")
    got = gam.gam_quant_linear(dirty, w, s)
    keep = [i for i in range(rows) if i not in (2, 4, 9)]
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[4]).all())
    # an infinity times weight q: +-inf by its sign, NaN where q is 0
    for row, col, sign in ((2, 5, 1), (9, 255, -1)):
        ref = np.where(q[:, col] == 0, np.nan, sign * np.sign(q[:, col] + 0.5 * (q[:, col] == 0)) * np.inf)
        assert np.array_equal(host(got[row]), ref, equal_nan=True)
    if dtype == "f32":
        big = torch.full((1, k), 3.0e38, device="cuda")
        big[0, 1:] = 0
        ref = 3.0000000054977558e38 * q[:, 0].astype(np.float64) * scale[:, 0].astype(np.float64)
        inside(gam.gam_quant_linear(big, w, s), ref, 4 * U * np.abs(ref))


def test_linear_no_rows_and_repeats():
    torch = _torch()
    x, _, q, scale, _ = linear_inputs(13, 64, 300, 1024, "bf16", False)
    w, s = dev(gam.gam_quant_linear_pack(q)), dev(scale)
    assert gam.gam_quant_linear(x[:0], w, s).shape == (0, 300)
    first = gam.gam_quant_linear(x, w, s)
    for _ in range(3):
        assert torch.equal(gam.gam_quant_linear(x, w, s), first)
    with pytest.raises(gam.GamError) as e:
        gam.gam_quant_linear(torch.zeros(65, 1024, dtype=torch.bfloat16, device="cuda"), w, s)
    assert e.value.name == "GAM_ERR_CAPACITY"


# ---- short convolution -------------------------------------------------------------

def conv_check(y, new, xf, w, b, lens, sf, act, dtype, exact_state):
    """taps + 1 fp32 fused multiply-adds, each off by u of the magnitudes' sum; swish as above."""
    B, T, d = xf.shape
    taps = w.shape[1]
    for i in range(B):
        n = min(max(int(lens[i]), 0), T)
        st = None if sf is None else sf[i]
        pre, state = oracle.causal_conv(xf[i, :n], w, b, st)
        mag, _ = oracle.causal_conv(np.abs(xf[i, :n]), np.abs(w), None if b is None else np.abs(b),
                                    None if st is None else np.abs(st))
        ref = oracle.op_activation(pre, act)
        tol = 1.1 * (taps + 1) * U * mag + 8 * U * np.abs(ref)
        inside(y[i, :n], ref, tol + half_step(np.abs(ref) + tol, _dt(dtype)), f"sequence {i}")
        assert bool((y[i, n:] == 0).all())
        assert np.array_equal(host(new[i]), state), f"state {i}"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,taps,act,bias,state,lens", [
    (1, 1, 64, 4, "swish", True, True, None), (3, 1, 7, 2, "none", False, False, None), (2, 2, 16, 8, "swish", True, True, None),
    (1, 130, 8, 3, "none", True, False, None), (5, 37, 40, 4, "swish", True, True, [37, 0, 1, 2, 36]),
    (4, 100, 33, 5, "none", False, True, [100, 17, 16, 3]), (2, 65, 1032, 6, "swish", True, False, [65, -3]),
    (2, 29, 24, 7, "swish", False, True, [1000, 5]), (64, 1, 256, 4, "swish", True, True, [i % 2 for i in range(64)]),
    (1, 3001, 24, 4, "none", True, True, [2999]), (3, 9, 40, 8, "none", True, True, [9, 3, 8]),
    (40, 50, 2048, 4, "swish", True, True, [(i * 7) % 51 for i in range(40)])])
def test_conv(dtype, B, T, d, taps, act, bias, state, lens):
    rng = np.random.default_rng(B * 100 + T + d + taps)
    x, xf = normal(rng, B, T, d, dtype=dtype)
    w = rng.normal(size=(d, taps)).astype(np.float32)
    b = rng.normal(size=d).astype(np.float32) if bias else None
    s, sf = normal(rng, B, taps - 1, d, dtype=dtype) if state else (None, None)
    if lens is not None:                       # frames behind the end are never read
        for i, n in enumerate(lens):
            x[i, max(n, 0):] = float("nan")
    ln = None if lens is None else dev(np.array(lens, np.int32))
    y, new = gam.gam_short_conv(x, dev(w), bias=None if b is None else dev(b), act=act, lengths=ln, state=s)
    conv_check(y, new, xf, w, b, [T] * B if lens is None else lens, sf, act, dtype, state)
    if state:                                  # the state may be updated in place
        y2, new2 = gam.gam_short_conv(x, dev(w), bias=None if b is None else dev(b), act=act, lengths=ln, state=s, state_out=s)
        assert new2 is s and _torch().equal(s, new) and _torch().equal(y2, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_strides_and_frame_by_frame(dtype):
    """Channels inside a wider row at an odd offset, time-major output; frames one at a time give the same bits."""
    torch = _torch()
    rng = np.random.default_rng(5)
    B, T, d, taps = 3, 11, 20, 4
    wide, wf = normal(rng, B, T, 2 * d + 3, dtype=dtype)
    x, xf = wide[..., 3:3 + d], wf[..., 3:3 + d]
    w = rng.normal(size=(d, taps)).astype(np.float32)
    out = torch.full((T, B, d + 1), 5.0, dtype=x.dtype, device="cuda")
    y, new = gam.gam_short_conv(x, dev(w), act="none", out=out.transpose(0, 1)[..., :d])
    conv_check(y, new, xf, w, None, [T] * B, None, "none", dtype, False)
    assert bool((out[..., d] == 5.0).all())
    state = torch.zeros(B, taps - 1, d, dtype=x.dtype, device="cuda")
    for t in range(T):
        step, _ = gam.gam_short_conv(x[:, t:t + 1], dev(w), act="none", state=state, state_out=state)
        assert torch.equal(step[:, 0], y[:, t])
    assert torch.equal(state, new)


def test_conv_no_frames_hands_the_state_on():
    torch = _torch()
    s = torch.randn(2, 3, 8, device="cuda")
    y, new = gam.gam_short_conv(torch.empty(2, 0, 8, device="cuda"), torch.randn(8, 4, device="cuda"), state=s)
    assert y.shape == (2, 0, 8) and torch.equal(new, s)


# ---- selective scan ----------------------------------------------------------------

def scan_inputs(seed, B, T, d, n, dtype, z=True, state=True, steps=(0.001, 0.1)):
    rng = np.random.default_rng(seed)
    f = {}
    t = {}
    for name, shape in (("x", (B, T, d)), ("z", (B, T, d)), ("b", (B, T, n)), ("c", (B, T, n))):
        t[name], f[name] = normal(rng, *shape, dtype=dtype)
    t["dt"], f["dt"] = normal(rng, B, T, d, dtype=dtype, std=0.5)
    step = np.exp(rng.uniform(np.log(steps[0]), np.log(steps[1]), size=d))
    for name, v in (("dt_bias", step + np.log(-np.expm1(-step))), ("d_skip", rng.normal(size=d)),
                    ("a", -np.arange(1, n + 1) * rng.uniform(0.5, 1.5, size=(d, n)))):
        t[name] = dev(v.astype(np.float32))
        f[name] = host(t[name])
    if not z:
        t["z"] = f["z"] = None
    t["state"], f["state"] = normal(rng, B, d, n) if state else (None, None)
    return t, f


def scan_check(y, new, f, lens, dtype, softplus=True):
    B, T, d = f["x"].shape
    for i in range(B):
        m = min(max(int(lens[i]), 0), T)
        ref, h, ey, eh = oracle.scan_clip(f["x"][i, :m], f["dt"][i, :m], f["a"], f["b"][i, :m], f["c"][i, :m], f["d_skip"],
                                          None if f["z"] is None else f["z"][i, :m], f["dt_bias"], softplus,
                                          None if f["state"] is None else f["state"][i])
        tol = 2 * ey                            # twice: an evaluation joined from pieces of the time axis
        inside(y[i, :m], ref, tol + half_step(np.abs(ref) + tol, _dt(dtype)), f"sequence {i}")
        assert bool((y[i, m:] == 0).all())
        inside(new[i], h, 2 * eh + U * np.abs(h), f"state {i}")


def scan_call(t, lengths=None, **more):
    return gam.gam_selective_scan(t["x"], t["dt"], t["a"], t["b"], t["c"], d_skip=t["d_skip"], z=t["z"],
                                  dt_bias=t["dt_bias"], state=t["state"], lengths=lengths, **more)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,n,z,state,lens", [
    (1, 1, 1, 1, True, True, None), (2, 1, 64, 16, True, True, None), (3, 1, 33, 5, False, True, [1, 0, 1]),
    (1, 2, 40, 8, True, False, None), (2, 17, 65, 3, True, True, [17, 9]), (5, 40, 24, 16, True, True, [40, 0, 1, 39, 16]),
    (2, 33, 130, 12, False, False, [33, 32]), (1, 300, 48, 32, True, True, None), (2, 70, 17, 64, True, True, [70, 1000]),
    (2, 130, 96, 33, False, True, [-5, 129]), (1, 1500, 16, 16, True, True, [1499]), (64, 3, 64, 16, True, True, None),
    (1, 700, 200, 20, True, False, None), (1, 900, 37, 9, True, True, [801]), (2, 640, 8, 64, False, True, [640, 3]),
    (1, 520, 24, 5, True, True, None), (40, 9, 1024, 16, True, True, [i % 10 for i in range(40)])])
def test_scan(dtype, B, T, d, n, z, state, lens):
    torch = _torch()
    t, f = scan_inputs(B * 31 + T + d + n, B, T, d, n, dtype, z, state)
    if lens is not None:                       # frames behind the end are never read
        for i, m in enumerate(lens):
            for name in ("x", "dt", "b", "c") + (("z",) if z else ()):
                t[name][i, max(m, 0):] = float("nan")
    ln = None if lens is None else dev(np.array(lens, np.int32))
    y, new = scan_call(t, ln)
    scan_check(y, new, f, [T] * B if lens is None else lens, dtype)
    y2, _ = scan_call(t, ln)
    assert torch.equal(y, y2)
    if state:
        y3, s3 = scan_call(t, ln, state_out=t["state"])
        assert s3 is t["state"] and torch.equal(s3, new) and torch.equal(y3, y)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_scan_without_softplus_and_large_steps(dtype):
    """Step sizes given as they are, and softplus of values where its naive form overflows or vanishes."""
    t, f = scan_inputs(7, 2, 40, 48, 16, dtype)
    t["dt"], f["dt"] = t["dt"].abs(), np.abs(f["dt"])
    t["dt_bias"], f["dt_bias"] = None, np.zeros(48)
    y, new = scan_call(t, dt_softplus=False)
    scan_check(y, new, f, [40, 40], dtype, softplus=False)
    t, f = scan_inputs(8, 1, 24, 32, 4, dtype)
    scale = np.linspace(-200, 200, 24)[None, :, None] * np.ones((1, 24, 32))
    t["dt"] = dev(scale.astype(np.float32), _dt(dtype))
    f["dt"] = host(t["dt"])
    y, new = scan_call(t)
    scan_check(y, new, f, [24], dtype)
    assert bool(_torch().isfinite(y).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_strides_and_pieces(dtype):
    """b, c and dt as slices of one projection, x and z as halves of another; a prompt in pieces, down to
    single frames, continues from its state."""
    torch = _torch()
    B, T, d, n = 2, 37, 30, 16
    t, f = scan_inputs(9, B, T, d, n, dtype)
    proj = torch.cat([t["dt"], t["b"], t["c"], t["x"][..., :1]], -1)
    t["dt"], t["b"], t["c"] = proj[..., :d], proj[..., d:d + n], proj[..., d + n:d + 2 * n]
    xz = torch.cat([t["x"][..., :1], t["x"], t["z"]], -1)
    t["x"], t["z"] = xz[..., 1:1 + d], xz[..., 1 + d:]
    whole, end = scan_call(t)
    scan_check(whole, end, f, [T] * B, dtype)
    state, parts = t["state"], []
    for lo, hi in ((0, 20), (20, 21), (21, 22), (22, 22), (22, 37)):
        part = dict(t, state=state, **{k: t[k][:, lo:hi] for k in ("x", "dt", "b", "c", "z")})
        y, state = scan_call(part)
        parts.append(y)
    scan_check(torch.cat(parts, 1), state, f, [T] * B, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,d,n", [(3, 1, 33, 5), (2, 60, 40, 16), (1, 1500, 16, 16), (40, 9, 1024, 16)])
def test_scan_steps_of_zero_keep_the_state(dtype, B, T, d, n):
    """A decay of 2^0 is 1 and an input of weight 0 is 0: such channels end with the state they began with, bit for bit."""
    torch = _torch()
    t, _ = scan_inputs(12 + T, B, T, d, n, dtype)
    t["dt"], t["dt_bias"] = t["dt"].abs(), None
    t["dt"][..., ::3] = 0
    _, new = scan_call(t, dt_softplus=False)
    assert torch.equal(new[:, ::3], t["state"][:, ::3]) and not torch.equal(new, t["state"])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("B,T,d,n", [(2, 3, 24, 8), (3, 70, 24, 8), (1, 1500, 16, 16), (40, 9, 1024, 16)])
def test_scan_infinite_rates_forget_their_state(dtype, B, T, d, n):
    """exp(s a) is 0 for a = -inf: such a state is its last frame's input, in ragged sequences too."""
    torch = _torch()
    t, f = scan_inputs(21 + T, B, T, d, n, dtype)
    t["a"][:, 1] = float("-inf")
    lens = [T - i % 3 for i in range(B)]
    t["c"][..., 1] = 0
    y, new = scan_call(t, dev(np.array(lens, np.int32)))
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(new).all())
    f["a"][:, 1], f["c"][..., 1] = -1e30, 0
    scan_check(y, new, f, lens, dtype)


def test_scan_no_frames_hands_the_state_on():
    torch = _torch()
    t, _ = scan_inputs(10, 2, 1, 24, 7, "f32")
    t = dict(t, **{k: t[k][:, :0] for k in ("x", "dt", "b", "c", "z")})
    y, new = scan_call(t)
    assert y.shape == (2, 0, 24) and torch.equal(new, t["state"])


def test_scan_nan_stays_in_its_channel_and_sequence():
    torch = _torch()
    t, _ = scan_inputs(11, 3, 50, 40, 16, "bf16")
    clean, _ = scan_call(t)
    t["x"] = t["x"].clone()
    t["x"][1, 20, 7] = float("nan")
    y, new = scan_call(t)
    hurt = torch.zeros_like(y, dtype=torch.bool)
    hurt[1, 20:, 7] = True
    assert bool(torch.isnan(y[hurt]).all()) and torch.equal(y[~hurt], clean[~hurt])


def test_offsets_past_32_bits():
    """Sequences more than 2^31 elements apart."""
    torch = _torch()
    far = 2 ** 31 + 12345
    t, f = scan_inputs(12, 2, 3, 16, 8, "f16")
    big = torch.empty(far + 64, dtype=torch.float16, device="cuda")
    def spread(v):
        w = big.as_strided(tuple(v.shape), (far, v.shape[2], 1))
        w.copy_(v)
        return w
    t["x"] = spread(t["x"])
    out = torch.empty(far + 64, dtype=torch.float16, device="cuda").as_strided((2, 3, 16), (far, 16, 1))
    y, new = scan_call(t, out=out)
    scan_check(y, new, f, [3, 3], "f16")
    w = np.random.default_rng(1).normal(size=(16, 4)).astype(np.float32)
    y, new = gam.gam_short_conv(t["x"], dev(w), act="none", out=out)
    conv_check(y, new, f["x"], w, None, [3, 3], None, "none", "f16", False)
    x = big.as_strided((2, 16), (far, 1))
    xo, u = gam.gam_residual_norm(x, x.clone(), out=out[:, 0])
    norm_check(xo, u, host(x), host(x.clone()), "f16", "f16", dict(alpha=1.0))


# ---- residual update with norms ------------------------------------------------------

def norm_sens(v, e, kind, weight, bias, eps, A=64):
    """Error of an fp32 norm of v given off by e: a sum of at most A additions in a row is off
    by A u of the magnitudes; then the first-order terms of the formula."""
    if kind == "none":
        return e
    w = 1.0 if weight is None else np.abs(weight)
    m = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    em = (np.abs(v).mean(-1, keepdims=True) * A * U + e.mean(-1, keepdims=True)) if kind == "layer" else 0.0
    c = v - m
    ec = e + em + U * np.abs(c)
    ms = (c * c).mean(-1, keepdims=True)
    r = 1 / np.sqrt(ms + eps)
    ems = 2 * (np.abs(c) * ec).mean(-1, keepdims=True) + (ec * ec).mean(-1, keepdims=True) + A * U * ms
    er = 0.5 * ems / (ms + eps) + 4 * U       # relative
    out = c * r * (1.0 if weight is None else weight)
    return w * r * ec + np.abs(out) * er + 3 * U * np.abs(out) + U * (0 if bias is None else np.abs(bias))


def norm_check(xo, u, xf, yf, xdtype, dtype, kw):
    rows, d = xf.shape
    g = kw.get("gate")
    per = rows // g.shape[0] if g is not None else 1
    post, pre, eps, alpha = kw.get("post", "none"), kw.get("pre", "layer"), kw.get("eps", 1e-5), kw.get("alpha", 1.0)
    refs = [oracle.residual_norm(xf[i], yf[i], alpha, kw.get("layer_scale"), None if g is None else g[i // per],
                                 kw.get("gate_act", "none"), post, kw.get("post_weight"), kw.get("post_bias"), pre,
                                 kw.get("pre_weight"), kw.get("pre_bias"), eps) for i in range(rows)]
    rx, ru = np.stack([r[0] for r in refs]), np.stack([r[1] for r in refs])
    gate = 1.0 if g is None else oracle.op_activation(np.repeat(g, per, 0), kw.get("gate_act", "none"))
    factor = np.abs(alpha * gate * (1.0 if kw.get("layer_scale") is None else kw["layer_scale"]))
    ex = factor * norm_sens(yf, np.zeros_like(yf), post, kw.get("post_weight"), kw.get("post_bias"), eps)
    ex = ex + 12 * U * np.abs(rx - xf) + U * np.abs(rx)       # gate's activation, the products, the addition
    inside(xo, rx, ex + half_step(np.abs(rx) + ex, _dt(xdtype)), "x_out")
    eu = norm_sens(rx, ex, pre, kw.get("pre_weight"), kw.get("pre_bias"), eps)
    inside(u, ru, 1.01 * eu + half_step(np.abs(ru) + eu, _dt(dtype)), "u")


@pytest.mark.parametrize("xdtype,dtype", [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,d,post,pre,gates,gate_act,ls,alpha", [
    (1, 1, "rms", "layer", 1, "tanh", True, 1.0), (1, 1024, "layer", "layer", 1, "sigmoid", False, 0.5),
    (3, 7, "none", "rms", 0, "none", False, 1.0), (9, 64, "layer", "rms", 3, "swish", True, 0.5),
    (5, 257, "rms", "layer", 5, "none", True, -2.0), (13, 768, "layer", "layer", 0, "none", False, 0.5),
    (4, 1000, "rms", "rms", 1, "sigmoid", True, 1.0), (3, 1030, "layer", "layer", 3, "tanh", False, 0.5),
    (7, 2048, "rms", "none", 7, "swish", True, 1.0), (2, 4099, "rms", "rms", 2, "swish", True, 0.5),
    (3, 4104, "layer", "layer", 1, "sigmoid", True, 0.25), (2, 8192, "layer", "layer", 0, "none", False, 0.5),
    (2, 16384, "rms", "layer", 2, "none", True, 0.5), (1, 16383, "layer", "rms", 1, "tanh", False, 0.5)])
def test_norm(xdtype, dtype, rows, d, post, pre, gates, gate_act, ls, alpha):
    torch = _torch()
    rng = np.random.default_rng(rows * 7 + d)
    x, xf = normal(rng, rows, d, dtype=xdtype, std=2.0)
    y, yf = normal(rng, rows, d, dtype=dtype)
    kw, kt = dict(post=post, pre=pre, gate_act=gate_act, alpha=alpha), {}
    for name, on in (("post_weight", post != "none"), ("post_bias", post == "layer"), ("pre_weight", pre != "none"),
                     ("pre_bias", pre == "layer"), ("layer_scale", ls)):
        if on:
            kt[name], kw[name] = normal(rng, d)
    if gates:
        kt["gate"], kw["gate"] = normal(rng, gates, d, dtype=dtype)
    call = {**{k: v for k, v in kw.items() if isinstance(v, (str, float))}, **kt}
    xo, u = gam.gam_residual_norm(x, y, **call)
    norm_check(xo, u, xf, yf, xdtype, dtype, kw)
    x2, u2 = gam.gam_residual_norm(x, y, x_out=x, out=y, **call)          # both in place
    assert x2 is x and u2 is y and torch.equal(x, xo) and torch.equal(y, u)


def test_norm_strides_odd_offsets_and_untouched_memory():
    torch = _torch()
    rng = np.random.default_rng(3)
    rows, d = 6, 72
    for off, extra in ((0, 8), (1, 5), (8, 16)):
        bx = torch.full((rows, d + off + extra), float("nan"), device="cuda")
        by = torch.full((rows, d + off + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
        bu = torch.full((rows + 2, d + off + extra), 9.0, dtype=torch.bfloat16, device="cuda")
        x, y, u = bx[:, off:off + d], by[:, off:off + d], bu[1:-1, off:off + d]
        x.copy_(dev(rng.normal(size=(rows, d)).astype(np.float32)))
        y.copy_(dev(rng.normal(size=(rows, d)).astype(np.float32)))
        xf, yf = host(x), host(y)
        xo, _ = gam.gam_residual_norm(x, y, alpha=0.5, post="rms", pre="layer", out=u)
        norm_check(xo, u, xf, yf, "f32", "bf16", dict(alpha=0.5, post="rms", pre="layer"))
        u.fill_(9.0)
        assert bool((bu == 9.0).all())


def test_norm_constant_and_zero_rows():
    """A row without variance leaves sqrt(eps) in the denominator: finite, and zero for LayerNorm."""
    torch = _torch()
    x = torch.zeros(3, 512, device="cuda")
    y = torch.full((3, 512), 4.0, device="cuda")
    y[1] = 0
    xo, u = gam.gam_residual_norm(x, y, post="layer", pre="rms")
    assert bool((xo == 0).all()) and bool((u == 0).all())
    xo, u = gam.gam_residual_norm(x, y, post="none", pre="layer")
    assert torch.equal(xo, y) and bool((u == 0).all())


def test_norm_large_mean():
    """The variance is taken around the mean: a mean 1000 times the deviation keeps its digits."""
    rng = np.random.default_rng(4)
    x, xf = normal(rng, 4, 1024)
    y = dev((1000 + rng.normal(size=(4, 1024))).astype(np.float32))
    xo, u = gam.gam_residual_norm(x * 0, y, post="layer", pre="layer")
    norm_check(xo, u, xf * 0, host(y), "f32", "f32", dict(post="layer", pre="layer"))


def test_norm_refuses_bad_gates():
    torch = _torch()
    x = torch.zeros(6, 64, device="cuda")
    with pytest.raises(gam.GamError) as e:
        gam.gam_residual_norm(x, x.clone(), gate=torch.zeros(4, 64, device="cuda"))
    assert e.value.name == "GAM_ERR_SHAPE"
    with pytest.raises(gam.GamError) as e:
        gam.gam_residual_norm(x, x.clone(), gate=torch.zeros(6, 64, dtype=torch.float16, device="cuda"))
    assert e.value.name == "GAM_ERR_INVALID_ARG"


# ---- the operators together -----------------------------------------------------------

class Block:
    """A state-space block on the framework's INT4-g64 weights: norm -> in-projection (x, z) -> causal
    convolution -> projection to (step rank, b, c) -> step projection -> scan -> out-projection ->
    half-weight residual with the branch's norm, and the next block's norm."""

    def __init__(self, seed, d=128, inner=256, rank=64, n=16, taps=4):
        rng = np.random.default_rng(seed)
        self.d, self.inner, self.rank, self.n, self.taps = d, inner, rank, n, taps
        self.w = {}
        for name, o, i in (("in", 2 * inner, d), ("proj", rank + 2 * n, inner), ("step", inner, rank), ("out", d, inner)):
            q = rng.integers(-7, 8, size=(o, i)).astype(np.int8)
            s = (rng.uniform(0.5, 1.5, size=(o, i // 64)) * 0.25 / i ** 0.5).astype(np.float16)
            self.w[name] = (dev(gam.gam_quant_linear_pack(q)), dev(s), q, s)
        f32 = np.float32
        step = np.exp(rng.uniform(-6, -2, size=inner))
        self.p = dict(conv=rng.normal(size=(inner, taps)).astype(f32) / 2, conv_b=rng.normal(size=inner).astype(f32) * 0.1,
                      a=(-np.arange(1, n + 1) * rng.uniform(0.5, 1.5, size=(inner, n))).astype(f32),
                      skip=np.ones(inner, f32), dt_bias=(step + np.log(-np.expm1(-step))).astype(f32),
                      post=1 + 0.1 * rng.normal(size=d).astype(f32), pre=1 + 0.1 * rng.normal(size=d).astype(f32),
                      pre_b=0.1 * rng.normal(size=d).astype(f32))
        self.t = {k: dev(v) for k, v in self.p.items()}

    def states(self, batch, dtype):
        torch = _torch()
        return (torch.zeros(batch, self.taps - 1, self.inner, dtype=dtype, device="cuda"),
                torch.zeros(batch, self.inner, self.n, device="cuda"))

    def linear(self, name, x, **kw):
        """Rows in calls of at most 64."""
        torch = _torch()
        w, s = self.w[name][:2]
        flat = x.reshape(-1, x.shape[-1])
        out = torch.empty(flat.shape[0], w.shape[0], dtype=x.dtype, device="cuda")
        for i in range(0, flat.shape[0], 64):
            gam.gam_quant_linear(flat[i:i + 64], w, s, out=out[i:i + 64], **kw)
        return out.view(*x.shape[:-1], -1)

    def __call__(self, x, u, states, lengths=None):
        """x fp32 [batch, t, d] residual, u its norm; the states are updated in place."""
        t, r, n = self.t, self.rank, self.n
        xz = self.linear("in", u)
        v, _ = gam.gam_short_conv(xz[..., :self.inner], t["conv"], bias=t["conv_b"], act="swish", lengths=lengths,
                                  state=states[0], state_out=states[0])
        pr = self.linear("proj", v)
        dt = self.linear("step", pr[..., :r])
        y, _ = gam.gam_selective_scan(v, dt, t["a"], pr[..., r:r + n], pr[..., r + n:], d_skip=t["skip"],
                                      z=xz[..., self.inner:], dt_bias=t["dt_bias"], lengths=lengths, state=states[1],
                                      state_out=states[1])
        o = self.linear("out", y)
        xo, uo = gam.gam_residual_norm(x.reshape(-1, self.d), o.reshape(-1, self.d), alpha=0.5, post="rms",
                                       post_weight=t["post"], pre="layer", pre_weight=t["pre"], pre_bias=t["pre_b"])
        return xo.view_as(x), uo.view_as(u)

    def oracle(self, x, u):
        """One sequence, fp64: x, u [t, d]."""
        p, r, n = self.p, self.rank, self.n
        lin = lambda name, v: oracle.quant_linear(v, *self.w[name][2:])  # noqa: E731
        xz = lin("in", u)
        v, conv = oracle.causal_conv(xz[:, :self.inner], p["conv"], p["conv_b"], act="swish")
        pr = lin("proj", v)
        y, h, _, _ = oracle.scan_clip(v, lin("step", pr[:, :r]), p["a"], pr[:, r:r + n], pr[:, r + n:], p["skip"],
                                      xz[:, self.inner:], p["dt_bias"])
        o = lin("out", y)
        out = [oracle.residual_norm(a, b, 0.5, post="rms", post_weight=p["post"], pre="layer", pre_weight=p["pre"],
                                    pre_bias=p["pre_b"]) for a, b in zip(x, o)]
        return np.stack([a for a, _ in out]), np.stack([b for _, b in out]), conv, h


def _block_inputs(dtype, B, T, d=128, seed=0):
    rng = np.random.default_rng(seed)
    x, xf = normal(rng, B, T, d)
    u, uf = normal(rng, B, T, d, dtype=dtype)
    return x, u, xf, uf


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("f16", 1e-2)])
def test_block_prompt_then_frames(dtype, tol):
    """A padded batch of prompts, then each stream frame by frame, against the oracle on the whole sequence.

    Relative 2-norm: in f16 six roundings of 2^-11 stand between input and output, each scaled by at most
    the next operators' gains (the post norm divides its branch's error and size alike), so 1e-2, twenty
    half steps, holds them; in f32 the sums of up to 256 products leave some 100 u = 6e-6 at worst."""
    torch = _torch()
    blk = Block(1)
    B, T, extra = 3, 33, 5
    lens = [33, 20, 7]
    x, u, xf, uf = _block_inputs(dtype, B, T + extra)
    states = blk.states(B, _dt(dtype))
    ln = dev(np.array(lens, np.int32))
    xo, uo = blk(x[:, :T].contiguous(), u[:, :T].contiguous(), states, ln)
    refs = [blk.oracle(np.concatenate([xf[i, :n], xf[i, T:]]), np.concatenate([uf[i, :n], uf[i, T:]]))
            for i, n in enumerate(lens)]
    for i, n in enumerate(lens):
        assert rel(host(xo[i, :n]), refs[i][0][:n]) <= tol and rel(host(uo[i, :n]), refs[i][1][:n]) <= tol
    for t in range(T, T + extra):
        xo, uo = blk(x[:, t:t + 1].contiguous(), u[:, t:t + 1].contiguous(), states)
        for i, n in enumerate(lens):
            assert rel(host(uo[i]), refs[i][1][n + t - T:n + t - T + 1]) <= tol
    for i in range(B):
        assert rel(host(states[0][i]), refs[i][2]) <= tol and rel(host(states[1][i]), refs[i][3]) <= tol


def test_block_step_in_a_graph_and_on_two_streams():
    """A frame's step captured once and replayed gives the eager bits; so do two blocks stepping on two
    streams at the same time, each with its own states."""
    torch = _torch()
    B, T = 4, 6
    blocks = [Block(1), Block(2)]
    x, u, _, _ = _block_inputs("f16", B, T)
    want = []
    for blk in blocks:
        st = blk.states(B, torch.float16)
        want.append([tuple(v.clone() for v in blk(x[:, t:t + 1].contiguous(), u[:, t:t + 1].contiguous(), st)) for t in range(T)])
    # captured
    blk = blocks[0]
    st = blk.states(B, torch.float16)
    xs, us = x[:, :1].clone(), u[:, :1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk(xs, us, blk.states(B, torch.float16))
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xo, uo = blk(xs, us, st)
    for t in range(T):
        xs.copy_(x[:, t:t + 1])
        us.copy_(u[:, t:t + 1])
        g.replay()
        assert torch.equal(xo, want[0][t][0]) and torch.equal(uo, want[0][t][1]), t
    # two streams
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sts = [blk.states(B, torch.float16) for blk in blocks]
    frames = [(x[:, t:t + 1].contiguous(), u[:, t:t + 1].contiguous()) for t in range(T)]
    torch.cuda.synchronize()
    got = [[], []]
    for t in range(T):
        for i, blk in enumerate(blocks):
            with torch.cuda.stream(streams[i]):
                got[i].append(blk(*frames[t], sts[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for t in range(T):
            assert torch.equal(got[i][t][0], want[i][t][0]) and torch.equal(got[i][t][1], want[i][t][1])


def test_stream_argument_and_device_checks():
    """A call's own stream argument orders it there, and its outputs belong to that stream."""
    torch = _torch()
    x = torch.randn(8, 256, device="cuda")
    y = torch.randn(8, 256, device="cuda")
    ref = gam.gam_residual_norm(x, y, alpha=0.5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gam.gam_residual_norm(x, y, alpha=0.5, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    with pytest.raises(gam.GamError) as e:
        gam.gam_residual_norm(x, y.cpu())
    assert e.value.name == "GAM_ERR_INVALID_ARG"
    with pytest.raises(gam.GamError) as e:
        gam.gam_residual_norm(x, y[:, ::2])
    assert e.value.name == "GAM_ERR_INVALID_ARG"


def test_tensors_that_require_gradients_are_refused():
    torch = _torch()
    x, y = torch.randn(3, 32, device="cuda"), torch.randn(3, 32, device="cuda")
    w = torch.ones(32, device="cuda", requires_grad=True)
    with pytest.raises(gam.GamError, match="pre_weight requires a gradient"):
        gam.gam_residual_norm(x, y, pre="rms", pre_weight=w)
    with torch.no_grad():
        a = gam.gam_residual_norm(x, y, pre="rms", pre_weight=w)
    b = gam.gam_residual_norm(x, y, pre="rms", pre_weight=w.detach())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
