"""Workloads of the streaming-block operators: what is measured and in which form.

Four operators that make up a block running frame by frame with a fixed-size
state: the few-row linear layer with 4-bit weights (one fp16 scale per 64), the
short causal convolution, the selective state-space scan, and the gated, scaled
residual update with the norms around it.  ``run`` computes them either from
elementary torch operations in 32 bits (``own`` false) or through the
framework's entry points (``own`` true).
"""
import torch

own = False

GROUP = 64
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one frame of one stream through a d768 projection: launch latency
        dict(name="linear-frame-768", op="linear", dtype="f16", rows=1, n=768, k=768, act="none", bias=True),
        # five hypotheses' frames through a 1025-class head in fp32: odd rows and columns
        dict(name="linear-head-1025-f32", op="linear", dtype="f32", rows=5, n=1025, k=1024, act="none", bias=True),
        # sixteen streams in step through a wide up-projection: the weight stream
        dict(name="linear-wide-16", op="linear", dtype="bf16", rows=16, n=16384, k=4096, act="swish", bias=False),
        # one frame of 64 streams (inner width of a d1024 block expanded twice)
        dict(name="conv-frame-64", op="conv", dtype="bf16", batch=64, t=1, d=2048, taps=4, act="swish", bias=True,
             state=True, ragged=False),
        # 32 clips of up to 30 s, right-padded
        dict(name="conv-clips-32", op="conv", dtype="f16", batch=32, t=749, d=2048, taps=4, act="swish", bias=True,
             state=False, ragged=True),
        # one frame of 64 streams: the states go through memory once
        dict(name="scan-frame-64", op="scan", dtype="bf16", batch=64, t=1, d=2048, n=16, z=True, state=True,
             ragged=False),
        # one 30 s window of the d768 model: few channels, a long axis
        dict(name="scan-window-1", op="scan", dtype="f16", batch=1, t=749, d=1536, n=16, z=True, state=False,
             ragged=False),
        # 32 clips of up to 30 s, right-padded: the largest call
        dict(name="scan-clips-32", op="scan", dtype="bf16", batch=32, t=749, d=2048, n=16, z=True, state=False,
             ragged=True),
        # odd sizes in fp32, continued from a state
        dict(name="scan-odd-f32", op="scan", dtype="f32", batch=3, t=517, d=1001, n=12, z=False, state=True,
             ragged=True),
        # one frame of one stream: launch latency
        dict(name="norm-frame", op="norm", xdtype="f32", dtype="f16", rows=1, d=1024, per_gate=1, gate_act="sigmoid",
             post="layer", pre="layer", layer_scale=False),
        # the valid frames of 32 clips of 30 s at d1024, half-weight residual, no gate
        dict(name="norm-clips-1024", op="norm", xdtype="f32", dtype="f16", rows=23968, d=1024, per_gate=0,
             gate_act="none", post="layer", pre="layer", layer_scale=False),
        # wide odd rows in bf16 with a gate per frame and a learnt scale per channel
        dict(name="norm-odd-4099", op="norm", xdtype="bf16", dtype="bf16", rows=2047, d=4099, per_gate=1,
             gate_act="swish", post="rms", pre="rms", layer_scale=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _width(rng, lo, hi):
    """A model's width: most are multiples of 32, some are odd."""
    d = _log(rng, lo, hi)
    return min(hi, (d + 31) // 32 * 32) if rng.random() < 0.6 else d


def draw(rng):
    op = rng.choice(("linear", "conv", "scan", "norm"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op == "linear":
        n = _width(rng, 64, 16384)
        k = GROUP * _log(rng, 1, min(256, (64 << 20) // (n * GROUP)))
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 64), n=n, k=k, act=rng.choice(("none", "swish")),
                    bias=rng.random() < 0.5)
    if op == "norm":
        d = _width(rng, 64, 16384)
        rows = _log(rng, 1, min(32768, (48 << 20) // d))
        per = rng.choice((0, 1, 1, 7))
        rows = rows * per if per > 1 and rows * per * d <= (48 << 20) else rows
        return dict(op=op, xdtype=rng.choice(("f32", dtype)), dtype=dtype, rows=rows, d=d,
                    per_gate=per if per and rows % per == 0 else 0,
                    gate_act=rng.choice(("none", "sigmoid", "swish", "tanh")),
                    post=rng.choice(("none", "layer", "rms")), pre=rng.choice(("layer", "rms")),
                    layer_scale=rng.random() < 0.5)
    d = _width(rng, 64, 4096)
    batch = _log(rng, 1, 64)
    common = dict(op=op, dtype=dtype, batch=batch, d=d, state=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "conv":
        t = 1 if rng.random() < 0.25 else _log(rng, 2, min(8192, (48 << 20) // (batch * d)))
        return dict(common, t=t, taps=rng.choice((2, 3, 4, 4, 4, 5, 8)), act=rng.choice(("none", "swish")),
                    bias=rng.random() < 0.7)
    n = rng.choice((8, 16, 16, 16, 32, 64, _log(rng, 1, 64)))
    t = 1 if rng.random() < 0.25 else _log(rng, 2, max(2, min(8192, (512 << 20) // (batch * d * n))))
    return dict(common, t=t, n=n, z=rng.random() < 0.7)


def _lengths(case):
    """Valid frames of each sequence: all of them, or spread from the longest down to one that is empty."""
    b, t = case["batch"], case["t"]
    if not case["ragged"]:
        return [t] * b
    spread = [t - ((i + b // 2) % b) * t // (b + 1) for i in range(b)]
    return [0 if b > 3 and i == b - 2 else v for i, v in enumerate(spread)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(to)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        # weights as a checkpoint packs them: u = q + 8 with q in -7 .. 7, eight to a word, v_2i in nibble i and
        # v_2i+1 in nibble 4 + i
        u = torch.randint(1, 16, (n, k // 8, 4, 2), generator=g, device="cuda", dtype=torch.int32)
        low = (u << (4 * torch.arange(4, device="cuda", dtype=torch.int32))[None, None, :, None]).sum(2)
        words = low[..., 0] | (low[..., 1] << 16)
        s["packed"] = words.to(torch.int32).view(torch.uint8).reshape(n, k // 2).contiguous()
        s["scale"] = ((uniform(n, k // GROUP) + 0.5) * (0.25 / k ** 0.5)).half()
        s["bias"] = normal(n, std=0.1) if case["bias"] else None
        s["x"] = normal(rows, k, to=dt)
        s["out"] = torch.empty(rows, n, dtype=dt, device="cuda")
        return s
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = normal(rows, d, std=2.0, to=DTYPES[case["xdtype"]])
        s["y"] = normal(rows, d, to=dt) + 0.5
        per = case["per_gate"]
        s["gate"] = normal(rows // per, d, to=dt) if per else None
        s["layer_scale"] = 1 + normal(d, std=0.2) if case["layer_scale"] else None
        for p in ("post", "pre"):
            kind = case[p]
            s[p + "_weight"] = 1 + normal(d, std=0.1) if kind != "none" else None
            s[p + "_bias"] = normal(d, std=0.1) if kind == "layer" else None
        s["x_out"], s["out"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        return s
    b, t, d = case["batch"], case["t"], case["d"]
    lens = _lengths(case)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if case["ragged"] else None
    s["x"] = normal(b, t, d, to=dt)
    s["out"] = torch.empty(b, t, d, dtype=dt, device="cuda")
    if case["op"] == "conv":
        taps = case["taps"]
        s["weight"] = normal(d, taps, std=taps ** -0.5)
        s["bias"] = normal(d, std=0.1) if case["bias"] else None
        s["state"] = normal(b, taps - 1, d, to=dt) if case["state"] else None
        s["state_out"] = torch.empty(b, taps - 1, d, dtype=dt, device="cuda")
        return s
    n = case["n"]
    # step sizes log-uniform in 0.001 .. 0.1 around the bias, decay rates 1 .. n, the usual start of such a layer
    step = torch.exp(uniform(d) * 4.6 - 6.9)
    s["dt"] = normal(b, t, d, std=0.5, to=dt)
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["a"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * (0.75 + 0.5 * uniform(d, n))
    # B and C as they leave one projection, side by side in a row
    bc = normal(b, t, 2 * n, to=dt)
    s["b"], s["c"] = bc[..., :n], bc[..., n:]
    s["d_skip"] = 1 + normal(d, std=0.1)
    s["z"] = normal(b, t, d, to=dt) if case["z"] else None
    s["state"] = normal(b, d, n) if case["state"] else None
    s["state_out"] = torch.empty(b, d, n, device="cuda")
    return s


# ---- plain forms -------------------------------------------------------------

def _act(v, kind):
    if kind == "swish":
        return v / (1 + torch.exp(-v))
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return torch.tanh(v) if kind == "tanh" else v


def _plain_linear(s):
    c, words = s["case"], s["packed"].view(torch.int32)
    shift = 4 * torch.arange(8, device=words.device, dtype=torch.int32).view(2, 4).t().reshape(8)
    q = ((words[..., None] >> shift) & 15) - 8                      # [n, k / 8, 8]
    w = q.view(c["n"], c["k"] // GROUP, GROUP).float() * s["scale"].float()[..., None]
    y = s["x"].float() @ w.view(c["n"], c["k"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return _act(y, c["act"]).to(s["x"].dtype)


def _valid(s):
    c = s["case"]
    t = torch.arange(c["t"], device=s["x"].device)
    lens = s["lengths"] if s["lengths"] is not None else torch.full((c["batch"],), c["t"], device=t.device)
    return t[None, :] < lens[:, None], lens.long()


def _plain_conv(s):
    c, x = s["case"], s["x"]
    b, t, d, taps = c["batch"], c["t"], c["d"], c["taps"]
    valid, lens = _valid(s)
    past = s["state"] if s["state"] is not None else torch.zeros(b, taps - 1, d, dtype=x.dtype, device=x.device)
    rows = torch.cat([past, x], 1)
    y = sum(rows[:, j:j + t].float() * s["weight"][:, j] for j in range(taps))
    if s["bias"] is not None:
        y = y + s["bias"]
    y = torch.where(valid[..., None], _act(y, c["act"]), torch.zeros_like(y)).to(x.dtype)
    at = lens[:, None] + torch.arange(taps - 1, device=x.device)
    return y, rows.gather(1, at[..., None].expand(b, taps - 1, d))


def _plain_scan(s):
    c, x = s["case"], s["x"].float()
    valid, _ = _valid(s)
    dt = s["dt"].float() + s["dt_bias"]
    dt = torch.where(dt > 20, dt, torch.log1p(torch.exp(dt.clamp(max=20.0))))
    dt = torch.where(valid[..., None], dt, torch.zeros_like(dt))    # a frame behind the end leaves the state alone
    xv = torch.where(valid[..., None], x, torch.zeros_like(x))
    bv = torch.where(valid[..., None], s["b"].float(), torch.zeros_like(s["b"].float()))
    decay = torch.exp(dt[..., None] * s["a"])                       # [batch, t, d, n]
    h = (dt * xv)[..., None] * bv[:, :, None, :]
    if s["state"] is not None:
        h[:, 0] += decay[:, 0] * s["state"]
    reach = 1
    while reach < c["t"]:                                           # each frame takes in twice as many before it
        h = torch.cat([h[:, :reach], h[:, reach:] + decay[:, reach:] * h[:, :-reach]], 1)
        decay = torch.cat([decay[:, :reach], decay[:, reach:] * decay[:, :-reach]], 1)
        reach *= 2
    y = (h * s["c"].float()[:, :, None, :]).sum(-1) + s["d_skip"] * x
    if s["z"] is not None:
        y = y * _act(s["z"].float(), "swish")
    y = torch.where(valid[..., None], y, torch.zeros_like(y))
    return y.to(s["x"].dtype), h[:, -1].clone()


def _norm(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    if kind != "none":
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * weight
    return v + bias if kind == "layer" else v


def _plain_norm(s):
    c = s["case"]
    branch = _norm(s["y"].float(), c["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        branch = branch * _act(s["gate"].float(), c["gate_act"]).repeat_interleave(c["per_gate"], 0)
    if s["layer_scale"] is not None:
        branch = branch * s["layer_scale"]
    x = s["x"].float() + 0.5 * branch
    return x.to(s["x"].dtype), _norm(x, c["pre"], s["pre_weight"], s["pre_bias"]).to(s["y"].dtype)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from conformer_speech_recognition_b200 import gam
        if op == "linear":
            return gam.gam_quant_linear(s["x"], s["packed"], s["scale"], bias=s["bias"], act=s["case"]["act"],
                                        out=s["out"])
        if op == "conv":
            return gam.gam_short_conv(s["x"], s["weight"], bias=s["bias"], act=s["case"]["act"],
                                      lengths=s["lengths"], state=s["state"], out=s["out"],
                                      state_out=s["state_out"])
        if op == "scan":
            return gam.gam_selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], d_skip=s["d_skip"], z=s["z"],
                                          dt_bias=s["dt_bias"], dt_softplus=True, lengths=s["lengths"],
                                          state=s["state"], out=s["out"], state_out=s["state_out"])
        return gam.gam_residual_norm(s["x"], s["y"], alpha=0.5, layer_scale=s["layer_scale"], gate=s["gate"],
                                     gate_act=s["case"]["gate_act"], post=s["case"]["post"],
                                     post_weight=s["post_weight"], post_bias=s["post_bias"], pre=s["case"]["pre"],
                                     pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=1e-5,
                                     x_out=s["x_out"], out=s["out"])
    return {"linear": _plain_linear, "conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](s)


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": n * k / 2 + n * k // GROUP * 2 + 4 * n * case["bias"] + rows * (k + n) * es,
                "flops": 2 * rows * n * k}
    if case["op"] == "norm":
        rows, d, per = case["rows"], case["d"], case["per_gate"]
        vectors = case["layer_scale"] + sum({"none": 0, "rms": 1, "layer": 2}[case[p]] for p in ("post", "pre"))
        return {"bytes": rows * d * 2 * (SIZE[case["xdtype"]] + es) + (rows // per * d * es if per else 0) + 4 * d * vectors,
                "flops": 14 * rows * d}
    b, t, d, frames = case["batch"], case["t"], case["d"], sum(_lengths(case))
    if case["op"] == "conv":
        taps = case["taps"]
        return {"bytes": (frames + b * t) * d * es + (1 + case["state"]) * b * (taps - 1) * d * es
                         + 4 * d * (taps + case["bias"]), "flops": 2 * taps * frames * d}
    n = case["n"]
    return {"bytes": frames * (d * (2 + case["z"]) + 2 * n) * es + b * t * d * es + (1 + case["state"]) * b * d * n * 4
                     + 4 * d * (n + 2), "flops": 7 * frames * d * n}


# ---- the definitions in 64 bits ------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    gate = {"none": lambda v: v, "sigmoid": torch.special.expit, "swish": lambda v: v * torch.special.expit(v),
            "tanh": torch.tanh}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        byte = s["packed"].view(n, k // 8, 4).long()                # byte j of a word: nibbles 2 j and 2 j + 1
        nibble = torch.stack([byte % 16, byte // 16], -1).view(n, k // 8, 2, 4)
        q = nibble.transpose(2, 3).reshape(n, k) - 8                # nibble 4 a + i holds weight 2 i + a
        y = f["x"] @ (q.double() * f["scale"].repeat_interleave(GROUP, 1)).T
        return gate[case["act"]](y + f["bias"] if case["bias"] else y)
    if case["op"] == "norm":
        def norm(v, kind, w, bias):
            if kind == "layer":
                return (v - v.mean(1, True)) * torch.rsqrt(v.var(1, unbiased=False, keepdim=True) + 1e-5) * w + bias
            return v * torch.rsqrt(v.pow(2).mean(1, True) + 1e-5) * w if kind == "rms" else v
        br = 0.5 * norm(f["y"], case["post"], f["post_weight"], f["post_bias"])
        if case["layer_scale"]:
            br = br * f["layer_scale"]
        if case["per_gate"]:
            br = br * gate[case["gate_act"]](f["gate"])[torch.arange(case["rows"], device=br.device) // case["per_gate"]]
        x = f["x"] + br
        return x, norm(x, case["pre"], f["pre_weight"], f["pre_bias"])
    b, t, d, lens = case["batch"], case["t"], case["d"], _lengths(case)
    y = torch.zeros(b, t, d, dtype=torch.float64, device="cuda")
    if case["op"] == "conv":
        taps, new = case["taps"], []
        for i in range(b):
            past = f["state"][i] if case["state"] else torch.zeros(taps - 1, d, dtype=torch.float64, device="cuda")
            seq = torch.cat([past, f["x"][i, :lens[i]]])
            new.append(seq[len(seq) - (taps - 1):])
            if lens[i]:
                v = torch.einsum("tdj,dj->td", seq.unfold(0, taps, 1), f["weight"])
                y[i, :lens[i]] = gate[case["act"]](v + f["bias"] if case["bias"] else v)
        return y, torch.stack(new)
    h = f["state"].clone() if case["state"] else torch.zeros(b, d, case["n"], dtype=torch.float64, device="cuda")
    step = torch.nn.functional.softplus(f["dt"] + f["dt_bias"], threshold=100)
    order = sorted(range(b), key=lambda i: -lens[i])                # longest first: the live ones are a prefix
    at = torch.tensor(order, device="cuda")
    h, step, x, bb, cc = h[at], step[at], f["x"][at], f["b"][at], f["c"][at]
    for i in range(t):
        live = sum(v > i for v in lens)
        if not live:
            break
        p = step[:live, i, :, None]
        h[:live] = torch.exp(p * f["a"]) * h[:live] + p * x[:live, i, :, None] * bb[:live, i, None, :]
        y[at[:live], i] = torch.einsum("bdn,bn->bd", h[:live], cc[:live, i]) + f["d_skip"] * x[:live, i]
    back = torch.empty_like(h)
    back[at] = h
    return (y * gate["swish"](f["z"]) if case["z"] else y), back
