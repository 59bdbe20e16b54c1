"""The channels-last sequence-mixer operators: what is measured, and their plain forms.

Three operators follow a convolution stage when a feature map (N, H, W, C) is read as
sequences of pixels, or a camera stream as a sequence of frames:

* group norm with an activation, channels last: tensors (N, P, C), P pixels an image;
* a short causal depthwise convolution along the sequence (B, L, D), whose left halo of
  K - 1 rows is carried in and out as a state;
* a selective state-space scan along the sequence: h_t = exp(delta_t A) h_{t-1} +
  delta_t u_t B_t, y_t = C_t . h_t + D u_t, gated by SiLU(z_t), with delta = softplus(dt + bias).

The convolution and the scan also have a form for one token that updates the carried
state in place.  A ragged batch gives a length per sequence; rows at or past it are not
read (they hold NaN here) and their outputs are zero.

`run` computes the plain form in 32 bits from elementary operations, or, where `own` is
true, calls the library.  `exact` is the definition in 64 bits, one token after another.
"""
import math

import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
BYTES = {F32: 4, BF16: 2, F16: 2}


# ---------------------------------------------------------------- the cases

def _gn(name, op, n, p, c, groups, dtype, act):
    return {"name": name, "op": op, "n": n, "p": p, "c": c, "groups": groups, "dtype": dtype, "act": act}


def _conv(name, op, b, l, d, k, dtype, act, state=False, ragged=False):
    return {"name": name, "op": op, "b": b, "l": l, "d": d, "k": k, "dtype": dtype, "act": act, "state": state,
            "ragged": ragged}


def _scan(name, op, b, l, d, n, groups, dtype, gate=True, state=False, ragged=False):
    return {"name": name, "op": op, "b": b, "l": l, "d": d, "n": n, "groups": groups, "dtype": dtype, "gate": gate,
            "state": state, "ragged": ragged}


def listed():
    return [
        # one small camera tile of a streaming detector: latency
        _gn("norm small map", "gn_fwd", 1, 16 * 32, 256, 32, BF16, "silu"),
        # the stem output of seven 512 x 4096 cameras: the largest map, inference
        _gn("norm stage-1 maps", "gn_fwd", 7, 128 * 1024, 256, 32, BF16, "silu"),
        # a training step on the depthwise workload's map
        _gn("norm training", "gn_train", 7, 128 * 512, 256, 32, F32, "silu"),
        # odd image and channel counts (the layer norm test's 97 x 113 map), exact-erf GELU
        _gn("norm odd training", "gn_train", 3, 97 * 113, 120, 24, BF16, "gelu"),
        # a prompt of pixel tokens read from half of an input projection's output
        _conv("conv prompt", "conv_fwd", 8, 4096, 1024, 4, BF16, "silu", state=True),
        # training on image rows of different widths
        _conv("conv ragged training", "conv_train", 56, 1023, 264, 4, F32, "silu", state=True, ragged=True),
        # one new frame for each of 64 streams
        _conv("conv one token", "conv_step", 64, 1, 2048, 4, BF16, "silu", state=True),
        # few tokens after a carried state: latency
        _scan("scan short prompt", "scan_fwd", 1, 33, 256, 16, 1, BF16, state=True),
        # one image as a raster of 16384 pixel tokens: few channels, a long axis
        _scan("scan long prompt", "scan_fwd", 1, 16384, 512, 16, 1, BF16),
        # image rows as sequences: 7 cameras x 32 rows of 1024 pixels
        _scan("scan row training", "scan_train", 224, 1024, 256, 16, 1, F32),
        # ragged rows, two channel groups with their own B and C, odd sizes, a carried state
        _scan("scan ragged training", "scan_train", 5, 1537, 328, 13, 2, BF16, state=True, ragged=True),
        # one new frame for each of 64 streams
        _scan("scan one token", "scan_step", 64, 1, 2048, 16, 1, BF16, state=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_train", "conv_fwd", "conv_train", "conv_step", "scan_fwd", "scan_train", "scan_step"])
    dtype = rng.choice([F32, BF16, F16])
    if op.startswith("gn"):
        per = rng.choice([1, 3, 4, 5, 8, 16])
        groups = _log(rng, 1, 64)
        c = per * groups
        n = _log(rng, 1, 16)
        # a gradient of a group of a few values is what cancellation leaves: from 16 pixels on
        least = 16 if op == "gn_train" else 1
        p = _log(rng, least, max(2 * least, min(1 << 17, (1 << 26) // (c * n))))
        case = _gn("", op, n, p, c, groups, dtype, rng.choice(["none", "silu", "gelu"]))
    elif op.startswith("conv"):
        d = _log(rng, 1, 2048)
        b = _log(rng, 1, 256)
        l = 1 if op == "conv_step" else _log(rng, 1, max(2, min(1 << 15, (1 << 25) // (b * d))))
        case = _conv("", op, b, l, d, rng.choice([2, 3, 4, 5]), dtype, rng.choice(["none", "silu"]),
                     op == "conv_step" or rng.random() < 0.5, op != "conv_step" and rng.random() < 0.4)
    else:
        groups = rng.choice([1, 1, 2, 4])
        d = groups * _log(rng, 1, 512)
        n = rng.choice([4, 7, 8, 16, 16, 32])
        b = _log(rng, 1, 128)
        l = 1 if op == "scan_step" else _log(rng, 1, max(2, min(1 << 14, (1 << 29) // (b * d * n))))
        case = _scan("", op, b, l, d, n, groups, dtype, rng.random() < 0.7, op == "scan_step" or rng.random() < 0.5,
                     op != "scan_step" and rng.random() < 0.4)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _lengths(b, l, seed):
    """Lengths of a ragged batch: spread over 0 .. l, an empty, a one-row and a full sequence among them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(0, l + 1, (b,), generator=g)
    for i, x in enumerate((l, 0, 1)):
        if i < b:
            v[(seed + i) % b] = x
    return v.to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    t = TORCH[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op.startswith("gn"):
        n, p, c = case["n"], case["p"], case["c"]
        # every channel with an offset and a scale of its own, as a convolution with a bias gives
        s["x"] = (torch.randn(n, p, c, generator=g, device="cuda") * (0.5 + uniform(c)) + normal(c)).to(t)
        s["gamma"], s["beta"] = normal(c, scale=0.1, shift=1.0), normal(c, scale=0.1)
        if op == "gn_train":
            s["gy"] = normal(n, p, c, dtype=t)
        return s

    b, l, d = case["b"], case["l"], case["d"]
    lens = _lengths(b, l, seed) if case["ragged"] else None
    s["lens"] = lens

    def blank(x):
        """NaN in the rows that a ragged batch does not have."""
        if lens is not None:
            gone = torch.arange(l, device="cuda") >= lens[:, None]
            x.masked_fill_(gone[:, :, None], float("nan"))
        return x

    if op.startswith("conv"):
        k = case["k"]
        # the first half of an input projection's output rows: a row stride of 2 d
        xz = blank(normal(b, l, 2 * d, dtype=t))
        s["x"] = xz[:, :, :d]
        s["w"], s["bias"] = (uniform(d, k) * 2 - 1) / math.sqrt(k), (uniform(d) * 2 - 1) / math.sqrt(k)
        s["state"] = normal(b, k - 1, d, dtype=t) if case["state"] else None
        if op == "conv_step":
            s["x"] = s["x"][:, 0]
        if op == "conv_train":
            s["gy"] = blank(normal(b, l, d, dtype=t))
        return s

    n, groups = case["n"], case["groups"]
    rank = max(1, d // 16)
    # B and C are slices of one projection's output rows (rank + 2 groups n wide); z is the second
    # half of the input projection's
    proj = blank(normal(b, l, rank + 2 * groups * n, dtype=t))
    s["B"], s["C"] = proj[:, :, rank:rank + groups * n], proj[:, :, rank + groups * n:]
    xz = blank(normal(b, l, 2 * d, dtype=t))
    s["z"] = xz[:, :, d:] if case["gate"] else None
    s["u"] = blank(normal(b, l, d, dtype=t))
    s["dt"] = blank(normal(b, l, d, scale=0.5, dtype=t))
    # A near -1 .. -n; step sizes spread over 0.001 .. 0.1 by the bias, softplus(bias) = step
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(d, n, scale=0.1))
    step = torch.exp(uniform(d) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = normal(d, scale=0.1, shift=1.0)
    s["state"] = normal(b, d, n, scale=0.3) if case["state"] else None
    if op == "scan_step":
        for key in ("B", "C", "z", "u", "dt"):
            s[key] = s[key][:, 0] if s[key] is not None else None
    if op == "scan_train":
        s["gy"] = blank(normal(b, l, d, dtype=t))
    return s


# ---------------------------------------------------------------- plain forms, 32 bits

def _act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return x


def _act_slope(x, kind):
    if kind == "silu":
        r = torch.sigmoid(x)
        return r * (1 + x * (1 - r))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    return torch.ones_like(x)


def _gn_plain(s):
    case = s["case"]
    n, p, c, groups, kind = (case[k] for k in ("n", "p", "c", "groups", "act"))
    t = s["x"].dtype
    x = s["x"].float().view(n, p, groups, c // groups)
    gamma, beta = s["gamma"].view(groups, -1), s["beta"].view(groups, -1)
    x = x - x.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt(x.square().mean((1, 3), keepdim=True) + 1e-5)
    x = x * rstd
    pre = x * gamma + beta
    out = {"y": _act(pre, kind).view(n, p, c).to(t)}
    if case["op"] == "gn_train":
        g = s["gy"].float().view(n, p, groups, c // groups) * _act_slope(pre, kind)
        out["ggamma"], out["gbeta"] = (g * x).sum((0, 1)).view(c), g.sum((0, 1)).view(c)
        g = g * gamma
        gx = rstd * (g - g.mean((1, 3), keepdim=True) - x * (g * x).mean((1, 3), keepdim=True))
        out["gx"] = gx.view(n, p, c).to(t)
    return out


def _live(s, l):
    """The rows that are there, (B, L, 1), or None where all are."""
    return None if s["lens"] is None else (torch.arange(l, device="cuda") < s["lens"][:, None])[:, :, None]


def _rows(x, live):
    x = x.float()
    return x if live is None else torch.where(live, x, torch.zeros_like(x))


def _conv_plain(s):
    case = s["case"]
    b, l, d, k, kind = (case[q] for q in ("b", "l", "d", "k", "act"))
    t = s["x"].dtype
    w, bias = s["w"], s["bias"]
    if case["op"] == "conv_step":
        win = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)  # (B, K, D)
        y = _act((win * w.t()).sum(1) + bias, kind)
        s["state"].copy_(win[:, 1:].to(t))
        return {"y": y.to(t), "state": s["state"]}
    live = _live(s, l)
    head = s["state"].float() if s["state"] is not None else torch.zeros(b, k - 1, d, device="cuda")
    x = torch.cat([head, _rows(s["x"], live)], 1)
    win = x.unfold(1, k, 1)  # (B, L, D, K)
    pre = (win * w).sum(-1) + bias
    out = {"y": _rows(_act(pre, kind), live).to(t)}
    ends = s["lens"].long() if s["lens"] is not None else torch.full((b,), l, device="cuda")
    last = (ends[:, None] + torch.arange(k - 1, device="cuda"))[:, :, None].expand(b, k - 1, d)
    out["state"] = x.gather(1, last).to(t)
    if case["op"] == "conv_train":
        g = _rows(s["gy"], live) * _rows(_act_slope(pre, kind), live)
        out["gw"], out["gb"] = (g[..., None] * win).sum((0, 1)), g.sum((0, 1))
        z = torch.zeros(b, k - 1, d, device="cuda")
        gx = (torch.cat([z, g, z], 1).unfold(1, k, 1) * w.flip(1)).sum(-1)  # of the carried rows, then of x
        out["gx"] = _rows(gx[:, k - 1:], live).to(t)
        if s["state"] is not None:
            out["gstate"] = gx[:, :k - 1].to(t)
    return out


def _recur(a, x):
    """h_t = a_t h_{t-1} + x_t along axis 1, every span of rows doubled until it covers the axis."""
    span = 1
    while span < x.shape[1]:
        x = torch.cat([x[:, :span], x[:, span:] + a[:, span:] * x[:, :-span]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return x


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_plain(s):
    case = s["case"]
    b, l, d, n, groups = (case[q] for q in ("b", "l", "d", "n", "groups"))
    t = s["u"].dtype
    A, D = s["A"], s["D"]
    one = case["op"] == "scan_step"
    live = None if one else _live(s, l)

    def rows(key):
        return _rows(s[key][:, None] if one else s[key], live)

    def wide(x):  # (B, L, groups n) for every channel of its group: (B, L, D, n)
        return x.view(b, -1, groups, 1, n).expand(-1, -1, -1, d // groups, -1).reshape(b, -1, d, n)

    u, B, C = rows("u"), wide(rows("B")), wide(rows("C"))
    raw = rows("dt") + s["dt_bias"]
    delta = _rows(_softplus(raw), live)
    a = torch.exp(delta[..., None] * A)
    x = (delta * u)[..., None] * B
    if s["state"] is not None:
        x[:, 0] += a[:, 0] * s["state"]
    h = _recur(a, x)
    ys = (h * C).sum(-1) + D * u
    z = rows("z") if case["gate"] else None
    y = ys * _act(z, "silu") if case["gate"] else ys
    if one:
        s["state"].copy_(h[:, 0])
        return {"y": y[:, 0].to(t), "state": s["state"]}
    out = {"y": _rows(y, live).to(t), "state": h[:, -1].clone()}
    if case["op"] == "scan_fwd":
        return out
    gy = rows("gy")
    if case["gate"]:
        out["gz"] = (gy * ys * _act_slope(z, "silu")).to(t)
        gy = gy * _act(z, "silu")
    # the state's gradient runs backwards: G_t = gy_t C_t + a_{t+1} G_{t+1}
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    G = _recur(after.flip(1), (gy[..., None] * C).flip(1)).flip(1)
    first = s["state"] if s["state"] is not None else torch.zeros(b, d, n, device="cuda")
    Gah = G * a * torch.cat([first[:, None], h[:, :-1]], 1)
    if s["state"] is not None:
        out["gstate"] = a[:, 0] * G[:, 0]
    GB = (G * B).sum(-1)
    out["gu"] = (GB * delta + D * gy).to(t)
    gdt = (GB * u + (Gah * A).sum(-1)) * torch.sigmoid(raw)
    gdt = _rows(gdt, live)
    out["gdt"], out["gdt_bias"] = gdt.to(t), gdt.sum((0, 1))
    out["gD"] = (gy * u).sum((0, 1))
    out["gA"] = (Gah * delta[..., None]).sum((0, 1))
    out["gB"] = (G * (delta * u)[..., None]).view(b, l, groups, -1, n).sum(3).reshape(b, l, -1).to(t)
    out["gC"] = (gy[..., None] * h).view(b, l, groups, -1, n).sum(3).reshape(b, l, -1).to(t)
    return out


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """The descriptor, outputs and workspaces that a program sets up once for its sizes."""
    from spatially_sharded_cnn_gb300 import hc
    case = s["case"]
    op, t = case["op"], TORCH[case["dtype"]]

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def space(got):
        hc.check(got[0], "workspace size")
        return empty(max(got[1], 16), dtype=torch.uint8), got[1]

    p = {"hc": hc}
    if op.startswith("gn"):
        n, px, c = case["n"], case["p"], case["c"]
        act = {"none": hc.HC_PW_NONE, "silu": hc.HC_PW_SILU, "gelu": hc.HC_PW_GELU}[case["act"]]
        p["d"] = hc.groupnorm_desc(N=n, P=px, C=c, groups=case["groups"], eps=1e-5, act=act, dtype=t)
        p["ws"], p["nb"] = space(hc.hc_groupnorm_workspace_size(p["d"], int(op == "gn_train")))
        p["out"] = {"y": empty(n, px, c, dtype=t)}
        if op == "gn_train":
            p["mean"], p["rstd"] = empty(n, case["groups"]), empty(n, case["groups"])
            p["out"].update(gx=empty(n, px, c, dtype=t), ggamma=empty(c), gbeta=empty(c))
    elif op.startswith("conv"):
        b, l, d, k = case["b"], case["l"], case["d"], case["k"]
        act = {"none": hc.HC_PW_NONE, "silu": hc.HC_PW_SILU}[case["act"]]
        p["d"] = hc.causal_conv_desc(B=b, L=l, D=d, K=k, act=act, dtype=t)
        if op == "conv_step":
            p["out"] = {"y": empty(b, d, dtype=t), "state": s["state"]}
            return p
        p["out"] = {"y": empty(b, l, d, dtype=t), "state": empty(b, k - 1, d, dtype=t)}
        if op == "conv_train":
            p["ws"], p["nb"] = space(hc.hc_causal_conv_workspace_size(p["d"]))
            p["out"].update(gx=empty(b, l, d, dtype=t), gw=empty(d, k), gb=empty(d))
            if s["state"] is not None:
                p["out"]["gstate"] = empty(b, k - 1, d, dtype=t)
    else:
        b, l, d, n, groups = case["b"], case["l"], case["d"], case["n"], case["groups"]
        p["d"] = hc.selective_scan_desc(B=b, L=l, D=d, groups=groups, d_state=n, softplus=1, dtype=t)
        if op == "scan_step":
            p["out"] = {"y": empty(b, d, dtype=t), "state": s["state"]}
            return p
        p["ws"], p["nb"] = space(hc.hc_selective_scan_workspace_size(p["d"], int(op == "scan_train")))
        p["out"] = {"y": empty(b, l, d, dtype=t), "state": empty(b, d, n)}
        p["saved"] = None
        if op == "scan_train":
            p["saved"] = space(hc.hc_selective_scan_saved_size(p["d"]))[0]
            p["out"].update(gu=empty(b, l, d, dtype=t), gdt=empty(b, l, d, dtype=t), gdt_bias=empty(d), gD=empty(d),
                            gA=empty(d, n), gB=empty(b, l, groups * n, dtype=t), gC=empty(b, l, groups * n, dtype=t))
            if case["gate"]:
                p["out"]["gz"] = empty(b, l, d, dtype=t)
            if s["state"] is not None:
                p["out"]["gstate"] = empty(b, d, n)
    return p


def _library(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    hc, d, out, op = p["hc"], p["d"], p["out"], s["case"]["op"]
    if op == "gn_fwd":
        hc.check(hc.hc_groupnorm_fwd(d, s["x"], s["gamma"], s["beta"], out["y"], ws=p["ws"], ws_bytes=p["nb"]))
    elif op == "gn_train":
        hc.check(hc.hc_groupnorm_fwd(d, s["x"], s["gamma"], s["beta"], out["y"], p["mean"], p["rstd"], p["ws"], p["nb"]))
        hc.check(hc.hc_groupnorm_bwd(d, s["x"], s["gamma"], s["beta"], p["mean"], p["rstd"], s["gy"], out["gx"],
                                     out["ggamma"], out["gbeta"], p["ws"], p["nb"]))
    elif op == "conv_step":
        hc.check(hc.hc_causal_conv_step(d, s["x"], s["w"], s["bias"], s["state"], out["y"]))
    elif op.startswith("conv"):
        hc.check(hc.hc_causal_conv_fwd(d, s["x"], s["w"], s["bias"], out["y"], s["state"], out["state"], s["lens"]))
        if op == "conv_train":
            hc.check(hc.hc_causal_conv_bwd(d, s["x"], s["w"], s["bias"], s["gy"], out["gx"], out["gw"], out["gb"],
                                           s["state"], None, out.get("gstate"), s["lens"], p["ws"], p["nb"]))
    elif op == "scan_step":
        hc.check(hc.hc_selective_scan_step(d, s["u"], s["dt"], s["A"], s["B"], s["C"], s["state"], out["y"], D=s["D"],
                                           z=s["z"], dt_bias=s["dt_bias"]))
    else:
        hc.check(hc.hc_selective_scan_fwd(d, s["u"], s["dt"], s["A"], s["B"], s["C"], out["y"], D=s["D"], z=s["z"],
                                          dt_bias=s["dt_bias"], h0=s["state"], hT=out["state"], lens=s["lens"],
                                          saved=p["saved"], ws=p["ws"], ws_bytes=p["nb"]))
        if op == "scan_train":
            hc.check(hc.hc_selective_scan_bwd(d, s["u"], s["dt"], s["A"], s["B"], s["C"], s["gy"], p["saved"],
                                              out["gu"], out["gdt"], out["gA"], out["gB"], out["gC"], D=s["D"],
                                              z=s["z"], dt_bias=s["dt_bias"], h0=s["state"], lens=s["lens"],
                                              gD=out["gD"], gz=out.get("gz"), gdt_bias=out["gdt_bias"],
                                              gh0=out.get("gstate"), ws=p["ws"], ws_bytes=p["nb"]))
    return out


def run(state):
    if own:
        return _library(state)
    op = state["case"]["op"]
    return _gn_plain(state) if op.startswith("gn") else _conv_plain(state) if op.startswith("conv") else _scan_plain(state)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op.startswith("gn"):
        m, c = case["n"] * case["p"] * case["c"], case["c"]
        # x and y, and for training gy and gx; about 10 operations an element forward, 20 backward
        if op == "gn_fwd":
            return {"bytes": 2 * m * e + 8 * c, "flops": 10 * m}
        return {"bytes": 4 * m * e + 16 * c, "flops": 30 * m}
    b, l, d = case["b"], case["l"], case["d"]
    m = b * l * d
    if op.startswith("conv"):
        k = case["k"]
        carried = b * (k - 1) * d * e
        if op == "conv_fwd" or op == "conv_step":
            return {"bytes": 2 * m * e + (1 + case["state"]) * carried + 4 * d * (k + 1), "flops": (2 * k + 6) * m}
        return {"bytes": 4 * m * e + (1 + 2 * case["state"]) * carried + 8 * d * (k + 1), "flops": (8 * k + 16) * m}
    n, groups = case["n"], case["groups"]
    shared, states = b * l * groups * n * e, 4 * b * d * n
    maps = 3 + case["gate"]  # u, dt, y and z
    params = 4 * d * (n + 2)
    # a state: delta A, exp, du B, one multiply-add each for h and y: 7 operations
    if op != "scan_train":
        return {"bytes": maps * m * e + 2 * shared + (1 + case["state"]) * states + params, "flops": 7 * n * m}
    # and for its gradient: the state's own, and one multiply-add each into gB, gC, gA, gu and gdt
    return {"bytes": 2 * maps * m * e + 4 * shared + (1 + 2 * case["state"]) * states + 2 * params,
            "flops": (7 + 16) * n * m}


# ---------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op.startswith("gn"):
        n, p, c, q = case["n"], case["p"], case["c"], case["c"] // case["groups"]
        x = f["x"].requires_grad_(op == "gn_train")
        gamma, beta = f["gamma"].requires_grad_(True), f["beta"].requires_grad_(True)
        v, m = torch.var_mean(x.view(n, p, -1, q), dim=(1, 3), correction=0)
        scale = gamma * ((v + 1e-5) ** -0.5).repeat_interleave(q, dim=1)[:, None]
        pre = (x - m.repeat_interleave(q, dim=1)[:, None]) * scale + beta
        if case["act"] == "silu":
            y = pre / (1 + torch.exp(-pre))
        elif case["act"] == "gelu":
            y = pre * torch.special.ndtr(pre)
        else:
            y = pre * 1
        out = {"y": y.detach()}
        if op == "gn_train":
            out["gx"], out["ggamma"], out["gbeta"] = torch.autograd.grad(y, (x, gamma, beta), f["gy"])
        return out

    b, l, d = case["b"], case["l"], case["d"]
    ends = f["lens"].long() if f["lens"] is not None else torch.full((b,), l, device="cuda")
    there = torch.arange(l, device="cuda")[None, :, None] < ends[:, None, None]

    def clean(key):
        v = f[key]
        return v[:, None] if op.endswith("step") else v.masked_fill(~there, 0.0)

    if op.startswith("conv"):
        k = case["k"]
        x = clean("x").requires_grad_(True)
        w, bias = f["w"].requires_grad_(True), f["bias"].requires_grad_(True)
        head = f["state"] if f["state"] is not None else x.new_zeros(b, k - 1, d)
        head = head.detach().requires_grad_(True)
        rows = torch.cat([head, x], 1)
        pre = bias + sum(rows[:, j:j + l] * w[:, j] for j in range(k))
        y = pre / (1 + torch.exp(-pre)) if case["act"] == "silu" else pre * 1
        state = torch.stack([rows[i, int(e):int(e) + k - 1] for i, e in enumerate(ends.tolist())]).detach()
        if op == "conv_step":
            return {"y": y[:, 0].detach(), "state": state}
        out = {"y": y.detach().masked_fill(~there, 0.0), "state": state}
        if op == "conv_train":
            gx, gw, gb, gs = torch.autograd.grad(y, (x, w, bias, head), clean("gy"))
            out.update(gx=gx.masked_fill(~there, 0.0), gw=gw, gb=gb)
            if f["state"] is not None:
                out["gstate"] = gs
        return out

    n, groups, per = case["n"], case["groups"], d // case["groups"]
    A, D = f["A"], f["D"]
    u, Bm, Cm, raw = clean("u"), clean("B"), clean("C"), clean("dt") + f["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw)).masked_fill(~there, 0.0)
    gate = torch.ones_like(u)
    if case["gate"]:
        z = clean("z")
        r = 1 / (1 + torch.exp(-z))
        gate = z * r
    h = f["state"].clone() if f["state"] is not None else u.new_zeros(b, d, n)
    first, kept, ys = h.clone(), [], torch.empty_like(u)

    def row(x, t):
        return x[:, t].reshape(b, groups, 1, n).expand(b, groups, per, n).reshape(b, d, n)

    for t in range(l):
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * u[:, t])[..., None] * row(Bm, t)
        ys[:, t] = (h * row(Cm, t)).sum(-1) + D * u[:, t]
        if op == "scan_train":
            kept.append(h)
    y = (ys * gate).masked_fill(~there, 0.0)
    if op == "scan_step":
        return {"y": y[:, 0], "state": h}
    out = {"y": y, "state": h}
    if op == "scan_fwd":
        return out
    gy = clean("gy")
    if case["gate"]:
        out["gz"] = gy * ys * (r + z * r * (1 - r))
        gy = gy * gate
    gu, gdt = torch.empty_like(u), torch.empty_like(u)
    gA, gB, gC = torch.zeros_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    G = torch.zeros_like(h)
    for t in reversed(range(l)):
        B1, C1, dl = row(Bm, t), row(Cm, t), delta[:, t, :, None]
        G = G + gy[:, t, :, None] * C1
        before = kept[t - 1] if t else first
        a = torch.exp(dl * A)
        through = G * a * before
        GB = (G * B1).sum(-1)
        gu[:, t] = GB * delta[:, t] + D * gy[:, t]
        gdt[:, t] = GB * u[:, t] + (through * A).sum(-1)
        gA += (through * dl).sum(0)
        gB[:, t] = (G * (dl * u[:, t, :, None])).view(b, groups, per, n).sum(2).reshape(b, -1)
        gC[:, t] = (gy[:, t, :, None] * kept[t]).view(b, groups, per, n).sum(2).reshape(b, -1)
        G = G * a
    gdt = (gdt / (1 + torch.exp(-raw))).masked_fill(~there, 0.0)
    out.update(gu=gu, gdt=gdt, gdt_bias=gdt.sum((0, 1)), gD=(gy * u).sum((0, 1)), gA=gA, gB=gB, gC=gC)
    if f["state"] is not None:
        out["gstate"] = G
    return out
