"""The operators of a channels-last sequence block: what is measured, and their plain forms.

Rows of a feature map (pixels) or of a camera stream (frames) pass through blocks of

* a layer norm over the channels of each row: tensors (B, L, C);
* a linear attention with a decay for each head: S_t = lambda_h S_{t-1} + k_t v_t^T,
  y_t = scale q_t S_t, over heads adjacent in a row: q, k (B, L, H * Dk), v, y (B, L, H * Dv),
  with the state S (B, H, Dk, Dv) carried in and out; and its form for one token;
* a gated feed-forward product: y = (act(x W_g) * (x W_u)) W_out over M rows of C channels,
  with W_in = [W_g | W_u] (C, 2 F) and W_out (F, C).

All three have a forward and a backward pass.  A ragged batch gives a length per sequence;
rows at or past it are not read (they hold NaN here), their outputs and gradients are zero.

`run` computes the plain form in 32 bits from elementary operations, or, where `own` is
true, calls the library.  `exact` is the definition in 64 bits, one token after another.
"""
import math

import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
BYTES = {F32: 4, BF16: 2, F16: 2}
EPS = 1e-5
CHUNK = 128  # rows that the plain attention takes as one block


# ---------------------------------------------------------------- the cases

def _ln(name, op, b, l, c, dtype, ragged=False):
    return {"name": name, "op": op, "b": b, "l": l, "c": c, "dtype": dtype, "ragged": ragged}


def _attn(name, op, b, l, h, dk, dv, dtype, state=False, ragged=False):
    return {"name": name, "op": op, "b": b, "l": l, "h": h, "dk": dk, "dv": dv, "dtype": dtype, "state": state,
            "ragged": ragged}


def _ffn(name, op, m, c, f, dtype, act):
    return {"name": name, "op": op, "m": m, "c": c, "f": f, "dtype": dtype, "act": act}


def listed():
    return [
        # one new frame of 64 streams: latency
        _ln("norm one token", "ln_fwd", 64, 1, 512, BF16),
        # a training step on image rows: 7 cameras x 32 rows of 1024 pixels
        _ln("norm row training", "ln_train", 224, 1024, 512, BF16),
        # ragged rows, channels that are no multiple of a wide load's
        _ln("norm ragged training", "ln_train", 5, 1537, 330, F32, ragged=True),
        # one new frame for each of 64 streams: the states are read and written
        _attn("attention one token", "attn_step", 64, 1, 16, 64, 64, BF16, state=True),
        # one image as a raster of 16384 pixel tokens: few heads, a long axis
        _attn("attention long prompt", "attn_fwd", 1, 16384, 8, 64, 64, BF16),
        # prompts of pixel tokens that go on from a carried state, wide heads
        _attn("attention wide prompt", "attn_fwd", 8, 4096, 8, 128, 128, BF16, state=True),
        # a training step on image rows
        _attn("attention row training", "attn_train", 224, 1024, 4, 64, 64, BF16),
        # ragged rows, odd head sizes, a carried state and its gradients
        _attn("attention ragged training", "attn_train", 5, 1537, 4, 41, 82, F32, state=True, ragged=True),
        # one new frame for each of 64 streams: the weights are read
        _ffn("feed-forward one token", "ffn_fwd", 64, 1024, 2816, BF16, "silu"),
        # the maps of seven cameras, inference
        _ffn("feed-forward maps", "ffn_fwd", 7 * 16384, 512, 2048, BF16, "gelu"),
        # a training step on image rows
        _ffn("feed-forward training", "ffn_train", 32768, 1024, 2816, BF16, "silu"),
        # widths that fill no tile, ragged rows packed one after another
        _ffn("feed-forward odd training", "ffn_train", 5 * 1537, 328, 872, F16, "gelu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_train", "attn_fwd", "attn_train", "attn_step", "ffn_fwd", "ffn_train"])
    if op.startswith("ln"):
        # a gradient of a few values is what cancellation leaves: from 16 channels on
        c = _log(rng, 16, 4096)
        b = _log(rng, 1, 256)
        l = _log(rng, 1, max(2, (1 << 26) // (b * c)))
        case = _ln("", op, b, l, c, rng.choice([F32, BF16, F16]), rng.random() < 0.3)
    elif op.startswith("attn"):
        h = _log(rng, 1, 16)
        dk, dv = (rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128, rng.randint(8, 128)]) for _ in range(2))
        b = _log(rng, 1, 256)
        l = 1 if op == "attn_step" else _log(rng, 1, max(2, min(1 << 15, (1 << 25) // (b * h * max(dk, dv)))))
        one = op == "attn_step"
        case = _attn("", op, b, l, h, dk, dv, rng.choice([F32, BF16, BF16, F16]), one or rng.random() < 0.5,
                     not one and rng.random() < 0.4)
    else:
        c, f = 8 * _log(rng, 1, 256), 8 * _log(rng, 1, 512)
        m = _log(rng, 1, max(2, min(1 << 17, (1 << 36) // (c * f))))
        case = _ffn("", op, m, c, f, rng.choice([BF16, F16]), rng.choice(["none", "silu", "gelu"]))
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
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    t = TORCH[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)

    s = {"case": case}
    if op.startswith("ffn"):
        m, c, f = case["m"], case["c"], case["f"]
        s["x"] = normal(m, c, dtype=t)
        s["w_in"], s["w_out"] = normal(c, 2 * f, scale=c ** -0.5, dtype=t), normal(f, c, scale=f ** -0.5, dtype=t)
        if op == "ffn_train":
            s["gy"] = normal(m, c, dtype=t)
        return s

    b, l = case["b"], case["l"]
    lens = _lengths(b, l, seed) if case["ragged"] else None
    s["lens"] = lens

    def blank(x):
        """NaN in the rows that a ragged batch does not have."""
        if lens is not None:
            gone = torch.arange(l, device="cuda") >= lens[:, None]
            x.masked_fill_(gone[:, :, None], float("nan"))
        return x

    if op.startswith("ln"):
        c = case["c"]
        # a residual stream: every channel with an offset and a scale of its own
        x = normal(b, l, c) * (0.5 + torch.rand(c, generator=g, device="cuda")) + normal(c, scale=0.5)
        s["x"] = blank(x.to(t))
        s["gamma"], s["beta"] = normal(c, scale=0.1, shift=1.0), normal(c, scale=0.1)
        if op == "ln_train":
            s["gy"] = blank(normal(b, l, c, dtype=t))
        return s

    h, dk, dv = case["h"], case["dk"], case["dv"]
    # q, k and v are slices of one projection's output rows
    qkv = blank(normal(b, l, h * (2 * dk + dv), dtype=t))
    s["q"], s["k"], s["v"] = qkv[:, :, :h * dk], qkv[:, :, h * dk:2 * h * dk], qkv[:, :, 2 * h * dk:]
    # heads that remember from 32 rows to a few thousand
    s["decay"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.rand(h, generator=g, device="cuda")))
    s["state"] = normal(b, h, dk, dv, scale=2.0) if case["state"] else None
    if op == "attn_step":
        for key in ("q", "k", "v"):
            s[key] = s[key][:, 0]
    if op == "attn_train":
        s["gy"] = blank(normal(b, l, h * dv, dtype=t))
        s["gstate_out"] = normal(b, h, dk, dv) if case["state"] else None
    return s


# ---------------------------------------------------------------- plain forms, 32 bits

def _live(s, l):
    """The rows that are there, (B, L, 1), or None where all are."""
    return None if s["lens"] is None else (torch.arange(l, device="cuda") < s["lens"][:, None])[:, :, None]


def _rows(x, live):
    x = x.float()
    return x if live is None else torch.where(live, x, torch.zeros_like(x))


def _ln_plain(s):
    t = s["x"].dtype
    live = _live(s, s["case"]["l"])
    x = _rows(s["x"], live)
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * rstd
    out = {"y": _rows(x * s["gamma"] + s["beta"], live).to(t)}
    if s["case"]["op"] == "ln_train":
        g = _rows(s["gy"], live)
        out["ggamma"], out["gbeta"] = (g * x).sum((0, 1)), g.sum((0, 1))
        g = g * s["gamma"]
        gx = rstd * (g - g.mean(-1, keepdim=True) - x * (g * x).mean(-1, keepdim=True))
        out["gx"] = _rows(gx, live).to(t)
    return out


def _attn_plain(s):
    case = s["case"]
    b, l, h, dk, dv = (case[k] for k in ("b", "l", "h", "dk", "dv"))
    t, a, scale = s["q"].dtype, s["decay"], case["dk"] ** -0.5
    if case["op"] == "attn_step":
        q, k, v = (s[key].float().view(b, h, -1) for key in ("q", "k", "v"))
        S = torch.exp(a)[:, None, None] * s["state"] + k[..., :, None] * v[..., None, :]
        s["state"].copy_(S)
        return {"y": (scale * q[..., None] * S).sum(-2).view(b, h * dv).to(t), "state": s["state"]}

    live = _live(s, l)
    n = min(CHUNK, l)
    chunks = -(-l // n)

    def split(key, d):  # (B, L, H * d) -> (B, H, chunks, n, d), zeros behind the last row
        x = _rows(s[key], live)
        x = torch.cat([x, x.new_zeros(b, chunks * n - l, h * d)], 1)
        return x.view(b, chunks, n, h, d).permute(0, 3, 1, 2, 4)

    def join(x, d):
        return _rows(x.permute(0, 2, 3, 1, 4).reshape(b, chunks * n, h * d)[:, :l], live).to(t)

    def power(count):  # decay to the power of `count`, for every head; zero where it is negative
        count = count.float()
        return torch.exp(a.view(h, *[1] * count.dim()) * count.clamp(min=0)) * (count >= 0)

    q, k, v = split("q", dk) * scale, split("k", dk), split("v", dv)
    row = torch.arange(n, device="cuda")
    among = torch.arange(chunks, device="cuda")
    mask = power(row[:, None] - row)[:, None]                     # (H, 1, n, n): rows i on rows j <= i
    start = power(row + 1)[:, None, :, None]                      # the state ahead of a chunk on row i
    end = power(n - 1 - row)[:, None, :, None]                    # row j on the state behind its chunk
    between = power(n * (among[:, None] - 1 - among))             # (H, c, c'): chunk c' on the state ahead of chunk c
    U = k.transpose(-1, -2) @ (end * v)                           # (B, H, chunks, Dk, Dv)
    S = (between @ U.reshape(b, h, chunks, dk * dv)).view(b, h, chunks, dk, dv)
    if s["state"] is not None:
        S = S + power(n * among)[..., None, None] * s["state"][:, :, None]
    P = (q @ k.transpose(-1, -2)) * mask
    out = {"y": join(P @ v + start * (q @ S), dv)}
    # the state behind each sequence's last row
    ends = s["lens"] if s["lens"] is not None else torch.full((b,), l, device="cuda")
    place = torch.arange(chunks * n, device="cuda").view(chunks, n)
    left = power(ends[:, None, None] - 1 - place).transpose(0, 1)[..., None]  # (B, H, chunks, n, 1)
    gone = power(ends).transpose(0, 1)[..., None, None]                      # (B, H, 1, 1)
    state = (k.transpose(-1, -2) @ (left * v)).sum(2)
    out["state"] = state if s["state"] is None else state + gone * s["state"]
    if case["op"] == "attn_train":
        g = split("gy", dv)
        G = (between.transpose(-1, -2) @ (q.transpose(-1, -2) @ (start * g)).reshape(b, h, chunks, dk * dv))
        G = G.view(b, h, chunks, dk, dv)  # the gradient of the state behind each chunk
        gP = (g @ v.transpose(-1, -2)) * mask
        gk = gP.transpose(-1, -2) @ q + end * (v @ G.transpose(-1, -2))
        gv = P.transpose(-1, -2) @ g + end * (k @ G)
        first = (q.transpose(-1, -2) @ (power(place + 1)[..., None] * g)).sum(2)
        if s["gstate_out"] is not None:
            last = s["gstate_out"][:, :, None]
            gk = gk + left * (v @ last.transpose(-1, -2))
            gv = gv + left * (k @ last)
            first = first + gone * s["gstate_out"]
        out["gq"] = join(scale * (gP @ k + start * (g @ S.transpose(-1, -2))), dk)
        out["gk"], out["gv"] = join(gk, dk), join(gv, dv)
        if s["state"] is not None:
            out["gstate"] = first
    return out


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


def _ffn_plain(s):
    kind, f, t = s["case"]["act"], s["case"]["f"], s["x"].dtype
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    pre = x @ w_in
    a, u = pre[:, :f], pre[:, f:]
    act = _act(a, kind)
    h = act * u
    out = {"y": (h @ w_out).to(t)}
    if s["case"]["op"] == "ffn_train":
        gy = s["gy"].float()
        gh = gy @ w_out.t()
        gpre = torch.cat([gh * u * _act_slope(a, kind), gh * act], 1)
        out["gx"], out["gw_in"], out["gw_out"] = (gpre @ w_in.t()).to(t), (x.t() @ gpre).to(t), (h.t() @ gy).to(t)
    return out


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """The descriptor, outputs and workspaces that a program sets up once for its sizes."""
    from spatially_sharded_cnn_gb300 import hc
    case = s["case"]
    op, t = case["op"], TORCH[case["dtype"]]
    train = op.endswith("train")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def space(got):
        hc.check(got[0], "workspace size")
        return empty(max(got[1], 16), dtype=torch.uint8), got[1]

    p = {"hc": hc}
    if op.startswith("ln"):
        b, l, c = case["b"], case["l"], case["c"]
        p["d"] = hc.layernorm_desc(B=b, L=l, C=c, eps=EPS, dtype=t)
        p["out"] = {"y": empty(b, l, c, dtype=t)}
        p["mean"] = p["rstd"] = None
        if train:
            p["ws"], p["nb"] = space(hc.hc_layernorm_workspace_size(p["d"]))
            p["mean"], p["rstd"] = empty(b, l), empty(b, l)
            p["out"].update(gx=empty(b, l, c, dtype=t), ggamma=empty(c), gbeta=empty(c))
    elif op.startswith("attn"):
        b, l, h, dk, dv = (case[k] for k in ("b", "l", "h", "dk", "dv"))
        p["d"] = hc.linear_attn_desc(B=b, L=l, H=h, Dk=dk, Dv=dv, scale=dk ** -0.5, dtype=t)
        if op == "attn_step":
            p["out"] = {"y": empty(b, h * dv, dtype=t), "state": s["state"]}
            return p
        p["ws"], p["nb"] = space(hc.hc_linear_attn_workspace_size(p["d"], int(train)))
        p["out"] = {"y": empty(b, l, h * dv, dtype=t), "state": empty(b, h, dk, dv)}
        if train:
            p["out"].update(gq=empty(b, l, h * dk, dtype=t), gk=empty(b, l, h * dk, dtype=t),
                            gv=empty(b, l, h * dv, dtype=t))
            if s["state"] is not None:
                p["out"]["gstate"] = empty(b, h, dk, dv)
    else:
        m, c, f = case["m"], case["c"], case["f"]
        act = {"none": hc.HC_PW_NONE, "silu": hc.HC_PW_SILU, "gelu": hc.HC_PW_GELU}[case["act"]]
        p["d"] = hc.gated_ffn_desc(M=m, C=c, F=f, act=act, dtype=t)
        p["ws"], p["nb"] = space(hc.hc_gated_ffn_workspace_size(p["d"], int(train)))
        p["out"] = {"y": empty(m, c, dtype=t)}
        if train:
            p["out"].update(gx=empty(m, c, dtype=t), gw_in=empty(c, 2 * f, dtype=t), gw_out=empty(f, c, dtype=t))
    return p


def _library(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    hc, d, out, op = p["hc"], p["d"], p["out"], s["case"]["op"]
    if op.startswith("ln"):
        hc.check(hc.hc_layernorm_fwd(d, s["x"], s["gamma"], s["beta"], out["y"], p["mean"], p["rstd"], lens=s["lens"]))
        if op == "ln_train":
            hc.check(hc.hc_layernorm_bwd(d, s["x"], s["gamma"], p["mean"], p["rstd"], s["gy"], out["gx"], out["ggamma"],
                                         out["gbeta"], lens=s["lens"], ws=p["ws"], ws_bytes=p["nb"]))
    elif op == "attn_step":
        hc.check(hc.hc_linear_attn_step(d, s["q"], s["k"], s["v"], s["state"], out["y"], log_decay=s["decay"]))
    elif op.startswith("attn"):
        hc.check(hc.hc_linear_attn_fwd(d, s["q"], s["k"], s["v"], out["y"], log_decay=s["decay"], h0=s["state"],
                                       hT=out["state"], lens=s["lens"], ws=p["ws"], ws_bytes=p["nb"]))
        if op == "attn_train":
            hc.check(hc.hc_linear_attn_bwd(d, s["q"], s["k"], s["v"], s["gy"], out["gq"], out["gk"], out["gv"],
                                           log_decay=s["decay"], h0=s["state"], ghT=s["gstate_out"],
                                           gh0=out.get("gstate"), lens=s["lens"], ws=p["ws"], ws_bytes=p["nb"]))
    else:
        hc.check(hc.hc_gated_ffn_fwd(d, s["x"], s["w_in"], s["w_out"], out["y"], ws=p["ws"], ws_bytes=p["nb"]))
        if op == "ffn_train":
            hc.check(hc.hc_gated_ffn_bwd(d, s["x"], s["w_in"], s["w_out"], s["gy"], out["gx"], out["gw_in"],
                                         out["gw_out"], ws=p["ws"], ws_bytes=p["nb"]))
    return out


def run(state):
    if own:
        return _library(state)
    op = state["case"]["op"]
    return _ln_plain(state) if op.startswith("ln") else _attn_plain(state) if op.startswith("attn") else _ffn_plain(state)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op.startswith("ffn"):
        m, c, f = case["m"], case["c"], case["f"]
        one = 2 * m * c * f  # operations of one of the products
        if op == "ffn_fwd":
            return {"bytes": (2 * m * c + 3 * c * f) * e, "flops": 3 * one}
        # x, gy, y and gx; the weights and their gradients
        return {"bytes": (4 * m * c + 6 * c * f) * e, "flops": 9 * one}
    b, l = case["b"], case["l"]
    # lengths of a ragged batch lie evenly between 0 and l: half of its input rows are there
    there = 0.5 if case["ragged"] else 1.0
    if op.startswith("ln"):
        m, c = b * l * case["c"], case["c"]
        if op == "ln_fwd":
            return {"bytes": int((1 + there) * m * e) + 8 * c, "flops": 8 * m}
        # x and gy in; y and gx out
        return {"bytes": int((2 + 2 * there) * m * e) + 16 * c, "flops": 20 * m}
    h, dk, dv = case["h"], case["dk"], case["dv"]
    rows, states = b * l * h, 4 * b * h * dk * dv
    # a row and head of the recurrence: k v^T into the decayed state, q times the state
    one = 5 * dk * dv
    if op != "attn_train":
        carried = (1 + case["state"]) * states
        return {"bytes": int(rows * (there * (2 * dk + dv) + dv) * e) + carried, "flops": int(there * rows * one)}
    carried = (1 + 3 * case["state"]) * states  # the state out; the one in, and the gradients of both
    # q, k, v and gy in; y, gq, gk and gv out; the state's gradient as the state, and three products with the two
    return {"bytes": int(rows * (there * (2 * dk + 2 * dv) + 2 * dk + 2 * dv) * e) + carried,
            "flops": int(there * rows * 14 * dk * dv)}


# ---------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op.startswith("ffn"):
        train = op == "ffn_train"
        x, w_in, w_out = (f[k].requires_grad_(train) for k in ("x", "w_in", "w_out"))
        gate, up = x @ w_in[:, :case["f"]], x @ w_in[:, case["f"]:]
        if case["act"] == "silu":
            gate = gate / (1 + torch.exp(-gate))
        elif case["act"] == "gelu":
            gate = gate * torch.special.ndtr(gate)
        y = (gate * up) @ w_out
        out = {"y": y.detach()}
        if train:
            out["gx"], out["gw_in"], out["gw_out"] = torch.autograd.grad(y, (x, w_in, w_out), f["gy"])
        return out

    b, l = case["b"], case["l"]
    ends = f["lens"].long() if f["lens"] is not None else torch.full((b,), l, device="cuda")
    there = torch.arange(l, device="cuda")[None, :, None] < ends[:, None, None]

    def clean(key):
        return f[key][:, None] if op.endswith("step") else f[key].masked_fill(~there, 0.0)

    if op.startswith("ln"):
        x = clean("x").requires_grad_(True)
        gamma, beta = f["gamma"].requires_grad_(True), f["beta"].requires_grad_(True)
        v, m = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        y = ((x - m) / torch.sqrt(v + EPS) * gamma + beta).masked_fill(~there, 0.0)
        out = {"y": y.detach()}
        if op == "ln_train":
            out["gx"], out["ggamma"], out["gbeta"] = torch.autograd.grad(y, (x, gamma, beta), clean("gy"))
        return out

    h, dk, dv = case["h"], case["dk"], case["dv"]
    scale, decay = dk ** -0.5, torch.exp(f["decay"])[None, :, None, None]
    on = there[:, :, :, None]  # a row that is not there leaves the state as it is

    def heads(x):
        return x.reshape(b, -1, h, x.shape[-1] // h)

    q, k, v = heads(clean("q")), heads(clean("k")), heads(clean("v"))
    g = heads(clean("gy")) if op == "attn_train" else None
    S = f["state"].clone() if f["state"] is not None else q.new_zeros(b, h, dk, dv)
    y, gq, gk, gv = torch.empty_like(v), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for i in range(l):
        S = torch.where(on[:, i, :, None], decay * S, S) + k[:, i, :, :, None] * v[:, i, :, None, :]
        y[:, i] = scale * torch.einsum("bhk,bhkv->bhv", q[:, i], S)
        if g is not None:
            gq[:, i] = scale * torch.einsum("bhv,bhkv->bhk", g[:, i], S)
    if op == "attn_step":
        return {"y": y.reshape(b, h * dv), "state": S}
    out = {"y": y.reshape(b, l, h * dv).masked_fill(~there, 0.0), "state": S}
    if g is None:
        return out
    G = f["gstate_out"].clone() if f["gstate_out"] is not None else torch.zeros_like(S)
    for i in reversed(range(l)):
        G = G + scale * q[:, i, :, :, None] * g[:, i, :, None, :]
        gk[:, i] = torch.einsum("bhv,bhkv->bhk", v[:, i], G)
        gv[:, i] = torch.einsum("bhk,bhkv->bhv", k[:, i], G)
        G = torch.where(on[:, i, :, None], decay * G, G)
    out.update(gq=gq.reshape(b, l, h * dk).masked_fill(~there, 0.0), gk=gk.reshape(b, l, h * dk).masked_fill(~there, 0.0),
               gv=gv.reshape(b, l, h * dv).masked_fill(~there, 0.0))
    if f["state"] is not None:
        out["gstate"] = G
    return out
