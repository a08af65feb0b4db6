"""The operators around the scan of a state space block, as cases to time and compare.

Four operators: the short causal convolution (forward, single token, backward), the selective scan
with a decay of its own for every channel and state entry (forward, single token, backward), the
gated norm behind the scan and the norm with residual before a block (each forward and backward).
Where ``own`` is false, ``run`` computes them in plain torch operations in 32 bits; where it is
true, it calls this package.
"""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token for each of a few sequences that decode together: latency alone counts
        dict(name="conv_decode", op="conv_step", io=BF16, batch=4, seqlen=1, nseq=4, channels=5376,
             width=4, split=128, pad=5120),
        # prompts of unequal length packed into one row of tokens, x, B and C of a small layer
        dict(name="conv_prompts", op="conv", io=BF16, batch=1, seqlen=5003, nseq=7, packed=True,
             channels=1792, width=4, split=128, pad=1536, initial=True),
        # a long prompt in two rows, x, B and C of a large layer, read from the projection's rows
        dict(name="conv_long", op="conv", io=BF16, batch=2, seqlen=8192, nseq=2, channels=5376,
             width=4, split=128, pad=5120, initial=False),
        # the same layer's training step: gradients of x, B and C come in 32 bits from the scan
        dict(name="conv_train", op="conv_backward", io=BF16, batch=2, seqlen=8192, nseq=2,
             channels=5376, width=4, split=128, pad=5120, initial=False, dy32=True),
        # one token for each of a serving batch
        dict(name="scan_decode", op="scan_step", io=BF16, batch=64, seqlen=1, nseq=64,
             channels=5120, dstate=16, groups=1, gate=True, pad=5120),
        # a few packed prompts in a small layer, in 32 bits
        dict(name="scan_prompts", op="scan", io=F32, batch=1, seqlen=3001, nseq=5, packed=True,
             channels=1536, dstate=16, groups=1, gate=True, pad=0, initial=True),
        # long prompts in a large layer
        dict(name="scan_long", op="scan", io=BF16, batch=2, seqlen=8192, nseq=2, channels=5120,
             dstate=16, groups=1, gate=True, pad=5120, initial=False),
        # a training step of the large layer
        dict(name="scan_train", op="scan_backward", io=BF16, batch=2, seqlen=4096, nseq=2,
             channels=5120, dstate=16, groups=1, gate=True, pad=5120, initial=False),
        # one token a sequence behind the scan of a large layer
        dict(name="gated_decode", op="gated", io=BF16, batch=64, seqlen=1, channels=5120, groups=1,
             first=False, pad=5120),
        # training: the wide grouped layer, the norm over each of its groups
        dict(name="gated_train", op="gated_backward", io=BF16, batch=2, seqlen=8192, channels=8192,
             groups=8, first=False, pad=8192),
        # a long prompt's residual stream in 32 bits, each channel of the block's output scaled
        dict(name="residual_long", op="residual", io=BF16, batch=2, seqlen=8192, channels=2560,
             res32=True, scale=True),
        # training of a small layer, all in 32 bits
        dict(name="residual_train", op="residual_backward", io=F32, batch=4, seqlen=2048,
             channels=768, res32=True, scale=False),
    ]


def _between(rng, low, high, step=1):
    """A whole multiple of `step` between the two, spread over the logarithm."""
    return max(low, step * round(math.exp(rng.uniform(math.log(low), math.log(high))) / step))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_step", "conv_backward", "scan", "scan", "scan_step",
                     "scan_backward", "scan_backward", "gated", "gated_backward", "residual",
                     "residual_backward"])
    c = dict(op=op, io=rng.choice([BF16, BF16, F32]))
    if op.endswith("_step"):
        c.update(batch=_between(rng, 1, 128), seqlen=1)
        c["nseq"] = c["batch"]
    elif op.startswith("conv") or op.startswith("scan"):
        rows = _between(rng, 1, 6000)
        if rng.random() < 0.5:
            c.update(batch=1, seqlen=rows, nseq=_between(rng, 1, 24), packed=True)
        else:
            batch = min(rows, _between(rng, 1, 8))
            c.update(batch=batch, seqlen=max(1, rows // batch), nseq=batch)
        c["initial"] = rng.random() < 0.5
    else:
        c.update(batch=_between(rng, 1, 4), seqlen=_between(rng, 1, 4000))
    if op.startswith("conv"):
        c.update(channels=_between(rng, 64, 6000, 8), width=rng.choice([2, 3, 4, 4, 4]),
                 pad=rng.choice([0, 64, 1544]))
        c["split"] = rng.choice([0, 8, 16])
        if op == "conv_backward":
            c["dy32"] = rng.random() < 0.5
    elif op.startswith("scan"):
        c.update(groups=rng.choice([1, 1, 2]), dstate=rng.choice([8, 16, 16, 16, 32]),
                 gate=rng.random() < 0.7, pad=rng.choice([0, 64, 520]))
        c["channels"] = c["groups"] * _between(rng, 64, 1600, 8)
    elif op.startswith("gated"):
        c.update(groups=rng.choice([1, 1, 4]), first=rng.random() < 0.5,
                 pad=rng.choice([0, 64, 520]))
        c["channels"] = c["groups"] * _between(rng, 32, 2000, 8)
    else:
        c.update(channels=_between(rng, 64, 8192, 8), scale=rng.random() < 0.5)
        c["res32"] = c["io"] == F32 or rng.random() < 0.5
    return c


# ---- inputs --------------------------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _slice(g, c, width, dtype):
    """[batch, seqlen, width] values that stand behind `pad` others in each row."""
    return _normal(g, c["batch"], c["seqlen"], c.get("pad", 0) + width, dtype=dtype)[
        ..., c.get("pad", 0):]


def _offsets(g, c):
    """Where each of nseq packed sequences starts, and the end: random cuts, some may be empty."""
    cuts = torch.randint(0, c["seqlen"] + 1, (c["nseq"] - 1,), generator=g, device="cuda")
    ends = torch.tensor([0, c["seqlen"]], device="cuda")
    return torch.cat([ends, cuts]).sort().values.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    io, op = TYPES[c["io"]], c["op"]
    B, L, C = c["batch"], c["seqlen"], c["channels"]
    s = dict(case=c, op=op)
    s["starts"] = _offsets(g, c) if c.get("packed") else None
    one = op.endswith("_step")
    if op.startswith("conv"):
        W = c["width"]
        s["x"] = _slice(g, c, C, io)
        s["weight"] = _normal(g, C, W, scale=W ** -0.5)
        s["bias"] = _normal(g, C, scale=0.1)
        s["state"] = _normal(g, c["nseq"], W - 1, C, dtype=io) if one or c.get("initial") else None
        n = c["split"]
        s["split"] = (C - 2 * n, n, n) if n else None
        if op == "conv_backward":
            to = torch.float32 if c["dy32"] else io
            s["dy"] = tuple(_normal(g, B, L, k, dtype=to) for k in s["split"] or (C,))
            s["dfinal"] = _normal(g, c["nseq"], W - 1, C) if c["initial"] else None
    elif op.startswith("scan"):
        N, G = c["dstate"], c["groups"]
        s["x"] = _normal(g, B, L, C, dtype=io)
        s["dt"] = _normal(g, B, L, C, dtype=io, scale=0.5)
        step = torch.exp(torch.rand(C, generator=g, device="cuda") * math.log(100) - math.log(1e3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["A"] = -(torch.rand(C, N, generator=g, device="cuda") * 15 + 1)
        # B and C stand side by side in the rows of one projection
        bc = _normal(g, B, L, 64 + 2 * G * N, dtype=io)[..., 64:]
        s["B"], s["C"] = (t.unflatten(-1, (G, N)) for t in bc.split(G * N, dim=-1))
        s["D"] = _normal(g, C, scale=0.1) + 1
        s["z"] = _slice(g, c, C, io) if c["gate"] else None
        s["state"] = _normal(g, c["nseq"], C, N) if one or c.get("initial") else None
        if op == "scan_backward":
            s["dy"] = _normal(g, B, L, C, dtype=io)
            s["dfinal"] = _normal(g, c["nseq"], C, N) if c["initial"] else None
    elif op.startswith("gated"):
        s["x"] = _normal(g, B, L, C, dtype=io)
        s["z"] = _slice(g, c, C, io)
        s["weight"] = _normal(g, C, scale=0.1) + 1
        if op == "gated_backward":
            s["dy"] = _normal(g, B, L, C, dtype=io)
    else:
        rt = torch.float32 if c["res32"] else io
        s["x"] = _normal(g, B, L, C, dtype=io)
        s["residual"] = _normal(g, B, L, C, dtype=rt, scale=3.0)
        s["weight"] = _normal(g, C, scale=0.1) + 1
        s["scale"] = _normal(g, C, scale=0.1) + 0.5 if c["scale"] else None
        if op == "residual_backward":
            s["dy"] = _normal(g, B, L, C, dtype=io)
            s["dres"] = _normal(g, B, L, C, dtype=rt)
    return s


EPS = 1e-5


# ---- what each pass cannot do without ------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    rows, C = c["batch"] * c["seqlen"], c["channels"]
    e = 2 if c["io"] == BF16 else 4
    el = rows * C
    if op.startswith("conv"):
        W, states = c["width"], c["nseq"] * (c["width"] - 1) * C
        params = C * (W + 1) * 4
        if op == "conv_backward":
            dy = 4 if c["dy32"] else e
            state_bytes = states * (4 + (e + 4 if c["initial"] else 0))
            return dict(bytes=el * (2 * e + dy) + 2 * params + state_bytes,
                        flops=el * (6 * W + 8))
        given = op == "conv_step" or c["initial"]
        return dict(bytes=2 * el * e + params + states * e * (2 if given else 1),
                    flops=el * (2 * W + 4))
    if op.startswith("scan"):
        N, G = c["dstate"], c["groups"]
        states, bc = c["nseq"] * C * N * 4, 2 * rows * G * N * e
        params = C * (N + 2) * 4
        z = 1 if c["gate"] else 0
        given = op == "scan_step" or c["initial"]
        if op == "scan_backward":
            state_bytes = states * (3 if given else 1)
            return dict(bytes=el * e * (5 + 2 * z) + 2 * bc + 2 * params + state_bytes,
                        flops=el * N * 22)
        return dict(bytes=el * e * (3 + z) + bc + params + states * (2 if given else 1),
                    flops=el * N * 7)
    if op.startswith("gated"):
        back = op == "gated_backward"
        return dict(bytes=el * e * (5 if back else 3) + C * 4 * (2 if back else 1),
                    flops=el * (20 if back else 10))
    r, scale = 4 if c["res32"] else e, 4 * C if c["scale"] else 0
    if op == "residual_backward":
        # x is read for the scale's gradient alone; without a scale one gradient serves both
        dx = el * e if c["scale"] or r != e else 0
        return dict(bytes=el * (e + 3 * r) + dx + (el * e + 2 * scale if c["scale"] else 0)
                    + 8 * C, flops=el * 14)
    return dict(bytes=el * 2 * (e + r) + 4 * C + scale, flops=el * 6)


# ---- the framework's calls -----------------------------------------------------------------------

def _own(s):
    import mamba_ssd_chunked_cumsum_amd as ssd

    c, op = s["case"], s["op"]
    if op == "conv":
        return ssd.conv(s["x"], s["weight"], s["bias"], s["state"], split=s["split"],
                        cu_seqlens=s["starts"])
    if op == "conv_step":
        x = s["x"].squeeze(1)
        return ssd.conv_step(s["state"], x, s["weight"], s["bias"], split=s["split"])
    if op == "conv_backward":
        dy = s["dy"] if s["split"] else s["dy"][0]
        return ssd.conv_backward(s["x"], s["weight"], s["bias"], dy, s["state"], s["dfinal"],
                                 cu_seqlens=s["starts"])
    if op == "scan":
        return ssd.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                  s["state"], dt_bias=s["dt_bias"], dt_softplus=True,
                                  cu_seqlens=s["starts"])
    if op == "scan_step":
        one = (None if s[k] is None else s[k].squeeze(1) for k in ("x", "dt", "B", "C", "z"))
        x, dt, B, C, z = one
        return ssd.selective_step(s["state"], x, dt, s["A"], B, C, s["D"], z,
                                  dt_bias=s["dt_bias"], dt_softplus=True)
    if op == "scan_backward":
        return ssd.selective_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                      s["dy"], s["state"], s["dfinal"], dt_bias=s["dt_bias"],
                                      dt_softplus=True, cu_seqlens=s["starts"])
    if op == "gated":
        return ssd.gated_norm(s["x"], s["z"], s["weight"], eps=EPS, ngroups=c["groups"],
                              norm_before_gate=c["first"])
    if op == "gated_backward":
        return ssd.gated_norm_backward(s["x"], s["z"], s["weight"], s["dy"], eps=EPS,
                                       ngroups=c["groups"], norm_before_gate=c["first"])
    if op == "residual":
        return ssd.residual_norm(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS)
    return ssd.residual_norm_backward(s["x"], s["residual"], s["weight"], s["dy"], s["dres"],
                                      scale=s["scale"], eps=EPS)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- plain forms ---------------------------------------------------------------------------------

def _rows(s, L, device):
    """(offsets [nseq + 1], the sequence of each row) of flattened rows; rows beyond the last
    sequence do not occur."""
    c = s["case"]
    if s["starts"] is not None:
        at = s["starts"].long()
    else:
        at = torch.arange(c["batch"] + 1, device=device) * L
    rows = torch.arange(c["batch"] * L, device=device)
    return at, torch.searchsorted(at[1:], rows, right=True)


def _window(s):
    """The inputs with each sequence's W - 1 earlier ones before it, as rows; and where the rows of
    tap k, of the tokens, before each sequence and at its end stand in them."""
    c, x = s["case"], s["x"].float()
    W, L = c["width"], c["seqlen"]
    if s["starts"] is None:
        state = x.new_zeros(x.shape[0], W - 1, x.shape[-1]) if s["state"] is None else s["state"]
        at = [(slice(None), slice(k, k + L)) for k in range(W)]
        return (torch.cat([state.float(), x], 1), at, at[W - 1], (slice(None), slice(0, W - 1)),
                (slice(None), slice(L, L + W - 1)))
    x = x[0]
    at, seq = _rows(s, L, x.device)
    ahead = torch.arange(at.numel() - 1, device=x.device) * (W - 1)
    back = torch.arange(W - 1, device=x.device)
    mine = torch.arange(L, device=x.device) + (seq + 1) * (W - 1)
    before, last = ((m + ahead)[:, None] + back for m in (at[:-1], at[1:]))
    rows = x.new_zeros(L + ahead.numel() * (W - 1), x.shape[-1])
    rows[mine] = x
    if s["state"] is not None:
        rows[before] = s["state"].float()
    return rows, [mine - (W - 1) + k for k in range(W)], mine, before, last


def _conv_sum(s, rows, taps):
    v = s["bias"]
    for k, tap in enumerate(taps):
        v = v + s["weight"][:, k] * rows[tap]
    return v


def _conv(s):
    io = s["x"].dtype
    rows, taps, _, _, last = _window(s)
    v = _conv_sum(s, rows, taps)
    y = (v / (1 + torch.exp(-v))).to(io).view(s["x"].shape)
    y = tuple(t.contiguous() for t in y.split(s["split"], -1)) if s["split"] else y
    return y, rows[last].to(io)


def _conv_step(s):
    io = s["x"].dtype
    rows = torch.cat([s["state"], s["x"]], 1)
    v = (rows.float() * s["weight"].t()).sum(1) + s["bias"]
    y = (v / (1 + torch.exp(-v))).to(io)
    y = tuple(t.contiguous() for t in y.split(s["split"], -1)) if s["split"] else y
    return y, rows[:, 1:].contiguous()


def _conv_backward(s):
    io = s["x"].dtype
    rows, taps, mine, before, last = _window(s)
    v = _conv_sum(s, rows, taps)
    sig = 1 / (1 + torch.exp(-v))
    dy = torch.cat([d.float() for d in s["dy"]], -1).view(v.shape)
    dv = dy * sig * (1 + v * (1 - sig))
    over = tuple(range(v.dim() - 1))
    drows, dw = torch.zeros_like(rows), []
    for k, tap in enumerate(taps):
        drows[tap] += s["weight"][:, k] * dv
        dw.append((rows[tap] * dv).sum(over))
    if s["dfinal"] is not None:
        drows[last] += s["dfinal"]
    return dict(dx=drows[mine].to(io).view(s["x"].shape), dweight=torch.stack(dw, 1),
                dbias=dv.sum(over), dinitial_state=drows[before].contiguous())


def _scan_rows(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; `longest`: of any sequence."""
    far = 1
    while far < longest:
        b = torch.cat([b[:far], torch.addcmul(b[far:], a[far:], b[:-far])])
        a = torch.cat([a[:far], a[far:] * a[:-far]])
        far *= 2
    return b


def _spread(t, C):
    """[rows, G, N] to [rows, C, N]: each group's values for its channels."""
    return t.repeat_interleave(C // t.shape[1], 1)


def _scan_parts(s):
    c = s["case"]
    C, N, G, L = c["channels"], c["dstate"], c["groups"], c["seqlen"]
    f = {k: s[k].float().reshape(-1, C) for k in ("x", "dt")}
    f["B"], f["C"] = (s[k].float().reshape(-1, G, N) for k in ("B", "C"))
    f["z"] = None if s["z"] is None else s["z"].float().reshape(-1, C)
    f["raw"] = f["dt"] + s["dt_bias"]
    f["dl"] = torch.where(f["raw"] > 20, f["raw"], torch.log1p(torch.exp(f["raw"])))
    f["at"], f["seq"] = _rows(s, L, f["x"].device)
    R = f["x"].shape[0]
    f["rows"] = torch.arange(R, device=f["x"].device)
    f["begin"] = f["rows"] == f["at"][f["seq"]]
    f["a"] = torch.exp(f["dl"][..., None] * s["A"])
    b = (f["dl"] * f["x"])[..., None] * _spread(f["B"], C)
    h0 = s["state"]
    f["h0"] = torch.zeros(c["nseq"], C, N, device=b.device) if h0 is None else h0
    first = (f["begin"].float()[:, None, None])
    if h0 is not None:
        b = b + first * f["a"] * h0[f["seq"]]
    f["h"] = _scan_rows(f["a"] * (1 - first), b, L)
    f["y"] = (f["h"] * _spread(f["C"], C)).sum(-1) + s["D"] * f["x"]
    return f


def _ends(f):
    """(last row of each sequence, whether it has any)."""
    return (f["at"][1:] - 1).clamp(min=0), (f["at"][1:] > f["at"][:-1])[:, None, None]


def _scan(s):
    f = _scan_parts(s)
    y = f["y"] if f["z"] is None else f["y"] * f["z"] / (1 + torch.exp(-f["z"]))
    last, some = _ends(f)
    return y.to(s["x"].dtype).view(s["x"].shape), torch.where(some, f["h"][last], f["h0"])


def _scan_step(s):
    c = s["case"]
    x, dt, B, C = (s[k].squeeze(1).float() for k in ("x", "dt", "B", "C"))
    raw = dt + s["dt_bias"]
    dl = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw)))
    B, C = (_spread(m, c["channels"]) for m in (B, C))
    h = torch.exp(dl[..., None] * s["A"]) * s["state"] + (dl * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].squeeze(1).float()
        y = y * z / (1 + torch.exp(-z))
    return y.to(s["x"].dtype), h


def _scan_backward(s):
    c, io, f = s["case"], s["x"].dtype, _scan_parts(s)
    C, N, G, L = c["channels"], c["dstate"], c["groups"], c["seqlen"]
    e = dy = s["dy"].float().view(-1, C)
    dz = None
    if f["z"] is not None:
        sig = 1 / (1 + torch.exp(-f["z"]))
        e = dy * f["z"] * sig
        dz = (dy * f["y"] * sig * (1 + f["z"] * (1 - sig))).to(io).view(s["x"].shape)
    last, some = _ends(f)
    end = f["rows"] == last[f["seq"]]
    g = e[..., None] * _spread(f["C"], C)
    if s["dfinal"] is not None:
        g = g + end.float()[:, None, None] * s["dfinal"][f["seq"]]
    later = torch.cat([f["a"][1:], f["a"][:1]]) * (1 - end.float())[:, None, None]
    g = _scan_rows(later.flip(0), g.flip(0), L).flip(0)
    before = torch.cat([f["h"][:1], f["h"][:-1]])
    if s["state"] is None:
        before = before * (1 - f["begin"].float())[:, None, None]
    else:
        before = torch.where(f["begin"][:, None, None], f["h0"][f["seq"]], before)
    r = g * f["a"] * before
    q = (g * _spread(f["B"], C)).sum(-1)
    ddl = f["x"] * q + (r * s["A"]).sum(-1)
    ddt = ddl * torch.where(f["raw"] > 20, 1.0, 1 / (1 + torch.exp(-f["raw"])))
    over = lambda t: t.view(-1, G, C // G, N).sum(2).to(io).view(s["B"].shape)  # noqa: E731
    first = f["at"][:-1].clamp(max=f["rows"].numel() - 1)
    none = torch.zeros_like(f["h0"]) if s["dfinal"] is None else s["dfinal"]
    return dict(dx=(s["D"] * e + f["dl"] * q).to(io).view(s["x"].shape),
                ddt=ddt.to(io).view(s["x"].shape), dA=(r * f["dl"][..., None]).sum(0),
                dB=over(g * (f["dl"] * f["x"])[..., None]), dC=over(f["h"] * e[..., None]),
                dD=(e * f["x"]).sum(0), dz=dz, ddt_bias=ddt.sum(0),
                dinitial_state=torch.where(some, f["a"][first] * g[first], none))


def _gated_parts(s):
    c = s["case"]
    G, C = c["groups"], c["channels"]
    x, z = (s[k].float().reshape(-1, G, C // G) for k in ("x", "z"))
    sig = 1 / (1 + torch.exp(-z))
    v = x if c["first"] else x * z * sig
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return x, z, sig, v * r, r, s["weight"].view(G, C // G)


def _gated(s):
    _, z, sig, n, _, w = _gated_parts(s)
    y = n * w * z * sig if s["case"]["first"] else n * w
    return y.to(s["x"].dtype).view(s["x"].shape)


def _gated_backward(s):
    x, z, sig, n, r, w = _gated_parts(s)
    dy = s["dy"].float().view(x.shape)
    slope = sig * (1 + z * (1 - sig))
    if s["case"]["first"]:
        dn = dy * w * z * sig
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        dz, dw = dy * w * n * slope, dy * n * z * sig
    else:
        dn = dy * w
        dv = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        dx, dz, dw = dv * z * sig, dv * x * slope, dy * n
    io, shape = s["x"].dtype, s["x"].shape
    return dict(dx=dx.to(io).view(shape), dz=dz.to(io).view(shape), dweight=dw.sum(0).view(-1))


def _residual(s):
    x, r = s["x"].float(), s["residual"].float()
    r = r + (x if s["scale"] is None else s["scale"] * x)
    y = s["weight"] * r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    return y.to(s["x"].dtype), r.to(s["residual"].dtype)


def _residual_backward(s):
    """`residual` stands for the sum that the forward returned."""
    x, r, dy = s["x"].float(), s["residual"].float(), s["dy"].float()
    inv = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n, dn = r * inv, dy * s["weight"]
    dr = inv * (dn - n * (dn * n).mean(-1, keepdim=True)) + s["dres"].float()
    sums = tuple(range(x.dim() - 1))
    dx = dr if s["scale"] is None else s["scale"] * dr
    return dict(dx=dx.to(s["x"].dtype), dresidual=dr.to(s["residual"].dtype),
                dweight=(dy * n).sum(sums),
                dscale=None if s["scale"] is None else (dr * x).sum(sums))


PLAIN = dict(conv=_conv, conv_step=_conv_step, conv_backward=_conv_backward, scan=_scan,
             scan_step=_scan_step, scan_backward=_scan_backward, gated=_gated,
             gated_backward=_gated_backward, residual=_residual,
             residual_backward=_residual_backward)


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _silu(v):
    return v * torch.sigmoid(v)


def _sequences(s):
    """(sequences, batch rows, first token, last token + 1): a dense batch together, packed ones
    one by one."""
    c = s["case"]
    if s["starts"] is None:
        return [(slice(0, c["batch"]), slice(0, c["batch"]), 0, c["seqlen"])]
    at = s["starts"].tolist()
    return [(slice(i, i + 1), slice(0, 1), a, b) for i, (a, b) in enumerate(zip(at, at[1:]))]


def _conv64(s, x, weight, bias, state):
    y, final = [], []
    for seqs, rows, a, b in _sequences(s):
        u = torch.cat([state[seqs], x[rows, a:b]], 1)
        final.append(u[:, b - a:])
        if b > a:
            taps = u.unfold(1, weight.shape[1], 1)
            y.append(_silu((taps * weight).sum(-1) + bias))
    return torch.cat(y, 1), torch.cat(final)


def _scan64(s, x, dt, A, B, C, D, z, dt_bias, state):
    per = x.shape[-1] // B.shape[-2]
    y, final = [], []
    dl = torch.nn.functional.softplus(dt + dt_bias, threshold=700)
    for seqs, rows, a, b in _sequences(s):
        h = state[seqs]
        for t in range(a, b):
            d = dl[rows, t]
            Bt, Ct = (m[rows, t].repeat_interleave(per, 1) for m in (B, C))
            h = torch.exp(d[..., None] * A) * h + (d * x[rows, t])[..., None] * Bt
            y.append((h * Ct).sum(-1))
        final.append(h)
    y = torch.stack(y, 1) + D * x
    return y if z is None else y * _silu(z), torch.cat(final)


def _rms64(v, groups):
    g = v.unflatten(-1, (groups, -1))
    return (g / torch.sqrt((g * g).mean(-1, keepdim=True) + EPS)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c, op, back = case, s["op"], s["op"].endswith("backward")
    one = op.endswith("_step")
    d = {k: v.double().requires_grad_(back) for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    d.setdefault("z", None)
    S, C = c.get("nseq"), c["channels"]
    if op.startswith("conv"):
        zero = torch.zeros(S, c["width"] - 1, C, dtype=torch.float64, device="cuda")
        state = d["state"] if "state" in d else zero.requires_grad_(back)
        y, final = _conv64(s, d["x"], d["weight"], d["bias"], state)
        if not back:
            parts = [t.squeeze(1) if one else t for t in (y.split(s["split"], -1) if s["split"]
                                                          else (y,))]
            return (tuple(parts) if s["split"] else parts[0]), final
        loss = (y * torch.cat([t.double() for t in s["dy"]], -1)).sum()
        loss = loss if s["dfinal"] is None else loss + (final * d["dfinal"]).sum()
        names = ("dx", "dweight", "dbias", "dinitial_state")
        of = (d["x"], d["weight"], d["bias"], state)
    elif op.startswith("scan"):
        zero = torch.zeros(S, C, c["dstate"], dtype=torch.float64, device="cuda")
        state = d["state"] if "state" in d else zero.requires_grad_(back)
        y, final = _scan64(s, *(d[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")),
                           state)
        if not back:
            return (y.squeeze(1) if one else y), final
        loss = (y * d["dy"]).sum()
        loss = loss if s["dfinal"] is None else loss + (final * d["dfinal"]).sum()
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dinitial_state")
        of = [d[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")] + [state]
        if d["z"] is not None:
            names, of = names + ("dz",), of + [d["z"]]
    elif op.startswith("gated"):
        if c["first"]:
            y = _rms64(d["x"], c["groups"]) * d["weight"] * _silu(d["z"])
        else:
            y = _rms64(d["x"] * _silu(d["z"]), c["groups"]) * d["weight"]
        if not back:
            return y
        loss, names = (y * d["dy"]).sum(), ("dx", "dz", "dweight")
        of = (d["x"], d["z"], d["weight"])
    elif not back:
        r = d["residual"] + (d["scale"] if c["scale"] else 1) * d["x"]
        return _rms64(r, 1) * d["weight"], r
    else:
        r = d["residual"]
        y = _rms64(r, 1) * d["weight"]
        dr, dw = torch.autograd.grad((y * d["dy"]).sum() + (r * d["dres"]).sum(),
                                     (r, d["weight"]))
        scale = d["scale"].detach() if c["scale"] else 1
        over = (dr * d["x"].detach()).sum((0, 1))
        return dict(dx=scale * dr, dresidual=dr, dweight=dw, dscale=over if c["scale"] else None)
    got = torch.autograd.grad(loss, of, allow_unused=True)
    return dict(zip(names, (torch.zeros_like(o) if g is None else g for g, o in zip(got, of))))
