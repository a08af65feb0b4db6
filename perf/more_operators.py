"""The operators of layers of linear recurrence beside the scan, as cases to time and compare.

Three operators: the gated linear recurrence, one state entry a channel (forward, single token,
backward); the rotation of B and C by positions of several axes, which gives the scan's decays a
phase (forward, for one token too, and backward); the group norm with its activation, over each
sequence's tokens and a group's channels (forward, backward; sequences of one token: over a
token's heads). Where ``own`` is false, ``run`` computes them in plain torch operations in 32 bits
(angles in 64); where it is true, it calls this package.
"""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token for each sequence of a serving batch, in a small layer: latency counts
        dict(name="recurrence_decode", op="recurrence_step", io=BF16, batch=64, seqlen=1, nseq=64,
             channels=2560, decay=True, gated=True, pad=2560),
        # prompts of unequal length packed into one row of tokens, continued from their states
        dict(name="recurrence_prompts", op="recurrence", io=BF16, batch=1, seqlen=5003, nseq=7,
             packed=True, channels=1536, decay=True, gated=True, pad=1536, initial=True),
        # long prompts in a large layer, both gates read from one projection's rows
        dict(name="recurrence_long", op="recurrence", io=BF16, batch=2, seqlen=8192, nseq=2,
             channels=5120, decay=True, gated=True, pad=5120, initial=False),
        # a training step of the large layer
        dict(name="recurrence_train", op="recurrence_backward", io=BF16, batch=2, seqlen=4096,
             nseq=2, channels=5120, decay=True, gated=True, pad=5120, initial=False),
        # training of a small layer in 32 bits, the gate itself the decay
        dict(name="recurrence_train_f32", op="recurrence_backward", io=F32, batch=4, seqlen=2048,
             nseq=4, channels=768, decay=False, gated=False, pad=0, initial=True),
        # B and C of one token for each sequence of a serving batch, far into their texts
        dict(name="rotate_decode", op="rotate", io=BF16, batch=64, seqlen=0, groups=1, dstate=128,
             nfreq=64, axes=1, far=1000000, interleaved=False, pad=5120, inverse=False),
        # B and C of the wide grouped layer over a video, by time, height and width
        dict(name="rotate_video", op="rotate", io=BF16, batch=2, seqlen=16384, groups=8,
             dstate=256, nfreq=128, axes=3, far=20000, interleaved=False, pad=0, inverse=False),
        # their gradients in a small layer, in 32 bits as the scan's backward gives them
        dict(name="rotate_train", op="rotate", io=F32, batch=4, seqlen=2048, groups=1, dstate=128,
             nfreq=64, axes=2, far=2000, interleaved=True, pad=0, inverse=True),
        # packed clips of unequal length behind a small convolution, in 32 bits
        dict(name="group_norm_clips", op="group_norm", io=F32, batch=1, seqlen=3001, nseq=5,
             packed=True, channels=768, groups=32, silu=True, pad=0, stats=False),
        # every head of every token behind the scan of a large layer, to be trained on
        dict(name="group_norm_heads", op="group_norm", io=BF16, batch=16384, seqlen=1, nseq=16384,
             channels=5120, groups=80, silu=False, pad=0, stats=True),
        # long sequences behind a convolution, statistics over a sequence's tokens
        dict(name="group_norm_long", op="group_norm", io=BF16, batch=2, seqlen=8192, nseq=2,
             channels=2560, groups=32, silu=True, pad=0, stats=False),
        # the same, a training step's gradients
        dict(name="group_norm_train", op="group_norm_backward", io=BF16, batch=2, seqlen=8192,
             nseq=2, channels=2560, groups=32, silu=True, pad=0),
    ]


def _between(rng, low, high, step=1):
    """A whole multiple of `step` between the two, spread over the logarithm."""
    return max(low, step * round(math.exp(rng.uniform(math.log(low), math.log(high))) / step))


def draw(rng):
    op = rng.choice(["recurrence", "recurrence", "recurrence_step", "recurrence_backward",
                     "recurrence_backward", "rotate", "rotate", "group_norm", "group_norm",
                     "group_norm_backward", "group_norm_backward"])
    c = dict(op=op, io=rng.choice([BF16, BF16, F32]), pad=rng.choice([0, 64, 520]))
    if op == "rotate":
        c.update(batch=_between(rng, 1, 8), groups=rng.choice([1, 1, 2, 4, 8]),
                 dstate=16 * _between(rng, 1, 16), interleaved=rng.random() < 0.5,
                 axes=rng.choice([1, 2, 3]), far=_between(rng, 100, 1000000),
                 inverse=rng.random() < 0.4)
        c["seqlen"] = rng.choice([0, _between(rng, 1, 6000), _between(rng, 1, 6000)])
        if not c["seqlen"]:
            c["batch"] = _between(rng, 1, 128)
        c["nfreq"] = c["dstate"] // rng.choice([2, 2, 4])
        return c
    if op == "recurrence_step":
        c.update(batch=_between(rng, 1, 128), seqlen=1)
        c["nseq"] = c["batch"]
    elif op.startswith("group_norm") and rng.random() < 0.35:  # the heads of single tokens
        c.update(batch=_between(rng, 1, 6000), seqlen=1)
        c["nseq"] = c["batch"]
    else:
        rows = _between(rng, 1, 6000)
        if rng.random() < 0.5:
            c.update(batch=1, seqlen=rows, nseq=_between(rng, 1, 24), packed=True)
        else:
            batch = min(rows, _between(rng, 1, 8))
            c.update(batch=batch, seqlen=max(1, rows // batch), nseq=batch)
    if op.startswith("recurrence"):
        c.update(channels=_between(rng, 64, 6000, 8), decay=rng.random() < 0.6,
                 gated=rng.random() < 0.6, initial=rng.random() < 0.5)
    else:
        c.update(groups=rng.choice([1, 4, 8, 16, 32]), silu=rng.random() < 0.6)
        c["channels"] = c["groups"] * _between(rng, 8, 5000 // c["groups"], 8)
        if op == "group_norm":
            c["stats"] = rng.random() < 0.5
    return c


# ---- inputs --------------------------------------------------------------------------------------

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _slice(g, pad, width, dtype, *lead):
    """[*lead, width] values that stand behind `pad` others in each row."""
    return _normal(g, *lead, pad + width, dtype=dtype)[..., pad:]


def _offsets(g, c):
    """Where each of nseq packed sequences starts, and the end: random cuts, some may be empty."""
    cuts = torch.randint(0, c["seqlen"] + 1, (c["nseq"] - 1,), generator=g, device="cuda")
    ends = torch.tensor([0, c["seqlen"]], device="cuda")
    return torch.cat([ends, cuts]).sort().values.to(torch.int32)


def _sections(c):
    """Frequencies of each axis: a quarter for time, what is left shared by the others."""
    n, axes = c["nfreq"], c["axes"]
    if axes == 1:
        return (n,)
    first = n // 4 if axes == 3 else n // 2
    return (first, n - first) if axes == 2 else (first, (n - first) // 2,
                                                 n - first - (n - first) // 2)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    io, op, pad = TYPES[c["io"]], c["op"], c["pad"]
    s = dict(case=c, op=op)
    if op == "rotate":
        lead = (c["batch"], c["seqlen"]) if c["seqlen"] else (c["batch"],)
        G, N = c["groups"], c["dstate"]
        # B and C stand side by side in the rows of one projection
        bc = _slice(g, pad, 2 * G * N, io, *lead)
        s["B"], s["C"] = (t.unflatten(-1, (G, N)) for t in bc.split(G * N, -1))
        if c["inverse"]:  # gradients come dense from the scan's backward
            s["B"], s["C"] = s["B"].contiguous(), s["C"].contiguous()
        s["positions"] = torch.randint(0, c["far"], (c["axes"], *lead), generator=g,
                                       device="cuda").to(torch.int32)
        j = torch.arange(c["nfreq"], device="cuda", dtype=torch.float64) / c["nfreq"]
        s["frequencies"] = (10000.0 ** -j).float()
        s["sections"] = _sections(c)
        return s
    B, L, C, S = c["batch"], c["seqlen"], c["channels"], c["nseq"]
    s["starts"] = _offsets(g, c) if c.get("packed") else None
    if op.startswith("recurrence"):
        s["x"] = _normal(g, B, L, C, dtype=io)
        # the gates stand side by side in the rows of one projection
        both = _slice(g, pad, 2 * C if c["gated"] else C, io, B, L)
        s["gate"], s["input_gate"] = both.split(C, -1) if c["gated"] else (both, None)
        s["decay"] = None
        if c["decay"]:  # forgets between 0.001 and 0.1 of the state where the gate is open
            rate = -torch.log(0.9 + 0.099 * _uniform(g, C)) / 8
            s["decay"] = torch.log(torch.expm1(rate))
        given = op == "recurrence_step" or c["initial"]
        s["state"] = _normal(g, S, C) if given else None
        if op == "recurrence_backward":
            s["dy"] = _normal(g, B, L, C, dtype=io)
            s["dfinal"] = _normal(g, S, C) if c["initial"] else None
        return s
    s["x"] = _slice(g, pad, C, io, B, L)
    s["weight"] = _normal(g, C, scale=0.1) + 1
    s["bias"] = _normal(g, C, scale=0.1)
    if op == "group_norm_backward":
        s["dy"] = _normal(g, B, L, C, dtype=io)
        s["stats"] = _stats(s)
    return s


EPS = 1e-5
SHARPNESS = 8.0


# ---- what each pass cannot do without ------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    e = 2 if c["io"] == BF16 else 4
    if op == "rotate":
        rows = c["batch"] * max(1, c["seqlen"])
        el = 2 * rows * c["groups"] * c["dstate"]
        return dict(bytes=2 * el * e + rows * c["axes"] * 4 + c["nfreq"] * 4, flops=el * 3)
    rows, C, S = c["batch"] * c["seqlen"], c["channels"], c["nseq"]
    el = rows * C
    if op.startswith("recurrence"):
        ins, params = 3 if c["gated"] else 2, 4 * C if c["decay"] else 0
        if op == "recurrence_backward":
            states = 4 * S * C * (3 if c["initial"] else 1)
            return dict(bytes=el * e * (2 * ins + 1) + 2 * params + states, flops=el * 40)
        given = op == "recurrence_step" or c["initial"]
        return dict(bytes=el * e * (ins + 1) + params + 4 * S * C * (2 if given else 1),
                    flops=el * 15)
    if op == "group_norm_backward":
        return dict(bytes=el * e * 3 + 16 * C + 8 * S * c["groups"], flops=el * 25)
    return dict(bytes=el * e * 2 + 8 * C + (8 * S * c["groups"] if c["stats"] else 0),
                flops=el * 10)


# ---- the framework's calls -----------------------------------------------------------------------

def _own(s):
    import mamba_ssd_chunked_cumsum_amd as ssd

    c, op = s["case"], s["op"]
    if op == "recurrence":
        return ssd.recurrence(s["x"], s["gate"], s["decay"], s["input_gate"], s["state"],
                              sharpness=SHARPNESS, cu_seqlens=s["starts"])
    if op == "recurrence_step":
        one = (None if s[k] is None else s[k].squeeze(1) for k in ("x", "gate", "input_gate"))
        x, gate, input_gate = one
        return ssd.recurrence_step(s["state"], x, gate, s["decay"], input_gate,
                                   sharpness=SHARPNESS)
    if op == "recurrence_backward":
        return ssd.recurrence_backward(s["x"], s["gate"], s["decay"], s["input_gate"], s["dy"],
                                       s["state"], s["dfinal"], sharpness=SHARPNESS,
                                       cu_seqlens=s["starts"])
    if op == "rotate":
        call = ssd.rotate_backward if c["inverse"] else ssd.rotate
        return call(s["B"], s["C"], s["positions"], s["frequencies"], sections=s["sections"],
                    interleaved=c["interleaved"])
    act = "silu" if c["silu"] else None
    if op == "group_norm":
        return ssd.group_norm(s["x"], s["weight"], s["bias"], ngroups=c["groups"], eps=EPS,
                              activation=act, cu_seqlens=s["starts"], want_stats=c["stats"])
    return ssd.group_norm_backward(s["x"], s["weight"], s["bias"], s["stats"], s["dy"],
                                   ngroups=c["groups"], activation=act, cu_seqlens=s["starts"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- plain forms ---------------------------------------------------------------------------------

def _rows(s):
    """(offsets [nseq + 1], the sequence of each row) of flattened rows; every row is in one."""
    c, device = s["case"], s["x"].device
    if s["starts"] is not None:
        at = s["starts"].long()
    else:
        at = torch.arange(c["batch"] + 1, device=device) * c["seqlen"]
    rows = torch.arange(c["batch"] * c["seqlen"], device=device)
    return at, torch.searchsorted(at[1:], rows, right=True)


def _scan_rows(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; `longest`: of any sequence."""
    far = 1
    while far < longest:
        b = torch.cat([b[:far], torch.addcmul(b[far:], a[far:], b[:-far])])
        a = torch.cat([a[:far], a[far:] * a[:-far]])
        far *= 2
    return b


def _sigmoid(v):
    """(sigmoid(v), sigmoid(-v)), each exact where it is small too."""
    e = torch.exp(-v.abs())
    big, small = 1 / (1 + e), e / (1 + e)
    return torch.where(v >= 0, big, small), torch.where(v >= 0, small, big)


def _decays(s, gate):
    """a, m (what the input is multiplied by), and with a decay u = -log a and 1 - r."""
    r, other = _sigmoid(gate)
    if s["decay"] is None:
        return r, other, None, None
    u = r * SHARPNESS * torch.log1p(torch.exp(s["decay"]))
    return torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)), u, other


def _recurrence_parts(s):
    c = s["case"]
    C = c["channels"]
    f = dict(x=s["x"].float().reshape(-1, C))
    f["a"], f["m"], f["u"], f["other"] = _decays(s, s["gate"].float().reshape(-1, C))
    f["v"] = f["x"]
    if s["input_gate"] is not None:
        f["si"], f["no"] = _sigmoid(s["input_gate"].float().reshape(-1, C))
        f["v"] = f["si"] * f["x"]
    f["at"], f["seq"] = _rows(s)
    f["rows"] = torch.arange(f["x"].shape[0], device=f["x"].device)
    f["first"] = (f["rows"] == f["at"][f["seq"]])[:, None].float()
    h0 = s["state"]
    f["h0"] = torch.zeros(c["nseq"], C, device=f["x"].device) if h0 is None else h0
    b = f["m"] * f["v"] + f["first"] * f["a"] * f["h0"][f["seq"]]
    f["h"] = _scan_rows(f["a"] * (1 - f["first"]), b, c["seqlen"])
    f["last"] = (f["at"][1:] - 1).clamp(min=0)
    f["some"] = (f["at"][1:] > f["at"][:-1])[:, None]
    return f


def _recurrence(s):
    f = _recurrence_parts(s)
    return (f["h"].to(s["x"].dtype).view(s["x"].shape),
            torch.where(f["some"], f["h"][f["last"]], f["h0"]))


def _recurrence_step(s):
    x, gate = s["x"].squeeze(1).float(), s["gate"].squeeze(1).float()
    a, m, _, _ = _decays(s, gate)
    v = x if s["input_gate"] is None else _sigmoid(s["input_gate"].squeeze(1).float())[0] * x
    h = a * s["state"] + m * v
    return h.to(s["x"].dtype), h


def _recurrence_backward(s):
    c, io, shape, f = s["case"], s["x"].dtype, s["x"].shape, _recurrence_parts(s)
    g = s["dy"].float().view(-1, c["channels"])
    end = (f["rows"] == f["last"][f["seq"]])[:, None].float()
    if s["dfinal"] is not None:
        g = g + end * s["dfinal"][f["seq"]]
    later = torch.cat([f["a"][1:], f["a"][:1]]) * (1 - end)
    g = _scan_rows(later.flip(0), g.flip(0), c["seqlen"]).flip(0)
    before = torch.where(f["first"] > 0, f["h0"][f["seq"]], torch.cat([f["h"][:1], f["h"][:-1]]))
    if s["decay"] is None:
        dgate, ddecay = g * (before - f["v"]) * f["a"] * f["m"], None
    else:
        q = g * (f["a"] * before - f["a"] * f["a"] / f["m"] * f["v"]) * -f["u"]
        dgate = q * f["other"]
        lam = s["decay"]  # u is proportional to softplus(decay)
        ddecay = q.sum(0) / (1 + torch.exp(-lam)) / torch.log1p(torch.exp(lam))
    dv = g * f["m"]
    dx, dinput = dv, None
    if s["input_gate"] is not None:
        dx = dv * f["si"]
        dinput = (dv * f["v"] * f["no"]).to(io).view(shape)
    first = f["at"][:-1].clamp(max=f["rows"].numel() - 1)
    none = torch.zeros_like(f["h0"]) if s["dfinal"] is None else s["dfinal"]
    return dict(dx=dx.to(io).view(shape), dgate=dgate.to(io).view(shape), ddecay=ddecay,
                dinput_gate=dinput,
                dinitial_state=torch.where(f["some"], f["a"][first] * g[first], none))


def _axis(s, device):
    """The axis of each frequency."""
    ends = torch.tensor(s["sections"], device=device).cumsum(0)
    return torch.searchsorted(ends, torch.arange(s["case"]["nfreq"], device=device), right=True)


def _angles(s):
    """[*lead, 1, nfreq], in 64 bits."""
    pos = s["positions"].double()[_axis(s, s["positions"].device)]
    angle = pos.movedim(0, -1) * s["frequencies"].double()
    return (-angle if s["case"]["inverse"] else angle).unsqueeze(-2)


def _turn(t, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        p, q = t[..., 0:2 * n:2], t[..., 1:2 * n:2]
        turned = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
    else:
        p, q = t[..., :n], t[..., n:2 * n]
        turned = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
    return torch.cat([turned, t[..., 2 * n:]], -1)


def _rotate(s):
    angle = _angles(s)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return tuple(_turn(t.float(), cos, sin, s["case"]["interleaved"]).to(t.dtype)
                 for t in (s["B"], s["C"]))


def _by_group(s):
    """x as [sequences or rows, tokens, groups, channels], and a sum over each sequence and
    group, [.., 1, groups, 1], given back to its tokens."""
    c = s["case"]
    G, C, L = c["groups"], c["channels"], c["seqlen"]
    if s["starts"] is None:
        x = s["x"].float().view(c["batch"], L, G, C // G)
        return x, L * (C // G), lambda t: t.sum((1, 3), keepdim=True), lambda t: t[:, 0, :, 0]
    at, seq = _rows(s)
    x = s["x"].float().view(L, 1, G, C // G)
    count = ((at[1:] - at[:-1])[seq] * (C // G))[:, None, None, None]

    def total(t):  # in 64 bits: differences of sums over all rows
        run = t.sum(3).double().cumsum(0).squeeze(1)
        run = torch.cat([torch.zeros_like(run[:1]), run])
        return (run[at[1:]] - run[at[:-1]])[seq].float().view(L, 1, G, 1)

    return x, count, total, lambda t: t[at[:-1].clamp(max=L - 1), 0, :, 0]


def _moments(s):
    x, count, total, _ = _by_group(s)
    mean = total(x) / count
    d = x - mean
    return d, mean, torch.rsqrt(total(d * d) / count + EPS)


def _stats(s):
    """[nseq, groups, 2]: mean and 1 / sqrt(variance + eps) of each; (0, 1 / sqrt(eps)) of a
    sequence without tokens."""
    _, mean, rstd = _moments(s)
    each = _by_group(s)[3]
    stats = torch.stack([each(mean.expand_as(rstd)), each(rstd)], -1)
    if s["starts"] is None:
        return stats
    some = (s["starts"][1:] > s["starts"][:-1])[:, None, None]
    return torch.where(some, stats, torch.tensor([0.0, EPS ** -0.5], device=stats.device))


def _group_norm(s):
    c = s["case"]
    d, _, rstd = _moments(s)
    w, b = (s[k].view(c["groups"], -1) for k in ("weight", "bias"))
    y = d * rstd * w + b
    y = y / (1 + torch.exp(-y)) if c["silu"] else y
    return y.to(s["x"].dtype).view(s["x"].shape), _stats(s) if c["stats"] else None


def _group_norm_backward(s):
    c, io = s["case"], s["x"].dtype
    x, count, total, _ = _by_group(s)
    st = s["stats"] if s["starts"] is None else s["stats"][_rows(s)[1]]
    mean, rstd = st[:, None, :, 0, None], st[:, None, :, 1, None]
    w, b = (s[k].view(c["groups"], -1) for k in ("weight", "bias"))
    n = (x - mean) * rstd
    dv = s["dy"].float().view(x.shape)
    if c["silu"]:
        v = n * w + b
        sig = 1 / (1 + torch.exp(-v))
        dv = dv * sig * (1 + v * (1 - sig))
    g = dv * w
    dx = rstd * (g - total(g) / count - n * (total(g * n) / count))
    return dict(dx=dx.to(io).view(s["x"].shape), dweight=(dv * n).sum((0, 1)).view(-1),
                dbias=dv.sum((0, 1)).view(-1))


PLAIN = dict(recurrence=_recurrence, recurrence_step=_recurrence_step,
             recurrence_backward=_recurrence_backward, rotate=_rotate, group_norm=_group_norm,
             group_norm_backward=_group_norm_backward)


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _sequences(s):
    """(sequences, batch rows, first token, last token + 1): a dense batch together, packed ones
    one by one."""
    c = s["case"]
    if s["starts"] is None:
        return [(slice(0, c["batch"]), slice(0, c["batch"]), 0, c["seqlen"])]
    at = s["starts"].tolist()
    return [(slice(i, i + 1), slice(0, 1), a, b) for i, (a, b) in enumerate(zip(at, at[1:]))]


def _recurrence64(s, x, gate, decay, input_gate, state):
    if decay is None:
        a = torch.sigmoid(gate)
        m = torch.sigmoid(-gate)
    else:
        log_a = -SHARPNESS * torch.nn.functional.softplus(decay) * torch.sigmoid(gate)
        a, m = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    b = m * (x if input_gate is None else torch.sigmoid(input_gate) * x)
    y, final = [], []
    for seqs, rows, begin, end in _sequences(s):
        h = state[seqs]
        for at, bt in zip(a[rows, begin:end].unbind(1), b[rows, begin:end].unbind(1)):
            h = at * h + bt
            y.append(h)
        final.append(h)
    return torch.stack(y, 1), torch.cat(final)


def _norm64(s, x, weight, bias):
    c = s["case"]
    y, stats = [], []
    for _, rows, begin, end in _sequences(s):
        t = x[rows, begin:end].unflatten(-1, (c["groups"], -1))
        if end == begin:
            stats.append(t.new_tensor([0.0, EPS ** -0.5]).expand(1, c["groups"], 2))
            continue
        mean = t.mean((1, 3), keepdim=True)
        rstd = (((t - mean) ** 2).mean((1, 3), keepdim=True) + EPS) ** -0.5
        y.append(((t - mean) * rstd).flatten(-2))
        stats.append(torch.stack([mean[:, 0, :, 0], rstd[:, 0, :, 0]], -1))
    y = torch.cat(y, 1) * weight + bias
    return y * torch.sigmoid(y) if c["silu"] else y, torch.cat(stats)


def exact(case, seed):
    s = prepare(case, seed)
    c, op, back = case, s["op"], s["op"].endswith("backward")
    if op == "rotate":
        out = []
        unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), _angles(s))
        n = c["nfreq"]
        for t in (s["B"].double(), s["C"].double()):
            if c["interleaved"]:
                z = torch.view_as_complex(t[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * unit
                turned = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(t[..., :n], t[..., n:2 * n]) * unit
                turned = torch.cat([z.real, z.imag], -1)
            out.append(torch.cat([turned, t[..., 2 * n:]], -1))
        return tuple(out)
    d = {k: v.double().requires_grad_(back) for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op.startswith("recurrence"):
        zero = torch.zeros(c["nseq"], c["channels"], dtype=torch.float64, device="cuda")
        state = d["state"] if "state" in d else zero.requires_grad_(back)
        y, final = _recurrence64(s, d["x"], d["gate"], d.get("decay"), d.get("input_gate"), state)
        if not back:
            return (y.squeeze(1) if op == "recurrence_step" else y), final
        loss = (y * d["dy"].detach()).sum()
        loss = loss if s["dfinal"] is None else loss + (final * d["dfinal"].detach()).sum()
        of = dict(dx=d["x"], dgate=d["gate"], ddecay=d.get("decay"),
                  dinput_gate=d.get("input_gate"), dinitial_state=state)
    else:
        y, stats = _norm64(s, d["x"], d["weight"], d["bias"])
        if not back:
            return y, stats if c["stats"] else None
        loss = (y * d["dy"].detach()).sum()
        of = dict(dx=d["x"], dweight=d["weight"], dbias=d["bias"])
    given = {k: v for k, v in of.items() if v is not None}
    got = dict(zip(given, torch.autograd.grad(loss, list(given.values()), allow_unused=True)))
    return {k: torch.zeros_like(given[k]) if k in given and got[k] is None else got.get(k)
            for k in of}
