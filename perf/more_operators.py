"""Measured cases of the operators of a selective state space layer: its short
causal convolution, its scan, and the norms after one block and before the
next fused with the gate, the residual scale and the residual sum.

Every case runs in two forms on the same inputs.  The plain form (``own`` is
false) is elementary torch arithmetic in 32 bits, rounded once at the end.
The other one calls this package's operators.  ``exact`` gives the same
outputs from the definitions in 64 bits.

Causal convolution over the tokens of b x l x d, K taps, x before the first
token from s0 (b x (K - 1) x d):
    y_t = act(bias + sum_j w_j x_(t - K + 1 + j)),  s1 = the last K - 1 inputs

Selective scan, per sequence and channel, with a state h of n values:
    dt_t = softplus(delta_t + delta_bias),  h_t = exp(dt_t A) h_(t-1) + dt_t u_t B_t
    y_t = (C_t . h_t + D u_t) silu(z_t)
B and C are shared by the d / g channels of a group.

Residual norm over rows of c:
    p = y / rms(y) w_post,  r = x + scale act(gate) p,  h = r / rms(r) w_pre,
    rms(v) = sqrt(mean(v^2) + eps)
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # one token of one sequence: latency of an interactive answer
        {"name": "conv token single", "op": "conv", "mode": "step", "b": 1, "l": 1, "d": 2048,
         "k": 4, "x": "bf16", "ragged": False, "bias": True},
        # a batch of short prompts of unequal length that go on from earlier tokens, channels that
        # no wide load divides
        {"name": "conv prompts ragged", "op": "conv", "mode": "fwd", "b": 5, "l": 333, "d": 515,
         "k": 3, "x": "f16", "ragged": True, "bias": False},
        # a training step of full sequences
        {"name": "conv train", "op": "conv", "mode": "train", "b": 8, "l": 2048, "d": 2048, "k": 4,
         "x": "bf16", "ragged": False, "bias": True},
        # one token of one sequence
        {"name": "scan token single", "op": "scan", "mode": "step", "b": 1, "l": 1, "d": 2048,
         "n": 16, "g": 1, "x": "bf16", "ragged": False, "gate": True},
        # one token of each of 128 sequences: a serving batch, bound by the states
        {"name": "scan token batch", "op": "scan", "mode": "step", "b": 128, "l": 1, "d": 4096,
         "n": 16, "g": 1, "x": "bf16", "ragged": False, "gate": True},
        # a prompt of one sequence
        {"name": "scan prompt", "op": "scan", "mode": "fwd", "b": 1, "l": 4096, "d": 2048, "n": 16,
         "g": 1, "x": "bf16", "ragged": False, "gate": True},
        # a batch of short prompts of unequal length, sizes that are no tile's, two groups
        {"name": "scan prompts ragged", "op": "scan", "mode": "fwd", "b": 5, "l": 333, "d": 600,
         "n": 20, "g": 2, "x": "f16", "ragged": True, "gate": True},
        # a training step of full sequences
        {"name": "scan train", "op": "scan", "mode": "train", "b": 8, "l": 2048, "d": 2048,
         "n": 16, "g": 1, "x": "bf16", "ragged": False, "gate": True},
        # a training step in fp32 of unequal sequences with a larger state and no gate
        {"name": "scan train f32", "op": "scan", "mode": "train", "b": 2, "l": 700, "d": 320,
         "n": 32, "g": 1, "x": "f32", "ragged": True, "gate": False},
        # between two blocks, one token: latency
        {"name": "norm token", "op": "norm", "train": False, "rows": 1, "c": 1024, "x": "bf16",
         "y": "bf16", "act": None, "scale": True},
        # between two blocks, a training step with an fp32 residual stream
        {"name": "norm train", "op": "norm", "train": True, "rows": 16384, "c": 2048, "x": "f32",
         "y": "bf16", "act": None, "scale": True},
        # the same with a gate, rows of an odd length
        {"name": "norm train gated odd", "op": "norm", "train": True, "rows": 3333, "c": 771,
         "x": "f16", "y": "f16", "act": "silu", "scale": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    x = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        c = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            c = max(8, c // 8 * 8)
        rows = _log(rng, 1, max(1, min(100000, 30000000 // c)))
        y = rng.choice(["bf16", "f16", "f32"]) if x == "f32" else x
        return {"op": op, "train": rng.random() < 0.6, "rows": rows, "c": c, "x": x, "y": y,
                "act": rng.choice([None, "silu", "sigmoid"]), "scale": rng.random() < 0.6}
    mode = rng.choice(["step", "fwd", "train"])
    if op == "conv":
        d = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        n = 1 if mode == "step" else _log(rng, 2, 6000)
        b = max(1, min(_log(rng, 1, 64), 30000000 // (n * d)))
        return {"op": op, "mode": mode, "b": b, "l": n, "d": d, "k": rng.choice([2, 3, 4, 4, 5, 8]),
                "x": x, "ragged": mode != "step" and rng.random() < 0.4,
                "bias": rng.random() < 0.7}
    g, n = rng.choice([1, 1, 2, 3]), rng.choice([1, 4, 8, 16, 16, 16, 20, 32, 64])
    d = g * _log(rng, 16, 1365)
    if mode == "step":
        b, t = max(1, min(_log(rng, 1, 192), 8000000 // (d * n))), 1
    else:
        t = _log(rng, 2, 6000 if mode == "fwd" else 3000)
        b = max(1, min(_log(rng, 1, 32), 250000000 // (t * d * n)))
        t = min(t, max(1, 500000000 // (b * d * n)))
    return {"op": op, "mode": mode, "b": b, "l": t, "d": d, "n": n, "g": g, "x": x,
            "ragged": mode != "step" and rng.random() < 0.4, "gate": rng.random() < 0.7}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _inputs(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = dict(case)
    dt = DTYPES[case["x"]]
    if case["op"] == "norm":
        rows, c = case["rows"], case["c"]
        yt = DTYPES[case["y"]]
        s["in"] = (normal(rows, c) * 1.5).to(dt)
        s["block"] = (normal(rows, c) * 0.7).to(yt)
        s["gate"] = normal(rows, c).to(yt) if case["act"] else None
        s["s"] = 0.5 + 0.2 * normal(c) if case["scale"] else None
        s["w_post"], s["w_pre"] = 1 + 0.2 * normal(c), 1 + 0.2 * normal(c)
        if case["train"]:
            s["dr"], s["dh"] = (0.5 * normal(rows, c)).to(dt), normal(rows, c).to(yt)
        return s
    b, n, d = case["b"], case["l"], case["d"]
    s["lengths"] = None
    if case["ragged"]:
        lens = torch.randint(0, n + 1, (b,), generator=gen, device=dev, dtype=torch.int32)
        lens[0] = n
        s["lengths"] = lens
    if case["op"] == "conv":
        k = case["k"]
        # one half of the projection that makes the operand and its gate
        s["in"] = normal(b, n, 2 * d).to(dt)[..., :d]
        s["w"] = (normal(k, d) / math.sqrt(k)).to(dt)
        s["bias"] = (0.1 * normal(d)).to(dt) if case["bias"] else None
        s["s0"] = normal(b, k - 1, d).to(dt)
        if case["mode"] == "step":
            s["s1"] = torch.empty_like(s["s0"])
        if case["mode"] == "train":
            s["dy"], s["ds"] = normal(b, n, d).to(dt), normal(b, k - 1, d).to(dt)
        return s
    g, m = case["g"], case["n"]
    s["u"] = torch.nn.functional.silu(normal(b, n, d)).to(dt)
    s["delta"] = (0.5 * normal(b, n, d)).to(dt)
    # the other half of the projection
    s["z"] = normal(b, n, 2 * d).to(dt)[..., d:] if case["gate"] else None
    # B and C as one projection leaves them, behind the low-rank steps
    rank = max(1, d // 16)
    mixed = normal(b, n, rank + 2 * g * m).to(dt)
    s["B"] = mixed[..., rank:rank + g * m].unflatten(-1, (g, m))
    s["C"] = mixed[..., rank + g * m:].unflatten(-1, (g, m))
    s["A"] = -(torch.arange(1, m + 1, device=dev) * torch.exp(0.1 * normal(d, m)))
    s["D"] = 1 + 0.1 * normal(d)
    # steps between 0.001 and 0.1 where delta is 0
    step = torch.exp(torch.rand(d, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["s0"] = 0.3 * normal(b, d, m)
    if case["mode"] == "step":
        s["s1"] = torch.empty_like(s["s0"])
    if case["mode"] == "train":
        s["dy"], s["ds"] = normal(b, n, d).to(dt), 0.1 * normal(b, d, m)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def run(s):
    if s["op"] == "conv":
        return _conv_own(s) if own else _conv_plain(s)
    if s["op"] == "scan":
        return _scan_own(s) if own else _scan_plain(s)
    return _norm_own(s) if own else _norm_plain(s)


# ------------------------------------------------- this package's operators ----

def _conv_own(s):
    import depthwise_convolution_dwc_amd as dwc

    if s["mode"] == "step":
        return dwc.causal_conv_step(s["in"], s["w"], s["bias"], s["s0"], act="silu",
                                    out_state=s["s1"])
    kw = {"s0": s["s0"], "lengths": s["lengths"], "act": "silu"}
    y, s1 = dwc.causal_conv(s["in"], s["w"], s["bias"], **kw)
    if s["mode"] == "fwd":
        return y, s1
    return (y, s1) + dwc.causal_conv_bwd(s["dy"], s["ds"], s["in"], s["w"], s["bias"], **kw)


def _scan_own(s):
    import depthwise_convolution_dwc_amd as dwc

    a = (s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["s0"])
    if s["mode"] == "step":
        return dwc.selective_scan_step(*a, softplus=True, out_state=s["s1"])
    y, s1 = dwc.selective_scan(*a, lengths=s["lengths"], softplus=True)
    if s["mode"] == "fwd":
        return y, s1
    return (y, s1) + dwc.selective_scan_bwd(s["dy"], s["ds"], *a, lengths=s["lengths"],
                                            softplus=True)


def _norm_own(s):
    import depthwise_convolution_dwc_amd as dwc

    kw = {"gate": s["gate"], "scale": s["s"], "w_post": s["w_post"], "w_pre": s["w_pre"],
          "act": s["act"] or "none"}
    r, h, post, pre = dwc.residual_norm(s["in"], s["block"], eps=EPS, **kw)
    if not s["train"]:
        return r, h
    return (r, h) + dwc.residual_norm_bwd(s["dr"], s["dh"], s["in"], s["block"], post, pre, **kw)


# -------------------------------------------------------------- plain forms ----

def _conv_plain(s):
    dt, k, n = DTYPES[s["x"]], s["k"], s["l"]
    x, w, s0 = s["in"].float(), s["w"].float(), s["s0"].float()
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(n, device=x.device) < s["lengths"][:, None])[..., None]
        x = torch.where(live, x, 0.0)
    full = torch.cat([s0, x], 1)
    pre = sum(w[j] * full[:, j:j + n] for j in range(k))
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    sig = 1.0 / (1.0 + torch.exp(-pre))
    y = pre * sig
    if live is None:
        ends = torch.full((x.shape[0],), n, device=x.device)
        s1 = full[:, n:]
    else:
        y = torch.where(live, y, 0.0)
        ends = s["lengths"].long()
        at = ends[:, None] + torch.arange(k - 1, device=x.device)
        s1 = full.gather(1, at[..., None].expand(-1, -1, x.shape[2]))
    y, s1 = y.to(dt), s1.to(dt)
    if s["mode"] != "train":
        return y, s1
    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    e = dy * (sig + pre * sig * (1.0 - sig))
    dfull = torch.zeros_like(full)
    dw = []
    for j in range(k):
        dfull[:, j:j + n] += w[j] * e
        dw.append((e * full[:, j:j + n]).sum((0, 1)))
    at = ends[:, None] + torch.arange(k - 1, device=x.device)
    dfull.scatter_add_(1, at[..., None].expand(-1, -1, x.shape[2]), s["ds"].float())
    return (y, s1, dfull[:, k - 1:].to(dt), torch.stack(dw),
            e.sum((0, 1)) if s["bias"] is not None else None, dfull[:, :k - 1].to(dt))


def _softplus(x):
    return x.clamp_min(0.0) + torch.log1p(torch.exp(-x.abs()))


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _wide(t, d):
    """b x l x g x n for each channel: b x l x d x n."""
    g = t.shape[2]
    return t[:, :, :, None].expand(-1, -1, -1, d // g, -1).flatten(2, 3)


def _scan_tokens(u, delta, a, b, c, skip, z, bias, s0, lengths):
    """The scan in 32 bits, chunks of tokens side by side: each from a state of zero, then the
    chunks' states one after the other."""
    nb, n, d = u.shape
    m = a.shape[1]
    dt = _softplus(delta + bias)
    live = None
    if lengths is not None:
        live = (torch.arange(n, device=u.device) < lengths[:, None])[..., None]
        dt, u = torch.where(live, dt, 0.0), torch.where(live, u, 0.0)
    t = min(CHUNK, n)
    pad = -n % t

    def split(v):
        return torch.nn.functional.pad(v, (0, 0, 0, pad)).unflatten(1, (-1, t))

    du, dc = split(dt * u), split(dt)
    wide_b, wide_c = (split(_wide(v, d).flatten(2)).unflatten(-1, (d, m)) for v in (b, c))
    decay = torch.exp(dc[..., None] * a)
    into = du[..., None] * wide_b
    h, local = torch.zeros_like(into[:, :, 0]), []
    for keep, add in zip(decay.unbind(2), into.unbind(2)):
        h = keep * h + add
        local.append(h)
    local = torch.stack(local, 2)
    since = torch.exp(dc.cumsum(2)[..., None] * a)
    state, first = s0, []
    for keep, add in zip(since[:, :, -1].unbind(1), local[:, :, -1].unbind(1)):
        first.append(state)
        state = keep * state + add
    h = local + since * torch.stack(first, 1)[:, :, None]
    y = (h * wide_c).sum(-1).flatten(1, 2)[:, :n] + skip * u
    if z is not None:
        y = y * _silu(z)
    return (y if live is None else torch.where(live, y, 0.0)), state


def _scan_plain(s):
    dt = DTYPES[s["x"]]
    f = lambda t: t.float() if t is not None else None  # noqa: E731
    a = [f(s[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "bias", "s0")]
    if s["mode"] != "train":
        y, s1 = _scan_tokens(*a, s["lengths"])
        return y.to(dt), s1
    leaves = [t.detach().requires_grad_() if t is not None else None for t in a]
    y, s1 = _scan_tokens(*leaves, s["lengths"])
    some = [t for t in leaves if t is not None]
    g = iter(torch.autograd.grad([y, s1], some, [s["dy"].float(), s["ds"]]))
    g = [next(g) if t is not None else None for t in leaves]
    for i in (0, 1, 3, 4, 6):
        g[i] = g[i].to(dt) if g[i] is not None else None
    return (y.detach().to(dt), s1.detach(), *g)


def _act(g, act):
    """(act(g), its derivative)"""
    if g is None:
        return 1.0, 0.0
    sig = 1.0 / (1.0 + torch.exp(-g))
    if act == "sigmoid":
        return sig, sig * (1.0 - sig)
    return g * sig, sig + g * sig * (1.0 - sig)


def _norm_plain(s):
    xt, yt = s["in"].dtype, s["block"].dtype
    x, y = s["in"].float(), s["block"].float()
    gate = s["gate"].float() if s["gate"] is not None else None
    scale = s["s"] if s["s"] is not None else 1.0
    r1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    yh = y * r1
    p = yh * s["w_post"]
    act, slope = _act(gate, s["act"])
    r = x + scale * act * p
    r2 = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    rh = r * r2
    out = (r.to(xt), (rh * s["w_pre"]).to(yt))
    if not s["train"]:
        return out
    dh = s["dh"].float()
    e = dh * s["w_pre"]
    t = s["dr"].float() + r2 * (e - rh * (e * rh).mean(-1, keepdim=True))
    dp = t * scale * act
    e1 = dp * s["w_post"]
    dy = r1 * (e1 - yh * (e1 * yh).mean(-1, keepdim=True))
    return out + (t.to(xt), dy.to(yt),
                  (t * scale * p * slope).to(yt) if gate is not None else None,
                  (t * act * p).sum(0) if s["s"] is not None else None,
                  (dp * yh).sum(0), (dh * rh).sum(0))


# ------------------------------------------------------ definitions, 64 bits ----

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "conv":
        return _conv_exact(s)
    if case["op"] == "scan":
        return _scan_exact(s)
    return _norm_exact(s)


def _conv_exact(s):
    """By shifted copies of each sequence's own tokens, one sequence at a time."""
    k, n, d = s["k"], s["l"], s["d"]
    w = s["w"].double()
    bias = s["bias"].double() if s["bias"] is not None else torch.zeros_like(w[0])
    b, train = s["in"].shape[0], s["mode"] == "train"
    y = torch.zeros(b, n, d, dtype=torch.float64, device=w.device)
    s1 = torch.zeros(b, k - 1, d, dtype=torch.float64, device=w.device)
    dx, ds0 = torch.zeros_like(y), torch.zeros_like(s1)
    dw, dbias = torch.zeros_like(w), torch.zeros_like(bias)
    lens = [n] * b if s["lengths"] is None else s["lengths"].tolist()
    for i, m in enumerate(lens):
        seq = torch.cat([s["s0"][i].double(), s["in"][i, :m].double()])
        s1[i] = seq[m:]
        pre = bias.expand(m, d).clone()
        for j in range(k):
            pre += w[j] * seq[j:j + m]
        y[i, :m] = pre / (1.0 + torch.exp(-pre))
        if not train:
            continue
        sig = torch.sigmoid(pre)
        e = s["dy"][i, :m].double() * sig * (1.0 + pre * (1.0 - sig))
        dseq = torch.zeros_like(seq)
        dseq[m:] += s["ds"][i].double()
        for j in range(k):
            dseq[j:j + m] += w[j] * e
            dw[j] += (e * seq[j:j + m]).sum(0)
        dbias += e.sum(0)
        dx[i, :m], ds0[i] = dseq[k - 1:], dseq[:k - 1]
    if not train:
        return y, s1
    return y, s1, dx, dw, dbias if s["bias"] is not None else None, ds0


def _scan_exact(s):
    """Token by token, and back by the adjoint of each token's update."""
    nb, n, d = s["u"].shape
    g, m = s["g"], s["n"]
    a, skip = s["A"].double(), s["D"].double()
    u = s["u"].double()
    raw = s["delta"].double() + s["bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    bb, cc = s["B"].double(), s["C"].double()
    z = s["z"].double() if s["z"] is not None else None
    silu = z * torch.sigmoid(z) if z is not None else 1.0
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(n, device=u.device)[None] < s["lengths"][:, None])[..., None]
        dt, u = dt * live, u * live
    each = lambda t: t.repeat_interleave(d // g, 1)  # b x g x n -> b x d x n  # noqa: E731
    train = s["mode"] == "train"
    h, o, kept = s["s0"].double(), torch.empty_like(u), []
    for t in range(n):
        if train:
            kept.append(h)
        step = dt[:, t, :, None]
        h = torch.exp(step * a) * h + step * u[:, t, :, None] * each(bb[:, t])
        o[:, t] = (h * each(cc[:, t])).sum(-1) + skip * u[:, t]
    y = o * silu
    if live is not None:
        y = y * live
    if not train:
        return y, h
    s1 = h
    dy = s["dy"].double()
    if live is not None:
        dy = dy * live
    do, dz = dy * silu, None
    if z is not None:
        sig = torch.sigmoid(z)
        dz = dy * o * sig * (1.0 + z * (1.0 - sig))
    du, ddt = skip * do, torch.empty_like(u)
    db, dc = torch.empty_like(bb), torch.empty_like(cc)
    da, gr = torch.zeros_like(a), s["ds"].double()
    shared = lambda t: t.unflatten(1, (g, d // g)).sum(2)  # noqa: E731
    for t in reversed(range(n)):
        step = dt[:, t, :, None]
        gr = gr + each(cc[:, t]) * do[:, t, :, None]
        dc[:, t] = shared(do[:, t, :, None] * h)
        db[:, t] = shared(gr * (step * u[:, t, :, None]))
        along = (gr * each(bb[:, t])).sum(-1)
        decay = torch.exp(step * a)
        before = kept.pop()
        through = gr * decay * before
        ddt[:, t] = (through * a).sum(-1) + u[:, t] * along
        du[:, t] += dt[:, t] * along
        da += (step * through).sum(0)
        h, gr = before, gr * decay
    ddelta = ddt * torch.sigmoid(raw)
    if live is not None:
        ddelta, du, db, dc = (t * live if t.dim() == 3 else t * live[..., None]
                              for t in (ddelta, du, db, dc))
    return (y, s1, du, ddelta, da, db, dc, (do * u).sum((0, 1)), dz, ddelta.sum((0, 1)), gr)


def _norm_exact(s):
    x, y, c = s["in"].double(), s["block"].double(), s["c"]
    post, pre = s["w_post"].double(), s["w_pre"].double()
    scale = s["s"].double() if s["s"] is not None else torch.ones_like(post)
    if s["gate"] is None:
        act, slope = torch.ones_like(y), None
    else:
        gate = s["gate"].double()
        sig = torch.sigmoid(gate)
        act, slope = sig, sig * torch.sigmoid(-gate)
        if s["act"] == "silu":
            act, slope = gate * sig, sig * (1.0 + gate * torch.sigmoid(-gate))
    q1 = 1.0 / torch.sqrt((y ** 2).sum(1, keepdim=True) / c + EPS)
    r = x + scale * act * (y * q1 * post)
    q2 = 1.0 / torch.sqrt((r ** 2).sum(1, keepdim=True) / c + EPS)
    h = r * q2 * pre
    if not s["train"]:
        return r, h
    dh = s["dh"].double()
    e = dh * pre
    t = s["dr"].double() + q2 * e - r * q2 ** 3 * (e * r).sum(1, keepdim=True) / c
    dp = t * scale * act
    e = dp * post
    dy = q1 * e - y * q1 ** 3 * (e * y).sum(1, keepdim=True) / c
    p = y * q1 * post
    return (r, h, t, dy, t * scale * p * slope if slope is not None else None,
            (t * act * p).sum(0) if s["s"] is not None else None, (dp * y * q1).sum(0),
            (dh * r * q2).sum(0))


def work(case):
    e = BYTES[case["x"]]
    if case["op"] == "norm":
        n, c, f = case["rows"] * case["c"], case["c"], BYTES[case["y"]]
        gate = f if case["act"] else 0
        vectors = 4 * c * (2 + case["scale"])
        # x, y and the gate read, r and h written
        fwd = n * (2 * e + 2 * f + gate)
        if not case["train"]:
            return {"bytes": fwd + vectors, "flops": 12 * n}
        # and dr and dh read, dx, dy and the gate's gradient written
        return {"bytes": fwd + n * (2 * e + 2 * f + gate) + 2 * vectors, "flops": 40 * n}
    b, n, d = case["b"], case["l"], case["d"]
    t = b * n * d
    if case["op"] == "conv":
        k = case["k"]
        ends = 2 * b * (k - 1) * d * e
        vectors = d * (k + case["bias"])
        if case["mode"] != "train":
            return {"bytes": 2 * t * e + ends + vectors * e, "flops": t * (2 * k + 5)}
        return {"bytes": 4 * t * e + 2 * ends + vectors * (e + 4), "flops": t * (6 * k + 20)}
    g, m = case["g"], case["n"]
    tokens = t * e * (3 + case["gate"]) + 2 * b * n * g * m * e  # u, delta, z, B, C read, y written
    vectors, ends = 4 * d * (m + 2), 8 * b * d * m
    flops = t * (7 * m + 20)
    if case["mode"] != "train":
        return {"bytes": tokens + vectors + ends, "flops": flops}
    # and dy read, the gradients written
    tokens += t * e * (3 + case["gate"]) + 2 * b * n * g * m * e
    return {"bytes": tokens + 2 * vectors + 2 * ends, "flops": 3 * flops}
