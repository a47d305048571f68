"""Measured cases of what stands around a recurrent token mixer's rule.

Three operators over packed sequences, each in its plain form (elementary
torch operations in 32 bits, sums over all tokens in 64) and as the library's
calls; "form" is the direction (fwd, bwd) or the token step (step):

  scan  the gated linear recurrence per channel, h = e^g h + m w x, m = 1,
        1 - e^g ("convex") or sqrt(1 - e^(2 g)) ("unit")
  conv  the short causal convolution per channel, with its state and SiLU
  norm  layer or RMS norm of rows, with weight, bias and a SiLU gate

``exact`` evaluates the definitions in 64 bits, the recurrence token by token
where the plain form doubles the scanned length.
"""

from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
EPS = {"layer": 1e-5, "rms": 1e-6}


# ---------------------------------------------------------------- cases --

def _scan(form, name=None, **kw):
    return _named({"op": "scan", "form": form, **kw}, name)


def _conv(form, name=None, **kw):
    return _named({"op": "conv", "form": form, **kw}, name)


def _norm(form, name=None, **kw):
    return _named({"op": "norm", "form": form, **kw}, name)


def _named(case, name):
    return case if name is None else {"name": name, **case}


def listed():
    return [
        # one very long document on a small model: few channels, the whole GPU on one sequence
        _scan("fwd", "scan_long", seqs=1, longest=65536, shortest=65536, D=1024, io="bf16", g="bf16", w=False, scale="convex",
              init=False),
        # a packed prefill batch of ragged prompts, the library's varlen shape at 32 heads of 128 channels
        _scan("fwd", "scan_varlen", seqs=8, longest=8192, shortest=256, D=4096, io="bf16", g="f32", w=True, scale="unit", init=True),
        # decode of a serving batch
        _scan("step", "scan_decode", seqs=128, longest=1, shortest=1, D=4096, io="bf16", g="f32", w=True, scale="unit", init=True),
        # a small training step, an odd number of channels: latency
        _scan("bwd", "scan_bwd_short", seqs=5, longest=333, shortest=1, D=321, io="fp16", g="f32", w=True, scale="unit", init=True),
        # a packed training batch of the varlen shape
        _scan("bwd", "scan_bwd_varlen", seqs=8, longest=8192, shortest=256, D=4096, io="bf16", g="f32", w=True, scale="unit",
              init=True),
        # decode: q, k and v of 16 + 16 + 32 heads of 128 channels at once
        _conv("step", "conv_decode", seqs=128, longest=1, shortest=1, D=8192, io="bf16", taps=4, bias=False, act="silu", init=True),
        # the packed prefill batch's q, k and v
        _conv("fwd", "conv_varlen", seqs=8, longest=8192, shortest=256, D=8192, io="bf16", taps=4, bias=True, act="silu", init=True),
        # and its training step
        _conv("bwd", "conv_bwd_varlen", seqs=8, longest=8192, shortest=256, D=8192, io="bf16", taps=4, bias=True, act="silu",
              init=False),
        # decode: the rule's output of 32 heads of 128, gated
        _norm("fwd", "norm_decode", tokens=128, heads=32, D=128, io="bf16", kind="rms", weight="f32", bias=False, gate=True),
        # the residual stream of a prefill batch, kept in 32 bits
        _norm("fwd", "norm_stream", tokens=16384, heads=1, D=4096, io="f32", kind="layer", weight="f32", bias=True, gate=False),
        # a small training step of an odd width: latency
        _norm("bwd", "norm_bwd_odd", tokens=333, heads=1, D=1001, io="fp16", kind="layer", weight="f32", bias=True, gate=False),
        # a training step's gated output norm
        _norm("bwd", "norm_bwd_gated", tokens=16384, heads=32, D=128, io="bf16", kind="rms", weight="f32", bias=False, gate=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng: random.Random):
    op = rng.choice(["scan", "scan", "conv", "norm"])
    io = rng.choice(["bf16", "bf16", "fp16", "f32"])
    if op == "norm":
        # (a row of one or two elements has no gradient but what eps leaves, the difference of two like numbers)
        D = rng.choice([64, 128, 256, _spread(rng, 8, 8192), 8 * _spread(rng, 1, 1024)])
        heads = rng.choice([1, rng.randint(1, 32)]) if D <= 256 else 1
        tokens = _spread(rng, 1, min(32768, 2 ** 26 // (D * heads)))
        return _norm(rng.choice(["fwd", "bwd"]), tokens=tokens, heads=heads, D=D, io=io, kind=rng.choice(["layer", "rms"]),
                     weight=rng.choice(["f32", "io"]), bias=rng.random() < 0.5, gate=rng.random() < 0.5)
    form = rng.choice(["fwd", "bwd", "step"] if op == "conv" else ["fwd", "fwd", "bwd", "step"])
    D = rng.choice([_spread(rng, 1, 8192), 64 * rng.randint(1, 64)])
    if form == "step":
        seqs, longest = _spread(rng, 1, 256), rng.choice([1, 1, 3, 8])
    else:
        most = 2 ** 26
        longest = _spread(rng, 1, min(65536, most // D))
        seqs = _spread(rng, 1, max(1, min(64, most // (longest * D))))
    if op == "conv":
        return _conv(form, seqs=seqs, longest=longest, shortest=rng.randint(1, longest), D=D, io=io, taps=rng.choice([2, 3, 4, 4]),
                     bias=rng.random() < 0.5, act=rng.choice(["silu", "silu", "none"]), init=form == "step" or rng.random() < 0.5)
    return _scan(form, seqs=seqs, longest=longest, shortest=rng.randint(1, longest), D=D, io=io, g=rng.choice(["f32", "f32", "io"]),
                 w=rng.random() < 0.6, scale=rng.choice(["none", "convex", "unit"]), init=form == "step" or rng.random() < 0.5)


def _type(case, what):
    return TYPES[case["io"] if case[what] == "io" else case[what]]


def _lengths(case, seed=0):
    """The case's lengths (the longest always among them), in an order that goes by the seed."""
    r = random.Random(case["seqs"] * 1000003 + case["longest"] * 1009 + case["shortest"])
    lens = [case["longest"]] + [r.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"] - 1)]
    random.Random(seed).shuffle(lens)
    return lens


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    io, D = TYPES[case["io"]], case["D"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    if case["op"] == "norm":
        shape = (case["tokens"], case["heads"], D)
        wt = _type(case, "weight")
        # a residual stream has channels that are off centre
        s = {"case": case, "x": (2.0 * normal(*shape) + 0.5 * normal(D)).to(io), "weight": (1.0 + 0.3 * normal(D)).to(wt),
             "bias": (0.2 * normal(D)).to(wt) if case["bias"] else None, "gate": normal(*shape).to(io) if case["gate"] else None}
        if case["form"] == "bwd":
            s["d_out"] = normal(*shape).to(io)
        return s
    lens = _lengths(case, seed)
    T, N = sum(lens), len(lens)
    s = {"case": case, "lens": lens, "cu": torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32), "x": normal(T, D).to(io)}
    if case["op"] == "conv":
        K = case["taps"]
        s["weight"] = (normal(D, K) * K ** -0.5).to(io)
        s["bias"] = (0.2 * normal(D)).to(io) if case["bias"] else None
        s["S0"] = normal(N, K - 1, D).to(io) if case["init"] else None
        if case["form"] == "bwd":
            s["d_out"], s["dST"] = normal(T, D).to(io), normal(N, K - 1, D).to(io)
        return s
    # decay rates of the channels spread over three decades, as trained recurrences have them, gated by the token
    rate = torch.exp(math.log(1e-3) + uniform(D) * math.log(1e3))
    s["g"] = (-rate * torch.sigmoid(normal(T, D)) - 1e-5).to(_type(case, "g"))
    s["w"] = torch.sigmoid(normal(T, D)).to(io) if case["w"] else None
    s["S0"] = normal(N, D) if case["init"] else None
    if case["form"] == "bwd":
        s["d_out"], s["dST"] = normal(T, D).to(io), normal(N, D)
    return s


# ----------------------------------------------------------- plain forms --

def _doubled(a, u):
    """h_t = a_t h_{t-1} + u_t over the first dimension, from zero: every pass doubles the tokens that a row sums up."""
    d, T = 1, u.shape[0]
    while d < T:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _drive(s, g):
    """The factor m of the inputs and its derivative by g."""
    a, kind = g.exp(), s["case"]["scale"]
    if kind == "none":
        return torch.ones_like(g), torch.zeros_like(g)
    if kind == "convex":
        return -torch.expm1(g), -a
    m = (-torch.expm1(2.0 * g)).sqrt()
    return m, torch.where(m > 0, -a * a / m, 0.0)


def _plain_scan(s):
    c, first, last = s["case"], s["cu"][:-1].long(), s["cu"][1:].long() - 1
    g, v = s["g"].float(), s["x"].float()
    if s["w"] is not None:
        v = v * s["w"].float()
    a, u = g.exp(), _drive(s, g)[0] * v
    if s["S0"] is not None:
        u[first] += a[first] * s["S0"]
    a[first] = 0.0
    h = _doubled(a, u)
    return h.to(TYPES[c["io"]]), h[last]


def _plain_scan_bwd(s):
    c, io, first, last = s["case"], TYPES[s["case"]["io"]], s["cu"][:-1].long(), s["cu"][1:].long() - 1
    g, x = s["g"].float(), s["x"].float()
    w = torch.ones_like(x) if s["w"] is None else s["w"].float()
    a, (m, dm) = g.exp(), _drive(s, g)
    u, inner = m * w * x, a.clone()
    if s["S0"] is not None:
        u[first] += a[first] * s["S0"]
    inner[first] = 0.0
    h = _doubled(inner, u)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = s["S0"] if s["S0"] is not None else 0.0
    dh = s["d_out"].float()
    dh[last] += s["dST"]
    after = torch.cat([inner[1:], torch.zeros_like(a[:1])])  # the next token's decay, none behind a sequence's last
    dh = _doubled(after.flip(0), dh.flip(0)).flip(0)
    got = {"dx": (m * w * dh).to(io), "dg": (dh * (a * before + dm * w * x)).to(s["g"].dtype),
           "d_initial_state": a[first] * dh[first]}
    if s["w"] is not None:
        got["dw"] = (m * x * dh).to(io)
    return got


def _with_state(s):
    """The inputs with each sequence's K - 1 rows of state before it, [T + N (K - 1), D], and the places of the tokens in it."""
    c, K = s["case"], s["case"]["taps"]
    N, D = len(s["lens"]), c["D"]
    n = torch.searchsorted(s["cu"][1:].long(), torch.arange(s["x"].shape[0], device=s["x"].device), right=True)
    at = torch.arange(s["x"].shape[0], device=n.device) + (n + 1) * (K - 1)
    rows = s["cu"][:-1].long()[:, None] + torch.arange(N, device=n.device)[:, None] * (K - 1) + torch.arange(K - 1, device=n.device)
    z = s["x"].new_zeros(s["x"].shape[0] + N * (K - 1), D, dtype=torch.float32)
    z[at] = s["x"].float()
    if s["S0"] is not None:
        z[rows.flatten()] = s["S0"].float().flatten(0, 1)
    return z, at, rows


def _products(s, z, at):
    """The convolution before the activation, [T, D]."""
    K = s["case"]["taps"]
    w = s["weight"].float()
    p = sum(z[at - (K - 1) + j] * w[:, j] for j in range(K))
    return p if s["bias"] is None else p + s["bias"].float()


def _last_rows(s, rows):
    """Where each sequence's last K - 1 inputs are in _with_state's order."""
    return rows + (s["cu"][1:] - s["cu"][:-1]).long()[:, None]


def _plain_conv(s):
    c, io = s["case"], TYPES[s["case"]["io"]]
    z, at, rows = _with_state(s)
    p = _products(s, z, at)
    y = p * torch.sigmoid(p) if c["act"] == "silu" else p
    return y.to(io), z[_last_rows(s, rows)].to(io)


def _plain_conv_bwd(s):
    c, K, io = s["case"], s["case"]["taps"], TYPES[s["case"]["io"]]
    z, at, rows = _with_state(s)
    dp, w = s["d_out"].float(), s["weight"].float()
    if c["act"] == "silu":
        p = _products(s, z, at)
        sig = torch.sigmoid(p)
        dp = dp * sig * (1.0 + p * (1.0 - sig))
    wide = torch.zeros_like(z)
    wide[at] = dp
    wide = torch.cat([wide, wide.new_zeros(K - 1, wide.shape[1])])
    dz = torch.zeros_like(z)
    L = z.shape[0]
    for j in range(K):
        # row i feeds the token K - 1 - j rows on, where that is still a token (rows of state between have none)
        dz += wide[K - 1 - j:K - 1 - j + L] * w[:, j]
    dz[_last_rows(s, rows).flatten()] += s["dST"].float().flatten(0, 1)
    got = {"dx": dz[at].to(io), "d_initial_state": dz[rows].to(io),
           "dweight": torch.stack([(dp * z[at - (K - 1) + j]).sum(0, dtype=torch.float64) for j in range(K)], 1).to(io)}
    if s["bias"] is not None:
        got["dbias"] = dp.sum(0, dtype=torch.float64).to(io)
    return got


def _centred(s):
    """Normalised rows, and the factor they were normalised by, in 32 bits."""
    x, kind = s["x"].float(), s["case"]["kind"]
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS[kind]).rsqrt()
    return x * r, r


def _affine(s, n):
    p = n * s["weight"].float()
    return p if s["bias"] is None else p + s["bias"].float()


def _plain_norm(s):
    y = _affine(s, _centred(s)[0])
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(TYPES[s["case"]["io"]])


def _plain_norm_bwd(s):
    io = TYPES[s["case"]["io"]]
    n, r = _centred(s)
    dp, got = s["d_out"].float(), {}
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        got["dgate"] = (dp * _affine(s, n) * (sig * (1.0 + z * (1.0 - sig)))).to(io)
        dp = dp * (z * sig)
    wt = s["weight"].dtype
    got["dweight"] = (dp * n).sum((0, 1), dtype=torch.float64).to(wt)
    if s["bias"] is not None:
        got["dbias"] = dp.sum((0, 1), dtype=torch.float64).to(wt)
    m = dp * s["weight"].float()
    dx = m - n * (m * n).mean(-1, keepdim=True)
    if s["case"]["kind"] == "layer":
        dx = dx - m.mean(-1, keepdim=True)
    got["dx"] = (r * dx).to(io)
    return got


# ------------------------------------------------------ the library's calls --

def _own_scan(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    call = gdn2.linear_scan_recurrent_fwd if s["case"]["form"] == "step" else gdn2.linear_scan_fwd
    return call(s["x"], s["g"], s["w"], initial_state=s["S0"], cu_seqlens=s["cu"], input_scale=s["case"]["scale"])


def _own_scan_bwd(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    got = gdn2.linear_scan_bwd(s["x"], s["g"], s["w"], s["d_out"], initial_state=s["S0"], cu_seqlens=s["cu"], d_final_state=s["dST"],
                               input_scale=s["case"]["scale"])
    return {n: got[n] for n in ("dx", "dg", "d_initial_state", "dw") if got[n] is not None}


def _own_conv(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    call = gdn2.short_conv_recurrent_fwd if s["case"]["form"] == "step" else gdn2.short_conv_fwd
    return call(s["x"], s["weight"], s["bias"], initial_state=s["S0"], cu_seqlens=s["cu"], activation=s["case"]["act"])


def _own_conv_bwd(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    got = gdn2.short_conv_bwd(s["x"], s["weight"], s["bias"], s["d_out"], initial_state=s["S0"], cu_seqlens=s["cu"],
                              d_final_state=s["dST"], activation=s["case"]["act"])
    return {n: got[n] for n in ("dx", "d_initial_state", "dweight", "dbias") if got[n] is not None}


def _own_norm(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    return gdn2.layer_norm(s["x"], s["weight"], s["bias"], gate=s["gate"], norm=s["case"]["kind"])


def _own_norm_bwd(s):
    from linear_attention_rnn_gdn2_amd import gdn2
    got = gdn2.layer_norm_bwd(s["x"], s["d_out"], s["weight"], s["bias"], gate=s["gate"], norm=s["case"]["kind"])
    return {n: got[n] for n in ("dgate", "dweight", "dbias", "dx") if got[n] is not None}


def run(state):
    op, back = state["case"]["op"], state["case"]["form"] == "bwd"
    if own:
        if op == "scan":
            return _own_scan_bwd(state) if back else _own_scan(state)
        if op == "conv":
            return _own_conv_bwd(state) if back else _own_conv(state)
        return _own_norm_bwd(state) if back else _own_norm(state)
    if op == "scan":
        return _plain_scan_bwd(state) if back else _plain_scan(state)
    if op == "conv":
        return _plain_conv_bwd(state) if back else _plain_conv(state)
    return _plain_norm_bwd(state) if back else _plain_norm(state)


# -------------------------------------------------------------------- work --

def _size(case, what):
    return 4 if _type(case, what) == torch.float32 else 2


def work(case):
    D, io, back = case["D"], 4 if case["io"] == "f32" else 2, case["form"] == "bwd"
    if case["op"] == "norm":
        rows = case["tokens"] * case["heads"]
        each = (5 if back else 3) if case["gate"] else (3 if back else 2)
        vectors = D * _size(case, "weight") * (2 if case["bias"] else 1) * (2 if back else 1)
        return {"bytes": rows * D * io * each + vectors, "flops": rows * D * (20 if back else 10)}
    T, N = sum(_lengths(case)), case["seqs"]
    if case["op"] == "conv":
        K = case["taps"]
        state = N * (K - 1) * D * io * (2 + case["init"] if back else 1 + case["init"])
        vectors = D * (K + case["bias"]) * io * (2 if back else 1)
        return {"bytes": T * D * io * (3 if back else 2) + state + vectors, "flops": T * D * ((6 if back else 2) * K + 8)}
    g, w = _size(case, "g"), 1 if case["w"] else 0
    state = N * D * 4 * (2 + case["init"] if back else 1 + case["init"])
    # x, w, g and the output or its gradient in; the gradients out
    rows = (io * (3 + 2 * w) + 2 * g) if back else (io * (2 + w) + g)
    return {"bytes": T * D * rows + state, "flops": T * D * (24 if back else 8)}


# -------------------------------------------------------- 64-bit definition --

def _padded64(s, name):
    """[length, N, D] in 64 bits, zeros before a sequence's tokens."""
    L, start = max(s["lens"]), 0
    x = s[name].double()
    y = x.new_zeros(L, len(s["lens"]), x.shape[1])
    for i, l in enumerate(s["lens"]):
        y[L - l:, i] = x[start:start + l]
        start += l
    return y


def _joined(s, y):
    L = max(s["lens"])
    return torch.cat([y[L - l:, i] for i, l in enumerate(s["lens"])])


def _factor64(kind, g):
    if kind == "none":
        return torch.ones_like(g), torch.zeros_like(g)
    a = torch.exp(g)
    if kind == "convex":
        return -torch.expm1(g), -a
    m = torch.sqrt(-torch.expm1(2.0 * g))
    return m, -(a * a) / m.clamp_min(1e-300) * (m > 0)


def _exact_scan(s):
    """Token by token; sequences lie at the end of the padded length, so that all of them end together."""
    c, L = s["case"], max(s["lens"])
    g, x = _padded64(s, "g"), _padded64(s, "x")
    v = x if s["w"] is None else x * _padded64(s, "w")
    m, dm = _factor64(c["scale"], g)
    inside = torch.zeros(L, len(s["lens"]), 1, dtype=torch.bool, device=x.device)
    for i, l in enumerate(s["lens"]):
        inside[L - l:, i] = True
    a, u = torch.where(inside, g.exp(), 1.0), m * v * inside
    h = s["S0"].double() if s["S0"] is not None else x.new_zeros(x.shape[1:])
    first, hs = h, torch.empty_like(x)
    for t in range(L):
        h = torch.addcmul(u[t], a[t], h)
        hs[t] = h
    if c["form"] != "bwd":
        return _joined(s, hs), h
    dh, out = s["dST"].double(), _padded64(s, "d_out")
    ds = torch.empty_like(x)
    for t in reversed(range(L)):
        dh = out[t] + dh
        ds[t] = dh
        dh = a[t] * dh
    before = torch.cat([first[None], hs[:-1]])
    got = {"dg": _joined(s, ds * (a * before + dm * v)), "d_initial_state": dh}
    if s["w"] is None:
        got["dx"] = _joined(s, m * ds)
    else:
        got["dx"] = _joined(s, m * ds * _padded64(s, "w"))
        got["dw"] = _joined(s, m * ds * x)
    return got


def _exact_conv(s):
    """Sequence by sequence, differentiable."""
    c, K = s["case"], s["case"]["taps"]
    leaves = {n: s[n].double() for n in ("x", "weight", "bias", "S0") if s[n] is not None}
    if "S0" not in leaves:
        leaves["S0"] = leaves["x"].new_zeros(len(s["lens"]), K - 1, c["D"])
    back = c["form"] == "bwd"
    if back:
        sums = {n: torch.zeros_like(leaves[n]) for n in leaves}
    outs, ends, start = [], [], 0
    for i, l in enumerate(s["lens"]):
        x, S0 = leaves["x"][start:start + l], leaves["S0"][i]
        w, b = leaves["weight"], leaves.get("bias")
        if back:
            x, S0, w = (t.detach().requires_grad_() for t in (x, S0, w))
            b = None if b is None else b.detach().requires_grad_()
        z = torch.cat([S0, x])
        p = (z.unfold(0, K, 1) * w).sum(-1)
        p = p if b is None else p + b
        y = p / (1.0 + torch.exp(-p)) if c["act"] == "silu" else p
        if back:
            ((y * s["d_out"][start:start + l].double()).sum() + (z[l:] * s["dST"][i].double()).sum()).backward()
            sums["x"][start:start + l], sums["S0"][i] = x.grad, S0.grad
            sums["weight"] += w.grad
            if b is not None:
                sums["bias"] += b.grad
        else:
            outs.append(y)
            ends.append(z[l:])
        start += l
    if not back:
        return torch.cat(outs), torch.stack(ends)
    names = {"x": "dx", "S0": "d_initial_state", "weight": "dweight", "bias": "dbias"}
    return {names[n]: t for n, t in sums.items()}


def _exact_norm(s):
    c = s["case"]
    leaves = {n: s[n].double() for n in ("x", "gate", "weight", "bias") if s[n] is not None}
    if c["form"] == "bwd":
        leaves = {n: t.requires_grad_() for n, t in leaves.items()}
    x = leaves["x"]
    if c["kind"] == "layer":
        x = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + EPS["layer"]).sqrt()
    else:
        x = x / ((x * x).sum(-1, keepdim=True) / c["D"] + EPS["rms"]).sqrt()
    y = x * leaves["weight"]
    if "bias" in leaves:
        y = y + leaves["bias"]
    if "gate" in leaves:
        y = y * leaves["gate"] / (1.0 + torch.exp(-leaves["gate"]))
    if c["form"] != "bwd":
        return y
    got = torch.autograd.grad(y, list(leaves.values()), s["d_out"].double())
    return {"d" + n: t for n, t in zip(leaves, got)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "conv": _exact_conv, "norm": _exact_norm}[case["op"]](s)
