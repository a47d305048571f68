"""Inputs and float64 references of the gated linear recurrence, the short
convolution and the layer norm.

Tolerances. A result of a 16-bit type is rounded once, by at most finfo.eps /
2 relative (``close`` adds it). Before that all arithmetic is float32, 2^-24 =
6e-8 per rounding:

  recurrence  every step rounds the state twice; a decay of rate r is
      remembered for M = 1 / r steps, so independent roundings leave sqrt(M)
      * sqrt(2) * 2^-24 in the 2-norm, 6.7e-7 at M = 64 (the rates here are
      0.02 and more, but for tests that say otherwise). e^g - 1 adds 1.1e-7, the
      factor m and the gated input six roundings more, 1.5e-7 together:
      SCAN_REL = 2e-6 is asked. dg is a sum of two products of such values,
      which may cancel to a part of either: DG_REL = 5e-6.
  convolution five products and a sigmoid (a reciprocal and an exponential
      of 2^-23 each): under ten roundings, CONV_REL = 1e-6.
  norm        sums over a row in pieces of 8 and a tree: under 30 roundings of
      which the sums' are independent, NORM_REL = 1e-6; dx is a difference of
      three terms of like size: NORM_DX_REL = 3e-6.
  sums over tokens or rows (weights' gradients) run over up to 256 terms in
      one register, then a tree: a sum of n terms of random sign is off by
      0.4 sqrt(n) * 2^-24 of itself, 4e-7, and joined parts the same again:
      SUM_REL = 3e-6.

Single elements may be off by the 2-norm's tolerance times sqrt(64 and more
channels) of the largest value: ELEMENT = 20 times the tolerance.
"""

import numpy as np
import torch

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SCAN_REL, DG_REL, CONV_REL, NORM_REL, NORM_DX_REL, SUM_REL = 2e-6, 5e-6, 1e-6, 1e-6, 3e-6, 3e-6
ELEMENT = 20


def close(tag, x, ref, rel):
    half = torch.finfo(x.dtype).eps / 2 if x.dtype != F32 else 0.0
    a, r = x.detach().cpu().double().numpy(), ref.detach().cpu().double().numpy()
    assert a.shape == r.shape, f"{tag}: {a.shape} {r.shape}"
    if not r.size:
        return
    assert np.isfinite(a).all(), f"{tag}: not finite"
    norm, err = np.linalg.norm(r), np.abs(a - r)
    got = np.linalg.norm(err) / norm if norm > 0 else np.linalg.norm(err)
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps  # a step under the smallest normal number
    worst = (err - half * np.abs(r) - tiny).max() / max(np.abs(r).max(), 1e-30)
    print(f"{tag}: rel-L2 {got:.2e} (allowed {rel + half:.2e}), element {worst:.2e}", flush=True)
    assert got <= rel + half and worst <= ELEMENT * rel, f"{tag}: rel-L2 {got:.3e}, element {worst:.3e}"


def cu_of(lens, dtype=torch.int32):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=dtype)


def gpu(d, names):
    return {n: None if d.get(n) is None else d[n].cuda() for n in names}


# ------------------------------------------------------------ recurrence --

SCAN_ARGS = ("x", "g", "w", "initial_state", "cu_seqlens")


def scan_inputs(lens, D, seed, io=BF16, gtype=F32, w=True, init=True, cu=torch.int32, lowest=0.02):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rate = lowest * torch.exp(torch.rand(D, generator=gen) * np.log(2.0 / lowest))
    return dict(x=torch.randn(T, D, generator=gen).to(io), g=(-rate * (0.5 + torch.rand(T, D, generator=gen))).to(gtype),
                w=torch.rand(T, D, generator=gen).to(io) if w else None,
                initial_state=torch.randn(N, D, generator=gen) if init else None,
                cu_seqlens=None if cu is None else cu_of(lens, cu), lens=lens,
                d_out=torch.randn(T, D, generator=gen).to(io), d_final_state=torch.randn(N, D, generator=gen))


def factor64(kind, g):
    if kind == "none":
        return torch.ones_like(g)
    return -torch.expm1(g) if kind == "convex" else torch.sqrt(-torch.expm1(2 * g))


def scan64(d, kind):
    """Token by token in float64: (out, final_state)."""
    x, g = d["x"].double(), d["g"].double()
    u = factor64(kind, g) * (x if d["w"] is None else x * d["w"].double())
    outs, ends, t = [], [], 0
    for n, l in enumerate(d["lens"]):
        h = x.new_zeros(x.shape[1]) if d["initial_state"] is None else d["initial_state"][n].double()
        for _ in range(l):
            h = g[t].exp() * h + u[t]
            outs.append(h)
            t += 1
        ends.append(h)
    return (torch.stack(outs) if outs else x[:0]), torch.stack(ends)


def scan64_grads(d, kind):
    """The gradients by autograd of scan64: dx, dg, dw, d_initial_state."""
    leaf = dict(d)
    names = [n for n in ("x", "g", "w", "initial_state") if d[n] is not None]
    for n in names:
        leaf[n] = d[n].double().requires_grad_()
    if d["initial_state"] is None:
        leaf["initial_state"] = torch.zeros(len(d["lens"]), d["x"].shape[1], dtype=torch.float64, requires_grad=True)
        names.append("initial_state")
    out, end = scan64(leaf, kind)
    loss = (out * d["d_out"].double()).sum()
    if d["d_final_state"] is not None:
        loss = loss + (end * d["d_final_state"].double()).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names], allow_unused=True)
    return {("d_" if n == "initial_state" else "d") + n: torch.zeros_like(leaf[n]) if t is None else t
            for n, t in zip(names, got)}


# ----------------------------------------------------------- convolution --

CONV_ARGS = ("x", "weight", "bias", "initial_state", "cu_seqlens")


def conv_inputs(lens, D, K, seed, io=BF16, wtype=None, bias=True, init=True, cu=torch.int32):
    gen = torch.Generator().manual_seed(seed)
    T, N, wt = sum(lens), len(lens), wtype or io
    return dict(x=torch.randn(T, D, generator=gen).to(io), weight=(0.6 * torch.randn(D, K, generator=gen)).to(wt),
                bias=(0.3 * torch.randn(D, generator=gen)).to(wt) if bias else None,
                initial_state=torch.randn(N, K - 1, D, generator=gen).to(io) if init else None,
                cu_seqlens=None if cu is None else cu_of(lens, cu), lens=lens,
                d_out=torch.randn(T, D, generator=gen).to(io), d_final_state=torch.randn(N, K - 1, D, generator=gen).to(io))


def conv64(d, act):
    x, w = d["x"].double(), d["weight"].double()
    K, outs, ends, t = w.shape[1], [], [], 0
    for n, l in enumerate(d["lens"]):
        s = x.new_zeros(K - 1, x.shape[1]) if d["initial_state"] is None else d["initial_state"][n].double()
        z = torch.cat([s, x[t:t + l]])
        p = sum(z[j:j + l] * w[:, j] for j in range(K))
        if d["bias"] is not None:
            p = p + d["bias"].double()
        outs.append(p * torch.sigmoid(p) if act == "silu" else p)
        ends.append(z[l:])
        t += l
    return torch.cat(outs), torch.stack(ends)


def conv64_grads(d, act):
    leaf = dict(d)
    names = [n for n in ("x", "weight", "bias", "initial_state") if d[n] is not None]
    for n in names:
        leaf[n] = d[n].double().requires_grad_()
    if d["initial_state"] is None:
        leaf["initial_state"] = torch.zeros(len(d["lens"]), d["weight"].shape[1] - 1, d["x"].shape[1], dtype=torch.float64,
                                            requires_grad=True)
        names.append("initial_state")
    out, end = conv64(leaf, act)
    loss = (out * d["d_out"].double()).sum()
    if d["d_final_state"] is not None:
        loss = loss + (end * d["d_final_state"].double()).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names])
    return {("d_" if n == "initial_state" else "d") + n: t for n, t in zip(names, got)}


# ------------------------------------------------------------------ norm --

NORM_ARGS = ("x", "weight", "bias", "gate")


def norm_inputs(T, H, D, seed, io=BF16, wtype=F32, btype=None, weight=True, bias=True, gate=True, offset=0.5):
    gen = torch.Generator().manual_seed(seed)
    return dict(x=(2 * torch.randn(T, H, D, generator=gen) + offset).to(io),
                weight=(1 + 0.3 * torch.randn(D, generator=gen)).to(wtype) if weight else None,
                bias=(0.3 * torch.randn(D, generator=gen)).to(btype or wtype) if bias else None,
                gate=torch.randn(T, H, D, generator=gen).to(io) if gate else None,
                d_out=torch.randn(T, H, D, generator=gen).to(io))


def norm64(d, kind, eps=None):
    x = d["x"].double() if not d["x"].requires_grad else d["x"]
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / (x.square().mean(-1, keepdim=True) + (eps or (1e-5 if kind == "layer" else 1e-6))).sqrt()
    if d["weight"] is not None:
        y = y * d["weight"].double()
    if d["bias"] is not None:
        y = y + d["bias"].double()
    if d["gate"] is not None:
        z = d["gate"].double()
        y = y * z * torch.sigmoid(z)
    return y


def norm64_grads(d, kind, eps=None):
    names = [n for n in NORM_ARGS if d[n] is not None]
    leaf = dict(d)
    for n in names:
        leaf[n] = d[n].double().requires_grad_()
    got = torch.autograd.grad(norm64(leaf, kind, eps), [leaf[n] for n in names], d["d_out"].double())
    return {"d" + n: t for n, t in zip(names, got)}
