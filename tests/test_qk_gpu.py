"""GPU tests of the q/k norms with the position rotation and their gradients,
against float64 autograd of the definition, and of the whole chain q/k
preparation -> delta rule -> gradients.

Tolerances: a 16-bit result is rounded once (finfo.eps / 2); the float32
arithmetic before it has about ten roundings of 2^-24 after sums of 128
terms, under 1e-6 in the 2-norm; the weights' gradients are float32 sums of
up to 2^15 terms in a fixed order, sqrt(2^15) * 2^-24 = 1.1e-5 at most.
"""

import pytest
import torch

from tests.delta_ref import F32_REL, close, make
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
REL = 1e-6
DW_REL = 1.1e-5


def rows64(x, w, norm, eps, rope, positions, interleaved):
    """The definition in float64: [T, heads, K]."""
    K = x.shape[-1]
    if norm == "l2":
        x = x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(eps or 1e-12)
    elif norm == "rms":
        x = x / (x.square().mean(-1, keepdim=True) + (eps or 1e-6)).sqrt()
    if w is not None:
        x = x * w
    if rope is None:
        return x
    rot = rope.shape[1]
    row = rope.double()[positions.long()][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, a * s + b * c
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:K]], -1)


def inputs(T, H, HK, K, io, wt, rot, seed, pos_type=torch.int32, P=500):
    gen = torch.Generator().manual_seed(seed)
    d = dict(q=(3 * torch.randn(T, H, K, generator=gen)).to(io), k=(0.2 * torch.randn(T, HK, K, generator=gen)).to(io),
             dq_out=torch.randn(T, H, K, generator=gen).to(io), dk_out=torch.randn(T, HK, K, generator=gen).to(io))
    d["q_weight"] = None if wt is None else (1 + 0.3 * torch.randn(K, generator=gen)).to(wt)
    d["k_weight"] = None if wt is None else (1 + 0.3 * torch.randn(K, generator=gen)).to(wt)
    from linear_attention_rnn_gdn2_amd.gdn2 import rope_table
    d["rope"] = rope_table(P, rot, device="cpu") if rot else None
    d["positions"] = torch.randint(0, P, (T,), generator=gen, dtype=pos_type) if rot else None
    return d


def gpu(d, names):
    return {n: None if d[n] is None else d[n].cuda() for n in names}


ARGS = ("q", "k", "q_weight", "k_weight", "rope", "positions")


@pytest.mark.parametrize("T,H,HK,K,io,norm,wt,rot,inter,pt", [
    (1, 1, 1, 64, BF16, "l2", None, 0, False, torch.int32),
    (5, 3, 2, 64, F16, "rms", F32, 64, False, torch.int64),
    (77, 2, 5, 128, BF16, "rms", BF16, 64, False, torch.int32),
    (300, 4, 1, 128, F16, "l2", F32, 128, True, torch.int32),
    (33, 1, 7, 64, BF16, "none", None, 32, True, torch.int64),
    (19, 16, 16, 128, BF16, "l2", None, 16, False, torch.int32),
    (40, 2, 2, 128, BF16, "none", F32, 0, False, torch.int32),
    (23, 3, 3, 64, F16, "rms", F16, 6, True, torch.int32)])
def test_forward_and_backward(lib, T, H, HK, K, io, norm, wt, rot, inter, pt):
    d = inputs(T, H, HK, K, io, wt, rot, seed=T + K, pos_type=pt)
    a = gpu(d, ARGS)
    kw = dict(norm=norm, interleaved=inter)
    y = lib.qk_norm_rope(**a, **kw)
    g = lib.qk_norm_rope_bwd(**a, dq_out=d["dq_out"].cuda(), dk_out=d["dk_out"].cuda(), **kw)
    torch.cuda.synchronize()
    for i, n in enumerate(("q", "k")):
        x = d[n].double().requires_grad_()
        w = d[n + "_weight"]
        w = None if w is None else w.double().requires_grad_()
        r = rows64(x, w, norm, None, d["rope"], d["positions"], inter)
        close(n, y[i], r.detach(), REL)
        r.backward(d[f"d{n}_out"].double())
        close("d" + n, g["d" + n], x.grad, REL)
        if w is None:
            assert g[f"d{n}_weight"] is None
        else:
            close(f"d{n}_weight", g[f"d{n}_weight"], w.grad, DW_REL)


def test_zero_and_tiny_rows(lib):
    """Rows of zeros and rows under eps: finite, and the gradient without the projection that the clamp removes."""
    d = inputs(4, 2, 2, 64, BF16, None, 0, seed=1)
    d["q"][1] = 0
    d["k"][2] = 0
    d["q"][3] = (d["q"][3].float() * 1e-3).to(BF16)
    for norm, eps in (("l2", 0.5), ("rms", 1e-3)):
        y = lib.qk_norm_rope(**gpu(d, ARGS), norm=norm, eps=eps)
        g = lib.qk_norm_rope_bwd(**gpu(d, ARGS), dq_out=d["dq_out"].cuda(), dk_out=d["dk_out"].cuda(), norm=norm, eps=eps)
        for i, n in enumerate(("q", "k")):
            x = d[n].double()
            s = x.square().sum(-1, keepdim=True)
            r = 1 / s.sqrt().clamp_min(eps) if norm == "l2" else 1 / (s / 64 + eps).sqrt()
            close(n, y[i], x * r, REL)
            dy = d[f"d{n}_out"].double()
            dot = (x * dy).sum(-1, keepdim=True) * r ** 3 * (1.0 if norm == "l2" else 1 / 64)
            if norm == "l2":
                dot = torch.where(s.sqrt() > eps, dot, 0.0)
            close("d" + n, g["d" + n], r * dy - x * dot, REL)


def test_default_equals_in_kernel_norm(lib):
    """The default (L2) followed by the rule equals the rule with qk_l2norm, but for the 16-bit rounding between them."""
    d = make([150], 2, 2, 64, 64, seed=2)
    d["q"], d["k"] = (4 * d["q"].float()).to(BF16), (4 * d["k"].float()).to(BF16)
    a = {n: None if d[n] is None else d[n].cuda() for n in ("q", "k", "v", "g", "beta", "initial_state", "cu_seqlens")}
    fused = lib.delta_chunk_fwd(**a, qk_l2norm=True)
    q, k = lib.qk_norm_rope(a["q"], a["k"])
    two = lib.delta_chunk_fwd(**dict(a, q=q, k=k))
    for x, y in zip(fused, two):
        assert (x.double() - y.double()).norm() <= 3 * 2.0 ** -8 * y.double().norm()


def test_strided_rows_and_clamped_positions(lib):
    """Views of one projection in and out; positions outside the table read its first or last row."""
    d = inputs(50, 2, 2, 64, BF16, F32, 64, seed=3, P=40)
    a = gpu(d, ARGS)
    want = lib.qk_norm_rope(**a)
    fused = torch.stack([a["q"], a["k"]], 1).contiguous()
    room_q, room_k = (torch.full((50, 3, 64), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    got = lib.qk_norm_rope(**dict(a, q=fused[:, 0], k=fused[:, 1]), q_out=room_q[:, :2], k_out=room_k[:, 1:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room_q[:, 2] == 7.0).all() and (room_k[:, 0] == 7.0).all()
    dy = d["dq_out"].cuda(), d["dk_out"].cuda()
    wb = lib.qk_norm_rope_bwd(**a, dq_out=dy[0], dk_out=dy[1])
    gb = lib.qk_norm_rope_bwd(**dict(a, q=fused[:, 0], k=fused[:, 1]), dq_out=dy[0], dk_out=dy[1])
    assert all(torch.equal(wb[n], gb[n]) for n in wb)
    far = dict(a, positions=torch.where(a["positions"] % 2 == 0, a["positions"] + 1000, a["positions"] - 1000))
    near = dict(a, positions=torch.where(a["positions"] % 2 == 0, 39, 0).to(torch.int32))
    x, y = lib.qk_norm_rope(**far), lib.qk_norm_rope(**near)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_no_tokens(lib):
    d = inputs(0, 1, 2, 64, BF16, F32, 32, seed=4)
    assert lib.qk_norm_rope(**gpu(d, ARGS))[0].shape == (0, 1, 64)
    g = lib.qk_norm_rope_bwd(**gpu(d, ARGS), dq_out=d["dq_out"].cuda(), dk_out=d["dk_out"].cuda())
    torch.cuda.synchronize()
    assert (g["dq_weight"] == 0).all() and (g["dk_weight"] == 0).all()


def test_graph_replays(lib):
    d, e = (inputs(70, 2, 1, 128, BF16, F32, 64, seed=s) for s in (5, 6))
    names = ARGS + ("dq_out", "dk_out")
    a, o = gpu(d, names), gpu(e, names)

    def call(x):
        f = lib.qk_norm_rope(**{n: x[n] for n in ARGS}, norm="rms")
        b = lib.qk_norm_rope_bwd(**x, norm="rms")
        return list(f) + [b[n] for n in sorted(b)]

    want = [call(a), call(o)]
    static = {n: x.clone() for n, x in a.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(static)
    for i in range(4):
        for n in static:
            static[n].copy_((a, o)[i % 2][n])
        eager = call((o, a)[i % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[i % 2]))
        assert all(torch.equal(x, y) for x, y in zip(eager, want[1 - i % 2]))


@pytest.mark.parametrize("io", [BF16, F16])
def test_chain_with_gradients(lib, io):
    """q/k preparation, the rule, and both backward passes, as a training step
    runs them, against float64 autograd token by token. Between the operators
    q, k and their gradients are rounded to 16 bits, each by half a step; the
    reference takes q and k as rounded (so the rule's inputs are equal), and
    dq, dk rounded once more pass through a linear map: two roundings."""
    T, H, HV, K = 90, 1, 2, 64
    d = make([70, 20], H, HV, K, K, seed=7, io=io)
    raw = inputs(T, H, H, K, io, F32, 32, seed=8)
    a = gpu(raw, ARGS)
    v, g, beta, s0, cu, do, dst = (d[n].cuda() for n in ("v", "g", "beta", "initial_state", "cu_seqlens", "d_out", "d_final_state"))
    q, k = lib.qk_norm_rope(**a)
    out, state = lib.delta_chunk_fwd(q, k, v, g, beta, initial_state=s0, cu_seqlens=cu)
    gr = lib.delta_chunk_bwd(q, k, v, g, beta, do, initial_state=s0, cu_seqlens=cu, d_final_state=dst)
    gp = lib.qk_norm_rope_bwd(**a, dq_out=gr["dq"], dk_out=gr["dk"])
    torch.cuda.synchronize()

    x = {n: raw[n].double().requires_grad_() for n in ("q", "k", "q_weight", "k_weight")}
    y = [rows64(x[n], x[n + "_weight"], "l2", None, raw["rope"], raw["positions"], False) for n in ("q", "k")]
    # the values the rule saw, with the gradient of the unrounded ones
    y = [t + (r.cpu().double() - t).detach() for t, r in zip(y, (q, k))]
    leaf = {n: d[n].double().requires_grad_() for n in ("v", "g", "beta", "initial_state")}
    outs, states = [], []
    for n in range(2):
        S = leaf["initial_state"][n]
        for t in range([0, 70][n], [70, 90][n]):
            qt, kt = (z[t].repeat_interleave(HV // H, 0) for z in y)
            S = S * leaf["g"][t].exp()[:, None, None]
            u = leaf["beta"][t][:, None] * (leaf["v"][t] - (S * kt[..., None]).sum(1))
            S = S + kt[..., None] * u[:, None]
            outs.append(K ** -0.5 * (S * qt[..., None]).sum(1))
        states.append(S)
    o64, s64 = torch.stack(outs), torch.stack(states)
    close("out", out, o64.detach(), F32_REL)
    close("state", state, s64.detach(), F32_REL)
    ((o64 * d["d_out"].double()).sum() + (s64 * d["d_final_state"].double()).sum()).backward()
    half = torch.finfo(io).eps / 2
    for n in ("v", "g", "beta"):
        close("d" + n, gr["d" + n], leaf[n].grad, 3e-5)
    close("d_initial_state", gr["d_initial_state"], leaf["initial_state"].grad, F32_REL)
    for n in ("q", "k"):
        # the norm's map has norm at most 1 / |x|: the rounding of dq reaches dx relative to |dq|, not to
        # its projection, so it is compared with that
        scale = float(gr["d" + n].double().norm() / raw[n].double().norm(dim=-1).min())
        err = float((gp["d" + n].cpu().double() - x[n].grad).norm())
        wmax = float(raw[n + "_weight"].abs().max())
        assert err <= 2 * half * wmax * scale, (n, err, scale)
        wg = x[n + "_weight"].grad
        err = float((gp[f"d{n}_weight"].cpu().double() - wg).norm())
        assert err <= 2 * half * float(gr["d" + n].double().norm()), (n, err)


@pytest.mark.parametrize("T,H,HK,K,io,inter", [(9001, 3, 2, 64, BF16, False), (4100, 2, 7, 128, F16, True)])
def test_more_tokens_than_waves(lib, T, H, HK, K, io, inter):
    """Waves that walk over several tokens, odd head counts, weights' gradients over thousands of rows."""
    d = inputs(T, H, HK, K, io, F32, 32, seed=T)
    a = gpu(d, ARGS)
    y = lib.qk_norm_rope(**a, norm="rms", interleaved=inter)
    g = lib.qk_norm_rope_bwd(**a, dq_out=d["dq_out"].cuda(), dk_out=d["dk_out"].cuda(), norm="rms", interleaved=inter)
    for i, n in enumerate(("q", "k")):
        x, w = d[n].double().requires_grad_(), d[n + "_weight"].double().requires_grad_()
        r = rows64(x, w, "rms", None, d["rope"], d["positions"], inter)
        close(n, y[i], r.detach(), REL)
        r.backward(d[f"d{n}_out"].double())
        close("d" + n, g["d" + n], x.grad, REL)
        close(f"d{n}_weight", g[f"d{n}_weight"], w.grad, DW_REL)


@pytest.mark.parametrize("inter", [False, True])
def test_columns_that_are_not_turned(lib, inter):
    """Infinities and NaN in columns behind the turned ones stay where they are, in both directions."""
    d = inputs(9, 2, 2, 64, BF16, None, 32, seed=4)
    clean = lib.qk_norm_rope(**gpu(d, ARGS), norm="none", interleaved=inter)
    d["q"][3, 1, 40], d["k"][5, 0, 63], d["q"][0, 0, 32] = float("inf"), float("nan"), float("-inf")
    got = lib.qk_norm_rope(**gpu(d, ARGS), norm="none", interleaved=inter)
    back = lib.qk_norm_rope_bwd(**gpu(d, ARGS), dq_out=d["q"].cuda(), dk_out=d["k"].cuda(), norm="none", interleaved=inter)
    for i, n in enumerate(("q", "k")):
        odd = ~torch.isfinite(d[n])
        assert torch.equal(~torch.isfinite(got[i].cpu()), odd) and torch.equal(~torch.isfinite(back["d" + n].cpu()), odd)
        assert torch.equal(got[i].cpu()[~odd], clean[i].cpu()[~odd])
        assert torch.equal(torch.nan_to_num(got[i].cpu()[odd].float()), torch.nan_to_num(d[n][odd].float()))
