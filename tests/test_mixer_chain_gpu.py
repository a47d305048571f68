"""GPU tests of the operators of a token mixer run one after the other, as a
block uses them, forward and backward."""

import pytest
import torch

from tests.delta_ref import F32_REL
from tests.delta_ref import close as close_delta
from tests.mixer_ref import (BF16, CONV_REL, NORM_DX_REL, NORM_REL, SUM_REL, close, conv64, conv64_grads, conv_inputs, cu_of,
                             norm64, norm64_grads, scan64)
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu


def test_norm_convolution_recurrence_gated_norm(lib):
    """A recurrent block in float32, both directions, against float64 autograd of the whole.

    Each operator leaves at most 3e-6 (mixer_ref) and its map of the error before it is bounded: the norms' by 1 / 2 times the
    weight's 2 (rows of spread 2), the convolution's by the taps' sum (under 4), the recurrence's by 1 / (1 - a) (under 64, but for
    random errors sqrt of that). Norms of outputs grow alike, so relative errors add up: 4 operators there and 4 back, 2.4e-5 at
    most, and 2e-5 is asked."""
    rel = 2e-5
    lens, D = [150, 0, 1, 90, 400], 96
    T, N = sum(lens), len(lens)
    gen = torch.Generator().manual_seed(1)

    def normal(*s):
        return torch.randn(s, generator=gen)

    p = dict(x=2 * normal(T, D) + 0.5, nw=1 + 0.3 * normal(D), nb=0.3 * normal(D), cw=0.5 * normal(D, 4), cb=0.2 * normal(D),
             cs=normal(N, 3, D), g=-0.02 - torch.rand(T, D, generator=gen), w=torch.rand(T, D, generator=gen), s=normal(N, D),
             ow=1 + 0.3 * normal(D), z=normal(T, D))
    cu, dy = cu_of(lens), normal(T, D)
    a = {n: t.cuda() for n, t in p.items()}
    cug = cu.cuda()
    h1 = lib.layer_norm(a["x"], a["nw"], a["nb"])
    h2, _ = lib.short_conv_fwd(h1, a["cw"], a["cb"], initial_state=a["cs"], cu_seqlens=cug)
    h3, s3 = lib.linear_scan_fwd(h2, a["g"], a["w"], initial_state=a["s"], cu_seqlens=cug, input_scale="unit")
    y = lib.layer_norm(h3, a["ow"], gate=a["z"], norm="rms")
    g4 = lib.layer_norm_bwd(h3, dy.cuda(), a["ow"], gate=a["z"], norm="rms")
    g3 = lib.linear_scan_bwd(h2, a["g"], a["w"], g4["dx"], initial_state=a["s"], cu_seqlens=cug, input_scale="unit")
    g2 = lib.short_conv_bwd(h1, a["cw"], a["cb"], g3["dx"], initial_state=a["cs"], cu_seqlens=cug)
    g1 = lib.layer_norm_bwd(a["x"], g2["dx"], a["nw"], a["nb"])

    q = {n: t.double().requires_grad_() for n, t in p.items()}
    r1 = norm64(dict(x=q["x"], weight=q["nw"], bias=q["nb"], gate=None), "layer")
    r2, _ = conv64(dict(x=r1, weight=q["cw"], bias=q["cb"], initial_state=q["cs"], lens=lens), "silu")
    r3, _ = scan64(dict(x=r2, g=q["g"], w=q["w"], initial_state=q["s"], lens=lens), "unit")
    r4 = norm64(dict(x=r3, weight=q["ow"], bias=None, gate=q["z"]), "rms")
    r4.backward(dy.double())
    close("y", y, r4, rel)
    for n, t in (("x", g1["dx"]), ("nw", g1["dweight"]), ("nb", g1["dbias"]), ("cw", g2["dweight"]), ("cb", g2["dbias"]),
                 ("cs", g2["d_initial_state"]), ("g", g3["dg"]), ("w", g3["dw"]), ("s", g3["d_initial_state"]),
                 ("ow", g4["dweight"]), ("z", g4["dgate"])):
        close("d" + n, t, q[n].grad, rel)


def test_convolution_delta_rule_gated_norm(lib):
    """q, k and v of one convolution as views of one tensor, the q/k norm, the delta rule and the gated norm of its heads, in
    bf16, with all gradients; each stage against float64 of the tensors that it was given."""
    lens, H, HV, K, V = [130, 3, 200], 2, 4, 64, 64
    T, N, D = sum(lens), len(lens), (2 * H + HV) * 64
    d = conv_inputs(lens, D, 4, seed=2)
    gen = torch.Generator().manual_seed(3)
    g, beta = -torch.rand(T, HV, generator=gen), torch.rand(T, HV, generator=gen).to(BF16)
    z, w, dy = (torch.randn(T, HV, V, generator=gen).to(BF16), 1 + 0.3 * torch.randn(V, generator=gen),
                torch.randn(T, HV, V, generator=gen).to(BF16))
    cu = d["cu_seqlens"].cuda()
    cw, cb, cs = d["weight"].cuda(), d["bias"].cuda(), d["initial_state"].cuda()
    x, gg, bb, zz, ww = d["x"].cuda(), g.cuda(), beta.cuda(), z.cuda(), w.cuda()
    y1, s1 = lib.short_conv_fwd(x, cw, cb, initial_state=cs, cu_seqlens=cu)
    ro, re = conv64(d, "silu")
    close("conv", y1, ro, CONV_REL)
    q, k, v = (y1[:, b:e].unflatten(1, (-1, 64)) for b, e in ((0, H * 64), (H * 64, 2 * H * 64), (2 * H * 64, D)))
    qn, kn = lib.qk_norm_rope(q, k)
    o, s = lib.delta_chunk_fwd(qn, kn, v, gg, bb, cu_seqlens=cu)
    y = lib.layer_norm(o, ww, gate=zz, norm="rms")
    nd = dict(x=o.cpu(), weight=w, bias=None, gate=z, d_out=dy)
    close("y", y, norm64(nd, "rms"), NORM_REL)

    gn = lib.layer_norm_bwd(o, dy.cuda(), ww, gate=zz, norm="rms")
    for n, r in norm64_grads(nd, "rms").items():
        close(n, gn[n], r, SUM_REL if n == "dweight" else NORM_DX_REL)
    vd = v.contiguous()
    gr = lib.delta_chunk_bwd(qn, kn, vd, gg, bb, gn["dx"], cu_seqlens=cu)
    dq = lib.qk_norm_rope_bwd(q, k, gr["dq"], gr["dk"])
    dy1 = torch.cat([dq["dq"].flatten(1), dq["dk"].flatten(1), gr["dv"].flatten(1)], 1)
    gc = lib.short_conv_bwd(x, cw, cb, dy1, initial_state=cs, cu_seqlens=cu)
    for n, r in conv64_grads(dict(d, d_out=dy1.cpu(), d_final_state=None), "silu").items():
        close(n, gc[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)

    # the rule between them, on the convolution's own rows
    from tests.delta_ref import forward64
    ro, rs = forward64(dict(q=qn.cpu(), k=kn.cpu(), v=vd.cpu(), g=g, beta=beta, initial_state=None, cu_seqlens=d["cu_seqlens"]))
    close_delta("rule", o, ro, F32_REL)
    close_delta("rule's state", s, rs, F32_REL)

    # decode goes on from the prefill's states, the convolution's in place
    xt = torch.randn(N, D, generator=gen).to(BF16).cuda()
    ct = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    held = s1.clone()
    t1, t2 = lib.short_conv_recurrent_fwd(xt, cw, cb, initial_state=held, cu_seqlens=ct, final_state=held)
    ends = cu.long()[1:]
    for n in range(N):
        whole, _ = lib.short_conv_fwd(torch.cat([x[cu[n]:ends[n]], xt[n:n + 1]]), cw, cb, initial_state=cs[n:n + 1])
        assert torch.equal(whole[-1], t1[n])
    assert torch.equal(t2[:, -1], xt)


def test_two_threads_on_two_streams(lib):
    """Calls of two host threads at once, each on its own stream, give the bits of the calls alone."""
    import threading

    from tests.mixer_ref import norm_inputs, scan_inputs

    def make(seed):
        s, c, n = scan_inputs([700, 0, 300], 130, seed), conv_inputs([700, 0, 300], 130, 4, seed), norm_inputs(500, 2, 130, seed)
        return [{k: t.cuda() if torch.is_tensor(t) else t for k, t in d.items()} for d in (s, c, n)]

    def calls(ins):
        s, c, n = ins
        kw = dict(initial_state=s["initial_state"], cu_seqlens=s["cu_seqlens"])
        out = list(lib.linear_scan_fwd(s["x"], s["g"], s["w"], input_scale="unit", **kw))
        g = lib.linear_scan_bwd(s["x"], s["g"], s["w"], s["d_out"], d_final_state=s["d_final_state"], input_scale="unit", **kw)
        out += [g[k] for k in sorted(g)]
        g = lib.short_conv_bwd(c["x"], c["weight"], c["bias"], c["d_out"], initial_state=c["initial_state"], cu_seqlens=c["cu_seqlens"])
        out += [g[k] for k in sorted(g)]
        g = lib.layer_norm_bwd(n["x"], n["d_out"], n["weight"], n["bias"], gate=n["gate"])
        return out + [g[k] for k in sorted(g)]

    ins = [make(5), make(6)]
    want = [calls(i) for i in ins]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[k] = calls(ins[k])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for k in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[k], want[k]))
