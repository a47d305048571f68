"""Inputs and float64 references of the scalar-gated delta rule's tests.

The reference is the channel-wise oracle at the scalar rule's point: g and
beta constant over a head's channels and w = beta (FlashInfer
``chunk_gated_delta_rule2`` docs, the reduction to the scalar rule). Gradients
follow by the chain rule: dg is the sum of the channels' dg, dbeta the sum of
the channels' dbeta plus the sum of dw.

Tolerances. A value rounded once to a 16-bit type is off by at most
finfo.eps / 2 relative. Before that rounding, the kernels' products take
float32 operands in two fp16 parts, each cut off below its 11 bits: a part
leaves out at most 2^-10 of what it stands for, the pair 2^-20 of the operand,
and the product of the two low parts, 2^-20 of the product, is dropped. A
product of two such operands is off by up to 3 * 2^-20, and by sqrt(3) * 2^-20
in the 2-norm when the errors are independent. Five products follow each
other from the inputs to a float32 result: sqrt(15) * 2^-20 = 3.7e-6, and
F32_REL = 4e-6 is asked. dg multiplies two such chains (S and dS): 2^0.5 times
that, DG_REL = 6e-6. On single elements the same error is relative to the sum
of the terms' magnitudes, about sqrt(128) times a typical value: ELEMENT = 5 *
3 * 2^-20 * sqrt(128) = 1.6e-4 of the largest value. A forward output of bf16
takes the state, P and U in one part rounded to nearest, 2^-12 of each: up to
2^-11 = 4.9e-4 of the largest value more, ELEMENT16 = 6.5e-4.
"""

import numpy as np
import torch

F32_REL = 4e-6
DG_REL = 6e-6
ELEMENT = 1.6e-4
ELEMENT16 = 6.5e-4


def make(lens, H, HV, K, V, seed, io=torch.bfloat16, gtype=torch.float32, init=True, beta_max=2.0, strong=False):
    """CPU tensors of one packed batch (unit-norm q and k rows, decays spread
    over the heads; ``strong``: single tokens that decay by e^-30)."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def unit(shape):
        x = torch.randn(shape, generator=gen)
        return (x / x.norm(dim=-1, keepdim=True)).to(io)

    rate = torch.exp(-6.0 * torch.rand(HV, generator=gen))
    g = -rate * torch.rand(T, HV, generator=gen)
    if strong and T:
        g[torch.rand(T, HV, generator=gen) < 0.1] = -30.0
    d = dict(q=unit((T, H, K)), k=unit((T, H, K)), v=torch.randn((T, HV, V), generator=gen).to(io), g=g.to(gtype),
             beta=(beta_max * torch.rand(T, HV, generator=gen)).to(io),
             initial_state=0.3 * torch.randn((N, HV, K, V), generator=gen) if init else None,
             cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
    d["d_out"] = torch.randn((T, HV, V), generator=gen).to(io)
    d["d_final_state"] = torch.randn((N, HV, K, V), generator=gen)
    return d


def channelwise(d):
    """The channel-wise oracle's arguments for the scalar rule's inputs."""
    T, HV, V = d["v"].shape
    K = d["q"].shape[2]
    g = torch.zeros(T, HV) if d.get("g") is None else d["g"]
    beta = torch.ones(T, HV) if d.get("beta") is None else d["beta"]
    return dict(q=d["q"], k=d["k"], v=d["v"], g=g.double()[..., None].expand(T, HV, K).contiguous(),
                beta=beta.double()[..., None].expand(T, HV, K).contiguous(),
                w=beta.double()[..., None].expand(T, HV, V).contiguous())


def forward64(d, scale=None, qk_l2norm=False):
    from oracle.c_oracle import gdn2_recurrence_c
    a = channelwise(d)
    return gdn2_recurrence_c(a["q"], a["k"], a["v"], a["g"], a["beta"], a["w"], scale, d["initial_state"], d["cu_seqlens"],
                             qk_l2norm=qk_l2norm)


def backward64(d, scale=None):
    from oracle.c_oracle import gdn2_recurrence_bwd_c
    a = channelwise(d)
    r = gdn2_recurrence_bwd_c(a["q"], a["k"], a["v"], a["g"], a["beta"], a["w"], scale, d["initial_state"], d["cu_seqlens"],
                              d["d_out"], d["d_final_state"])
    return {"dq": r["dq"], "dk": r["dk"], "dv": r["dv"], "dg": r["dg"].sum(-1),
            "dbeta": r["dbeta"].sum(-1) + r["dw"].sum(-1), "d_initial_state": r["d_initial_state"]}


def close(tag, x, ref, rel):
    """x against the float64 reference: `rel` in the 2-norm and ELEMENT (of a
    bf16 result ELEMENT16) on single elements, plus half a step of x's type
    where it has 16 bits."""
    element = ELEMENT16 if x.dtype == torch.bfloat16 else ELEMENT
    half = torch.finfo(x.dtype).eps / 2 if x.dtype != torch.float32 else 0.0
    a, r = x.detach().cpu().double().numpy(), np.asarray(ref, dtype=np.float64)
    assert a.shape == r.shape, f"{tag}: {a.shape} {r.shape}"
    if not r.size:
        return
    assert np.isfinite(a).all(), f"{tag}: not finite"
    norm, err = np.linalg.norm(r), np.abs(a - r)
    got = np.linalg.norm(err) / norm if norm > 0 else np.linalg.norm(err)
    worst = (err - half * np.abs(r)).max() / max(np.abs(r).max(), 1e-30)
    print(f"{tag}: rel-L2 {got:.2e} (allowed {rel + half:.2e}), element {worst:.2e}", flush=True)
    assert got <= rel + half and worst <= element, f"{tag}: rel-L2 {got:.3e}, element {worst:.3e}"
