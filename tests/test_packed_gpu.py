"""GPU tests of packed batches with more sequences than the 64 that a wave
looks up at once: equal lengths, multiples of the 8 tokens of one load, one-token
and empty ones beside a long one. References in float64 on the GPU, tolerances
from tests/mixer_ref.py (sums over all tokens: 256 and fewer in one register, a
workgroup's four, then up to a hundred workgroups': 2.7e-7, and 1e-7 for the
rest, next to the terms' own CONV_REL, so SUM_REL holds)."""

import pytest
import torch

from tests.mixer_ref import BF16, CONV_REL, F32, SCAN_REL, SUM_REL, conv64, conv64_grads, cu_of, factor64
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu


def near(tag, x, ref, rel):
    """mixer_ref's measure of the 2-norm, on the GPU: these tensors are large."""
    assert x.shape == ref.shape and torch.isfinite(x).all(), tag
    half = torch.finfo(x.dtype).eps / 2 if x.dtype != F32 else 0.0
    err = float((x.double() - ref).norm() / ref.norm())
    print(f"{tag}: rel-L2 {err:.2e} (allowed {rel + half:.2e})", flush=True)
    assert err <= rel + half, f"{tag}: rel-L2 {err:.3e}"


def inputs(lens, D, seed, io):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, N = sum(lens), len(lens)
    rate = 0.02 * torch.exp(torch.rand(D, generator=gen, device="cuda") * 4.6)
    return dict(x=torch.randn(T, D, generator=gen, device="cuda").to(io),
                g=-rate * (0.5 + torch.rand(T, D, generator=gen, device="cuda")),
                w=torch.rand(T, D, generator=gen, device="cuda").to(io),
                initial_state=torch.randn(N, D, generator=gen, device="cuda"), cu_seqlens=cu_of(lens).cuda())


def scan64_doubling(a, lens, kind):
    """h_t = e^g h_{t-1} + u by doubling spans, each sequence's first token with its initial state in u and no decay."""
    decay, u = a["g"].double().exp(), factor64(kind, a["g"].double()) * (a["w"].double() * a["x"].double())
    cu, full = a["cu_seqlens"].long(), torch.tensor(lens, device="cuda") > 0
    first, last = cu[:-1][full], cu[1:][full] - 1
    u[first] += decay[first] * a["initial_state"].double()[full]
    decay[first] = 0.0
    span = 1
    while span < max(lens):
        u[span:] = u[span:] + decay[span:] * u[:-span]
        decay[span:] = decay[span:] * decay[:-span]
        span *= 2
    end = a["initial_state"].double().clone()
    end[full] = u[last]
    return u, end


EIGHTS = [8 * ((7 * i) % 12 + 1) for i in range(1024)]
TINY = [(5 * i) % 4 for i in range(2000)]
MIXED = [20] * 12 + [1] * 64 + [8] * 51 + [16384]
EDGES = [1] * 16 + [0] * 47 + [16] + [3, 0, 1] * 40 + [16500]
LONG = [2, 0, 1] * 21 + [1] + [3, 0, 1] * 25 + [2 ** 20] + [1] * 30


@pytest.mark.parametrize("lens,D,two_passes", [
    ([64] * 1000, 4096, False), (EIGHTS, 4096, False), (TINY, 4096, False), ([8] * 65 + [100], 4096, False),
    (LONG, 8, True)])
def test_recurrence(lib, lens, D, two_passes):
    a = inputs(lens, D, len(lens), F32)
    assert (lib.linear_scan_fwd_workspace(sum(lens), len(lens), D) > 0) == two_passes
    room = torch.full((len(lens), D), float("nan"), device="cuda")
    out, end = lib.linear_scan_fwd(**a, input_scale="unit", final_state=room)
    ro, re = scan64_doubling(a, lens, "unit")
    near("out", out, ro, SCAN_REL)
    near("final_state", end, re, SCAN_REL)


@pytest.mark.parametrize("lens,D", [(MIXED, 4032), (EDGES, 4032), ([1, 0] * 2100, 4096)])
def test_convolution_and_its_gradients(lib, lens, D):
    a = inputs(lens, D, len(lens), BF16)
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, N, K = sum(lens), len(lens), 4

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    d = dict(x=a["x"], weight=0.6 * normal(D, K), bias=0.3 * normal(D), initial_state=normal(N, K - 1, D).to(BF16),
             cu_seqlens=a["cu_seqlens"], lens=lens, d_out=normal(T, D).to(BF16), d_final_state=normal(N, K - 1, D).to(BF16))
    args = [d[n] for n in ("x", "weight", "bias")]
    kw = {n: d[n] for n in ("initial_state", "cu_seqlens")}
    out, end = lib.short_conv_fwd(*args, **kw, final_state=torch.full((N, K - 1, D), float("nan"), dtype=BF16, device="cuda"))
    ro, re = conv64(d, "silu")
    near("out", out, ro, CONV_REL)
    assert torch.equal(end.double(), re)
    del ro, re
    dx = torch.full((T, D), float("nan"), dtype=BF16, device="cuda")
    g = lib.short_conv_bwd(*args, d["d_out"], **kw, d_final_state=d["d_final_state"], grads={"dx": dx})
    for n, r in conv64_grads(d, "silu").items():
        near(n, g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)
