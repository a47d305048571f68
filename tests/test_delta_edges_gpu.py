"""GPU tests of the scalar-gated delta rule at its edges: how bf16 outputs
round, state resets written as the lowest value, and the variants that only
large batches take (tolerances of float32 results: see tests/delta_ref.py)."""

import numpy as np
import pytest
import torch

from tests.delta_ref import F32_REL, backward64, close, forward64, make
from tests.test_delta_gpu import BF16, F16, F32, check_fwd, check_grads, fwd, grads, lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,HV,K,V", [([600], 2, 2, 128, 128), ([333, 500], 1, 3, 64, 64), ([2400], 2, 2, 128, 64)])
def test_bf16_outputs_are_rounded_without_bias(lib, lens, H, HV, K, V):
    """A bf16 output is off by its own rounding and by those of S, P and U (one fp16 part each, to nearest).

    Rounding to nearest leaves an error that is uniform over a step: with significands in [1, 2) its root mean square
    is at most 2^-7 / sqrt(12) of the value for bf16, and 2^-10 / sqrt(12) for each factor in fp16, two of which meet
    in P U. Of independent errors the projection on the result is their size over the square root of their number:
    five times that is allowed. (Cut off towards zero, an fp16 factor is half of 2^-10 times 2/3 to 3/4 too small, all
    outputs alike: 3.5e-4.)"""
    d = make(lens, H, HV, K, V, seed=71, beta_max=1.0)
    out, _ = fwd(lib, d)
    ref = forward64(d)[0]
    err = out.cpu().double().numpy() - ref
    rms = np.sqrt(2.0 ** -14 / 12 + 2 * 2.0 ** -20 / 12)
    size, bias = np.linalg.norm(err) / np.linalg.norm(ref), (err * ref).sum() / (ref * ref).sum()
    allowed = 5 * rms / ref.size ** 0.5
    print(f"rel-L2 {size:.3e} (allowed {rms:.3e}), bias {bias:.2e} (allowed {allowed:.2e})", flush=True)
    assert size <= rms and abs(bias) <= allowed


RESETS = [(F32, -1e6), (F32, -1e10), (F32, -1e12), (F32, -1e15), (F32, torch.finfo(F32).min), (BF16, torch.finfo(BF16).min),
          (F16, torch.finfo(F16).min)]


def with_resets(value, gtype, D, seed):
    """Single tokens that forget everything: inside chunks, at their ends, two in a row, at a sequence's start and end."""
    d = make([150, 70, 40], 1, 2, D, D, seed=seed, gtype=gtype, beta_max=1.0)
    for t, head in ((20, 0), (63, 0), (64, 0), (65, 0), (100, 0), (30, 1), (149, 1), (150, 0), (190, 1), (225, 0), (226, 0), (259, 0)):
        d["g"][t, head] = value
    return d


@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("gtype,value", RESETS)
def test_resets(lib, recurrent, gtype, value):
    """Tokens after a reset see nothing before it, and each other as if it were not there."""
    d = with_resets(value, gtype, 128, 72)
    check_fwd(f"{value}", fwd(lib, d, recurrent), forward64(d))


@pytest.mark.parametrize("gtype,value", RESETS)
def test_reset_gradients(lib, gtype, value):
    d = with_resets(value, gtype, 64, 73)
    check_grads(f"{value}", grads(lib, d), backward64(d))


def ragged(n, seed, longest):
    """n lengths up to `longest`, a quarter of them chunk borders, single tokens and empty sequences."""
    rng = np.random.default_rng(seed)
    return [int(rng.choice([0, 1, 63, 64, 65, 128])) if i % 4 == 1 else int(rng.integers(1, longest + 1)) for i in range(n)]


# (sequences, q/k heads, value heads): 64 columns of the state per workgroup with 65 to 256 chains of 128 columns, 128
# with more; batches whose chains are dealt to the XCDs (N H a multiple of 8) and ones that are not, beyond 64 sequences too
MANY = [(64, 1, 2), (45, 2, 4), (136, 1, 2), (130, 1, 2), (60, 2, 6)]


@pytest.mark.parametrize("N,H,HV", MANY)
@pytest.mark.parametrize("io", [BF16, F16])
def test_many_chains(lib, N, H, HV, io):
    d = make(ragged(N, N, 140), H, HV, 128, 128, seed=N + HV, io=io, beta_max=1.0)
    check_fwd("many", fwd(lib, d), forward64(d))
    check_grads("many", grads(lib, d), backward64(d))


@pytest.mark.parametrize("N,H,HV,K,V", [(136, 1, 2, 64, 128), (130, 1, 2, 128, 64), (64, 1, 2, 64, 128), (300, 1, 1, 64, 64)])
@pytest.mark.parametrize("io", [BF16, F16])
def test_many_chains_of_mixed_sizes(lib, N, H, HV, K, V, io):
    d = make(ragged(N, N + 1, 100), H, HV, K, V, seed=N + K, io=io, beta_max=1.0)
    check_fwd("many", fwd(lib, d), forward64(d))


@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("io", [BF16, F16])
def test_l2norm_of_128(lib, recurrent, io):
    """In-kernel norms of 128-element rows of any size, zero rows among them."""
    d = make([100, 3, 64], 2, 4, 128, 128, seed=74, io=io)
    d["q"] = (d["q"].float() * 5.0).to(io)
    d["k"] = (d["k"].float() * torch.linspace(0.1, 9.0, 167)[:, None, None]).to(io)
    d["k"][17, 1] = 0
    d["q"][101] = 0
    check_fwd("l2norm", fwd(lib, d, recurrent, qk_l2norm=True), forward64(d, qk_l2norm=True))


def segments(lib, T, N, HV, D):
    """The segments of each sequence of a call with K = V = D, from what its workspace holds for them."""
    items = (T // 64 + N) * HV
    more = lib.delta_chunk_bwd_workspace(T, N, HV, HV, D, D) - items * (26880 + 8 * D * D + 514 * D)
    return 1 + more // (N * HV * 3 * D * D * 4)


@pytest.mark.parametrize("lens,H,HV,D,io,least", [
    ([16500], 1, 1, 64, BF16, 32), ([16500], 1, 1, 128, F16, 32), ([8000, 9000], 1, 2, 64, F16, 16), ([3000], 1, 4, 128, BF16, 4)])
def test_split_of_many_segments(lib, lens, H, HV, D, io, least):
    """Split runs of this head size, up to the most segments there are: forward and gradients."""
    assert segments(lib, sum(lens), len(lens), HV, D) >= least
    d = make(lens, H, HV, D, D, seed=75, io=io, beta_max=1.0)
    check_fwd("split", fwd(lib, d), forward64(d))
    check_grads("split", grads(lib, d), backward64(d))


@pytest.mark.parametrize("layout", ["kv", "vk"])
def test_split_run_with_bf16_states(lib, layout):
    assert segments(lib, 2400, 1, 2, 64) > 1
    d = make([2400], 1, 2, 64, 64, seed=76, beta_max=1.0)
    d["initial_state"] = d["initial_state"].to(BF16)
    ref = forward64(dict(d, initial_state=d["initial_state"].float()))
    if layout == "vk":
        d["initial_state"] = d["initial_state"].transpose(2, 3).contiguous()
    fin = torch.empty_like(d["initial_state"], device="cuda")
    out, fin = fwd(lib, d, final_state=fin, state_layout=layout)
    close("out", out, ref[0], F32_REL)
    close("state", fin.transpose(2, 3) if layout == "vk" else fin, ref[1], F32_REL)


@pytest.mark.parametrize("io", [BF16, F16])
def test_one_long_sequence_among_short_ones(lib, io):
    d = make([64] * 20 + [9000] + [7, 0, 65] * 10, 1, 2, 128, 128, seed=77, io=io, beta_max=1.0)
    check_fwd("unlike", fwd(lib, d), forward64(d))
    check_grads("unlike", grads(lib, d), backward64(d))


def test_far_offsets_against_float64(lib):
    """655360 tokens of 32 heads, workspaces of several 2^32 bytes: the last head of the last sequence."""
    N, L, H, K = 8, 81920, 32, 64
    gen = torch.Generator(device="cuda").manual_seed(78)

    def unit():
        x = torch.randn((N * L, H, K), generator=gen, device="cuda", dtype=F32)
        return (x / x.norm(dim=-1, keepdim=True)).to(BF16)

    a = dict(q=unit(), k=unit(), v=unit(), g=-0.1 * torch.rand((N * L, H), generator=gen, device="cuda"),
             beta=torch.rand((N * L, H), generator=gen, device="cuda").to(BF16))
    do = unit()
    cu = torch.arange(0, N * L + 1, L, device="cuda", dtype=torch.int32)
    one = {n: x[-L:, -1:].cpu() for n, x in dict(a, d_out=do).items()}
    one.update(initial_state=None, d_final_state=None, cu_seqlens=torch.tensor([0, L], dtype=torch.int32))
    out, fin = lib.delta_chunk_fwd(**a, cu_seqlens=cu)
    check_fwd("far", (out[-L:, -1:], fin[-1:, -1:]), forward64(one))
    del out
    got = lib.delta_chunk_bwd(**a, d_out=do, cu_seqlens=cu)
    check_grads("far", {n: x[-1:, -1:] if n == "d_initial_state" else x[-L:, -1:] for n, x in got.items()}, backward64(one))


@pytest.mark.parametrize("K,V", [(16, 16), (8, 64), (96, 96), (64, 128)])
def test_unsupported_head_sizes_are_refused(lib, K, V):
    """Head sizes that the gradients do not take, the smallest too, are refused by the library."""
    q, v, g = torch.zeros(9, 2, K, dtype=BF16, device="cuda"), torch.zeros(9, 2, V, dtype=BF16, device="cuda"), torch.zeros(9, 2, device="cuda")
    with pytest.raises(lib.Gdn2Error) as e:
        lib.delta_chunk_bwd(q, q.clone(), v, g, g.to(BF16), v.clone())
    assert e.value.status == "UNSUPPORTED"
    if (K, V) == (64, 128):
        return
    for call in (lib.delta_chunk_fwd, lib.delta_recurrent_fwd):
        with pytest.raises(lib.Gdn2Error) as e:
            call(q, q.clone(), v)
        assert e.value.status == "UNSUPPORTED"
