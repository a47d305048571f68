"""GPU tests of the scalar-gated delta rule at its edges: how bf16 outputs
round, and state resets written as the lowest value (tolerances of float32
results: see tests/delta_ref.py)."""

import numpy as np
import pytest
import torch

from tests.delta_ref import backward64, forward64, make
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
