"""GPU tests of the scalar-gated delta rule at its edges: how bf16 outputs
round (tolerances of float32 results: see tests/delta_ref.py)."""

import numpy as np
import pytest

from tests.delta_ref import forward64, make
from tests.test_delta_gpu import fwd, lib  # noqa: F401

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
