"""GPU tests of the convolution's, the recurrence's and the norm's calls at
their edges: workspaces of calls that need none, widths whose last workgroup
holds a single channel."""

import pytest
import torch

from tests.mixer_ref import (BF16, CONV_ARGS, CONV_REL, F32, NORM_ARGS, SCAN_ARGS, SUM_REL, close, conv64, conv64_grads,
                             conv_inputs, gpu, norm_inputs, scan_inputs)
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [0, 1, 256])
def test_a_workspace_that_is_not_needed_stays(lib, size):
    """Calls without tokens (and scans that run whole) ask for 0 bytes: what they are given is left as it was, whatever its size
    and alignment."""
    room = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    ws = room[4096 + size % 2:4096 + size % 2 + size]
    d = conv_inputs([0, 0], 130, 4, seed=1, io=BF16, wtype=F32)
    a = gpu(d, CONV_ARGS)
    assert lib.short_conv_bwd_workspace(0, 130, 4) == 0
    g = lib.short_conv_bwd(a["x"], a["weight"], a["bias"], d["d_out"].cuda(), initial_state=a["initial_state"],
                           cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), workspace=ws)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all() and torch.equal(g["d_initial_state"].cpu(), d["d_final_state"])
    d = norm_inputs(0, 2, 130, seed=2)
    g = lib.layer_norm_bwd(**gpu(d, NORM_ARGS), d_out=d["d_out"].cuda(), workspace=ws)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    for lens in ([0, 0], [3, 40]):
        d = scan_inputs(lens, 130, seed=3)
        a = gpu(d, SCAN_ARGS)
        assert lib.linear_scan_fwd_workspace(sum(lens), 2, 130) == lib.linear_scan_bwd_workspace(sum(lens), 2, 130) == 0
        lib.linear_scan_fwd(**a, workspace=ws)
        lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                            workspace=ws)
    torch.cuda.synchronize()
    assert (room == 7).all()


@pytest.mark.parametrize("D", [127, 129, 385, 2049])
@pytest.mark.parametrize("K", [2, 4])
def test_weight_sums_of_a_last_single_channel(lib, D, K):
    d = conv_inputs([70, 0, 3, 200], D, K, seed=D, io=F32)
    a = gpu(d, CONV_ARGS)
    out, _ = lib.short_conv_fwd(**a)
    g = lib.short_conv_bwd(a["x"], a["weight"], a["bias"], d["d_out"].cuda(), initial_state=a["initial_state"],
                           cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda())
    close("out", out, conv64(d, "silu")[0], CONV_REL)
    for n, r in conv64_grads(d, "silu").items():
        close(n, g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)
