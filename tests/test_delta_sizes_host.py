"""CPU tests of the sizes that the scalar-gated delta rule's and the q/k
preparation's entries take: workspaces of refused sizes, and the launch limits
(descriptors alone: the checks read no memory)."""

import ctypes

import pytest
import torch

from tests.test_delta_host import gdn2  # noqa: F401


@pytest.mark.parametrize("args", [
    (130, 2, 2, 4, 16, 16), (130, 2, 2, 4, 1, 1), (130, 2, 2, 4, 96, 96), (130, 2, 2, 4, 64, 128), (130, 2, 3, 4, 64, 64),
    (130, 2, 2, 4, 1 << 30, 1 << 30), (64, 1 << 20, 1, 1 << 18, 1 << 27, 1 << 27), (1 << 31, 1, 1, 1, 64, 64),
    (1 << 62, 1, 1, 1, 64, 64), (64, (1 << 31) - 1, 1, (1 << 31) - 1, 64, 64), (64, 1, 1, 1 << 18, 64, 64), (130, -1, 2, 4, 64, 64)])
def test_no_backward_workspace_for_refused_sizes(gdn2, args):
    """(Head sizes under 32 divided by zero here and ended the process.)"""
    assert gdn2.delta_chunk_bwd_workspace(*args) == 0


@pytest.mark.parametrize("args", [(1 << 31, 1, 1), (1 << 62, 1, 1), (64, (1 << 31) - 1, (1 << 31) - 1), (64, 5592405, 2), (64, -1, 2)])
def test_no_forward_workspace_for_refused_sizes(gdn2, args):
    assert gdn2.delta_chunk_fwd_workspace(*args) == 0


def test_no_preparation_workspace_for_refused_sizes(gdn2):
    for args in ((9, 2, 2, 32), (1 << 31, 2, 2, 64), (9, (1 << 31) - 1, (1 << 31) - 1, 64)):
        assert gdn2.qk_norm_rope_bwd_workspace(*args) == 0


def segments(mod, T, N, HV, D):
    """The segments of each sequence of a call with K = V = D, from what its workspace holds for them."""
    items = (T // 64 + N) * HV
    more = mod.delta_chunk_bwd_workspace(T, N, HV, HV, D, D) - items * (26880 + 8 * D * D + 514 * D)
    return 1 + more // (N * HV * 3 * D * D * 4)


@pytest.mark.parametrize("T,N,HV,D,want", [
    (1535, 1, 1, 64, 1), (1536, 1, 1, 64, 3), (1536, 1, 8, 128, 3), (4096, 1, 16, 128, 5), (16500, 1, 1, 64, 32),
    # no more than three segments are resident at once
    (1536, 1, 32, 128, 1), (2047, 1, 32, 128, 1), (2048, 1, 32, 128, 3), (8192, 1, 32, 128, 3), (4095, 2, 16, 128, 1),
    (4096, 2, 16, 128, 3), (1 << 20, 1, 65, 128, 1)])
def test_split_rule(gdn2, T, N, HV, D, want):
    """Sequences are split where that was measured faster."""
    assert segments(gdn2, T, N, HV, D) == want


def tensor(mod, at, dtype, *shape):
    """The descriptor of a dense tensor at an address of its own (`at` times 2^44), which nothing reads."""
    d = mod.Gdn2Tensor()
    d.data, d.dtype, d.ndim = (at + 1) << 44, mod._DTYPES[dtype], len(shape)
    step = 1
    for i in reversed(range(len(shape))):
        d.shape[i], d.stride[i] = shape[i], step
        step *= shape[i]
    return ctypes.addressof(d), d


def rule_status(mod, entry, T, H, HV, D, io=torch.bfloat16):
    qk, v, gates = (T, H, D), (T, HV, D), (T, HV)
    shapes = {"fwd": [qk, qk, v, None, None], "bwd": [qk, qk, v, gates, gates, v, qk, qk, v, gates, gates]}
    ds = [None if s is None else tensor(mod, i, io, *s) for i, s in enumerate(shapes["bwd" if entry == "bwd" else "fwd"])]
    a = [None if d is None else d[0] for d in ds]
    lib = mod.load_library()
    if entry == "bwd":
        rc = lib.gdn2_delta_chunk_bwd_check(*a[:5], 0.0, None, None, a[5], None, *a[6:], None)
    else:
        out = tensor(mod, 30, io, *v)
        fn = lib.gdn2_delta_recurrent_fwd_check if entry == "recurrent" else lib.gdn2_delta_chunk_fwd_check
        rc = fn(*a, 0.0, None, None, out[0], None, None)
    return mod.STATUS[rc]


@pytest.mark.parametrize("entry", ["fwd", "recurrent", "bwd"])
@pytest.mark.parametrize("HV", [1, 32])
def test_chunk_limit(gdn2, entry, HV):
    """Chunks times value heads, 768 threads each: 5592405 are one launch, one chunk more is refused."""
    T = (5592405 // HV - 1) * 64 + 63  # the last token of the last chunk that fits
    assert rule_status(gdn2, entry, T, HV, HV, 64) == "OK"
    assert rule_status(gdn2, entry, T + 1, HV, HV, 64) == "SHAPE"


@pytest.mark.parametrize("D", [64, 128])
def test_row_limit_of_the_backward(gdn2, D):
    """64 tokens' rows of the value heads are addressed with 32 bits."""
    HV = (1 << 24) // D
    assert rule_status(gdn2, "bwd", 5, 1, HV - 1, D) == "OK"
    assert rule_status(gdn2, "bwd", 5, 1, HV, D) == "SHAPE"


def test_token_limit(gdn2):
    for entry in ("fwd", "recurrent", "bwd"):
        assert rule_status(gdn2, entry, 1 << 31, 1, 1, 64) == "SHAPE"
