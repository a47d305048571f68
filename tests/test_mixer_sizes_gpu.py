"""GPU tests of the recurrence and the convolution at the slices, chunks and
numbers of partial sums that large calls run, against float64 on the GPU.

How long a slice or a chunk is goes by the call's size and shows in its
workspace, which every test compares first. Tolerances from tests/mixer_ref.py;
the weights' sums: up to 256 terms one after the other leave 0.4 sqrt(256 / 2)
2^-24 = 2.7e-7 of their size, up to 150 workgroups' sums in 16 runs and a tree
under 0.4 sqrt(26) 2^-24 = 1.2e-7, and each term is off by CONV_REL at most,
independently: SUM_REL = 3e-6 holds."""

import pytest
import torch

from tests.mixer_ref import BF16, CONV_REL, F16, F32, SCAN_REL, SUM_REL, conv64, conv64_grads, cu_of
from tests.test_delta_gpu import lib  # noqa: F401
from tests.test_packed_gpu import inputs, near, scan64_doubling

pytestmark = pytest.mark.gpu


def up(n):
    return (n + 255) // 256 * 256


# sequences that end inside, at and just behind slices, short and empty ones between long ones
def cut(T, short=(1, 0, 7, 64, 2, 0, 300, 33, 3, 3)):
    short = list(short)
    left = T - sum(short)
    half = len(short) // 2
    return [left // 2 - 5] + short[:half] + [left // 4] + short[half:] + [left - left // 2 + 5 - left // 4]


@pytest.mark.parametrize("T,D,K,io,slice_tokens", [
    (9500, 64, 4, F32, 16), (9500, 65, 3, BF16, 16), (17003, 512, 4, F32, 32), (34001, 512, 2, F16, 64), (34005, 1024, 4, BF16, 128),
    (34005, 1985, 4, F32, 256)])
def test_convolution_slices(lib, T, D, K, io, slice_tokens):
    lens = cut(T)
    N, slices = len(lens), -(-T // (4 * slice_tokens))
    assert sum(lens) == T and min(lens) >= 0
    assert lib.short_conv_bwd_workspace(T, D, K) == up(slices * (K + 1) * D * 4)
    assert slice_tokens > 16 or slices > 128  # (the partial sums' second round)
    gen = torch.Generator(device="cuda").manual_seed(T + D)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    d = dict(x=normal(T, D).to(io), weight=0.6 * normal(D, K), bias=0.3 * normal(D), initial_state=normal(N, K - 1, D).to(io),
             cu_seqlens=cu_of(lens).cuda(), lens=lens, d_out=normal(T, D).to(io), d_final_state=normal(N, K - 1, D).to(io))
    args, kw = [d[n] for n in ("x", "weight", "bias")], {n: d[n] for n in ("initial_state", "cu_seqlens")}
    out, end = lib.short_conv_fwd(*args, **kw)
    ro, re = conv64(d, "silu")
    near("out", out, ro, CONV_REL)
    assert torch.equal(end.double(), re)
    g = lib.short_conv_bwd(*args, d["d_out"], **kw, d_final_state=d["d_final_state"])
    for n, r in conv64_grads(d, "silu").items():
        near(n, g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)


@pytest.mark.parametrize("T,D,io,chunk,short", [
    (16500, 512, F32, 16, None), (33005, 512, BF16, 32, None), (65111, 512, F32, 56, None), (65606, 1023, F16, 128, (1, 9)),
    (131171, 1024, BF16, 256, (1, 9)), (131171, 2050, F32, 256, ())])
def test_recurrence_chunks(lib, T, D, io, chunk, short):
    lens = cut(T) if short is None else cut(T, short)
    ranges = -(-T // (8 * chunk))
    assert lib.linear_scan_fwd_workspace(T, len(lens), D) == 2 * up(ranges * D * 4) + 2 * up(8 * ranges * D * 4)
    a = inputs(lens, D, T, io)
    for kind in ("none", "unit"):
        out, end = lib.linear_scan_fwd(**a, input_scale=kind)
        ro, re = scan64_doubling(a, lens, kind)
        near("out", out, ro, SCAN_REL)
        near("final_state", end, re, SCAN_REL)
