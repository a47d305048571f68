"""GPU tests of the short causal convolution, its gradients and its token step
against float64 (tolerances: tests/mixer_ref.py)."""

import pytest
import torch

from tests.mixer_ref import (BF16, CONV_ARGS, CONV_REL, F16, F32, SUM_REL, close, conv64, conv64_grads, conv_inputs, cu_of,
                             gpu)
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu

# lengths under, at and just over the taps, the 8 tokens of one load, the 32 and 128 of a wave and a workgroup; empty sequences
LENS = {"one": [1], "short": [1, 2, 3, 4, 0, 2, 1, 5], "single": [333], "edges": [32, 31, 33, 0, 128, 127, 1, 129],
        "empty": [0, 0, 5, 0], "many": [(7 * i) % 5 for i in range(200)], "long": [1500, 700]}


def backward(lib, a, d, act, **kw):
    return lib.short_conv_bwd(a["x"], a["weight"], a["bias"], d["d_out"].cuda(), initial_state=a["initial_state"],
                              cu_seqlens=a["cu_seqlens"],
                              d_final_state=None if d["d_final_state"] is None else d["d_final_state"].cuda(), activation=act, **kw)


@pytest.mark.parametrize("lens,D,K,io,wtype,act,bias,init,cu", [
    ("one", 1, 4, BF16, None, "silu", True, True, torch.int32),
    ("one", 64, 2, F32, None, "none", False, False, None),
    ("short", 66, 4, F32, None, "silu", True, True, torch.int32),
    ("short", 67, 3, F16, F32, "none", True, True, torch.int64),
    ("short", 130, 4, BF16, BF16, "silu", False, False, torch.int32),
    ("short", 5, 2, F32, None, "silu", True, True, torch.int32),
    ("single", 129, 4, F16, None, "silu", True, True, None),
    ("edges", 64, 4, BF16, F32, "silu", True, True, torch.int32),
    ("edges", 200, 3, F32, None, "none", False, True, torch.int64),
    ("empty", 70, 4, F32, None, "silu", True, True, torch.int32),
    ("many", 96, 4, F32, None, "silu", True, True, torch.int32),
    ("many", 3, 2, BF16, None, "none", True, False, torch.int32),
    ("long", 257, 4, BF16, None, "silu", True, True, torch.int32),
    ("long", 128, 4, F32, None, "silu", False, False, torch.int32)])
def test_forward_step_and_backward(lib, lens, D, K, io, wtype, act, bias, init, cu):
    d = conv_inputs(LENS[lens], D, K, seed=D + K, io=io, wtype=wtype, bias=bias, init=init, cu=cu)
    a = gpu(d, CONV_ARGS)
    out, end = lib.short_conv_fwd(**a, activation=act)
    step, send = lib.short_conv_recurrent_fwd(**a, activation=act)
    g = backward(lib, a, d, act)
    torch.cuda.synchronize()
    ro, re = conv64(d, act)
    close("out", out, ro, CONV_REL)
    assert torch.equal(end.cpu().double(), re) and torch.equal(send, end)
    close("step", step, ro, CONV_REL)
    assert (g["dbias"] is None) == (not bias)
    for n, r in conv64_grads(d, act).items():
        assert g[n].dtype == (io if n in ("dx", "d_initial_state") else wtype or io)
        close(n, g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)


def test_without_some_gradients(lib):
    """No final state's gradient, no gradient of the initial state, only one of the weights' sums."""
    d = conv_inputs(LENS["edges"], 64, 4, seed=1, io=F32)
    d["d_final_state"] = None
    a = gpu(d, CONV_ARGS)
    g = backward(lib, a, d, "silu", need_d_initial_state=False)
    assert g["d_initial_state"] is None
    for n, r in conv64_grads(d, "silu").items():
        if g[n] is not None:
            close(n, g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)


def test_gradient_against_differences(lib):
    """Central differences of the kernels' own loss, steps of 2^-6: the third derivatives leave 2^-12 / 6 times their size (order
    1), the outputs' roundings 2^-18 * sqrt(terms): 2e-3 is asked."""
    d = conv_inputs([60, 2, 40], 8, 4, seed=2, io=F32)
    a = gpu(d, CONV_ARGS)
    do, de = d["d_out"].cuda().double(), d["d_final_state"].cuda().double()
    g = backward(lib, a, d, "silu")

    def loss(b):
        out, end = lib.short_conv_fwd(**b)
        return float((out.double() * do).sum() + (end.double() * de).sum())

    gen = torch.Generator().manual_seed(3)
    for name in ("x", "weight", "bias", "initial_state"):
        v, h = torch.randn(a[name].shape, generator=gen).cuda(), 2.0 ** -6
        up, down = (loss(dict(a, **{name: a[name] + s * h * v})) for s in (1, -1))
        t = g[("d_" if name == "initial_state" else "d") + name].double()
        assert abs((up - down) / (2 * h) - float((t * v.double()).sum())) <= 2e-3 * float(t.norm() * v.double().norm())


@pytest.mark.parametrize("D", [96, 97])
def test_strided_rows_and_guards(lib, D):
    lens = [100, 0, 61, 300]
    T = sum(lens)
    d = conv_inputs(lens, D, 4, seed=4)
    a = gpu(d, CONV_ARGS)
    do = d["d_out"].cuda()
    want, wantb = lib.short_conv_fwd(**a), backward(lib, a, d, "silu")
    for off in (1, 2):
        fused = torch.zeros(T, 2 * D + 8, dtype=BF16, device="cuda")
        x, dy = fused[:, off:off + D], fused[:, D + off + 1:2 * D + off + 1]
        x.copy_(a["x"]), dy.copy_(do)
        for call in (lib.short_conv_fwd, lib.short_conv_recurrent_fwd):
            room = torch.full((T, D + 6), 7.0, dtype=BF16, device="cuda")
            out, end = call(**dict(a, x=x), out=room[:, off:off + D])
            assert torch.equal(out, want[0]) and torch.equal(end, want[1])
            assert (room[:, :off] == 7).all() and (room[:, off + D:] == 7).all()
        room.fill_(7.0)
        g = lib.short_conv_bwd(x, a["weight"], a["bias"], dy, initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                               d_final_state=d["d_final_state"].cuda(), grads={"dx": room[:, off:off + D]})
        assert all(torch.equal(g[n], wantb[n]) for n in ("dx", "d_initial_state"))
        for n in ("dweight", "dbias"):
            close(n, g[n], wantb[n].double(), 2 ** -8)
        assert (room[:, :off] == 7).all() and (room[:, off + D:] == 7).all()


@pytest.mark.parametrize("D", [64, 7])
def test_tokens_behind_the_last_sequence(lib, D):
    lens, pad = [90, 0, 2, 300], 150
    d = conv_inputs(lens + [pad], D, 4, seed=5)
    T, N = sum(lens), len(lens)
    ref = dict(d, lens=lens, cu_seqlens=cu_of(lens), **{n: d[n][:T] for n in ("x", "d_out")},
               **{n: d[n][:N] for n in ("initial_state", "d_final_state")})
    for n in ("x", "d_out"):
        d[n][T:] = float("nan")
    a = gpu(dict(d, cu_seqlens=ref["cu_seqlens"], initial_state=ref["initial_state"]), CONV_ARGS)
    ro, re = conv64(ref, "silu")
    for call in (lib.short_conv_fwd, lib.short_conv_recurrent_fwd):
        room = torch.full((T + pad, D), 7.0, dtype=BF16, device="cuda")
        out, end = call(**a, out=room)
        close("out", out[:T], ro, CONV_REL)
        assert torch.equal(end.cpu().double(), re) and (room[T:] == 7).all()
    room.fill_(7.0)
    g = backward(lib, a, dict(d, d_final_state=ref["d_final_state"]), "silu", grads={"dx": room})
    for n, r in conv64_grads(ref, "silu").items():
        close(n, g[n][:T] if n == "dx" else g[n], r, SUM_REL if n in ("dweight", "dbias") else CONV_REL)
    assert (room[T:] == 7).all()


def test_infinities_stay_in_their_sequence_and_channel(lib):
    d = conv_inputs([70, 90, 40], 64, 4, seed=6)
    bad = dict(d, x=d["x"].clone(), d_out=d["d_out"].clone())
    bad["x"][70, 5], bad["x"][159, 5], bad["d_out"][100, 5] = float("inf"), float("nan"), float("inf")
    res = []
    for v in (d, bad):
        a = gpu(v, CONV_ARGS)
        f, g = lib.short_conv_fwd(**a), backward(lib, a, v, "silu")
        res.append((f[0], g["dx"], f[1], g["d_initial_state"], g["dweight"], g["dbias"]))
    for i, (x, y) in enumerate(zip(*res)):
        x, y = x.clone(), y.clone()
        at = (slice(70, 160), 5) if i < 2 else (1, slice(None), 5) if i < 4 else (5,)
        assert not torch.isfinite(y[at]).all() or i == 3
        x[at] = y[at] = 0
        assert torch.equal(x, y)


@pytest.mark.parametrize("D,K", [(130, 4), (33, 3), (64, 2)])
def test_step_in_place(lib, D, K):
    d = conv_inputs([1, 0, 3, 1, 8, 2], D, K, seed=7)
    a = gpu(d, CONV_ARGS)
    out, end = lib.short_conv_recurrent_fwd(**a)
    held = a["initial_state"].clone()
    out2, end2 = lib.short_conv_recurrent_fwd(**dict(a, initial_state=held), final_state=held)
    assert end2 is held and torch.equal(out2, out) and torch.equal(held, end)


def test_prefill_then_decode(lib):
    d = conv_inputs([300], 64, 4, seed=8)
    a = gpu(d, CONV_ARGS)
    kw = {n: a[n] for n in ("weight", "bias")}
    out, end = lib.short_conv_fwd(**a)
    for cut in (1, 2, 64, 299):
        o1, s1 = lib.short_conv_fwd(a["x"][:cut], **kw, initial_state=a["initial_state"])
        o2, s2 = lib.short_conv_recurrent_fwd(a["x"][cut:], **kw, initial_state=s1)
        assert torch.equal(torch.cat([o1, o2]), out) and torch.equal(s2, end)


def test_no_tokens(lib):
    d = conv_inputs([0, 0], 70, 4, seed=9)
    a = gpu(d, CONV_ARGS)
    for call in (lib.short_conv_fwd, lib.short_conv_recurrent_fwd):
        out, end = call(**a)
        assert out.shape == (0, 70) and torch.equal(end, a["initial_state"])
        assert (call(**dict(a, initial_state=None))[1] == 0).all()
    g = backward(lib, a, d, "silu")
    assert torch.equal(g["d_initial_state"].cpu(), d["d_final_state"]) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_graphs_streams_and_repeated_calls(lib):
    ds = [conv_inputs([500, 0, 400], 64, 4, seed=s) for s in (10, 11)]
    names = CONV_ARGS + ("d_out", "d_final_state")
    ins = [gpu(d, names) for d in ds]

    def call(x):
        f = lib.short_conv_fwd(**{n: x[n] for n in CONV_ARGS})
        b = lib.short_conv_bwd(x["x"], x["weight"], x["bias"], x["d_out"], initial_state=x["initial_state"],
                               cu_seqlens=x["cu_seqlens"], d_final_state=x["d_final_state"])
        return list(f) + [b[n] for n in sorted(b)]

    want = [call(x) for x in ins]
    side = torch.cuda.Stream()
    static = {n: t.clone() for n, t in ins[0].items()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(static)
    for i in range(4):
        for n in static:
            static[n].copy_(ins[i % 2][n])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            eager = call(ins[1 - i % 2])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want[i % 2]))
        assert all(torch.equal(x, y) for x, y in zip(eager, want[1 - i % 2]))


def test_far_offsets(lib):
    """A sequence behind 2^31 elements gives what it gives alone."""
    D, near, far = 4096, 2 ** 19 + 100, 90
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(near + far, D, generator=gen, device="cuda", dtype=BF16)
    w = torch.randn(D, 4, generator=gen, device="cuda", dtype=BF16)
    cu = cu_of([near, far]).cuda()
    alone, end = lib.short_conv_fwd(x[near:], w)
    both, ends = lib.short_conv_fwd(x, w, cu_seqlens=cu)
    step, _ = lib.short_conv_recurrent_fwd(x, w, cu_seqlens=cu_of([512] * 1024 + [100, far]).cuda())
    assert torch.equal(both[near:], alone) and torch.equal(step[near:], alone) and torch.equal(ends[1:], end)
    del both, step
    want = lib.short_conv_bwd(x[near:], w, None, x[near:])
    got = lib.short_conv_bwd(x, w, None, x, cu_seqlens=cu)
    assert torch.equal(got["dx"][near:], want["dx"]) and torch.equal(got["d_initial_state"][1:], want["d_initial_state"])
