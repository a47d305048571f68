"""GPU tests of the gated linear recurrence, its gradients and its token step
against float64 token by token (tolerances: tests/mixer_ref.py)."""

import pytest
import torch

from tests.mixer_ref import (BF16, DG_REL, F16, F32, SCAN_ARGS, SCAN_REL, close, cu_of, gpu, scan64, scan64_grads,
                             scan_inputs)
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu

# lengths: one token, odd ones, tiles of 64 just missed, empty sequences at both ends and between, one long one,
# more sequences than one look-up holds (64), and batches that run as groups of whole sequences
LENS = {"one": [1], "single": [333], "tile": [64], "ragged": [63, 0, 65, 1, 128, 7], "empty": [0, 0, 5, 0], "long": [1500],
        "tiles": [600, 0, 1, 300, 64], "many": [(7 * i) % 5 for i in range(150)], "pairs": [3] * 300}


@pytest.mark.parametrize("lens,D,io,gtype,kind,w,init,cu", [
    ("one", 1, BF16, F32, "unit", True, True, torch.int32),
    ("single", 3, F32, F32, "none", False, False, None),
    ("single", 130, F16, F16, "convex", True, True, torch.int64),
    ("tile", 65, BF16, BF16, "unit", True, False, torch.int32),
    ("ragged", 64, F16, F32, "unit", True, True, torch.int64),
    ("ragged", 200, F32, F32, "convex", True, True, torch.int32),
    ("empty", 66, BF16, F32, "none", True, True, torch.int32),
    ("empty", 2, F32, F32, "unit", False, False, torch.int32),
    ("long", 70, BF16, F32, "unit", True, True, None),
    ("long", 33, F32, F32, "none", False, True, torch.int32),
    ("tiles", 128, F16, F32, "convex", False, True, torch.int32),
    ("tiles", 129, BF16, BF16, "none", True, False, torch.int64),
    ("many", 96, F32, F32, "unit", True, True, torch.int32),
    ("pairs", 64, BF16, F32, "convex", True, True, torch.int32)])
def test_forward_step_and_backward(lib, lens, D, io, gtype, kind, w, init, cu):
    lens = LENS[lens]
    d = scan_inputs(lens, D, seed=len(lens) + D, io=io, gtype=gtype, w=w, init=init, cu=cu)
    a = gpu(d, SCAN_ARGS)
    out, end = lib.linear_scan_fwd(**a, input_scale=kind)
    step, send = lib.linear_scan_recurrent_fwd(**a, input_scale=kind)
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"],
                            cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), input_scale=kind)
    torch.cuda.synchronize()
    ro, re = scan64(d, kind)
    for tag, o, e in (("scan", out, end), ("step", step, send)):
        close(tag + " out", o, ro, SCAN_REL)
        close(tag + " final_state", e, re, SCAN_REL)
    r = scan64_grads(d, kind)
    assert (g["dw"] is None) == (not w)
    for n in r:
        assert g[n].dtype == {"dx": io, "dw": io, "dg": gtype, "d_initial_state": F32}[n]
        close(n, g[n], r[n], DG_REL if n == "dg" else SCAN_REL)


@pytest.mark.parametrize("lens,D", [([(11 * i + 3) % 37 for i in range(300)], 64), ([(11 * i + 3) % 37 for i in range(40)], 4096),
                                    ([70, 300, 0, 300, 1, 129], 4096), ([65 + 2 * (i * i % 40) for i in range(64)], 96),
                                    ([65 + 2 * (i * i % 40) for i in range(65)], 96)])
def test_groups_of_sequences(lib, lens, D):
    """Batches that run whole: several sequences (empty ones among them) per group, and each its own group, by length, equal and
    empty ones too, as many as one look-up holds and one more."""
    N = len(lens)
    assert lib.linear_scan_fwd_workspace(sum(lens), N, D) == 0
    d = scan_inputs(lens, D, seed=N, io=F32)
    out, end = lib.linear_scan_fwd(**gpu(d, SCAN_ARGS), input_scale="unit")
    ro, re = scan64(d, "unit")
    close("out", out, ro, SCAN_REL)
    close("final_state", end, re, SCAN_REL)


@pytest.mark.parametrize("lens,D", [([19200 + 17], 3), ([7000, 1, 0, 9000, 3000], 3), ([1300, 900], 2100), ([2000], 33)])
def test_two_passes(lib, lens, D):
    """Few long sequences: chunks of 8 and more tokens per wave, more tiles than one pass of the join holds, both widths of the
    join (up to 2048 channels and beyond)."""
    d = scan_inputs(lens, D, seed=1, io=F32, lowest=0.1)
    a = gpu(d, SCAN_ARGS)
    assert lib.linear_scan_fwd_workspace(sum(lens), len(lens), D) > 0
    out, end = lib.linear_scan_fwd(**a, input_scale="convex")
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"],
                            cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), input_scale="convex")
    ro, re = scan64(d, "convex")
    close("out", out, ro, SCAN_REL)
    close("final_state", end, re, SCAN_REL)
    for n, r in scan64_grads(d, "convex").items():
        close(n, g[n], r, DG_REL if n == "dg" else SCAN_REL)


def test_slow_decays(lib):
    """g = -1e-5 over 6000 tokens: e^g rounded to float32 would be off by up to 2^-25 per step, 9e-5 over half the length. The
    state's roundings are independent, sqrt(6000 / 3) * sqrt(2) * 2^-24 = 3.8e-6."""
    T = 6000
    d = scan_inputs([T], 64, seed=2, io=F32, w=False)
    d["g"] = torch.full((T, 64), -1e-5) * (1 + torch.arange(64) / 64)
    d["x"] = d["x"].abs()
    for call in (lib.linear_scan_fwd, lib.linear_scan_recurrent_fwd):
        out, end = call(**gpu(d, SCAN_ARGS))
        ro, re = scan64(d, "none")
        close("out", out, ro, 4e-6)
        close("final_state", end, re, 4e-6)


@pytest.mark.parametrize("gtype", [F32, BF16, F16])
@pytest.mark.parametrize("kind", ["none", "convex", "unit"])
def test_forgetting(lib, gtype, kind):
    """g of minus infinity and of the type's lowest value forget the state: what follows is as from a zero state, gradients are
    finite and zero for what was forgotten."""
    T, D, cut = 200, 66, 77
    d = scan_inputs([T], D, seed=3, io=F16 if gtype == F16 else BF16, gtype=gtype)
    d["g"][cut] = float("-inf")
    d["g"][cut + 50] = torch.finfo(gtype).min
    d["g"][cut + 51] = torch.finfo(gtype).min
    a = gpu(d, SCAN_ARGS)
    ref = dict(d, g=d["g"].double().clamp_min(-1e4))  # e^-10000 is 0 in float64
    out, end = lib.linear_scan_fwd(**a, input_scale=kind)
    step, _ = lib.linear_scan_recurrent_fwd(**a, input_scale=kind)
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"],
                            cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), input_scale=kind)
    ro, re = scan64(ref, kind)
    close("out", out, ro, SCAN_REL)
    close("step", step, ro, SCAN_REL)
    close("final_state", end, re, SCAN_REL)
    for n, r in scan64_grads(ref, kind).items():
        close(n, g[n], r, DG_REL if n == "dg" else SCAN_REL)
    assert (g["dg"][cut] == 0).all()


def test_no_decay_at_all(lib):
    """g = 0 (and -0): the sum of the inputs; with "convex" and "unit" nothing enters, and the infinite slope of the second is 0."""
    d = scan_inputs([150, 90], 64, seed=4, io=F32)
    d["g"] = torch.zeros_like(d["g"])
    d["g"][::2] = -0.0
    a = gpu(d, SCAN_ARGS)
    for kind in ("none", "convex", "unit"):
        out, end = lib.linear_scan_fwd(**a, input_scale=kind)
        g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"],
                                cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), input_scale=kind)
        ro, re = scan64(d, kind)
        close("out", out, ro, SCAN_REL)
        close("final_state", end, re, SCAN_REL)
        if kind == "unit":
            assert (g["dx"] == 0).all() and (g["dw"] == 0).all() and torch.isfinite(g["dg"]).all()
        else:
            for n, r in scan64_grads(d, kind).items():
                close(n, g[n], r, DG_REL if n == "dg" else SCAN_REL)


def test_gradient_against_differences(lib):
    """The kernels' own loss moved by small steps: central differences of a float32 loss summed in float64. With steps of 2^-6 the
    third derivative (of order 1 here) leaves 2^-12 / 6 = 4e-5 and the outputs' roundings 2^-24 / 2^-6 * sqrt(terms): 2e-3 is asked."""
    d = scan_inputs([90, 40], 8, seed=5, io=F32)
    a = gpu(d, SCAN_ARGS)
    do, de = d["d_out"].cuda().double(), d["d_final_state"].cuda().double()
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"],
                            cu_seqlens=a["cu_seqlens"], d_final_state=d["d_final_state"].cuda(), input_scale="unit")

    def loss(b):
        out, end = lib.linear_scan_fwd(**b, input_scale="unit")
        return float((out.double() * do).sum() + (end.double() * de).sum())

    gen = torch.Generator().manual_seed(6)
    for name, key in (("x", "dx"), ("g", "dg"), ("w", "dw"), ("initial_state", "d_initial_state")):
        v = torch.randn(a[name].shape, generator=gen).cuda()
        if name == "g":
            v = v * a["g"].abs()  # stays negative
        h = 2.0 ** -6
        up, down = (loss(dict(a, **{name: a[name] + s * h * v})) for s in (1, -1))
        want = float((g[key].double() * v.double()).sum())
        scale = float((g[key].double().norm() * v.double().norm()))
        print(name, (up - down) / (2 * h), want, scale)
        assert abs((up - down) / (2 * h) - want) <= 2e-3 * scale


@pytest.mark.parametrize("D", [96, 97])
def test_strided_rows_and_guards(lib, D):
    """Inputs and outputs as views of wider tensors at odd and even offsets; what lies beside them stays."""
    lens = [100, 0, 61, 500]
    T = sum(lens)
    d = scan_inputs(lens, D, seed=7)
    a = gpu(d, SCAN_ARGS)
    do, de = d["d_out"].cuda(), d["d_final_state"].cuda()
    want = lib.linear_scan_fwd(**a, input_scale="unit")
    wantb = lib.linear_scan_bwd(a["x"], a["g"], a["w"], do, initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                                d_final_state=de, input_scale="unit")
    for off in (1, 2):
        fused = torch.zeros(T, 3 * D + 8, dtype=BF16, device="cuda")
        x, w = fused[:, off:off + D], fused[:, D + off + 1:2 * D + off + 1]
        x.copy_(a["x"]), w.copy_(a["w"])
        room = torch.full((T, D + 6), 7.0, dtype=BF16, device="cuda")
        out, end = lib.linear_scan_fwd(x, a["g"], w, initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                                       input_scale="unit", out=room[:, off:off + D])
        assert torch.equal(out, want[0]) and torch.equal(end, want[1])
        assert (room[:, :off] == 7).all() and (room[:, off + D:] == 7).all()
        room.fill_(7.0)
        step, _ = lib.linear_scan_recurrent_fwd(x, a["g"], w, initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                                                input_scale="unit", out=room[:, off:off + D])
        assert (step.float() - want[0].float()).norm() <= 2 ** -7 * want[0].float().norm()
        assert (room[:, :off] == 7).all() and (room[:, off + D:] == 7).all()
        rooms = {n: torch.full((T, D + 6), 7.0, dtype=F32 if n == "dg" else BF16, device="cuda") for n in ("dx", "dg", "dw")}
        gb = lib.linear_scan_bwd(x, a["g"], w, do, initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"], d_final_state=de,
                                 input_scale="unit", grads={n: t[:, off:off + D] for n, t in rooms.items()})
        assert all(torch.equal(gb[n], wantb[n]) for n in wantb)
        assert all((t[:, :off] == 7).all() and (t[:, off + D:] == 7).all() for t in rooms.values())
    # one row of gates for every token
    row = a["w"][:1]
    x1 = lib.linear_scan_fwd(**dict(a, w=row.expand(T, D)))
    x2 = lib.linear_scan_fwd(**dict(a, w=row.expand(T, D).contiguous()))
    assert torch.equal(x1[0], x2[0])


@pytest.mark.parametrize("D", [64, 7])
def test_tokens_behind_the_last_sequence(lib, D):
    lens, pad = [90, 0, 600], 150
    d = scan_inputs(lens + [pad], D, seed=8)
    T = sum(lens)
    ref = dict(d, lens=lens, cu_seqlens=cu_of(lens), **{n: d[n][:T] for n in ("x", "g", "w", "d_out")},
               **{n: d[n][:3] for n in ("initial_state", "d_final_state")})
    for n in ("x", "g", "w", "d_out"):
        d[n][T:] = float("nan")
    a = gpu(dict(d, cu_seqlens=ref["cu_seqlens"], initial_state=ref["initial_state"]), SCAN_ARGS)
    ro, re = scan64(ref, "unit")
    for call in (lib.linear_scan_fwd, lib.linear_scan_recurrent_fwd):
        room = torch.full((T + pad, D), 7.0, dtype=BF16, device="cuda")
        out, end = call(**a, input_scale="unit", out=room)
        close("out", out[:T], ro, SCAN_REL)
        close("final_state", end, re, SCAN_REL)
        assert (room[T:] == 7).all()
    rooms = {n: torch.full((T + pad, D), 7.0, dtype=F32 if n == "dg" else BF16, device="cuda") for n in ("dx", "dg", "dw")}
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), initial_state=a["initial_state"], cu_seqlens=a["cu_seqlens"],
                            d_final_state=ref["d_final_state"].cuda(), input_scale="unit", grads=rooms)
    for n, r in scan64_grads(ref, "unit").items():
        close(n, g[n][:T] if n in rooms else g[n], r, DG_REL if n == "dg" else SCAN_REL)
    assert all((t[T:] == 7).all() for t in rooms.values())


@pytest.mark.parametrize("N", [3, 300])
def test_infinities_stay_in_their_sequence_and_channel(lib, N):
    """In batches that run as tiles and as groups."""
    lens = [(13 * i) % 9 + 200 // N for i in range(N)] if N > 3 else [300, 200, 130]
    d = scan_inputs(lens, 64, seed=9)
    bad = dict(d, **{n: d[n].clone() for n in ("x", "g", "w", "d_out", "initial_state")})
    s, ch = N // 2, 5
    b, e = int(d["cu_seqlens"][s]), int(d["cu_seqlens"][s + 1])
    bad["x"][b], bad["g"][e - 1, ch], bad["d_out"][(b + e) // 2, ch] = float("inf"), float("nan"), float("nan")
    bad["x"][b, :ch], bad["x"][b, ch + 1:] = d["x"][b, :ch], d["x"][b, ch + 1:]
    res = []
    for v in (d, bad):
        a = gpu(v, SCAN_ARGS)
        f = lib.linear_scan_fwd(**a, input_scale="unit")
        g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], v["d_out"].cuda(), initial_state=a["initial_state"],
                                cu_seqlens=a["cu_seqlens"], d_final_state=v["d_final_state"].cuda(), input_scale="unit")
        res.append(((f[0], g["dx"], g["dg"], g["dw"]), (f[1], g["d_initial_state"])))
    for x, y in zip(res[0][0], res[1][0]):
        x, y = x.clone(), y.clone()
        assert not torch.isfinite(y[b:e, ch]).all()
        x[b:e, ch] = y[b:e, ch] = 0
        assert torch.equal(x, y)
    for x, y in zip(res[0][1], res[1][1]):
        x, y = x.clone(), y.clone()
        x[s, ch] = y[s, ch] = 0
        assert torch.equal(x, y)


@pytest.mark.parametrize("state", [F32, BF16])
@pytest.mark.parametrize("D", [130, 33])
def test_step_in_place_and_16_bit_states(lib, state, D):
    lens = [1, 0, 3, 1, 1, 8]
    d = scan_inputs(lens, D, seed=10)
    d["initial_state"] = d["initial_state"].to(state)
    a = gpu(d, SCAN_ARGS)
    ro, re = scan64(d, "unit")
    for call in (lib.linear_scan_fwd, lib.linear_scan_recurrent_fwd):
        out, end = call(**a, input_scale="unit", final_state=torch.empty_like(a["initial_state"]))
        close("out", out, ro, SCAN_REL)
        close("final_state", end, re, SCAN_REL)
    held = a["initial_state"].clone()
    out2, end2 = lib.linear_scan_recurrent_fwd(**dict(a, initial_state=held), input_scale="unit", final_state=held)
    assert end2 is held and torch.equal(out2, out) and torch.equal(held, end)


def test_prefill_then_decode(lib):
    """A sequence cut at any place gives what it gives whole."""
    d = scan_inputs([700], 64, seed=11, io=F32)
    a = gpu(d, SCAN_ARGS)
    out, end = lib.linear_scan_fwd(**a, input_scale="unit")
    for cut in (1, 64, 650):
        part = {n: a[n][:cut] for n in ("x", "g", "w")}
        rest = {n: a[n][cut:] for n in ("x", "g", "w")}
        o1, s1 = lib.linear_scan_fwd(**part, initial_state=a["initial_state"], input_scale="unit")
        o2, s2 = lib.linear_scan_recurrent_fwd(**rest, initial_state=s1, input_scale="unit")
        close("out", torch.cat([o1, o2]), out.double(), 2 * SCAN_REL)
        close("final_state", s2, end.double(), 2 * SCAN_REL)


def test_no_tokens(lib):
    d = scan_inputs([0, 0], 70, seed=12)
    a = gpu(d, SCAN_ARGS)
    for call in (lib.linear_scan_fwd, lib.linear_scan_recurrent_fwd):
        out, end = call(**a)
        assert out.shape == (0, 70) and torch.equal(end, a["initial_state"])
        assert (call(**dict(a, initial_state=None))[1] == 0).all()
    g = lib.linear_scan_bwd(a["x"], a["g"], a["w"], d["d_out"].cuda(), cu_seqlens=a["cu_seqlens"],
                            d_final_state=d["d_final_state"].cuda())
    assert torch.equal(g["d_initial_state"].cpu(), d["d_final_state"])
    one = {n: a[n] for n in ("x", "g", "w")}
    out, end = lib.linear_scan_fwd(**one, initial_state=a["initial_state"][:1])
    assert torch.equal(end, a["initial_state"][:1])
    g = lib.linear_scan_bwd(one["x"], one["g"], one["w"], d["d_out"].cuda())
    assert (g["d_initial_state"] == 0).all()


def test_graphs_streams_and_repeated_calls(lib):
    """Two captured graphs, replayed with other inputs between eager calls on another stream, give the eager bits."""
    ds = [scan_inputs([500, 0, 400], 64, seed=s) for s in (13, 14)]
    names = SCAN_ARGS + ("d_out", "d_final_state")
    ins = [gpu(d, names) for d in ds]

    def call(x):
        f = lib.linear_scan_fwd(**{n: x[n] for n in SCAN_ARGS}, input_scale="unit")
        b = lib.linear_scan_bwd(x["x"], x["g"], x["w"], x["d_out"], initial_state=x["initial_state"], cu_seqlens=x["cu_seqlens"],
                                d_final_state=x["d_final_state"], input_scale="unit")
        return list(f) + [b[n] for n in sorted(b)]

    want = [call(x) for x in ins]
    assert all(torch.equal(x, y) for x, y in zip(want[0], call(ins[0])))
    side = torch.cuda.Stream()
    graphs = []
    for x in ins:
        static = {n: t.clone() for n, t in x.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(static)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(static)
        graphs.append((graph, static, got))
    for i in range(4):
        for k, (graph, static, got) in enumerate(graphs):
            for n in static:
                static[n].copy_(ins[(i + k) % 2][n])
        side.wait_stream(torch.cuda.current_stream())
        for graph, _, _ in graphs:
            graph.replay()
        with torch.cuda.stream(side):
            eager = call(ins[i % 2])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(eager, want[i % 2]))
        for k, (_, _, got) in enumerate(graphs):
            assert all(torch.equal(x, y) for x, y in zip(got, want[(i + k) % 2]))


def test_far_offsets(lib):
    """A sequence behind 2^31 elements gives what it gives alone."""
    D, near, far = 4096, 2 ** 19 + 100, 90
    gen = torch.Generator(device="cuda").manual_seed(15)
    x = torch.randn(near + far, D, generator=gen, device="cuda", dtype=BF16)
    g = -torch.rand(near + far, D, generator=gen, device="cuda", dtype=BF16)
    cu = cu_of([near, far]).cuda()
    alone, end = lib.linear_scan_fwd(x[near:], g[near:], input_scale="unit")
    both, ends = lib.linear_scan_fwd(x, g, cu_seqlens=cu, input_scale="unit")
    short = cu_of([512] * 1024 + [100, far]).cuda()
    step, _ = lib.linear_scan_recurrent_fwd(x, g, cu_seqlens=short, input_scale="unit")
    close("out", both[near:], alone.double(), SCAN_REL + 2 ** -8)
    close("step", step[near:], alone.double(), SCAN_REL + 2 ** -8)
    close("final_state", ends[1:], end.double(), SCAN_REL)
    del both, step
    want = lib.linear_scan_bwd(x[near:], g[near:], None, x[near:], input_scale="unit")
    got = lib.linear_scan_bwd(x, g, None, x, cu_seqlens=cu, input_scale="unit")
    for n in ("dx", "dg"):
        close(n, got[n][near:], want[n].double(), DG_REL + 2 ** -8)
    close("d_initial_state", got["d_initial_state"][1:], want["d_initial_state"].double(), SCAN_REL)
