"""GPU tests of the layer and RMS norm with weight, bias and gate, and of its
gradients, against float64 autograd (tolerances: tests/mixer_ref.py)."""

import pytest
import torch

from tests.mixer_ref import (BF16, F16, F32, NORM_ARGS, NORM_DX_REL, NORM_REL, SUM_REL, close, gpu, norm64, norm64_grads,
                             norm_inputs)
from tests.test_delta_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu


def rel_of(n):
    return SUM_REL if n in ("dweight", "dbias") else NORM_DX_REL


def run(lib, d, kind, eps=None, **kw):
    a = gpu(d, NORM_ARGS)
    y = lib.layer_norm(**a, norm=kind, eps=eps)
    g = lib.layer_norm_bwd(**a, d_out=d["d_out"].cuda(), norm=kind, eps=eps, **kw)
    torch.cuda.synchronize()
    return y, g


# widths at and around a lane's piece (4 or 8), a row's 8 to 64 lanes, two pieces per lane, and 4 to 16 waves per row
@pytest.mark.parametrize("T,H,D,io,kind,wt,bias,gate", [
    (3, 2, 1, F32, "rms", F32, True, True), (5, 1, 3, BF16, "layer", F32, True, False), (70, 3, 64, BF16, "rms", F32, False, True),
    (33, 5, 128, F16, "rms", F16, True, True), (40, 2, 100, F32, "layer", F32, True, True), (9, 1, 256, BF16, "layer", BF16, True, True),
    (17, 1, 257, F16, "layer", F32, True, False), (300, 1, 513, F32, "rms", F32, False, False),
    (11, 1, 1001, F16, "layer", F32, True, False), (7, 1, 1024, BF16, "rms", BF16, False, True),
    (6, 2, 1025, BF16, "layer", F32, True, True), (5, 1, 2048, F32, "layer", F32, True, True),
    (9, 1, 4096, BF16, "layer", F32, True, False), (5, 1, 4097, F32, "rms", F32, True, True),
    (4, 1, 8191, F16, "layer", F16, True, True), (3, 1, 8200, F32, "layer", F32, True, True),
    (3, 1, 16384, BF16, "layer", F32, True, True), (3, 1, 16384, F32, "layer", F32, True, True), (2, 1, 16383, BF16, "rms", BF16, True, False)])
def test_forward_and_backward(lib, T, H, D, io, kind, wt, bias, gate):
    d = norm_inputs(T, H, D, seed=T + D, io=io, wtype=wt, bias=bias, gate=gate)
    y, g = run(lib, d, kind)
    close("y", y, norm64(d, kind), NORM_REL)
    r = norm64_grads(d, kind)
    assert {n for n in g if g[n] is not None} == set(r)
    for n in r:
        assert g[n].dtype == (wt if n in ("dweight", "dbias") else io)
        if n == "dx" and D == 1:
            # r (m - n mean(m n)) with one element is r m (1 - n^2), 1 - n^2 = eps r^2 of 1e-6: what float32 holds of it is three
            # roundings of 2^-24 relative to r m, which is what dx is compared with (under LAYER it is 0)
            x = d["x"].double()
            m = d["d_out"].double() * d["weight"].double() * (d["gate"].double() * torch.sigmoid(d["gate"].double()) if gate else 1.0)
            size = (m / (x.square() + 1e-6).sqrt()).abs().max()
            assert float((g[n].cpu().double() - r[n]).abs().max()) <= 4 * 2.0 ** -24 * float(size)
            continue
        close(n, g[n], r[n], rel_of(n))


def test_rows_of_one_element(lib):
    d = norm_inputs(40, 1, 1, seed=20, io=F32)
    y, g = run(lib, d, "layer")
    close("y", y, norm64(d, "layer"), NORM_REL)
    assert (g["dx"] == 0).all() and (g["dweight"] == 0).all()


@pytest.mark.parametrize("weight,bias,gate", [(False, False, False), (False, True, True), (True, False, False)])
def test_without_some_arguments(lib, weight, bias, gate):
    d = norm_inputs(50, 2, 128, seed=1, io=F16, wtype=F32, btype=F16, weight=weight, bias=bias, gate=gate)
    for kind in ("layer", "rms"):
        y, g = run(lib, d, kind)
        close("y", y, norm64(d, kind), NORM_REL)
        for n, r in norm64_grads(d, kind).items():
            close(n, g[n], r, rel_of(n))


@pytest.mark.parametrize("T,H,D", [(5000, 4, 64), (3000, 1, 1000), (2100, 1, 2048)])
def test_many_rows(lib, T, H, D):
    """More rows than workgroups: sums over rows that one workgroup takes in turn."""
    d = norm_inputs(T, H, D, seed=2, io=BF16)
    y, g = run(lib, d, "layer")
    close("y", y, norm64(d, "layer"), NORM_REL)
    for n, r in norm64_grads(d, "layer").items():
        close(n, g[n], r, rel_of(n))


def test_constant_and_zero_rows(lib):
    """Rows without variance: eps alone holds them; eps given."""
    d = norm_inputs(6, 1, 200, seed=3, io=F32)
    d["x"][1], d["x"][2] = 0.0, 3.0
    for kind, eps in (("layer", None), ("rms", None), ("layer", 0.5), ("rms", 0.25)):
        y, g = run(lib, d, kind, eps)
        close("y", y, norm64(d, kind, eps), NORM_REL)
        for n, r in norm64_grads(d, kind, eps).items():
            # (at var = 0 dx is 1 / sqrt(eps) times a difference of like terms)
            close(n, g[n], r, rel_of(n))


def test_gradient_against_differences(lib):
    """Central differences of the kernel's own loss, steps of 2^-6: 2^-12 / 6 times third derivatives of order 1, and roundings of
    2^-18 * sqrt(terms): 2e-3 is asked."""
    d = norm_inputs(30, 1, 40, seed=4, io=F32)
    for kind in ("layer", "rms"):
        a = gpu(d, NORM_ARGS)
        do = d["d_out"].cuda().double()
        g = run(lib, d, kind)[1]
        gen = torch.Generator().manual_seed(5)
        for name in NORM_ARGS:
            v, h = torch.randn(a[name].shape, generator=gen).cuda(), 2.0 ** -6
            up, down = (float((lib.layer_norm(**dict(a, **{name: a[name] + s * h * v}), norm=kind).double() * do).sum()) for s in (1, -1))
            t = g["d" + name].double()
            assert abs((up - down) / (2 * h) - float((t * v.double()).sum())) <= 2e-3 * float(t.norm() * v.double().norm())


@pytest.mark.parametrize("D", [64, 65, 600])
def test_strided_rows_and_guards(lib, D):
    """Heads as views of a wider projection at odd and even offsets, token and head strides of their own, in and out."""
    T, H = 40, 3
    d = norm_inputs(T, H, D, seed=6)
    a, do = gpu(d, NORM_ARGS), d["d_out"].cuda()
    want, wantb = run(lib, d, "layer")

    def room(off, value=7.0):
        t = torch.full((T, H + 1, D + 6), value, dtype=BF16, device="cuda")
        return t, t[:, :H, off:off + D]

    for off in (1, 4):
        ins = {}
        for n, t in (("x", a["x"]), ("gate", a["gate"]), ("d_out", do)):
            ins[n] = room(off)[1]
            ins[n].copy_(t)
        outs = {n: room(off) for n in ("out", "dx", "dgate")}
        y = lib.layer_norm(ins["x"], a["weight"], a["bias"], gate=ins["gate"], out=outs["out"][1])
        g = lib.layer_norm_bwd(ins["x"], ins["d_out"], a["weight"], a["bias"], gate=ins["gate"],
                               grads={n: outs[n][1] for n in ("dx", "dgate")})
        # (a row that is no multiple of 16 bytes may be summed in another order: which elements a lane takes goes by the layout)
        close("y", y, norm64(d, "layer"), NORM_REL)
        for n, r in norm64_grads(d, "layer").items():
            close(n, g[n], r, rel_of(n))
        if D % 8 == 0:
            assert torch.equal(y, want) and all(torch.equal(g[n], wantb[n]) for n in wantb)
        for whole, view in outs.values():
            view.fill_(7.0)
            assert (whole == 7).all()
    # token-major and head-major outputs, a gate that all tokens share, rows as [T, D]
    hm = torch.empty(H, T, D, dtype=BF16, device="cuda").transpose(0, 1)
    close("y", lib.layer_norm(a["x"], a["weight"], a["bias"], gate=a["gate"], out=hm), norm64(d, "layer"), NORM_REL)
    one = a["gate"][:1].expand(T, H, D)
    close("y", lib.layer_norm(a["x"], gate=one), norm64(dict(d, weight=None, bias=None, gate=one.cpu()), "layer"), NORM_REL)
    flat = lib.layer_norm(a["x"].reshape(T * H, D), a["weight"], a["bias"], gate=a["gate"].reshape(T * H, D))
    assert torch.equal(flat.reshape(T, H, D), want)


@pytest.mark.parametrize("D,io", [(64, BF16), (65, BF16), (1004, F16), (1002, F32), (333, F32), (4095, BF16)])
def test_rows_anywhere_in_a_line(lib, D, io):
    """Rows [T, D] that begin at every place of a 16-byte line, all tensors alike or each at its own; sums over all of them."""
    T = 37
    d = norm_inputs(T, 1, D, seed=21, io=io)
    r, ry = norm64_grads(d, "layer"), norm64(d, "layer")
    w, b = d["weight"].cuda(), d["bias"].cuda()
    for pad, offs in ((5, (1, 1, 1, 1, 1)), (5, (3, 1, 0, 2, 4)), (8, (1, 1, 1, 1, 1)), (0, (0, 0, 0, 0, 0))):
        rooms = [torch.full((T, D + pad), 7.0, dtype=io, device="cuda") for _ in range(6)]
        x, z, dy, y, dx = (t[:, o:o + D] for t, o in zip(rooms, offs))
        dz = rooms[5][:, offs[1]:offs[1] + D]
        for t, n in ((x, "x"), (z, "gate"), (dy, "d_out")):
            t.copy_(d[n][:, 0])
        lib.layer_norm(x, w, b, gate=z, out=y)
        g = lib.layer_norm_bwd(x, dy, w, b, gate=z, grads={"dx": dx, "dgate": dz})
        close("y", y[:, None], ry, NORM_REL)
        for n in r:
            close(n, g[n][:, None] if n in ("dx", "dgate") else g[n], r[n], rel_of(n))
        for t in (y, dx, dz):
            t.fill_(7.0)
        assert all((t == 7).all() for t in rooms[3:])


@pytest.mark.parametrize("T,D", [(1, 1001), (3, 1001), (9, 7), (2, 15)])
def test_fewer_rows_than_places_in_a_line(lib, T, D):
    d = norm_inputs(T, 1, D, seed=22, io=BF16)
    y, g = run(lib, d, "layer")
    close("y", y, norm64(d, "layer"), NORM_REL)
    for n, r in norm64_grads(d, "layer").items():
        close(n, g[n], r, rel_of(n))


def test_infinities_stay_in_their_row(lib):
    for D in (100, 3000):
        d = norm_inputs(9, 1, D, seed=7)
        clean = run(lib, d, "layer")
        d["x"][3, 0, 7], d["x"][5, 0, 99], d["gate"][6, 0, 0] = float("inf"), float("nan"), float("-inf")
        got = run(lib, d, "layer")
        keep = torch.tensor([0, 1, 2, 4, 7, 8]).cuda()
        for x, y in ((clean[0], got[0]), (clean[1]["dx"], got[1]["dx"]), (clean[1]["dgate"], got[1]["dgate"])):
            assert torch.equal(x[keep], y[keep])


def test_no_rows(lib):
    d = norm_inputs(0, 2, 64, seed=8)
    y, g = run(lib, d, "rms")
    assert y.shape == (0, 2, 64) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_graphs_streams_and_repeated_calls(lib):
    ds = [norm_inputs(300, 2, 128, seed=s) for s in (9, 10)]
    ins = [gpu(d, NORM_ARGS + ("d_out",)) for d in ds]

    def call(x):
        b = lib.layer_norm_bwd(**x, norm="rms")
        return [lib.layer_norm(**{n: x[n] for n in NORM_ARGS}, norm="rms")] + [b[n] for n in sorted(b)]

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
    """Rows behind 2^31 elements give what they give alone."""
    D, near, far = 4096, 2 ** 19 + 10, 30
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(near + far, D, generator=gen, device="cuda", dtype=BF16)
    w = torch.rand(D, generator=gen, device="cuda")
    assert torch.equal(lib.layer_norm(x, w)[near:], lib.layer_norm(x[near:], w))
    assert torch.equal(lib.layer_norm_bwd(x, x, w)["dx"][near:], lib.layer_norm_bwd(x[near:], x[near:], w)["dx"])
