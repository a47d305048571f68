"""CPU tests of the argument checks of the gated linear recurrence's, the short
convolution's and the layer norm's entries: the ``_check`` functions run the
validation alone, on descriptors of host memory."""

import ctypes

import pytest
import torch

from tests.test_delta_host import gdn2  # noqa: F401

BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def scan_case(T=70, D=10, N=2, io=BF16, g=F32):
    return dict(x=zeros(T, D, dtype=io), g=zeros(T, D, dtype=g), w=zeros(T, D, dtype=io), initial_state=zeros(N, D, dtype=F32),
                cu_seqlens=zeros(N + 1, dtype=I32), out=zeros(T, D, dtype=io), final_state=zeros(N, D, dtype=F32))


def scan_back(T=70, D=10, N=2, io=BF16, g=F32):
    c = scan_case(T, D, N, io, g)
    del c["out"], c["final_state"]
    return dict(c, d_out=zeros(T, D, dtype=io), d_final_state=zeros(N, D, dtype=F32),
                grads=dict(dx=zeros(T, D, dtype=io), dg=zeros(T, D, dtype=g), dw=zeros(T, D, dtype=io),
                           d_initial_state=zeros(N, D, dtype=F32)))


def conv_case(T=70, D=10, K=4, N=2, io=BF16, wt=None):
    wt = wt or io
    return dict(x=zeros(T, D, dtype=io), weight=zeros(D, K, dtype=wt), bias=zeros(D, dtype=wt),
                initial_state=zeros(N, K - 1, D, dtype=io), cu_seqlens=zeros(N + 1, dtype=I32), out=zeros(T, D, dtype=io),
                final_state=zeros(N, K - 1, D, dtype=io))


def conv_back(T=70, D=10, K=4, N=2, io=BF16, wt=None):
    c = conv_case(T, D, K, N, io, wt)
    del c["out"], c["final_state"]
    wt = wt or io
    return dict(c, d_out=zeros(T, D, dtype=io), d_final_state=zeros(N, K - 1, D, dtype=io),
                grads=dict(dx=zeros(T, D, dtype=io), dweight=zeros(D, K, dtype=wt), dbias=zeros(D, dtype=wt),
                           d_initial_state=zeros(N, K - 1, D, dtype=io)))


def norm_case(T=7, H=3, D=10, io=BF16, wt=F32):
    return dict(x=zeros(T, H, D, dtype=io), weight=zeros(D, dtype=wt), bias=zeros(D, dtype=wt), gate=zeros(T, H, D, dtype=io),
                out=zeros(T, H, D, dtype=io))


def norm_back(T=7, H=3, D=10, io=BF16, wt=F32):
    c = norm_case(T, H, D, io, wt)
    del c["out"]
    return dict(c, d_out=zeros(T, H, D, dtype=io),
                grads=dict(dx=zeros(T, H, D, dtype=io), dgate=zeros(T, H, D, dtype=io), dweight=zeros(D, dtype=wt),
                           dbias=zeros(D, dtype=wt)))


ENTRIES = {"scan": ("check_linear_scan", scan_case, {}), "scan_step": ("check_linear_scan", scan_case, {"recurrent": True}),
           "scan_bwd": ("check_linear_scan_bwd", scan_back, {}), "conv": ("check_short_conv", conv_case, {}),
           "conv_step": ("check_short_conv", conv_case, {"recurrent": True}), "conv_bwd": ("check_short_conv_bwd", conv_back, {}),
           "norm": ("check_layer_norm", norm_case, {}), "norm_bwd": ("check_layer_norm_bwd", norm_back, {})}


def status(gdn2, entry, c, **kw):
    fn, _, fixed = ENTRIES[entry]
    return gdn2.STATUS[getattr(gdn2, fn)(**c, **fixed, **kw)]


def changed(c, name, value):
    return dict(c, grads=dict(c["grads"], **{name: value})) if name in c.get("grads", {}) else dict(c, **{name: value})


def test_accepted(gdn2):
    for e, (_, make, _) in ENTRIES.items():
        for io in (BF16, F16, F32):
            for D in (1, 10, 64, 4097):
                assert status(gdn2, e, make(D=D, io=io)) == "OK", (e, io, D, gdn2.last_error())
        assert status(gdn2, e, make(T=0)) == "OK"
        c = make()
        optional = [n for n in ("w", "bias", "initial_state", "cu_seqlens", "final_state", "d_final_state", "gate", "weight")
                    if n in c and not (n == "weight" and "conv" in e)]
        for n in optional:
            b = dict(c, **{n: None})
            if n == "cu_seqlens":
                b = {k: v[:1] if k.endswith("_state") else v for k, v in b.items()}
                if "grads" in b:
                    b["grads"] = dict(b["grads"], d_initial_state=b["grads"]["d_initial_state"][:1])
            if "grads" in b and n in ("w", "bias", "gate", "weight"):
                b["grads"] = dict(b["grads"], **{"d" + n: None})
            assert status(gdn2, e, b) == "OK", (e, n, gdn2.last_error())
        if "cu_seqlens" in c:
            assert status(gdn2, e, dict(c, cu_seqlens=c["cu_seqlens"].long())) == "OK"
        # views of wider rows at an odd element, any strides
        wide = torch.zeros(*c["x"].shape[:-1], 25, dtype=BF16)[..., 3:13]
        assert status(gdn2, e, dict(c, x=wide)) == "OK"
        # inputs may repeat a row
        assert status(gdn2, e, dict(c, x=c["x"][:1].expand(c["x"].shape))) == "OK"
    for g in (BF16, F32):
        assert status(gdn2, "scan", scan_case(g=g)) == "OK"
    for s in (BF16, F32):
        c = scan_case()
        assert status(gdn2, "scan", dict(c, initial_state=c["initial_state"].to(s), final_state=c["final_state"].to(s))) == "OK"
    for K in (2, 3, 4):
        for wt in (BF16, F32):
            assert status(gdn2, "conv_bwd", conv_back(K=K, wt=wt)) == "OK"
    assert status(gdn2, "norm", norm_case(D=16384)) == "OK"
    assert gdn2.STATUS[gdn2.check_layer_norm(zeros(5, 10), out=zeros(5, 10))] == "OK"


BAD = [
    ("scan", "x", None, "NULL_ARG"), ("scan", "g", None, "NULL_ARG"), ("scan", "out", None, "NULL_ARG"),
    ("scan", "x", zeros(70, 10, dtype=torch.float64), "DTYPE"), ("scan", "g", zeros(70, 10, dtype=F16), "DTYPE"),
    ("scan", "w", zeros(70, 10, dtype=F32), "DTYPE"), ("scan", "out", zeros(70, 10, dtype=F32), "DTYPE"),
    ("scan", "initial_state", zeros(2, 10, dtype=F16), "DTYPE"), ("scan", "g", zeros(70, 11, dtype=F32), "SHAPE"),
    ("scan", "w", zeros(69, 10), "SHAPE"), ("scan", "x", zeros(70, 1, 10), "SHAPE"), ("scan", "initial_state", zeros(3, 10, dtype=F32), "SHAPE"),
    ("scan", "final_state", zeros(10, 2, dtype=F32).T, "LAYOUT"), ("scan", "x", zeros(10, 70).T, "LAYOUT"),
    ("scan", "out", zeros(1, 10).expand(70, 10), "LAYOUT"), ("scan", "out", zeros(700).as_strided((70, 10), (9, 1)), "LAYOUT"),
    ("scan", "cu_seqlens", zeros(1, dtype=I32), "SHAPE"), ("scan", "cu_seqlens", zeros(3, dtype=F32), "DTYPE"),
    ("scan_bwd", "d_out", None, "NULL_ARG"), ("scan_bwd", "dx", None, "NULL_ARG"), ("scan_bwd", "dg", None, "NULL_ARG"),
    ("scan_bwd", "w", None, "NULL_ARG"), ("scan_bwd", "dg", zeros(70, 10), "DTYPE"), ("scan_bwd", "dx", zeros(70, 10, dtype=F32), "DTYPE"),
    ("scan_bwd", "d_final_state", zeros(2, 10), "DTYPE"), ("scan_bwd", "d_initial_state", zeros(2, 10), "DTYPE"),
    ("scan_bwd", "dw", zeros(1, 10).expand(70, 10), "LAYOUT"),
    ("conv", "x", None, "NULL_ARG"), ("conv", "weight", None, "NULL_ARG"), ("conv", "out", None, "NULL_ARG"),
    ("conv", "weight", zeros(10, 5), "UNSUPPORTED"), ("conv", "weight", zeros(10, 1), "UNSUPPORTED"),
    ("conv", "weight", zeros(11, 4), "SHAPE"), ("conv", "weight", zeros(4, 10).T, "LAYOUT"), ("conv", "weight", zeros(10, 4, dtype=F16), "DTYPE"),
    ("conv", "bias", zeros(10, dtype=F32), "DTYPE"), ("conv", "bias", zeros(11), "SHAPE"), ("conv", "initial_state", zeros(2, 4, 10), "SHAPE"),
    ("conv", "final_state", zeros(2, 3, 10, dtype=F32), "DTYPE"), ("conv", "cu_seqlens", zeros(3, dtype=torch.int16), "DTYPE"),
    ("conv_bwd", "dx", None, "NULL_ARG"), ("conv_bwd", "bias", None, "NULL_ARG"), ("conv_bwd", "dweight", zeros(10, 3), "SHAPE"),
    ("conv_bwd", "dweight", zeros(10, 4, dtype=F32), "DTYPE"), ("conv_bwd", "d_final_state", zeros(2, 3, 10, dtype=F32), "DTYPE"),
    ("norm", "x", None, "NULL_ARG"), ("norm", "out", None, "NULL_ARG"), ("norm", "weight", zeros(10, dtype=F16), "DTYPE"),
    ("norm", "gate", zeros(7, 3, 10, dtype=F32), "DTYPE"), ("norm", "gate", zeros(7, 2, 10), "SHAPE"), ("norm", "weight", zeros(9, dtype=F32), "SHAPE"),
    ("norm", "x", zeros(7, 3, 0), "UNSUPPORTED"), ("norm", "x", zeros(1, 1, 16385), "UNSUPPORTED"), ("norm", "x", zeros(7, 0, 10), "SHAPE"),
    ("norm", "out", zeros(7, 1, 10).expand(7, 3, 10), "LAYOUT"), ("norm", "x", zeros(7, 10, 3).transpose(1, 2), "LAYOUT"),
    ("norm_bwd", "d_out", None, "NULL_ARG"), ("norm_bwd", "dgate", None, "NULL_ARG"), ("norm_bwd", "gate", None, "NULL_ARG"),
    ("norm_bwd", "weight", None, "NULL_ARG"), ("norm_bwd", "bias", None, "NULL_ARG"), ("norm_bwd", "dbias", zeros(10), "DTYPE"),
]


@pytest.mark.parametrize("entry,name,value,want", BAD)
def test_refused(gdn2, entry, name, value, want):
    for e in ([entry, entry + "_step"] if entry in ("scan", "conv") else [entry]):
        assert status(gdn2, e, changed(ENTRIES[e][1](), name, value)) == want, gdn2.last_error()
        assert gdn2.last_error()


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_overlaps(gdn2, entry):
    """No output may share memory with an input or another output; a state may in the token steps."""
    make = ENTRIES[entry][1]
    c = make(T=70, D=70, N=70) if "norm" not in entry else make()
    outs = list(c["grads"]) if "grads" in c else [n for n in ("out", "final_state") if n in c]
    flat = {**{n: t for n, t in c.items() if n != "grads"}, **c.get("grads", {})}
    for o in outs:
        for n, t in flat.items():
            if n == o or t is None or t.shape != flat[o].shape or t.dtype != flat[o].dtype:
                continue
            want = "OK" if "step" in entry and {o, n} == {"initial_state", "final_state"} else "ALIAS"
            assert status(gdn2, entry, changed(c, o, t)) == want, (o, n)
    if "step" in entry:  # in place means the same buffer, not one that overlaps
        s = flat["final_state"]
        big = torch.zeros(2 * s.numel(), dtype=s.dtype)
        moved = big[8:8 + s.numel()].view(s.shape)
        assert status(gdn2, entry, dict(c, initial_state=big[:s.numel()].view(s.shape), final_state=moved)) == "ALIAS"


def test_misaligned_states_and_weights(gdn2):
    c = scan_case(D=11)
    assert status(gdn2, "scan", dict(c, initial_state=torch.zeros(23)[1:].view(2, 11))) == "LAYOUT"
    raw = torch.zeros(70 * 10 * 2 + 1, dtype=torch.uint8)
    assert raw.data_ptr() % 2 == 0
    d = gdn2.describe(zeros(70, 10))
    d.data = raw.data_ptr() + 1
    lib = gdn2.load_library()
    rest = [gdn2.describe(c0) for c0 in scan_case().values()]
    rest[0] = d
    rc = lib.gdn2_linear_scan_fwd_check(*[ctypes.addressof(r) for r in rest], None)
    assert gdn2.STATUS[rc] == "LAYOUT"


def test_options(gdn2):
    lib = gdn2.load_library()
    for c, cls, entry, bad in ((scan_case(), gdn2.Gdn2ScanOptions, lib.gdn2_linear_scan_fwd_check, (3, -1)),
                               (conv_case(), gdn2.Gdn2ConvOptions, lib.gdn2_short_conv_fwd_check, (2, -1))):
        keep, d = gdn2._describe_all(list(c.values()))
        size = ctypes.sizeof(cls)
        assert entry(*d, None) == 0 and entry(*d, ctypes.addressof(cls(size, 1))) == 0
        for v in bad:
            assert gdn2.STATUS[entry(*d, ctypes.addressof(cls(size, v)))] == "SHAPE"
        assert gdn2.STATUS[entry(*d, ctypes.addressof(cls(size - 1, 0)))] == "SHAPE"
    c = norm_case()
    keep, d = gdn2._describe_all([c[n] for n in ("x", "gate", "weight", "bias", "out")])
    cls = gdn2.Gdn2NormOptions
    size = ctypes.sizeof(cls)
    assert lib.gdn2_layer_norm_fwd_check(*d, None) == 0
    for o in (cls(size, 2, 0.0), cls(size, 0, -1.0), cls(size, 0, float("nan")), cls(size, 1, float("inf")), cls(size - 1, 0, 0.0)):
        assert gdn2.STATUS[lib.gdn2_layer_norm_fwd_check(*d, ctypes.addressof(o))] == "SHAPE"
    for bad in (lambda: gdn2.check_linear_scan(**scan_case(), input_scale="rms"),
                lambda: gdn2.check_short_conv(**conv_case(), activation="relu"),
                lambda: gdn2.check_layer_norm(**norm_case(), norm="l2")):
        with pytest.raises(ValueError):
            bad()


def test_workspaces(gdn2):
    """Sizes, 0 for what the entry refuses, and the refusal of a missing, small, misaligned or overlapping workspace."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert gdn2.linear_scan_fwd_workspace(1000, 1, 70) == 2 * up(16 * 70 * 4) + 2 * up(8 * 16 * 70 * 4)
    assert gdn2.linear_scan_bwd_workspace(1000, 1, 70) == 3 * up(16 * 70 * 4)
    assert gdn2.linear_scan_fwd_workspace(256, 1, 70) == gdn2.linear_scan_bwd_workspace(64, 1, 70) == 0
    assert gdn2.short_conv_bwd_workspace(1000, 70, 4) == up(-(-1000 // 64) * 5 * 70 * 4)
    assert gdn2.layer_norm_bwd_workspace(1000, 3, 64) >= 2 * 64 * 4
    for f in (gdn2.linear_scan_fwd_workspace, gdn2.linear_scan_bwd_workspace):
        for T, N, D in ((-1, 1, 8), (0, 1, 8), (1000, 0, 8), (1000, 1, 0), (1000, 1, -3), (2 ** 31 - 1, 1, 8), (2 ** 30, 1, 2 ** 24),
                        (1000, 1, 2 ** 24 + 1), (2 ** 62, 1, 8)):
            assert f(T, N, D) == 0, (T, N, D)
    for T, D, K in ((-1, 8, 4), (1000, 0, 4), (1000, 8, 1), (1000, 8, 5), (2 ** 31, 8, 4), (2 ** 30, 2 ** 24, 4)):
        assert gdn2.short_conv_bwd_workspace(T, D, K) == 0
    for T, H, D in ((-1, 1, 8), (0, 1, 8), (10, 0, 8), (10, 1, 0), (10, 1, 16385), (2 ** 30, 2, 8), (2 ** 62, 4, 8)):
        assert gdn2.layer_norm_bwd_workspace(T, H, D) == 0
    lib = gdn2.load_library()
    c = scan_back(T=1000)
    need = gdn2.linear_scan_bwd_workspace(1000, 2, 10)
    order = ["x", "g", "w", "initial_state", "cu_seqlens", "d_out", "d_final_state"]
    keep, d = gdn2._describe_all([c[n] for n in order] + [c["grads"][n] for n in gdn2.SCAN_GRADS])
    room = torch.zeros(need + 20000 + 512, dtype=torch.uint8)
    base = (room.data_ptr() + 255) // 256 * 256
    for ws, size in ((None, need), (base, need - 1), (base + 16, need)):
        assert gdn2.STATUS[lib.gdn2_linear_scan_bwd(*d, None, ws, size, None)] == "WORKSPACE"
    x = room[base - room.data_ptr():][:1000 * 20].view(BF16).view(1000, 10)
    keep, d = gdn2._describe_all([x] + [c[n] for n in order[1:]] + [c["grads"][n] for n in gdn2.SCAN_GRADS])
    assert gdn2.STATUS[lib.gdn2_linear_scan_bwd(*d, None, base, need, None)] == "ALIAS"


@pytest.mark.parametrize("T,N,D,ok", [(2 ** 31 - 65537, 1, 1, False), (2 ** 20, 1, 2 ** 14, True), (2 ** 22, 1, 2 ** 14, False),
                                      (70, 1, 2 ** 24, True), (70, 1, 2 ** 24 + 1, False)])
def test_launch_limits(gdn2, T, N, D, ok):
    """Sizes that one launch cannot hold are refused (descriptors without memory behind them, rows repeated)."""
    x, g = zeros(1, 1).expand(T, D), zeros(1, 1, dtype=F32).expand(T, D)
    ds = []
    for t in (x, g, x, x):
        d = gdn2.describe(t)
        d.stride[0], d.stride[1] = (D, 1)
        ds.append(d)
    ds[3].data = 1 << 60  # an output apart from the inputs
    lib = gdn2.load_library()
    p = [ctypes.addressof(d) for d in ds]
    rc = lib.gdn2_linear_scan_fwd_check(p[0], p[1], None, None, None, p[3], None, None)
    assert (gdn2.STATUS[rc] == "OK") == ok, gdn2.last_error()
    assert ok or gdn2.STATUS[rc] == "SHAPE"


def test_binding_refuses(gdn2):
    """CPU tensors, wrong ranks: before the library is called."""
    c = scan_case()
    with pytest.raises(ValueError, match="GPU"):
        gdn2.linear_scan_fwd(c["x"], c["g"])
    with pytest.raises(ValueError, match="GPU"):
        gdn2.short_conv_fwd(zeros(4, 8), zeros(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        gdn2.layer_norm(zeros(4, 8))
