"""CPU tests of the argument checks of the scalar-gated delta rule's and the
q/k preparation's entries: the ``_check`` functions run the validation alone,
on descriptors of host memory."""

import os

import pytest
import torch

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def gdn2():
    from linear_attention_rnn_gdn2_amd import gdn2 as mod
    if not os.path.exists(mod.LIB_PATH):
        from linear_attention_rnn_gdn2_amd._build import build_library
        build_library()
    mod.load_library()
    return mod


def case(T=70, H=2, HV=4, K=64, V=64, N=2, io=BF16):
    return dict(q=torch.zeros(T, H, K, dtype=io), k=torch.zeros(T, H, K, dtype=io), v=torch.zeros(T, HV, V, dtype=io),
                g=torch.zeros(T, HV), beta=torch.zeros(T, HV, dtype=io), initial_state=torch.zeros(N, HV, K, V),
                cu_seqlens=torch.zeros(N + 1, dtype=torch.int32), out=torch.zeros(T, HV, V, dtype=io),
                final_state=torch.zeros(N, HV, K, V))


def status(gdn2, **kw):
    return gdn2.STATUS[gdn2.check_delta(**kw)]


@pytest.mark.parametrize("recurrent", [False, True])
def test_accepted(gdn2, recurrent):
    for K in (64, 128):
        for V in (64, 128):
            for io in (BF16, F16):
                assert status(gdn2, **case(K=K, V=V, io=io), recurrent=recurrent) == "OK"
    c = case()
    for n in ("g", "beta", "initial_state", "final_state"):
        assert status(gdn2, **dict(c, **{n: None}), recurrent=recurrent) == "OK"
    for g in (BF16, F16):
        assert status(gdn2, **dict(c, g=c["g"].to(g)), recurrent=recurrent) == "OK"
    # gates with any strides and any alignment of an element
    wide = torch.zeros(70, 9)
    assert status(gdn2, **dict(c, g=wide[:, 3:7]), recurrent=recurrent) == "OK"
    assert status(gdn2, **dict(c, g=torch.zeros(4, 70).T, beta=torch.zeros(1, 4, dtype=BF16).expand(70, 4)),
                  recurrent=recurrent) == "OK"
    fused = torch.zeros(70, 3, 4, 64, dtype=BF16)
    f = case(H=4)
    assert status(gdn2, **dict(f, q=fused[:, 0], k=fused[:, 1], v=fused[:, 2]), recurrent=recurrent) == "OK"
    assert status(gdn2, **dict(c, cu_seqlens=c["cu_seqlens"].long()), recurrent=recurrent) == "OK"
    vk = case(K=64, V=128)
    vk["initial_state"] = vk["final_state"] = None
    assert status(gdn2, **dict(vk, initial_state=torch.zeros(2, 4, 128, 64)), state_layout="vk", qk_l2norm=True,
                  recurrent=recurrent) == "OK"


BAD = [
    ("q", None, "NULL_ARG"), ("k", None, "NULL_ARG"), ("v", None, "NULL_ARG"), ("out", None, "NULL_ARG"),
    ("q", torch.zeros(70, 2, 64), "DTYPE"), ("k", torch.zeros(70, 2, 64, dtype=F16), "DTYPE"),
    ("v", torch.zeros(70, 4, 64, dtype=F16), "DTYPE"), ("beta", torch.zeros(70, 4), "DTYPE"),
    ("g", torch.zeros(70, 4, dtype=torch.int32), "DTYPE"), ("g", torch.zeros(70, 4, dtype=torch.float64), "DTYPE"),
    ("g", torch.zeros(70, 4, 64), "SHAPE"), ("g", torch.zeros(69, 4), "SHAPE"), ("beta", torch.zeros(70, 2, dtype=BF16), "SHAPE"),
    ("k", torch.zeros(71, 2, 64, dtype=BF16), "SHAPE"), ("out", torch.zeros(70, 4, 128, dtype=BF16), "SHAPE"),
    ("v", torch.zeros(70, 3, 64, dtype=BF16), "HEADS"), ("v", torch.zeros(70, 4, 96, dtype=BF16), "UNSUPPORTED"),
    ("initial_state", torch.zeros(3, 4, 64, 64), "SHAPE"), ("initial_state", torch.zeros(2, 4, 64, 64, dtype=F16), "DTYPE"),
    ("final_state", torch.zeros(2, 4, 64, 64).transpose(2, 3), "LAYOUT"), ("cu_seqlens", torch.zeros(1, dtype=torch.int32), "SHAPE"),
    ("cu_seqlens", torch.zeros(3), "DTYPE"), ("q", torch.zeros(70, 64, 2, dtype=BF16).transpose(1, 2), "LAYOUT"),
    ("q", torch.zeros(70, 2, 68, dtype=BF16)[:, :, :64], "LAYOUT"),
    ("out", torch.zeros(1, 4, 64, dtype=BF16).expand(70, 4, 64), "LAYOUT"),
]


@pytest.mark.parametrize("recurrent", [False, True])
@pytest.mark.parametrize("name,value,want", BAD)
def test_refused(gdn2, recurrent, name, value, want):
    c = case()
    if name == "v" and want != "DTYPE" and value is not None:  # sizes that go by v
        c.update(out=torch.zeros_like(value), g=None, beta=None, initial_state=None, final_state=None)
    assert status(gdn2, **dict(c, **{name: value}), recurrent=recurrent) == want, gdn2.last_error()


def test_refused_options_and_overlaps(gdn2):
    c = case()
    assert status(gdn2, **c, seq_split=4) == "UNSUPPORTED"
    assert status(gdn2, **c, seq_split=-1) == "OK"
    assert status(gdn2, **c, seq_split=4, recurrent=True) == "OK"
    assert status(gdn2, **dict(c, out=c["v"])) == "ALIAS"
    assert status(gdn2, **dict(c, final_state=c["initial_state"])) == "ALIAS"
    assert status(gdn2, **dict(c, final_state=c["initial_state"]), recurrent=True) == "OK"
    both = torch.zeros(3, 4, 64, 64)
    assert status(gdn2, **dict(c, initial_state=both[:2], final_state=both[1:]), recurrent=True) == "ALIAS"
    half = c["initial_state"].to(BF16)
    assert status(gdn2, **dict(c, initial_state=half, final_state=half), recurrent=True) == "OK"
    with pytest.raises(ValueError):
        gdn2.check_delta(**c, state_layout="x")
    # the launch limit (only descriptors: no memory of that size exists)
    big = dict(case(T=1), g=None, beta=None, initial_state=None, final_state=None)
    for n in ("q", "k", "v", "out"):
        big[n] = torch.empty(1 << 30, big[n].shape[1], 64, dtype=BF16, device="meta")
    assert gdn2.STATUS[gdn2.check_delta(**big)] in ("SHAPE", "NULL_ARG")


def bwd_case(T=70, H=2, HV=4, D=64, N=2, io=BF16):
    c = case(T, H, HV, D, D, N, io)
    c.pop("out"), c.pop("final_state")
    c["d_out"], c["d_final_state"] = torch.zeros_like(c["v"]), torch.zeros_like(c["initial_state"])
    c["grads"] = dict(dq=torch.zeros_like(c["q"]), dk=torch.zeros_like(c["k"]), dv=torch.zeros_like(c["v"]),
                      dg=torch.zeros_like(c["g"]), dbeta=torch.zeros_like(c["beta"]),
                      d_initial_state=torch.zeros_like(c["initial_state"]))
    return c


def bwd_status(gdn2, c):
    return gdn2.STATUS[gdn2.check_delta_bwd(**c)]


def test_backward_checks(gdn2):
    for D in (64, 128):
        for io in (BF16, F16):
            assert bwd_status(gdn2, bwd_case(D=D, io=io)) == "OK"
    for n in ("initial_state", "d_final_state", "cu_seqlens"):
        c = bwd_case(N=1)
        c[n] = None
        assert bwd_status(gdn2, c) == "OK"
    for n in ("g", "beta", "d_out", "q"):
        c = bwd_case()
        c[n] = None
        assert bwd_status(gdn2, c) == "NULL_ARG", n
    c = bwd_case()
    c["grads"]["d_initial_state"] = None
    assert bwd_status(gdn2, c) == "OK"
    for n in ("dq", "dg", "dbeta"):
        c = bwd_case()
        c["grads"][n] = None
        assert bwd_status(gdn2, c) == "NULL_ARG", n
    c = bwd_case()
    c["v"] = c["d_out"] = c["grads"]["dv"] = torch.zeros(70, 4, 128, dtype=BF16)
    assert bwd_status(gdn2, c) == "UNSUPPORTED"
    c = bwd_case()
    c["grads"]["dg"] = c["grads"]["dg"].to(BF16)
    assert bwd_status(gdn2, c) == "DTYPE"
    c = bwd_case()
    c["g"] = torch.zeros(4, 70).T
    assert bwd_status(gdn2, c) == "LAYOUT"
    c = bwd_case()
    c["grads"]["dk"] = c["grads"]["dq"]
    assert bwd_status(gdn2, c) == "ALIAS"
    c = bwd_case()
    c["grads"]["dv"] = c["d_out"]
    assert bwd_status(gdn2, c) == "ALIAS"
    c = bwd_case()
    c["initial_state"] = c["initial_state"].to(BF16)
    assert bwd_status(gdn2, c) == "DTYPE"


def test_workspace_sizes(gdn2):
    """(T / 64 + N) HV records; the backward's checkpoints beside them; monotone; nothing for nothing."""
    assert gdn2.delta_chunk_fwd_workspace(130, 2, 4) == (130 // 64 + 2) * 4 * 26880
    assert gdn2.delta_chunk_fwd_workspace(0, 2, 4) == 0
    items = (130 // 64 + 2) * 4
    want = items * (26880 + 8 * 64 * 64 + 514 * 64) + 2 * 130 * 4 * 64 * 4
    got = gdn2.delta_chunk_bwd_workspace(130, 2, 2, 4, 64, 64)
    assert want <= got <= want + 8 * 256
    assert gdn2.delta_chunk_bwd_workspace(130, 2, 4, 4, 64, 64) < got
    assert gdn2.delta_chunk_bwd_workspace(0, 2, 2, 4, 64, 64) == 0
    assert gdn2.qk_norm_rope_bwd_workspace(0, 2, 4, 64) == 0
    assert 0 < gdn2.qk_norm_rope_bwd_workspace(1, 2, 4, 64) <= gdn2.qk_norm_rope_bwd_workspace(100000, 2, 4, 64) <= 2048 * 1024


def qk_case(T=9, H=3, HK=2, K=64, io=BF16, rot=32):
    return dict(q=torch.zeros(T, H, K, dtype=io), k=torch.zeros(T, HK, K, dtype=io), q_weight=torch.zeros(K),
                k_weight=torch.zeros(K, dtype=io), rope=torch.zeros(50, rot), positions=torch.zeros(T, dtype=torch.int32),
                q_out=torch.zeros(T, H, K, dtype=io), k_out=torch.zeros(T, HK, K, dtype=io))


def qk_status(gdn2, c, **kw):
    return gdn2.STATUS[gdn2.check_qk_norm_rope(**c, **kw)]


def test_qk_accepted(gdn2):
    for K in (64, 128):
        for io in (BF16, F16):
            for norm in ("l2", "rms", "none"):
                assert qk_status(gdn2, qk_case(K=K, io=io), norm=norm) == "OK"
    assert qk_status(gdn2, qk_case(rot=6), interleaved=True) == "OK"
    assert qk_status(gdn2, dict(qk_case(), q_weight=None, k_weight=None, rope=None, positions=None)) == "OK"
    assert qk_status(gdn2, dict(qk_case(), positions=torch.zeros(9, dtype=torch.int64))) == "OK"


@pytest.mark.parametrize("name,value,want", [
    ("q", None, "NULL_ARG"), ("k_out", None, "NULL_ARG"), ("positions", None, "NULL_ARG"), ("rope", None, "NULL_ARG"),
    ("k", torch.zeros(8, 2, 64, dtype=BF16), "SHAPE"), ("k", torch.zeros(9, 2, 64, dtype=F16), "DTYPE"),
    ("q_weight", torch.zeros(32), "SHAPE"), ("q_weight", torch.zeros(64, dtype=F16), "DTYPE"),
    ("rope", torch.zeros(50, 24), "UNSUPPORTED"), ("rope", torch.zeros(50, 128), "UNSUPPORTED"),
    ("rope", torch.zeros(0, 32), "SHAPE"), ("rope", torch.zeros(50, 32, dtype=BF16), "DTYPE"),
    ("positions", torch.zeros(8, dtype=torch.int32), "SHAPE"), ("positions", torch.zeros(9), "DTYPE"),
    ("q_out", torch.zeros(1, 3, 64, dtype=BF16).expand(9, 3, 64), "LAYOUT"), ("q", torch.zeros(9, 3, 96, dtype=BF16), "SHAPE")])
def test_qk_refused(gdn2, name, value, want):
    assert qk_status(gdn2, dict(qk_case(), **{name: value})) == want, gdn2.last_error()


def test_qk_refused_options(gdn2):
    c = qk_case()
    for eps in (-1.0, float("inf"), float("nan")):
        assert qk_status(gdn2, c, eps=eps) == "SHAPE"
    with pytest.raises(ValueError):
        gdn2.check_qk_norm_rope(**c, norm="max")
    assert qk_status(gdn2, dict(c, q_out=c["q"])) == "ALIAS"
    one = torch.zeros(9, 3, 64, dtype=BF16)
    assert qk_status(gdn2, dict(c, k=torch.zeros(9, 3, 64, dtype=BF16), q_out=one, k_out=one)) == "ALIAS"


def test_qk_backward_checks(gdn2):
    c = qk_case()
    c["dq_out"], c["dk_out"] = torch.zeros_like(c.pop("q_out")), torch.zeros_like(c.pop("k_out"))
    g = dict(dq=torch.zeros_like(c["q"]), dk=torch.zeros_like(c["k"]), dq_weight=torch.zeros(64),
             dk_weight=torch.zeros(64, dtype=BF16))

    def st(c, g):
        return gdn2.STATUS[gdn2.check_qk_norm_rope_bwd(**c, grads=g)]

    assert st(c, g) == "OK"
    assert st(c, dict(g, dq_weight=None)) == "OK"
    assert st(dict(c, q_weight=None), g) == "NULL_ARG"
    assert st(c, dict(g, dk_weight=torch.zeros(64))) == "DTYPE"
    assert st(c, dict(g, dq=c["dq_out"])) == "ALIAS"
    assert st(dict(c, dk_out=None), g) == "NULL_ARG"


def test_rope_table(gdn2):
    t = gdn2.rope_table(1000, 8, base=100.0, position_scale=0.5, device="cpu")
    assert t.shape == (1000, 8) and t.dtype == F32
    pos, i = 777, 3
    angle = torch.tensor(777 * 0.5 * 100.0 ** (-2 * i / 8), dtype=torch.float64)
    assert t[pos, i] == angle.cos().float() and t[pos, 4 + i] == angle.sin().float()
    with pytest.raises(ValueError):
        gdn2.rope_table(10, 7, device="cpu")


def test_host_tensors_are_refused(gdn2):
    c = case()
    for call in (gdn2.delta_chunk_fwd, gdn2.delta_recurrent_fwd):
        with pytest.raises(ValueError):
            call(**c)
    with pytest.raises(ValueError):
        gdn2.qk_norm_rope(c["q"], c["k"])
    with pytest.raises(ValueError):
        gdn2.qk_norm_rope_bwd(c["q"], c["k"], c["q"], c["k"])
    b = bwd_case()
    with pytest.raises(ValueError):
        gdn2.delta_chunk_bwd(**b)


@pytest.mark.parametrize("recurrent", [False, True])
def test_chain_limit(gdn2, recurrent):
    """768 threads per (sequence, value head): 5592405 chains are one launch, one more is refused."""
    c = dict(case(T=64, H=1, HV=1), initial_state=None, final_state=None)
    for n, want in ((5592405 - 1, "OK"), (5592406, "SHAPE")):
        c["cu_seqlens"] = torch.zeros(n + 1, dtype=torch.int32)
        assert status(gdn2, **c, recurrent=recurrent) == want


def test_split_workspace(gdn2):
    """Segments are added where few long sequences are split, 8 MiB at most, and nowhere else."""
    def more(T, N, HV):
        return gdn2.delta_chunk_fwd_workspace(T, N, HV) - (T // 64 + N) * HV * 26880
    assert more(4096, 1, 16) == 4 * 16 * 131072 and more(37517, 8, 32) == 0 and more(1000, 1, 1) == 0
    for T in (1536, 2304, 5000, 40000, 1 << 20):
        for N in (1, 2, 3, 8):
            for HV in range(1, 70):
                assert 0 <= more(T, N, HV) <= 8 << 20

    def more_bwd(T, N, HV, D):
        return gdn2.delta_chunk_bwd_workspace(T, N, HV, HV, D, D) - (T // 64 + N) * HV * (26880 + 8 * D * D + 514 * D)
    assert more_bwd(4096, 1, 16, 128) == 4 * 16 * (131072 + 65536) and 0 <= more_bwd(1000, 1, 1, 64) < 8 * 256
    for T in (2304, 40000):
        for N in (1, 3):
            for HV in range(1, 70):
                assert 0 <= more_bwd(T, N, HV, 64) and more_bwd(T, N, HV, 128) < (12 << 20) + 8 * 256
