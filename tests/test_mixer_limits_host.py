"""CPU tests of the sizes that one launch holds, just under and just over, for
the recurrence's gradients, the convolution and the token steps (descriptors
without memory behind them; the checks alone)."""

import ctypes

import pytest
import torch

from tests.test_delta_host import gdn2  # noqa: F401

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
THREADS = 2 ** 32 - 1  # that one launch can hold


class Made:
    def __init__(self, gdn2):
        self.gdn2, self.keep = gdn2, []

    def __call__(self, *shape, dtype=BF16, out=0):
        d = self.gdn2.describe(torch.zeros((1,) * len(shape), dtype=dtype))
        stride = 1
        for i in reversed(range(len(shape))):
            d.shape[i], d.stride[i] = shape[i], stride
            stride *= shape[i]
        d.data = (64 if out == 0 else out << 58)  # outputs apart from the inputs and each other
        self.keep.append(d)
        return ctypes.addressof(d)


def verdict(gdn2, rc):
    return gdn2.STATUS[rc]


def most_tokens(threads, per_part, cols, more=0):
    """T with the most parts of per_part tokens that `cols` columns of workgroups leave room for."""
    return (THREADS // threads // cols - more) * per_part


@pytest.mark.parametrize("D", [1, 64, 65, 4096, 2 ** 20])
def test_recurrence_and_its_gradients(gdn2, D):
    lib, t = gdn2.load_library(), Made(gdn2)
    T = most_tokens(512, 64, -(-D // 64))
    for tokens, want in ((T, "OK"), (T + 1, "SHAPE")):
        if tokens > 2 ** 31 - 65537:
            continue
        x, g = t(tokens, D), t(tokens, D, dtype=F32)
        rc = lib.gdn2_linear_scan_fwd_check(x, g, None, None, None, t(tokens, D, out=1), None, None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()
        rc = lib.gdn2_linear_scan_bwd_check(x, g, None, None, None, x, None, t(tokens, D, out=1), t(tokens, D, dtype=F32, out=2), None, None,
                                            None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()
        assert (gdn2.linear_scan_bwd_workspace(tokens, 1, D) > 0) == (want == "OK" and tokens > 64)


@pytest.mark.parametrize("D", [1, 64, 65, 4096, 2 ** 20])
def test_convolution_and_its_gradients(gdn2, D):
    lib, t = gdn2.load_library(), Made(gdn2)
    T = most_tokens(256, 32, -(-D // 64), more=1) + 31  # (32 tokens in one workgroup, where slices are shortest)
    w = t(D, 4)
    for tokens, want in ((T, "OK"), (T + 1, "SHAPE")):
        x = t(tokens, D)
        assert verdict(gdn2, lib.gdn2_short_conv_fwd_check(x, w, None, None, None, t(tokens, D, out=1), None, None)) == want
        rc = lib.gdn2_short_conv_bwd_check(x, w, None, None, None, x, None, t(tokens, D, out=1), t(D, 4, out=2), None, None, None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()
        assert (gdn2.short_conv_bwd_workspace(tokens, D, 4) > 0) == (want == "OK")


@pytest.mark.parametrize("D", [1, 256, 257, 8192, 2 ** 24])
def test_token_steps(gdn2, D):
    lib, t = gdn2.load_library(), Made(gdn2)
    N = THREADS // 256 // -(-D // 256)
    w = t(D, 4)
    for n, want in ((N, "OK"), (N + 1, "SHAPE")):
        x, cu = t(70, D), t(n + 1, dtype=I32)
        rc = lib.gdn2_linear_scan_recurrent_fwd_check(x, t(70, D, dtype=F32), None, None, cu, t(70, D, out=1), None, None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()
        rc = lib.gdn2_short_conv_recurrent_fwd_check(x, w, None, None, cu, t(70, D, out=1), None, None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()


def test_most_tokens_and_sequences(gdn2):
    lib, t = gdn2.load_library(), Made(gdn2)
    for T, N, want in ((2 ** 31 - 65537, 70, "OK"), (2 ** 31 - 65536, 70, "SHAPE"), (70, 2 ** 24 - 1, "OK"), (70, 2 ** 31 - 65536, "SHAPE")):
        x, cu = t(T, 1), t(N + 1, dtype=I32)
        rc = lib.gdn2_linear_scan_recurrent_fwd_check(x, t(T, 1, dtype=F32), None, None, cu, t(T, 1, out=1), None, None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()
    for T, H, want in ((2 ** 31 - 1, 1, "OK"), (2 ** 31, 1, "SHAPE"), (2 ** 30, 1, "OK"), (2 ** 30, 2, "SHAPE")):
        rc = lib.gdn2_layer_norm_fwd_check(t(T, H, 1), None, None, None, t(T, H, 1, out=1), None)
        assert verdict(gdn2, rc) == want, gdn2.last_error()


def test_interleaved_outputs_are_refused(gdn2):
    """Overlaps go by whole spans: gradients that are views of one joint buffer, although no element is shared."""
    both = torch.zeros(7, 3, 20, dtype=BF16)
    x, gate, d_out = (torch.zeros(7, 3, 10, dtype=BF16) for _ in range(3))
    for dx, dgate, want in ((both[..., :10], both[..., 10:], "ALIAS"), (both[..., :10], torch.zeros(7, 3, 10, dtype=BF16), "OK")):
        rc = gdn2.check_layer_norm_bwd(x, d_out, gate=gate, grads={"dx": dx, "dgate": dgate})
        assert verdict(gdn2, rc) == want


def test_no_eps_is_the_default(gdn2):
    assert gdn2._norm_options("rms", None).eps == gdn2._norm_options("rms", 0.0).eps == 0.0
