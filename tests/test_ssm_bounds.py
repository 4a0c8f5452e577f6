"""Bounds and overlaps at the convolution's C entry points (CPU only): refused before
anything is launched."""
import ctypes

from delta_rule_sequence_efla_amd import efla

NUL, FAKE = None, ctypes.c_void_p(4096)
INVALID, UNSUPPORTED = 1, 2


def empty_gradient(B, D, W):
    """Sequences without tokens: ds_final is copied to ds0, B (W - 1) D threads of a launch."""
    return efla.lib().efla_conv_bwd(NUL, D, FAKE, NUL, NUL, NUL, D, FAKE, NUL, D, FAKE, NUL, ctypes.c_void_p(1 << 44), B, 0, D, W,
                                    1, 1, NUL, 0, NUL)


def test_states_of_empty_sequences_past_one_launch():
    B, D = 1 << 15, 43691  # 3 B D = 2^32 + 2^15, and B D below the bounds of the forward pass
    assert empty_gradient(B, D, 4) == UNSUPPORTED
    assert empty_gradient(B, 60000, 4) == UNSUPPORTED


MEM = 1 << 44


def at(x):
    return ctypes.c_void_p(MEM + x)


def forward(x, y, row=64, yrow=None, B=2, L=32, D=64):
    return efla.lib().efla_conv_fwd(at(x), row, FAKE, NUL, NUL, at(y), yrow or row, NUL, B, L, D, 4, 1, 1, NUL)


def packed(x, y, row=64, T=64, D=64):
    return efla.lib().efla_conv_fwd_varlen(at(x), row, FAKE, NUL, FAKE, NUL, 2, 2, NUL, at(y), row, NUL, T, D, 4, 1, 1, NUL)


def gradient(x, dy, dx, s0=None, dsf=None, ds0=None, row=64):
    p = [NUL if t is None else at(t) for t in (s0, dsf, ds0)]
    return efla.lib().efla_conv_bwd(at(x), row, FAKE, NUL, p[0], at(dy), row, p[1], at(dx), row, FAKE, NUL, p[2], 2, 32, 64, 4, 1,
                                    1, FAKE, 1 << 30, NUL)


def test_outputs_over_inputs():
    """64 rows of 64 bf16 channels, 128 bytes: the convolution's rows are read by more than the wavefront that writes them."""
    for call in (forward, packed):
        for y in (0, 16, 128 * 5, 128 * 63 + 112, -128 * 63, -128 * 64 + 16):
            assert call(0, y) == INVALID, y
        for y in (0, 112, 256 * 3 + 48, -256 * 63 + 112, 256 - 112):  # rows of a tensor twice as wide
            assert call(0, y, row=128) == INVALID, y
    assert forward(0, 64, B=1, L=1, yrow=4096) == INVALID
    far = 1 << 20
    for shift in (0, 64, -64):
        assert gradient(0, far, shift) == INVALID and gradient(far, 0, shift) == INVALID
    assert gradient(0, far, 2 * far, dsf=4 * far, ds0=4 * far) == INVALID
    assert gradient(0, far, 2 * far, s0=4 * far, ds0=4 * far + 2 * 3 * 128 - 16) == INVALID
