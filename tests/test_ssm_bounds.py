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
