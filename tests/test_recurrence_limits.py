"""The sizes from which the gated recurrence's calls are refused, from both sides. An output that is off its alignment stands
for the next check, so that no call reaches a launch."""
import ctypes

import pytest

from fft_long_convolution_libhyena_amd import binding
from fft_long_convolution_libhyena_amd.binding import RecurrenceInputsStruct, RecurrenceParamsStruct

INVALID, UNSUPPORTED = 1, 2
P = 4096  # stands for a device address; never followed


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def common(dim):
    return ctypes.byref(RecurrenceParamsStruct(dim, 1, 0, P)), ctypes.byref(RecurrenceInputsStruct(P, dim, P, dim, P, dim))


# 2^23 pairs of 80 tokens and 128 channels are too many
@pytest.mark.parametrize("dim,most", [(8, 671088560), (128, 671088560), (136, 335544240), (1 << 20, 81840)])
def test_whole_sequences(lib, dim, most):
    p, i = common(dim)
    for tokens, want in ((most, INVALID), (most + 1, UNSUPPORTED)):
        assert lib.hyena_recurrence_forward(p, 1, tokens, None, i, None, P + 8, P, None, P, 1 << 50, None) == want
        assert lib.hyena_recurrence_backward(p, 1, tokens, None, i, None, None, P, None, P + 8, P, P, P, None, P, 1 << 50, None) == want
        assert (lib.hyena_recurrence_workspace_bytes(p, 1, tokens, None) > 0) == (want == INVALID)
        assert (lib.hyena_recurrence_backward_workspace_bytes(p, 1, tokens, None, None) > 0) == (want == INVALID)


def test_steps_are_held_to_their_own_grid_alone(lib):
    for dim, B, T, want in ((8192, 1, 1 << 24, INVALID), (8, 1 << 23, 255, INVALID), (512, (1 << 24) - 1, 1, INVALID),
                            (512, 1 << 24, 1, UNSUPPORTED), (520, 1 << 23, 1, UNSUPPORTED),  # 2^24 pairs of a row and 512 channels
                            (8, 1 << 12, (1 << 19) - 1, INVALID), (8, 1 << 12, 1 << 19, UNSUPPORTED)):  # 2^31 - 256 tokens
        p, i = common(dim)
        # misaligned states stop what the shared checks pass; the grid's are behind them
        got = lib.hyena_recurrence_step(p, B, T, i, P if want == UNSUPPORTED else P + 8, 1 << 24, None, P, None)
        assert got == want, (dim, B, T)
