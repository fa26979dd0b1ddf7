"""A workspace that holds for a call holds for every smaller one, of fewer tokens or of fewer channels: a program may
size one for its largest call and share it among all."""
import ctypes

import pytest

from fft_long_convolution_libhyena_amd import binding
from fft_long_convolution_libhyena_amd.binding import QKNormParamsStruct, RecurrenceParamsStruct, ResidualNormParamsStruct

P = 4096  # stands for a device address; never followed
TOKENS = sorted({*range(0, 700), *range(700, 20000, 37), *range(20000, 400000, 997), 2688, 2689, 2752, 4096, 16384, 16385})
DIMS = sorted({*range(8, 1100, 8), *range(1104, 40000, 1256), 1 << 15, (1 << 15) + 8})


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def recurrence(lib, dim, tokens, which):
    p = ctypes.byref(RecurrenceParamsStruct(dim, 1, 0, P))
    if which == "forward":
        return lib.hyena_recurrence_workspace_bytes(p, 1, tokens, None)
    return lib.hyena_recurrence_backward_workspace_bytes(p, 1, tokens, None, P if which == "backward of carries" else None)


WHICH = ["forward", "backward", "backward of carries"]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("dim", [8, 128, 136, 768, 1000, 2048, 33000])
def test_recurrence_never_falls_with_the_tokens(lib, dim, which):
    sizes = [recurrence(lib, dim, t, which) for t in TOKENS]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("tokens", [1, 64, 65, 500, 2688, 9000, 50000])
def test_recurrence_never_falls_with_the_channels(lib, tokens, which):
    sizes = [recurrence(lib, d, tokens, which) for d in DIMS]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("heads_q,heads_k,dim", [(6, 6, 128), (12, 4, 64), (1, 1, 8), (3, 1, 256), (2000, 1, 16)])
def test_head_norm_never_falls_with_the_tokens(lib, heads_q, heads_k, dim):
    p = ctypes.byref(QKNormParamsStruct(heads_q, heads_k, dim, 0, 0, 0, 1, 1e-6, P, P, None))
    sizes = [lib.hyena_qk_norm_backward_workspace_bytes(p, t) for t in TOKENS]
    assert sizes == sorted(sizes) and sizes[1] > 0


@pytest.mark.parametrize("dim", [8, 256, 264, 768, 1032, 16384])
def test_residual_norm_never_falls_with_the_rows(lib, dim):
    p = ctypes.byref(ResidualNormParamsStruct(dim, 1, 0, 0, 1e-6, P))
    sizes = [lib.hyena_residual_norm_backward_workspace_bytes(p, t) for t in TOKENS]
    assert sizes == sorted(sizes) and sizes[1] > 0
