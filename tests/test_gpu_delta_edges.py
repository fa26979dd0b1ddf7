"""Gated delta rule on the GPU: calls at the edges of what include/hyena.h allows."""
import pytest
import torch

import _delta as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_empty_sequences_need_no_workspace(packed, dtype):
    """Without tokens the states are passed on and their gradients back, with no workspace."""
    import ctypes

    from fft_long_convolution_libhyena_amd import DeltaRule
    from fft_long_convolution_libhyena_amd.binding import DeltaInputsStruct

    N, hv, dk, dv = 3, 2, 64, 40
    r = DeltaRule(1, hv, dk, dv, dtype)
    none = DeltaInputsStruct(None, dk, None, dk, None, hv * dv, None, None)
    starts = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    start = starts.data_ptr() if packed else None
    s, ds = torch.randn(2, N, hv, dk, dv, device="cuda")
    out, dout = torch.empty_like(s), torch.empty_like(s)
    stream = torch.cuda.current_stream().cuda_stream
    assert r.lib.hyena_delta_forward(r._params(None), N, 0, start, ctypes.byref(none), s.data_ptr(), None, out.data_ptr(), None, 0,
                                     stream) == 0
    assert r.lib.hyena_delta_backward(r._params(None), N, 0, start, ctypes.byref(none), s.data_ptr(), None, ds.data_ptr(), None,
                                      None, None, None, None, dout.data_ptr(), None, 0, stream) == 0
    assert torch.equal(out, s) and torch.equal(dout, ds)
