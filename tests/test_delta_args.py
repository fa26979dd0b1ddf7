"""Refusals of the delta rule's entry points: every argument error is found on the host,
before any device call, so these run without a GPU."""
import ctypes

import pytest

from fft_long_convolution_libhyena_amd import binding
from fft_long_convolution_libhyena_amd.binding import DeltaInputsStruct, DeltaParamsStruct

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 4096  # stands for a device address; never followed


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def params(**kw):
    d = dict(heads_k=2, heads_v=4, dim_k=64, dim_v=64, dtype=1, scale=0.125)
    d.update(kw)
    return DeltaParamsStruct(*(d[n] for n, _ in DeltaParamsStruct._fields_))


def inputs(**kw):
    d = dict(q=P, ldq=128, k=P, ldk=128, v=P, ldv=256, g=P, beta=P)
    d.update(kw)
    return DeltaInputsStruct(*(d[n] for n, _ in DeltaInputsStruct._fields_))


def forward(lib, p=None, N=2, tokens=128, start=None, i=None, s_in=None, o=P, s_out=P, ws=P, ws_bytes=1 << 40):
    p, i = p or params(), i or inputs()
    return lib.hyena_delta_forward(ctypes.byref(p), N, tokens, start, ctypes.byref(i), s_in, o, s_out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(heads_k=0), INVALID), (dict(heads_v=0), INVALID), (dict(heads_k=3), INVALID), (dict(dim_k=0), INVALID),
    (dict(dim_v=-8), INVALID), (dict(dtype=5), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(dim_k=12), UNSUPPORTED), (dict(dim_k=136), UNSUPPORTED), (dict(dim_v=20), UNSUPPORTED),
    (dict(dim_v=264), UNSUPPORTED), (dict(heads_k=1, heads_v=65536), UNSUPPORTED),
])
def test_params(lib, kw, want):
    p = params(**kw)
    wide = dict(ldq=1 << 20, ldk=1 << 20, ldv=1 << 30)
    assert forward(lib, p, i=inputs(**wide)) == want
    assert lib.hyena_delta_workspace_bytes(ctypes.byref(p), 2, 128, None) == 0
    assert lib.hyena_delta_step(ctypes.byref(p), 2, 1, ctypes.byref(inputs(**wide)), P, 4, None, P, None) == want


@pytest.mark.parametrize("kw", [dict(N=0), dict(tokens=-1), dict(tokens=127), dict(start=P + 4), dict(o=None),
                                dict(o=P + 8), dict(s_in=P + 4), dict(s_out=P + 8), dict(ws=P + 8)])
def test_forward_arguments(lib, kw):
    assert forward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(q=P + 8),
                                dict(g=P + 1), dict(beta=P + 3), dict(ldq=120), dict(ldk=132), dict(ldv=255), dict(ldv=(1 << 31) + 8)])
def test_inputs(lib, kw):
    assert forward(lib, i=inputs(**kw)) == INVALID
    assert lib.hyena_delta_step(ctypes.byref(params()), 2, 1, ctypes.byref(inputs(**kw)), P, 4, None, P, None) == INVALID


def test_sizes_beyond_the_launch(lib):
    assert forward(lib, N=1 << 25, tokens=0) == UNSUPPORTED
    assert forward(lib, N=1, tokens=(1 << 31) + 1) == UNSUPPORTED
    assert forward(lib, params(heads_v=65534, dim_v=8), N=1 << 12, tokens=1 << 12,
                   i=inputs(ldv=65534 * 8)) == UNSUPPORTED


def test_workspace(lib):
    need = lib.hyena_delta_workspace_bytes(ctypes.byref(params()), 2, 128, None)
    assert need > 0
    assert forward(lib, ws_bytes=need - 1) == WORKSPACE
    assert forward(lib, ws=None) == WORKSPACE
    # packed sequences may need one more chunk each than their tokens fill
    assert lib.hyena_delta_workspace_bytes(ctypes.byref(params()), 2, 128, P) > need
    assert lib.hyena_delta_workspace_bytes(ctypes.byref(params()), 2, 0, None) == 0
    assert lib.hyena_delta_workspace_bytes(None, 2, 128, None) == 0


def backward(lib, p=None, N=2, tokens=128, start=None, i=None, ws=P, ws_bytes=1 << 40, **kw):
    a = dict(s_in=None, dout=P, ds_out=None, dq=P, dk=P, dv=P, dg=P, dbeta=P, ds_in=None)
    a.update(kw)
    p, i = p or params(), i or inputs()
    return lib.hyena_delta_backward(ctypes.byref(p), N, tokens, start, ctypes.byref(i), a["s_in"], a["dout"], a["ds_out"],
                                    a["dq"], a["dk"], a["dv"], a["dg"], a["dbeta"], a["ds_in"], ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(N=0), dict(tokens=129), dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None),
                                dict(dg=None), dict(dbeta=None), dict(dq=P + 8), dict(s_in=P + 4), dict(ds_out=P + 4),
                                dict(ds_in=P + 4), dict(ws=P + 8), dict(i=inputs(ldq=120))])
def test_backward_arguments(lib, kw):
    assert backward(lib, **kw) == INVALID


def test_backward_workspace(lib):
    need = lib.hyena_delta_backward_workspace_bytes(ctypes.byref(params()), 2, 128, None)
    assert need > lib.hyena_delta_workspace_bytes(ctypes.byref(params()), 2, 128, None) > 0
    assert backward(lib, ws_bytes=need - 1) == WORKSPACE
    assert backward(lib, ws=None) == WORKSPACE
    assert backward(lib, params(dim_k=136), i=inputs(ldq=1 << 20, ldk=1 << 20)) == UNSUPPORTED
    assert lib.hyena_delta_backward_workspace_bytes(None, 2, 128, None) == 0
    assert lib.hyena_delta_backward_workspace_bytes(ctypes.byref(params()), 2, 127, None) == 0


def test_null_structs(lib):
    assert lib.hyena_delta_forward(None, 2, 128, None, ctypes.byref(inputs()), None, P, P, P, 1 << 40, None) == INVALID
    assert lib.hyena_delta_forward(ctypes.byref(params()), 2, 128, None, None, None, P, P, P, 1 << 40, None) == INVALID
    assert lib.hyena_delta_step(None, 2, 1, ctypes.byref(inputs()), P, 4, None, P, None) == INVALID
    assert lib.hyena_delta_step(ctypes.byref(params()), 2, 1, None, P, 4, None, P, None) == INVALID


@pytest.mark.parametrize("B,T,states,num,slots,o,want", [
    (0, 1, P, 4, None, P, INVALID), (2, 0, P, 4, None, P, INVALID), (2, 1, None, 4, None, P, INVALID),
    (2, 1, P, 0, None, P, INVALID), (2, 1, P, 1, None, P, INVALID), (2, 1, P + 4, 4, None, P, INVALID),
    (2, 1, P, 4, P + 2, P, INVALID), (2, 1, P, 4, None, None, INVALID), (2, 1, P, 4, None, P + 2, INVALID),
    (2, 1 << 25, P, 4, None, P, UNSUPPORTED), (1 << 25, 1, P, 1 << 26, None, P, UNSUPPORTED),
    (2, 1, P, 1 << 31, None, P, UNSUPPORTED)])
def test_step_arguments(lib, B, T, states, num, slots, o, want):
    assert lib.hyena_delta_step(ctypes.byref(params()), B, T, ctypes.byref(inputs()), states, num, slots, o, None) == want


def test_binding_refuses_before_the_library():
    import torch

    from fft_long_convolution_libhyena_amd import DeltaRule

    with pytest.raises(ValueError):
        DeltaRule(1, 1, 64, 64, dtype="f16")
    r = DeltaRule(1, 1, 64, 64, dtype="f32")
    q = torch.zeros(2, 3, 1, 64)
    with pytest.raises(ValueError):  # not on a GPU
        r.forward(q, q, q, torch.zeros(2, 3, 1), torch.zeros(2, 3, 1))
    with pytest.raises(ValueError):  # packed rows without offsets
        r.forward(q[0], q[0], q[0], torch.zeros(3, 1), torch.zeros(3, 1))
    with pytest.raises(ValueError):  # offsets with batched rows
        r.forward(q, q, q, torch.zeros(2, 3, 1), torch.zeros(2, 3, 1), seq_start=torch.zeros(3, dtype=torch.int64))
