"""Refusals of the residual norm's entry points and of the head norm's with several axes, found on the
host before any device call."""
import ctypes

import pytest
import torch

from fft_long_convolution_libhyena_amd import QKNorm, ResidualNorm, binding
from fft_long_convolution_libhyena_amd.binding import QKNormParamsStruct, ResidualNormParamsStruct

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 4096  # stands for a device address; never followed


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def params(**kw):
    d = dict(dim=256, dtype=1, residual_dtype=0, block=0, eps=1e-6, w=P)
    d.update(kw)
    return ResidualNormParamsStruct(*(d[n] for n, _ in ResidualNormParamsStruct._fields_))


def forward(lib, p=None, rows=3, x=P, ldx=256, res=P, ldr=256, y=P, scales=None, s=P):
    return lib.hyena_residual_norm_forward(ctypes.byref(p or params()), rows, x, ldx, res, ldr, y, scales, s, None)


def backward(lib, p=None, rows=3, s=P, lds=256, dy=P, ds=P, dx=P, dres=P, dw=P, ws=P, ws_bytes=1 << 40):
    return lib.hyena_residual_norm_backward(ctypes.byref(p or params()), rows, s, lds, dy, ds, dx, dres, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dim=0), INVALID), (dict(dtype=3), INVALID), (dict(residual_dtype=3), INVALID), (dict(block=64), INVALID),
    (dict(block=-128), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(w=P + 2), INVALID), (dict(dtype=0, residual_dtype=1), UNSUPPORTED), (dict(dim=20), UNSUPPORTED),
    (dict(dim=16392), UNSUPPORTED)])
def test_params(lib, kw, want):
    p = params(**kw)
    assert forward(lib, p, ldx=1 << 20, ldr=1 << 20) == want and backward(lib, p, lds=1 << 20) == want
    assert lib.hyena_residual_norm_backward_workspace_bytes(ctypes.byref(p), 3) == 0


def test_arguments(lib):
    for kw in (dict(rows=-1), dict(x=None), dict(y=None), dict(x=P + 8), dict(res=P + 4), dict(y=P + 8), dict(s=P + 2), dict(scales=P + 2),
               dict(ldx=248), dict(ldx=260), dict(ldr=258), dict(ldx=(1 << 31) + 8)):
        assert forward(lib, **kw) == INVALID, kw
    for kw in (dict(rows=-1), dict(s=None), dict(dy=None), dict(s=P + 8), dict(dy=P + 8), dict(ds=P + 8), dict(dx=P + 8), dict(dres=P + 8),
               dict(dw=P + 2), dict(lds=252 - 4), dict(lds=258), dict(dx=None, dres=None, dw=None), dict(ws=P + 8)):
        assert backward(lib, **kw) == INVALID, kw
    assert forward(lib, rows=(1 << 31) + 1) == UNSUPPORTED and backward(lib, rows=(1 << 31) + 1) == UNSUPPORTED
    need = lib.hyena_residual_norm_backward_workspace_bytes(ctypes.byref(params()), 3)
    assert need > 0 and backward(lib, ws_bytes=need - 1) == WORKSPACE and backward(lib, ws=None) == WORKSPACE
    assert lib.hyena_residual_norm_backward_workspace_bytes(ctypes.byref(params()), 0) == 0
    assert forward(lib, rows=0, x=None, res=None, y=None, s=None) == OK
    assert lib.hyena_residual_norm_forward(None, 3, P, 256, P, 256, P, None, P, None) == INVALID
    assert lib.hyena_residual_norm_backward(None, 3, P, 256, P, P, P, P, P, P, 1 << 30, None) == INVALID


def test_axes(lib):
    def call(axis=P, axes=3, rot=16, null=False):
        p = QKNormParamsStruct(4, 2, 64, rot, 0, 0, 1, 1e-6, P, P, P)
        p = None if null else ctypes.byref(p)
        f = lib.hyena_qk_norm_axes_forward(p, axis, axes, 3, P, 248, P, 128, P, P, P, None)  # ldq is refused last
        b = lib.hyena_qk_norm_axes_backward(p, axis, axes, 3, P, 248, P, 128, P, P, P, P, P, P, P, P, 1 << 30, None)
        assert f == b
        return f

    assert call(axes=0) == INVALID and call(axis=None) == INVALID and call(axis=P + 2) == INVALID and call(null=True) == INVALID
    assert call(axes=9) == UNSUPPORTED
    assert call() == INVALID  # only the stride is left to refuse


@pytest.fixture
def launches(monkeypatch):
    """The calls that would have been launched: (name, arguments); CPU tensors stand for the device's."""
    seen = []
    monkeypatch.setattr(binding, "_gpu_of", lambda t, name: t.device)
    monkeypatch.setattr(binding, "_launch", lambda torch, name, fn, device, *args: seen.append((name, args)))
    return seen


def test_binding(launches):
    for kw in (dict(dtype="f16"), dict(block=64), dict(w=torch.ones(8)), dict(w=torch.ones(16).double())):
        with pytest.raises(ValueError):
            ResidualNorm(16, **kw)
    m = ResidualNorm(16, torch.ones(16), wide_residual=True)
    x, r = torch.zeros(4, 16).bfloat16(), torch.zeros(4, 16)
    for call in (lambda: m.forward(r, r), lambda: m.forward(x, x), lambda: m.forward(x, r[:3]), lambda: m.forward(x, r, y=r),
                 lambda: m.forward(x[0], r[0]), lambda: m.backward(x, x), lambda: m.backward(r, r), lambda: m.backward(r, x, x),
                 lambda: m.backward(r, x, r, workspace=torch.empty(1, dtype=torch.uint8).expand(1 << 20))):
        with pytest.raises(ValueError):
            call()
    assert not launches
    y, s = m.forward(x)
    assert y.dtype == torch.bfloat16 and s.dtype == torch.float32 and launches[-1][1][4] is None
    same = ResidualNorm(16, None, bits8=True, block=128)
    y, scales, s = same.forward(x)
    assert s is x and y.dtype == torch.float8_e4m3fn and scales.shape == (4, 1)
    dx, dres, dw = same.backward(x, x)
    assert dres is dx and dw is None and launches[-1][1][-2:] == (None, 0)


def test_head_norm_binding_with_axes(launches):
    freq, axis = torch.ones(8), torch.zeros(8, dtype=torch.int32)
    for kw in (dict(freq=None, axis=axis), dict(freq=freq, axis=axis.long()), dict(freq=freq, axis=axis[:4]),
               dict(freq=freq, axis=torch.zeros(16, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError):
            QKNorm(2, 1, 64, **kw)
    m = QKNorm(2, 1, 64, freq=freq, axis=axis)
    q, k = torch.zeros(6, 2, 64).bfloat16(), torch.zeros(6, 1, 64).bfloat16()
    for pos in (None, torch.zeros(6, dtype=torch.int64), torch.zeros(5, 3, dtype=torch.int64), torch.zeros(6, 3)):
        with pytest.raises(ValueError):
            m.forward(q, k, pos)
    assert not launches
    m.forward(q, k, torch.zeros(6, 3, dtype=torch.int64))
    name, args = launches[-1]
    assert name == "hyena_qk_norm_axes_forward" and args[1:4] == (axis.data_ptr(), 3, 6)
    QKNorm(2, 1, 64, freq=freq).forward(q, k, torch.zeros(6, dtype=torch.int64))
    assert launches[-1][0] == "hyena_qk_norm_forward" and launches[-1][1][1] == 6
    m.backward(q, k, q, k, torch.zeros(6, 3, dtype=torch.int64))
    assert launches[-1][0] == "hyena_qk_norm_axes_backward" and launches[-1][1][1:4] == (axis.data_ptr(), 3, 6)
