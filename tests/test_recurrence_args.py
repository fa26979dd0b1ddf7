"""Refusals of the gated recurrence's entry points, found on the host before any device call."""
import ctypes

import pytest
import torch

from fft_long_convolution_libhyena_amd import GatedRecurrence, binding
from fft_long_convolution_libhyena_amd.binding import RecurrenceInputsStruct, RecurrenceParamsStruct

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 4096  # stands for a device address; never followed


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def params(**kw):
    d = dict(dim=256, dtype=1, clear=0, rate=P)
    d.update(kw)
    return RecurrenceParamsStruct(*(d[n] for n, _ in RecurrenceParamsStruct._fields_))


def inputs(**kw):
    d = dict(x=P, ldx=256, r=P, ldr=256, i=P, ldi=768)
    d.update(kw)
    return RecurrenceInputsStruct(*(d[n] for n, _ in RecurrenceInputsStruct._fields_))


def forward(lib, p=None, N=2, tokens=128, start=None, i=None, s_in=None, y=P, s_out=P, carries=None, ws=P, ws_bytes=1 << 40):
    return lib.hyena_recurrence_forward(ctypes.byref(p or params()), N, tokens, start, ctypes.byref(i or inputs()), s_in, y, s_out,
                                        carries, ws, ws_bytes, None)


def backward(lib, p=None, N=2, tokens=128, start=None, i=None, ws=P, ws_bytes=1 << 40, **kw):
    a = dict(s_in=None, carries=None, dy=P, ds=None, dx=P, dr=P, di=P, drate=P, ds_in=None)
    a.update(kw)
    return lib.hyena_recurrence_backward(ctypes.byref(p or params()), N, tokens, start, ctypes.byref(i or inputs()),
                                         *(a[k] for k in ("s_in", "carries", "dy", "ds", "dx", "dr", "di", "drate", "ds_in")), ws,
                                         ws_bytes, None)


def step(lib, p=None, B=2, T=1, i=None, states=P, num=4, slots=None, y=P):
    return lib.hyena_recurrence_step(ctypes.byref(p or params()), B, T, ctypes.byref(i or inputs()), states, num, slots, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dim=0), INVALID), (dict(dtype=5), INVALID), (dict(rate=None), INVALID), (dict(rate=P + 2), INVALID),
    (dict(dim=12), UNSUPPORTED), (dict(dim=(1 << 20) + 8), UNSUPPORTED)])
def test_params(lib, kw, want):
    p, i = params(**kw), inputs(ldx=1 << 21, ldr=1 << 21, ldi=1 << 21)
    assert forward(lib, p, i=i) == want and backward(lib, p, i=i) == want and step(lib, p, i=i) == want
    assert lib.hyena_recurrence_workspace_bytes(ctypes.byref(p), 2, 128, None) == 0
    assert lib.hyena_recurrence_backward_workspace_bytes(ctypes.byref(p), 2, 128, None, None) == 0


@pytest.mark.parametrize("kw", [dict(x=None), dict(r=None), dict(i=None), dict(x=P + 8), dict(ldx=248), dict(ldr=260),
                                dict(ldi=(1 << 31) + 8)])
def test_inputs(lib, kw):
    assert forward(lib, i=inputs(**kw)) == INVALID and backward(lib, i=inputs(**kw)) == INVALID
    assert step(lib, i=inputs(**kw)) == INVALID


def test_stride_of_whole_sequences(lib):
    i = inputs(ldx=(1 << 22) + 8)
    assert forward(lib, i=i) == INVALID and backward(lib, i=i) == INVALID


def test_sizes(lib):
    for kw in (dict(N=0), dict(tokens=-1), dict(tokens=127), dict(start=P + 4)):
        assert forward(lib, **kw) == INVALID and backward(lib, **kw) == INVALID
    for kw in (dict(N=1 << 25, tokens=0), dict(N=1, tokens=(1 << 31) - 127), dict(N=1, tokens=(1 << 31) - 256)):
        assert forward(lib, **kw) == UNSUPPORTED and backward(lib, **kw) == UNSUPPORTED
    assert lib.hyena_recurrence_workspace_bytes(ctypes.byref(params()), 2, 0, None) == 0
    assert lib.hyena_recurrence_forward(None, 2, 128, None, ctypes.byref(inputs()), None, P, P, None, P, 1 << 40, None) == INVALID
    assert lib.hyena_recurrence_forward(ctypes.byref(params()), 2, 128, None, None, None, P, P, None, P, 1 << 40, None) == INVALID


def test_arrays(lib):
    for kw in (dict(y=None), dict(y=P + 8), dict(s_in=P + 4), dict(s_out=P + 8), dict(carries=P + 4)):
        assert forward(lib, **kw) == INVALID
    for kw in (dict(dy=None), dict(dx=None), dict(dr=None), dict(di=P + 8), dict(drate=None), dict(drate=P + 2), dict(s_in=P + 4),
               dict(ds=P + 4), dict(ds_in=P + 8), dict(carries=P + 4)):
        assert backward(lib, **kw) == INVALID


def test_workspace(lib):
    need = lib.hyena_recurrence_workspace_bytes(ctypes.byref(params()), 1, 4096, None)
    if need:
        assert forward(lib, N=1, tokens=4096, ws_bytes=need - 1) == WORKSPACE and forward(lib, N=1, tokens=4096, ws=None) == WORKSPACE
        assert forward(lib, N=1, tokens=4096, ws=P + 8) == INVALID
    need = lib.hyena_recurrence_backward_workspace_bytes(ctypes.byref(params()), 2, 128, None, None)
    assert need >= lib.hyena_recurrence_backward_workspace_bytes(ctypes.byref(params()), 2, 128, None, P) > 0
    assert backward(lib, ws_bytes=need - 1) == WORKSPACE and backward(lib, ws=None) == WORKSPACE
    assert backward(lib, ws=P + 8) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(states=None), INVALID), (dict(num=0), INVALID), (dict(num=1), INVALID),
    (dict(states=P + 4), INVALID), (dict(slots=P + 2), INVALID), (dict(y=None), INVALID), (dict(y=P + 8), INVALID),
    (dict(T=1 << 25), UNSUPPORTED), (dict(B=1 << 25, num=1 << 26), UNSUPPORTED), (dict(num=1 << 31), UNSUPPORTED),
    (dict(B=1 << 24, num=1 << 24), UNSUPPORTED)])
def test_step(lib, kw, want):
    assert step(lib, **kw) == want


@pytest.fixture
def launches(monkeypatch):
    """The calls that would have been launched: (name, arguments); CPU tensors stand for the device's."""
    seen = []
    monkeypatch.setattr(binding, "_gpu_of", lambda t, name: t.device)
    monkeypatch.setattr(binding, "_launch", lambda torch, name, fn, device, *args: seen.append((name, args)))
    return seen


def test_binding(launches):
    with pytest.raises(ValueError):
        GatedRecurrence(16, torch.ones(16), dtype="f16")
    for rate in (None, torch.ones(8), torch.ones(16).double(), torch.ones(32)[::2]):
        with pytest.raises(ValueError):
            GatedRecurrence(16, rate)
    m = GatedRecurrence(16, torch.ones(16), dtype="f32")
    x = torch.zeros(2, 300, 16)
    start = torch.tensor([0, 300], dtype=torch.int64)
    for call in (lambda: m.forward(x[0], x[0], x[0]), lambda: m.forward(x, x, x, seq_start=start),
                 lambda: m.forward(x, x.bfloat16(), x), lambda: m.forward(x, x[:, :299], x), lambda: m.forward(x, None, x),
                 lambda: m.forward(x, x, x, state=torch.zeros(3, 16)), lambda: m.forward(x, x, x, carries=torch.zeros(9, 16)),
                 lambda: m.forward(x, x, x, carries=torch.zeros(8, 16).double()),
                 lambda: m.forward(x, x, torch.zeros(2, 300, 32)[..., ::2]), lambda: m.forward(x, x, torch.zeros(2, 300, 20)[..., 2:18]),
                 lambda: m.forward(x[0], x[0], x[0], seq_start=start.int()), lambda: m.forward(x[0], x[0], x[0], seq_start=start[:1]),
                 lambda: m.backward(x, x, x, x[0]), lambda: m.backward(x, x, x, x, dstate_out=torch.zeros(2, 8)),
                 lambda: m.step(x, x, x, torch.zeros(2, 8)), lambda: m.step(x, x, x, torch.zeros(2, 16), slots=torch.zeros(2)),
                 lambda: m.forward(x, x, x, workspace=torch.empty(1, dtype=torch.uint8).expand(1 << 20)),
                 lambda: m.backward(x, x, x, x, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError):
            call()
    assert not launches
    rows = torch.zeros(2, 300, 52)  # views with one stride between tokens
    m.forward(rows[..., :16], rows[..., 16:32], rows[..., 32:48], carries=torch.zeros(m.carries_shape(600)))
    name, args = launches[-1]
    got = ctypes.cast(args[4], ctypes.POINTER(RecurrenceInputsStruct)).contents
    assert name == "hyena_recurrence_forward" and args[1:3] == (2, 600) and (got.ldx, got.ldr, got.ldi) == (52, 52, 52)
    assert got.r - got.x == 64
