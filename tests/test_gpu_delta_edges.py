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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_where_a_value_that_is_not_finite_shows(name, bad, dtype):
    """q's in its token; v's in its column from the token on, the others' in their value heads
    from there on: earlier tokens, other heads and other sequences keep their bits."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    hk, hv, dk, dv, lens = 2, 4, 64, 40, [200, 90]
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=17)
    r = DeltaRule(hk, hv, dk, dv, dtype)

    def call():
        return r.forward(*(d[n].cuda() for n in ("q", "k", "v", "g", "beta")), state=d["state"].cuda(), seq_start=D.starts(lens, "cuda"))

    o0, s0 = call()
    d[name][100, 1, ...] = bad  # head 1, token 36 of the second chunk
    if name == "v":
        d[name][100, 1, :] = 0.5
        d[name][100, 1, 3] = bad
    o, s = call()
    heads = {"q": [2, 3], "k": [2, 3]}.get(name, [1])
    same = torch.ones_like(o, dtype=torch.bool)
    if name == "q":
        same[100, heads] = False
    elif name == "v":
        same[100:200, 1] = False
    else:
        same[100:200, heads] = False
    assert torch.equal(o[same], o0[same]) and bool(torch.isfinite(o[same]).all())
    if name == "v":  # its other columns were changed here, but are finite
        fine = torch.isfinite(o[64:200, 1])
        assert bool(fine[..., [i for i in range(dv) if i != 3]].all()) and not bool(fine[36:, 3].any())
    others = [i for i in range(hv) if i not in heads]
    assert torch.equal(s[1], s0[1]) and torch.equal(s[0, others], s0[0, others])
    if name != "g" or bad != float("inf"):  # exp(inf) may meet a zero or an infinity first
        assert not bool(torch.isfinite(o[100, heads] if name != "v" else o[100, 1, 3]).all())
    if name == "q":
        assert torch.equal(s, s0)
    elif name == "v":
        keep = [i for i in range(dv) if i != 3]
        assert bool(torch.isfinite(s[0, 1][:, keep]).all()) and not bool(torch.isfinite(s[0, 1][:, 3]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_no_sequence_have_no_gradient(dtype):
    """A padded packed batch, as a captured training step has it: the rows around the sequences
    hold anything and come back as zeros."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    dims, lens, front, back = (1, 2, 64, 72), [70, 0, 33], 5, 60
    d = D.make(lens, *dims, dtype, seed=18)
    x = []
    for n in ("q", "k", "v", "g", "beta", "do"):
        t = torch.full((front + sum(lens) + back, *d[n].shape[1:]), float("nan"), dtype=d[n].dtype)
        t[front:-back] = d[n]
        x.append(t.cuda())
    start = D.starts(lens, "cuda") + front
    r = DeltaRule(*dims, dtype=dtype)
    torch.use_deterministic_algorithms(True, warn_only=True)  # torch.empty gives NaN
    try:
        o, _ = r.forward(*x[:5], seq_start=start)
        grads = r.backward(*x, seq_start=start)[:5]
    finally:
        torch.use_deterministic_algorithms(False)
    plain = r.backward(*(d[n].cuda() for n in ("q", "k", "v", "g", "beta", "do")), seq_start=D.starts(lens, "cuda"))[:5]
    for t in (o, *grads):
        assert bool((t[:front] == 0).all()) and bool((t[-back:] == 0).all())
    for a, b in zip(grads, plain):
        assert torch.equal(a[front:-back], b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 40), (128, 128), (40, 72)])
@pytest.mark.parametrize("at", [0, 5, 36, 63])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_what_is_not_finite_reaches_no_earlier_token(name, at, dk, dv, dtype):
    """The mixer is causal: tokens in front of a NaN or an infinity keep their bits, also those of
    its own chunk of 64, and no token behind it looks as if nothing had happened."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    hk, hv, lens = 1, 2, [170, 64]
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=19)
    r = DeltaRule(hk, hv, dk, dv, dtype)

    def call():
        return r.forward(*(d[n].cuda() for n in ("q", "k", "v", "g", "beta")), state=d["state"].cuda(), seq_start=D.starts(lens, "cuda"))

    o0, s0 = call()
    for bad in (float("nan"), float("inf"), float("-inf")):
        if name == "g" and bad == float("-inf"):
            continue  # a reset, and finite
        keep = d[name].clone()
        t = 64 + at
        d[name][t] = bad
        if name == "v":
            d[name][t, :, 1:] = keep[t, :, 1:]
        o, s = call()
        d[name] = keep
        assert torch.equal(o[:t], o0[:t]), bad
        assert torch.equal(o[170:], o0[170:]) and torch.equal(s[1], s0[1])
        if name == "q":
            assert torch.equal(o[t + 1:], o0[t + 1:]) and not bool(torch.isfinite(o[t]).any()) and torch.equal(s, s0)
        elif name == "v":
            assert torch.equal(o[..., 1:], o0[..., 1:]) and torch.equal(s[..., 1:], s0[..., 1:])
            assert not bool(torch.isfinite(o[t:170, :, 0]).any()) and not bool(torch.isfinite(s[0, ..., 0]).any())
        else:
            assert not bool(torch.isfinite(o[t:170]).any()) and not bool(torch.isfinite(s[0]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["k", "v"])
def test_what_is_not_finite_reaches_no_earlier_token_of_a_cut_sequence(name, dtype):
    from fft_long_convolution_libhyena_amd import DeltaRule

    lens, at = [2300], 1100
    d = D.make(lens, 1, 2, 64, 64, dtype, seed=20, decay=1e-2)
    r = DeltaRule(1, 2, 64, 64, dtype)
    call = lambda: r.forward(*(d[n].cuda() for n in ("q", "k", "v", "g", "beta")), state=d["state"].cuda(),  # noqa: E731
                             seq_start=D.starts(lens, "cuda"))
    o0, _ = call()
    d[name][at, :, 0] = float("nan")
    o, s = call()
    assert torch.equal(o[:at], o0[:at])
    after = slice(0, 1) if name == "v" else slice(None)
    assert bool(o[at:, :, after].isnan().all()) and bool(s[..., after].isnan().all())
    if name == "v":
        assert torch.equal(o[..., 1:], o0[..., 1:])
