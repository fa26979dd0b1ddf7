"""Backward of the gated delta rule on the GPU against the 64-bit recurrence's gradients
(autograd over tests/_delta.py) and against differences of the library's own forward.

Tolerances (relative 2-norm) count roundings, which add in squares:
  bf16 dq, dk, dbeta: the output and at most six operands (S0, dS1, u, r, W, M + M^T)
    are rounded to bf16, half a step 2^-8 each: sqrt(7) 2^-8.
  bf16 dg: the same, in sums over a chunk whose terms partly cancel: twice that.
  bf16 dv: r comes from operands of two parts (2^-16) and is rounded once: 2^-8 and 1%.
  the fp32 dstate of a bf16 call: dS, T, dU, r, P and exp(G) dO in two parts, the product
    of second parts left out: sqrt(7) 2^-16.
  fp32: two chained sums of up to 128 + 64 terms: 2 * 192 * 2^-24.
"""
import math

import pytest
import torch

import _delta as D

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate")
F32 = 2 * 192 * 2.0 ** -24
TOL = {"bf16": dict(dq=math.sqrt(7) * 2 ** -8, dk=math.sqrt(7) * 2 ** -8, dv=1.01 * 2 ** -8, dg=2 * math.sqrt(7) * 2 ** -8,
                    dbeta=math.sqrt(7) * 2 ** -8, dstate=math.sqrt(7) * 2 ** -16),
       "f32": {n: F32 for n in NAMES}}


def gpu(x):
    return None if x is None else x.cuda()


def run(d, dtype, dims, scale=None, use_state=True, use_dstate=True, seq_start=None):
    from fft_long_convolution_libhyena_amd import DeltaRule

    lens = d["lens"]
    start = D.starts(lens, "cuda") if seq_start is None else seq_start
    return DeltaRule(*dims, dtype=dtype).backward(
        *(d[n].cuda() for n in ("q", "k", "v", "g", "beta", "do")), state=gpu(d["state"]) if use_state else None,
        dstate_out=gpu(d["dstate"]) if use_dstate else None, scale=scale, seq_start=start)


def check(got, want, dtype):
    for name, x, y in zip(NAMES, got, want):
        assert x.shape == y.shape
        if y.numel():
            assert D.rel(x, y) <= TOL[dtype][name], (name, D.rel(x, y))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [
    ([1], 1, 1, 8, 8),
    ([64], 2, 2, 128, 128),
    ([65, 0, 1], 2, 4, 128, 128),
    ([200, 64, 3, 129], 1, 3, 72, 40),
    ([130], 2, 2, 40, 256),
    ([333, 70], 1, 1, 64, 104),
    ([0], 1, 1, 64, 64),
])
def test_gradients(lens, hk, hv, dk, dv, dtype):
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=len(lens) + dk)
    check(run(d, dtype, (hk, hv, dk, dv)), D.backward(d, dk ** -0.5), dtype)


# Long enough to be cut into pieces, with slow decays and weak writes so that states and their
# gradients reach far. Each carry adds the roundings of two operands (2^-16) or sums of 128
# terms, in the state's scan and in its gradient's; fp32 states also sum over ~55 chunks.
LONG = {"bf16": dict(TOL["bf16"], dstate=math.sqrt(7 + 2 * 2) * 2 ** -16),
        "f32": {n: 2 * (192 + 2 * 128 + 55) * 2.0 ** -24 for n in NAMES}}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [
    ([3500], 1, 2, 64, 72),
    ([2050], 1, 1, 128, 128),
    ([1700, 0, 33], 1, 1, 40, 96),
    ([70, 2500, 1999], 2, 2, 128, 40),
])
def test_gradients_cut_into_pieces(lens, hk, hv, dk, dv, dtype):
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=sum(lens), decay=1e-3)
    d["beta"] = d["beta"] * 0.0625
    got, again = (run(d, dtype, (hk, hv, dk, dv)) for _ in range(2))
    for name, x, y, z in zip(NAMES, got, D.backward(d, dk ** -0.5), again):
        assert D.rel(x, y) <= LONG[dtype][name], (name, D.rel(x, y))
        assert bool((x == z).all()), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("use_state,use_dstate", [(False, False), (False, True), (True, False)])
def test_without_states(dtype, use_state, use_dstate):
    d = D.make([140, 63], 2, 2, 64, 64, dtype, seed=3)
    check(run(d, dtype, (2, 2, 64, 64), 0.6, use_state, use_dstate), D.backward(d, 0.6, use_state, use_dstate), dtype)


def test_zero_strength_and_resets_have_their_gradients():
    """beta = 0 writes nothing but has a gradient; a reset passes none on."""
    d = D.make([150], 1, 2, 64, 64, "f32", seed=5)
    d["beta"][10:90, 0] = 0
    d["g"][::17, 1] = -300.0
    got, want = run(d, "f32", (1, 2, 64, 64)), D.backward(d, 64 ** -0.5)
    check(got, want, "f32")
    assert float(got[4][20:80, 0].abs().max()) > 0


def test_gate_gradients_of_carried_states():
    """With nothing written and no outputs' gradient, dg is <dS, S> decayed, here a tenth of
    what it is for unrelated dS and S. Both enter in two bf16 parts, off by 2^-16 at most in
    each product (errors add in squares; three, with the product of second parts), and the
    result is rounded once."""
    lens, hv, dk, dv = [70, 5, 64], 2, 64, 64
    d = D.make(lens, 1, hv, dk, dv, "bf16", seed=41)
    d["beta"].zero_()
    d["do"].zero_()
    s, ds = d["state"], d["dstate"]
    along = (s * ds).sum((2, 3), keepdim=True) / (ds * ds).sum((2, 3), keepdim=True)
    size = (s * ds).square().sum((2, 3)).sqrt()
    d["state"] = s + ds * (0.1 * (size / (ds * ds).sum((2, 3)))[:, :, None, None] - along)
    got = run(d, "bf16", (1, hv, dk, dv))[3].cpu().double()
    want = D.backward(d, dk ** -0.5)[3]
    spread = (d["state"].double() * d["dstate"].double()).square().sum((2, 3)).sqrt()
    bound = torch.cat([spread[i].expand(n, hv) for i, n in enumerate(lens)]) * 3 ** 0.5 * 2.0 ** -16
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + bound).all())


def test_batch_layout_matches_packed():
    from fft_long_convolution_libhyena_amd import DeltaRule

    B, T, dims = 3, 70, (2, 4, 64, 64)
    d = D.make([T] * B, *dims, "bf16", seed=6)
    packed = run(d, "bf16", dims, use_state=False, use_dstate=False)
    g = [d[n].cuda().unflatten(0, (B, T)) for n in ("q", "k", "v", "g", "beta", "do")]
    out = DeltaRule(*dims).backward(*g)
    for x, y in zip(out[:5], packed[:5]):
        assert torch.equal(x.flatten(0, 1), y)
    assert torch.equal(out[5], packed[5])


def test_repeatable_and_strided_inputs():
    from fft_long_convolution_libhyena_amd import DeltaRule

    hk, hv, dk, dv = 2, 4, 64, 64
    lens = [90, 200]
    d = D.make(lens, hk, hv, dk, dv, "bf16", seed=7, packed_rows=True)
    q, k, v = d["rows"].cuda().split([hk * dk, hk * dk, hv * dv], 1)
    r = DeltaRule(hk, hv, dk, dv)
    args = (q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv)), d["g"].cuda(), d["beta"].cuda(),
            d["do"].cuda())
    a = r.backward(*args, seq_start=D.starts(lens, "cuda"))
    b = run(d, "bf16", (hk, hv, dk, dv), use_state=False, use_dstate=False)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_rows_outside_sequences_stay():
    """Gradients of rows that belong to no sequence are not written."""
    dims = (1, 1, 64, 64)
    d = D.make([50, 40], *dims, "bf16", seed=8)
    from fft_long_convolution_libhyena_amd import DeltaRule

    r = DeltaRule(*dims)
    x = {}
    for n in ("q", "k", "v", "g", "beta", "do"):
        t = torch.full((140, *d[n].shape[1:]), float("nan"), dtype=torch.bfloat16)
        t[10:100] = d[n]
        x[n] = t.cuda()
    start = torch.tensor([10, 60, 100], device="cuda")
    inputs = r._inputs(x["q"], x["k"], x["v"], x["g"], x["beta"], (140,), x["q"].device)
    outs = [torch.full_like(x[n], 7.0) for n in ("q", "k", "v", "g", "beta")]
    ws = torch.empty(r.backward_workspace_bytes(2, 140, True), dtype=torch.uint8, device="cuda")
    st = r.lib.hyena_delta_backward(r._params(None), 2, 140, start.data_ptr(), inputs, None,
                                    x["do"].data_ptr(), None, *(o.data_ptr() for o in outs), None, ws.data_ptr(), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want = D.backward(d, 64 ** -0.5, use_state=False, use_dstate=False)
    check([o[10:100] for o in outs], want[:5], "bf16")
    for o in outs:
        assert bool((o[:10] == 7).all()) and bool((o[100:] == 7).all())


def test_against_differences():
    """dq, dk, dv, dg, dbeta along a random direction against the fp32 forward's own
    difference quotient (central, error of second order in the step)."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    dims = (1, 2, 64, 64)
    d = D.make([130], *dims, "f32", seed=9)
    r = DeltaRule(*dims, dtype="f32")
    x = [d[n].cuda()[None] for n in ("q", "k", "v", "g", "beta")]
    do = d["do"].cuda()[None]
    grads = r.backward(*x, do)[:5]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i in range(5):
        way = torch.randn(x[i].shape, device="cuda", generator=gen)
        want = float((grads[i].double() * way).sum())

        def loss(step):
            y = list(x)
            y[i] = x[i] + step * way
            return float((r.forward(*y)[0].double() * do).sum())

        # fp32 outputs are off by about 192 * 2^-24 of sum |o do| <= sum |grad way| / step scale;
        # the step balances that against the second-order term
        h = 2.0 ** -8
        got = (loss(h) - loss(-h)) / (2 * h)
        size = float((grads[i].double().abs() * way.abs()).sum())
        assert abs(got - want) <= 0.01 * size


def test_captured_backward_replays():
    from fft_long_convolution_libhyena_amd import DeltaRule

    dims = (1, 2, 64, 64)
    d = D.make([100, 100], *dims, "bf16", seed=10)
    x = [d[n].cuda().unflatten(0, (2, 100)) for n in ("q", "k", "v", "g", "beta", "do")]
    r = DeltaRule(*dims)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.backward(*x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = r.backward(*x)
    for i in range(3):
        x[5].mul_(0.5 + i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, r.backward(*x)):
            assert torch.equal(a, b)
