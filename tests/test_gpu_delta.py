"""Gated delta rule on the GPU against the plain 64-bit recurrence (tests/_delta.py).

Tolerances (relative 2-norm) count roundings, which add in squares:
  bf16 outputs: the output, the state, u and P are each rounded to bf16 once, half a
    step 2^-8 each: sqrt(4) 2^-8.
  the fp32 state of a bf16 call: state, T, residual and written values enter as two
    bf16 parts, and the product of second parts is left out: 5 errors of 2^-16.
  fp32: sums of up to 128 + 64 terms, each addition off by at most 2^-24: 192 * 2^-24.
"""
import math

import pytest
import torch

import _delta as D

pytestmark = pytest.mark.gpu

TOL_O = {"bf16": 2 * 2.0 ** -8, "f32": 192 * 2.0 ** -24}
TOL_S = {"bf16": math.sqrt(5) * 2.0 ** -16, "f32": 192 * 2.0 ** -24}


def rule(d, hk, hv, dk, dv, dtype):
    from fft_long_convolution_libhyena_amd import DeltaRule

    return DeltaRule(hk, hv, dk, dv, dtype)


def on_gpu(d):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in d.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [
    ([1], 1, 1, 8, 8),
    ([63], 1, 2, 64, 64),
    ([64], 2, 2, 128, 128),
    ([65, 0, 1], 2, 4, 128, 128),
    ([200, 64, 3, 129], 1, 3, 72, 40),
    ([130], 2, 2, 40, 256),
    ([0], 1, 1, 64, 64),
    ([333, 70], 3, 3, 96, 104),
])
def test_forward_packed(lens, hk, hv, dk, dv, dtype):
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=len(lens) + dk)
    g = on_gpu(d)
    r = rule(d, hk, hv, dk, dv, dtype)
    o, s = r.forward(g["q"], g["k"], g["v"], g["g"], g["beta"], state=g["state"], seq_start=D.starts(lens, "cuda"))
    ro, rs = D.forward(d, dk ** -0.5)
    assert D.rel(s, rs) <= TOL_S[dtype]
    if sum(lens):
        assert D.rel(o, ro) <= TOL_O[dtype]
    assert o.dtype == d["q"].dtype and s.dtype == torch.float32


# Sequences long enough to be cut into pieces, slow decays and weak writes so that the state
# in front of a piece reaches far into it. Cutting adds, per carry, the roundings of M's and
# S's operands (two of 2^-16) or sums of 128 terms more; fp32 states also sum over ~55 chunks.
TOL_LONG = {"bf16": math.sqrt(5 + 2 * 2) * 2.0 ** -16, "f32": (192 + 2 * 128 + 55) * 2.0 ** -24}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,hk,hv,dk,dv", [
    ([3500], False, 1, 1, 64, 64),
    ([3500, 3500], False, 1, 2, 40, 72),
    ([4100], True, 2, 2, 128, 96),
    ([3201, 0, 70], True, 1, 2, 128, 40),
    ([1, 3300, 3137], True, 1, 1, 72, 128),
])
def test_forward_cut_into_pieces(lens, packed, hk, hv, dk, dv, dtype):
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=sum(lens), decay=1e-3)
    d["beta"] = d["beta"] * 0.0625
    g = on_gpu(d)
    r = rule(d, hk, hv, dk, dv, dtype)
    if packed:
        args, start = [g[n] for n in ("q", "k", "v", "g", "beta")], D.starts(lens, "cuda")
    else:
        args, start = [g[n].unflatten(0, (len(lens), lens[0])) for n in ("q", "k", "v", "g", "beta")], None
    o, s = r.forward(*args, state=g["state"], seq_start=start)
    o2, s2 = r.forward(*args, state=g["state"], seq_start=start)
    ro, rs = D.forward(d, dk ** -0.5)
    assert D.rel(s, rs) <= TOL_LONG[dtype]
    assert D.rel(o.reshape(ro.shape), ro) <= max(TOL_O[dtype], TOL_LONG[dtype])
    assert bool((o == o2).all()) and bool((s == s2).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cut_sequences_keep_their_state_in_place(dtype):
    """A cut sequence's first piece and its last both meet the state's memory."""
    lens, hk, hv, dk, dv = [2000, 1900], 1, 2, 64, 64
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=12, decay=1e-3)
    d["beta"] = d["beta"] * 0.0625
    g = on_gpu(d)
    args, start = [g[n] for n in ("q", "k", "v", "g", "beta")], D.starts(lens, "cuda")
    r = rule(d, hk, hv, dk, dv, dtype)
    o, s = r.forward(*args, state=g["state"], seq_start=start)
    st = g["state"].clone()
    o2, s2 = r.forward(*args, state=st, seq_start=start, state_out=st)
    ro, rs = D.forward(d, dk ** -0.5)
    assert s2.data_ptr() == st.data_ptr()
    assert bool((o == o2).all()) and bool((s == s2).all())
    assert D.rel(s, rs) <= TOL_LONG[dtype] and D.rel(o, ro) <= max(TOL_O[dtype], TOL_LONG[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 100), (3, 257), (2, 0)])
def test_forward_batch_without_state(B, T, dtype):
    hk, hv, dk, dv = 2, 4, 64, 72
    d = D.make([T] * B, hk, hv, dk, dv, dtype, seed=B + T)
    g = {n: x.cuda().unflatten(0, (B, T)) for n, x in d.items() if n in ("q", "k", "v", "g", "beta")}
    o, s = rule(d, hk, hv, dk, dv, dtype).forward(g["q"], g["k"], g["v"], g["g"], g["beta"], scale=0.7)
    ro, rs = D.forward(d, 0.7, use_state=False)
    assert o.shape == (B, T, hv, dv)
    if T:
        assert D.rel(o.flatten(0, 1), ro) <= TOL_O[dtype]
    assert D.rel(s, rs) <= TOL_S[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_strided_rows_and_in_place_state(dtype):
    hk, hv, dk, dv = 2, 4, 64, 64
    lens = [70, 33]
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=5, packed_rows=True)
    rows = d["rows"].cuda()
    q, k, v = rows.split([hk * dk, hk * dk, hv * dv], 1)
    q, k, v = q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv))
    assert not q.is_contiguous()
    st = d["state"].cuda()
    o, s = rule(d, hk, hv, dk, dv, dtype).forward(q, k, v, d["g"].cuda(), d["beta"].cuda(), state=st,
                                                  seq_start=D.starts(lens, "cuda"), state_out=st)
    ro, rs = D.forward(d, dk ** -0.5)
    assert s.data_ptr() == st.data_ptr()
    assert D.rel(o, ro) <= TOL_O[dtype] and D.rel(s, rs) <= TOL_S[dtype]


def test_other_rows_stay_untouched_and_nan_does_not_leak():
    """Rows in front of, behind and between sequences are neither read nor written."""
    hk, hv, dk, dv = 1, 2, 64, 64
    d = D.make([50, 40], hk, hv, dk, dv, "bf16", seed=8)
    pad = {}
    for n in ("q", "k", "v", "g", "beta"):
        x = torch.full((140, *d[n].shape[1:]), float("nan"), dtype=d[n].dtype)
        x[10:100] = d[n]
        pad[n] = x.cuda()
    start = torch.tensor([10, 60, 100], device="cuda")
    o = torch.full((140, hv, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    _, s = rule(d, hk, hv, dk, dv, "bf16").forward(pad["q"], pad["k"], pad["v"], pad["g"], pad["beta"],
                                                   state=d["state"].cuda(), seq_start=start, o=o)
    ro, rs = D.forward(d, dk ** -0.5)
    assert D.rel(o[10:100], ro) <= TOL_O["bf16"] and D.rel(s, rs) <= TOL_S["bf16"]
    assert bool((o[:10] == 7).all()) and bool((o[100:] == 7).all())


def test_nan_stays_in_its_sequence_and_head():
    hk, hv, dk, dv = 2, 2, 64, 64
    d = D.make([100, 100], hk, hv, dk, dv, "bf16", seed=9)
    d["v"][30, 1, 3] = float("nan")
    g = on_gpu(d)
    o, s = rule(d, hk, hv, dk, dv, "bf16").forward(g["q"], g["k"], g["v"], g["g"], g["beta"],
                                                   seq_start=D.starts([100, 100], "cuda"))
    bad = torch.isnan(o)
    assert bool(bad[30:100, 1, 3].all()) and not bool(bad[:, 0].any()) and not bool(bad[100:].any())
    assert not bool(bad[..., :3].any()) and not bool(bad[..., 4:].any())


@pytest.mark.parametrize("gate", [float("-inf"), -1e4, -300.0, -30.0])
def test_strong_decay_and_resets(gate):
    """A reset forgets everything before it and leaves the other decays exact."""
    hk, hv, dk, dv = 1, 2, 64, 32
    d = D.make([150], hk, hv, dk, dv, "f32", seed=11)
    d["g"][::13, 0] = gate
    d["g"][70:80, 1] = gate
    g = on_gpu(d)
    o, s = rule(d, hk, hv, dk, dv, "f32").forward(g["q"], g["k"], g["v"], g["g"], g["beta"], state=g["state"],
                                                  seq_start=D.starts([150], "cuda"))
    ro, rs = D.forward(d, dk ** -0.5)
    assert D.rel(o, ro) <= TOL_O["f32"] and D.rel(s, rs) <= TOL_S["f32"]


def test_keep_and_zero_strength():
    """g = 0 and beta = 0 pass the state through; beta = 1 with g = 0 replaces the key's answer."""
    hk = hv = 1
    d = D.make([128], hk, hv, 64, 64, "f32", seed=12)
    d["g"].zero_()
    d["beta"].zero_()
    g = on_gpu(d)
    r = rule(d, hk, hv, 64, 64, "f32")
    o, s = r.forward(g["q"], g["k"], g["v"], g["g"], g["beta"], state=g["state"], seq_start=D.starts([128], "cuda"))
    assert torch.equal(s, g["state"])
    d["beta"].fill_(1.0)
    g = on_gpu(d)
    o, s = r.forward(g["q"], g["k"], g["v"], g["g"], g["beta"], state=g["state"], seq_start=D.starts([128], "cuda"))
    assert D.rel((s[0, 0].double().T @ g["k"][-1, 0].double()), d["v"][-1, 0]) <= 192 * 2.0 ** -24 * 2


def test_results_do_not_depend_on_neighbours():
    """A sequence gives the same bits alone, in a batch, and packed behind others."""
    hk, hv, dk, dv = 2, 4, 128, 128
    lens = [77, 200, 130]
    d = D.make(lens, hk, hv, dk, dv, "bf16", seed=13)
    g = on_gpu(d)
    r = rule(d, hk, hv, dk, dv, "bf16")
    o, s = r.forward(g["q"], g["k"], g["v"], g["g"], g["beta"], state=g["state"], seq_start=D.starts(lens, "cuda"))
    sl = slice(77, 277)
    o1, s1 = r.forward(*(g[n][sl][None] for n in ("q", "k", "v", "g", "beta")), state=g["state"][1:2])
    assert torch.equal(o[sl], o1[0]) and torch.equal(s[1], s1[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,hk,hv,dk,dv", [(1, 1, 1, 1, 8, 8), (3, 1, 2, 4, 128, 128), (5, 3, 1, 3, 72, 40),
                                             (2, 7, 2, 2, 64, 256), (9, 1, 3, 3, 96, 104)])
def test_step(B, T, hk, hv, dk, dv, dtype):
    d = D.make([T] * B, hk, hv, dk, dv, dtype, seed=B + T)
    pool = torch.randn(B + 3, hv, dk, dv)
    slots = torch.randperm(B + 3)[:B]
    d["state"] = pool[slots]
    g = {n: x.cuda().unflatten(0, (B, T)) for n, x in d.items() if n in ("q", "k", "v", "g", "beta")}
    states = pool.cuda()
    o = rule(d, hk, hv, dk, dv, dtype).step(g["q"], g["k"], g["v"], g["g"], g["beta"], states,
                                            slots=slots.to(torch.int32).cuda())
    ro, rs = D.forward(d, dk ** -0.5)
    # fp32 arithmetic throughout; a bf16 output is rounded once
    assert D.rel(o.flatten(0, 1), ro) <= (2.0 ** -8 if dtype == "bf16" else TOL_O["f32"])
    assert D.rel(states[slots.cuda()], rs) <= TOL_S["f32"]
    rest = [i for i in range(B + 3) if i not in slots.tolist()]
    assert torch.equal(states[rest].cpu(), pool[rest])


def test_step_slots_repeated_and_out_of_range():
    """Rows of one slot are successive tokens; rows without a state give zeros."""
    hk, hv, dk, dv = 1, 2, 64, 64
    B = 70
    names = [3, 1, 3, -1, 3, 1, 99] + [0] * (B - 7)
    d = D.make([1] * B, hk, hv, dk, dv, "f32", seed=21)
    pool = torch.randn(4, hv, dk, dv)
    g = {n: d[n].cuda()[:, None] for n in ("q", "k", "v", "g", "beta")}
    states = pool.cuda()
    r = rule(d, hk, hv, dk, dv, "f32")
    o = r.step(g["q"], g["k"], g["v"], g["g"], g["beta"], states,
               slots=torch.tensor(names, dtype=torch.int32, device="cuda"))
    assert bool((o[3] == 0).all()) and bool((o[6] == 0).all())
    for slot in (0, 1, 3):
        idx = [i for i, s in enumerate(names) if s == slot]
        x = [d[n][idx].double() for n in ("q", "k", "v", "g", "beta")]
        ro, rs = D.recurrence(*x, pool[slot].double(), dk ** -0.5)
        assert D.rel(o[idx, 0], ro) <= TOL_O["f32"] and D.rel(states[slot], rs) <= TOL_S["f32"]
    assert torch.equal(states[2].cpu(), pool[2])


def test_prefill_then_steps_is_one_long_forward():
    """The state a prefill leaves is the one the recurrent form continues from."""
    hk, hv, dk, dv = 2, 4, 128, 128
    B, T, extra = 2, 90, 6
    d = D.make([T + extra] * B, hk, hv, dk, dv, "bf16", seed=23)
    g = {n: d[n].cuda().unflatten(0, (B, T + extra)) for n in ("q", "k", "v", "g", "beta")}
    r = rule(d, hk, hv, dk, dv, "bf16")
    _, st = r.forward(*(g[n][:, :T].contiguous() for n in ("q", "k", "v", "g", "beta")))
    outs = [r.step(*(g[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "g", "beta")), st) for t in range(T, T + 3)]
    outs.append(r.step(*(g[n][:, T + 3:].contiguous() for n in ("q", "k", "v", "g", "beta")), st))
    ro, rs = D.forward(d, dk ** -0.5, use_state=False)
    ro = ro.unflatten(0, (B, T + extra))[:, T:]
    assert D.rel(torch.cat(outs, 1), ro) <= 2.0 ** -8 + TOL_S["bf16"]
    assert D.rel(st, rs) <= TOL_S["bf16"] + TOL_S["f32"]


def test_captured_forward_and_step_replay():
    """Captured once, replayed with eager work between: every replay equals the eager result."""
    hk, hv, dk, dv = 2, 4, 64, 64
    B, T = 2, 100
    d = D.make([T] * B, hk, hv, dk, dv, "bf16", seed=24)
    g = {n: d[n].cuda().unflatten(0, (B, T)) for n in ("q", "k", "v", "g", "beta")}
    one = {n: x[:, :1].contiguous() for n, x in g.items()}
    r = rule(d, hk, hv, dk, dv, "bf16")
    names = ("q", "k", "v", "g", "beta")
    first = torch.zeros(r.state_shape(B), device="cuda")
    st = first.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward(*(g[n] for n in names))
        r.step(*(one[n] for n in names), st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = r.forward(*(g[n] for n in names), state=first)
        st.copy_(s)
        so = r.step(*(one[n] for n in names), st)
    for i in range(3):
        g["v"].mul_(0.5 + i)
        graph.replay()
        torch.cuda.synchronize()
        eo, es = r.forward(*(g[n] for n in names), state=first)
        est = es.clone()
        eso = r.step(*(one[n] for n in names), est)
        assert torch.equal(o, eo) and torch.equal(s, es) and torch.equal(st, est) and torch.equal(so, eso)


def test_runs_on_the_callers_stream():
    hk, hv, dk, dv = 1, 1, 64, 64
    d = D.make([300], hk, hv, dk, dv, "bf16", seed=25)
    g = on_gpu(d)
    r = rule(d, hk, hv, dk, dv, "bf16")
    args = [g[n][None] for n in ("q", "k", "v", "g", "beta")]
    want, ws = r.forward(*args)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(r.forward(*args))
    torch.cuda.synchronize()
    for o, s in outs:
        assert torch.equal(o, want) and torch.equal(s, ws)


def test_captured_cut_sequences_replay():
    """A sequence long enough to be cut, forward and backward, captured once; replays follow
    new inputs, with eager work between them."""
    lens, hk, hv, dk, dv = [2300], 1, 2, 64, 64
    ds = [D.make(lens, hk, hv, dk, dv, "bf16", seed=s, decay=1e-2) for s in (31, 32, 33)]
    r = rule(ds[0], hk, hv, dk, dv, "bf16")
    start = D.starts(lens, "cuda")
    bufs = {n: ds[0][n].cuda() for n in ("q", "k", "v", "g", "beta", "state", "do", "dstate")}

    def both(b):
        o, s = r.forward(*(b[n] for n in ("q", "k", "v", "g", "beta")), state=b["state"], seq_start=start)
        return [o, s, *r.backward(*(b[n] for n in ("q", "k", "v", "g", "beta", "do")), state=b["state"],
                                  dstate_out=b["dstate"], seq_start=start)]

    both(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(bufs)
    for d in ds:
        want = both({n: d[n].cuda() for n in bufs})
        torch.cuda.synchronize()
        for n in bufs:
            bufs[n].copy_(d[n])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert bool((x == y).all())
