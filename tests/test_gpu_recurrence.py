"""Gated linear recurrence on the GPU against its 64-bit recurrence.

Tolerances (relative 2-norm, E = 2^-24). For |r| <= 10 a sigmoid is off by at most 16 E of itself (its
argument's rounding 10, exponential, sum and reciprocal), log a by 18, a therefore by 18 |log a| + 2 <= 11 (rates up to
0.5), b by a root, two sigmoids' worth and products: 40. A state holds each term through at most T factors and as many
products and sums, off by at most (11 + 2) T + 40 <= 16 (T + 4) E of the term; the terms' errors, of either sign as the
terms, leave that share of the state. The backward passes T factors back as well: twice that. bf16 results add
half a step, 2^-8, of their own rounding.
The accuracy test below holds the kernels to what the same formula loses in fp32 on the CPU.
"""
import pytest
import torch

import _recurrence as R

pytestmark = pytest.mark.gpu


def f32(lens):
    return 16 * (max(lens) + 4) * 2.0 ** -24


def fwd(lens, dtype):
    return f32(lens) + (2.0 ** -8 if dtype == "bf16" else 0)


def bwd(lens, dtype):
    return f32(lens) + fwd(lens, dtype)


LENS = [
    [1], [2], [15], [16], [17], [127], [128], [129], [700],
    [0, 5, 0, 0, 1, 1, 1, 3, 0], [16, 16, 16], [100, 28, 128, 1, 300], [1] * 40, [0, 0, 260, 0],
]


def rule(d, dim, dtype):
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    return GatedRecurrence(dim, d["rate"].cuda(), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [8, 200])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_packed(lens, dim, dtype):
    d = R.make(lens, dim, dtype, seed=len(lens) + dim)
    m = rule(d, dim, dtype)
    start = R.starts(lens)
    x = R.gpu(d, "x", "r", "i")
    for use in (True, False):
        state = d["state"].cuda() if use else None
        carries = torch.empty(m.carries_shape(sum(lens)), device="cuda")
        y, s = m.forward(*x, state=state, seq_start=start, carries=carries)
        y0, s0 = R.forward(d, use)
        assert R.rel(y, y0) <= fwd(lens, dtype) and R.rel(s, s0) <= f32(lens)
        dstate = d["dstate"].cuda() if use else None
        want = R.backward(d, use, use)
        for c in (None, carries):
            got = m.backward(*x, d["dy"].cuda(), state=state, dstate_out=dstate, seq_start=start, carries=c)
            for k, (g, w) in enumerate(zip(got, want)):
                assert R.rel(g, w) <= (bwd(lens, dtype) if k < 3 else 2 * f32(lens)), (use, k)


def over_one_grid(tokens):
    """Columns with which the forward's chunks of 64 tokens would take more than 256 workgroups: then they have 160."""
    return 128 * (256 // ((tokens + 63) // 64)) + 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS + [[159], [160], [161], [19, 1, 140, 20, 0, 21], [320, 1]], ids=str)
def test_packed_of_many_columns(lens, dtype):
    test_packed(lens, over_one_grid(sum(lens)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,dim", [(1, 1, 768), (3, 5, 136), (2, 333, 96), (5, 128, 128), (4, 16, 264), (1, 520, 1000)])
def test_batched(N, T, dim, dtype):
    d, lens = R.make([T] * N, dim, dtype, seed=T + dim), [T]
    m = rule(d, dim, dtype)
    rows = torch.cat([d[k] for k in ("x", "r", "i")], 1).cuda().unflatten(0, (N, T))  # views of a projection
    x = rows.split(dim, -1)
    y, s = m.forward(*x, state=d["state"].cuda())
    y0, s0 = R.forward(d)
    assert y.shape == (N, T, dim) and R.rel(y.flatten(0, 1), y0) <= fwd(lens, dtype) and R.rel(s, s0) <= f32(lens)
    got = m.backward(*x, d["dy"].cuda().unflatten(0, (N, T)), state=d["state"].cuda(), dstate_out=d["dstate"].cuda())
    for k, (g, w) in enumerate(zip(got, R.backward(d))):
        assert R.rel(g.flatten(0, 1) if k < 3 else g, w) <= (bwd(lens, dtype) if k < 3 else 2 * f32(lens)), k
    packed = m.forward(*(d[k].cuda() for k in ("x", "r", "i")), state=d["state"].cuda(), seq_start=R.starts([T] * N))
    assert torch.equal(packed[0], y.flatten(0, 1)) and torch.equal(packed[1], s)


@pytest.mark.parametrize("dim", [16, 264])
@pytest.mark.parametrize("lens", [[9001], [4096, 100, 5000]], ids=str)
def test_many_chunks(lens, dim):
    """Long enough that states pass through groups of chunks; slow decays carry them all the way."""
    d = R.make(lens, dim, "f32", seed=3, slow=1e-5, fast=1e-2)
    m = rule(d, dim, "f32")
    x = R.gpu(d, "x", "r", "i")
    start = R.starts(lens)
    y, s = m.forward(*x, state=d["state"].cuda(), seq_start=start)
    tol = f32(lens)
    y0, s0 = R.forward(d)
    assert R.rel(y, y0) <= tol and R.rel(s, s0) <= tol
    got = m.backward(*x, d["dy"].cuda(), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=start)
    for g, w in zip(got, R.backward(d)):
        assert R.rel(g, w) <= 2 * tol
    again = m.backward(*x, d["dy"].cuda(), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=start)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_no_more_is_lost_than_the_formula_loses():
    """Errors of the fp32 kernels against those of the same recurrence in fp32, token by token, on the
    CPU: at most twice (both are sums of as many independent roundings)."""
    d = R.make([2000], 64, "f32", seed=9, slow=1e-3, fast=0.1)
    m = rule(d, 64, "f32")
    x = R.gpu(d, "x", "r", "i")
    start = R.starts([2000])
    y, s = m.forward(*x, state=d["state"].cuda(), seq_start=start)
    la = -d["rate"] * torch.sigmoid(d["r"])
    a, b = la.exp(), (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(d["i"]) * d["x"]
    h, plain = d["state"][0], []
    for t in range(2000):
        h = a[t] * h + b[t]
        plain.append(h)
    y0, _ = R.forward(d)
    assert R.rel(y, y0) <= 2 * R.rel(torch.stack(plain), y0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_wide_open_and_shut(dtype):
    """sig(r) and sig(i) of 0 and 1: the state stays, or forgets at once; gradients stay finite."""
    lens = [64]
    d = R.make(lens, 16, dtype, seed=5)
    big = torch.tensor([-3e4, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 3e4])
    d["r"][:, :8] = big.to(d["r"].dtype)
    d["i"][:, 8:] = big.to(d["i"].dtype)
    d["rate"][2::3] = 40.0
    m = rule(d, 16, dtype)
    x = R.gpu(d, "x", "r", "i")
    start = R.starts([64])
    y, s = m.forward(*x, state=d["state"].cuda(), seq_start=start)
    y0, s0 = R.forward(d)
    assert R.rel(y, y0) <= fwd(lens, dtype) and R.rel(s, s0) <= f32(lens)
    assert bool((y[:, 0].double().cpu() == d["state"][0, 0].to(y.dtype).double()).all())  # sig(r) = 0: kept
    got = m.backward(*x, d["dy"].cuda(), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=start)
    want = R.backward(d)
    for k, (g, w) in enumerate(zip(got, want)):
        assert bool(torch.isfinite(g).all())
        fine = torch.isfinite(w)  # 64-bit autograd divides 0 by 0 where a gate is shut
        assert R.rel(g.cpu()[fine], w[fine]) <= (bwd(lens, dtype) if k < 3 else 2 * f32(lens)), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("z", [8.0, 14.0, 18.0])
def test_gates_all_open_keep_the_digits_of_their_gradients(z, dtype):
    """sig' = sig (1 - sig) where 1 - sig is 3e-4 .. 2e-8: relative to itself, not to 1. (z is exact in bf16; its
    exponential's argument is off by at most z E, the rest as above.)"""
    lens = [100]
    d = R.make(lens, 16, dtype, seed=12)
    d["r"].fill_(z)
    d["i"].fill_(z)
    m = rule(d, 16, dtype)
    got = m.backward(*R.gpu(d, "x", "r", "i", "dy"), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=R.starts(lens))
    want = R.backward(d)
    for k, (g, w) in enumerate(zip(got, want)):
        assert R.rel(g, w) <= (bwd(lens, dtype) if k < 3 else 2 * f32(lens)) + 2 * z * 2.0 ** -24, k


def test_gradients_against_differences():
    """Central differences of the kernels' own fp32 forward along random directions, in fp32 sums: a
    step of 1e-2 leaves curvature of about 1e-4 and rounding of 2^-24 * sqrt(n) / 1e-2, both under 1 percent of
    a directional derivative, which is of the size of the gradient's norm."""
    d = R.make([90, 45], 24, "f32", seed=6, slow=1e-2)
    m = rule(d, 24, "f32")
    start = R.starts([90, 45])
    gen = torch.Generator().manual_seed(1)

    def loss(p):
        from fft_long_convolution_libhyena_amd import GatedRecurrence

        y, s = GatedRecurrence(24, p["rate"].cuda(), "f32").forward(*R.gpu(p, "x", "r", "i"), state=p["state"].cuda(), seq_start=start)
        return float((y.cpu().double() * d["dy"].double()).sum() + (s.cpu().double() * d["dstate"].double()).sum())

    got = m.backward(*R.gpu(d, "x", "r", "i"), d["dy"].cuda(), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=start)
    for name, g in zip(("x", "r", "i", "rate", "state"), got):
        g = g.cpu().double()
        way = g / g.norm() + 0.1 * torch.randn(g.shape, generator=gen).double() / g.numel() ** 0.5
        eps = 1e-2 if name != "rate" else 1e-2 * float(d["rate"].min())
        hi, lo = (loss(dict(d, **{name: (d[name].double() + sign * eps * way).float()})) for sign in (1, -1))
        slope = float((g * way).sum())
        assert abs((hi - lo) / (2 * eps) - slope) <= 1e-2 * abs(slope), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["x", "r", "i", "state"])
@pytest.mark.parametrize("dim", [16, over_one_grid(370)])
def test_where_a_value_that_is_not_finite_shows(name, bad, dtype, dim):
    """In its channel of its sequence from its token on; everything else keeps its bits."""
    lens = [150, 0, 20, 200]
    d = R.make(lens, dim, dtype, seed=7)
    m = rule(d, dim, dtype)

    def call():
        return m.forward(*R.gpu(d, "x", "r", "i"), state=d["state"].cuda(), seq_start=R.starts(lens))

    y0, s0 = call()
    if name == "state":
        d["state"][2, 5] = bad
    else:
        d[name][160, 5] = bad
    y, s = call()
    same, kept = torch.ones_like(y, dtype=torch.bool), torch.ones_like(s, dtype=torch.bool)
    same[(150 if name == "state" else 160):170, 5] = False
    kept[2, 5] = False
    assert torch.equal(y[same], y0[same]) and torch.equal(s[kept], s0[kept])
    if name in ("x", "state") or bad != bad:
        assert not bool(torch.isfinite(y[160, 5])) and not bool(torch.isfinite(s[2, 5]))
    # backward: the channel's gradients in that sequence, and its drate
    got = m.backward(*R.gpu(d, "x", "r", "i", "dy"), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=R.starts(lens))
    others = torch.ones(sum(lens), dim, dtype=torch.bool, device="cuda")
    others[150:170, 5] = False
    for g in got[:3]:
        assert bool(torch.isfinite(g[others]).all())
    assert bool(torch.isfinite(got[3][[c for c in range(dim) if c != 5]]).all()) and bool(torch.isfinite(got[4][kept]).all())


@pytest.mark.parametrize("dim", [40, over_one_grid(368)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_no_sequence(dtype, dim):
    """A padded packed batch: the rows around the sequences hold NaN, have no results and no gradients,
    and given outputs keep what they hold there."""
    lens, front, back = [70, 0, 33], 5, 260
    d = R.make(lens, dim, dtype, seed=8)
    m = rule(d, dim, dtype)
    x = []
    for n in ("x", "r", "i", "dy"):
        t = torch.full((front + sum(lens) + back, dim), float("nan"), dtype=d[n].dtype)
        t[front:-back] = d[n]
        x.append(t.cuda())
    start = R.starts(lens, front=front)
    torch.use_deterministic_algorithms(True, warn_only=True)  # torch.empty gives NaN
    try:
        y, s = m.forward(*x[:3], state=d["state"].cuda(), seq_start=start)
        grads = m.backward(*x, state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=start)
    finally:
        torch.use_deterministic_algorithms(False)
    assert R.rel(y[front:-back], R.forward(d)[0]) <= fwd(lens, dtype) and R.rel(s, R.forward(d)[1]) <= f32(lens)
    for k, (g, w) in enumerate(zip(grads, R.backward(d))):
        assert R.rel(g[front:-back] if k < 3 else g, w) <= (bwd(lens, dtype) if k < 3 else 2 * f32(lens)), k
    for t in (y, *grads[:3]):
        assert not bool(t[:front].any()) and not bool(t[-back:].any())
    given = torch.full_like(y, 7.0)
    m.forward(*x[:3], state=d["state"].cuda(), seq_start=start, y=given)
    assert bool((given[:front] == 7).all()) and bool((given[-back:] == 7).all())
    assert torch.equal(given[front:-back], y[front:-back])


@pytest.mark.parametrize("clear", [0, 1])
@pytest.mark.parametrize("tokens,start", [(300, [7, 7, 200]), (300, [300, 300, 300]), (300, [0, 100, 300]), (1, [0, 0, 0])])
def test_rows_of_no_sequence_are_left_or_cleared(tokens, start, clear):
    """Every output of rows, through the C calls, without state gradients and with the workspace's words or without."""
    import ctypes

    from fft_long_convolution_libhyena_amd.binding import RecurrenceInputsStruct

    dim = 24
    d = R.make([tokens], dim, "bf16", seed=14)
    m = rule(d, dim, "bf16")
    x, r, i, dy = R.gpu(d, "x", "r", "i", "dy")
    at = torch.tensor(start, device="cuda")
    p = m._params(None, clear)
    need = m.lib.hyena_recurrence_backward_workspace_bytes(p, 2, tokens, at.data_ptr(), None)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y, dx, dr, di = (torch.full_like(x, 7.0) for _ in range(4))
    drate = torch.empty(dim, device="cuda")
    ins = ctypes.byref(RecurrenceInputsStruct(x.data_ptr(), dim, r.data_ptr(), dim, i.data_ptr(), dim))
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert m.lib.hyena_recurrence_forward(p, 2, tokens, at.data_ptr(), ins, None, y.data_ptr(), None, None, ws.data_ptr(),
                                          need, st) == 0
    assert m.lib.hyena_recurrence_backward(p, 2, tokens, at.data_ptr(), ins, None, None, dy.data_ptr(), None, dx.data_ptr(),
                                           dr.data_ptr(), di.data_ptr(), drate.data_ptr(), None, ws.data_ptr(), need, st) == 0
    want = m.forward(x, r, i, seq_start=at)[0], *m.backward(x, r, i, dy, seq_start=at)[:3]
    for t, w in zip((y, dx, dr, di), want):
        assert torch.equal(t[start[0]:start[-1]], w[start[0]:start[-1]])
        for rest in (t[:start[0]], t[start[-1]:]):
            assert bool((rest == (0 if clear else 7)).all())


@pytest.mark.parametrize("dim", [72, 520])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_in_place(dtype, dim):
    """state_out may be the initial states: sequences within a wave, a chunk and over many, and empty ones."""
    lens = [3, 0, 500, 1, 4000, 40, 0, 700]
    d = R.make(lens, dim, dtype, seed=13)
    m = rule(d, dim, dtype)
    x, start = R.gpu(d, "x", "r", "i"), R.starts(lens)
    y, s = m.forward(*x, state=d["state"].cuda(), seq_start=start)
    for _ in range(3):
        pool = d["state"].cuda()
        y2, s2 = m.forward(*x, state=pool, seq_start=start, state_out=pool)
        assert s2 is pool and torch.equal(s2, s) and torch.equal(y2, y)
    rows = [v[:4200].unflatten(0, (6, 700)) for v in x]
    y, s = m.forward(*rows, state=d["state"][:6].cuda())
    pool = d["state"][:6].cuda()
    assert torch.equal(m.forward(*rows, state=pool, state_out=pool)[0], y) and torch.equal(pool, s)


def test_more_than_32_bits_of_elements():
    """Two sequences of 2^20 rows of 2304 channels, 4.8e9 elements: constant gates and inputs reach b / (1 - a), and
    the backward's sums their closed forms."""
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB of free memory")
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    T, dim = 1 << 20, 2304
    rate = torch.linspace(0.1, 0.4, dim).cuda()
    m = GatedRecurrence(dim, rate)
    x = torch.ones(2, T, dim, dtype=torch.bfloat16, device="cuda")
    x[1] = -2
    zero = torch.zeros_like(x)
    y, s = m.forward(x, zero, zero)
    a = torch.exp(-rate.double() / 2)
    b = (1 - a * a).sqrt() / 2
    full = b / (1 - a)
    for n, v in ((0, 1.0), (1, -2.0)):
        assert R.rel(s[n], v * full) <= 1e-5 and R.rel(y[n, 0], v * b) <= 2.0 ** -8
        for t in (5000, T // 2 + 7, T - 1):
            assert R.rel(y[n, t], v * full) <= 2.0 ** -8 + 1e-5
    del y
    dx, dr, di, drate, dstate = m.backward(x, zero, zero, x)
    at = T // 2 + 3  # far from both ends: dh = v / (1 - a), h = v full
    for n, v in ((0, 1.0), (1, -2.0)):
        dh = v / (1 - a)
        assert R.rel(dx[n, at], dh * b) <= 2.0 ** -8 + 1e-5 and R.rel(di[n, at], dh * b * v / 2) <= 2.0 ** -8 + 1e-5
        assert R.rel(dx[n, T - 1], v * b) <= 2.0 ** -8 + 1e-5
    assert bool(torch.isfinite(drate).all())
    del x, zero, dx, dr, di
    torch.cuda.empty_cache()


def test_no_tokens():
    m = rule(R.make([1], 16), 16, "bf16")
    s = torch.randn(3, 16, device="cuda")
    x = torch.empty(3, 0, 16, dtype=torch.bfloat16, device="cuda")
    y, out = m.forward(x, x, x, state=s)
    assert y.shape == x.shape and torch.equal(out, s)
    got = m.backward(x, x, x, x, dstate_out=s)
    assert torch.equal(got[4], s) and not bool(got[3].any())
    packed = m.forward(x[0], x[0], x[0], seq_start=torch.zeros(4, dtype=torch.int64, device="cuda"))
    assert not bool(packed[1].any())


@pytest.mark.parametrize("dim", [16, over_one_grid(300)])
def test_offsets_that_break_the_rules_stay_inside(dim):
    """Offsets below 0, beyond the rows or decreasing: any result, but nothing outside the arrays."""
    tokens, N = 300, 4
    d = R.make([tokens], dim, "f32", seed=2)
    m = rule(d, dim, "f32")
    room = torch.full((3, tokens + 20, dim), 7.0, device="cuda")
    states = torch.full((N + 2, dim), 7.0, device="cuda")
    for bad in ([-50, 10, 400, 200, 1 << 40], [300, 200, 100, 50, 0], [0, 0, 0, 0, 0], [1 << 62, -1, 5, 7, -(1 << 62)]):
        start = torch.tensor(bad, dtype=torch.int64, device="cuda")
        y, s = room[0, 10:-10], states[1:-1]
        m.forward(*R.gpu(d, "x", "r", "i"), seq_start=start, y=y, state_out=s)
        m.backward(*R.gpu(d, "x", "r", "i", "dy"), seq_start=start)
        torch.cuda.synchronize()
        assert bool((room[0, :10] == 7).all()) and bool((room[0, -10:] == 7).all())
        assert bool((states[0] == 7).all()) and bool((states[-1] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,dim", [(1, 1, 768), (5, 1, 200), (7, 3, 2056), (300, 2, 16)])
def test_step(B, T, dim, dtype):
    d = R.make([T] * B, dim, dtype, seed=B + dim)
    m = rule(d, dim, dtype)
    gen = torch.Generator().manual_seed(B)
    slots = torch.randperm(B + 3, generator=gen)[:B].to(torch.int32)
    pool = torch.randn(B + 3, dim, generator=gen)
    d["state"] = pool[slots.long()]
    states = pool.cuda()
    y = m.step(*(d[k].cuda().unflatten(0, (B, T)) for k in ("x", "r", "i")), states, slots=slots.cuda())
    y0, s0 = R.forward(d)
    tol = f32([T])
    assert R.rel(y.flatten(0, 1), y0) <= tol + (2.0 ** -8 if dtype == "bf16" else 0)
    full = pool.double()
    full[slots.long()] = s0
    assert R.rel(states, full) <= tol
    free = torch.ones(B + 3, dtype=torch.bool)
    free[slots.long()] = False
    assert torch.equal(states.cpu()[free], pool[free])


def test_step_shared_slots_padding_and_continuing():
    """Rows that name one slot are its successive tokens; a slot outside the pool gives zeros; steps go on
    from a forward's states."""
    B, dim = 9, 72
    d = R.make([1] * B, dim, "f32", seed=4)
    m = rule(d, dim, "f32")
    x = [d[k].cuda() for k in ("x", "r", "i")]
    slots = torch.tensor([2, 0, 2, -1, 2, 5, 0, 1000, 1], dtype=torch.int32, device="cuda")
    pool = torch.randn(5, dim, device="cuda")
    states = pool.clone()
    y = m.step(*(v[:, None] for v in x), states, slots=slots)[:, 0]
    assert not bool(y[[3, 5, 7]].any())
    for slot in (0, 1, 2):
        rows = (slots == slot).nonzero()[:, 0]
        want, s = m.forward(*(v[rows][None] for v in x), state=pool[slot:slot + 1].clone())
        assert R.rel(y[rows], want[0]) <= 2 * f32([3]) and R.rel(states[slot], s[0]) <= 2 * f32([3])
    assert torch.equal(states[3:], pool[3:])
    y1, s1 = m.forward(*(v[None] for v in x))
    y2, s2 = m.forward(*(v[None, :6] for v in x))
    y3 = m.step(*(v[None, 6:] for v in x), s2)
    assert R.rel(y3, y1[:, 6:]) <= 2 * f32([9]) and R.rel(s2, s1) <= 2 * f32([9])


def test_step_on_the_last_tokens_of_long_rows():
    """A view with one token of each of a few long rows: strides beyond what whole sequences take."""
    B, T, dim = 3, 60000, 136
    d = R.make([1] * B, dim, "bf16", seed=14)
    m = rule(d, dim, "bf16")
    long = torch.zeros(3, B, T, dim, dtype=torch.bfloat16, device="cuda")
    for k, n in enumerate(("x", "r", "i")):
        long[k, :, -1] = d[n].cuda()
    states = [d["state"].cuda() for _ in range(2)]
    y = m.step(*long[:, :, -1:], states[0])
    assert T * dim > 1 << 22 and y.is_contiguous()
    assert torch.equal(y, m.step(*(d[n].cuda()[:, None] for n in ("x", "r", "i")), states[1])) and torch.equal(*states)


def test_capture_replays_and_streams():
    """A captured training step replayed on new inputs, with eager work between, and the same calls on two
    streams at once, against eager results."""
    N, T, dim = 2, 1000, 136
    d = R.make([T] * N, dim, "bf16", seed=11)
    m = rule(d, dim, "bf16")
    x = [d[k].cuda().unflatten(0, (N, T)) for k in ("x", "r", "i", "dy")]
    state = d["state"].cuda()

    def step():
        carries = torch.empty(m.carries_shape(N * T), device="cuda")
        out = m.forward(*x[:3], state=state, carries=carries)
        return out + m.backward(*x, state=state, dstate_out=state, carries=carries)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        for v in x:
            v.copy_(v.roll(1, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        state.mul_(0.5)
    want = step()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for side in sides:
            with torch.cuda.stream(side):
                got.append(step())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_widest_rows_and_many_sequences():
    """2^20 channels; 70000 sequences of no token, one or two, packed and in a batch."""
    d = R.make([3, 0, 2], 1 << 20, "bf16", seed=15)
    m = rule(d, 1 << 20, "bf16")
    y, s = m.forward(*R.gpu(d, "x", "r", "i"), state=d["state"].cuda(), seq_start=R.starts(d["lens"]))
    y0, s0 = R.forward(d)
    assert R.rel(y, y0) <= fwd([3], "bf16") and R.rel(s, s0) <= f32([3])
    got = m.backward(*R.gpu(d, "x", "r", "i", "dy"), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(), seq_start=R.starts(d["lens"]))
    for k, (g, w) in enumerate(zip(got, R.backward(d))):
        assert R.rel(g, w) <= (bwd([3], "bf16") if k < 3 else 2 * f32([3])), k

    N, dim = 70000, 8
    d = R.make([1] * N, dim, "f32", seed=16)
    m = rule(d, dim, "f32")
    x, dy, state = R.gpu(d, "x", "r", "i"), d["dy"].cuda(), d["state"].cuda()
    lens = torch.randint(0, 3, (N,), generator=torch.Generator().manual_seed(16))
    lens = lens[lens.cumsum(0) <= N]
    start = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    # every sequence in 64 bits at once: its first token, then its second
    x64, r64, i64 = (d[k].double() for k in ("x", "r", "i"))
    la = -d["rate"].double() * torch.sigmoid(r64)
    a, b = la.exp(), (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(i64) * x64
    h = d["state"][:len(lens)].double()
    y0 = torch.zeros(N, dim, dtype=torch.float64)
    for t in range(2):
        some = lens > t
        at = start[:-1][some] + t
        h[some] = a[at] * h[some] + b[at]
        y0[at] = h[some]
    y, s = m.forward(*x, state=state[:len(lens)], seq_start=start.cuda())
    assert R.rel(y, y0) <= f32([2]) and R.rel(s, h) <= f32([2])
    grads = m.backward(*x, dy, state=state[:len(lens)], seq_start=start.cuda())
    dx = d["dy"].double().clone()  # of a sequence's last token dh = dy, of the one in front dy + a dh
    before = (start[1:] - 2)[lens > 1]
    dx[before] += a[before + 1] * d["dy"][before + 1].double()
    dx[int(start[-1]):] = 0
    assert R.rel(grads[0], dx * (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(i64)) <= 2 * f32([2])
    y, s = m.forward(*(v[:, None] for v in x), state=state)
    want = a * d["state"].double() + b
    assert R.rel(y[:, 0], want) <= f32([1]) and R.rel(s, want) <= f32([1])


def test_graphs_that_share_a_workspace():
    """Two captured calls of different sizes with one workspace, replayed in turn and between eager calls with it."""
    d = [R.make([n], 136, "bf16", seed=n) for n in (3000, 700)]
    m = [rule(v, 136, "bf16") for v in d]
    x = [[v[k].cuda()[None] for k in ("x", "r", "i", "dy")] for v in d]
    ws = torch.empty(max(m[0].backward_workspace_bytes(1, 3000), m[0].workspace_bytes(1, 3000)), dtype=torch.uint8, device="cuda")

    def step(k):
        return m[k].forward(*x[k][:3], workspace=ws) + m[k].backward(*x[k], workspace=ws)

    want, graphs, outs = [step(k) for k in range(2)], [], []
    torch.cuda.synchronize()
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            outs.append(step(k))
    for k in (0, 1, 1, 0, 0, 1):
        for t in outs[k]:
            t.zero_()
        graphs[k].replay()
        eager = step(1 - k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k])), k
        assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - k])), k
