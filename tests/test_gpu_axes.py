"""Head norm with a position for each of several axes, against its plain form in 64 bits (tolerances:
those of one axis, whose operations it has), and the operators of a block run behind each other.
"""
import pytest
import torch

import _delta as D
import _recurrence as R

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
FWD = {"bf16": 2.0 ** -8, "f32": (256 / 2 + 16) * E}
BWD = {"bf16": 2.0 ** -8 + 416 * E, "f32": 416 * E}
DW = (512 + 416) * E
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def reference(x, w, pos, axis, freq, kind, pairs, eps=1e-6):
    """64-bit y of x [tokens, heads, dim] with positions [tokens, axes]; differentiable."""
    size = x.square().sum(-1, keepdim=True) / (x.shape[-1] if kind == "rms" else 1) + eps
    y = x / size.sqrt()
    y = y if w is None else y * w
    f = freq.numel()
    ang = (pos.double()[:, axis.long()] * freq.double())[:, None]
    c, s = ang.cos(), ang.sin()
    a, b = (y[..., 0:2 * f:2], y[..., 1:2 * f:2]) if pairs else (y[..., :f], y[..., f:2 * f])
    u, v = a * c - b * s, a * s + b * c
    head = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([head, y[..., 2 * f:]], -1)


def make(tokens, hq, hk, dim, axis, axes, dtype, seed, far, weights):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    rot = len(axis)
    return dict(q=rn(tokens, hq, dim).to(DT[dtype]), k=(3 * rn(tokens, hk, dim)).to(DT[dtype]), dq_out=rn(tokens, hq, dim).to(DT[dtype]),
                dk_out=rn(tokens, hk, dim).to(DT[dtype]), w_q=1 + 0.3 * rn(dim) if weights else None,
                w_k=1 + 0.3 * rn(dim) if weights else None, axis=torch.tensor(axis, dtype=torch.int32),
                freq=10000.0 ** (-torch.arange(rot).float() / max(rot, 1)),
                pos=torch.randint(-20, far + 50, (tokens, axes), generator=gen))


def gpu(x):
    return None if x is None else x.cuda()


def norm(d, hq, hk, dim, dtype, kind, pairs):
    from fft_long_convolution_libhyena_amd import QKNorm

    return QKNorm(hq, hk, dim, dtype=dtype, kind=kind, w_q=gpu(d["w_q"]), w_k=gpu(d["w_k"]), freq=gpu(d["freq"]), pairs=pairs,
                  axis=gpu(d["axis"]))


CASES = [  # tokens, heads_q, heads_k, dim, axis of every pair, axes, far, weights
    (1, 1, 1, 8, [0, 1, 1, 0], 2, 0, True),
    (5, 6, 6, 128, [0] * 16 + [1] * 24 + [2] * 24, 3, 1000000, True),
    (37, 3, 1, 72, [0, 1, 2] * 4, 3, 100, False),         # by turns
    (130, 12, 4, 64, [0] * 7 + [1] * 9, 2, 100000, True),   # a section that ends inside four pairs
    (9, 2, 7, 256, list(range(8)) * 16, 8, 0, False),
    (300, 2, 1, 32, [0] * 8, 1, 1000, True),
    (6, 2, 1, 64, [], 2, 0, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,pairs", [("rms", False), ("l2", True), ("l2", False), ("rms", True)])
@pytest.mark.parametrize("tokens,hq,hk,dim,axis,axes,far,weights", CASES)
def test_forward_and_backward(tokens, hq, hk, dim, axis, axes, far, weights, kind, pairs, dtype):
    d = make(tokens, hq, hk, dim, axis, axes, dtype, tokens + dim, far, weights)
    m = norm(d, hq, hk, dim, dtype, kind, pairs)
    pos = gpu(d["pos"])
    out = m.forward(d["q"].cuda(), d["k"].cuda(), pos)
    got = m.backward(d["q"].cuda(), d["k"].cuda(), d["dq_out"].cuda(), d["dk_out"].cuda(), pos)
    for i, n in enumerate("qk"):
        x = d[n].double().requires_grad_()
        w = d["w_" + n].double().requires_grad_() if weights else None
        y = reference(x, w, d["pos"], d["axis"], d["freq"], kind, pairs)
        assert D.rel(out[i], y) <= FWD[dtype]
        grads = torch.autograd.grad((y * d[f"d{n}_out"].double()).sum(), [x] + ([w] if weights else []))
        assert D.rel(got[i], grads[0]) <= BWD[dtype]
        if weights:
            assert D.rel(got[2 + i], grads[1]) <= DW


def test_one_position_on_every_axis_is_one_axis():
    """The same position on all axes gives the bits of the call with one position."""
    from fft_long_convolution_libhyena_amd import QKNorm

    d = make(50, 3, 2, 64, [0, 1, 2, 1] * 8, 3, "bf16", 5, 1000, True)
    pos = d["pos"][:, :1].contiguous().cuda()
    q, k = d["q"].cuda(), d["k"].cuda()
    several = norm(d, 3, 2, 64, "bf16", "rms", False)
    one = QKNorm(3, 2, 64, w_q=gpu(d["w_q"]), w_k=gpu(d["w_k"]), freq=gpu(d["freq"]))
    for a, b in zip(several.forward(q, k, pos.expand(50, 3).contiguous()), one.forward(q, k, pos[:, 0].contiguous())):
        assert torch.equal(a, b)
    # an axis that a token does not have is held to those it has
    d["axis"] = torch.tensor([-1, 0, 7, 1 << 30] * 8, dtype=torch.int32)
    for a, b in zip(norm(d, 3, 2, 64, "bf16", "rms", False).forward(q, k, pos), one.forward(q, k, pos[:, 0].contiguous())):
        assert torch.equal(a, b)


def test_batch_shape_no_tokens_and_capture():
    d = make(66, 3, 2, 64, [0] * 16 + [1] * 16, 2, "bf16", 6, 100, True)
    m = norm(d, 3, 2, 64, "bf16", "l2", True)
    q, k, pos = d["q"].cuda(), d["k"].cuda(), d["pos"].cuda()
    want = m.forward(q, k, pos)
    got = m.forward(q.unflatten(0, (2, 33)), k.unflatten(0, (2, 33)), pos.unflatten(0, (2, 33)))
    assert all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, want))
    assert m.forward(q[:0], k[:0], pos[:0])[0].shape == (0, 3, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.forward(q, k, pos) + m.backward(q, k, q, k, pos)
    for i in range(3):
        pos.add_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, m.forward(q, k, pos) + m.backward(q, k, q, k, pos))), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,pairs", [(8, False), (64, True), (128, False), (256, True)])
def test_calls_beyond_the_cache(dim, pairs, dtype):
    """More than 256 MiB: the same bits for every token as in a call of few."""
    few, hq, hk = 100, 2, 1
    axis = [k % 3 for k in range(dim // 4 // 4 * 4)]
    d = make(few, hq, hk, dim, axis, 3, dtype, dim, 1000, True)
    m = norm(d, hq, hk, dim, dtype, "rms", pairs)
    n = -(-(300 << 20) // ((hq + hk) * dim * 2 * (4 if dtype == "f32" else 2)) // few) + 1
    small = [d[k].cuda() for k in ("q", "k", "dq_out", "dk_out", "pos")]
    q, k, dq, dk, pos = (t.repeat(n, *[1] * (t.dim() - 1)) for t in small)
    for a, b in zip(m.forward(q, k, pos), m.forward(small[0], small[1], small[4])):
        assert torch.equal(a, b.repeat(n, 1, 1))
    for a, b in zip(m.backward(q, k, dq, dk, pos)[:2], m.backward(*small)[:2]):
        assert torch.equal(a, b.repeat(n, 1, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_for_a_video(dtype):
    """A block as a layer runs it: residual norm, projection, head norm over time, height and width, gated delta rule,
    residual norm, projection, gated recurrence; then the gradients back through all of it, against 64 bits."""
    from fft_long_convolution_libhyena_amd import DeltaRule, GatedRecurrence, QKNorm, ResidualNorm

    heads, hd, grid = 2, 32, (4, 5, 6)
    dim, T = heads * hd, 4 * 5 * 6
    gen = torch.Generator().manual_seed(31)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = DT[dtype]
    x, stream = rn(T, dim).to(dt), rn(T, dim).to(dt)
    w1, w2 = 1 + 0.2 * rn(dim), 1 + 0.2 * rn(dim)
    proj1, proj2 = (rn(dim, 3 * dim) / dim ** 0.5).to(dt), (rn(dim, 3 * dim) / dim ** 0.5).to(dt)
    g, beta = (-0.1 * torch.rand((T, heads), generator=gen)).to(dt), torch.sigmoid(rn(T, heads)).to(dt)
    rate = 0.01 + 0.1 * torch.rand(dim, generator=gen)
    pos = torch.cartesian_prod(*(torch.arange(n) for n in grid))
    axis = torch.tensor([0] * 4 + [1] * 6 + [2] * 6, dtype=torch.int32)
    freq = 100.0 ** (-torch.arange(16).float() / 16)
    dy, dsum = rn(T, dim).to(dt), rn(T, dim).to(dt)

    n1, n2 = (ResidualNorm(dim, w.cuda(), dtype=dtype) for w in (w1, w2))
    heads_norm = QKNorm(heads, heads, hd, dtype=dtype, kind="l2", freq=freq.cuda(), axis=axis.cuda())
    rule, rec = DeltaRule(heads, heads, hd, hd, dtype), GatedRecurrence(dim, rate.cuda(), dtype)
    c = {k: v.cuda() for k, v in dict(x=x, stream=stream, p1=proj1, p2=proj2, g=g, beta=beta, pos=pos, dy=dy, dsum=dsum).items()}
    y1, s1 = n1.forward(c["x"], c["stream"])
    q, k, v = ((y1 @ c["p1"]).split(dim, -1))
    q, k, v = (t.unflatten(-1, (heads, hd))[None] for t in (q, k, v))
    qn, kn = heads_norm.forward(q, k, c["pos"][None])
    o, _ = rule.forward(qn, kn, v, c["g"][None], c["beta"][None])
    y2, s2 = n2.forward(o[0].flatten(1), s1)
    xr, r, i = (t[None] for t in (y2 @ c["p2"]).split(dim, -1))
    carries = torch.empty(rec.carries_shape(T), device="cuda")
    y, _ = rec.forward(xr, r, i, carries=carries)
    back = rec.backward(xr, r, i, c["dy"][None], carries=carries)
    dy2 = torch.cat([t[0] for t in back[:3]], -1) @ c["p2"].t().contiguous()
    do, ds1, dw2 = n2.backward(s2, dy2, c["dsum"])
    dqn, dkn, dv, dg, dbeta, _ = rule.backward(qn, kn, v, c["g"][None], c["beta"][None], do.unflatten(-1, (heads, hd))[None])
    dq, dk, _, _ = heads_norm.backward(q, k, dqn, dkn, c["pos"][None])
    dy1 = torch.cat([t[0].flatten(1) for t in (dq, dk, dv)], -1) @ c["p1"].t().contiguous()
    dx, _, dw1 = n1.backward(s1, dy1, ds1)

    leaves = [t.double().requires_grad_() for t in (x, stream, w1, w2, g, beta, rate)]
    X, S, W1, W2, G, Be, Ra = leaves
    rms = lambda s, w: s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    S1 = X + S
    Q, K, V = (t.unflatten(-1, (heads, hd)) for t in (rms(S1, W1) @ proj1.double()).split(dim, -1))
    Q, K = (reference(t, None, pos, axis, freq, "l2", False) for t in (Q, K))
    O, _ = D.recurrence(Q, K, V, G, Be, torch.zeros(heads, hd, hd, dtype=torch.float64), hd ** -0.5)
    S2 = S1 + O.flatten(1)
    Y, _ = R.recurrence(*(rms(S2, W2) @ proj2.double()).split(dim, -1), Ra, torch.zeros(dim, dtype=torch.float64))
    want = torch.autograd.grad((Y * dy.double()).sum() + (S2 * dsum.double()).sum(), leaves)
    # On the way to y a value is rounded to bf16 ten times (norms, sums, products, heads, o), and on the way back as often
    # again, each time half a step 2^-8 of a part of it; such errors add in squares, and each may enter a result through three
    # of its factors: 2^-8 * 3 * sqrt(10) forward, sqrt(30) back. fp32: the same of the parts' bounds, the largest 16 * 124 E.
    unit = 2.0 ** -8 if dtype == "bf16" else 16 * 124 * E
    assert D.rel(y[0], Y) <= unit * 3 * 10 ** 0.5
    for got, exact in zip((dx, dx, dw1, dw2, dg[0], dbeta[0], back[3]), want):
        assert D.rel(got, exact) <= unit * 3 * 30 ** 0.5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_block(dtype):
    """Serving: ragged prompts through residual norm and recurrence into a pool of states, then single tokens."""
    from fft_long_convolution_libhyena_amd import GatedRecurrence, ResidualNorm

    dim, lens, extra = 48, [130, 1, 67], 3
    total = [n + extra for n in lens]
    d = R.make(total, dim, dtype, seed=41)
    gen = torch.Generator().manual_seed(42)
    stream = torch.randn(sum(total), dim, generator=gen).to(DT[dtype])
    w = 1 + 0.2 * torch.randn(dim, generator=gen)
    norm_, rec = ResidualNorm(dim, w.cuda(), dtype=dtype), GatedRecurrence(dim, d["rate"].cuda(), dtype)
    begin = [sum(total[:i]) for i in range(len(total))]
    prompt = torch.cat([torch.arange(b, b + n) for b, n in zip(begin, lens)])
    u, _ = norm_.forward(d["x"][prompt].cuda(), stream[prompt].cuda())
    y, states = rec.forward(u, d["r"][prompt].cuda(), d["i"][prompt].cuda(), state=d["state"].cuda(), seq_start=R.starts(lens))
    pool = torch.full((5, dim), float("nan"), device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = states
    out = [y[sum(lens[:i]):sum(lens[:i + 1])] for i in range(len(lens))]
    for t in range(extra):
        at = torch.tensor([b + n + t for b, n in zip(begin, lens)])
        u, _ = norm_.forward(d["x"][at].cuda()[:, None], stream[at].cuda()[:, None])
        y1 = rec.step(u, *(d[n][at].cuda()[:, None] for n in ("r", "i")), pool, slots=slots)
        out = [torch.cat([a, b]) for a, b in zip(out, y1)]
    s = d["x"].double() + stream.double()
    ref = dict(d, x=s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double())
    y0, s0 = R.forward(ref)
    f32 = 16 * 140 * E
    # bf16: the normed rows' rounding and the outputs' own add in squares; states have the first
    assert D.rel(torch.cat(out), y0) <= f32 + (2.0 ** -8 * 2 ** 0.5 if dtype == "bf16" else 0)
    assert D.rel(pool[slots.long()], s0) <= f32 + (2.0 ** -8 if dtype == "bf16" else 0)
    assert bool(pool[[1, 3]].isnan().all())
