"""Residual norm on the GPU against its plain form in 64 bits.

Tolerances (relative 2-norm, E = 2^-24). fp32: the addition one rounding, which its square doubles; a sum of n squares at
most n of them, halved by the root; root, reciprocal and two products 6: (n / 2 + 8) E. Sums run over 64 to 512 threads of at most 32
values and ten exchanges each, so n is held at 48, whatever dim. The backward has a second such sum and 10 more operations:
(48 + 24 + 24) E. The weight's gradient sums rows in chains of at most 512 here: 512 E more. bf16 adds half a
step, 2^-8, and e4m3 half a step 2^-4 of each value, or, below its smallest normal 2^-6, half of 2^-9 (in
units of the scale).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
FWD = {"bf16": 2.0 ** -8, "f32": (24 + 8) * E}
DW = (512 + 96) * E
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n else 1.0)


def make(rows, dim, dtype, wide, seed=0, weight=True):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    res = torch.float32 if wide else DT[dtype]
    return dict(x=rn(rows, dim).to(DT[dtype]), residual=(2 * rn(rows, dim)).to(res), dy=rn(rows, dim).to(DT[dtype]),
                dsum=rn(rows, dim).to(res), w=1 + 0.3 * rn(dim) if weight else None)


def reference(s, w, eps=1e-6):
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w


def norm(d, dim, dtype, wide, **kw):
    from fft_long_convolution_libhyena_amd import ResidualNorm

    return ResidualNorm(dim, None if d["w"] is None else d["w"].cuda(), dtype=dtype, wide_residual=wide, **kw)


TYPES = [("bf16", False), ("bf16", True), ("f32", False)]
SIZES = [(1, 8), (3, 16), (5, 256), (4, 264), (7, 768), (66, 520), (9, 1000), (5, 1032), (6, 1544), (3, 2048), (5, 2056), (2, 4104),
         (3, 8200), (2, 16384), (4099, 64)]


@pytest.mark.parametrize("dtype,wide", TYPES)
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_backward(rows, dim, dtype, wide):
    weight = rows % 2 == 1
    d = make(rows, dim, dtype, wide, seed=dim, weight=weight)
    m = norm(d, dim, dtype, wide)
    w = d["w"].double() if weight else None
    y, s = m.forward(d["x"].cuda(), d["residual"].cuda())
    total = d["x"].double() + d["residual"].double()
    assert rel(y, reference(total, w)) <= FWD[dtype]
    assert s.dtype == d["residual"].dtype and torch.equal(s.cpu(), (d["x"].float() + d["residual"].float()).to(s.dtype))
    # without a residual: s is x itself, or x in fp32
    y, s = m.forward(d["x"].cuda())
    assert rel(y, reference(d["x"].double(), w)) <= FWD[dtype] and torch.equal(s.cpu(), d["x"].to(s.dtype))
    for use in (True, False):
        leaf = d["residual"].double().requires_grad_()
        wl = w.clone().requires_grad_() if weight else None
        grads = torch.autograd.grad((reference(leaf, wl) * d["dy"].double()).sum(), [leaf] + ([wl] if weight else []))
        ds = grads[0] + d["dsum"].double() if use else grads[0]
        dx, dres, dw = m.backward(d["residual"].cuda(), d["dy"].cuda(), d["dsum"].cuda() if use else None)
        # the gradient's terms can cancel; their roundings are of the terms' size
        inv = 1 / (leaf.detach().square().mean(-1, keepdim=True) + 1e-6).sqrt()
        terms = 2 * float((inv * d["dy"].double() * (w if weight else 1)).norm()) + (float(d["dsum"].double().norm()) if use else 0)
        for got in (dx, dres):
            half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0
            assert float((got.cpu().double() - ds).norm()) <= half * float(ds.norm()) + 96 * E * terms
        assert (dw is None) == (not weight)
        if weight:
            assert rel(dw, grads[1]) <= DW * max(1.0, rows ** 0.5)  # a sum of signed terms may cancel to its root
        assert dres is dx or wide


@pytest.mark.parametrize("dtype,wide", TYPES)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,dim", [(1, 8), (5, 128), (3, 136), (4, 768), (66, 520), (3, 2048), (2, 2056), (3, 4224), (2, 16384)])
def test_8_bits(rows, dim, block, dtype, wide):
    d = make(rows, dim, dtype, wide, seed=dim + 1)
    m = norm(d, dim, dtype, wide, bits8=True, block=block)
    q, scales, s = m.forward(d["x"].cuda(), d["residual"].cuda())
    n = -(-dim // block) if block else 1
    assert q.dtype == torch.float8_e4m3fn and scales.shape == (rows, n)
    y = reference(d["x"].double() + d["residual"].double(), d["w"].double())
    width = block or dim
    padded = torch.nn.functional.pad(y, (0, n * width - dim)).unflatten(1, (n, width))
    want = padded.abs().amax(-1) / 448
    assert float(((scales.cpu().double() - want) / want).abs().max()) <= (24 + 10) * E
    q, by = q.cpu().double(), scales.cpu().double().repeat_interleave(width, 1)[:, :dim]
    # half a step of the value, or of the smallest numbers; y and the division round in fp32 first
    step = torch.maximum(y.abs() * 2.0 ** -4, by * 2.0 ** -10) + y.abs() * 64 * E
    assert bool(((q * by - y).abs() <= step).all())
    assert bool((q.abs().unflatten(1, (1, dim)).amax(-1) == 448).all())  # the largest is represented
    assert torch.equal(s.cpu(), (d["x"].float() + d["residual"].float()).to(s.dtype))


@pytest.mark.parametrize("dim", [72, 4096])
@pytest.mark.parametrize("block", [0, 128])
def test_zeros_tiny_and_not_finite_rows(dim, block):
    d = make(6, dim, "f32", False, seed=1)
    d["x"][1] = 0
    d["residual"][1] = 0
    d["x"][2, 5] = float("nan")
    d["x"][3, 3] = float("inf")
    d["x"][4] *= 1e-30
    d["residual"][4] *= 1e-30
    m = norm(d, dim, "f32", False, eps=1e-30)
    y, _ = m.forward(d["x"].cuda(), d["residual"].cuda())
    assert bool((y[1] == 0).all()) and bool(torch.isfinite(y[[0, 4, 5]]).all())
    assert not bool(torch.isfinite(y[2]).any()) and bool(torch.isnan(y[3, 3]))
    m8 = norm(d, dim, "f32", False, eps=1e-30, bits8=True, block=block)
    q, scales, _ = m8.forward(d["x"].cuda(), d["residual"].cuda())
    q = q.float()
    assert bool((q[1] == 0).all()) and bool((scales[1] == 1).all())
    assert bool(torch.isfinite(q[[0, 4, 5]]).all()) and bool(torch.isfinite(scales).all())
    assert bool(torch.isnan(q[2]).all()) and bool(torch.isnan(q[3, 3]))
    dx, _, dw = m.backward(d["x"].cuda(), d["dy"].cuda())
    assert bool(torch.isfinite(dx[[0, 1, 5]]).all())


@pytest.mark.parametrize("dtype,wide", TYPES)
@pytest.mark.parametrize("dim", [264, 768, 1544, 4104])
def test_calls_beyond_the_cache(dim, dtype, wide):
    """Calls of more than 256 MiB take other instructions for the same arithmetic: every row has the bits it has in a
    small call, and the weight's gradient is the rows' sum (600 fp32 additions each way; signs cancel to the root of the rows)."""
    rows = -(-(300 << 20) // (dim * 8))
    few = 64
    d = make(few, dim, dtype, wide, seed=dim)
    small = [d[k].cuda() for k in ("x", "residual", "dy", "dsum")]
    big = [t.repeat(-(-rows // few), 1)[:rows] for t in small]
    for kw in (dict(), dict(bits8=True, block=128), dict(bits8=True)):
        m = norm(d, dim, dtype, wide, **kw)
        got, want = m.forward(big[0], big[1]), m.forward(small[0], small[1])
        for a, b in zip(got, want):
            a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
            assert torch.equal(a, b.repeat(-(-rows // few), 1)[:rows])
    dx, dres, dw = m.backward(*big[1:])
    sx, sres, _ = m.backward(*small[1:])
    assert torch.equal(dx, sx.repeat(-(-rows // few), 1)[:rows]) and torch.equal(dres, sres.repeat(-(-rows // few), 1)[:rows])
    s = d["residual"].double()
    each = (d["dy"].double() * s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt()).cuda()
    assert rel(dw, each.repeat(-(-rows // few), 1)[:rows].sum(0)) <= (600 + 96) * E * few ** 0.5


def test_views_batches_and_in_place():
    dim, B, T = 64, 2, 33
    d = make(B * T, dim, "bf16", False, seed=2)
    m = norm(d, dim, "bf16", False)
    rows = torch.cat([d["x"], d["residual"], torch.zeros(B * T, 8).bfloat16()], 1).cuda().unflatten(0, (B, T))
    y, s = m.forward(rows[..., :dim], rows[..., dim:2 * dim])
    y2, s2 = m.forward(d["x"].cuda(), d["residual"].cuda())
    assert y.shape == (B, T, dim) and torch.equal(y.flatten(0, 1), y2) and torch.equal(s.flatten(0, 1), s2)
    stream = d["residual"].cuda()
    y3, s3 = m.forward(d["x"].cuda(), stream, sum_out=stream)
    assert s3 is stream and torch.equal(s3, s2) and torch.equal(y3, y2)
    a = m.backward(rows[..., dim:2 * dim], d["dy"].cuda().unflatten(0, (B, T)), d["dsum"].cuda().unflatten(0, (B, T)))
    b = m.backward(d["residual"].cuda(), d["dy"].cuda(), d["dsum"].cuda())
    assert torch.equal(a[0].flatten(0, 1), b[0]) and torch.equal(a[2], b[2])


def test_single_outputs_of_the_backward():
    """Any of the three may be left out, and dresidual may be dsum."""
    dim, rows = 520, 70
    d = make(rows, dim, "bf16", True, seed=6)
    m = norm(d, dim, "bf16", True)
    s, dy, ds = d["residual"].cuda(), d["dy"].cuda(), d["dsum"].cuda()
    dx, dres, dw = m.backward(s, dy, ds)
    ws = torch.empty(m.backward_workspace_bytes(rows), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(x=None, r=None, w=None):
        p = [t.data_ptr() if t is not None else None for t in (x, r, w)]
        assert m.lib.hyena_residual_norm_backward(m._params(), rows, s.data_ptr(), dim, dy.data_ptr(), ds.data_ptr(), *p,
                                                  ws.data_ptr() if w is not None else None, ws.numel(), stream) == 0

    for want, key in ((dx, "x"), (dres, "r"), (dw, "w")):
        got = torch.full_like(want, 7)
        call(**{key: got})
        assert torch.equal(got, want)
    call(r=ds)
    assert torch.equal(ds, dres)


def test_no_rows():
    d = make(1, 64, "bf16", False)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    m = norm(d, 64, "bf16", False)
    y, s = m.forward(e, e)
    dx, dres, dw = m.backward(e, e)
    assert y.shape == s.shape == dx.shape == (0, 64) and not bool(dw.any())


def test_capture_replays_and_streams():
    dim = 1000
    d = make(3000, dim, "bf16", True, seed=3)
    m, m8 = norm(d, dim, "bf16", True), norm(d, dim, "bf16", True, bits8=True, block=128)
    x, res, dy = (d[k].cuda() for k in ("x", "residual", "dy"))

    def step():
        y, s = m.forward(x, res)
        q, scales, _ = m8.forward(x, res)
        return (y, s, q.view(torch.uint8), scales) + m.backward(s, dy, res)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(x.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), k
    want = step()
    torch.cuda.synchronize()
    got = []
    for side in [torch.cuda.Stream() for _ in range(2)]:
        for _ in range(2):
            with torch.cuda.stream(side):
                got.append(step())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
