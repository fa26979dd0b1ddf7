"""The gated recurrence over many chunks and groups of chunks, held to what the same formulas lose in fp32, token by token
on the CPU: outputs, final states and all gradients, as a whole and in every 16 rows, so that nothing at one border
between chunks hides in the rest.

Kernel and plain form round a, the products and the sums as often a token (the kernel's a half a step off, its joins of runs one
rounding in 20 tokens more), so their errors are sums of as many independent roundings: at most twice the plain form's as a
whole and, where the largest of some hundred blocks is compared with the largest, three times. On top come errors that
every value has for itself: sigmoids from an exponential whose argument is rounded (|z| E, of some hundred values 2 E in
the mean), root, reciprocals and products (8 E): below 16 E, E = 2^-24. bf16 results add half a step, 2^-8.
"""
import pytest
import torch

import _recurrence as R

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def plain(d, dt):
    """y, states, dx, dr, di, drate, dstate by the formulas, token by token, in dt."""
    x, r, i, dy = (d[k].to(dt) for k in ("x", "r", "i", "dy"))
    rate, state, dstate = (d[k].to(dt) for k in ("rate", "state", "dstate"))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    la = -rate * sr
    a, m = 1 + torch.expm1(la), (-torch.expm1(2 * la)).sqrt()  # a half a step off: exp's error counts once a token outlived
    b = m * si * x
    y, before, dh = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    last, dfirst, at = torch.empty_like(state), torch.empty_like(state), 0
    for n, length in enumerate(d["lens"]):
        h = state[n]
        for t in range(at, at + length):
            before[t] = h
            h = a[t] * h + b[t]
            y[t] = h
        last[n] = h
        g = dstate[n]
        for t in reversed(range(at, at + length)):
            dh[t] = dy[t] + g
            g = a[t] * dh[t]
        dfirst[n] = g
        at += length
    w = dh * a * (before - a / m * si * x) * la
    return y, last, dh * m * si, w * (1 - sr), dh * m * x * si * (1 - si), w.sum(0) / rate, dfirst


def blocks(a, b):
    """The largest error of 16 rows, relative to those rows."""
    a, b = a.detach().double().cpu(), b.double()
    pad = -a.shape[0] % 16
    e, n = (torch.nn.functional.pad(t, (0, 0, 0, pad)).unflatten(0, (-1, 16)).flatten(1).norm(dim=1) for t in (a - b, b))
    return float((e / n).max())


def compare(lens, dim, slow, fast, dtype):
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    d = R.make(lens, dim, dtype, seed=sum(lens) + dim, slow=slow, fast=fast)
    want, lossy = plain(d, torch.float64), plain(d, torch.float32)
    m = GatedRecurrence(dim, d["rate"].cuda(), dtype)
    x, start = R.gpu(d, "x", "r", "i"), R.starts(lens)
    state, dstate = R.gpu(d, "state", "dstate")
    carries = torch.empty(m.carries_shape(sum(lens)), device="cuda")
    y = m.forward(*x, state=state, seq_start=start, carries=carries)
    names = ("y", "states", "dx", "dr", "di", "drate", "dstate")
    for c in (None, carries):
        got = y + m.backward(*x, d["dy"].cuda(), state=state, dstate_out=dstate, seq_start=start, carries=c)
        for name, g, w, f in zip(names, got, want, lossy):
            half = 2.0 ** -8 if g.dtype == torch.bfloat16 else 0
            assert R.rel(g, w) <= half + 2 * R.rel(f, w) + 16 * E, (name, R.rel(g, w) / E, R.rel(f, w) / E)
            if g.shape[0] == sum(lens):
                assert blocks(g, w) <= half + 3 * blocks(f, w) + 16 * E, (name, blocks(g, w) / E, blocks(f, w) / E)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("slow,fast", [(1e-5, 1e-2), (1e-3, 0.5)])
@pytest.mark.parametrize("lens,dim", [([9001], 16), ([9001], 264), ([4096, 100, 5000], 264), ([2700, 3, 0, 2697], 24),
                                      ([14000], 136), ([161], 33288)], ids=str)
def test_many_chunks_lose_no_more(lens, dim, slow, fast, dtype):
    compare(lens, dim, slow, fast, dtype)


@pytest.mark.parametrize("rate", [1e-5, 1e-4, 1e-3])
def test_decays_that_are_alike_lose_no_more(rate):
    """Runs of tokens with nearly the same decay next to 1, whose product rounds to the same side each time."""
    compare([20001], 64, rate, 1.01 * rate, "f32")


def test_gradients_beyond_32_bits_of_elements():
    """Two sequences of 2^20 rows of 2304 channels with constant gates and inputs v: far from the ends h = v m / (2 (1 - a)) and
    dh = v / (1 - a), so dr = -v^2 a w / (4 m (1 - a)) (r = i = 0, w = rate / 2), and drate is the sum of twice that over all
    tokens / rate, but for the ends, where it differs by at most 3 times dr's for 1 / (1 - a) <= 21 tokens."""
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB of free memory")
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    T, dim = 1 << 20, 2304
    rate = torch.linspace(0.1, 0.4, dim).cuda()
    m = GatedRecurrence(dim, rate)
    x = torch.ones(2, T, dim, dtype=torch.bfloat16, device="cuda")
    x[1] = -2
    zero = torch.zeros_like(x)
    dx, dr, di, drate, dstate = m.backward(x, zero, zero, x)
    w = rate.double() / 2
    a = torch.exp(-w)
    one = -a * w / (4 * (1 - a * a).sqrt() * (1 - a))
    for n, v in ((0, 1.0), (1, -2.0)):
        for t in (5000, T // 2 + 3, T - 5000):
            assert R.rel(dr[n, t], v * v * one) <= 2.0 ** -8 + 1e-5, (n, t)
    ends = 63 / T  # of the sum; fp32 sums of 80 tokens add at most 80 E
    assert R.rel(drate, 2 * one * T * (1 + 4) / rate.double()) <= ends + 1e-5
    del x, zero, dx, dr, di
    torch.cuda.empty_cache()
