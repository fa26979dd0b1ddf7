"""Plain 64-bit form of the gated linear recurrence for the tests: one token after the other,
exactly as include/hyena.h states it, on the CPU."""
import torch


def make(lens, dim, dtype="bf16", seed=0, slow=1e-3, fast=0.5):
    """Seeded CPU inputs of packed sequences, already rounded to the dtype: a dict of x, r, i, rate,
    state, dy, dstate (and lens). Rates from `slow` to `fast` over the channels."""
    gen = torch.Generator().manual_seed(seed)
    total = sum(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def randn(*s):
        return torch.randn(s, generator=gen)

    return dict(x=randn(total, dim).to(dt), r=(2 * randn(total, dim)).to(dt), i=randn(total, dim).to(dt),
                rate=slow * (fast / slow) ** torch.rand(dim, generator=gen), state=randn(len(lens), dim),
                dy=randn(total, dim).to(dt), dstate=randn(len(lens), dim), lens=list(lens))


def recurrence(x, r, i, rate, h):
    """One sequence, 64-bit [T, dim]: (y, final state)."""
    la = -rate * torch.sigmoid(r)
    a, b = la.exp(), (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(i) * x
    y = []
    for t in range(x.shape[0]):
        h = a[t] * h + b[t]
        y.append(h)
    return (torch.stack(y) if y else torch.zeros_like(x)), h


def forward(d, use_state=True):
    """(y [tokens, dim], states [N, dim]) in 64 bits."""
    y, states, at = [], [], 0
    for n, length in enumerate(d["lens"]):
        h = d["state"][n].double() if use_state else torch.zeros_like(d["state"][n], dtype=torch.float64)
        o, h = recurrence(*(d[k][at:at + length].double() for k in ("x", "r", "i")), d["rate"].double(), h)
        y.append(o)
        states.append(h)
        at += length
    return torch.cat(y), torch.stack(states)


def backward(d, use_state=True, use_dstate=True):
    """Gradients of sum(y * dy) + sum(states * dstate): dx, dr, di, drate, dstate_in."""
    names = ("x", "r", "i", "rate", "state")
    p = dict(d, **{k: d[k].double().requires_grad_() for k in names})
    if not use_state:
        p["state"] = torch.zeros_like(p["state"]).requires_grad_()
    y, states = forward(p)
    loss = (y * d["dy"].double()).sum() + ((states * d["dstate"].double()).sum() if use_dstate else 0)
    return torch.autograd.grad(loss, [p[k] for k in names])


def starts(lens, device="cuda", front=0):
    return torch.tensor([front] + list(lens), dtype=torch.int64).cumsum(0).to(device)


def gpu(d, *names):
    return [d[n].cuda() for n in names]


def rel(a, b):
    """2-norm of the difference over the 2-norm of b (absolute where b is zero)."""
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n else 1.0)
