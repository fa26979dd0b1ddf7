"""Plain 64-bit form of the gated delta rule for the tests: one token after the other,
exactly as include/hyena.h states it, on the CPU."""
import torch

EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative to the value


def make(lens, hk, hv, dk, dv, dtype="bf16", seed=0, packed_rows=False, unit=True, decay=0.1):
    """Seeded CPU inputs of packed sequences, already rounded to the dtype: a dict of
    q, k, v, g, beta, state, do, dstate (and lens)."""
    gen = torch.Generator().manual_seed(seed)
    total = sum(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def randn(*s):
        return torch.randn(s, generator=gen)

    q, k = randn(total, hk, dk), randn(total, hk, dk) + 0.5
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6) for x in (q, k))
    d = dict(q=q.to(dt), k=k.to(dt), v=randn(total, hv, dv).to(dt),
             g=(-decay * torch.rand((total, hv), generator=gen)).to(dt),
             beta=torch.sigmoid(randn(total, hv)).to(dt), state=randn(len(lens), hv, dk, dv) * 0.3,
             do=randn(total, hv, dv).to(dt), dstate=randn(len(lens), hv, dk, dv))
    if packed_rows:  # q, k, v as column ranges of one projection's rows
        rows = torch.cat([d[x].flatten(1) for x in ("q", "k", "v")], 1)
        d["rows"] = rows
    d["lens"] = list(lens)
    return d


def recurrence(q, k, v, g, beta, state, scale):
    """One sequence, 64-bit tensors [T, H, ...] with q, k of Hk heads: (o, final state)."""
    group = v.shape[1] // k.shape[1]
    o = []
    for t in range(v.shape[0]):
        kt, qt = k[t].repeat_interleave(group, 0), q[t].repeat_interleave(group, 0)
        state = state * g[t].exp()[:, None, None]
        err = v[t] - (state * kt[:, :, None]).sum(1)
        state = state + kt[:, :, None] * (beta[t][:, None] * err)[:, None, :]
        o.append(scale * (state * qt[:, :, None]).sum(1))
    return (torch.stack(o) if o else torch.zeros_like(v)), state


def forward(d, scale, use_state=True):
    """(o [tokens, hv, dv], states [N, hv, dk, dv]) in 64 bits."""
    outs, states, at = [], [], 0
    x = {n: d[n].double() for n in ("q", "k", "v", "g", "beta")}
    for i, n in enumerate(d["lens"]):
        s0 = d["state"][i].double() if use_state else torch.zeros_like(d["state"][i]).double()
        o, s = recurrence(*(x[m][at:at + n] for m in ("q", "k", "v", "g", "beta")), s0, scale)
        outs.append(o)
        states.append(s)
        at += n
    return torch.cat(outs), torch.stack(states)


def backward(d, scale, use_state=True, use_dstate=True):
    """Gradients of sum(o * do) + sum(state * dstate): dq, dk, dv, dg, dbeta, dstate_in."""
    leaves = {n: d[n].double().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    s0 = (d["state"].double() if use_state else torch.zeros_like(d["state"]).double()).requires_grad_()
    x = dict(d, **leaves, state=s0)
    outs, states, at = [], [], 0
    for i, n in enumerate(d["lens"]):
        o, s = recurrence(*(x[m][at:at + n] for m in ("q", "k", "v", "g", "beta")), s0[i], scale)
        outs.append(o)
        states.append(s)
        at += n
    loss = (torch.cat(outs) * d["do"].double()).sum()
    if use_dstate:
        loss = loss + (torch.stack(states) * d["dstate"].double()).sum()
    grads = torch.autograd.grad(loss, [leaves[n] for n in ("q", "k", "v", "g", "beta")] + [s0], allow_unused=True)
    return [torch.zeros_like(y) if z is None else z for z, y in
            zip(grads, [leaves[n] for n in ("q", "k", "v", "g", "beta")] + [s0])]


def starts(lens, device):
    return torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0).to(device)


def rel(a, b):
    """2-norm of the difference over the 2-norm of b (absolute where b is zero)."""
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    n = float(b.norm())
    return float((a - b).norm()) / (n if n else 1.0)
