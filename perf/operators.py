"""Cases of the gated delta rule (chunked forward and backward, recurrent step) and of
the query/key head norm with rotation, with their plain forms.

The gated delta rule keeps per sequence and value head a state S [Dk, Dv] (S = the
given initial state, or 0). With a = exp(g), for every token in order:
    S <- a S;   S <- S + beta k (v - S^T k)^T;   o = scale S^T q.
Value heads share query/key heads in groups of Hv / Hk.

The head norm divides each head's vector by its root mean square ("rms") or its
length ("l2"), multiplies by an optional weight and turns the first 2 F components
in pairs by the angles position * freq[0..F).

`run` computes these in plain fp32 torch operations when `own` is false (the delta
rule in chunks of 64 tokens, whose in-chunk coupling is a unit lower triangular
system) and calls the library when it is true.
"""
import math

import torch

own = False

_CHUNK = 64


# --------------------------------------------------------------------------- cases

def listed():
    d = dict(hk=6, hv=6, dk=128, dv=128, dtype="bf16")
    return [
        # one token of one sequence: a width-768 layer answering a single user
        dict(d, name="step one sequence", op="step", n=1, t=1, pool=1),
        # one token of each of 96 sequences whose states sit in a pool, keys shared by two value heads
        dict(name="step batch", op="step", n=96, t=1, pool=128, hk=8, hv=16, dk=128, dv=128, dtype="bf16"),
        # a few drafted tokens each, fp32, heads of 64
        dict(name="step drafts f32", op="step", n=16, t=5, pool=16, hk=12, hv=12, dk=64, dv=64, dtype="f32"),
        # prompts of unequal lengths (one empty, one of a single token) packed behind each other, carried states
        dict(name="prefill ragged", op="forward", lens="1531,1,777,0,64,2050,513", state=True, packed=True, hk=6,
             hv=12, dk=128, dv=128, dtype="bf16"),
        # a training batch of a width-768 layer: 8 sequences of 8192
        dict(d, name="forward 8 x 8192", op="forward", n=8, t=8192, state=False, packed=True),
        # one long document
        dict(d, name="forward 1 x 65536", op="forward", n=1, t=65536, state=True, packed=False),
        # a short odd fp32 batch, value heads of another width
        dict(name="forward 2 x 333 f32", op="forward", n=2, t=333, state=True, packed=False, hk=4, hv=4, dk=64, dv=96,
             dtype="f32"),
        # the training batch's gradients
        dict(d, name="backward 8 x 8192", op="backward", n=8, t=8192, state=False, packed=True),
        # packed fp32 documents with carried states and shared keys, gradients of everything
        dict(name="backward ragged f32", op="backward", lens="700,129,1,450", state=True, packed=False, hk=2, hv=4,
             dk=64, dv=64, dtype="f32"),
        # queries and keys of the training batch, unit length with rotation over the whole head
        dict(name="norm 65536 tokens", op="norm", tokens=65536, hq=6, hk=6, dim=128, rot=64, kind="l2", weights=False,
             pairs=False, far=0, dtype="bf16"),
        # its gradient in the weighted rms form, half of each head rotated
        dict(name="norm backward", op="norm_backward", tokens=16384, hq=12, hk=4, dim=64, rot=16, kind="rms",
             weights=True, pairs=True, far=0, dtype="bf16"),
        # single tokens of a few sequences, far into them
        dict(name="norm 5 tokens", op="norm", tokens=5, hq=6, hk=6, dim=128, rot=32, kind="rms", weights=True,
             pairs=False, far=1000000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["step", "forward", "forward", "backward", "norm", "norm_backward"])
    if op.startswith("norm"):
        dim = rng.choice([32, 64, 96, 128])
        return dict(op=op, tokens=_log(rng, 1, 50000), hq=rng.randint(1, 12), hk=rng.randint(1, 6), dim=dim,
                    rot=rng.choice([0, dim // 8, dim // 4, dim // 2]), kind=rng.choice(["rms", "l2"]),
                    weights=rng.random() < 0.5, pairs=rng.random() < 0.5, far=rng.choice([0, 100000]), dtype=dtype)
    hk = rng.randint(1, 6)
    c = dict(op=op, hk=hk, hv=hk * rng.choice([1, 1, 2, 3]), dk=rng.choice([32, 64, 72, 128]),
             dv=rng.choice([32, 64, 72, 128]), dtype=dtype)
    if op == "step":
        n = _log(rng, 1, 160)
        return dict(c, n=n, t=rng.choice([1, 1, 2, 5]), pool=n + rng.randint(0, 20))
    state, packed = rng.random() < 0.5, rng.random() < 0.5
    if rng.random() < 0.5:
        lens = [0 if rng.random() < 0.1 else _log(rng, 1, 3000) for _ in range(rng.randint(1, 8))] + [rng.randint(1, 200)]
        return dict(c, lens=",".join(map(str, lens)), state=state, packed=packed)
    t = _log(rng, 1, 12000)
    return dict(c, n=max(1, min(8, 16000 // t)), t=t, state=state, packed=packed)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if "lens" in case else [case["t"]] * case["n"]


def _esize(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    e = _esize(case)
    if case["op"].startswith("norm"):
        vals = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        if case["op"] == "norm":
            return {"bytes": 2 * vals * e + 8 * case["tokens"], "flops": 6 * vals}
        return {"bytes": 3 * vals * e + 8 * case["tokens"], "flops": 14 * vals}
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    tokens, seqs = sum(_lens(case)), len(_lens(case))
    qk, vo, gb, st = tokens * hk * dk * 2 * e, tokens * hv * dv * e, tokens * hv * 2 * e, seqs * hv * dk * dv * 4
    if case["op"] == "backward":
        return {"bytes": 2 * (qk + vo + gb) + vo + (3 * st if case["state"] else 0),
                "flops": 22 * tokens * hv * dk * dv}
    states = 2 * st if case["op"] == "step" or case["state"] else st
    return {"bytes": qk + 2 * vo + gb + states, "flops": 7 * tokens * hv * dk * dv}


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"].startswith("norm"):
        n, dim, rot = case["tokens"], case["dim"], case["rot"]
        s["q"], s["k"] = (randn(n, h, dim).to(dt) for h in (case["hq"], case["hk"]))
        s["positions"] = torch.arange(n, device="cuda") + case["far"]
        s["freq"] = 10000.0 ** (-torch.arange(rot, device="cuda", dtype=torch.float32) / rot) if rot else None
        s["w_q"], s["w_k"] = (1 + 0.2 * randn(dim), 1 + 0.2 * randn(dim)) if case["weights"] else (None, None)
        if case["op"] == "norm_backward":
            s["dq_out"], s["dk_out"] = (randn(n, h, dim).to(dt) for h in (case["hq"], case["hk"]))
        if own:
            from fft_long_convolution_libhyena_amd import QKNorm

            s["norm"] = QKNorm(case["hq"], case["hk"], dim, dtype=case["dtype"], kind=case["kind"], eps=1e-6,
                               w_q=s["w_q"], w_k=s["w_k"], freq=s["freq"], pairs=case["pairs"])
        return s
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    lens = _lens(case)
    total = sum(lens)
    rows = (total,) if "lens" in case else (case["n"], case["t"])
    # what a layer has after its short convolution: SiLU of near-normal values, queries and keys of unit length
    q, k, v = (torch.nn.functional.silu(randn(*rows, h, d)) for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    q, k = (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt() for x in (q, k))
    if case.get("packed"):  # views of one projection's rows, as a layer's split leaves them
        parts = torch.cat([x.flatten(-2) for x in (q, k, v)], -1).to(dt)
        s["q"], s["k"], s["v"] = (x.unflatten(-1, (h, -1)) for x, h in zip(
            parts.split([hk * dk, hk * dk, hv * dv], -1), (hk, hk, hv)))
    else:
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
    # decay rates of 1 to 16 per head times a softplus time step around 0.01 .. 0.1, write strengths in (0, 1)
    rate = torch.linspace(1, 16, hv, device="cuda")
    s["g"] = (-rate * torch.nn.functional.softplus(randn(*rows, hv) - 4)).to(dt)
    s["beta"] = torch.sigmoid(randn(*rows, hv)).to(dt)
    s["scale"] = dk ** -0.5
    s["lens"] = lens
    if "lens" in case:
        s["seq_start"] = torch.tensor([0] + lens, device="cuda").cumsum(0)
        s["pad"] = _padding(lens)
    else:
        s["seq_start"] = None
    if case["op"] == "step":
        s["states"] = 0.3 * randn(case["pool"], hv, dk, dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device="cuda")[:case["n"]].to(torch.int32)
    elif case["state"]:
        s["state"] = 0.3 * randn(len(lens), hv, dk, dv)
    else:
        s["state"] = None
    if case["op"] == "backward":
        s["do"] = randn(*rows, hv, dv).to(dt)
        s["dstate"] = randn(len(lens), hv, dk, dv) if case["state"] else None
    if own:
        from fft_long_convolution_libhyena_amd import DeltaRule

        s["rule"] = DeltaRule(hk, hv, dk, dv, dtype=case["dtype"])
    return s


def _padding(lens):
    """Index of every packed token in the padded [sequences, longest] layout."""
    longest = max(lens)
    return torch.cat([torch.arange(n) + i * longest for i, n in enumerate(lens)]).cuda()


# --------------------------------------------------------------------------- passes

def run(s):
    c = s["case"]
    if c["op"] == "norm":
        if own:
            return s["norm"].forward(s["q"], s["k"], s["positions"])
        turn = _angles(s)
        return tuple(_norm(s[x], s["w_" + x], turn, c) for x in "qk")
    if c["op"] == "norm_backward":
        if own:
            dq, dk, dwq, dwk = s["norm"].backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["positions"])
        else:
            turn = _angles(s)
            (dq, dwq), (dk, dwk) = (_norm_backward(s[x], s["w_" + x], s[f"d{x}_out"], turn, c) for x in "qk")
        return (dq, dk, dwq, dwk) if c["weights"] else (dq, dk)
    if c["op"] == "step":
        if own:
            o = s["rule"].step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], slots=s["slots"],
                               scale=s["scale"])
            return o, s["states"]
        return _step(s)
    if c["op"] == "forward":
        if own:
            return s["rule"].forward(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], scale=s["scale"],
                                     seq_start=s["seq_start"])
        return _forward(s)
    if own:
        out = s["rule"].backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], state=s["state"],
                                 dstate_out=s["dstate"], scale=s["scale"], seq_start=s["seq_start"])
        return out if s["state"] is not None else out[:5]
    return _backward(s)


def _angles(s):
    """cos and sin of position * freq [tokens, 1, F]; the angles are formed and reduced in 64 bits."""
    if s["freq"] is None:
        return None
    a = s["positions"].double()[:, None, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def _turn(x, turn, pairs, back=False):
    if turn is None:
        return x
    cos, sin = turn
    f = cos.shape[-1]
    sin = -sin if back else sin
    a, b = (x[..., 0:2 * f:2], x[..., 1:2 * f:2]) if pairs else (x[..., :f], x[..., f:2 * f])
    u, w = a * cos - b * sin, a * sin + b * cos
    head = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([head, x[..., 2 * f:]], -1)


def _inverse_norm(x, kind):
    ss = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((ss / x.shape[-1] if kind == "rms" else ss) + 1e-6)


def _norm(x, w, turn, c):
    x = x.float()
    y = x * _inverse_norm(x, c["kind"])
    if w is not None:
        y = y * w
    return _turn(y, turn, c["pairs"]).to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)


def _norm_backward(x, w, dy, turn, c):
    dt = x.dtype
    x, dy = x.float(), _turn(dy.float(), turn, c["pairs"], back=True)
    r = _inverse_norm(x, c["kind"])
    xn = x * r
    dw = None
    if w is not None:
        dw = (dy * xn).sum((0, 1))
        dy = dy * w
    along = (dy * xn).sum(-1, keepdim=True)
    if c["kind"] == "rms":
        along = along / x.shape[-1]
    return (r * (dy - xn * along)).to(dt), dw


def _heads(x, s, group=1):
    """[tokens..., H, D] or [tokens..., H] -> fp32 [sequences, H * group, T, ...], packed tokens padded with zeros."""
    x = x.float()
    if s["seq_start"] is not None:
        n, longest = len(s["lens"]), max(s["lens"])
        x = x.new_zeros((n * longest, *x.shape[1:])).index_copy(0, s["pad"], x).unflatten(0, (n, longest))
    x = x.transpose(1, 2)
    return x.repeat_interleave(group, 1) if group > 1 else x


def _tokens(x, s):
    """The inverse of _heads, without the groups."""
    x = x.transpose(1, 2)
    return x.flatten(0, 1)[s["pad"]] if s["seq_start"] is not None else x


def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower triangular a [..., 64, 64], joining diagonal blocks of doubling size."""
    n = a.shape[-1]
    t = a.new_ones((*a.shape[:-2], n, 1, 1))
    while t.shape[-1] < n:
        m = t.shape[-1]
        low = a.unflatten(-1, (-1, 2, m)).unflatten(-4, (-1, 2, m))[..., 1, :, :, 0, :]  # [.., block, m, block, m]
        low = low.diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        t1, t2 = t[..., 0::2, :, :], t[..., 1::2, :, :]
        t = torch.cat([torch.cat([t1, torch.zeros_like(t1)], -1), torch.cat([-(t2 @ low @ t1), t2], -1)], -2)
    return t[..., 0, :, :]


def _chunked(q, k, v, g, beta, state, scale):
    """fp32 [N, H, T, ...] -> (o, final state). In a chunk with decays D[i, j] = exp(g[j+1] + .. + g[i]):
    (I + tril(beta D k k^T, -1)) u = beta (v - decayed k S);  o = scale (decayed q S + tril(D q k^T) u);
    S <- decayed S + (decays to the chunk's end * k)^T u."""
    t, c = q.shape[2], _CHUNK
    pad = -t % c

    def chunks(x):
        return torch.cat([x, x.new_zeros((*x.shape[:2], pad, *x.shape[3:]))], 2).unflatten(2, (-1, c))

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    total = g.double().cumsum(-1)
    lower = torch.ones(c, c, device=q.device).tril().bool()
    decay = (total[..., :, None] - total[..., None, :]).masked_fill(~lower, -math.inf).float().exp()
    to_end = (total[..., -1:] - total).float().exp()[..., None]
    from_start = total.float().exp()[..., None]
    kt = k.transpose(-1, -2).contiguous()
    inv = _unit_lower_inverse((beta[..., None] * decay * (k @ kt)).tril(-1))
    mix = decay * (q @ kt)
    k_in, q_in, k_out = from_start * k, from_start * q, (to_end * k).transpose(-1, -2).contiguous()
    out = []
    for i in range(q.shape[2]):
        u = inv[:, :, i] @ (beta[:, :, i, :, None] * (v[:, :, i] - k_in[:, :, i] @ state))
        out.append(q_in[:, :, i] @ state + mix[:, :, i] @ u)
        state = from_start[:, :, i, -1:] * state + k_out[:, :, i] @ u
    return scale * torch.cat(out, 2)[:, :, :t], state


def _operands(s):
    c = s["case"]
    group = c["hv"] // c["hk"]
    state = s["state"]
    if state is None:
        state = torch.zeros(len(s["lens"]), c["hv"], c["dk"], c["dv"], device="cuda")
    return [_heads(s["q"], s, group), _heads(s["k"], s, group), _heads(s["v"], s), _heads(s["g"], s),
            _heads(s["beta"], s), state]


def _forward(s):
    o, state = _chunked(*_operands(s), s["scale"])
    return _tokens(o, s).to(s["v"].dtype), state


def _backward(s):
    c = s["case"]
    leaves = [x.detach().float().requires_grad_() for x in (s["q"], s["k"], s["v"], s["g"], s["beta"])]
    p = dict(s, **dict(zip(("q", "k", "v", "g", "beta"), leaves)))
    if s["state"] is not None:
        p["state"] = s["state"].detach().requires_grad_()
    with torch.enable_grad():
        o, state = _chunked(*_operands(p), s["scale"])
        o = _tokens(o, s)
        if s["state"] is None:
            grads = torch.autograd.grad(o, leaves, s["do"].float())
        else:
            grads = torch.autograd.grad((o, state), leaves + [p["state"]], (s["do"].float(), s["dstate"]))
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    return tuple(x.to(dt) for x in grads[:5]) + tuple(grads[5:])


def _step(s):
    group = s["case"]["hv"] // s["case"]["hk"]
    q, k, v, g, beta = (s[x].float() for x in ("q", "k", "v", "g", "beta"))
    q, k = (x.repeat_interleave(group, 2) for x in (q, k))
    st = s["states"][s["slots"].long()]
    out = []
    for t in range(q.shape[1]):
        st = st * g[:, t].exp()[..., None, None]
        err = beta[:, t, :, None] * (v[:, t] - (st * k[:, t, :, :, None]).sum(-2))
        st = st + k[:, t, :, :, None] * err[:, :, None, :]
        out.append(s["scale"] * (st * q[:, t, :, :, None]).sum(-2))
    s["states"].index_copy_(0, s["slots"].long(), st)  # the pool is updated in place, as a serving loop does
    return torch.stack(out, 1).to(s["v"].dtype), s["states"]


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    lens, hv, group = _lens(case), case["hv"], case["hv"] // case["hk"]
    n, longest = len(lens), max(lens)

    def rows(x, rep=1):  # token-major [T, N, H, ...]
        x = x.double()
        if "lens" in case:
            y = x.new_zeros((n, longest, *x.shape[1:]))
            at = 0
            for i, m in enumerate(lens):
                y[i, :m] = x[at:at + m]
                at += m
            x = y
        x = x.transpose(0, 1)
        return x.repeat_interleave(rep, 2) if rep > 1 else x

    def back(x):  # [T, N, H, ...] -> as the input
        return torch.cat([x[:m, i] for i, m in enumerate(lens)]) if "lens" in case else x.transpose(0, 1)

    q, k, v, g, b = rows(s["q"], group), rows(s["k"], group), rows(s["v"]), rows(s["g"]), rows(s["beta"])
    a = g.exp()[..., None, None]
    scale = s["scale"]
    if case["op"] == "step":
        st = s["states"].double()[s["slots"].long()]
    elif s["state"] is not None:
        st = s["state"].double()
    else:
        st = torch.zeros(n, hv, case["dk"], case["dv"], device="cuda", dtype=torch.float64)

    def advance(st, t):
        st = a[t] * st
        e = v[t] - torch.matmul(k[t][..., None, :], st)[..., 0, :]
        return st, e, st + k[t][..., :, None] * (b[t][..., None] * e)[..., None, :]

    if case["op"] != "backward":
        o = torch.empty_like(v)
        for t in range(v.shape[0]):
            st = advance(st, t)[2]
            o[t] = scale * torch.matmul(q[t][..., None, :], st)[..., 0, :]
        if case["op"] == "step":
            full = s["states"].double()
            full[s["slots"].long()] = st
            return back(o), full
        return back(o), st

    do = rows(s["do"])
    ds = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(st)
    span, marks = 128, []
    for t in range(v.shape[0]):
        if t % span == 0:
            marks.append(st)
        st = advance(st, t)[2]
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, b))
    for m in reversed(range(len(marks))):
        st, kept = marks[m], []
        for t in range(m * span, min((m + 1) * span, v.shape[0])):
            kept.append(advance(st, t))
            st = kept[-1][2]
        for t in reversed(range(m * span, min((m + 1) * span, v.shape[0]))):
            before, e, after = kept.pop()
            dq[t] = scale * torch.matmul(after, do[t][..., None])[..., 0]
            ds = ds + scale * q[t][..., :, None] * do[t][..., None, :]
            w = torch.matmul(k[t][..., None, :], ds)[..., 0, :]
            db[t] = (w * e).sum(-1)
            de = b[t][..., None] * w
            dv[t] = de
            dk[t] = torch.matmul(ds, (b[t][..., None] * e)[..., None])[..., 0] - torch.matmul(before, de[..., None])[..., 0]
            ds = ds - k[t][..., :, None] * de[..., None, :]
            dg[t] = (ds * before).sum((-1, -2))
            ds = a[t] * ds
    if group > 1:
        dq, dk = (x.unflatten(2, (-1, group)).sum(3) for x in (dq, dk))
    out = tuple(back(x) for x in (dq, dk, dv, dg, db))
    return out + (ds,) if s["state"] is not None else out


def _exact_norm(case, s):
    f, dim, pairs = case["rot"], case["dim"], case["pairs"]
    idx = torch.arange(f, device="cuda")
    first, second = (2 * idx, 2 * idx + 1) if pairs else (idx, idx + f)
    z = torch.ones(case["tokens"], 1, f, dtype=torch.complex128, device="cuda")
    if f:
        ang = s["positions"].double()[:, None, None] * s["freq"].double()
        z = torch.polar(torch.ones_like(ang), ang)
    grads, outs, dws = [], [], []
    for name in "qk":
        x, w = s[name].double(), s["w_" + name]
        w = torch.ones(dim, device="cuda", dtype=torch.float64) if w is None else w.double()
        size = (x * x).sum(-1, keepdim=True) / (dim if case["kind"] == "rms" else 1) + 1e-6
        if case["op"] == "norm":
            y = x / size.sqrt() * w
            r = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = r.real, r.imag
            outs.append(y)
            continue
        dy = s[f"d{name}_out"].double().clone()
        r = torch.complex(dy[..., first], dy[..., second]) * z.conj()
        dy[..., first], dy[..., second] = r.real, r.imag
        dws.append((dy * x / size.sqrt()).sum((0, 1)))
        dy = dy * w
        dot = (dy * x).sum(-1, keepdim=True) / (dim if case["kind"] == "rms" else 1)
        grads.append(dy / size.sqrt() - x * dot / size ** 1.5)
    if case["op"] == "norm":
        return tuple(outs)
    return tuple(grads + dws) if case["weights"] else tuple(grads)
