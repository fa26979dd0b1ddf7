"""Gated delta rule on the GPU: bf16 results are those of 64 bits, rounded once.

An unrounded result off by d_i rounds to the other side of a border in at most d_i of step_i
cases, and is then one step off: the square of the difference to the exact result's own
rounding is at most sum step_i d_i. Steps are at most 2^-7 of the value, so by Cauchy's
inequality the relative 2-norm of that difference is at most sqrt(2^-7 delta), delta being
that of d. (Rounding an operand to one bf16 part alone makes it 1e-3 and more.)

A first bf16 part leaves at most 2^-8 of a value and a second rounds what is left, by at most
2^-9 of it: TWO. A product of two such values leaves out that of the second parts: CROSS. Such
errors add in squares.
"""
import math

import pytest
import torch

import _delta as D

pytestmark = pytest.mark.gpu

TWO, CROSS = 2.0 ** -17, 2.0 ** -16


def rounded(delta):
    return math.sqrt(2.0 ** -7 * delta)


@pytest.mark.parametrize("lens,hk,hv,dk,dv,use_state", [
    ([64], 1, 1, 64, 64, False),
    ([300, 77], 1, 2, 128, 128, True),
    ([150], 2, 4, 72, 40, True),
    ([1900], 1, 1, 64, 64, True),  # cut into pieces
])
def test_outputs_are_rounded_once(lens, hk, hv, dk, dv, use_state):
    """S, u and P enter in two bf16 parts each, and the products of P's and u's second parts are
    left out (q has one part); sums of up to 128 + 64 fp32 terms."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    d = D.make(lens, hk, hv, dk, dv, "bf16", seed=dk + len(lens))
    g = {n: d[n].cuda() for n in ("q", "k", "v", "g", "beta", "state")}
    o, _ = DeltaRule(hk, hv, dk, dv).forward(*(g[n] for n in ("q", "k", "v", "g", "beta")),
                                             state=g["state"] if use_state else None, seq_start=D.starts(lens, "cuda"))
    want = D.forward(d, dk ** -0.5, use_state)[0].to(torch.bfloat16)
    assert D.rel(o, want) <= rounded(math.sqrt(3 * TWO ** 2 + CROSS ** 2) + 192 * 2.0 ** -24)


def with_residuals(lens, hk, hv, dk, dv, dtype, seed, share):
    """Inputs whose v is what the state answers to k, but for a residual of `share` of it."""
    d = D.make(lens, hk, hv, dk, dv, dtype, seed=seed)
    at = 0
    for n, state in zip(lens, d["state"].double()):
        for t in range(at, at + n):
            one = [d[m][t:t + 1].double() for m in ("q", "k", "v", "g", "beta")]
            kt = one[1][0].repeat_interleave(hv // hk, 0)
            answer = (state * one[3][0].exp()[:, None, None] * kt[:, :, None]).sum(1)
            way = one[2][0] / one[2][0].norm(dim=-1, keepdim=True)
            d["v"][t] = (answer + share * answer.norm(dim=-1, keepdim=True) * way).to(d["v"].dtype)
            one[2] = d["v"][t:t + 1].double()
            state = D.recurrence(*one, state, 1.0)[1]
        at += n
    return d


def gradients(d, dims, dtype="bf16", scale=None):
    from fft_long_convolution_libhyena_amd import DeltaRule

    return DeltaRule(*dims, dtype=dtype).backward(
        *(d[n].cuda() for n in ("q", "k", "v", "g", "beta", "do")), state=d["state"].cuda(), dstate_out=d["dstate"].cuda(),
        scale=scale, seq_start=D.starts(d["lens"], "cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [0.05, 0.01])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([150, 64], 1, 2, 128, 128), ([100], 2, 2, 64, 72)])
def test_strengths_gradients_where_the_state_predicts_the_values(lens, hk, hv, dk, dv, share, dtype):
    """dbeta is r . (v - answer): with v close to the answer neither may enter rounded by itself.
    The residual comes from products with S and T in two (fp32: three) parts (and sums of 192
    terms of 2^-24) of an answer 1 / share times as large; r, the residual and the result are
    rounded once at most in bf16 calls (fp32: two chained sums)."""
    d = with_residuals(lens, hk, hv, dk, dv, dtype, dk, share)
    d["beta"][::7] = 0  # no residual may need beta to be seen
    got, want = gradients(d, (hk, hv, dk, dv), dtype)[4], D.backward(d, dk ** -0.5)[4]
    tol = (math.sqrt(3) * 2.0 ** -8 + math.sqrt(2) * TWO / share if dtype == "bf16"
           else 192 * 2.0 ** -24 * (2 + 1 / share))
    assert D.rel(got, want) <= tol
    assert D.rel(got[::7], want[::7]) <= tol


def test_values_without_strength_do_not_reach_other_gradients():
    """A token with beta = 0 writes nothing, however large its value is."""
    dims = (1, 2, 64, 64)
    d = D.make([150], *dims, "bf16", seed=3)
    d["beta"][40] = 0
    plain = gradients(d, dims)
    d["v"][40] = 1e15
    got, want = gradients(d, dims), D.backward(d, 64 ** -0.5)
    for i in (0, 1, 2, 3, 5):  # 1e15 times 2^-90 is 1e-12
        assert D.rel(got[i], plain[i]) <= 2.0 ** -8, i
    rest = [t for t in range(150) if t != 40]
    assert D.rel(got[4][rest], plain[4][rest]) <= 2.0 ** -8
    assert D.rel(got[4][40], want[4][40]) <= 2 * 2.0 ** -8


@pytest.mark.parametrize("lens,hk,hv,dk,dv", [
    ([64], 1, 1, 64, 64),
    ([300, 77], 1, 2, 128, 128),
    ([150, 0, 33], 2, 4, 72, 40),
    ([130], 1, 1, 40, 256),
    ([1900], 1, 2, 64, 64),  # cut into pieces
])
def test_gradients_are_rounded_once(lens, hk, hv, dk, dv):
    """Seven operands of two parts on the way to u or r and two in the gradients' own products (W,
    M), four that were kept in 24 bits, 16 of them significant, and so are off by 2^-16 (S0, dS1,
    u, r); products of second parts are left out in five (T e and T^T dU, u dS1^T, r S0^T,
    r u^T); three chained sums of up to 192 fp32 terms. dg sums a chunk's
    differences of such products, which partly cancel: twice that."""
    d = D.make(lens, hk, hv, dk, dv, "bf16", seed=dk + len(lens))
    delta = math.sqrt(9 * TWO ** 2 + 4 * 2.0 ** -32 + 5 * CROSS ** 2) + 3 * 192 * 2.0 ** -24
    got, want = gradients(d, (hk, hv, dk, dv)), D.backward(d, dk ** -0.5)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        tol = rounded(2 * delta if name == "dg" else delta)
        off = D.rel(got[i], want[i].to(torch.bfloat16))
        assert off <= tol, (name, off, tol)


def test_states_take_what_is_written_in_fp32():
    """With keys along the axes and no state before, the state's row i is exp(G_last - G_i) beta_i
    v_i alone, of which a bf16 call's operands hold all 24 bits in three parts: off by 2^-24 each
    for two products, the decay (twice, its exponent and the exp2) and the third part. Two parts
    would leave 2^-17 at most, 2e-6 in the mean."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    lens, hv, dk, dv = [64, 50], 2, 64, 72
    d = D.make(lens, 1, hv, dk, dv, "bf16", seed=4)
    d["k"] = torch.eye(64)[torch.cat([torch.randperm(n, generator=torch.Generator().manual_seed(n)) for n in lens])][:, None].bfloat16()
    g = {n: d[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    _, s = DeltaRule(1, hv, dk, dv).forward(*g.values(), seq_start=D.starts(lens, "cuda"))
    assert D.rel(s, D.forward(d, 1.0, use_state=False)[1]) <= 5 * 2.0 ** -24


@pytest.mark.parametrize("lens,dk,dv", [([64, 30], 64, 64), ([300, 77], 128, 72)])
def test_state_gradients_take_the_outputs_in_fp32(lens, dk, dv):
    """With beta = 0 the initial state's gradient is the sum of exp(G) scale q do over the tokens
    and the decayed final one: exact products of q with three parts of the rest, off by 2^-24
    for each of two products and a decay (twice), and fp32 sums of 64 terms and of the chunks;
    errors add in squares. Two parts would leave 2e-6 and more."""
    d = D.make(lens, 1, 2, dk, dv, "bf16", seed=dk)
    d["beta"].zero_()
    got, want = gradients(d, (1, 2, dk, dv))[5], D.backward(d, dk ** -0.5)[5]
    assert D.rel(got, want) <= math.sqrt(4 + 64 + max(lens) // 64 + 1) * 2.0 ** -24


def test_state_gradients_follow_the_residuals_in_fp32():
    """With keys along the axes r is dU and the initial state's gradient a sum of -exp(G) beta k r
    and exp(G) scale q do: here of the first alone, do reaching it through P^T (q = k), with
    all of dU and r in three parts. Off by 2^-24 for P's product and decay, three products and
    two decays more."""
    lens, hv, dk, dv = [64], 2, 64, 64
    d = D.make(lens, 1, hv, dk, dv, "bf16", seed=6)
    d["k"] = torch.eye(64)[:, None].bfloat16()
    d["q"] = d["k"].clone()
    d["dstate"].zero_()
    got, want = gradients(d, (1, hv, dk, dv))[5], D.backward(d, dk ** -0.5)[5]
    # exp(G) (scale do - beta r), r = scale do: exact but for what the two leave, 1 / (1 - beta) more
    size = (d["do"].double() ** 2 * dk ** -1.0).sum().sqrt()
    assert float((got.double().cpu() - want).norm()) <= 8 * 2.0 ** -24 * float(size)
