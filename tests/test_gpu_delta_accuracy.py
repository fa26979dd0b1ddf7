"""Gated delta rule on the GPU: bf16 results are those of 64 bits, rounded once.

An unrounded result off by d_i rounds to the other side of a border in at most d_i of step_i
cases, and is then one step off: the square of the difference to the exact result's own
rounding is at most sum step_i d_i. Steps are at most 2^-7 of the value, so by Cauchy's
inequality the relative 2-norm of that difference is at most sqrt(2^-7 delta), delta being
that of d. (Rounding an operand to one bf16 part alone makes it 1e-3 and more.)
"""
import math

import pytest
import torch

import _delta as D

pytestmark = pytest.mark.gpu


def rounded(delta):
    return math.sqrt(2.0 ** -7 * delta)


@pytest.mark.parametrize("lens,hk,hv,dk,dv,use_state", [
    ([64], 1, 1, 64, 64, False),
    ([300, 77], 1, 2, 128, 128, True),
    ([150], 2, 4, 72, 40, True),
    ([1900], 1, 1, 64, 64, True),  # cut into pieces
])
def test_outputs_are_rounded_once(lens, hk, hv, dk, dv, use_state):
    """S, u and P enter in two bf16 parts each, off by half a step of the second, 2^-9 of 2^-9;
    the products of second parts are left out, 2^-18 for each of the two sums. Five errors of
    2^-18 in squares, and sums of up to 128 + 64 fp32 terms."""
    from fft_long_convolution_libhyena_amd import DeltaRule

    d = D.make(lens, hk, hv, dk, dv, "bf16", seed=dk + len(lens))
    g = {n: d[n].cuda() for n in ("q", "k", "v", "g", "beta", "state")}
    o, _ = DeltaRule(hk, hv, dk, dv).forward(*(g[n] for n in ("q", "k", "v", "g", "beta")),
                                             state=g["state"] if use_state else None, seq_start=D.starts(lens, "cuda"))
    want = D.forward(d, dk ** -0.5, use_state)[0].to(torch.bfloat16)
    assert D.rel(o, want) <= rounded(math.sqrt(5) * 2.0 ** -18 + 192 * 2.0 ** -24)
