"""The residual norm's 8-bit codes are those of y / scale, rounded to nearest even: bit for bit, next to the borders
between two codes too.

Rows of +-1 have a mean square of exactly 1 (256, 1024 and 4096 columns; eps of 1e-30 is lost in it), so y = +-w exactly
and the weights choose it. The scale is the largest |w| / 448 in fp32, rounded once, as on the CPU.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# halfway between neighbouring e4m3 values, from its smallest step (2^-9) up
TIES = [(2 * k + 1) * 2.0 ** -10 for k in range(16)] + [(2 * m + 1) * 2.0 ** (e - 4) for e in range(-5, 9) for m in range(8, 16)]
TIES = torch.tensor([t for t in TIES if t < 448])


def weights(dim, seed):
    """Values next to the borders for a largest one of its own in every 128 columns, largest at the end."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.empty(dim)
    for at in range(0, dim, 128):
        n = min(128, dim - at)
        most = 2.0 ** torch.randint(-3, 4, (1,), generator=gen).item() * (1 + torch.rand(1, generator=gen))
        t = TIES[torch.randint(len(TIES), (n,), generator=gen)]
        w[at:at + n] = t * (most / 448)
        w[at + n - 1] = most
    return w


def codes(y, block):
    """(codes, scales, whether a product with the scale's reciprocal would have given another code)."""
    b = y.unflatten(-1, (-1, block))
    scale = b.abs().amax(-1, keepdim=True) / 448
    q = (b / scale).to(torch.float8_e4m3fn)
    other = (b * (1 / scale)).to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), scale[..., 0], (q.float() != other.float()).flatten(-2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("dim", [256, 1024, 4096])
def test_codes_are_those_of_a_division(dim, block, dtype):
    from fft_long_convolution_libhyena_amd import ResidualNorm

    differ = 0
    for seed in range(8):
        gen = torch.Generator().manual_seed(100 + seed)
        sign = 2.0 * torch.randint(0, 2, (5, dim), generator=gen) - 1
        w = weights(dim, seed)
        if block == 0:  # one scale a row: ties of that one
            w = (TIES[torch.randint(len(TIES), (dim,), generator=gen)] * (w.max() / 448)).index_fill(0, torch.tensor([dim - 1]), float(w.max()))
        x = sign.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
        q, scales, _ = ResidualNorm(dim, w.cuda(), dtype=dtype, eps=1e-30, bits8=True, block=block).forward(x)
        want, by, other = codes(sign * w, block or dim)
        assert torch.equal(scales.cpu(), by)
        assert torch.equal(q.view(torch.uint8).cpu(), want), seed
        differ += int(other.sum())
    assert differ > 20  # the inputs tell a division from a product


def test_signs_of_zeros():
    from fft_long_convolution_libhyena_amd import ResidualNorm

    x = torch.ones(1, 256)
    w = torch.zeros(256)
    w[1::2] = -0.0
    w[7] = 3.0
    q, _, _ = ResidualNorm(256, w.cuda(), dtype="f32", eps=1e-30, bits8=True).forward(x.cuda())
    assert torch.equal(q.view(torch.uint8).cpu(), codes(x * w, 256)[0])
