"""The head norm at the largest number of tokens that fits the card."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_tokens_than_one_launch_has_workgroups():
    """2^27 tokens at 8 a workgroup of 256 threads would be 2^32 threads: workgroups walk on."""
    from fft_long_convolution_libhyena_amd import QKNorm

    tokens, dim = 1 << 27, 136
    if torch.cuda.mem_get_info()[0] < 4 * tokens * dim * 2:  # three arrays and room
        pytest.skip("needs 146 GB of free memory")
    q = torch.zeros(tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 7, (1 << 26) + 3, tokens - 65, tokens - 9, tokens - 8, tokens - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    q[at] = torch.randn(len(at), 1, dim, device="cuda", generator=gen).bfloat16()
    out = QKNorm(1, 1, dim, kind="l2").forward(q, q)
    want = q[at].double() / (q[at].double().square().sum(-1, keepdim=True) + 1e-6).sqrt()
    for x in out:
        assert float((x[at].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
    del q, out, x
    torch.cuda.empty_cache()
