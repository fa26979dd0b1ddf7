"""A step of more tokens than whole sequences may have: every row has the bits that it has in a small call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_more_than_2_to_the_23_chunks_of_tokens():
    B, T, dim = 1 << 23, 81, 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    m = GatedRecurrence(dim, torch.linspace(0.05, 0.4, dim).cuda())
    x = torch.empty(B, T, dim, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    states = torch.arange(B, device="cuda").remainder(7).float()[:, None].expand(B, dim).contiguous()
    before = states.clone()
    y = m.step(x, x, x, states)
    for rows in (slice(0, 100), slice(B // 2 - 50, B // 2 + 50), slice(B - 100, B)):
        s = before[rows].clone()
        part = x[rows].contiguous()
        assert torch.equal(m.step(part, part, part, s), y[rows]) and torch.equal(s, states[rows])
    del x, y
    torch.cuda.empty_cache()
