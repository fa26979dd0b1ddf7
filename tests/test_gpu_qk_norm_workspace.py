"""A workspace sized for the longer of two backward calls of the head norm serves the shorter one, whose workgroups are more."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes", [0, 2])
@pytest.mark.parametrize("hq,hk,dim,most,less", [(12, 4, 64, 2017, 2016), (6, 6, 128, 1361, 1360)])
def test_shorter_calls_fit(hq, hk, dim, most, less, axes):
    from fft_long_convolution_libhyena_amd import QKNorm

    gen = torch.Generator().manual_seed(most)
    rn = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    axis = (torch.arange(8) % 2).to(torch.int32).cuda() if axes else None
    m = QKNorm(hq, hk, dim, dtype="f32", w_q=rn(dim), w_k=rn(dim), freq=torch.rand(8, generator=gen).cuda(), axis=axis)
    ws = torch.empty(m.backward_workspace_bytes(most, torch.device("cuda:0")), dtype=torch.uint8, device="cuda")
    for n in (most, less):
        pos = torch.arange(n).cuda()
        pos = pos[:, None].expand(n, 2).contiguous() if axes else pos
        q, k, dq, dk = rn(n, hq, dim), rn(n, hk, dim), rn(n, hq, dim), rn(n, hk, dim)
        for a, b in zip(m.backward(q, k, dq, dk, pos, workspace=ws), m.backward(q, k, dq, dk, pos)):
            assert torch.equal(a, b)
