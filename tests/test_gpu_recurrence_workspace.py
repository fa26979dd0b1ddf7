"""One workspace, sized for the longest call, shared with shorter ones whose chunks are cut otherwise and need more
words: eager and captured calls give the bits that they give with workspaces of their own."""
import pytest
import torch

import _recurrence as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,less", [((4096, 768), (2688, 768)), ((2700, 896), (2688, 768)), ((700, 8200), (65, 8192))])
def test_calls_of_either_chunks_share_a_workspace(most, less):
    from fft_long_convolution_libhyena_amd import GatedRecurrence

    data = [R.make([t], dim, "bf16", seed=t) for t, dim in (most, less)]
    rules = [GatedRecurrence(d["rate"].numel(), d["rate"].cuda()) for d in data]
    ins = [[d[k].cuda()[None] for k in ("x", "r", "i", "dy")] for d in data]
    ws = [torch.empty(f(1, most[0]), dtype=torch.uint8, device="cuda")
          for f in (rules[0].workspace_bytes, rules[0].backward_workspace_bytes)]

    def call(k, own=False):
        w = [None, None] if own else ws
        return rules[k].forward(*ins[k][:3], workspace=w[0]) + rules[k].backward(*ins[k], workspace=w[1])

    want = [call(k, own=True) for k in range(2)]
    graphs, outs = [], []
    for k in range(2):
        call(k)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            outs.append(call(k))
    for k in (0, 1, 1, 0, 1):
        for t in outs[k]:
            t.zero_()
        graphs[k].replay()
        eager = call(1 - k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - k]))
