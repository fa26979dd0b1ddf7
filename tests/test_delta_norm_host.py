"""What the bindings of the delta rule and the norms do on the host before any launch: the
launch itself is replaced, so these run without a GPU (CPU tensors stand for the device's)."""
import pytest
import torch

from fft_long_convolution_libhyena_amd import DeltaRule, QKNorm, binding


@pytest.fixture
def launches(monkeypatch):
    """The calls that would have been launched: (name, arguments)."""
    seen = []
    monkeypatch.setattr(binding, "_gpu_of", lambda t, name: t.device)
    monkeypatch.setattr(binding, "_launch", lambda torch, name, fn, device, *args: seen.append((name, args)))
    return seen


def norm_inputs(tokens=3):
    return [torch.zeros(tokens, h, 64, dtype=torch.bfloat16) for h in (2, 1, 2, 1)]


@pytest.mark.parametrize("workspace", [
    torch.empty(1 << 20, dtype=torch.uint8, device="meta"),        # not where q is
    torch.empty(1, dtype=torch.uint8).expand(1 << 20),             # more elements than memory
    torch.empty(1 << 20, dtype=torch.uint8)[::2],
])
def test_norm_backward_refuses_a_workspace_it_cannot_write(launches, workspace):
    m = QKNorm(2, 1, 64, w_q=torch.ones(64), w_k=torch.ones(64))
    with pytest.raises(ValueError):
        m.backward(*norm_inputs(), workspace=workspace)
    assert not launches


def test_norm_backward_takes_a_dense_workspace(launches):
    m = QKNorm(2, 1, 64, w_q=torch.ones(64), w_k=torch.ones(64))
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    m.backward(*norm_inputs(), workspace=ws)
    m.backward(*norm_inputs())
    plain = QKNorm(2, 1, 64)  # no weights: none is needed, and one that is given is not looked at
    plain.backward(*norm_inputs())
    plain.backward(*norm_inputs(), workspace=torch.empty(8, dtype=torch.uint8, device="meta"))
    assert [n for n, _ in launches] == ["hyena_qk_norm_backward"] * 4
    assert launches[0][1][-2:] == (ws.data_ptr(), 1 << 20)
    need = m.backward_workspace_bytes(3, torch.device("cpu"))
    assert need > 0 and launches[1][1][-1] == need and launches[2][1][-2:] == launches[3][1][-2:] == (None, 0)


@pytest.mark.parametrize("backward", [False, True])
def test_delta_rule_refuses_a_workspace_it_cannot_write(launches, backward):
    r = DeltaRule(1, 1, 64, 64)
    x = [torch.zeros(1, 3, 1, 64, dtype=torch.bfloat16) for _ in range(3)]
    x += [torch.zeros(1, 3, 1, dtype=torch.bfloat16) for _ in range(2)]
    for ws in (torch.empty(1 << 24, dtype=torch.uint8, device="meta"), torch.empty(1, dtype=torch.uint8).expand(1 << 24)):
        with pytest.raises(ValueError):
            r.backward(*x, x[2], workspace=ws) if backward else r.forward(*x, workspace=ws)
    assert not launches


def test_rows_of_no_sequence_are_cleared_in_what_the_call_allocates(launches):
    """They have no result: o's are dropped, and their gradient is 0. A caller's o is left as it was."""
    r, tokens = DeltaRule(1, 2, 64, 64), 7
    x = [torch.zeros(tokens, h, 64, dtype=torch.bfloat16) for h in (1, 1, 2)]
    x += [torch.zeros(tokens, 2, dtype=torch.bfloat16) for _ in range(2)]
    start = torch.tensor([1, 3, 6])
    cleared = lambda: [(a[:4], list(a[4]), list(a[5])) for n, a in launches if n == "hyena_delta_clear_rows"]  # noqa: E731
    o, _ = r.forward(*x, seq_start=start)
    want = [((2, tokens, start.data_ptr(), 1), [o.data_ptr()], [2 * 64 * 2])]
    assert cleared() == want and launches[-1][0] == "hyena_delta_forward"
    r.forward(*x, seq_start=start, o=o)
    r.forward(*(t[None] for t in x))  # every row belongs to a sequence
    r.backward(*(t[None] for t in x), x[2][None])
    assert cleared() == want
    grads = r.backward(*x, x[2], seq_start=start)[:5]
    want.append(((2, tokens, start.data_ptr(), 5), [t.data_ptr() for t in grads], [128, 128, 256, 4, 4]))
    assert cleared() == want and launches[-1][0] == "hyena_delta_backward"
