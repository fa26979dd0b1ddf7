"""The delta rule's limits of size, found on the host: what a launch cannot take is refused
before anything is enqueued, what it can is not."""
import ctypes

import pytest

from test_delta_args import INVALID, P, UNSUPPORTED, WORKSPACE, backward, forward, inputs, lib, params  # noqa: F401


def small(**kw):
    return params(**dict(dict(heads_k=1, heads_v=1, dim_k=8, dim_v=8), **kw))


def rows(p):
    return inputs(ldq=p.heads_k * p.dim_k, ldk=p.heads_k * p.dim_k, ldv=p.heads_v * p.dim_v)


# dtype (0 fp32, 1 bf16), value heads, dim_v, sequences of one token that a launch no longer takes
LIMITS = [(1, 1, 8, 1 << 24), (1, 4, 64, 1 << 21), (0, 4, 64, (1 << 32) // 192 // 16 + 2), (1, 2, 256, 1 << 20),
          (0, 2, 256, (1 << 32) // 192 // 32 + 4)]


@pytest.mark.parametrize("dtype,hv,dv,N", LIMITS)
def test_whole_sequences(lib, dtype, hv, dv, N):  # noqa: F811
    p = small(heads_v=hv, dim_v=dv, dtype=dtype)
    for start in (None, P):
        assert forward(lib, p, N=N, tokens=N, start=start, i=rows(p)) == UNSUPPORTED
        assert backward(lib, p, N=N, tokens=N, start=start, i=rows(p)) == UNSUPPORTED
        assert lib.hyena_delta_workspace_bytes(ctypes.byref(p), N, N, start) == 0
        assert lib.hyena_delta_backward_workspace_bytes(ctypes.byref(p), N, N, start) == 0
    less = N - 16
    assert forward(lib, p, N=less, tokens=less, i=rows(p), ws=None) == WORKSPACE
    assert backward(lib, p, N=less, tokens=less, i=rows(p), ws=None) == WORKSPACE


def test_many_chunks_of_one_sequence(lib):  # noqa: F811
    p, n = small(), 1 << 30  # 2^24 chunks
    assert forward(lib, p, N=1, tokens=n, i=rows(p)) == UNSUPPORTED
    assert forward(lib, p, N=1, tokens=n - 64, i=rows(p), ws=None) == WORKSPACE


@pytest.mark.parametrize("hv,dv,B", [(1, 128, 1 << 24), (4, 128, 1 << 22), (4, 256, 1 << 22), (4, 64, 1 << 23)])
def test_steps(lib, hv, dv, B):  # noqa: F811
    p = small(heads_v=hv, dim_v=dv)
    assert lib.hyena_delta_step(ctypes.byref(p), B, 1, ctypes.byref(rows(p)), P, B, None, P, None) == UNSUPPORTED


def test_no_tokens_need_no_workspace(lib):  # noqa: F811
    """Packed sequences that are all empty have no chunks, whatever their number."""
    for start in (None, P):
        for N in (1, 2, 1000):
            assert lib.hyena_delta_workspace_bytes(ctypes.byref(params()), N, 0, start) == 0
            assert lib.hyena_delta_backward_workspace_bytes(ctypes.byref(params()), N, 0, start) == 0


@pytest.mark.parametrize("which", ["ldq", "ldk", "ldv"])
def test_strides_between_tokens(lib, which):  # noqa: F811
    """At most 2^22 elements: a chunk's 64 rows are addressed with 32 bits."""
    assert forward(lib, i=inputs(**{which: 1 << 22}), ws=None) == WORKSPACE
    assert forward(lib, i=inputs(**{which: (1 << 22) + 8})) == INVALID
    assert backward(lib, i=inputs(**{which: 1 << 22}), ws=None) == WORKSPACE
    assert backward(lib, i=inputs(**{which: (1 << 22) + 8})) == INVALID


@pytest.mark.parametrize("kw", [dict(heads_k=1, heads_v=65528, dim_v=72), dict(heads_k=65528, heads_v=65528, dim_k=72, dim_v=8)])
def test_rows_wider_than_a_stride(lib, kw):  # noqa: F811
    p, wide = params(**kw), dict(ldq=1 << 23, ldk=1 << 23, ldv=1 << 23)
    assert forward(lib, p, N=1, tokens=64, i=inputs(**wide)) == UNSUPPORTED
    assert lib.hyena_delta_workspace_bytes(ctypes.byref(p), 1, 64, None) == 0
    assert lib.hyena_delta_step(ctypes.byref(p), 1, 1, ctypes.byref(inputs(**wide)), P, 1, None, P, None) == UNSUPPORTED


def test_clearing_rows(lib):  # noqa: F811
    def clear(N=2, tokens=8, start=P, count=2, arrays=(P, P + 2), sizes=(16, 6)):
        n = len(arrays)
        return lib.hyena_delta_clear_rows(N, tokens, start, count, (ctypes.c_void_p * n)(*arrays), (ctypes.c_int64 * n)(*sizes), None)

    for kw in (dict(N=0), dict(tokens=-1), dict(start=None), dict(start=P + 4), dict(count=0), dict(count=9),
               dict(arrays=(None, P)), dict(arrays=(P + 1, P)), dict(sizes=(0, 6)), dict(sizes=(16, 7)), dict(sizes=(-2, 6))):
        assert clear(**kw) == INVALID, kw
    assert lib.hyena_delta_clear_rows(2, 8, P, 1, None, None, None) == INVALID
    assert clear(tokens=0) == 0
