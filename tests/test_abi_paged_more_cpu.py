"""More of the paged calls without a GPU: overlapping arrays, tensors of another
device."""
import pytest

from test_abi_paged_cpu import INVALID, P, _append, _chunk, _dims


def test_append_refuses_queries_that_overlap_in_part():
    size = 4 * 8 * 32 * 2                                   # four tokens, eight heads of 32 bf16 channels
    for off in (16, size - 16):
        assert _append(q=P, qo=P + off) == INVALID
        assert _append(q=P + off, qo=P) == INVALID
    none = dict(B=0)                                        # no sequences: the arguments are sound and nothing runs
    assert _append(q=P, qo=P + size, **none) == 0 and _append(q=P + size, qo=P, **none) == 0
    assert _append(q=P, qo=P, **none) == 0
    assert _append(q=P, qo=P + 16, chunk=_chunk(N=0), **none) == 0
    f32 = _dims(dtype="f32")
    assert _append(d=f32, q=P, qo=P + 2 * size - 16) == INVALID
    assert _append(d=f32, q=P, qo=P + 2 * size, **none) == 0
