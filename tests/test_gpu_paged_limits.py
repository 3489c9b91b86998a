"""The paged calls at their limits: full tables, device arrays that do not
ascend, repeated calls in place, pieces against whole chunks."""
import numpy as np
import pytest
import torch

import temporally_compressed_latent_b200 as mtla
from paged_harness import BASE, Batch

pytestmark = pytest.mark.gpu

TINY = dict(dtype="f32", H=4, d_h=16, r=64, d_R=8)


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
@pytest.mark.parametrize("n", [1, 2, 20])
def test_append_and_attention_refuse_the_same_sequences(n, dims):
    """Of three sequences one fills its table to the last row and one needs a row more: no call takes the latter."""
    s, pr = 2, 8
    new, past = [n, n, n], [9, 48 - n, 49 - n]
    for call in ("append", "attn"):
        b = Batch(new, past, s=s, page_rows=pr, seed=41, **dims)
        b.fill_groups()
        b.paged = mtla.paged_cache(b.d_pages, b.num_pages, pr, b.stride, b.d_table[:, :3].contiguous(), 3)
        o = getattr(b, call)()
        b.take = [n, n, 0]
        getattr(b, "check_" + call)(o)
        assert int(b.err.item()) == mtla.DEVERR_CAPACITY
