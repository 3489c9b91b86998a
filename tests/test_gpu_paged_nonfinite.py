"""NaN and infinities in what mtla_paged_attn reads: they reach every query that
sees them, and no other, whether an item's columns are one block's or several
blocks' work.

A query that sees a NaN, or scores +inf somewhere, has no softmax: its head's
outputs are NaN.  A column that scores -inf has probability zero; 0 x inf makes
the output NaN in the channels in which that column is infinite, and only there."""
import math

import numpy as np
import pytest
import torch

from paged_harness import HALF, U32, Batch, f64

pytestmark = pytest.mark.gpu

TINY = dict(dtype="f32", H=4, d_h=16, r=64, d_R=8)
WIDE = dict(dtype="bf16", H=5, d_h=64, r=384, d_R=64)
NAN, INF = float("nan"), float("inf")


def put_state(b, seq, place, channel, value):
    tok = int(b.start[seq]) + place
    b.d["state"][tok, channel] = value
    b.v["state"][tok, channel] = value


def put_row(b, seq, row, channel, value):
    pg, slot = b.where(seq, row)
    b.d_pages[pg, slot, channel] = value
    b.cache[seq][row, channel] = value


def reference(b, seq, i):
    """Output [H, r], lse [H] and the error bound of a finite output, from the columns that the query sees."""
    v, tok, t = b.v, b.start[seq] + i, b.past[seq] + 1 + i
    rows = np.concatenate([b.cache[seq][: -(-t // b.s) - 1], v["state"][tok][None]])
    q = np.concatenate([v["q_abs"][tok], v["q_rope"][tok]], axis=1)
    scale = 1 / math.sqrt(b.d_h)
    out, lse, tol, ltol = np.full((b.H, b.r), NAN), np.full(b.H, NAN), np.zeros((b.H, 1)), np.zeros(b.H)
    bad = ~np.isfinite(rows[:, : b.r]).all(axis=0)                # channels in which a visible column is not finite
    with np.errstate(invalid="ignore"):
        x = (q[:, None, :] * rows[None]).sum(axis=2) * scale
    for h in range(b.H):
        if np.isnan(x[h]).any() or (x[h] == INF).any():
            continue
        use = x[h] > -INF
        if not use.any():                                         # nothing but -inf: 0 / 0, and ln 0
            lse[h] = -INF
            continue
        y, k = x[h][use], rows[use]
        p = np.exp(y - y.max())
        out[h], lse[h] = p @ k[:, : b.r] / p.sum(), y.max() + np.log(p.sum())
        out[h][bad] = NAN
        # as in Batch.check_attn: a score's D products in fp32, its scaling, the exponential; a probability's rounding
        # as an operand; sums of L terms
        gap = (b.D + 4) * U32 * (np.abs(q[h]) @ np.abs(k).T * scale).max() + 4 * U32 * np.abs(y).max() + 2.0 ** -21
        tol[h] = (2 * gap + (HALF["bf16"] if b.dtype == "bf16" else 0.0) + (len(k) + 16) * U32) * np.abs(k[:, : b.r]).max()
        ltol[h] = gap + (len(k) + 16) * U32 + 4 * U32 * np.abs(lse[h]) + 1e-30
    return out, lse, tol, ltol


def check(b, o, where=None):
    """Every query's output and lse, NaN for NaN (where: (sequence, place) pairs, default all)."""
    torch.cuda.synchronize()
    out, lse = f64(o["out"]), f64(o["lse"])
    od = "f32" if o["out"].dtype == torch.float32 else "bf16"
    clean = 0
    for seq, i in where or [(s, i) for s in range(b.B) for i in range(b.take[s])]:
        ref, ref_l, tol, ltol = reference(b, seq, i)
        tok = b.start[seq] + i
        what = f"sequence {seq} token {i}"
        np.testing.assert_array_equal(np.isnan(out[tok]), np.isnan(ref), err_msg=what)
        np.testing.assert_array_equal(np.isnan(lse[tok]), np.isnan(ref_l), err_msg=what)
        fine = ~np.isnan(ref)
        assert np.isfinite(out[tok][fine]).all(), what
        near = (np.abs(out[tok] - ref) <= (tol + HALF[od] * (np.abs(ref) + tol)) * 1.01 + 1e-30) | ~fine
        assert near.all(), what
        with np.errstate(invalid="ignore"):
            assert ((np.abs(lse[tok] - ref_l) <= ltol) | np.isnan(ref_l) | (lse[tok] == ref_l)).all(), what
        clean += bool(fine.all())
    return clean


def blind(b, bad):
    """Tokens that see none of the columns in `bad`: ("state", seq, place) or ("row", seq, row)."""
    def sees(seq, i):
        rows = -(-(b.past[seq] + 1 + i) // b.s) - 1
        return any(s == seq and (k == i if kind == "state" else k < rows) for kind, s, k in bad)
    return [(s, i) for s in range(b.B) for i in range(b.take[s]) if not sees(s, i)]


SHORT = [5, 1, 8, 3], [11, 4, 17, 0]                  # one key tile an item: no item is split
LONG = [5, 40, 1, 16], [3000, 900, 2500, 1501]        # many key tiles an item, split over blocks


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("dims", [{}, dict(H=16), TINY, WIDE], ids=["main", "h16", "tiny", "wide"])
@pytest.mark.parametrize("new,past", [SHORT, LONG], ids=["short", "long"])
def test_later_values_do_not_reach_earlier_tokens(new, past, dims, value):
    """A later token's own state, and a group that a later token closes, latent or RoPE channel."""
    b = Batch(new, past, s=2, page_rows=8, seed=51, **dims)
    b.fill_groups()
    bad = []
    for seq, (n, t0) in enumerate(zip(new, past)):
        if n < 3:
            continue
        put_state(b, seq, n - 1, 3, value)
        put_state(b, seq, n // 2, b.r + 1 if seq % 2 else b.r - 1, value)
        closed = (t0 + n) // 2 - 1                      # the last group that the chunk closes
        put_row(b, seq, closed, 0 if seq % 2 else b.r // 2, value)
        bad += [("state", seq, n - 1), ("state", seq, n // 2), ("row", seq, closed)]
    for od in ("f32", b.dtype):
        o = b.attn(out_dtype=od)
        rest = blind(b, bad)
        assert check(b, o, rest) == len(rest) >= sum(new) - 3 * len(bad)
        if new is SHORT[0]:
            check(b, o)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("dims", [{}, dict(H=16), TINY, WIDE], ids=["main", "h16", "tiny", "wide"])
@pytest.mark.parametrize("new,past", [([1] * 32, [4096] * 32), ([1] * 32, [21] * 32), LONG], ids=["split", "whole", "long"])
def test_seen_values_reach_the_output(new, past, dims, value):
    """A token's own state (in a cut item it can be a part's only visible column), an old cache row, a query; with a
    query that is zero where the state is not finite."""
    b = Batch(new, past, s=2, page_rows=8, seed=52, **dims)
    b.fill_groups()
    for seq, n in enumerate(new):
        if seq % 4 < 3 or n > 1:
            put_state(b, seq, n - 1, 5, value)
        if seq % 4 == 1:
            put_row(b, seq, past[seq] // 4, b.r - 1, value)
        if seq % 4 == 2:
            tok = int(b.start[seq]) + n - 1
            b.d["q_abs"][tok, 0, 5] = 0.0
            b.v["q_abs"][tok, 0, 5] = 0.0
        if seq % 4 == 3:
            tok = int(b.start[seq]) + n // 2
            b.d["q_abs"][tok, :, 2] = value
            b.v["q_abs"][tok, :, 2] = value
    for od in ("f32", b.dtype):
        check(b, b.attn(out_dtype=od))
    assert int(b.err.item()) == 0
