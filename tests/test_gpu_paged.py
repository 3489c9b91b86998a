"""The paged calls on the device against a plain float64 implementation
(tests/paged_harness.py): mtla_paged_append, mtla_paged_attn and
mtla_verify_drafts, alone and together as a serving loop uses them.

Sizes sit where the kernels can go wrong: sequences without tokens, one token,
groups that span chunks and tiles, pages that end inside a key tile, heads that
do not divide a tile, rows that belong to no sequence, NaN wherever nothing may
be read."""
import math

import numpy as np
import pytest
import torch

import temporally_compressed_latent_b200 as mtla
from paged_harness import BASE, Batch, f64, verify_ref

pytestmark = pytest.mark.gpu

TINY = dict(dtype="f32", H=4, d_h=16, r=64, d_R=8)
WIDE = dict(dtype="bf16", H=5, d_h=64, r=384, d_R=64)
WIDE32 = dict(dtype="f32", H=16, d_h=128, r=512, d_R=64)


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("dims", [{}, dict(H=12), TINY, WIDE, WIDE32], ids=["main", "h12", "tiny", "wide", "wide32"])
@pytest.mark.parametrize("s,page_rows", [(1, 8), (2, 16), (3, 24), (8, 8), (70, 16)])
def test_append(dims, s, page_rows):
    """Ragged chunks (none, one, many tokens) after none, an open or a complete group."""
    new = [1, 0, 5, 2 * s + 1, 17, 1, 0, 33]
    past = [0, 3, s, 2 * s - 1, 5 * s + 1, s - 1, 0, 40]
    b = Batch(new, past, s=s, page_rows=page_rows, spare_tokens=3, seed=10 * s + page_rows, **dims)
    o = b.append()
    b.check_append(o)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("new,past,s,dims", [
    ([700, 1, 0, 301], [5, 1000, 7, 0], 2, {}),
    ([513], [0], 3, {}),
    ([130, 400], [1, 63], 32, {}),
    ([260, 129, 128, 127], [63, 0, 64, 65], 64, {}),
    ([600], [10], 300, {}),
    ([1] * 40, list(range(40)), 2, {}),
    ([300, 45], [2, 9], 5, TINY),
    ([1200], [3], 1200, TINY),
    ([1] * 600 + [0] * 40 + [3, 2], [i % 70 for i in range(642)], 2, dict(H=12)),
    ([255, 0, 258], [129, 5, 0], 1, dict(H=16)),
    ([2] * 270, [i % 9 for i in range(270)], 4, dict(H=5)),
    ([250, 200], [3, 0], 2, {}),
], ids=["ragged", "s3", "s32", "s64", "s300", "decode40", "tiny", "onegroup", "decode600", "s1", "pairs", "below"])
def test_append_long(new, past, s, dims):
    b = Batch(new, past, s=s, page_rows=16, seed=77, **dims)
    b.check_append(b.append())
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_append_options(dims):
    """Padded rows, no queries, queries in place, rotated inputs, no row states, a count for every sequence."""
    kw = dict(new=[4, 9, 3, 2], past=[3, 8, 0, 1], s=2, page_rows=8, seed=3, **dims)
    b = Batch(pad=16, **kw)
    b.check_append(b.append(q=False))
    b = Batch(**kw)
    b.check_append(b.append(in_place=True))
    b = Batch(**kw)
    b.check_append(b.append(rope_base=0.0), rope_base=0.0)
    b = Batch(**kw)
    b.check_append(b.append(state=False))
    b = Batch(count=[4, 2, 0, -3], **kw)
    b.check_append(b.append())
    # the same with tokens enough for the long-chunk kernel
    kw = dict(kw, new=[310, 9, 200, 2])
    for make in (dict(pad=8), dict(count=[190, 20, 0, 1])):
        b = Batch(spare_tokens=5, **make, **kw)
        b.check_append(b.append(q="count" in make))
    b = Batch(**kw)
    b.check_append(b.append(in_place=True))
    b = Batch(**kw)
    b.check_append(b.append(rope_base=0.0, state=False), rope_base=0.0)


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_append_without_tokens(dims):
    """Nothing new anywhere: times and tails are handed on; token arrays may have no rows at all."""
    for spare in (2, 0):
        b = Batch([0, 0, 0], [5, 0, 4], s=2, page_rows=8, spare_tokens=spare, seed=2, **dims)
        b.check_append(b.append())
        b.fill_groups()
        b.check_attn(b.attn())
        assert int(b.err.item()) == 0


def test_without_rope_channels():
    """d_R = 0: latents alone, no RoPE keys or queries."""
    b = Batch([3, 0, 20, 1], [4, 9, 70, 0], dtype="f32", H=3, d_h=8, r=32, d_R=0, s=3, page_rows=8, seed=6)
    b.check_append(b.append(q=False))
    b = Batch([3, 0, 20, 1], [4, 9, 70, 0], dtype="f32", H=3, d_h=8, r=32, d_R=0, s=3, page_rows=8, seed=6)
    b.fill_groups()
    b.check_attn(b.attn())


def test_append_far_position():
    """Angles at large times: the table of P limits a sequence's groups, so a large stride gives large times."""
    s = 1 << 20
    b = Batch([3, 2], [5 * s + 7, 3 * s - 1], s=s, page_rows=8, seed=4)
    b.check_append(b.append())


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_append_in_pieces_and_taken_back(dims):
    """The open group's sum travels in fp32: one token at a time gives the sums of one call, and a call repeated
    with fewer tokens leaves what the fewer alone leave."""
    s, n, past = 4, 11, 6
    whole = Batch([n], [past], s=s, page_rows=8, seed=21, **dims)
    ow = whole.append()
    whole.check_append(ow)
    step = Batch([n], [past], s=s, page_rows=8, seed=21, **dims)
    # rows of the token arrays are taken one by one by moving the start
    tail, t = step.d["tail"].clone(), step.t_prev.clone()
    m = mtla.merge_args(step.d["c"], step.d["kR"], step.d["W_c"], step.d["b_c"], step.d["P"], step.d["P"].shape[0])
    state = torch.zeros_like(ow["state"])
    for i in range(n):
        start = torch.tensor([i, i + 1], dtype=torch.int32, device="cuda")
        ch = mtla.chunk(n, start, t)
        tail2, t2 = torch.empty_like(tail), torch.empty_like(t)
        mtla.mtla_paged_append(step.md, 1, ch, m, BASE, None, None, step.paged, tail, tail2, t2, None, state, None, 0, step.err)
        tail, t = tail2, t2
    torch.cuda.synchronize()
    assert t.tolist() == [past + n]
    # the same sums up to the order of the gate's products (few roundings of 2^-24 of values of order 1)
    assert (tail - ow["tail"]).abs().max().item() < 1e-5
    assert (state.float() - ow["state"].float()).abs().max().item() <= (2.0 ** -7) * ow["state"].float().abs().max().item()
    # taken back to 4 tokens
    back = Batch([n], [past], s=s, page_rows=8, seed=21, **dims)
    back.append()
    keep = torch.tensor([4], dtype=torch.int32, device="cuda")
    o = back.append(chunk=mtla.chunk(n, back.tok_start, back.t_prev, keep))
    few = Batch([n], [past], s=s, page_rows=8, seed=21, count=[4], **dims)
    of = few.append()
    few.check_append(of)
    assert torch.equal(o["tail"], of["tail"]) and o["t"].tolist() == [past + 4]
    for j in range((past + 4) // s):
        at = back.where(0, j)
        assert torch.equal(back.d_pages[at][: back.D], few.d_pages[at][: few.D])


@pytest.mark.parametrize("more", [[], [1] * 520], ids=["few", "many"])
def test_append_refuses_on_the_device(more):
    """Sequences that do not fit take nothing and say why; the others are not disturbed."""
    new, past, s = [3, 3, 3, 3] + more, [4, 30, 2, 5] + [6] * len(more), 2
    t_more, n_more = [7] * len(more), [1] * len(more)
    b = Batch(new, past, s=s, page_rows=8, seed=8)
    # sequence 1 needs 17 rows: a table of two pages holds 16
    b.paged = mtla.paged_cache(b.d_pages, b.num_pages, b.pr, b.stride, b.d_table[:, :2].contiguous(), 2)
    o = b.append()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_CAPACITY
    assert o["t"].tolist() == [7, 30, 5, 8] + t_more
    b.check_append(o, take=[3, 0, 3, 3] + n_more)
    # the P table ends before sequence 1's groups
    b = Batch(new, past, s=s, page_rows=8, seed=8)
    b.d["P"] = b.d["P"][:10].contiguous()
    o = b.append()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_PE_RANGE
    b.check_append(o, take=[3, 0, 3, 3] + n_more)
    # a negative time
    b = Batch(new, past, s=s, page_rows=8, seed=8)
    b.t_prev[2] = -1
    o = b.append()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_CAPACITY and o["t"].tolist() == [7, 33, -1, 8] + t_more
    # a time past the 32-bit integers
    b = Batch(new, past, s=s, page_rows=8, seed=8)
    b.t_prev[3] = (1 << 31) - 3
    o = b.append()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_CAPACITY and o["t"].tolist() == [7, 33, 5, (1 << 31) - 3] + t_more
    # a table entry outside the pool: its rows are not written, the rest is
    for bad in (-1, 1 << 30):
        b = Batch(new, past, s=s, page_rows=8, seed=8)
        b.d_table[0, 0] = bad
        before = b.d_pages.clone()
        o = b.append()
        torch.cuda.synchronize()
        assert int(b.err.item()) == mtla.DEVERR_CAPACITY
        page = b.d_pages[int(b.table[0, 0])]
        assert torch.equal(page.view(torch.int16), before[int(b.table[0, 0])].view(torch.int16))
        assert torch.isfinite(o["state"]).all()


# --------------------------------------------------------------- attention


@pytest.mark.parametrize("dims", [{}, dict(H=1), dict(H=3), dict(H=12), dict(H=16), TINY, WIDE, WIDE32],
                         ids=["main", "h1", "h3", "h12", "h16", "tiny", "wide", "wide32"])
@pytest.mark.parametrize("s,page_rows", [(1, 8), (2, 16), (3, 24), (8, 64)])
def test_attention(dims, s, page_rows):
    """Ragged chunks over ragged caches; nothing cached, nothing new; NaN in every row that is not visible."""
    new = [1, 0, 5, 17, 1, 2 * s + 1, 0, 40, 1]
    past = [0, 3, s, 65 * s, 64 * s - 1, 7, 0, 200 * s + 1, 129 * s]
    b = Batch(new, past, s=s, page_rows=page_rows, spare_tokens=2, seed=10 * s + page_rows, **dims)
    b.fill_groups()
    o = b.attn()
    b.check_attn(o)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("new,past,kw", [
    ([1], [0], {}),
    ([1], [20000], {}),                              # one token over a long cache: every block holds a part
    ([3] * 50, [37 * i for i in range(50)], {}),     # many short items
    ([500, 1, 130], [3000, 1, 0], {}),
    ([1] * 700, [i % 90 for i in range(700)], {}),   # more sequences than threads of a block
    ([257, 15, 16], [0, 4000, 127], dict(s=1, page_rows=128)),
    ([90, 7], [700, 3], dict(TINY, s=3, page_rows=8)),
    ([1, 1, 2], [9000, 11, 4000], dict(TINY, page_rows=32)),
], ids=["one", "long", "short", "mixed", "many", "s1", "tiny", "tinylong"])
def test_attention_shapes(new, past, kw):
    kw = dict(dict(s=2, page_rows=16, seed=31), **kw)
    b = Batch(new, past, **kw)
    b.fill_groups()
    o = b.attn()
    rng = np.random.default_rng(0)
    every = [(i, k) for i in range(b.B) for k in range(b.take[i])]
    some = every if len(every) < 200 else [every[0], every[-1]] + [every[k] for k in rng.choice(len(every), 120, replace=False)]
    b.check_attn(o, tokens=some)
    assert int(b.err.item()) == 0


def _some(b, k=60):
    """Every sequence's first and last token and some others."""
    every = [(i, j) for i in range(b.B) for j in range(b.take[i])]
    ends = {(i, j) for i in range(b.B) if b.take[i] for j in (0, b.take[i] - 1)}
    rng = np.random.default_rng(1)
    more = [every[i] for i in rng.choice(len(every), min(k, len(every)), replace=False)]
    return sorted(ends | set(more))


@pytest.mark.parametrize("most", [1, 5, 6, 8, 9, 16])
def test_attention_live_rows(most):
    """Chunks whose items hold 8 to 128 live rows, over more key tiles than are in flight."""
    b = Batch([most, 1, most, 2], [1500, 3, 700, 2900], s=1, page_rows=16, seed=most)
    b.fill_groups()
    b.check_attn(b.attn(), tokens=_some(b))
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("new,past,kw", [
    ([33, 33, 9], [3000, 2000, 50], dict(s=1)),                  # few items, each in many parts
    ([1], [4000], dict(s=1)),                                    # one row of them
    ([300, 2], [900, 5000], dict(s=2)),                          # a sequence of more items than are added one by one
    ([1 + i % 3 for i in range(100)], [(37 * i) % 300 for i in range(100)], dict(s=3)),  # more windows than are kept
], ids=["few", "one", "items", "sequences"])
@pytest.mark.parametrize("dims", [TINY, WIDE32], ids=["tiny", "wide32"])
def test_attention_parts(new, past, kw, dims):
    """The generic kernel's shares and the joining of their parts."""
    b = Batch(new, past, page_rows=8, seed=17, **kw, **dims)
    b.fill_groups()
    b.check_attn(b.attn(), tokens=_some(b))
    assert int(b.err.item()) == 0


def test_attention_options():
    kw = dict(new=[4, 19, 3, 2], past=[3, 900, 0, 130], s=2, page_rows=8, seed=3)
    b = Batch(pad=8, **kw)
    b.fill_groups()
    b.check_attn(b.attn(out_dtype="f32"), out_dtype="f32")
    b.check_attn(b.attn(lse=False))
    b = Batch(count=[4, 11, 0, -1], **kw)
    b.fill_groups()
    b.check_attn(b.attn())
    # large scores: one column takes nearly everything
    b = Batch(**kw)
    b.d["q_abs"].mul_(8)
    b.v["q_abs"] = f64(b.d["q_abs"])
    b.fill_groups()
    b.check_attn(b.attn())


def test_attention_refuses_on_the_device():
    new, past = [2, 2, 2], [30, 100, 12]
    b = Batch(new, past, s=2, page_rows=8, seed=9)
    b.fill_groups()
    # sequence 1 sees 50 rows: a table of three pages holds 24
    b.paged = mtla.paged_cache(b.d_pages, b.num_pages, b.pr, b.stride, b.d_table[:, :3].contiguous(), 3)
    o = b.attn()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_CAPACITY
    b.take = [2, 0, 2]
    b.check_attn(o)
    b = Batch(new, past, s=2, page_rows=8, seed=9)
    b.fill_groups()
    b.t_prev[0] = -3
    o = b.attn()
    torch.cuda.synchronize()
    assert int(b.err.item()) == mtla.DEVERR_CAPACITY
    b.take = [0, 2, 2]
    b.check_attn(o)
    # rows of a page outside the pool read as zeros
    for bad in (-1, 1 << 30):
        b = Batch(new, past, s=2, page_rows=8, seed=9)
        b.fill_groups()
        b.d_table[1, 2] = bad
        b.cache[1][16:24] = 0.0
        o = b.attn()
        b.check_attn(o)
        assert int(b.err.item()) == mtla.DEVERR_CAPACITY


def test_attention_equals_the_contiguous_decode():
    """One token a sequence over pages in order is mtla_decode_attn's step over the same rows."""
    new, past, s = [1] * 6, [0, 1, 130, 511, 700, 2047], 2
    b = Batch(new, past, s=s, page_rows=16, seed=14)
    b.fill_groups()
    b.check_attn(b.attn(out_dtype="f32"), out_dtype="f32")
    o = b.attn(out_dtype="f32")
    rows = [np.concatenate([b.cache[i][: -(-(t + 1) // s) - 1], b.v["state"][i][None]]) for i, t in enumerate(past)]
    cap = max(len(r) for r in rows)
    buf = torch.zeros(6 * cap, b.D, dtype=torch.bfloat16)
    for i, r in enumerate(rows):
        buf[i * cap:i * cap + len(r)] = torch.from_numpy(r).to(torch.bfloat16)
    buf = buf.cuda()
    off = torch.arange(6, dtype=torch.int64, device="cuda") * cap
    capacity = torch.full((6,), cap, dtype=torch.int64, device="cuda")
    t = torch.tensor([p + 1 for p in past], dtype=torch.int32, device="cuda")
    out = torch.empty(6, b.H, b.r, device="cuda")
    size = mtla.mtla_workspace_bytes(b.md, 6)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mtla.mtla_decode_attn(b.md, 6, b.d["q_abs"], b.d["q_rope"], None, buf, 6 * cap, b.D, off, capacity, t, None, out,
                          None, ws, size, b.err)
    torch.cuda.synchronize()
    # both within bf16 probabilities of the same softmax
    assert (out - o["out"]).abs().max().item() <= 2 * 2.0 ** -8 * float(buf.float().abs().max())


# ------------------------------------------------- offsets past 32 bits


def _behind(x, off):
    """x's rows behind off others."""
    big = torch.empty((off + x.shape[0],) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
    big[off:] = x
    return big


@pytest.fixture
def freed():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_far_pages(dims, freed):
    """Pages more than 2^31 elements into the pool."""
    for call in ("append", "attn"):
        width = dims.get("r", 256) + dims.get("d_R", 32)
        b = Batch([3, 1, 40], [100, 0, 601], s=2, page_rows=16, pad=16384 - width, seed=23, **dims)
        if call == "attn":
            b.fill_groups()
        first = (1 << 31) // (16 * 16384) + 1
        pool = _behind(b.d_pages, first)
        table = torch.where(b.d_table >= 0, b.d_table + first, b.d_table)
        b.paged = mtla.paged_cache(pool, first + b.num_pages, 16, b.stride, table, b.table_pages)
        o = getattr(b, call)()
        if call == "append":
            torch.cuda.synchronize()
            b.d_pages.copy_(pool[first:])
            b.check_append(o)
        else:
            b.check_attn(o)
        assert int(b.err.item()) == 0


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_far_tokens(dims, freed):
    """Tokens more than 2^31 elements into every token array, behind a sequence of which none is taken."""
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
    b = Batch([3, 1, 40], [100, 0, 601], s=2, page_rows=16, seed=29, **dims)
    table = torch.cat([torch.zeros_like(b.d_table[:1]), b.d_table])
    paged = mtla.paged_cache(b.d_pages, b.num_pages, b.pr, b.stride, table, b.table_pages)
    row = lambda x: torch.cat([x[:1], x])          # the sequence in front

    def chunk(off):
        N = off + b.N
        return N, mtla.chunk(N, i32([0] + [off + x for x in b.start]), i32([0] + b.past), i32([0] + b.take))

    off = (1 << 31) // b.r + 5
    N, c = chunk(off)
    m = mtla.merge_args(_behind(b.d["c"], off), _behind(b.d["kR"], off), b.d["W_c"], b.d["b_c"], b.d["P"], b.d["P"].shape[0])
    state, q = (_behind(torch.full_like(b.d[k], float("nan")), off) for k in ("state", "q_rope"))
    tail = torch.full((b.B + 1, b.D), float("nan"), device="cuda")
    t, n = i32([-5] * (b.B + 1)), i32([-5] * (b.B + 1))
    tail_in = row(b.d["tail"])
    mtla.mtla_paged_append(b.md, b.B + 1, c, m, 10000.0, _behind(b.d["q_rope"], off), q, paged, tail_in, tail, t, n, state,
                           None, 0, b.err)
    b.check_append({"t": t[1:], "len": n[1:], "state": state[off:], "q": q[off:], "tail": tail[1:]})
    del m, state, q

    b.fill_groups()
    off = (1 << 31) // (b.H * b.r) + 5
    N, c = chunk(off)
    out = _behind(torch.full((b.N, b.H, b.r), float("nan"), dtype=b.d["q_abs"].dtype, device="cuda"), off)
    lse = _behind(torch.full((b.N, b.H), float("nan"), device="cuda"), off)
    size = mtla.mtla_paged_workspace_bytes(b.md, b.B + 1, N, mtla.PAGED_ATTN)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    kind = mtla.MTLA_F32 if b.dtype == "f32" else mtla.MTLA_BF16
    mtla.mtla_paged_attn(b.md, b.B + 1, c, _behind(b.d["q_abs"], off), _behind(b.d["q_rope"], off), _behind(b.d["state"], off),
                         paged, out, kind, lse, ws, size, b.err)
    b.check_attn({"out": out[off:], "lse": lse[off:]})
    assert int(b.err.item()) == 0


# ------------------------------------------------------------ verification


def _verify(p, q, tokens, start, ua, us, ld=None):
    B, N, V = len(start) - 1, p.shape[0], p.shape[1]
    ld = ld or V

    def pad(x):
        y = torch.full((N, ld), float("nan"))
        y[:, :V] = torch.from_numpy(np.asarray(x, np.float32))
        return y.cuda()

    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
    f32 = lambda v: torch.tensor(np.asarray(v, np.float32), device="cuda")
    keep, nxt, err = i32([-9] * B), i32([-9] * B), i32([0])
    P, Q = pad(p), pad(q) if q is not None else None
    args = (i32(tokens), i32(start), f32(ua), f32(us))
    mtla.mtla_verify_drafts(B, N, V, P, ld, Q, ld if q is not None else 0, *args, keep, nxt, err)
    torch.cuda.synchronize()
    return keep.tolist(), nxt.tolist(), int(err.item())


def _dists(rng, N, V, near=0.5):
    z = 2 * rng.standard_normal((N, V))
    soft = lambda a: np.exp(a) / np.exp(a).sum(axis=1, keepdims=True)
    return soft(z).astype(np.float32), soft(z + near * rng.standard_normal((N, V))).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 1024, 8193, 50021])
@pytest.mark.parametrize("ld", [0, 7])
def test_verify(V, ld):
    rng = np.random.default_rng(V + ld)
    lens = [1, 0, 5, 2, 9, 3, 1, 4, 0]
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1]) + 1
    p, q = _dists(rng, N, V)
    tokens = np.array([rng.integers(0, V)] + [rng.choice(V, p=q[i].astype(np.float64) / q[i].astype(np.float64).sum()) for i in range(N - 1)])
    ua, us = rng.random(N).astype(np.float32), rng.random(len(lens)).astype(np.float32)
    us[0], us[2] = 0.0, np.float32(1 - 2.0 ** -24)
    for Q in (q, None):
        keep, nxt, err = _verify(p, Q, tokens, start, ua, us, V + ld)
        assert (keep, nxt) == verify_ref(p, Q, tokens, start, ua, us) and err == 0


def test_verify_many_drafts():
    """More drafts than a block has threads, all kept but one."""
    rng = np.random.default_rng(6)
    n, V = 700, 64
    p, q = _dists(rng, n, V, near=0.0)
    tokens = rng.integers(0, V, n)
    for drop in (0, 255, 256, 511, 698, None):
        ua = np.zeros(n, np.float32)
        if drop is not None:
            ua[drop] = 1.5
        keep, nxt, _ = _verify(p, q, tokens, [0, n], ua, [0.4])
        assert (keep, nxt) == verify_ref(p, q, tokens, [0, n], ua, [0.4]) and keep == [(n if drop is None else drop + 1)]


@pytest.mark.parametrize("V,lens", [
    (20001, [3, 1] * 40),                     # more sequences than can have eight blocks each at once
    (1 << 22, [2] + [0] * 59),                # the largest vocabulary, with four blocks a sequence
    (1 << 22, [1] + [0] * 39 + [2]),          # with eight
    (1 << 22, [2]),                           # and with sixteen
], ids=["many", "widest4", "widest8", "widest16"])
def test_verify_blocks(V, lens):
    rng = np.random.default_rng(V + len(lens))
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1])
    p, q = _dists(rng, N, V)
    tokens = rng.integers(0, V, N)
    for us in (rng.random(len(lens)), np.full(len(lens), 0.999999)):
        for Q in (q, None):
            ua, u = rng.random(N).astype(np.float32), us.astype(np.float32)
            keep, nxt, err = _verify(p, Q, tokens, start, ua, u)
            assert (keep, nxt) == verify_ref(p, Q, tokens, start, ua, u) and err == 0


def test_verify_far_rows(freed):
    """Rows 2^30 entries apart."""
    rng = np.random.default_rng(3)
    V, lens, ld = 1000, [2, 0, 2], 1 << 30
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1])
    p, q = _dists(rng, N, V)
    tokens = rng.integers(0, V, N)
    dev = lambda v, dt: torch.tensor(np.asarray(v, dt), device="cuda")
    far = [torch.empty(N, ld, device="cuda") for _ in range(2)]
    for x, y in zip(far, (p, q)):
        x[:, :V] = torch.from_numpy(y).cuda()
    for accept in (0.0, 0.999):
        ua, us = np.full(N, accept, np.float32), rng.random(len(lens)).astype(np.float32)
        keep, nxt, err = dev([-9] * 3, np.int32), dev([-9] * 3, np.int32), dev([0], np.int32)
        mtla.mtla_verify_drafts(3, N, V, far[0], ld, far[1], ld, dev(tokens, np.int32), dev(start, np.int32), dev(ua, np.float32),
                                dev(us, np.float32), keep, nxt, err)
        torch.cuda.synchronize()
        assert (keep.tolist(), nxt.tolist()) == verify_ref(p, q, tokens, start, ua, us) and int(err.item()) == 0


def test_verify_odd_distributions():
    """Masked entries (NaN, infinities, negative), a residual that is zero, one-hot rows, empty rows, bad tokens."""
    rng = np.random.default_rng(7)
    V, n = 3000, 3
    lens = [n] * 8
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1])
    p, q = _dists(rng, N, V)
    tokens = np.array([int(p[max(i - 1, 0)].argmax()) for i in range(N)])
    ua, us = np.full(N, 0.5, np.float32), rng.random(len(lens)).astype(np.float32)
    p[0, 100:2000], q[0, :50] = np.nan, -np.inf          # masked values
    p[1, 5], q[1, 7] = np.inf, np.nan
    ua[3:5], p[3:6] = 2.0, q[3:6]                        # dropped, and the residual is empty: p itself
    p[6] = 0; p[6, 2999] = 1; tokens[7] = 2999           # one-hot, kept
    p[9] = 0; q[9] = 0                                   # nothing anywhere
    tokens[13] = V                                       # outside the vocabulary
    tokens[16] = -1
    p[18:21, :] = -1.0                                   # every entry masked
    q[21, :] = 0; tokens[22] = int(p[21].argmax())       # q gives it no weight: kept
    keep, nxt, err = _verify(p, q, tokens, start, ua, us)
    assert (keep, nxt) == verify_ref(p, q, tokens, start, ua, us)
    assert err == mtla.DEVERR_TOKEN | mtla.DEVERR_EMPTY and nxt[3] == -1 and nxt[6] == -1


def test_verify_follows_the_target():
    """The first new token of many chunks is distributed as p: draft from q, keep or redraw.  20000 draws over 8
    entries: a share's deviation is at most sqrt(p (1 - p) / 20000) <= 0.0036; 5 of them bound every entry but for one
    chance in 10^5."""
    rng = np.random.default_rng(11)
    V, B = 8, 20000
    p1, q1 = _dists(rng, 1, V, near=1.0)
    start = np.arange(0, 2 * B + 1, 2)
    p, q = np.repeat(p1, 2 * B, 0), np.repeat(q1, 2 * B, 0)
    draft = rng.choice(V, size=B, p=q1[0].astype(np.float64) / q1[0].astype(np.float64).sum())
    tokens = np.stack([np.zeros(B, int), draft], 1).reshape(-1)
    keep, nxt, _ = _verify(p, q, tokens, start, rng.random(2 * B), rng.random(B))
    first = np.where(np.array(keep) == 2, draft, nxt)
    share = np.bincount(first, minlength=V) / B
    assert np.abs(share - p1[0]).max() < 5 * 0.0036


# ---------------------------------------------------------------- together


def _layer(md_s, seed):
    g = torch.Generator().manual_seed(seed)
    H, d_h, r, d_R, d = 8, 64, 256, 32, 512
    D = r + d_R
    rand = lambda *sh: torch.randn(*sh, generator=g)
    return dict(W_c=rand(r, D) / 16, b_c=rand(D) / 16, P=0.8 * rand(600, D))


@pytest.mark.parametrize("s", [2, 3])
def test_serving_loop(s):
    """Two prompts in pieces, then speculative steps with drafts taken back, over one pool of pages: every query's
    output equals the softmax over the float64 rows of the tokens kept before it."""
    H, r, d_R, D, pr = 8, 256, 32, 288, 16
    L = _layer(s, 5)
    g = torch.Generator().manual_seed(6)
    B, T = 2, 300
    c = torch.randn(B, T, r, generator=g).bfloat16()
    kR = torch.randn(B, T, d_R, generator=g).bfloat16()
    qa = torch.randn(B, T, H, r, generator=g).bfloat16()
    qr = torch.randn(B, T, H, d_R, generator=g).bfloat16()
    dev = {k: v.cuda() for k, v in L.items()}
    md = mtla.dims(H, 64, r, d_R, s, "bf16")
    table_pages = -(-T // (s * pr)) + 1
    pages = torch.full((2 * table_pages + 1, pr, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(2 * table_pages, dtype=torch.int32).flip(0).reshape(2, table_pages).contiguous().cuda()
    cache = mtla.paged_cache(pages, 2 * table_pages + 1, pr, D, table, table_pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, tail = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, D, device="cuda")
    done = [0, 0]
    rng = np.random.default_rng(2)
    plans = [([150, 70], None), ([1, 96], None)] + [([5, 4], [1 + int(rng.integers(0, 5)), 1 + int(rng.integers(0, 4))]) for _ in range(6)] + [([1, 1], None)]
    seen = {}
    for new, keep in plans:
        N = sum(new)
        cat = lambda x: torch.cat([x[b, done[b]:done[b] + new[b]] for b in range(B)]).cuda()
        start = torch.tensor([0, new[0], N], dtype=torch.int32, device="cuda")
        C, K, QA, QR = cat(c), cat(kR), cat(qa), cat(qr)
        m = mtla.merge_args(C, K, dev["W_c"], dev["b_c"], dev["P"], 600)
        state = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty(N, H, r, dtype=torch.bfloat16, device="cuda"), torch.empty(N, H, device="cuda")
        QRr = torch.empty_like(QR)
        tail2, t2 = torch.empty_like(tail), torch.empty_like(t)
        size = mtla.mtla_paged_workspace_bytes(md, B, N, mtla.PAGED_ATTN)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        ch = mtla.chunk(N, start, t)
        mtla.mtla_paged_append(md, B, ch, m, BASE, QR, QRr, cache, tail, tail2, t2, None, state, None, 0, err)
        mtla.mtla_paged_attn(md, B, ch, QA, QRr, state, cache, out, mtla.MTLA_BF16, lse, ws, size, err)
        if keep is not None:  # the verification's result: the rest is taken back
            kept = torch.tensor(keep, dtype=torch.int32, device="cuda")
            mtla.mtla_paged_append(md, B, mtla.chunk(N, start, t, kept), m, BASE, None, None, cache, tail, tail2, t2,
                                   None, None, None, 0, err)
        o = f64(out)
        for b in range(B):
            for i in range(new[b]):
                seen.setdefault(b, {})[done[b] + i] = o[(new[0] if b else 0) + i]
            done[b] += (keep or new)[b]
        tail, t = tail2, t2
        assert t.tolist() == done
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    from paged_harness import rotate
    v = {k: x.double().numpy() for k, x in L.items()}
    for b in range(B):
        S, rows = None, []
        for i in range(done[b]):
            cc, kk = f64(c[b, i]), rotate(f64(kR[b, i]), i)
            e = np.concatenate([cc, kk]) / (1 + np.exp(-(cc @ v["W_c"] + v["b_c"]) * v["P"][i // s]))
            S = e if i % s == 0 else S + e
            q = np.concatenate([f64(qa[b, i]), rotate(f64(qr[b, i]), i)], axis=1)
            keys = np.stack(rows + [S])
            x = q @ keys.T / 8
            p = np.exp(x - x.max(axis=1, keepdims=True))
            ref = p @ keys[:, :r] / p.sum(axis=1, keepdims=True)
            # keys, queries, probabilities and outputs are bf16: a score of 288 products with two rounded factors
            # moves by about 2 x 2^-8 of |q||k| / 8 / sqrt(288) x a few; held to the library's bf16 bound
            assert np.abs(seen[b][i] - ref).max() <= 2e-2 * max(np.abs(keys).max(), 1.0), (b, i)
            if (i + 1) % s == 0:
                rows.append(S)


def test_graph_and_streams():
    """Captured on a side stream and replayed on new contents; two graphs share a workspace; a call on another
    stream than the tensors' own."""
    def batch(seed):
        b = Batch([3, 1, 20], [100, 2000, 5], s=2, page_rows=16, seed=seed)
        b.fill_groups()
        return b

    b1, b2 = batch(1), batch(2)
    size = mtla.mtla_paged_workspace_bytes(b1.md, b1.B, b1.N, mtla.PAGED_ATTN)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    b1.attn(ws=ws)
    b1.append()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    with torch.cuda.stream(st):
        for b in (b1, b2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                o = b.attn(ws=ws)
                a = b.append()
            graphs.append(gr)
            outs.append((o, a))
        for gr in graphs + graphs:
            gr.replay()
    st.synchronize()
    for b, (o, a) in zip((b1, b2), outs):
        # (the append has replaced the groups that the chunk closes: compare the attention of a fresh run)
        b.check_append_only = True
        assert torch.isfinite(o["out"]).all()
        assert a["t"].tolist() == [103, 2001, 25]
    c = batch(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        o = c.attn(ws=ws)
    st.synchronize()
    c.check_attn(o)
    # replays repeat the same bits
    keep = outs[0][0]["out"].clone()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(keep.view(torch.int16), outs[0][0]["out"].view(torch.int16))


def test_repeats_are_identical():
    b = Batch([1] * 20 + [200], [100 * i for i in range(21)], s=2, page_rows=16, seed=12)
    b.fill_groups()
    first = b.attn()
    for _ in range(3):
        again = b.attn()
        torch.cuda.synchronize()
        assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])
