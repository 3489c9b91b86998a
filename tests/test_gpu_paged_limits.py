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


@pytest.mark.parametrize("dims,N", [({}, 64), (TINY, 64), (dict(TINY, s=12), 64), ({}, 600)], ids=["main", "tiny", "far", "many"])
def test_starts_that_do_not_ascend(dims, N):
    """Whatever tok_start holds, no call looks outside its arrays: a token that a search leads to the wrong sequence
    is nobody's, and times follow the windows."""
    rng = np.random.default_rng(N)
    B = 100
    for trial in range(6):
        b = Batch([1] * (B - 1) + [N - B + 1] if N > B else [1] * N + [0] * (B - N), [9] * B, page_rows=8,
                  seed=43, J_extra=N, **{"s": 2, **dims})
        b.fill_groups()
        start = rng.integers(-5, N + 6, B + 1) if trial else np.arange(B, -1, -1)
        b.tok_start.copy_(torch.from_numpy(start.astype(np.int32)))
        b.table[:] = 0                                   # rows for any window: page 0 again and again
        table = torch.zeros(B, 80, dtype=torch.int32, device="cuda")
        b.paged = mtla.paged_cache(b.d_pages, b.num_pages, b.pr, b.stride, table, 80)
        o = b.append()
        a = b.attn()
        first = np.clip(start[:-1], 0, N)
        n = np.clip(np.minimum(start[1:], N) - first, 0, None)
        torch.cuda.synchronize()
        assert o["t"].tolist() == (9 + n).tolist() and int(b.err.item()) == 0
        seen = np.zeros(N, bool)
        for f, k in zip(first, n):
            seen[f:f + k] = True
        assert torch.isnan(a["out"][torch.from_numpy(~seen).cuda()]).all()
        keep, nxt = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        p = torch.rand(N, 50, device="cuda")
        mtla.mtla_verify_drafts(B, N, 50, p, 50, None, 0, torch.zeros(N, dtype=torch.int32, device="cuda"), b.tok_start,
                                torch.zeros(N, device="cuda"), torch.full((B,), 0.5, device="cuda"), keep, nxt, b.err)
        torch.cuda.synchronize()
        assert ((keep.cpu().numpy() == 0) == (n == 0)).all() and int(b.err.item()) == 0


@pytest.mark.parametrize("dims,new", [({}, [7, 3]), (TINY, [7, 3]), ({}, [600, 3])], ids=["main", "tiny", "many"])
def test_taken_back_after_queries_in_place(dims, new):
    """The first call rotates the queries where they are; the repeated one takes none, and they stay rotated once."""
    b = Batch(new, [4, 9], s=2, page_rows=8, seed=44, **dims)
    first = b.append(in_place=True)
    torch.cuda.synchronize()
    once = first["q"].clone()
    keep = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    back = b.append(q=False, chunk=mtla.chunk(b.N, b.tok_start, b.t_prev, keep))
    torch.cuda.synchronize()
    assert torch.equal(first["q"], once)
    few = Batch(new, [4, 9], s=2, page_rows=8, seed=44, count=[2, 3], **dims)
    few.check_append(few.append())
    alone = few.append(q=False)
    torch.cuda.synchronize()
    assert torch.equal(back["tail"], alone["tail"]) and torch.equal(back["t"], alone["t"])
    Q = b.append_ref()[-1]
    q = first["q"].double().cpu().numpy()
    for i, ref in Q.items():
        gap = 2.0 ** -20 * np.abs(b.v["q_rope"][i]).max()
        half = 2.0 ** -8 if b.dtype == "bf16" else 2.0 ** -24
        np.testing.assert_array_less(np.abs(q[i] - ref), gap + half * (np.abs(ref) + gap) + 1e-30)


def test_host_tensors_are_refused():
    """Before anything is launched; pinned host memory is the device's too."""
    b = Batch([2, 1], [4, 9], s=2, page_rows=8, seed=45)
    for k in ("c", "q_rope", "tail"):
        keep, b.d[k] = b.d[k], b.d[k].cpu()
        with pytest.raises(ValueError, match="the host"):
            b.append()
        b.d[k] = keep
    for k in ("q_abs", "state"):
        keep, b.d[k] = b.d[k], b.d[k].cpu()
        with pytest.raises(ValueError, match="the host"):
            b.attn()
        b.d[k] = keep
    b.check_append(b.append())
    p = torch.rand(3, 50, device="cuda")
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pin = lambda n: torch.full((n,), -9, dtype=torch.int32).pin_memory()
    keep, nxt, err = pin(1), pin(1), torch.zeros(1, dtype=torch.int32).pin_memory()
    u = torch.zeros(3, device="cuda")
    mtla.mtla_verify_drafts(1, 3, 50, p, 50, p, 50, dev([0, 1, 77]), dev([0, 3]), u, u[:1], keep, nxt, err)
    torch.cuda.synchronize()
    assert keep.item() == 2 and 0 <= nxt.item() < 50 and err.item() == mtla.DEVERR_TOKEN


def _in_pieces(b, cuts):
    """The tokens of a one-sequence batch in pieces; tail, time and states as append() gives them."""
    m = mtla.merge_args(b.d["c"], b.d["kR"], b.d["W_c"], b.d["b_c"], b.d["P"], b.d["P"].shape[0])
    tail, t = b.d["tail"].clone(), b.t_prev.clone()
    state, q = torch.full_like(b.d["state"], float("nan")), torch.full_like(b.d["q_rope"], float("nan"))
    n = torch.zeros_like(t)
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        start = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        tail2, t2 = torch.empty_like(tail), torch.empty_like(t)
        mtla.mtla_paged_append(b.md, 1, mtla.chunk(b.N, start, t), m, BASE, b.d["q_rope"], q, b.paged, tail, tail2, t2, n,
                               state, None, 0, b.err)
        tail, t = tail2, t2
    torch.cuda.synchronize()
    return {"state": state, "tail": tail, "t": t, "len": n, "q": q}


@pytest.mark.parametrize("dims,N,s,past", [
    ({}, 40, 4, 6), ({}, 300, 2, 5), ({}, 1300, 2, 5), ({}, 900, 1, 0), ({}, 1000, 3, 1), ({}, 700, 9, 13), ({}, 1500, 64, 50),
    (TINY, 200, 3, 4), (dict(TINY, r=128), 150, 30, 11), (dict(H=5, r=384, d_R=64), 90, 5, 2),
])
def test_pieces_give_the_bits_of_the_whole(dims, N, s, past):
    """Within a kernel (chosen by the widths and the rows of the token arrays) a token's sums do not depend on the
    call it comes in: the same bits, but for the RoPE channels of the tensor-core kernel, whose angles are exact at
    every eighth column of a tile."""
    make = lambda: Batch([N], [past], s=s, page_rows=16, seed=46, **dims)
    whole = make()
    ow = whole.append()
    whole.check_append(ow)
    same = whole.r if not dims and N >= 512 else whole.D           # channels whose bits do not change
    # a rotated key is within 2^-20 of its size on either side, a group holds s of them, and each sum is rounded
    size = whole.d["kR"].float().abs().max().item() if whole.d_R else 0.0
    gap = s * (2 * 2.0 ** -20 * size + 2 * 2.0 ** -24 * s * size)
    half = 2.0 ** -8 if whole.dtype == "bf16" else 0.0             # stored rows: a rounding each

    def equal(x, y, stored, what):
        x, y = x.float(), y.float()
        assert torch.equal(x[..., :same], y[..., :same]), what
        far = (x[..., same:] - y[..., same:]).abs() - gap - (half if stored else 0.0) * (x[..., same:].abs() + y[..., same:].abs())
        assert same == whole.D or far.max().item() <= 0, what

    rng = np.random.default_rng(N + s)
    for trial in range(3):
        most = (5, 60, 400)[trial]
        cuts = [0]
        while cuts[-1] < N:
            cuts.append(min(N, cuts[-1] + int(rng.integers(1, most + 1))))
        b = make()
        o = _in_pieces(b, cuts)
        for k in ("t", "len", "q"):
            assert torch.equal(o[k], ow[k]), (k, trial)
        equal(o["state"], ow["state"], True, ("state", trial))
        equal(o["tail"], ow["tail"], False, ("tail", trial))
        for j in range(past // s, -(-(past + N) // s)):
            at = b.where(0, j)
            equal(b.d_pages[at][: b.D], whole.d_pages[at][: b.D], True, ("row", j, trial))


@pytest.mark.parametrize("s,past", [(2, 5), (7, 3), (64, 1)])
def test_pieces_across_the_kernels(s, past):
    """Token arrays of fewer than 512 rows take the kernel with the weights in fp32, longer ones that with two bf16
    parts: a sequence may pass from one to the other and keeps the bounds of the latter."""
    N = 1024
    whole = Batch([N], [past], s=s, page_rows=16, seed=47)
    b = Batch([N], [past], s=s, page_rows=16, seed=47)
    tail, t = b.d["tail"].clone(), b.t_prev.clone()
    state, q = torch.full_like(b.d["state"], float("nan")), torch.full_like(b.d["q_rope"], float("nan"))
    n = torch.zeros_like(t)
    for lo, hi in ((0, 130), (130, 700), (700, 701), (701, N)):
        k = hi - lo
        rows = lambda x: x[lo:hi].clone()
        m = mtla.merge_args(rows(b.d["c"]), rows(b.d["kR"]), b.d["W_c"], b.d["b_c"], b.d["P"], b.d["P"].shape[0])
        part, qp = torch.empty_like(state[lo:hi]), torch.empty_like(q[lo:hi])
        start = torch.tensor([0, k], dtype=torch.int32, device="cuda")
        tail2, t2 = torch.empty_like(tail), torch.empty_like(t)
        mtla.mtla_paged_append(b.md, 1, mtla.chunk(k, start, t), m, BASE, rows(b.d["q_rope"]), qp, b.paged, tail, tail2, t2,
                               n, part, None, 0, b.err)
        state[lo:hi], q[lo:hi] = part, qp
        tail, t = tail2, t2
    b.check_append({"state": state, "tail": tail, "t": t, "len": n, "q": q})
    whole.check_append(whole.append())
    assert int(b.err.item()) == 0


def test_calls_from_several_host_threads():
    """Every thread its own batch, stream and workspace; some of the calls are a kernel's first."""
    import threading
    kinds = [dict(new=[3, 1, 20], past=[100, 2000, 5]), dict(new=[520, 4], past=[3, 8]),
             dict(new=[5, 2], past=[30, 700], **TINY), dict(new=[9], past=[50], H=5, r=384, d_R=64)]
    jobs = []
    for k, kw in enumerate(kinds * 2):
        a = Batch(s=2, page_rows=16, seed=60 + k, **kw)
        b = Batch(s=2, page_rows=16, seed=60 + k, **kw)
        b.fill_groups()
        jobs.append((a, b))
    torch.cuda.synchronize()
    out, failed = {}, []
    gate = threading.Barrier(len(jobs))

    def work(k):
        try:
            a, b = jobs[k]
            st = torch.cuda.Stream()
            gate.wait(timeout=60)
            with torch.cuda.stream(st):
                for _ in range(8):
                    out[k] = a.append(), b.attn()
            st.synchronize()
        except Exception as e:  # noqa: BLE001 (handed to the test)
            failed.append((k, e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for k, (a, b) in enumerate(jobs):
        a.check_append(out[k][0])
        b.check_attn(out[k][1])
        assert int(a.err.item()) == 0 and int(b.err.item()) == 0
