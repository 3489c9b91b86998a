"""Chunks long enough that every block of the append takes several full tiles, and
replays of captured calls on new contents, each compared with the float64
implementation."""
import numpy as np
import pytest
import torch

import temporally_compressed_latent_b200 as mtla
from paged_harness import BASE, HALF, U32, Batch, verify_ref

pytestmark = pytest.mark.gpu

TINY = dict(dtype="f32", H=4, d_h=16, r=64, d_R=8)


class Dense:
    """A long ragged append: float64 by whole arrays (Batch's goes token by token)."""

    def __init__(self, new, past, s, *, dtype="bf16", H=8, d_h=64, r=256, d_R=32, page_rows=16, seed=0):
        self.new, self.past, self.s, self.r, self.d_R, self.D, self.dtype = new, past, s, r, d_R, r + d_R, dtype
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
        B, N = len(new), sum(new)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *sh: torch.randn(*sh, generator=g, device="cuda")
        rows = [-(-(t + n) // s) for t, n in zip(past, new)]
        pages = [-(-x // page_rows) for x in rows]
        total = sum(pages)
        table = torch.full((B, max(pages)), -1, dtype=torch.int32)
        perm, at = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32), 0
        for b, k in enumerate(pages):
            table[b, :k] = perm[at:at + k]
            at += k
        self.table, self.pr = table, page_rows
        i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.c, self.kR, self.q = rand(N, r).to(dt), rand(N, d_R).to(dt), rand(N, H, d_R).to(dt)
        self.W_c, self.b_c, self.P = rand(r, self.D) / r ** 0.5, rand(self.D) / r ** 0.5, 0.8 * rand(max(rows), self.D)
        self.tail, self.pages = rand(B, self.D), torch.full((total, page_rows, self.D), float("nan"), dtype=dt, device="cuda")
        md = mtla.dims(H, d_h, r, d_R, s, dtype)
        self.state, self.tail_out = torch.full_like(self.c[:, :1], float("nan")).repeat(1, self.D), torch.full_like(self.tail, float("nan"))
        self.q_out, self.t, self.n = torch.full_like(self.q, float("nan")), i32([-1] * B), i32([-1] * B)
        err = i32([0])
        mtla.mtla_paged_append(md, B, mtla.chunk(N, i32(self.start), i32(past)), mtla.merge_args(self.c, self.kR, self.W_c, self.b_c, self.P, max(rows)),
                               BASE, self.q, self.q_out, mtla.paged_cache(self.pages, total, page_rows, self.D, table.cuda(), max(pages)),
                               self.tail, self.tail_out, self.t, self.n, self.state, None, 0, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0

    def rotated(self, x, pos):
        f = BASE ** (-2.0 * torch.arange(self.d_R // 2, dtype=torch.float64, device="cuda") / self.d_R)
        a = pos.double()[:, None] * f
        co, si = torch.cos(a), torch.sin(a)
        if x.dim() == 3:
            co, si = co[:, None], si[:, None]
        x = x.double()
        return torch.stack([x[..., 0::2] * co - x[..., 1::2] * si, x[..., 0::2] * si + x[..., 1::2] * co], dim=-1).flatten(-2)

    def check(self):
        """Every state, tail, cache row and query, within the bounds of Batch.append_ref."""
        s, h = self.s, HALF[self.dtype]
        assert self.t.tolist() == [t + n for t, n in zip(self.past, self.new)]
        assert self.n.tolist() == [-(-(t + n) // s) for t, n in zip(self.past, self.new)]
        W, flat = self.W_c.double(), self.pages.view(-1, self.D)
        seen = torch.zeros(flat.shape[0], dtype=torch.bool, device="cuda")

        def near(got, ref, gap, half):
            far = (got.double() - ref).abs() - gap - half * (ref.abs() + gap) - 1e-30
            assert torch.isfinite(got).all() and far.max().item() < 0

        for b, (n, t0) in enumerate(zip(self.new, self.past)):
            at = slice(int(self.start[b]), int(self.start[b]) + n)
            pos = torch.arange(t0, t0 + n, device="cuda")
            P = self.P[pos // s].double()
            c, kR = self.c[at].double(), self.kR[at]
            x = torch.cat([c, self.rotated(kR, pos)], dim=1)
            e = x / (1 + torch.exp(-(c @ W + self.b_c.double()) * P))
            size = c.abs() @ W.abs() + self.b_c.double().abs()
            turn = torch.cat([torch.zeros(n, self.r, device="cuda"), (2.0 ** -20 * kR.float().abs().amax(1, keepdim=True)).expand(n, self.d_R)], 1)
            gap = x.abs() * P.abs() / 4 * size * (2.0 ** -17 + (self.r + 4) * U32) + 2.0 ** -20 * x.abs() + turn
            # sums from each group's start: rows of s slots, the first group's earlier part in its slot 0
            g0, off = t0 // s, t0 % s
            groups = -(-(off + n) // s)
            slots = lambda v: torch.cat([torch.zeros(off, self.D, dtype=torch.float64, device="cuda"), v,
                                         torch.zeros(groups * s - off - n, self.D, dtype=torch.float64, device="cuda")]).view(groups, s, self.D)
            E, G = slots(e), slots(gap)
            if off:
                E[0, 0] = self.tail[b].double()
            S = E.cumsum(1)
            G = (G + U32 * S.abs()).cumsum(1)
            S, G = S.reshape(-1, self.D)[off:off + n], G.reshape(-1, self.D)[off:off + n]
            near(self.state[at], S, G, h)
            near(self.tail_out[b], S[-1], G[-1], U32)
            ends = torch.clamp((torch.arange(g0, g0 + groups, device="cuda") + 1) * s, max=t0 + n) - 1 - t0
            j = torch.arange(g0, g0 + groups)
            where = (self.table[b, j // self.pr].long() * self.pr + j % self.pr).cuda()
            near(flat[where], S[ends], G[ends], h)
            seen[where] = True
            near(self.q_out[at], self.rotated(self.q[at], pos), 2.0 ** -20 * self.q[at].double().abs().amax((1, 2))[:, None, None], h)
        assert torch.isnan(flat[~seen].float()).all(), "other cache rows changed"


@pytest.mark.parametrize("s", [1, 2, 3, 9, 64])
def test_tensor_core_append_over_many_tiles(s):
    """Each of a channel tile's 49 CTAs takes four tiles of 128 columns or more (of which s - 1 repeat)."""
    rng = np.random.default_rng(s)
    N = 49 * 4 * (128 - (s - 1)) + 77
    cut = np.sort(rng.choice(np.arange(1, N), 9, replace=False))
    new = [int(x) for x in np.diff(np.concatenate([[0], cut, [N]]))] + [1, 2, s + 1]
    past = [int(x) for x in rng.integers(0, 3000, len(new))]
    Dense(new, past, s, seed=s).check()


@pytest.mark.parametrize("s,H", [(2, 5), (3, 16)])
def test_tensor_core_append_of_many_short_chunks(s, H):
    """Sequences of one to nine tokens over several tiles a CTA."""
    rng = np.random.default_rng(s + H)
    new = [int(x) for x in rng.integers(1, 10, 5200)]
    past = [int(x) for x in rng.integers(0, 60, len(new))]
    Dense(new, past, s, H=H, page_rows=8, seed=H).check()


@pytest.mark.parametrize("dims,N", [(TINY, 9001), (dict(dtype="bf16", H=5, d_h=64, r=384, d_R=64), 4100), (dict(TINY, r=508, d_R=68), 3000)],
                         ids=["tiny", "wide", "widest"])
@pytest.mark.parametrize("s", [1, 2, 9, 10, 40])
def test_generic_append_over_many_rounds(dims, N, s):
    """Tiles of several rounds: the rows before a tile in its first one (s <= 9), or sought."""
    new = [N - 700, 1, 333, 2, 364]
    past = [5, 0, s, 3 * s - 1, 1000]
    Dense(new, past, s, seed=N + s, **dims).check()


def _hold(b, c):
    """Puts the contents of batch c (no larger, as many tokens and sequences) where b's captured calls look."""
    b.t_prev.copy_(c.t_prev)
    b.tok_start.copy_(c.tok_start)
    b.d_table.fill_(-7)
    b.d_table[:, : c.table_pages].copy_(c.d_table)
    b.d_pages.fill_(float("nan"))
    b.d_pages[: c.num_pages].copy_(c.d_pages)
    for k, x in c.d.items():
        b.d[k][: x.shape[0]].copy_(x)
    b.err.zero_()


@pytest.mark.parametrize("dims", [{}, TINY], ids=["main", "tiny"])
def test_replays_follow_new_contents(dims):
    """Attention of two batches in two graphs that share a workspace, and their appends in graphs of their own: replayed
    after lengths, starts, tables, pages and inputs have changed, every result is that of the new contents."""
    N, kw = 24, dict(s=2, page_rows=16, **dims)
    large = [Batch([3, 1, 20], [1990, 2000, 1995], seed=70 + k, J_extra=8, **kw) for k in range(2)]
    size = mtla.mtla_paged_workspace_bytes(large[0].md, 3, N, mtla.PAGED_ATTN)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    for b in large:
        b.fill_groups()
        b.attn(ws=ws)
        b.append()
    torch.cuda.synchronize()
    graphs = {}
    with torch.cuda.stream(st):
        for k, b in enumerate(large):
            for call in ("attn", "append"):
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr, stream=st):
                    o = b.attn(ws=ws) if call == "attn" else b.append()
                graphs[call, k] = gr, o
    st.synchronize()
    shapes = [([10, 0, 14], [900, 31, 1500]), ([1, 22, 1], [2000, 3, 0]), ([8, 8, 8], [0, 1, 1001]), ([24, 0, 0], [77, 0, 9])]
    for i, (new, past) in enumerate(shapes):
        for call in ("attn", "append"):
            held = []
            for k, b in enumerate(large):
                # the second graph's contents are another shape's
                n, p = shapes[(i + k) % len(shapes)]
                c = Batch(n, p, seed=80 + 2 * i + k, **kw)
                if call == "attn":
                    c.fill_groups()
                _hold(b, c)
                held.append(c)
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                for k in (0, 1, 0, 1):
                    graphs[call, k][0].replay()
            st.synchronize()
            for k, (b, c) in enumerate(zip(large, held)):
                o = graphs[call, k][1]
                if call == "append":
                    c.d_pages.copy_(b.d_pages[: c.num_pages])
                    c.check_append(o)
                else:
                    c.check_attn(o)
                assert int(b.err.item()) == 0


def test_verification_replays_follow_new_contents():
    rng = np.random.default_rng(5)
    B, N, V = 4, 13, 9001
    dev = lambda v, t: torch.tensor(np.asarray(v), dtype=t, device="cuda")
    p, q = torch.zeros(N, V, device="cuda"), torch.zeros(N, V, device="cuda")
    tokens, start = dev([0] * N, torch.int32), dev([0, 3, 3, 12, 13], torch.int32)
    ua, us = torch.zeros(N, device="cuda"), torch.zeros(B, device="cuda")
    keep, nxt, err = (dev([-9] * n, torch.int32) for n in (B, B, 1))
    call = lambda: mtla.mtla_verify_drafts(B, N, V, p, V, q, V, tokens, start, ua, us, keep, nxt, err)
    call()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for lens in ([3, 0, 9, 1], [13, 0, 0, 0], [1, 1, 1, 1], [4, 4, 4, 1]):
        z = 2 * rng.standard_normal((N, V))
        soft = lambda a: (np.exp(a) / np.exp(a).sum(1, keepdims=True)).astype(np.float32)
        P, Q = soft(z), soft(z + 0.4 * rng.standard_normal((N, V)))
        tok = [int(rng.integers(0, V))] + [int(rng.choice(V, p=Q[i].astype(np.float64) / Q[i].astype(np.float64).sum())) for i in range(N - 1)]
        s, a, u = np.concatenate([[0], np.cumsum(lens)]), rng.random(N).astype(np.float32), rng.random(B).astype(np.float32)
        for dst, src in ((p, P), (q, Q), (tokens, tok), (start, s), (ua, a), (us, u), (err, [0])):
            dst.copy_(torch.from_numpy(np.asarray(src)))
        gr.replay()
        torch.cuda.synchronize()
        assert (keep.tolist(), nxt.tolist()) == verify_ref(P, Q, tok, s, a, u) and int(err.item()) == 0
