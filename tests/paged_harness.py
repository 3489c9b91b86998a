"""Test-side plumbing of the paged calls: inputs, a plain float64 implementation
written token by token from the formulas, and the error bounds that the storage
types allow.

Pages, row states and tables are filled with NaN (or nonsense) wherever a call
must not look, so a read out of place shows in the results."""
from __future__ import annotations

import math

import numpy as np
import torch

import temporally_compressed_latent_b200 as mtla

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # relative error of one rounding to nearest
U32 = 2.0 ** -24
BASE = 10000.0


def f64(t):
    return t.detach().double().cpu().numpy()


def rotate(x, pos):
    """Channel pairs of x [..., d_R] turned by pos base^(-2k/d_R)."""
    d = x.shape[-1]
    if d == 0:
        return x
    ang = pos * BASE ** (-2.0 * np.arange(d // 2) / d)
    out = np.empty_like(x)
    out[..., 0::2] = x[..., 0::2] * np.cos(ang) - x[..., 1::2] * np.sin(ang)
    out[..., 1::2] = x[..., 0::2] * np.sin(ang) + x[..., 1::2] * np.cos(ang)
    return out


class Batch:
    """A ragged chunk over a paged cache: device tensors and what they hold in float64."""

    def __init__(self, new, past, *, dtype="bf16", H=8, d_h=64, r=256, d_R=32, s=2, page_rows=16, pad=0, spare_tokens=0,
                 count=None, seed=0, J_extra=0, shuffle=True):
        self.new, self.past = list(new), list(past)
        self.take = [n if count is None else max(0, min(n, c)) for n, c in zip(new, count or new)]
        self.dtype, self.H, self.d_h, self.r, self.d_R, self.s, self.pr = dtype, H, d_h, r, d_R, s, page_rows
        self.D = r + d_R
        self.B, self.N = len(self.new), sum(self.new) + spare_tokens
        dt = TDT[dtype]
        g = torch.Generator().manual_seed(seed)
        rand = lambda *sh: torch.randn(*sh, generator=g)
        self.rows = [-(-(t + n) // s) for t, n in zip(self.past, self.new)]
        pages = [-(-x // page_rows) for x in self.rows]
        self.table_pages = max(max(pages), 1)
        total = sum(pages) + 2
        perm = (torch.randperm(total, generator=g) if shuffle else torch.arange(total)).tolist()
        # entries behind a sequence's pages name a page that is never valid
        self.table = torch.full((self.B, self.table_pages), -7, dtype=torch.int32)
        at = 0
        for b, k in enumerate(pages):
            for i in range(k):
                self.table[b, i] = perm[at]
                at += 1
        self.num_pages = total
        self.stride = self.D + pad
        self.pages = torch.full((total, page_rows, self.stride), float("nan"), dtype=dt)
        self.cache = []                       # float64 rows before the chunk
        for b in range(self.B):
            rows = rand(self.past[b] // s + 1, self.D).to(dt)
            # complete groups; the open group's row holds anything (its sum is in the tail)
            for j in range(self.past[b] // s):
                self.pages[self.where(b, j)][: self.D] = rows[j]
            self.cache.append(f64(rows))
        start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.start = start
        self.h = {
            "c": rand(self.N, r).to(dt), "kR": rand(self.N, d_R).to(dt), "q_rope": rand(self.N, H, d_R).to(dt),
            "q_abs": rand(self.N, H, r).to(dt), "W_c": rand(r, self.D) / math.sqrt(r), "b_c": rand(self.D) / math.sqrt(r),
            "P": 0.8 * rand(max(self.rows + [1]) + J_extra, self.D), "tail": rand(self.B, self.D),
            "state": rand(self.N, self.D).to(dt),
        }
        for b in range(self.B):               # a tail is only read where a group is open
            if self.past[b] % s == 0:
                self.h["tail"][b] = float("nan")
        for i in range(self.N):               # rows that no sequence takes
            if not any(start[b] <= i < start[b] + self.take[b] for b in range(self.B)):
                for k in ("c", "kR", "q_rope", "q_abs", "state"):
                    self.h[k][i] = float("nan")
        self.v = {k: f64(x) for k, x in self.h.items()}
        dev = lambda x: x.cuda()
        self.d = {k: dev(x) for k, x in self.h.items()}
        self.d_pages, self.d_table = dev(self.pages), dev(self.table)
        i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")
        self.t_prev, self.tok_start = i32(self.past), i32(start)
        self.tok_count = None if count is None else i32(count)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.md = mtla.dims(H, d_h, r, d_R, s, dtype)
        self.chunk = mtla.chunk(self.N, self.tok_start, self.t_prev, self.tok_count)
        self.paged = mtla.paged_cache(self.d_pages, total, page_rows, self.stride, self.d_table, self.table_pages)

    def where(self, b, j):
        return int(self.table[b, j // self.pr]), j % self.pr

    # ------------------------------------------------------------- append
    def append(self, rope_base=BASE, q=True, in_place=False, state=True, chunk=None):
        m = mtla.merge_args(self.d["c"], self.d["kR"], self.d["W_c"], self.d["b_c"], self.d["P"], self.d["P"].shape[0])
        nan = lambda *sh, dt=torch.float32: torch.full(sh, float("nan"), dtype=dt, device="cuda")
        o = {"state": nan(self.N, self.D, dt=TDT[self.dtype]) if state else None, "tail": nan(self.B, self.D),
             "t": torch.full((self.B,), -5, dtype=torch.int32, device="cuda"),
             "len": torch.full((self.B,), -5, dtype=torch.int32, device="cuda"),
             "q": None if not q else (self.d["q_rope"].clone() if in_place else nan(self.N, self.H, self.d_R, dt=TDT[self.dtype]))}
        size = mtla.mtla_paged_workspace_bytes(self.md, self.B, self.N, mtla.PAGED_APPEND)
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        mtla.mtla_paged_append(self.md, self.B, chunk or self.chunk, m, rope_base,
                               None if not q else (o["q"] if in_place else self.d["q_rope"]), o["q"], self.paged,
                               self.d["tail"], o["tail"], o["t"], o["len"], o["state"], ws, size, self.err)
        o["ws"] = ws
        return o

    def append_ref(self, rope_base=BASE, take=None):
        """Every token's S_t, the touched cache rows, the tails, the rotated queries; and how far fp32 arithmetic
        over bf16-split weights may leave S_t: a gate's pre-activation is a sum of r products of which each keeps
        a relative error of 2^-17 (W_c in two bf16 parts: 2^-9 of 2^-9, and half as much again for the sums in
        fp32, r + 4 roundings of 2^-24), its sigmoid has slope at most 1/4, and the sums take one rounding a token."""
        v, s = self.v, self.s
        S, slack, Q, rows, tails, tslack = {}, {}, {}, {}, {}, {}
        for b in range(self.B):
            run = v["tail"][b] if self.past[b] % s else np.zeros(self.D)
            gap = np.zeros(self.D)
            tails[b], tslack[b] = v["tail"][b], np.zeros(self.D)
            for i in range((take or self.take)[b]):
                tok, t = self.start[b] + i, self.past[b] + 1 + i
                j = -(-t // s)
                kR = rotate(v["kR"][tok], t - 1) if rope_base else v["kR"][tok]
                x = np.concatenate([v["c"][tok], kR])
                z = (v["c"][tok] @ v["W_c"] + v["b_c"]) * v["P"][j - 1]
                e = x / (1 + np.exp(-z))
                size = np.abs(v["c"][tok]) @ np.abs(v["W_c"]) + np.abs(v["b_c"])
                # (the rotated entries carry an angle error of 2^-23 turns and three roundings)
                turn = np.concatenate([np.zeros(self.r), np.full(self.d_R, 2.0 ** -20 * np.abs(v["kR"][tok]).max(initial=0))])
                g = np.abs(x) * np.abs(v["P"][j - 1]) / 4 * size * (2.0 ** -17 + (self.r + 4) * U32) + 2.0 ** -20 * np.abs(x) + turn
                opens = (t - 1) % s == 0
                run, gap = (e, g) if opens else (run + e, gap + g)
                gap = gap + U32 * np.abs(run)
                S[tok], slack[tok] = run, gap
                rows[b, j - 1] = (run, gap)
                tails[b], tslack[b] = run, gap
                Q[tok] = rotate(v["q_rope"][tok], t - 1) if rope_base else v["q_rope"][tok]
        return S, slack, rows, tails, tslack, Q

    def check_append(self, o, rope_base=BASE, take=None):
        take = take or self.take
        S, slack, rows, tails, tslack, Q = self.append_ref(rope_base, take)
        h = HALF[self.dtype]
        torch.cuda.synchronize()
        near = lambda got, ref, gap, what: np.testing.assert_array_less(
            np.abs(got - ref), gap + h * (np.abs(ref) + gap) + 1e-30, err_msg=what)
        assert o["t"].tolist() == [t + n for t, n in zip(self.past, take)]
        assert o["len"].tolist() == [-(-(t + n) // self.s) for t, n in zip(self.past, take)]
        state = f64(o["state"]) if o["state"] is not None else None
        q = f64(o["q"]) if o["q"] is not None else None
        for i in range(self.N):
            if state is not None:
                if i in S:
                    near(state[i], S[i], slack[i], f"state of token {i}")
                else:
                    assert np.isnan(state[i]).all(), f"row {i} belongs to no sequence"
            if q is not None:
                if i in Q:
                    near(q[i], Q[i], 2.0 ** -20 * np.abs(self.v["q_rope"][i]).max(initial=0), f"query of token {i}")
                else:
                    assert np.isnan(q[i]).all()
        tail = f64(o["tail"])
        for b in range(self.B):
            if take[b] == 0:
                np.testing.assert_array_equal(tail[b], self.v["tail"][b])
            else:
                gap = tslack[b] + U32 * np.abs(tails[b]) + 1e-30
                np.testing.assert_array_less(np.abs(tail[b] - tails[b]), gap)
        got = self.d_pages.cpu()
        touched = {}
        for (b, j), (ref, gap) in rows.items():
            pg, slot = self.where(b, j)
            near(f64(got[pg, slot, : self.D]), ref, gap, f"cache row {j} of sequence {b}")
            touched[pg, slot] = True
        want = self.pages.clone()
        for pg, slot in touched:
            want[pg, slot, : self.D] = got[pg, slot, : self.D]
        assert torch.equal(got.view(torch.int16 if self.dtype == "bf16" else torch.int32),
                           want.view(torch.int16 if self.dtype == "bf16" else torch.int32)), "other cache rows changed"

    # ---------------------------------------------------------- attention
    def attn(self, out_dtype=None, lse=True, chunk=None, ws=None):
        od = out_dtype or self.dtype
        out = torch.full((self.N, self.H, self.r), float("nan"), dtype=TDT[od], device="cuda")
        l = torch.full((self.N, self.H), float("nan"), device="cuda") if lse else None
        size = mtla.mtla_paged_workspace_bytes(self.md, self.B, self.N, mtla.PAGED_ATTN)
        if ws is None:
            ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        mtla.mtla_paged_attn(self.md, self.B, chunk or self.chunk, self.d["q_abs"], self.d["q_rope"], self.d["state"],
                             self.paged, out, {"f32": mtla.MTLA_F32, "bf16": mtla.MTLA_BF16}[od], l, ws, size, self.err)
        return {"out": out, "lse": l, "ws": ws}

    def fill_groups(self, seed=5):
        """The complete groups that the chunk itself closes (as the append would have left them); the open group's row too."""
        g = torch.Generator().manual_seed(seed)
        for b in range(self.B):
            rows = torch.randn(self.rows[b], self.D, generator=g).to(TDT[self.dtype])
            rows[: self.past[b] // self.s] = torch.from_numpy(self.cache[b][: self.past[b] // self.s]).to(TDT[self.dtype])
            for j in range((self.past[b] + self.take[b]) // self.s):
                self.pages[self.where(b, j)][: self.D] = rows[j]
            self.cache[b] = f64(rows)
        self.d_pages.copy_(self.pages)

    def attn_ref(self, b, i):
        """Output, lse and (error of a score, largest value) of token i of sequence b."""
        v, tok, t = self.v, self.start[b] + i, self.past[b] + 1 + i
        rows = np.concatenate([self.cache[b][: -(-t // self.s) - 1], v["state"][tok][None]])
        q = np.concatenate([v["q_abs"][tok], v["q_rope"][tok]], axis=1)
        scale = 1 / math.sqrt(self.d_h)
        x = q @ rows.T * scale
        m = x.max(axis=1, keepdims=True)
        p = np.exp(x - m)
        l = p.sum(axis=1, keepdims=True)
        # a score: D products summed in fp32, scaled to log2 units (two more roundings, one of the difference to
        # the maximum), and the exponential's own 2^-22
        gap = ((self.D + 4) * U32 * (np.abs(q) @ np.abs(rows).T * scale).max(axis=1) + 4 * U32 * np.abs(x).max(axis=1) + 2.0 ** -21)
        return p @ rows[:, : self.r] / l, (m + np.log(l))[:, 0], gap, np.abs(rows[:, : self.r]).max(), len(rows)

    def check_attn(self, o, out_dtype=None, tokens=None):
        """tokens: (sequence, place) pairs to compare (default: all)."""
        torch.cuda.synchronize()
        out, lse = f64(o["out"]), f64(o["lse"]) if o["lse"] is not None else None
        taken = {self.start[b] + i for b in range(self.B) for i in range(self.take[b])}
        for i in range(self.N):
            if i not in taken:
                assert np.isnan(out[i]).all() and (lse is None or np.isnan(lse[i]).all()), f"row {i} belongs to no sequence"
            else:
                assert np.isfinite(out[i]).all(), i
        for b, i in tokens or [(b, i) for b in range(self.B) for i in range(self.take[b])]:
            ref, ref_l, gap, big, L = self.attn_ref(b, i)
            tok = self.start[b] + i
            # a probability: its score's error and, for bf16, its rounding as a tensor-core operand; numerator and
            # denominator each, sums of L terms in fp32; then the output's rounding
            p_err = 2 * gap[:, None] + (HALF["bf16"] if self.dtype == "bf16" else 0.0) + (L + 16) * U32
            tol = p_err * big + HALF[out_dtype or self.dtype] * (np.abs(ref) + p_err * big)
            np.testing.assert_array_less(np.abs(out[tok] - ref), tol * 1.01 + 1e-30, err_msg=f"sequence {b} token {i}")
            if lse is not None:
                np.testing.assert_array_less(np.abs(lse[tok] - ref_l), gap + (L + 16) * U32 + 4 * U32 * np.abs(ref_l) + 1e-30,
                                             err_msg=f"lse, sequence {b} token {i}")


def verify_ref(p, q, tokens, start, ua, us):
    """Speculative sampling in float64, draft by draft."""
    clean = lambda a: np.where(np.isfinite(a) & (a > 0), a, 0.0).astype(np.float64)
    keep, nxt = [], []
    for b in range(len(start) - 1):
        n = start[b + 1] - start[b]
        if n == 0:
            keep.append(0)
            nxt.append(-1)
            continue
        k = 1
        while k < n:
            i = start[b] + k - 1
            x = tokens[i + 1]
            if not 0 <= x < p.shape[1]:
                break
            qx = clean(q[i])[x] if q is not None else 1.0
            if not float(ua[i]) * qx < clean(p[i])[x]:
                break
            k += 1
        i = start[b] + k - 1
        w = clean(p[i])
        if k < n:
            one = np.zeros_like(w)
            if q is None and 0 <= tokens[i + 1] < len(w):
                one[tokens[i + 1]] = np.inf
            rest = np.maximum(w - (clean(q[i]) if q is not None else one), 0.0)
            w = rest if rest.sum() > 0 else w
        keep.append(k)
        cdf = np.cumsum(w)
        nxt.append(-1 if cdf[-1] == 0 else int(np.argmax(cdf > float(us[b]) * cdf[-1])))
    return keep, nxt
