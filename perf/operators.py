"""The operators that serve a ragged chunk of new tokens over a paged MTLA cache:

* ``append``: the chunk's tokens merged into the paged compressed cache, with the RoPE rotation of their
  keys and queries on the way (``mtla_paged_append``);
* ``attn``: the chunk's queries attending the cache through the block table (``mtla_paged_attn``);
* ``verify``: drafted tokens checked against the target's probabilities (``mtla_verify_drafts``).

A case names its shape by plain numbers: B sequences, n new tokens each (with ``ragged`` between one and n,
drawn from ``layout``), ``ctx`` earlier tokens each (with ``ragged`` between half of it and all of it), and
the layer's H, d_h, r, d_R and s.  ``run`` computes an operator in elementary torch operations, or, with
``own``, makes the call into the library.
"""
import math
import random

import torch

own = False

BF16_DIMS = {"dtype": "bf16", "H": 8, "d_h": 64, "r": 256, "d_R": 32}  # the layer of the decode and prefill workloads
F32_DIMS = {"dtype": "f32", "H": 4, "d_h": 16, "r": 64, "d_R": 8}      # the tiny fp32 layer of the end-to-end tests
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0


def listed():
    a = lambda name, dims, **k: {"name": name, "op": "append", "layout": 1, "ragged": False, "page_rows": 64, **dims, **k}
    t = lambda name, dims, **k: {"name": name, "op": "attn", "layout": 1, "ragged": False, "page_rows": 64, **dims, **k}
    v = lambda name, **k: {"name": name, "op": "verify", "layout": 1, "ragged": False, **k}
    return [
        # one token of one sequence: the interactive decode step, where latency is all
        a("append one token", BF16_DIMS, B=1, n=1, ctx=1001, s=2),
        # a decode step of a batch of 32 (the decode workload's batch and lengths)
        a("append batch of 32", BF16_DIMS, B=32, n=1, ctx=4095, s=2),
        # prompt chunks of a busy server, ragged, after earlier context
        a("append prompt chunks", BF16_DIMS, B=8, n=4096, ctx=8192, s=2, ragged=True, page_rows=16),
        # four drafts a sequence in the tiny fp32 layer, stride 3
        a("append fp32 drafts", F32_DIMS, B=24, n=5, ctx=700, s=3, ragged=True, page_rows=8),
        # the interactive decode step over a short conversation
        t("attention one token", BF16_DIMS, B=1, n=1, ctx=301, s=2),
        # the decode workload: 32 sequences of 4096 tokens, one new token each
        t("attention batch of 32", BF16_DIMS, B=32, n=1, ctx=4096, s=2),
        # speculative decode of a large ragged batch: up to five tokens a sequence, lengths 4096 to 8192
        t("attention ragged drafts", BF16_DIMS, B=128, n=5, ctx=8192, s=2, ragged=True, page_rows=16),
        # chunked prefill over long contexts
        t("attention long chunks", BF16_DIMS, B=4, n=1024, ctx=16384, s=2, page_rows=128),
        # chunks in the tiny fp32 layer
        t("attention fp32 chunks", F32_DIMS, B=8, n=33, ctx=1500, s=3, ragged=True, page_rows=16),
        # four drafts of one sequence, a small vocabulary
        v("verify one sequence", B=1, n=5, V=32000),
        # a batch of 32 with ragged drafts over a vocabulary that is no multiple of anything
        v("verify ragged batch", B=32, n=8, V=50021, ragged=True),
        # a large batch and a large vocabulary
        v("verify large batch", B=96, n=4, V=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attn", "attn", "attn", "verify"])
    layout, ragged = rng.randrange(1 << 20), rng.random() < 0.6
    if op == "verify":
        B, V, n = _log(rng, 1, 96), _log(rng, 1000, 131072), rng.randint(1, 9)
        return {"op": op, "layout": layout, "ragged": ragged, "B": B, "n": max(1, min(n, 96 * 4 * 131072 // (B * V))), "V": V}
    f32 = rng.random() < 0.2
    dims = dict(F32_DIMS if f32 else BF16_DIMS)
    if not f32:
        dims["H"] = rng.choice([4, 8, 8, 8, 12, 16])
    s = rng.choice([1, 2, 2, 2, 3, 4, 8])
    B = _log(rng, 1, 32 if f32 else 256)
    n = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 64 if f32 else 2048)])
    ctx = rng.choice([rng.randint(0, 64), _log(rng, 65, 1500 if f32 else 16384)])
    if op == "append":
        n = max(1, min(n, (128 if f32 else 16384) // B))
        ctx = min(ctx, s * (120 if f32 else 32768) // B + 1)
    else:
        # cache rows of all sequences, and visible (query, head, row) triples, below those of the largest listed case
        ctx = min(ctx, s * (12000 if f32 else 600000) // B)
        most = 8 * 33 * 4 * 500 if f32 else 4 * 1024 * 8 * 8192
        n = max(1, min(n, most // (B * dims["H"] * ((ctx + n) // s + 1)), (33 * 8 if f32 else 4096) // B))
    return {"op": op, "layout": layout, "ragged": ragged, "page_rows": rng.choice([8, 16, 16, 32, 64, 128]), **dims, "B": B, "n": n, "ctx": ctx, "s": s}


def _lengths(case):
    """New tokens and earlier tokens of every sequence."""
    rng, B, n, ctx = random.Random(case["layout"]), case["B"], case["n"], case.get("ctx", 0)
    if not case["ragged"]:
        return [n] * B, [ctx] * B
    new = [rng.randint(1, n) for _ in range(B)]
    new[rng.randrange(B)] = n
    return new, [rng.randint(ctx // 2, ctx) for _ in range(B)]


def _up(a, b):
    return -(-a // b)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + case["layout"])
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    new, past = _lengths(case)
    B, N = case["B"], sum(new)
    start = [0]
    for x in new:
        start.append(start[-1] + x)
    st = {"case": case, "B": B, "N": N, "n_max": max(new), "tok_start": i32(start), "dev_err": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["op"] == "verify":
        # target and draft distributions that mostly agree, drafts drawn from the draft's by Gumbel noise
        V = case["V"]
        logits = 2.0 * rand(N, V)
        st["p"] = torch.softmax(logits, dim=1)
        st["q"] = torch.softmax(logits + 0.5 * rand(N, V), dim=1)
        gumbel = -torch.log(-torch.log(torch.rand(N, V, generator=g, device=dev).clamp_(1e-20, 1 - 1e-7)))
        drawn = (torch.log(st["q"]) + gumbel).argmax(dim=1).to(torch.int32)  # token that row i's draft proposes next
        st["tokens"] = torch.cat([drawn[-1:], drawn[:-1]])                   # ... is token i + 1 of the chunk
        st["u_accept"] = torch.rand(N, generator=g, device=dev)
        st["u_sample"] = torch.rand(B, generator=g, device=dev)
        st["n_keep"], st["next_token"] = torch.zeros(B, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
        return st
    dt, s, H, r, d_R, pr = TYPES[case["dtype"]], case["s"], case["H"], case["r"], case["d_R"], case["page_rows"]
    D = r + d_R
    rows = [_up(t + x, s) for t, x in zip(past, new)]
    n_pages = [_up(x, pr) for x in rows]
    total, table_pages = sum(n_pages) + 3, max(n_pages)
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    # sequence b's pages in table order, scattered over the pool; unused entries name page 0
    at = torch.arange(table_pages, device=dev)[None, :]
    first = torch.tensor([sum(n_pages[:b]) for b in range(B)], device=dev)[:, None]
    used = at < torch.tensor(n_pages, device=dev)[:, None]
    st["block_table"] = torch.where(used, perm[(first + at).clamp(max=total - 1)], torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
    st["t_prev"] = i32(past)
    st["pages"] = rand(total, pr, D).to(dt)
    st["table_pages"], st["rows_max"] = table_pages, max(rows)
    if case["op"] == "append":
        J = max(rows)
        st["c"], st["kR"] = rand(N, r).to(dt), rand(N, d_R).to(dt)
        st["q_rope"] = rand(N, H, d_R).to(dt)
        st["W_c"], st["b_c"] = rand(r, D) / math.sqrt(r), rand(D) / math.sqrt(r)
        st["P"], st["J_max"] = 0.8 * rand(J, D), J
        st["tail_in"] = 0.5 * rand(B, D)
        st["tail_out"], st["row_state"] = torch.zeros(B, D, device=dev), torch.zeros(N, D, dtype=dt, device=dev)
        st["q_rope_out"] = torch.zeros_like(st["q_rope"])
        st["t_out"], st["cache_len"] = torch.zeros(B, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
    else:
        st["q_abs"], st["q_rope"] = rand(N, H, r).to(dt), rand(N, H, d_R).to(dt)
        st["row_state"] = rand(N, D).to(dt)
        st["out"], st["lse"] = torch.zeros(N, H, r, dtype=dt, device=dev), torch.zeros(N, H, device=dev)
    return st


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


# ----------------------------------------------------------------- plain forms


def _tokens(st):
    """Every token's sequence, place in its chunk and position (1-based)."""
    start = st["tok_start"].long()
    i = torch.arange(st["N"], device=start.device)
    seq = torch.searchsorted(start[1:].contiguous(), i, right=True)
    place = i - start[seq]
    return seq, place, st["t_prev"].long()[seq] + 1 + place


def _rotate(x, t):
    """x [N, ..., d_R]: channel pairs rotated by (t - 1) base^(-2k / d_R); the angles in 64 bits."""
    d = x.shape[-1]
    freq = ROPE_BASE ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    angle = (t - 1).double()[:, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    a, b = x.float()[..., 0::2], x.float()[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)


def _plain_append(st):
    case, dt = st["case"], st["c"].dtype
    s, pr = case["s"], case["page_rows"]
    seq, place, t = _tokens(st)
    j = (t + s - 1) // s                                             # 1-based group
    z = (st["c"].float() @ st["W_c"] + st["b_c"]) * st["P"][j - 1]
    e = torch.sigmoid(z) * torch.cat([st["c"].float(), _rotate(st["kR"], t)], dim=1)
    # running sums inside groups: differences of one long sum, in 64 bits; the chunk's first group goes on from the tail
    total = torch.cumsum(e.double(), dim=0)
    i = torch.arange(st["N"], device=t.device)
    t_prev, count = st["t_prev"].long(), st["tok_start"].long().diff()
    in_group = torch.minimum((t - 1) % s, place)                     # tokens of the chunk before it in its group
    before = torch.where((i - in_group > 0)[:, None], total[(i - in_group - 1).clamp(min=0)], torch.zeros((), dtype=torch.float64, device=t.device))
    goes_on = ((t - 1) % s > place)[:, None]
    state = total - before + torch.where(goes_on, st["tail_in"][seq].double(), torch.zeros((), dtype=torch.float64, device=t.device))
    state = state.float()
    # every token of a group writes the group's last state of this chunk
    last = torch.minimum(i + (j * s - t), i + count[seq] - 1 - place)
    page = st["block_table"].long()[seq, (j - 1) // pr]
    st["pages"].view(-1, st["pages"].shape[-1])[page * pr + (j - 1) % pr] = state[last].to(dt)
    ends = (st["tok_start"].long()[1:] - 1).clamp(min=0)
    tail = torch.where((count > 0)[:, None], state[ends], st["tail_in"])
    t_out = t_prev + count
    return {"pages": st["pages"], "row_state": state.to(dt), "tail": tail, "t": t_out.int(), "cache_len": ((t_out + s - 1) // s).int(),
            "q_rope": _rotate(st["q_rope"], t).to(dt)}


def _plain_attn(st):
    case, dt = st["case"], st["q_abs"].dtype
    s, pr, r, H, B, n, L = case["s"], case["page_rows"], case["r"], case["H"], st["B"], st["n_max"], st["rows_max"]
    dev = st["q_abs"].device
    seq, place, t = _tokens(st)
    # every sequence padded to n queries and L rows
    tok = (st["tok_start"].long()[:-1, None] + torch.arange(n, device=dev)).clamp(max=st["N"] - 1)
    q = torch.cat([st["q_abs"], st["q_rope"]], dim=2).float()[tok]                  # [B, n, H, D]
    self_row = st["row_state"].float()[tok]                                         # [B, n, D]
    row = torch.arange(L, device=dev)
    page = st["block_table"].long()[:, row // pr]
    keys = st["pages"].view(-1, st["pages"].shape[-1])[page * pr + row % pr].float()  # [B, L, D]
    scale = 1.0 / math.sqrt(case["d_h"])
    seen = (st["t_prev"].long()[:, None] + 1 + torch.arange(n, device=dev) + s - 1) // s - 1  # complete groups before each query's own
    hidden = row[None, None, :] >= seen[:, :, None]                                 # [B, n, L]
    x = (q.reshape(B, n * H, -1) @ keys.transpose(1, 2)).reshape(B, n, H, L) * scale
    x = x.masked_fill(hidden[:, :, None, :], -math.inf)
    x_self = (q * self_row[:, :, None, :]).sum(-1) * scale                          # [B, n, H]
    top = torch.maximum(x.amax(dim=-1) if L else x_self, x_self)
    p, p_self = torch.exp(x - top[..., None]), torch.exp(x_self - top)
    total = p.sum(-1) + p_self
    o = (p.reshape(B, n * H, L) @ keys[:, :, :r]).reshape(B, n, H, r) + p_self[..., None] * self_row[:, :, None, :r]
    out, lse = o / total[..., None], top + torch.log(total)
    return {"out": out[seq, place].to(dt), "lse": lse[seq, place]}


def _plain_verify(st):
    B, n, p, q = st["B"], st["n_max"], st["p"], st["q"]
    start = st["tok_start"].long()
    count = start.diff()
    at = torch.arange(n, device=p.device)
    row = (start[:-1, None] + at).clamp(max=st["N"] - 1)
    nxt = (row + 1).clamp(max=st["N"] - 1)
    x = st["tokens"].long()[nxt]                                                    # the draft that row i judges
    ok = (st["u_accept"][row].double() * q[row, x].double() < p[row, x].double()) & (at[None, :] < count[:, None] - 1)
    keep = 1 + ok.long().cumprod(dim=1).sum(dim=1)
    last = start[:-1] + keep - 1
    target = p[last].double()
    residual = torch.where((keep < count)[:, None], (target - q[last].double()).clamp(min=0), target)
    weight = torch.where((residual.sum(dim=1) > 0)[:, None], residual, target)
    cdf = weight.cumsum(dim=1)
    token = torch.searchsorted(cdf, st["u_sample"].double()[:, None] * cdf[:, -1:], right=True)[:, 0]
    return {"n_keep": keep.int(), "next_token": token.int()}


_plain = {"append": _plain_append, "attn": _plain_attn, "verify": _plain_verify}


# ----------------------------------------------------------------- the library's calls


def _plan(st):
    """What a serving loop keeps between calls: dims, the argument structs and the workspace."""
    import temporally_compressed_latent_b200 as mtla
    case = st["case"]
    d = mtla.dims(case["H"], case["d_h"], case["r"], case["d_R"], case["s"], case["dtype"])
    chunk = mtla.chunk(st["N"], st["tok_start"], st["t_prev"])
    cache = mtla.paged_cache(st["pages"], st["pages"].shape[0], case["page_rows"], st["pages"].shape[2], st["block_table"], st["table_pages"])
    merge = None
    if case["op"] == "append":
        merge = mtla.merge_args(st["c"], st["kR"], st["W_c"], st["b_c"], st["P"], st["J_max"])
    size = mtla.mtla_paged_workspace_bytes(d, st["B"], st["N"], mtla.PAGED_APPEND if merge is not None else mtla.PAGED_ATTN)
    return d, chunk, cache, merge, torch.empty(max(size, 16), dtype=torch.uint8, device=st["pages"].device), size


def _own_append(st):
    import temporally_compressed_latent_b200 as mtla
    if "plan" not in st:
        st["plan"] = _plan(st)
    d, chunk, cache, merge, ws, size = st["plan"]
    mtla.mtla_paged_append(d, st["B"], chunk, merge, ROPE_BASE, st["q_rope"], st["q_rope_out"], cache, st["tail_in"], st["tail_out"], st["t_out"],
                           st["cache_len"], st["row_state"], ws, size, st["dev_err"])
    return {"pages": st["pages"], "row_state": st["row_state"], "tail": st["tail_out"], "t": st["t_out"], "cache_len": st["cache_len"], "q_rope": st["q_rope_out"]}


def _own_attn(st):
    import temporally_compressed_latent_b200 as mtla
    if "plan" not in st:
        st["plan"] = _plan(st)
    d, chunk, cache, _, ws, size = st["plan"]
    mtla.mtla_paged_attn(d, st["B"], chunk, st["q_abs"], st["q_rope"], st["row_state"], cache, st["out"], d.dtype, st["lse"], ws, size, st["dev_err"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_verify(st):
    import temporally_compressed_latent_b200 as mtla
    V = st["case"]["V"]
    mtla.mtla_verify_drafts(st["B"], st["N"], V, st["p"], V, st["q"], V, st["tokens"], st["tok_start"], st["u_accept"], st["u_sample"],
                            st["n_keep"], st["next_token"], st["dev_err"])
    return {"n_keep": st["n_keep"], "next_token": st["next_token"]}


_own = {"append": _own_append, "attn": _own_attn, "verify": _own_verify}


# ----------------------------------------------------------------- work and the definition in 64 bits


def work(case):
    new, past = _lengths(case)
    N = sum(new)
    if case["op"] == "verify":
        # the two gathered probabilities of every draft, then one row of each distribution a sequence (the draft's
        # row is not needed where every draft is accepted: counted all the same, since the case does not say)
        return {"bytes": case["B"] * 8 * case["V"] + 16 * N + 24 * case["B"], "flops": 4 * case["B"] * case["V"]}
    s, H, r, D = case["s"], case["H"], case["r"], case["r"] + case["d_R"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        groups = [(t // s, _up(t + x, s)) for t, x in zip(past, new)]  # touched groups of each sequence
        positions = len(set().union(*(range(a, b) for a, b in groups)))  # distinct rows of P
        moved = N * (2 * D + 2 * H * case["d_R"]) * e + sum(b - a for a, b in groups) * D * e
        return {"bytes": moved + positions * D * 4 + (r + 1) * D * 4 + 2 * case["B"] * D * 4, "flops": 2 * r * D * N}
    rows = sum(_up(t + x, s) - 1 for t, x in zip(past, new))
    seen = sum(sum(_up(t + 1 + i, s) for i in range(x)) for t, x in zip(past, new))
    return {"bytes": (rows + N) * D * e + N * H * (D + r) * e + 4 * N * H, "flops": seen * H * 2 * (D + r)}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact[case["op"]](case, st, *_lengths(case))


def _exact_rotate(x, first):
    """x [n, ..., d_R] at positions first, first + 1, ...: complex numbers times e^(i angle)."""
    d = x.shape[-1]
    k = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    pos = torch.arange(first, first + x.shape[0], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos[:, None] * torch.exp(-2 * k / d * math.log(ROPE_BASE))[None, :])
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], d // 2, 2).contiguous())
    z = z * (turn if x.dim() == 2 else turn[:, None])
    return torch.view_as_real(z).flatten(-2)


def _exact_append(case, st, new, past):
    s, pr = case["s"], case["page_rows"]
    table, pages = st["block_table"].tolist(), st["pages"].double()
    states, tails, queries, at = [], [], [], 0
    for b, (n, t0) in enumerate(zip(new, past)):
        c = st["c"][at:at + n].double()
        groups = torch.arange(t0, t0 + n, device=c.device) // s            # 0-based
        gate = 1 / (1 + torch.exp(-(c @ st["W_c"].double() + st["b_c"].double()) * st["P"].double()[groups]))
        entry = gate * torch.cat([c, _exact_rotate(st["kR"][at:at + n], t0)], dim=1)
        # one row of s slots a group, the earlier part of the first group in its slot 0
        g0, g1 = t0 // s, (t0 + n - 1) // s + 1
        slots = torch.zeros((g1 - g0) * s, entry.shape[1], dtype=torch.float64, device=c.device)
        off = t0 - g0 * s
        slots[off:off + n] = entry
        if off:
            slots[0] = st["tail_in"][b].double()
        sums = slots.view(g1 - g0, s, -1).cumsum(dim=1)
        flat = sums.reshape(-1, entry.shape[1])[off:off + n]
        states.append(flat)
        tails.append(flat[-1])
        ends = torch.clamp((torch.arange(g0, g1, device=c.device) + 1) * s, max=t0 + n) - 1 - t0
        where = torch.tensor([table[b][g // pr] * pr + g % pr for g in range(g0, g1)], device=c.device)
        pages.view(-1, pages.shape[-1])[where] = flat[ends]
        queries.append(_exact_rotate(st["q_rope"][at:at + n], t0))
        at += n
    t = torch.tensor([a + b for a, b in zip(past, new)], dtype=torch.int32)
    return {"pages": pages, "row_state": torch.cat(states), "tail": torch.stack(tails), "t": t, "cache_len": ((t + s - 1) // s).int(), "q_rope": torch.cat(queries)}


def _exact_attn(case, st, new, past):
    s, pr, r = case["s"], case["page_rows"], case["r"]
    flat, table = st["pages"].view(-1, st["pages"].shape[-1]), st["block_table"].long()
    outs, lses, at = [], [], 0
    for b, (n, t0) in enumerate(zip(new, past)):
        seen = torch.tensor([_up(t0 + 1 + i, s) - 1 for i in range(n)], device=flat.device)
        g = torch.arange(int(seen[-1]), device=flat.device)
        rows = flat[table[b, g // pr] * pr + g % pr].double()
        for lo in range(0, n, 64):
            hi = min(n, lo + 64)
            q = torch.cat([st["q_abs"][at + lo:at + hi], st["q_rope"][at + lo:at + hi]], dim=2).double()
            mine = st["row_state"][at + lo:at + hi].double()
            x = torch.cat([torch.einsum("nhd,ld->nhl", q, rows), torch.einsum("nhd,nd->nh", q, mine)[..., None]], dim=2) / math.sqrt(case["d_h"])
            x[:, :, :len(g)].masked_fill_((g[None, :] >= seen[lo:hi, None])[:, None, :], -math.inf)
            w = torch.softmax(x, dim=2)
            outs.append(torch.einsum("nhl,lr->nhr", w[:, :, :-1], rows[:, :r]) + w[:, :, -1:] * mine[:, None, :r])
            lses.append(torch.logsumexp(x, dim=2))
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_verify(case, st, new, past):
    keeps, tokens, at = [], [], 0
    ids, u = st["tokens"].tolist(), st["u_accept"].double().tolist()
    for b, n in enumerate(new):
        keep = 1
        while keep < n:
            i, x = at + keep - 1, ids[at + keep]
            if not u[i] * float(st["q"][i, x]) < float(st["p"][i, x]):
                break
            keep += 1
        i = at + keep - 1
        weight = st["p"][i].double().cpu()
        if keep < n:
            rest = torch.relu(weight - st["q"][i].double().cpu())
            weight = rest if float(rest.sum()) > 0 else weight
        cdf = torch.cumsum(weight, dim=0)
        tokens.append(int((cdf > float(st["u_sample"][b]) * float(cdf[-1])).nonzero()[0]))
        keeps.append(keep)
        at += n
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)
    return {"n_keep": i32(keeps), "next_token": i32(tokens)}


_exact = {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify}
