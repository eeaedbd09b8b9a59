"""Workloads of the operators around the paged cache: appending keys and values
to it (with the position rotation on the way), decode attention for batches that
share a prefix, and decode attention over blocks that a cheap score selects.

Each case names an operator and its sizes; `prepare` makes its inputs on the GPU,
`run` makes one call (`own`: the library's; else the operator's definition in
elementary torch operations), `exact` gives the definition's value in 64 bits.

Layouts as in include/pa.h: query and output [rows][heads][head_size], caches
[num_blocks][kv_heads][block_size][head_size], int32 tables and lengths.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one user's next token at the end of a 100,000-token conversation: pure latency
        dict(name="append_one_token", op="append", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=1, chunk_lo=0, chunk_hi=0, ctx_lo=99999, ctx_hi=99999,
             rotary_dim=128, interleaved=False, bounds=True, query=True, positions=False, lens_seed=1),
        # a full decode batch's next tokens
        dict(name="append_decode_256", op="append", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=256, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=700,
             rotary_dim=128, interleaved=False, bounds=True, query=True, positions=False, lens_seed=2),
        # prompts and prompt pieces of ragged lengths joining a running batch
        dict(name="append_prompts", op="append", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=37, chunk_lo=1, chunk_hi=441, ctx_lo=0, ctx_hi=300,
             rotary_dim=128, interleaved=False, bounds=True, query=True, positions=False, lens_seed=3),
        # a small fp32 model that rotates half of each head in adjacent pairs; the
        # positions are the caller's (behind a prefix that other sequences share)
        dict(name="append_f32_partial", op="append", dtype="f32", heads=4, kv_heads=1, head_size=64,
             block_size=8, seqs=19, chunk_lo=1, chunk_hi=129, ctx_lo=0, ctx_hi=77,
             rotary_dim=32, interleaved=True, bounds=False, query=True, positions=True, lens_seed=4),
        # a batch of requests behind one long system prompt: the prefix is a matrix product
        dict(name="prefix_256", op="prefix", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, groups=1, seqs=256, prefix_lo=8192, prefix_hi=8192,
             suffix_lo=16, suffix_hi=512, lens_seed=5),
        # a few samples of one very long document's answer: the prefix is a read
        dict(name="prefix_8_of_100k", op="prefix", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, groups=1, seqs=8, prefix_lo=100000, prefix_hi=100000,
             suffix_lo=1, suffix_hi=300, lens_seed=6),
        # several prompts, each with its own odd number of requests
        dict(name="prefix_groups_f16", op="prefix", dtype="f16", heads=32, kv_heads=4, head_size=64,
             block_size=8, groups=5, seqs=63, prefix_lo=1, prefix_hi=2999,
             suffix_lo=0, suffix_hi=200, lens_seed=7),
        # wide heads, larger pages
        dict(name="prefix_d256", op="prefix", dtype="bf16", heads=16, kv_heads=2, head_size=256,
             block_size=32, groups=2, seqs=64, prefix_lo=9001, prefix_hi=16001,
             suffix_lo=1, suffix_hi=1000, lens_seed=8),
        # a decode batch that reads 32 blocks (512 tokens) a head of up to 3584 tokens
        dict(name="sparse_256", op="sparse", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=256, chunk=0, len_lo=512, len_hi=3584, log_lens=False,
             selected=32, sinks=1, recent=2, partition=512, lens_seed=9),
        # one conversation of 100,000 tokens, 4096 of them read
        dict(name="sparse_1_of_100k", op="sparse", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=1, chunk=0, len_lo=100000, len_hi=100000, log_lens=False,
             selected=256, sinks=1, recent=4, partition=128, lens_seed=10),
        # four draft tokens a sequence to verify, each with its own blocks
        dict(name="sparse_drafts_f16", op="sparse", dtype="f16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=8, chunk=4, len_lo=1024, len_hi=8192, log_lens=False,
             selected=48, sinks=0, recent=1, partition=512, lens_seed=11),
        # lengths from a few tokens to very long ones in one batch, wide heads
        dict(name="sparse_mixed_d256", op="sparse", dtype="bf16", heads=16, kv_heads=2, head_size=256,
             block_size=32, seqs=64, chunk=0, len_lo=16, len_hi=131072, log_lens=True,
             selected=64, sinks=2, recent=2, partition=512, lens_seed=12),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "prefix", "sparse"])
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]) if D < 256 else rng.choice([1, 2, 4, 8])
    c = dict(op=op, heads=kv * G, kv_heads=kv, head_size=D, block_size=rng.choice([8, 16, 32, 64]),
             lens_seed=rng.randrange(1, 10 ** 6))
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["rotary_dim"] = rng.choice([0, 16, D // 2, D, D])
        c["interleaved"] = rng.random() < 0.4
        c["bounds"] = rng.random() < 0.6
        c["query"] = rng.random() < 0.8
        c["positions"] = rng.random() < 0.3
        if rng.random() < 0.5:
            c.update(seqs=_log_uniform(rng, 1, 256), chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=rng.randint(0, 700))
        else:
            n = _log_uniform(rng, 1, 64)
            top = _log_uniform(rng, 1, max(1, 6000 // n))
            c.update(seqs=n, chunk_lo=rng.choice([0, 1, top]), chunk_hi=max(1, top), ctx_lo=0,
                     ctx_hi=rng.randint(0, 300))
    elif op == "prefix":
        c["dtype"] = rng.choice(["bf16", "f16"])
        n = _log_uniform(rng, 1, 256)
        top = _log_uniform(rng, 16, 100000)
        while top * n * G * kv * D > 8192 * 256 * 32 * 64:
            top //= 2
        c.update(seqs=n, groups=rng.randint(1, min(n, 6)), prefix_lo=rng.choice([0, top // 2, top]),
                 prefix_hi=top, suffix_lo=rng.choice([0, 1]), suffix_hi=_log_uniform(rng, 1, 512))
    else:
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        n = _log_uniform(rng, 1, 256)
        top = _log_uniform(rng, 16, 100000)
        while top * n * kv * D > 3000 * 256 * 4 * 128:
            top //= 2
        chunk = rng.choice([0, 0, 0, 2, 5])
        sel = _log_uniform(rng, 4, 256)
        while sel * c["block_size"] * n * max(chunk, 1) * kv * G * D > 32 * 16 * 256 * 32 * 128:
            sel = max(4, sel // 2)
            if sel == 4:
                break
        c.update(seqs=n, chunk=chunk, len_lo=max(1, chunk, top // rng.choice([1, 2, 50])), len_hi=max(top, chunk, 1),
                 log_lens=rng.random() < 0.4, selected=sel, sinks=rng.choice([0, 1, 2]), recent=rng.choice([1, 2]),
                 partition=rng.choice([128, 256, 512]))
    # never more than the largest listed cases' bytes and operations
    while c["seqs"] > 1 and (work(c)["bytes"] > 2.5e8 or work(c)["flops"] > 3e10):
        c["seqs"] //= 2
        if op == "prefix":
            c["groups"] = min(c["groups"], c["seqs"])
    return c


def _lengths(case):
    """The case's integers: lengths (and what goes with them) that both `work`
    and `prepare` need, from the case alone."""
    rng = random.Random(case["lens_seed"])
    n = case["seqs"]
    if case["op"] == "append":
        ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        if case["chunk_hi"] == 0:
            new = [1] * n
        else:
            new = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(n)]
            new[0] = max(new[0], 1)
        return dict(ctx=ctx, new=new, lens=[a + b for a, b in zip(ctx, new)],
                    offset=[rng.randint(0, 5000) if case["positions"] else 0 for _ in range(n)])
    if case["op"] == "prefix":
        cuts = sorted(rng.randint(0, n) for _ in range(case["groups"] - 1))
        return dict(start=[0] + cuts + [n],
                    prefix=[rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["groups"])],
                    lens=[rng.randint(case["suffix_lo"], case["suffix_hi"]) for _ in range(n)])
    lo, hi = case["len_lo"], case["len_hi"]
    if case["log_lens"]:
        return dict(lens=[_log_uniform(rng, lo, hi) for _ in range(n)])
    return dict(lens=[rng.randint(lo, hi) for _ in range(n)])


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# Inputs

def _tables(lens, bs, g, spare, first=0):
    """Block tables of scattered pages (-1 where a sequence has none), from page
    `first` on; and the number of pages."""
    pages = [_ceil(L, bs) for L in lens]
    total = sum(pages)
    perm = torch.randperm(total + spare, generator=g, device=DEVICE)[:total].to(torch.int32) + first
    width = max(max(pages, default=0), 1)
    bt = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt, first + total + spare


def _randn(shape, dtype, g, mult=1.0):
    out = torch.empty(shape, dtype=dtype, device=DEVICE)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):  # pieces: no fp32 copy of a whole cache
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEVICE) * mult
    return out


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    z = _lengths(case)
    dt = DTYPES[case["dtype"]]
    H, K, D, bs = case["heads"], case["kv_heads"], case["head_size"], case["block_size"]
    st = dict(case=case, dtype=dt, lens=z["lens"], scale=1.0 / math.sqrt(D))
    if case["op"] == "prefix":
        # the prefixes' pages and the sequences' own, in one pool
        ptab, first = _tables(z["prefix"], bs, g, 1)
        bt, pool = _tables(z["lens"], bs, g, 1, first)
        st.update(prefix_tables=ptab, prefix_lens=_ints(z["prefix"]), prefix_start=_ints(z["start"]),
                  prefix=z["prefix"], start=z["start"])
    else:
        bt, pool = _tables(z["lens"], bs, g, 3)
    st.update(block_tables=bt, seq_lens=_ints(z["lens"]), max_len=max(z["lens"]))
    st["key_cache"] = _randn((pool, K, bs, D), dt, g, 1.0 if case["op"] == "append" else 2.0)
    st["value_cache"] = _randn((pool, K, bs, D), dt, g)
    if case["op"] == "append":
        rows = sum(z["new"])
        # the projection's output as a model has it: query, key and value heads of
        # a token side by side
        qkv = _randn((max(rows, 1), (H + 2 * K) * D), dt, g)[:rows]
        st["query"] = qkv[:, :H * D].view(rows, H, D) if case["query"] else None
        st["key"] = qkv[:, H * D:(H + K) * D].view(rows, K, D)
        st["value"] = qkv[:, (H + K) * D:].view(rows, K, D)
        st["query_out"] = torch.zeros(rows, H, D, dtype=dt, device=DEVICE) if case["query"] else None
        st["q_start"] = None if case["chunk_hi"] == 0 else _ints(_starts(z["new"]))
        st["new"], st["max_new"] = z["new"], max(z["new"])
        pos = [c + o + i for c, n, o in zip(z["ctx"], z["new"], z["offset"]) for i in range(n)]
        st["positions"] = _ints(pos) if case["positions"] else None
        R = case["rotary_dim"]
        st["cos_sin"] = None
        if R:
            top = max(pos, default=0) + 1
            inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R)
            ang = torch.arange(top, dtype=torch.float64, device=DEVICE)[:, None] * inv
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["key_bounds"] = None
        if case["bounds"]:
            st["key_bounds"] = _randn((pool, K, 2, D), dt, g)
            _set_bounds(st, z["ctx"])  # what earlier appends left
    elif case["op"] == "prefix":
        st["query"] = _randn((case["seqs"], H, D), dt, g)
    else:
        n = case["chunk"] or 1
        rows = case["seqs"] * n
        st["query"] = _randn((rows, H, D), dt, g)
        st["q_start"] = _ints([i * n for i in range(case["seqs"] + 1)]) if case["chunk"] else None
        st["rows_per_seq"] = n
        st["key_bounds"] = torch.zeros(pool, K, 2, D, dtype=dt, device=DEVICE)
        _set_bounds(st, z["lens"])
    if own:
        _prepare_own(st)
    return st


def _set_bounds(st, lens):
    """key_bounds of the pages of each sequence's first `lens` tokens."""
    bs = st["case"]["block_size"]
    kc, bt, kb = st["key_cache"], st["block_tables"], st["key_bounds"]
    full = [(s, L // bs) for s, L in enumerate(lens) if L // bs]
    if full:
        pages = torch.cat([bt[s, :n] for s, n in full]).long()
        for part in pages.split(1 << 14):
            k = kc[part]
            kb[part] = torch.stack([k.amax(2), k.amin(2)], 2)
    rest = [(s, L) for s, L in enumerate(lens) if L % bs]
    if rest:
        pages = torch.stack([bt[s, L // bs] for s, L in rest]).long()
        k = kc[pages]
        dead = torch.arange(bs, device=DEVICE)[None, :] >= _ints([L % bs for _, L in rest])[:, None]
        dead = dead[:, None, :, None]
        kb[pages] = torch.stack([k.masked_fill(dead, -math.inf).amax(2),
                                 k.masked_fill(dead, math.inf).amin(2)], 2)


def _prepare_own(st):
    import paged_decode_attention_v2_gb300 as pa
    c = st["case"]
    st["pa"] = pa
    H, K, D = c["heads"], c["kv_heads"], c["head_size"]
    if c["op"] == "append":
        st["workspace"] = pa.alloc_workspace(1, 1, 64, 0, 64)  # the status block alone
        return
    st["out"] = torch.empty_like(st["query"])
    if c["op"] == "prefix":
        st["workspace"] = pa.alloc_prefix_workspace(
            c["seqs"], len(st["prefix"]), H, K, D, st["max_len"], max(st["prefix"]), 512)
    else:
        rows = st["query"].shape[0]
        st["selected"] = torch.empty(rows, K, c["selected"], dtype=torch.int32, device=DEVICE)
        st["workspace"] = pa.alloc_sparse_workspace(
            rows, H, K, D, c["block_size"], st["max_len"], c["selected"], c["partition"])


# ---------------------------------------------------------------------------
# One pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "prefix": _own_prefix, "sparse": _own_sparse}[op](state)
    return {"append": _plain_append, "prefix": _plain_prefix, "sparse": _plain_sparse}[op](state)


def _append_outputs(st):
    out = {"key_cache": st["key_cache"], "value_cache": st["value_cache"]}
    if st["query"] is not None:
        out["query"] = st["query_out"]
    if st["key_bounds"] is not None:
        out["key_bounds"] = st["key_bounds"]
    return out


def _own_append(st):
    c = st["case"]
    st["pa"].pa_append_kv(
        st["key_cache"], st["value_cache"], st["key"], st["value"], st["block_tables"],
        st["seq_lens"], st["workspace"], query=st["query"], query_out=st["query_out"],
        key_bounds=st["key_bounds"], cos_sin=st["cos_sin"], positions=st["positions"],
        q_start=st["q_start"], rotary_dim=c["rotary_dim"], interleaved=c["interleaved"],
        max_seq_len=st["max_len"])
    return _append_outputs(st)


def _own_prefix(st):
    st["pa"].pa_prefix_forward(
        st["out"], st["query"], st["key_cache"], st["value_cache"], st["block_tables"],
        st["seq_lens"], st["prefix_tables"], st["prefix_lens"], st["prefix_start"], st["scale"],
        512, st["workspace"], max_seq_len=st["max_len"], max_prefix_len=max(st["prefix"]))
    return {"out": st["out"]}


def _own_sparse(st):
    c = st["case"]
    st["pa"].pa_sparse_forward(
        st["out"], st["selected"], st["query"], st["key_cache"], st["value_cache"],
        st["block_tables"], st["seq_lens"], st["scale"], c["partition"], st["workspace"],
        key_bounds=st["key_bounds"], sink_blocks=c["sinks"], recent_blocks=c["recent"],
        q_start=st["q_start"], max_seq_len=st["max_len"])
    return {"out": st["out"], "selected": st["selected"]}


# ---------------------------------------------------------------------------
# The plain forms

def _rotate(x, pos, cos_sin, R, interleaved):
    """x [rows, heads, D] in fp32, the first R elements of each head rotated by
    the angles of its row's position."""
    if not R:
        return x
    cs = cos_sin[pos]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * c - b * s
        y[..., 1:R:2] = b * c + a * s
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * c - b * s
        y[..., R // 2:R] = b * c + a * s
    return y


def _plain_append(st):
    c, dt = st["case"], st["dtype"]
    bs, R = c["block_size"], c["rotary_dim"]
    rows = st["key"].shape[0]
    r = torch.arange(rows, device=DEVICE)
    lens = st["seq_lens"].long()
    if st["q_start"] is None:
        seq, at = r, lens - 1
    else:
        qs = st["q_start"].long()
        seq = (r[:, None] >= qs[None, 1:]).sum(1)
        at = lens[seq] - (qs[seq + 1] - qs[seq]) + r - qs[seq]
    pos = st["positions"].long() if st["positions"] is not None else at
    k = _rotate(st["key"].float(), pos, st["cos_sin"], R, c["interleaved"])
    page = st["block_tables"][seq, at // bs].long()
    st["key_cache"][page, :, at % bs] = k.to(dt)
    st["value_cache"][page, :, at % bs] = st["value"]
    if st["query"] is not None:
        st["query_out"].copy_(_rotate(st["query"].float(), pos, st["cos_sin"], R, c["interleaved"]))
    if st["key_bounds"] is not None:
        # the touched pages' bounds over the tokens that the sequence now holds
        live = (at // bs * bs)[:, None] + torch.arange(bs, device=DEVICE)[None] < lens[seq][:, None]
        live = live[:, None, :, None]
        k = st["key_cache"][page]
        st["key_bounds"][page] = torch.stack([torch.where(live, k, -math.inf).amax(2),
                                              torch.where(live, k, math.inf).amin(2)], 2)
    return _append_outputs(st)


def _gather(cache, table, n, bs):
    """Keys (or values) of the first n tokens of each table row, in fp32:
    [rows, kv_heads, n, D]."""
    t = torch.arange(n, device=DEVICE)
    pages = table[:, t // bs].clamp_min(0).long()
    return cache[pages, :, t % bs].float().transpose(1, 2)


def _plain_prefix(st):
    c = st["case"]
    H, K, D, bs = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    G = H // K
    n = st["max_len"]
    q = st["query"].float().view(-1, K, G, D)
    out = torch.zeros_like(q)
    for i, P in enumerate(st["prefix"]):  # computed once for the sequences of a group
        a, b = st["start"][i], st["start"][i + 1]
        if a == b or P + n == 0:
            continue
        B = b - a
        kp = _gather(st["key_cache"], st["prefix_tables"][i:i + 1], P, bs)[0]
        vp = _gather(st["value_cache"], st["prefix_tables"][i:i + 1], P, bs)[0]
        qk = q[a:b].transpose(0, 1).reshape(K, B * G, D)
        sp = torch.matmul(qk, kp.transpose(1, 2)).view(K, B, G, P).transpose(0, 1) * st["scale"]
        ks = _gather(st["key_cache"], st["block_tables"][a:b], n, bs)
        ss = torch.matmul(q[a:b], ks.transpose(2, 3)) * st["scale"]
        dead = torch.arange(n, device=DEVICE)[None] >= st["seq_lens"][a:b, None]
        ss = ss.masked_fill(dead[:, None, None], -math.inf)
        s = torch.cat([sp, ss], 3)
        m = s.amax(3, keepdim=True)
        e = torch.where(s == -math.inf, 0.0, torch.exp(s - m))
        e = e / e.sum(3, keepdim=True).clamp_min(1e-30)
        ep = e[..., :P].transpose(0, 1).reshape(K, B * G, P)
        o = torch.matmul(ep, vp).view(K, B, G, D).transpose(0, 1)
        vs = _gather(st["value_cache"], st["block_tables"][a:b], n, bs)
        vs = vs.masked_fill(dead[:, None, :, None], 0.0)
        out[a:b] = o + torch.matmul(e[..., P:], vs)
    return {"out": out.view(-1, H, D).to(st["dtype"])}


def _plain_sparse(st):
    c = st["case"]
    H, K, D, bs = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    G, k = H // K, c["selected"]
    n = st["rows_per_seq"]
    rows = st["query"].shape[0]
    seq = torch.arange(rows, device=DEVICE) // n
    vis = st["seq_lens"].long()[seq] - n + torch.arange(rows, device=DEVICE) % n + 1  # keys a row sees
    bt = st["block_tables"]
    W = _ceil(st["max_len"], bs)
    pages = (vis + bs - 1) // bs
    # the scores: 64 bits, since nearly equal ones decide which block is read
    q = st["query"].double().view(rows, K, G, D)
    w = torch.stack([q.clamp_min(0).sum(2), q.clamp_max(0).sum(2)], 2)  # [rows, K, 2, D]
    score = torch.empty(rows, K, W, dtype=torch.float64, device=DEVICE)
    for a in range(0, W, 512):
        t = bt[:, a:min(a + 512, W)].clamp_min(0).long()
        kb = st["key_bounds"][t].double()  # [seqs, pages, K, 2, D]
        kb = kb.permute(0, 2, 1, 3, 4).reshape(len(st["lens"]), K, t.shape[1], 2 * D)
        wr = w.view(-1, n, K, 2 * D).permute(0, 2, 3, 1)
        score[:, :, a:a + t.shape[1]] = torch.matmul(kb, wr).permute(0, 3, 1, 2).reshape(rows, K, -1)
    j = torch.arange(W, device=DEVICE)[None]
    forced = (j < c["sinks"]) | (j >= pages[:, None] - c["recent"])
    score = score.masked_fill(forced[:, None], math.inf)
    score = score.masked_fill((j >= pages[:, None])[:, None], -math.inf)
    if W < k:
        score = torch.nn.functional.pad(score, (0, k - W), value=-math.inf)
    top, idx = torch.sort(score, dim=2, descending=True, stable=True)
    idx = idx[..., :k].masked_fill(top[..., :k] == -math.inf, 1 << 30).sort(2).values
    sel = idx.masked_fill(idx == 1 << 30, -1)
    out = torch.empty(rows, K, G, D, device=DEVICE)
    step = max(1, (1 << 27) // (K * k * bs * D))
    for a in range(0, rows, step):
        r = slice(a, min(a + step, rows))
        s = sel[r]
        page = torch.gather(bt[seq[r]][:, None].expand(-1, K, -1), 2, s.clamp_min(0).long()).long()
        h = torch.arange(K, device=DEVICE)[None, :, None]
        tok = s[..., None] * bs + torch.arange(bs, device=DEVICE)
        dead = ((tok >= vis[r][:, None, None, None]) | (s < 0)[..., None]).flatten(2)
        kk = st["key_cache"][page, h].float().flatten(2, 3)
        x = torch.matmul(st["query"][r].float().view(-1, K, G, D), kk.transpose(2, 3)) * st["scale"]
        x = x.masked_fill(dead[:, :, None], -math.inf)
        e = torch.exp(x - x.amax(3, keepdim=True))
        e = e / e.sum(3, keepdim=True)
        vv = st["value_cache"][page, h].float().flatten(2, 3).masked_fill(dead[..., None], 0.0)
        out[r] = torch.matmul(e, vv)
    return {"out": out.view(rows, H, D).to(st["dtype"]), "selected": sel.to(torch.int32)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "prefix": _exact_prefix, "sparse": _exact_sparse}[case["op"]](st)


def _exact_append(st):
    c = st["case"]
    bs, R = c["block_size"], c["rotary_dim"]
    kc, vc = st["key_cache"].double(), st["value_cache"].double()
    qo = st["query_out"].double() if st["query"] is not None else None
    kb = st["key_bounds"].double() if st["key_bounds"] is not None else None
    row = 0
    for s, (n, L) in enumerate(zip(st["new"], st["lens"])):
        if n == 0:
            continue
        rows = slice(row, row + n)
        at = torch.arange(L - n, L, device=DEVICE)
        pos = at if st["positions"] is None else st["positions"][rows].long()

        def turn(x):
            x = x.double()
            if not R:
                return x
            cs = st["cos_sin"][pos].double()
            z = torch.complex(cs[:, :R // 2], cs[:, R // 2:])[:, None]
            if c["interleaved"]:
                pair = x[..., :R].unflatten(-1, (R // 2, 2))
                y = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * z).flatten(-2)
            else:
                w = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
                y = torch.cat([w.real, w.imag], -1)
            return torch.cat([y, x[..., R:]], -1)

        page = st["block_tables"][s, at // bs].long()
        kc[page, :, at % bs] = turn(st["key"][rows])
        vc[page, :, at % bs] = st["value"][rows].double()
        if qo is not None:
            qo[rows] = turn(st["query"][rows])
        if kb is not None:
            for j in range((L - n) // bs, _ceil(L, bs)):
                p = int(st["block_tables"][s, j])
                k = kc[p, :, :min(bs, L - j * bs)]
                kb[p, :, 0] = k.max(1).values
                kb[p, :, 1] = k.min(1).values
        row += n
    out = {"key_cache": kc, "value_cache": vc}
    if qo is not None:
        out["query"] = qo
    if kb is not None:
        out["key_bounds"] = kb
    return out


def _tokens(cache, table, tok, bs):
    """Rows of the cache for token numbers `tok` of one table row: [K, n, D] in 64 bits."""
    return cache[table[tok // bs].long(), :, tok % bs].double().transpose(0, 1)


def _exact_prefix(st):
    c = st["case"]
    H, K, D, bs = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    out = torch.zeros(c["seqs"], K, H // K, D, dtype=torch.float64, device=DEVICE)
    q = st["query"].double().view(-1, K, H // K, D)
    for i, P in enumerate(st["prefix"]):
        tp = torch.arange(P, device=DEVICE)
        kp = _tokens(st["key_cache"], st["prefix_tables"][i], tp, bs)
        vp = _tokens(st["value_cache"], st["prefix_tables"][i], tp, bs)
        for s in range(st["start"][i], st["start"][i + 1]):
            ts = torch.arange(st["lens"][s], device=DEVICE)
            k = torch.cat([kp, _tokens(st["key_cache"], st["block_tables"][s], ts, bs)], 1)
            v = torch.cat([vp, _tokens(st["value_cache"], st["block_tables"][s], ts, bs)], 1)
            if k.shape[1]:
                out[s] = torch.softmax((q[s] @ k.transpose(1, 2)) * st["scale"], -1) @ v
    return {"out": out.view(-1, H, D)}


def _exact_sparse(st):
    c = st["case"]
    H, K, D, bs = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    G, k, n = H // K, c["selected"], st["rows_per_seq"]
    rows = st["query"].shape[0]
    q = st["query"].double().view(rows, K, G, D)
    out = torch.zeros(rows, K, G, D, dtype=torch.float64, device=DEVICE)
    sel = torch.full((rows, K, k), -1, dtype=torch.int32, device=DEVICE)
    for s, L in enumerate(st["lens"]):
        table = st["block_tables"][s]
        kb = st["key_bounds"][table[:_ceil(L, bs)].long()].double()  # [pages, K, 2, D]
        for i in range(n):
            r, vis = s * n + i, L - n + i + 1
            pages = _ceil(vis, bs)
            # a head's bound on q.k over a page: the larger end of each channel
            lim = torch.zeros(pages, K, dtype=torch.float64, device=DEVICE)
            for h in range(G):
                lim += torch.maximum(q[r, :, h] * kb[:pages, :, 0], q[r, :, h] * kb[:pages, :, 1]).sum(-1)
            lim[:c["sinks"]] = math.inf
            lim[max(pages - c["recent"], 0):] = math.inf
            order = torch.sort(-lim, dim=0, stable=True).indices[:k].sort(0).values  # [<=k, K]
            sel[r, :, :order.shape[0]] = order.T.to(torch.int32)
            tok = order.T[:, :, None] * bs + torch.arange(bs, device=DEVICE)
            tok = tok.flatten(1)
            for h in range(K):
                t = tok[h][tok[h] < vis]
                kk = st["key_cache"][table[t // bs].long(), h, t % bs].double()
                vv = st["value_cache"][table[t // bs].long(), h, t % bs].double()
                out[r, h] = torch.softmax((q[r, h] @ kk.T) * st["scale"], -1) @ vv
    return {"out": out.view(rows, H, D), "selected": sel}


# ---------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    z = _lengths(case)
    e = 4 if case["dtype"] == "f32" else 2
    H, K, D, bs = case["heads"], case["kv_heads"], case["head_size"], case["block_size"]
    if case["op"] == "append":
        rows = sum(z["new"])
        heads = 2 * K + (H if case["query"] else 0)
        R = case["rotary_dim"]
        b = 2 * rows * heads * D * e + rows * (R * 4 + 4) + len(z["lens"]) * 8
        if case["bounds"]:
            for n, L in zip(z["new"], z["lens"]):
                if n:
                    pages = _ceil(L, bs) - (L - n) // bs
                    b += (pages + (1 if (L - n) % bs else 0)) * K * 2 * D * e
        return {"bytes": float(b), "flops": float(3 * rows * (heads - K) * R)}
    if case["op"] == "prefix":
        keys = sum(P for P, a, b in zip(z["prefix"], z["start"], z["start"][1:]) if b > a) + sum(z["lens"])
        pairs = sum(P * (b - a) for P, a, b in zip(z["prefix"], z["start"], z["start"][1:])) + sum(z["lens"])
        return {"bytes": float(2 * keys * K * D * e + 2 * case["seqs"] * H * D * e + 4 * keys / bs),
                "flops": float(4 * pairs * H * D)}
    n = case["chunk"] or 1
    b = 2 * case["seqs"] * n * H * D * e
    f = 0
    for L in z["lens"]:
        pages = _ceil(L, bs)
        read = 0
        for i in range(n):
            vis = L - n + i + 1
            p = _ceil(vis, bs)
            tok = min(case["selected"], p) * bs - (p * bs - vis)
            read += tok
            f += 4 * tok * H * D + 4 * p * K * D
            b += 4 * K * min(case["selected"], p)
        b += pages * (K * 2 * D * e + 4)
        # the rows of one sequence may share blocks: no block more than once
        b += 2 * min(read, L) * K * D * e
    return {"bytes": float(b), "flops": float(f)}
