"""Workloads of the caches that hold less a token than keys and values in 16 bits,
and of the attention that reads them: keys and values in 4 bits (appending to such a
cache, and attention over it), and one shared latent vector a token (appending its
normalised latent and rotated key, and attention in the absorbed form).

Each case names an operator and its sizes; `prepare` makes its inputs on the GPU,
`run` makes one call (`own`: the library's; else the operator's definition in
elementary torch operations), `exact` gives the definition's value in 64 bits.

Layouts as in include/pa.h: query and output [rows][heads][head_size], int32 tables
and lengths, and
  4 bits   codes uint8 [num_blocks][kv_heads][block_size][head_size / 2] (element 2i in
           the low half of byte i), scales f16 [..][block_size][head_size / 64][2]: the
           lowest value and the step of every 64 elements; a code c stands for
           lowest + c * step
  latent   [num_blocks][block_size][latent_dim + rope_dim]
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"
GROUP = 64  # elements that share a lowest value and a step
ROPE = 64   # rotated elements of a latent cache's row
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one user's next token at the end of a 100,000-token conversation: pure latency
        dict(name="q4_append_one_token", op="q4_append", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=1, chunk_lo=0, chunk_hi=0, ctx_lo=99999, ctx_hi=99999,
             rotary_dim=128, interleaved=False, query=True, positions=False, lens_seed=1),
        # a full decode batch's next tokens
        dict(name="q4_append_decode_256", op="q4_append", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=256, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=700,
             rotary_dim=128, interleaved=False, query=True, positions=False, lens_seed=2),
        # prompts and prompt pieces of ragged lengths behind a shared prefix (positions are
        # the caller's), a quarter of each wide head rotated in adjacent pairs
        dict(name="q4_append_prompts_f16", op="q4_append", dtype="f16", heads=16, kv_heads=2, head_size=256,
             block_size=32, seqs=37, chunk_lo=1, chunk_hi=441, ctx_lo=0, ctx_hi=300,
             rotary_dim=64, interleaved=True, query=True, positions=True, lens_seed=3),
        # a decode batch over contexts of 512 to 3584 tokens
        dict(name="q4_decode_256", op="q4", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=256, chunk=0, len_lo=512, len_hi=3584, log_lens=False, lens_seed=4),
        # one conversation of 100,000 tokens
        dict(name="q4_1_of_100k", op="q4", dtype="bf16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=1, chunk=0, len_lo=100000, len_hi=100000, log_lens=False, lens_seed=5),
        # up to five draft tokens a sequence to verify
        dict(name="q4_drafts_f16", op="q4", dtype="f16", heads=32, kv_heads=4, head_size=128,
             block_size=16, seqs=8, chunk=5, len_lo=1024, len_hi=8192, log_lens=False, lens_seed=6),
        # lengths from a few tokens to very long ones in one batch, wide heads
        dict(name="q4_mixed_d256", op="q4", dtype="bf16", heads=16, kv_heads=2, head_size=256,
             block_size=32, seqs=64, chunk=0, len_lo=16, len_hi=32768, log_lens=True, lens_seed=7),
        # a decode batch's next latents and rotated query parts
        dict(name="latent_append_decode_256", op="latent_append", dtype="bf16", heads=32, latent=512,
             block_size=16, seqs=256, chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=700,
             norm=True, interleaved=True, query=True, positions=False, lens_seed=8),
        # prompts of ragged lengths joining a running batch
        dict(name="latent_append_prompts_f16", op="latent_append", dtype="f16", heads=16, latent=256,
             block_size=32, seqs=37, chunk_lo=1, chunk_hi=441, ctx_lo=0, ctx_hi=300,
             norm=True, interleaved=False, query=True, positions=False, lens_seed=9),
        # one conversation of 100,000 tokens on a GPU that holds a share of the heads: a read
        dict(name="latent_1_of_100k", op="latent", dtype="bf16", heads=16, latent=512,
             block_size=16, seqs=1, chunk=0, len_lo=100000, len_hi=100000, log_lens=False, lens_seed=10),
        # a decode batch with every head on one GPU: as much arithmetic as reading
        dict(name="latent_64_heads128", op="latent", dtype="bf16", heads=128, latent=512,
             block_size=64, seqs=64, chunk=0, len_lo=1024, len_hi=8192, log_lens=False, lens_seed=11),
        # up to three draft tokens a sequence to verify, a smaller latent
        dict(name="latent_drafts_f16", op="latent", dtype="f16", heads=24, latent=256,
             block_size=32, seqs=8, chunk=3, len_lo=100, len_hi=8192, log_lens=False, lens_seed=12),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4_append", "q4", "q4", "latent_append", "latent", "latent"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), block_size=rng.choice([8, 16, 32, 64]),
             lens_seed=rng.randrange(1, 10 ** 6))
    if op.startswith("q4"):
        kv = rng.choice([1, 2, 4, 8])
        c.update(head_size=rng.choice([64, 128, 128, 256]), kv_heads=kv,
                 heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]))
    else:
        c.update(latent=rng.choice([256, 512, 512]), heads=rng.choice([1, 5, 8, 16, 24, 32, 40, 64, 128]))
    if op.endswith("append"):
        c["interleaved"] = rng.random() < 0.5
        c["query"] = rng.random() < 0.8
        c["positions"] = rng.random() < 0.3
        if op == "q4_append":
            D = c["head_size"]
            c["rotary_dim"] = rng.choice([0, 16, D // 2, D, D])
        else:
            c["norm"] = rng.random() < 0.8
        if rng.random() < 0.5:
            c.update(seqs=_log_uniform(rng, 1, 256), chunk_lo=0, chunk_hi=0, ctx_lo=0, ctx_hi=rng.randint(0, 700))
        else:
            n = _log_uniform(rng, 1, 64)
            top = _log_uniform(rng, 1, max(1, 6000 // n))
            c.update(seqs=n, chunk_lo=rng.choice([0, 1, top]), chunk_hi=max(1, top), ctx_lo=0,
                     ctx_hi=rng.randint(0, 300))
    else:
        chunk = rng.choice([0, 0, 0, 2, 5])
        n = _log_uniform(rng, 1, 256)
        top = _log_uniform(rng, 16, 100000)
        while top * n > 400000:
            top //= 2
        top = max(top, chunk, 1)
        c.update(seqs=n, chunk=chunk, len_lo=max(1, chunk, top // rng.choice([1, 2, 50])), len_hi=top,
                 log_lens=rng.random() < 0.4)
    # never more than the largest listed cases' bytes and operations
    while c["seqs"] > 1 and (work(c)["bytes"] > 3e8 or work(c)["flops"] > 7e10):
        c["seqs"] //= 2
    return c


def _lengths(case):
    """The case's integers: lengths (and what goes with them) that both `work`
    and `prepare` need, from the case alone."""
    rng = random.Random(case["lens_seed"])
    n = case["seqs"]
    if case["op"].endswith("append"):
        ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        if case["chunk_hi"] == 0:
            new = [1] * n
        else:
            new = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(n)]
            new[0] = max(new[0], 1)
        return dict(ctx=ctx, new=new, lens=[a + b for a, b in zip(ctx, new)],
                    offset=[rng.randint(0, 5000) if case["positions"] else 0 for _ in range(n)])
    lo, hi = case["len_lo"], case["len_hi"]
    if case["log_lens"]:
        lens = [_log_uniform(rng, lo, hi) for _ in range(n)]
    else:
        lens = [rng.randint(lo, hi) for _ in range(n)]
    new = [1] * n
    if case["chunk"]:
        new = [rng.randint(0, case["chunk"]) for _ in range(n)]
        new[-1] = case["chunk"]
    return dict(lens=lens, new=new)


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# Inputs

def _tables(lens, bs, g, spare):
    """Block tables of scattered pages (-1 where a sequence has none), and the
    number of pages."""
    pages = [_ceil(L, bs) for L in lens]
    total = sum(pages)
    perm = torch.randperm(total + spare, generator=g, device=DEVICE)[:total].to(torch.int32)
    width = max(max(pages, default=0), 1)
    bt = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt, total + spare


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


def _random_q4(pool, K, bs, D, g, mult):
    """A cache in 4 bits of normal keys (or values), quantised in pieces."""
    codes = torch.empty(pool, K, bs, D // 2, dtype=torch.uint8, device=DEVICE)
    scales = torch.empty(pool, K, bs, D // GROUP, 2, dtype=torch.float16, device=DEVICE)
    step = max(1, (1 << 25) // (K * bs * D))
    for i in range(0, pool, step):
        n = min(step, pool - i)
        x = torch.randn(n, K, bs, D, generator=g, device=DEVICE) * mult
        codes[i:i + n], scales[i:i + n], _ = _quantise(x)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    z = _lengths(case)
    dt = DTYPES[case["dtype"]]
    H, bs, op = case["heads"], case["block_size"], case["op"]
    rows = sum(z["new"])
    bt, pool = _tables(z["lens"], bs, g, 3)
    st = dict(case=case, dtype=dt, lens=z["lens"], new=z["new"], block_tables=bt,
              seq_lens=_ints(z["lens"]), max_len=max(z["lens"]))
    many = case["chunk_hi"] if op.endswith("append") else case["chunk"]
    st["q_start"] = _ints(_starts(z["new"])) if many else None
    if op.startswith("q4"):
        K, D = case["kv_heads"], case["head_size"]
        st["scale"] = 1.0 / math.sqrt(D)
        st["key_cache"], st["key_scales"] = _random_q4(pool, K, bs, D, g, 2.0)
        st["value_cache"], st["value_scales"] = _random_q4(pool, K, bs, D, g, 1.0)
        if op == "q4":
            st["query"] = _randn((rows, H, D), dt, g)
        else:
            # the projection's output as a model has it: query, key and value heads of
            # a token side by side
            qkv = _randn((rows, (H + 2 * K) * D), dt, g)
            st["query"] = qkv[:, :H * D].view(rows, H, D) if case["query"] else None
            st["key"] = qkv[:, H * D:(H + K) * D].view(rows, K, D)
            st["value"] = qkv[:, (H + K) * D:].view(rows, K, D)
            st["query_out"] = torch.zeros(rows, H, D, dtype=dt, device=DEVICE) if case["query"] else None
            st["key_out"] = torch.zeros(rows, K, D, dtype=dt, device=DEVICE)
            st["value_out"] = torch.zeros(rows, K, D, dtype=dt, device=DEVICE)
    else:
        L = case["latent"]
        st["scale"] = 1.0 / math.sqrt(128 + ROPE)  # heads of 128 + 64 before the absorption
        st["cache"] = _randn((pool, bs, L + ROPE), dt, g)
        if op == "latent":
            # absorbed queries: a head's 128 elements through its up-projection
            st["query"] = _randn((rows, H, L + ROPE), dt, g)
            st["query"][..., :L] *= math.sqrt(128 / L)
        else:
            down = _randn((rows, L + ROPE), dt, g, 3.0)  # the down-projection's output
            st["latent"], st["rope_key"] = down[:, :L], down[:, L:]
            st["norm_weight"] = (1 + 0.1 * torch.randn(L, generator=g, device=DEVICE)).to(dt) if case["norm"] else None
            st["query"] = _randn((rows, H, L + ROPE), dt, g) if case["query"] else None
            q = _randn((rows, H, 128 + ROPE), dt, g)  # the query projection's output
            st["query_rope"] = q[..., 128:] if case["query"] else None
    if op.endswith("append"):
        pos = [c + o + i for c, n, o in zip(z["ctx"], z["new"], z["offset"]) for i in range(n)]
        st["positions"] = _ints(pos) if case["positions"] else None
        R = case["rotary_dim"] if op == "q4_append" else ROPE
        st["cos_sin"] = None
        if R:
            top = max(pos, default=0) + 1
            inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R)
            ang = torch.arange(top, dtype=torch.float64, device=DEVICE)[:, None] * inv
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import paged_decode_attention_v2_gb300 as pa
    c = st["case"]
    st["pa"] = pa
    if c["op"].endswith("append"):
        st["workspace"] = pa.alloc_workspace(1, 1, 64, 0, 64)  # the status block alone
        return
    if c["op"] == "q4":
        st["workspace"] = pa.alloc_q4_workspace(c["head_size"])
        st["out"] = torch.empty_like(st["query"])
    else:
        st["workspace"] = pa.alloc_latent_workspace(c["latent"])
        st["out"] = torch.empty(st["query"].shape[0], c["heads"], c["latent"], dtype=st["dtype"], device=DEVICE)


# ---------------------------------------------------------------------------
# One pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"q4_append": _own_q4_append, "q4": _own_q4, "latent_append": _own_latent_append,
                "latent": _own_latent}[op](state)
    return {"q4_append": _plain_q4_append, "q4": _plain_q4, "latent_append": _plain_latent_append,
            "latent": _plain_latent}[op](state)


def _q4_append_outputs(st):
    # the cache as it is (codes have to agree bit by bit), and the values that the new
    # tokens' codes stand for
    out = {k: st[k] for k in ("key_cache", "value_cache", "key_scales", "value_scales")}
    out["key"], out["value"] = st["key_out"], st["value_out"]
    if st["query"] is not None:
        out["query"] = st["query_out"]
    return out


def _own_q4_append(st):
    c = st["case"]
    st["pa"].pa_q4_append(
        st["key_cache"], st["value_cache"], st["key_scales"], st["value_scales"], st["key"],
        st["value"], st["block_tables"], st["seq_lens"], st["workspace"], query=st["query"],
        query_out=st["query_out"], key_out=st["key_out"], value_out=st["value_out"],
        cos_sin=st["cos_sin"], positions=st["positions"], q_start=st["q_start"],
        rotary_dim=c["rotary_dim"], interleaved=c["interleaved"], max_seq_len=st["max_len"])
    return _q4_append_outputs(st)


def _own_q4(st):
    st["pa"].pa_q4_forward(
        st["out"], st["query"], st["key_cache"], st["value_cache"], st["key_scales"],
        st["value_scales"], st["block_tables"], st["seq_lens"], st["scale"], st["workspace"],
        q_start=st["q_start"], max_seq_len=st["max_len"])
    return {"out": st["out"]}


def _latent_append_outputs(st):
    out = {"cache": st["cache"]}
    if st["query"] is not None:
        out["query"] = st["query"]
    return out


def _own_latent_append(st):
    st["pa"].pa_latent_append(
        st["cache"], st["latent"], st["rope_key"], st["block_tables"], st["seq_lens"],
        st["workspace"], st["cos_sin"], query=st["query"], query_rope=st["query_rope"],
        norm_weight=st["norm_weight"], eps=EPS, positions=st["positions"], q_start=st["q_start"],
        interleaved=st["case"]["interleaved"], max_seq_len=st["max_len"])
    return _latent_append_outputs(st)


def _own_latent(st):
    st["pa"].pa_latent_forward(
        st["out"], st["query"], st["cache"], st["block_tables"], st["seq_lens"], st["scale"],
        st["workspace"], q_start=st["q_start"], max_seq_len=st["max_len"])
    return {"out": st["out"]}


# ---------------------------------------------------------------------------
# The plain forms

def _quantise(x):
    """x [..., D] in fp32 as (codes, scales, the values that they stand for): of every 64
    elements the lowest value and a fifteenth of the range, both rounded to f16 (and
    no further from zero than f16's largest), and the nearest multiples of it."""
    y = x.unflatten(-1, (-1, GROUP))
    lo = y.amin(-1, keepdim=True).clamp(-65504.0, 65504.0).half()
    step = ((y.amax(-1, keepdim=True) - lo.float()) * (1.0 / 15.0)).clamp(0.0, 65504.0).half()
    q = (y - lo.float()) * torch.where(step > 0, torch.reciprocal(step.float()), 0.0)
    q = torch.round(q).clamp(0.0, 15.0)
    c = q.to(torch.uint8).flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([lo, step], -1),
            (lo.float() + q * step.float()).flatten(-2))


def _values(codes, scales):
    """The values, in fp32, that codes and scales stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (scales[..., :1].float() + c * scales[..., 1:].float()).flatten(-2)


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


def _places(st, rows):
    """The rows' sequences, tokens and positions."""
    r = torch.arange(rows, device=DEVICE)
    lens = st["seq_lens"].long()
    if st["q_start"] is None:
        seq, at = r, lens - 1
    else:
        qs = st["q_start"].long()
        seq = (r[:, None] >= qs[None, 1:]).sum(1)
        at = lens[seq] - (qs[seq + 1] - qs[seq]) + r - qs[seq]
    positions = st.get("positions")
    return seq, at, positions.long() if positions is not None else at


def _plain_q4_append(st):
    c, dt = st["case"], st["dtype"]
    bs, R = c["block_size"], c["rotary_dim"]
    seq, at, pos = _places(st, st["key"].shape[0])
    page = st["block_tables"][seq, at // bs].long()
    k = _rotate(st["key"].float(), pos, st["cos_sin"], R, c["interleaved"]).to(dt)
    for name, x in (("key", k), ("value", st["value"])):
        codes, scales, values = _quantise(x.float())
        st[name + "_cache"][page, :, at % bs] = codes
        st[name + "_scales"][page, :, at % bs] = scales
        st[name + "_out"].copy_(values)
    if st["query"] is not None:
        st["query_out"].copy_(_rotate(st["query"].float(), pos, st["cos_sin"], R, c["interleaved"]))
    return _q4_append_outputs(st)


def _plain_latent_append(st):
    c, dt = st["case"], st["dtype"]
    L, bs = c["latent"], c["block_size"]
    seq, at, pos = _places(st, st["latent"].shape[0])
    page = st["block_tables"][seq, at // bs].long()
    x = st["latent"].float()
    if st["norm_weight"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["norm_weight"].float()
    k = _rotate(st["rope_key"].float()[:, None], pos, st["cos_sin"], ROPE, c["interleaved"])[:, 0]
    st["cache"][page, at % bs] = torch.cat([x, k], -1).to(dt)
    if st["query"] is not None:
        st["query"][..., L:] = _rotate(st["query_rope"].float(), pos, st["cos_sin"], ROPE, c["interleaved"]).to(dt)
    return _latent_append_outputs(st)


def _chunk_rows(st):
    """For the plain attention: the rows as [sequences, longest chunk], padded with a
    sequence's last row, and whether each place is a row of its own."""
    n = max(max(st["new"]), 1)
    i = torch.arange(n, device=DEVICE)[None]
    new = _ints(st["new"]).long()[:, None]
    first = new.cumsum(0) - new
    return (first + torch.minimum(i, (new - 1).clamp_min(0))).clamp_max(sum(st["new"]) - 1), i < new


def _plain_attention(st, k, v, heads):
    """k, v [sequences, heads, tokens, ...] against the chunks' rows of st["query"]; heads
    of k and v are shared by `heads` query heads each."""
    idx, live = _chunk_rows(st)
    B, n = idx.shape
    q = st["query"][idx].float()  # [sequences, chunk, H, D]
    K, D = k.shape[1], q.shape[-1]
    q = q.view(B, n, K, heads, D).permute(0, 2, 1, 3, 4).reshape(B, K, n * heads, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    new = _ints(st["new"]).long()
    vis = st["seq_lens"].long()[:, None] - new[:, None] + torch.arange(n, device=DEVICE)[None] + 1
    vis = vis.clamp_min(1).repeat_interleave(heads, 1)  # [sequences, chunk * heads]
    dead = torch.arange(k.shape[2], device=DEVICE)[None, None] >= vis[..., None]
    x = x.masked_fill(dead[:, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(e / e.sum(-1, keepdim=True), v)  # [B, K, n * heads, Dv]
    o = o.view(B, K, n, heads, -1).permute(0, 2, 1, 3, 4).reshape(B, n, K * heads, -1)
    return {"out": o[live].to(st["dtype"])}


def _pages(st):
    """[sequences, tokens] page and place of every token up to the longest length."""
    bs = st["case"]["block_size"]
    t = torch.arange(st["max_len"], device=DEVICE)
    return st["block_tables"][:, t // bs].clamp_min(0).long(), t % bs


def _plain_q4(st):
    page, at = _pages(st)
    at = at.expand_as(page)
    dead = torch.arange(st["max_len"], device=DEVICE)[None] >= st["seq_lens"][:, None]
    k = _values(st["key_cache"][page, :, at], st["key_scales"][page, :, at]).transpose(1, 2)
    v = _values(st["value_cache"][page, :, at], st["value_scales"][page, :, at])
    v = v.masked_fill(dead[:, :, None, None], 0.0).transpose(1, 2)
    return _plain_attention(st, k, v, st["case"]["heads"] // st["case"]["kv_heads"])


def _plain_latent(st):
    page, at = _pages(st)
    dead = torch.arange(st["max_len"], device=DEVICE)[None] >= st["seq_lens"][:, None]
    k = st["cache"][page, at.expand_as(page)].float().masked_fill(dead[..., None], 0.0)[:, None]
    return _plain_attention(st, k, k[..., :st["case"]["latent"]], st["case"]["heads"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence

def exact(case, seed):
    st = prepare(case, seed)
    return {"q4_append": _exact_q4_append, "q4": _exact_q4, "latent_append": _exact_latent_append,
            "latent": _exact_latent}[case["op"]](st)


def _turn(x, cs, interleaved):
    """x [n, heads, R] in 64 bits as complex numbers times the unit ones of cs [n, R]."""
    R = x.shape[-1]
    z = torch.complex(cs[:, :R // 2], cs[:, R // 2:])[:, None]
    if interleaved:
        pair = x.unflatten(-1, (R // 2, 2))
        return torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * z).flatten(-2)
    w = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:].contiguous()) * z
    return torch.cat([w.real, w.imag], -1)


def _spans(st):
    """(sequence, rows, tokens, positions) of each sequence with new tokens."""
    row = 0
    for s, (n, L) in enumerate(zip(st["new"], st["lens"])):
        if n:
            rows, at = slice(row, row + n), torch.arange(L - n, L, device=DEVICE)
            yield s, rows, at, at if st.get("positions") is None else st["positions"][rows].long()
        row += n


def _exact_q4_append(st):
    c, dt = st["case"], st["dtype"]
    bs, R = c["block_size"], c["rotary_dim"]

    def stands_for(x):  # the 64-bit values of the codes of x [n, K, D]
        y = x.reshape(*x.shape[:-1], -1, GROUP)
        lo = y.min(-1).values.half().double()[..., None]
        step = ((y.max(-1).values[..., None] - lo) / 15).half().double()
        level = torch.round((y - lo) / step.clamp_min(1e-30)).clamp(0, 15)
        return torch.where(step > 0, lo + level * step, lo).reshape(x.shape), lo, step

    out = dict(key_cache=None, value_cache=None, key_scales=st["key_scales"].double(),
               value_scales=st["value_scales"].double(), key=st["key_out"].double(), value=st["value_out"].double())
    if st["query"] is not None:
        out["query"] = st["query_out"].double()
    for s, rows, at, pos in _spans(st):
        def turn(x):
            x = x.double()
            return torch.cat([_turn(x[..., :R], st["cos_sin"][pos].double(), c["interleaved"]), x[..., R:]], -1) if R else x

        page = st["block_tables"][s, at // bs].long()
        for name, x in (("key", turn(st["key"][rows]).to(dt).double()), ("value", st["value"][rows].double())):
            out[name][rows], lo, step = stands_for(x)
            out[name + "_scales"][page, :, at % bs] = torch.cat([lo, step], -1)
        if st["query"] is not None:
            out["query"][rows] = turn(st["query"][rows])
    return out


def _exact_latent_append(st):
    c = st["case"]
    L, bs = c["latent"], c["block_size"]
    out = {"cache": st["cache"].double()}
    if st["query"] is not None:
        out["query"] = st["query"].double()
    for s, rows, at, pos in _spans(st):
        cs = st["cos_sin"][pos].double()
        x = st["latent"][rows].double()
        if st["norm_weight"] is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / L + EPS) * st["norm_weight"].double()
        page = st["block_tables"][s, at // bs].long()
        out["cache"][page, at % bs] = torch.cat([x, _turn(st["rope_key"][rows].double()[:, None], cs, c["interleaved"])[:, 0]], -1)
        if st["query"] is not None:
            out["query"][rows, :, L:] = _turn(st["query_rope"][rows].double(), cs, c["interleaved"])
    return out


def _exact_q4(st):
    c = st["case"]
    H, K, D, bs = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    rows = st["query"].shape[0]
    out = torch.zeros(rows, K, H // K, D, dtype=torch.float64, device=DEVICE)
    q = st["query"].double().view(rows, K, H // K, D)

    def read(name, table, tok):  # [K, n, D]
        b = st[name + "_cache"][table[tok // bs].long(), :, tok % bs].long()
        s = st[name + "_scales"][table[tok // bs].long(), :, tok % bs].double().repeat_interleave(GROUP, 2)
        x = torch.empty(*b.shape[:-1], D, dtype=torch.float64, device=DEVICE)
        x[..., 0::2], x[..., 1::2] = (b % 16).double(), (b // 16).double()
        return (x * s[..., 1] + s[..., 0]).transpose(0, 1)

    row = 0
    for s, (n, L) in enumerate(zip(st["new"], st["lens"])):
        if not n:
            continue
        tok = torch.arange(L, device=DEVICE)
        k, v = read("key", st["block_tables"][s], tok), read("value", st["block_tables"][s], tok)
        for i in range(n):
            m = L - n + i + 1
            out[row] = torch.softmax((q[row] @ k[:, :m].transpose(1, 2)) * st["scale"], -1) @ v[:, :m]
            row += 1
    return {"out": out.view(rows, H, D)}


def _exact_latent(st):
    c = st["case"]
    bs, L = c["block_size"], c["latent"]
    rows = st["query"].shape[0]
    out = torch.zeros(rows, c["heads"], L, dtype=torch.float64, device=DEVICE)
    row = 0
    for s, (n, length) in enumerate(zip(st["new"], st["lens"])):
        tok = torch.arange(length, device=DEVICE)
        kv = st["cache"][st["block_tables"][s, tok // bs].long(), tok % bs].double()
        for i in range(n):
            m = length - n + i + 1
            out[row] = torch.softmax((st["query"][row].double() @ kv[:m].T) * st["scale"], -1) @ kv[:m, :L]
            row += 1
    return {"out": out}


# ---------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    z = _lengths(case)
    H, op = case["heads"], case["op"]
    rows = sum(z["new"])
    ints = 4 * len(z["lens"]) * (2 if op.endswith("append") else 1)
    if op == "q4_append":
        K, D, R = case["kv_heads"], case["head_size"], case["rotary_dim"]
        held = D // 2 + 4 * (D // GROUP)
        b = rows * 2 * K * (2 * D + held + 2 * D) + rows * (R * 4 + 4) + ints
        b += 4 * rows * H * D if case["query"] else 0
        f = 3 * rows * (K + (H if case["query"] else 0)) * R + rows * 2 * K * D * 6
        return {"bytes": float(b), "flops": float(f)}
    if op == "latent_append":
        L = case["latent"]
        b = 4 * rows * (L + ROPE) + rows * (ROPE * 4 + 4) + ints + (2 * L if case["norm"] else 0)
        b += 4 * rows * H * ROPE if case["query"] else 0
        return {"bytes": float(b), "flops": float(rows * (4 * L + 3 * ROPE * (H + 1)))}
    keys = sum(L for L, n in zip(z["lens"], z["new"]) if n)
    pairs = sum(L - n + i + 1 for L, n in zip(z["lens"], z["new"]) for i in range(n))
    pages = sum(_ceil(L, case["block_size"]) for L, n in zip(z["lens"], z["new"]) if n)
    if op == "q4":
        K, D = case["kv_heads"], case["head_size"]
        return {"bytes": float(2 * keys * K * (D // 2 + 4 * (D // GROUP)) + 4 * rows * H * D + 4 * pages + ints),
                "flops": float(4 * pairs * H * D)}
    L = case["latent"]
    return {"bytes": float(2 * keys * (L + ROPE) + 2 * rows * H * (2 * L + ROPE) + 4 * pages + ints),
            "flops": float(2 * pairs * H * (2 * L + ROPE))}
