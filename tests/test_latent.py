"""pa_latent_append and pa_latent_forward: a paged cache of shared latents against
its definition in 64 bits, their refusals (CPU), their reports of bad data and their
bounded waits."""
import math
import random

import pytest
import torch

import paged_decode_attention_v2_gb300 as pa

FAKE = 1 << 20  # aligned, never dereferenced by the host checks
ROPE = 64

APPEND = dict(cache=FAKE, query=FAKE, query_rope=FAKE, latent=FAKE, rope_key=FAKE, norm_weight=FAKE,
              eps=1e-6, query_stride=8 * 192, query_head_stride=192, latent_stride=576,
              rope_key_stride=576, cos_sin=FAKE, positions=FAKE, block_tables=FAKE, seq_lens=FAKE,
              q_start=FAKE, num_seqs=2, num_rows=5, num_heads=8, latent_dim=512, rope_dim=64,
              num_blocks=64, block_size=16, max_blocks_per_seq=8, max_seq_len=128, interleaved=0,
              max_position=200, dtype=pa.PA_DTYPE_BF16, workspace=FAKE, workspace_bytes=256, stream=0)
FORWARD = dict(out=FAKE, query=FAKE, cache=FAKE, block_tables=FAKE, seq_lens=FAKE, q_start=FAKE,
               num_seqs=2, num_rows=5, num_heads=8, latent_dim=512, rope_dim=64, num_blocks=64,
               block_size=16, max_blocks_per_seq=8, max_seq_len=128, scale=0.1,
               dtype=pa.PA_DTYPE_BF16, workspace=FAKE, workspace_bytes=1 << 40, stream=0, opts=None)

# The parity bar of the framework's 16-bit calls, for latents of deviation 1: a
# weight is rounded to the type (2^-8 of it for bf16, the sums taking it as rounded, so
# only unlike roundings of a row's weights count), the output again (2^-8 of it).
ATOL, RTOL = 4e-3, 1e-2


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return pa.load_library()


@pytest.mark.parametrize("over,status", [
    (dict(cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(latent=0), pa.PA_ERR_INVALID_ARG),
    (dict(rope_key=0), pa.PA_ERR_INVALID_ARG),
    (dict(cos_sin=0), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(query=0), pa.PA_ERR_INVALID_ARG),
    (dict(query_rope=0), pa.PA_ERR_INVALID_ARG),
    (dict(eps=-1.0), pa.PA_ERR_INVALID_ARG),
    (dict(eps=math.nan), pa.PA_ERR_INVALID_ARG),
    (dict(interleaved=2), pa.PA_ERR_INVALID_ARG),
    (dict(max_position=0), pa.PA_ERR_INVALID_ARG),
    (dict(latent=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(norm_weight=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(positions=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 128), pa.PA_ERR_INVALID_ARG),
    (dict(latent_stride=504), pa.PA_ERR_INVALID_ARG),
    (dict(latent_stride=516), pa.PA_ERR_INVALID_ARG),
    (dict(rope_key_stride=60), pa.PA_ERR_INVALID_ARG),
    (dict(query_head_stride=60), pa.PA_ERR_INVALID_ARG),
    (dict(query_stride=1400), pa.PA_ERR_INVALID_ARG),      # rows would overlap
    (dict(q_start=0), pa.PA_ERR_INVALID_ARG),
    (dict(num_rows=-1), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=7), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=pa.PA_DTYPE_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(latent_dim=384), pa.PA_ERR_UNSUPPORTED),
    (dict(rope_dim=32), pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=12, max_seq_len=96), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=129), pa.PA_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 28), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=255), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_append_refusals(lib, over, status):
    assert lib.pa_latent_append(*dict(APPEND, **over).values()) == status
    words = pa._LATENT_APPEND[1](*dict(APPEND, **over).values())
    assert lib.pa_call(2, words) == status


@pytest.mark.parametrize("over,status", [
    (dict(out=0), pa.PA_ERR_INVALID_ARG),
    (dict(cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(query=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(q_start=0), pa.PA_ERR_INVALID_ARG),
    (dict(scale=math.inf), pa.PA_ERR_INVALID_ARG),
    (dict(num_seqs=-1), pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=pa.PA_DTYPE_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(latent_dim=1024), pa.PA_ERR_UNSUPPORTED),
    (dict(rope_dim=0), pa.PA_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 28, max_seq_len=(1 << 30) + 1), pa.PA_ERR_UNSUPPORTED),
    (dict(num_rows=(1 << 31) - 1), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=4096), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_forward_refusals(lib, over, status):
    assert lib.pa_latent_forward(*dict(FORWARD, **over).values()) == status
    words = pa._LATENT_FORWARD[1](*dict(FORWARD, **dict(over, opts=0)).values())
    assert lib.pa_call(3, words) == status


def test_no_rows_is_no_work(lib):
    assert lib.pa_latent_append(*dict(APPEND, num_rows=0, latent=0, rope_key=0, query=0, query_rope=0).values()) == pa.PA_OK
    assert lib.pa_latent_forward(*dict(FORWARD, num_rows=0, query=0, out=0).values()) == pa.PA_OK


def test_workspace_sizes(lib):
    assert pa.pa_latent_workspace_bytes(384) == 0
    a, b = pa.pa_latent_workspace_bytes(256), pa.pa_latent_workspace_bytes(512)
    assert 0 < a < b and a % 256 == 0 and b % 256 == 0


def test_binding_refuses_host_tensors():
    cache = torch.zeros(4, 16, 320, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.pa_latent_append(cache, cache[0, :1, :256], cache[0, :1, 256:], i.view(1, 1), i, w, torch.zeros(4, 64))
    with pytest.raises(ValueError):
        pa.pa_latent_forward(torch.zeros(1, 1, 256), torch.zeros(1, 1, 320), cache, i.view(1, 1), i, 1.0, w)


# ---------------------------------------------------------------------------

def tables(lens, bs, g, spare=2):
    pages = [-(-max(L, 0) // bs) for L in lens]
    pool = sum(pages) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    bt = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
    return bt, pool


def turn(x, cs, il):
    """x [rows, heads, 64] in 64 bits, cs [rows, 64]."""
    c, s = cs[:, None, :32].double(), cs[:, None, 32:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if il else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, b * c + a * s
    return torch.stack([u, v], -1).flatten(-2) if il else torch.cat([u, v], -1)


def near(got, ref, dtype):
    """One rounding of fp32 arithmetic: half a step of the type, and 2^-20 of the largest
    term for the fp32 operations before it."""
    u = torch.finfo(dtype).eps / 2
    err = (got.double().cpu() - ref).abs()
    return (err <= 1.01 * u * ref.abs() + 2 ** -20 * ref.abs().amax().clamp_min(1e-30) + 2 ** -25).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L,bs,il,norm,query,decode", [
    (8, 512, 16, False, True, True, False), (1, 256, 8, True, True, True, False), (128, 512, 64, True, False, True, False),
    (5, 256, 32, False, True, False, False), (24, 512, 16, True, True, True, True)])
def test_append(dtype, H, L, bs, il, norm, query, decode):
    g = torch.Generator().manual_seed(H)
    new = [1] * 5 if decode else [5, 0, 1, 33, 700]
    lens = [n + c for n, c in zip(new, [0, 7, 15, 3, 60])]
    bt, pool = tables(lens, bs, g)
    rows, pad = sum(new), 0 if decode else 3
    down = (torch.randn(rows + pad, L + ROPE, generator=g) * 3).to(dtype)
    qfull = torch.randn(rows + pad, H, 128 + ROPE, generator=g).to(dtype)
    w = (1 + 0.2 * torch.randn(L, generator=g)).to(dtype) if norm else None
    cache = torch.randn(pool, bs, L + ROPE, generator=g).to(dtype)
    q = torch.randn(rows + pad, H, L + ROPE, generator=g).to(dtype)
    place = [(s, t) for s, (n, m) in enumerate(zip(new, lens)) for t in range(m - n, m)]
    ang = torch.arange(max(lens), dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    qs = [0]
    for n in new:
        qs.append(qs[-1] + n)
    d = "cuda"
    dc, dq, dd, dqf = cache.to(d), q.to(d), down.to(d), qfull.to(d)
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    pa.pa_latent_append(dc, dd[:, :L], dd[:, L:], bt.to(d), torch.tensor(lens, dtype=torch.int32, device=d), ws, cs.to(d),
                        query=dq if query else None, query_rope=dqf[..., 128:] if query else None,
                        norm_weight=w.to(d) if norm else None, eps=1e-5,
                        q_start=None if decode else torch.tensor(qs, dtype=torch.int32, device=d), interleaved=il)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    x = down[:rows].double()
    c = x[:, :L]
    if norm:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w.double()
    rcs = cs[[t for _, t in place]]
    ref = torch.cat([c, turn(x[:, None, L:], rcs, il)[:, 0]], -1)
    got = dc.cpu()
    at = [(int(bt[s, t // bs]), t % bs) for s, t in place]
    assert near(torch.stack([got[p, o] for p, o in at]), ref, dtype)
    for p, o in at:
        got[p, o] = cache[p, o]
    assert torch.equal(got, cache)  # nothing else
    gq = dq.cpu()
    if query:
        assert near(gq[:rows, :, L:], turn(qfull[:rows, :, 128:].double(), rcs, il), dtype)
        gq[:rows, :, L:] = q[:rows, :, L:]
    assert torch.equal(gq, q)


@pytest.mark.gpu
def test_append_bad_data():
    g = torch.Generator().manual_seed(1)
    for what in ("page", "length", "position", "chunk"):
        lens, new = [22, 4], [2, 3]
        bt, pool = tables(lens, 16, g)
        cache = torch.randn(pool, 16, 320, generator=g).bfloat16().cuda()
        before = cache.clone()
        own = bt[0, :2].long() if what != "chunk" else bt[1, :1].long()
        cs = torch.ones(64, 64)
        qs = [0, 2, 5]
        if what == "page":
            bt[0, 1] = 999
        elif what == "length":
            lens[0] = 10 ** 6
        elif what == "position":
            cs = cs[:10]
        else:
            qs = [0, 4, 3]  # (a chunk of sequence 0, and one that ends before it starts)
        x = torch.randn(5, 320, generator=g).bfloat16().cuda()
        ws = pa.alloc_workspace(1, 1, 64, 0, 64)
        pa.pa_latent_append(cache, x[:, :256], x[:, 256:], bt.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            ws, cs.cuda(), q_start=torch.tensor(qs, dtype=torch.int32, device="cuda"))
        assert pa.pa_read_device_status(ws) == pa.PA_ERR_DEVICE_BAD_INPUT
        assert torch.equal(cache[own], before[own]), what


# ---------------------------------------------------------------------------

class Attend:
    def __init__(self, seed, dtype, H, L, bs, lens, new=None, pad=0, qmult=1.0, cmult=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, L=L, bs=bs, lens=lens, scale=scale or 1 / math.sqrt(L + ROPE))
        self.new = new if new is not None else [1] * len(lens)
        self.chunks = new is not None
        self.bt, pool = tables(lens, bs, g)
        self.rows = sum(self.new)
        self.q = (torch.randn(self.rows + pad, H, L + ROPE, generator=g) * qmult).to(dtype)
        self.q[self.rows:] = float("nan")  # padding: never looked at by a row of its own
        self.cache = (torch.randn(pool, bs, L + ROPE, generator=g) * cmult).to(dtype)
        held = torch.zeros(pool, bs, dtype=torch.bool)
        for s, n in enumerate(lens):
            for t in range(max(n, 0)):
                held[self.bt[s, t // bs].long(), t % bs] = True
        self.cache[~held] = float("nan")

    def reference(self):
        c = self.cache.double()
        out = torch.full((len(self.q), self.H, self.L), 7.0, dtype=torch.float64)
        row = 0
        for s, (n, L) in enumerate(zip(self.new, self.lens)):
            t = torch.arange(max(L, 0))
            kv = c[self.bt[s, t // self.bs].long(), t % self.bs]
            for i in range(n):
                m = L - n + i + 1
                out[row] = torch.softmax(self.q[row].double() @ kv[:m].T * self.scale, -1) @ kv[:m, :self.L] if m > 0 else 0.0
                row += 1
        return out

    def device(self):
        d = "cuda"
        self.a = [t.to(d) for t in (self.q, self.cache, self.bt, torch.tensor(self.lens, dtype=torch.int32))]
        qs = [0]
        for n in self.new:
            qs.append(qs[-1] + n)
        self.qs = torch.tensor(qs, dtype=torch.int32, device=d) if self.chunks else None
        self.ws = pa.alloc_latent_workspace(self.L)
        return self

    def run(self, ws=None, out=None, stream=None, **kw):
        if out is None:
            out = torch.full((len(self.q), self.H, self.L), 7.0, dtype=self.dtype, device="cuda")
        pa.pa_latent_forward(out, *self.a, self.scale, self.ws if ws is None else ws, q_start=self.qs, stream=stream, **kw)
        return out

    def check(self, out, atol=ATOL, rtol=RTOL):
        ref = self.reference()
        err = (out.double().cpu() - ref).abs()
        assert (err <= atol + rtol * ref.abs()).all(), float((err - rtol * ref.abs()).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L,bs", [(1, 512, 16), (16, 512, 8), (64, 512, 64), (65, 512, 32), (128, 512, 16), (128, 256, 8),
                                    (24, 256, 16), (63, 256, 64)])
def test_decode(dtype, H, L, bs):
    c = Attend(1, dtype, H, L, bs, [0, 1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 0, 517]).device()
    c.check(c.run())
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L,bs", [(5, 512, 8), (64, 512, 64), (128, 512, 16), (33, 256, 32), (100, 256, 16)])
def test_chunks(dtype, H, L, bs):
    c = Attend(2, dtype, H, L, bs, [5, 40, 33, 1, 130, 64], [5, 0, 3, 1, 6, 17], pad=3).device()
    c.check(c.run())  # (rows behind the last sequence stay 7)
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("H,L,lens", [(4, 512, [30000]), (3, 256, [11000, 3, 12000]), (2, 512, [200] * 300), (80, 256, [6000, 1, 2500])])
def test_long_and_many(H, L, lens):
    c = Attend(3, torch.bfloat16, H, L, 16, lens).device()
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("H,L,new", [(4, 256, False), (80, 512, False), (24, 512, True)])
@pytest.mark.parametrize("lens", [[1] * 250 + [7000] + [2] * 40, [64] * 3, [100, 6000] + [5] * 60])
def test_short_beside_long(H, L, new, lens):
    """Shares that hold many whole units, parts of one, or end where a unit begins."""
    c = Attend(8, torch.bfloat16, H, L, 16, lens, [min(n, 3) for n in lens] if new else None).device()
    out = c.run()
    c.check(out)
    assert torch.equal(out, c.run())  # whoever takes which share


@pytest.mark.gpu
def test_peaked_scores():
    """Scores of +-1000, and none at all: maxima that rise late and by much."""
    for kw in (dict(qmult=8.0), dict(qmult=60.0), dict(qmult=0.0), dict(scale=-0.2)):
        for dtype in (torch.bfloat16, torch.float16):
            c = Attend(4, dtype, 16, 512, 16, [900, 40, 1], **kw).device()
            ref = c.reference()
            out = c.run().double().cpu()
            # scores of magnitude X are sums of 576 products in fp32: off by X 576 2^-24 at
            # most, and the output by that times the spread of the latents
            X = float((c.q[:c.rows].double().abs().sum(-1).amax() * 5 + 1) * abs(c.scale))
            assert ((out - ref).abs() <= ATOL + X * 576 * 2 ** -24 * 8 + RTOL * ref.abs()).all(), kw


@pytest.mark.gpu
@pytest.mark.parametrize("rise", ["up", "down", "steps"])
def test_maxima_that_rise(rise):
    """Keys in an order that makes every tile's largest score the largest so far."""
    c = Attend(5, torch.float16, 7, 256, 16, [1000])
    t = torch.arange(1000, dtype=torch.float64)
    lift = {"up": t / 25, "down": -t / 25, "steps": (t // 64) * 9.0}[rise]
    c.q[:, :, 256] = 1.0
    flat = c.cache[c.bt[0].long()].flatten(0, 1)
    flat[:1000, 256] = (lift / c.scale / 16).half()
    c.q[:, :, 256] = 16.0
    c.cache[c.bt[0].long()] = flat.view(-1, 16, 320)
    c.device()
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "length", "negative", "chunk"])
def test_bad_data(what):
    c = Attend(6, torch.bfloat16, 20, 512, 16, [100, 40, 70], [3, 2, 4] if what == "chunk" else None).device()
    ref = c.reference()
    q, cache, bt, sl = c.a
    if what == "page":
        bt[1, 1] = 10 ** 6
    elif what == "length":
        sl[1] = 10 ** 6
    elif what == "negative":
        sl[1] = -5
    else:
        c.qs = torch.tensor([0, 3, 5, 99], dtype=torch.int32, device="cuda")
    out = c.run().double().cpu()
    assert pa.pa_read_device_status(c.ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    for r in ([0, 2] if len(out) == 3 else [0, 1, 2, 3, 4]):
        assert ((out[r] - ref[r]).abs() <= ATOL + RTOL * ref[r].abs()).all()
    if what in ("length", "negative"):
        assert (out[1] == 0).all()
    d = Attend(7, torch.bfloat16, 8, 512, 16, [50]).device()
    d.check(d.run(ws=c.ws))
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
def test_bounded_waits():
    """Softmax warps that wait for a barrier nobody releases give up after the limit; the
    workspace serves again once initialised."""
    c = Attend(8, torch.bfloat16, 16, 512, 16, [300, 20]).device()
    c.run(debug_flags=pa.PA_DEBUG_STALL_CONSUMERS, wait_limit_ns=2_000_000)
    assert pa.pa_read_device_status(c.ws) == pa.PA_ERR_DEVICE_TIMEOUT
    pa.pa_workspace_init(c.ws)
    c.check(c.run())
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
def test_graph_shared_workspace_and_streams():
    a = Attend(10, torch.bfloat16, 128, 512, 16, [3000, 5, 700]).device()
    b = Attend(11, torch.bfloat16, 12, 512, 8, [44, 900], [7, 3]).device()
    oa = torch.zeros(3, 128, 512, dtype=torch.bfloat16, device="cuda")
    ob = torch.zeros(10, 12, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run(out=oa)
        b.run(ws=a.ws, out=ob)
        side.synchronize()
        graphs = []
        for c, o in ((a, oa), (b, ob)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                c.run(ws=a.ws, out=o)
            graphs.append(g)
        for _ in range(3):
            for g, o in zip(graphs, (oa, ob)):
                o.fill_(7.0)
                g.replay()
    side.synchronize()
    a.check(oa)
    b.check(ob)
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        x = a.run(out=oa)
        y = b.run(stream=s2, out=ob)
    torch.cuda.synchronize()
    a.check(x)
    b.check(y)


@pytest.mark.gpu
def test_far_pages():
    """Pages beyond 2^31 elements and 2^32 bytes."""
    bs, L = 64, 512
    nb = 70000
    cache = torch.empty(nb, bs, L + ROPE, dtype=torch.bfloat16, device="cuda")
    c = Attend(12, torch.bfloat16, 16, L, bs, [100, 65])
    src = c.cache
    far = {int(p): nb - 1 - 31 * i for i, p in enumerate(c.bt[c.bt >= 0].tolist())}
    for p, f in far.items():
        cache[f] = src[p].cuda()
    c.device()
    bt = c.bt.clone()
    for p, f in far.items():
        bt[c.bt == p] = f
    c.a[1], c.a[2] = cache, bt.cuda()
    c.check(c.run())
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
def test_decode_loop():
    """A prompt, then tokens one by one: appended, then attended to, against 64 bits over
    the rows that the cache then holds."""
    H, L, bs, dt = 20, 256, 16, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    rng = random.Random(4)
    prompt, steps = [37, 5, 90], 8
    B, top = len(prompt), max(prompt) + steps * 3
    width = -(-top // bs)
    cache = torch.zeros(B * width, bs, L + ROPE, dtype=dt, device="cuda")
    bt = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    ang = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    ws = pa.alloc_latent_workspace(L)
    w = torch.ones(L, dtype=dt, device="cuda")
    lens = [0] * B
    for k in range(steps + 1):
        new = prompt if k == 0 else [rng.randint(1, 3) for _ in range(B)]
        lens = [a + b for a, b in zip(lens, new)]
        rows = sum(new)
        qs = [0]
        for n in new:
            qs.append(qs[-1] + n)
        qs = torch.tensor(qs, dtype=torch.int32, device="cuda")
        down = torch.randn(rows, L + ROPE, generator=g).to(dt).cuda()
        query = torch.randn(rows, H, L + ROPE, generator=g).to(dt).cuda()
        rope = torch.randn(rows, H, ROPE, generator=g).to(dt).cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        pa.pa_latent_append(cache, down[:, :L], down[:, L:], bt, sl, ws, cs, query=query, query_rope=rope, norm_weight=w, eps=1e-6, q_start=qs)
        out = torch.empty(rows, H, L, dtype=dt, device="cuda")
        pa.pa_latent_forward(out, query, cache, bt, sl, 0.06, ws, q_start=qs)
        assert pa.pa_read_device_status(ws) == pa.PA_OK
        row = 0
        for s, n in enumerate(new):
            t = torch.arange(lens[s], device="cuda")
            kv = cache[bt[s, t // bs].long(), t % bs].double()
            for i in range(n):
                m = lens[s] - n + i + 1
                ref = torch.softmax(query[row].double() @ kv[:m].T * 0.06, -1) @ kv[:m, :L]
                assert ((out[row].double() - ref).abs() <= ATOL + RTOL * ref.abs()).all()
                row += 1


@pytest.mark.gpu
@pytest.mark.parametrize("H,L,lens", [(5, 256, [640, 65]), (16, 512, [3000, 64]), (80, 512, [640, 1000])])
def test_small_f16_weights(H, L, lens):
    """Weights of 2^-26 beside one of 1, every 64 keys, whose values make up for it: f16's
    smallest number is 2^-24.  A weight is off by 2^-32 of the largest at most."""
    c = Attend(30, torch.float16, H, L, 16, lens, scale=1.0)
    c.q.zero_()
    c.q[..., L] = 1.0
    for s, n in enumerate(lens):
        t = torch.arange(n)
        c.cache[c.bt[s, t // 16].long(), t % 16, :L] = 57344.0
        c.cache[c.bt[s, t // 16].long(), t % 16, L] = -18.25
        t = torch.arange(0, n, 64)
        c.cache[c.bt[s, t // 16].long(), t % 16, :L] = 0.0
        c.cache[c.bt[s, t // 16].long(), t % 16, L] = 0.0
    ref = c.reference()
    assert (ref > 0.02).all()
    err = (c.device().run().double().cpu() - ref).abs()
    assert (err <= 63 * 2 ** -32 * 57344 * 1.01 + (2 ** -11 + 2 ** -20) * ref).all(), float(err.max())


@pytest.mark.gpu
@pytest.mark.parametrize("deviation", [4.0, 6.0, 10.0])
def test_peaky_logits_within_the_parity_bar(deviation):
    """Few keys carry a row's weight, so that the rounding of single weights shows: 10
    million outputs, of 150 sequences that read the same 600 keys, whole units a share.
    Weights of up to 2^8, each off by half a step, left the bar by a factor of up to 1.4;
    where a key that outweighs half of all before it has a weight of 1, exact, the worst of
    12 million (simulated in 64 bits) is at 0.83 of it."""
    c = Attend(33, torch.bfloat16, 128, 512, 64, [600] + [0] * 149, scale=deviation / (512 + ROPE) ** 0.5)
    c.lens, c.bt = [600] * 150, c.bt[:1].expand(150, -1).contiguous()
    out = c.device().run()
    kv = c.a[1][c.a[2][0].long()].flatten(0, 1)[:600].double()
    for s in range(0, 150, 10):
        ref = torch.softmax(c.a[0][s:s + 10].double() @ kv.T * c.scale, -1) @ kv[:, :512]
        over = ((out[s:s + 10].double() - ref).abs() / (ATOL + RTOL * ref.abs())).max()
        assert over <= 1.0, float(over)


@pytest.mark.parametrize("over", [
    dict(),                                                                # other strides, same words
    dict(query_rope=FAKE + 520 * 2, query_head_stride=576, query_stride=8 * 576),  # eight elements on
    dict(query_rope=FAKE + (512 + 576) * 2, query_head_stride=576, query_stride=8 * 576),  # a head on
    dict(query_rope=FAKE + (512 - 576) * 2, query_head_stride=576, query_stride=8 * 576),
    dict(query_rope=FAKE - 64 * 2, query_head_stride=64, query_stride=512),
])
def test_append_refuses_queries_that_overlap(lib, over):
    """Words that are written before another head's are read."""
    assert lib.pa_latent_append(*dict(APPEND, **over).values()) == pa.PA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L,rows,at", [(8, 512, 700, 512), (1, 256, 3, 256), (24, 256, 1, 256), (8, 512, 700, 0)])
@pytest.mark.parametrize("il", [False, True])
def test_append_in_place(dtype, H, L, rows, at, il):
    """query_rope as the last elements of query's heads, or others that are not written."""
    g = torch.Generator().manual_seed(40)
    bt, pool = tables([rows + 9], 16, g)
    q = torch.randn(rows, H, L + ROPE, generator=g).to(dtype)
    down = torch.randn(rows, L + ROPE, generator=g).to(dtype).cuda()
    ang = torch.arange(rows + 9, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    cache = torch.zeros(pool, 16, L + ROPE, dtype=dtype, device="cuda")
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dq = q.cuda()
    pa.pa_latent_append(cache, down[:, :L], down[:, L:], bt.cuda(), i32([rows + 9]), ws, cs.cuda(), query=dq,
                        query_rope=dq[..., at:at + ROPE], q_start=i32([0, rows]), interleaved=il)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    got = dq.cpu()
    assert near(got[..., L:], turn(q[..., at:at + ROPE].double(), cs[9:], il), dtype)
    assert torch.equal(got[..., :L], q[..., :L])


@pytest.mark.gpu
def test_append_queries_heads_first():
    """query_rope as a view of [heads][rows][64]: heads further apart than rows."""
    g = torch.Generator().manual_seed(41)
    H, L, rows, dt = 6, 256, 37, torch.bfloat16
    bt, pool = tables([rows], 16, g)
    rope = torch.randn(H, rows, ROPE, generator=g).to(dt)
    down = torch.randn(rows, L + ROPE, generator=g).to(dt).cuda()
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    cache = torch.zeros(pool, 16, L + ROPE, dtype=dt, device="cuda")
    q = torch.zeros(rows, H, L + ROPE, dtype=dt, device="cuda")
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pa.pa_latent_append(cache, down[:, :L], down[:, L:], bt.cuda(), i32([rows]), ws, cs.cuda(), query=q,
                        query_rope=rope.cuda().transpose(0, 1), q_start=i32([0, rows]))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    assert near(q.cpu()[..., L:], turn(rope.transpose(0, 1).double(), cs, False), dt)
    assert (q[..., :L] == 0).all()


# ---------------------------------------------------------------------------
# Bounds from a case's own data, where the parity bar says little: few keys that
# carry the result, scores of +-1000, f16.

def rounding_bound(c, ref):
    """What rounding may do to c's outputs (ref, in 64 bits), by output.

    Scores: 36 MMAs of 16 products, two roundings each at most, of terms that add up to T:
    72 of 2^-23 T with those after it, so below 2^-16 T; that moves weights against each
    other by a factor of exp(+-2 2^-16 T).  Weights are rounded to the type, u = eps / 2
    (f16: or 2^-32 of the largest, the smallest number against weights that start at 2^7),
    the sum taking them as rounded.  Sums: fp32, fewer than 2^7 additions a share, of which
    two roundings each.  The output: half a step of its type."""
    u = torch.finfo(c.dtype).eps / 2
    kvs, out, row = c.cache.double(), torch.zeros_like(ref), 0
    for s, (n, L) in enumerate(zip(c.new, c.lens)):
        t = torch.arange(L)
        kv = kvs[c.bt[s, t // c.bs].long(), t % c.bs]
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                row += 1
                continue
            q = c.q[row].double()
            p = torch.softmax(q @ kv[:m].T * c.scale, -1)
            T = (q.abs() @ kv[:m].abs().T * abs(c.scale)).amax(-1)
            off = torch.stack([(p[h, :, None] * (kv[:m, :c.L] - ref[row, h]).abs()).sum(0) for h in range(c.H)])
            far = torch.stack([(kv[:m, :c.L] - ref[row, h]).abs().amax(0) for h in range(c.H)])
            tiny = p.amax(-1, keepdim=True) * (m * 2.0 ** -32 if c.dtype == torch.float16 else 0.0) * far
            out[row] = (u * 1.01 + torch.expm1(2 * 2 ** -16 * T)[:, None]) * off + tiny + 2 ** -16 * (p @ kv[:m, :c.L].abs())
            row += 1
    return out + u * (ref.abs() + out) + 2 ** -25


def lose_newest(c):
    """The case's exact outputs without each sequence's newest key."""
    d = object.__new__(Attend)
    d.__dict__.update(c.__dict__)
    d.lens = [max(L - 1, 0) for L in c.lens]
    return d.reference()


def far_case(dtype, qmult, L=512, seed=31):
    """Every other head looks for the newest key."""
    c = Attend(seed, dtype, 16, L, 16, [900, 40, 33])
    for s, n in enumerate(c.lens):
        c.q[s, ::2] = c.cache[c.bt[s, (n - 1) // 16].long(), (n - 1) % 16]
    c.q = (c.q.double() * qmult).to(dtype)
    return c


@pytest.mark.parametrize("qmult", [1.0, 8.0, 60.0])
def test_bounds_notice_what_is_lost(qmult):
    """Zeros, and outputs without the newest key, leave the bound (an oracle's mistake)."""
    for dtype in (torch.bfloat16, torch.float16):
        c = far_case(dtype, qmult)
        ref = c.reference()
        tol = rounding_bound(c, ref)
        assert (ref.abs() > tol).double().mean() > 0.75
        assert ((lose_newest(c) - ref).abs() > tol)[:, ::2].any(-1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("qmult,L", [(1.0, 512), (8.0, 512), (60.0, 512), (60.0, 256)])
def test_far_scores_within_rounding(dtype, qmult, L):
    c = far_case(dtype, qmult, L).device()
    ref = c.reference()
    err = (c.run().double().cpu() - ref).abs()
    assert (err <= rounding_bound(c, ref)).all(), float((err - rounding_bound(c, ref)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L,bs,new", [(16, 512, 16, None), (128, 512, 64, None), (24, 256, 8, [5, 1, 17]),
                                        (16, 512, 32, [5, 1, 64])])
def test_within_rounding(dtype, H, L, bs, new):
    c = Attend(32, dtype, H, L, bs, [700, 33, 150], new).device()
    ref = c.reference()
    err = (c.run().double().cpu() - ref).abs()
    assert (err <= rounding_bound(c, ref)).all(), float((err - rounding_bound(c, ref)).max())


# ---------------------------------------------------------------------------
# Appends and attention together, captured; streams; what the appends' tests left out

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,L", [(torch.bfloat16, 20, 256), (torch.float16, 80, 512)])
def test_append_and_attend_as_graphs(dtype, H, L):
    """A prompt, then decode steps and draft chunks of which some tokens are taken back, each
    an append and the attention behind it: captured once and replayed as the lengths grow,
    beside the same calls one by one on a cache of their own.  Every output against 64 bits
    over the rows that the cache then holds."""
    bs, B, scale = 16, 3, 0.06
    g = torch.Generator().manual_seed(51)
    rng = random.Random(52)
    lens, width = [37, 5, 90], 9
    caches = [torch.zeros(B * width, bs, L + ROPE, dtype=dtype, device="cuda") for _ in range(2)]
    bt = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    ang = torch.arange(width * bs, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    w = (1 + 0.2 * torch.randn(L, generator=g)).to(dtype).cuda()
    ws = pa.alloc_latent_workspace(L)

    class Step:
        def __init__(self, new, chunks):
            self.new, n = new, sum(new)
            self.down = torch.zeros(n, L + ROPE, dtype=dtype, device="cuda")
            self.rope = torch.zeros(n, H, ROPE, dtype=dtype, device="cuda")
            self.q = torch.zeros(n, H, L + ROPE, dtype=dtype, device="cuda")
            self.sl = torch.zeros(B, dtype=torch.int32, device="cuda")
            starts = [sum(new[:i]) for i in range(B + 1)]
            self.qs = torch.tensor(starts, dtype=torch.int32, device="cuda") if chunks else None
            self.out = torch.zeros(n, H, L, dtype=dtype, device="cuda")

        def calls(self, cache):
            pa.pa_latent_append(cache, self.down[:, :L], self.down[:, L:], bt, self.sl, ws, cs, query=self.q,
                                query_rope=self.rope, norm_weight=w, eps=1e-6, q_start=self.qs)
            pa.pa_latent_forward(self.out, self.q, cache, bt, self.sl, scale, ws, q_start=self.qs)

        def fill(self):
            for t in (self.down, self.rope, self.q):
                t.copy_(torch.randn(t.shape, generator=g))
            self.sl.copy_(torch.tensor(lens))

        def check(self):
            row = 0
            for s, (n, m) in enumerate(zip(self.new, lens)):
                t = torch.arange(m, device="cuda")
                kv = caches[0][bt[s, t // bs].long(), t % bs].double()
                for i in range(m - n + 1, m + 1):
                    ref = torch.softmax(self.q[row].double() @ kv[:i].T * scale, -1) @ kv[:i, :L]
                    assert ((self.out[row].double() - ref).abs() <= ATOL + RTOL * ref.abs()).all()
                    row += 1

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        prompt = Step(list(lens), True)
        prompt.fill()
        for cache in caches:
            prompt.calls(cache)
        prompt.check()
        kinds = [Step([1] * B, False), Step([3, 1, 2], True)]
        graphs = []
        for k in kinds:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                k.calls(caches[0])
            graphs.append(graph)
        for i in range(8):
            k = kinds[i % 2]
            lens = [a + b for a, b in zip(lens, k.new)]
            k.fill()
            graphs[i % 2].replay()
            got = [t.clone() for t in (k.out, k.q)]
            k.check()
            k.calls(caches[1])
            assert all(torch.equal(a, b) for a, b in zip(got, (k.out, k.q)))
            assert torch.equal(*caches)
            if i % 2:  # drafts that were not right: their places are written again
                lens = [a - rng.randint(0, b - 1) for a, b in zip(lens, k.new)]
        assert pa.pa_read_device_status(ws) == pa.PA_OK


@pytest.mark.gpu
def test_two_streams_bit_by_bit():
    """A workspace each: every call gives the bits that it gives alone."""
    a = Attend(10, torch.bfloat16, 128, 512, 16, [3000, 5, 700]).device()
    b = Attend(11, torch.bfloat16, 12, 512, 8, [44, 900], [7, 3]).device()
    alone = [c.run().clone() for c in (a, b)]
    outs = [torch.empty_like(x) for x in alone]
    s2 = torch.cuda.Stream()
    for _ in range(20):
        for o in outs:
            o.fill_(7.0)
        s2.wait_stream(torch.cuda.current_stream())
        b.run(stream=s2, out=outs[1])
        a.run(out=outs[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, alone))


def append_rows(dtype, L, rows, lens, bt, cache, down, cs, w=None, eps=0.0, positions=None):
    """Rows of one sequence appended by the call; what the cache should hold of them, in 64 bits."""
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    d = down.cuda()
    pa.pa_latent_append(cache, d[:, :L], d[:, L:], bt.cuda(), i32(lens), ws, cs.cuda(), norm_weight=None if w is None else w.cuda(),
                        eps=eps, positions=positions, q_start=i32([0, rows]))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    x = down.double()
    c = x[:, :L]
    if w is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps) * w.double()
    at = torch.arange(lens[0] - rows, lens[0]) if positions is None else positions.cpu().long()
    return torch.cat([c, turn(x[:, None, L:], cs[at], False)[:, 0]], -1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("L", [256, 512])
def test_append_rows_near_zero(dtype, L):
    """Rows whose mean square is far below eps, and of zeros: the root is eps's."""
    g = torch.Generator().manual_seed(42)
    rows = 40
    down = torch.randn(rows, L + ROPE, generator=g)
    down[:, :L] *= 10.0 ** -torch.linspace(0, 4, rows)[:, None]
    down[7, :L] = 0.0
    down, w = down.to(dtype), (1 + 0.2 * torch.randn(L, generator=g)).to(dtype)
    bt, pool = tables([rows], 16, g)
    cache = torch.zeros(pool, 16, L + ROPE, dtype=dtype, device="cuda")
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    ref = append_rows(dtype, L, rows, [rows], bt, cache, down, cs, w, 1e-5)
    t = torch.arange(rows)
    got = cache.cpu()[bt[0, t // 16].long(), t % 16]
    for r in range(rows):  # (each row's bound by its own size)
        assert near(got[r, :L], ref[r, :L], dtype) and near(got[r, L:], ref[r, L:], dtype)
    assert (got[7, :L] == 0).all()


@pytest.mark.gpu
def test_append_positions():
    """Positions of the caller's: the keys' angles, not their places."""
    g = torch.Generator().manual_seed(43)
    rows, L, dtype = 50, 512, torch.bfloat16
    down = torch.randn(rows, L + ROPE, generator=g).to(dtype)
    bt, pool = tables([rows + 30], 16, g)
    cache = torch.zeros(pool, 16, L + ROPE, dtype=dtype, device="cuda")
    ang = torch.arange(700, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, 700, (rows,), generator=g).to(torch.int32).cuda()
    ref = append_rows(dtype, L, rows, [rows + 30], bt, cache, down, cs, positions=pos)
    t = torch.arange(30, rows + 30)
    assert near(cache.cpu()[bt[0, t // 16].long(), t % 16], ref, dtype)


@pytest.mark.gpu
def test_append_far_pages():
    """Pages beyond 2^31 elements and 2^32 bytes; nothing else is written."""
    L, bs, nb, dtype, rows = 512, 64, 70000, torch.bfloat16, 100
    g = torch.Generator().manual_seed(44)
    cache = torch.zeros(nb, bs, L + ROPE, dtype=dtype, device="cuda")
    down = torch.randn(rows, L + ROPE, generator=g).to(dtype)
    bt = torch.tensor([[nb - 1, nb - 9]], dtype=torch.int32)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    ref = append_rows(dtype, L, rows, [rows], bt, cache, down, cs)
    t = torch.arange(rows)
    assert near(cache[bt[0, t // bs].long().cuda(), (t % bs).cuda()].cpu(), ref, dtype)
    for p in bt[0].tolist():
        cache[p] = 0.0
    assert not cache.any()


@pytest.mark.gpu
def test_first_start_is_zero():
    """Rows before the first chunk are nobody's: reported, and left as they were."""
    c = Attend(34, torch.bfloat16, 20, 512, 16, [100, 40], [3, 2], pad=2).device()
    ref = c.reference()
    c.qs += 2
    c.a[0].copy_(c.a[0].roll(2, 0))
    out = c.run().double().cpu()
    assert pa.pa_read_device_status(c.ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    assert (out[:2] == 7.0).all()
    assert ((out[2:7] - ref[:5]).abs() <= ATOL + RTOL * ref[:5].abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("top", [1e4, 1e7, 1e8, 1e9])
def test_weights_stay_in_range_however_far_the_scores(dtype, top):
    """Scores near `top`, rising by a few units a key, where fp32's spacing is up to 64:
    latents that are all 3 come back as 3, as no weight passes the type's largest."""
    c = Attend(45, dtype, 16, 256, 16, [900, 77, 2000], scale=top / 2.0 ** 22)
    c.q.zero_()
    c.cache[..., :256] = 3.0
    c.q[..., 256], c.q[..., 257] = 2.0 ** 11, min(12 / c.scale / 2000, 6e4)
    for sign in (1.0, -1.0):
        for s, n in enumerate(c.lens):
            t = torch.arange(n)
            c.cache[c.bt[s, t // 16].long(), t % 16, 256] = sign * 2.0 ** 11
            c.cache[c.bt[s, t // 16].long(), t % 16, 257] = t.to(dtype)
            c.cache[c.bt[s, t // 16].long(), t % 16, 258:] = 0.0
        out = c.device().run().double()
        assert ((out - 3.0).abs() <= 3 * (torch.finfo(dtype).eps / 2 + 2 ** -16)).all()
