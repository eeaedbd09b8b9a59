"""pa_q4_append and pa_q4_forward: a cache in 4 bits against its definition in 64
bits (the codes bit by bit against the definition's own 32-bit operations), their
refusals (CPU) and their reports of bad data."""
import math
import random

import pytest
import torch

import paged_decode_attention_v2_gb300 as pa

FAKE = 1 << 20  # aligned, never dereferenced by the host checks

APPEND = dict(key_cache=FAKE, value_cache=FAKE, key_scales=FAKE, value_scales=FAKE, query_out=FAKE + 4096,
              key_out=FAKE, value_out=FAKE, query=FAKE, key=FAKE, value=FAKE, query_stride=1280,
              key_stride=1280, value_stride=1280, cos_sin=FAKE, positions=FAKE, block_tables=FAKE,
              seq_lens=FAKE, q_start=FAKE, num_seqs=2, num_rows=5, num_heads=8, num_kv_heads=1,
              head_size=128, num_blocks=64, block_size=16, max_blocks_per_seq=8, max_seq_len=128,
              rotary_dim=128, interleaved=0, max_position=200, dtype=pa.PA_DTYPE_BF16, workspace=FAKE,
              workspace_bytes=256, stream=0)
FORWARD = dict(out=FAKE, query=FAKE, key_cache=FAKE, value_cache=FAKE, key_scales=FAKE,
               value_scales=FAKE, block_tables=FAKE, seq_lens=FAKE, q_start=FAKE, num_seqs=2,
               num_rows=5, num_heads=8, num_kv_heads=1, head_size=128, num_blocks=64, block_size=16,
               max_blocks_per_seq=8, max_seq_len=128, scale=0.1, dtype=pa.PA_DTYPE_BF16,
               workspace=FAKE, workspace_bytes=1 << 40, stream=0)

# The parity bar of the framework's 16-bit calls, for values of deviation 1: a
# weight is off by f16's half step (2^-11 of it), so an output by at most 2^-11 of
# the spread of the values (8: 4e-3), and rounded to the type (2^-8 of it, below 1e-2).
ATOL, RTOL = 4e-3, 1e-2


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return pa.load_library()


@pytest.mark.parametrize("over,status", [
    (dict(key_cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(value_scales=0), pa.PA_ERR_INVALID_ARG),
    (dict(value=0), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(query_out=0), pa.PA_ERR_INVALID_ARG),
    (dict(query=0), pa.PA_ERR_INVALID_ARG),
    (dict(cos_sin=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_position=0), pa.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=24), pa.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=144), pa.PA_ERR_INVALID_ARG),
    (dict(interleaved=2), pa.PA_ERR_INVALID_ARG),
    (dict(key_scales=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(key_out=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(q_start=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 128), pa.PA_ERR_INVALID_ARG),
    (dict(key_stride=1284), pa.PA_ERR_INVALID_ARG),
    (dict(value_stride=120), pa.PA_ERR_INVALID_ARG),
    (dict(query_out=FAKE), pa.PA_ERR_INVALID_ARG),         # in place with another stride
    (dict(q_start=0), pa.PA_ERR_INVALID_ARG),              # one row a sequence, 5 rows for 2
    (dict(num_rows=-1), pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=9, num_kv_heads=2), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=pa.PA_DTYPE_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(head_size=96), pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=12, max_seq_len=96), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=17), pa.PA_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=255), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_append_refusals(lib, over, status):
    assert lib.pa_q4_append(*dict(APPEND, **over).values()) == status


@pytest.mark.parametrize("over,status", [
    (dict(out=0), pa.PA_ERR_INVALID_ARG),
    (dict(key_scales=0), pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(value_cache=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(q_start=0), pa.PA_ERR_INVALID_ARG),
    (dict(scale=math.inf), pa.PA_ERR_INVALID_ARG),
    (dict(num_seqs=-1), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=9), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=pa.PA_DTYPE_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(head_size=512), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=32), pa.PA_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 28, max_seq_len=(1 << 30) + 1), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=4096), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_forward_refusals(lib, over, status):
    assert lib.pa_q4_forward(*dict(FORWARD, **over).values()) == status


def test_no_rows_is_no_work(lib):
    a = dict(APPEND, num_rows=0, key=0, value=0, query=0, query_out=0, positions=0)
    assert lib.pa_q4_append(*a.values()) == pa.PA_OK
    assert lib.pa_q4_forward(*dict(FORWARD, num_rows=0, query=0, out=0).values()) == pa.PA_OK
    assert lib.pa_q4_forward(*dict(FORWARD, num_seqs=0, q_start=0, num_rows=0).values()) == pa.PA_OK


def test_workspace_sizes(lib):
    assert pa.pa_q4_workspace_bytes(96) == 0
    sizes = [pa.pa_q4_workspace_bytes(d) for d in (64, 128, 256)]
    assert 0 < sizes[0] < sizes[1] < sizes[2] and all(n % 256 == 0 for n in sizes)


def test_packed_calls(lib):
    """pa_call's words reach the call in order, and an int beyond 32 bits is refused."""
    pack = pa._Q4_APPEND[1]
    assert lib.pa_call(0, pack(*dict(APPEND, num_rows=0).values())) == pa.PA_OK
    assert lib.pa_call(0, pack(*dict(APPEND, workspace_bytes=255).values())) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert lib.pa_call(0, pack(*dict(APPEND, num_rows=1 << 32).values())) == pa.PA_ERR_INVALID_ARG
    pack = pa._Q4_FORWARD[1]
    assert lib.pa_call(1, pack(*dict(FORWARD, scale=math.nan).values())) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_call(1, pack(*dict(FORWARD, workspace_bytes=1).values())) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert lib.pa_call(99, pack(*FORWARD.values())) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_call(1, None) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    codes = torch.zeros(4, 1, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(4, 1, 16, 1, 2, dtype=torch.float16)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.pa_q4_append(codes, codes, scales, scales, x, x, i.view(1, 1), i, w)
    with pytest.raises(ValueError):
        pa.pa_q4_forward(x, x, codes, codes, scales, scales, i.view(1, 1), i, 1.0, w)


# ---------------------------------------------------------------------------

def quantise(x):
    """(codes, scales, values) of x [..., D] in fp32, each operation rounded by itself."""
    y = x.float().unflatten(-1, (-1, 64))
    lo = y.amin(-1, keepdim=True).clamp(-65504.0, 65504.0).half()
    step = ((y.amax(-1, keepdim=True) - lo.float()) * torch.tensor(1.0 / 15.0)).clamp(0.0, 65504.0).half()
    inv = torch.where(step > 0, torch.tensor(1.0) / step.float(), torch.tensor(0.0))
    q = torch.round((y - lo.float()) * inv).clamp(0.0, 15.0)
    c = q.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([lo, step], -1), (lo.float() + q * step.float()).flatten(-2)


def values(codes, scales):
    """What codes and scales stand for, in 64 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double().unflatten(-1, (-1, 64))
    return (scales[..., :1].double() + c * scales[..., 1:].double()).flatten(-2)


def rotate(x, cs, R, il):
    """x [rows, heads, D] in x's type (32 or 64 bits), cs [rows, R]."""
    y = x.clone()
    if R:
        c, s = cs[:, None, :R // 2].to(x.dtype), cs[:, None, R // 2:].to(x.dtype)
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if il else (x[..., :R // 2], x[..., R // 2:R])
        u, v = a * c - b * s, b * c + a * s
        if il:
            y[..., 0:R:2], y[..., 1:R:2] = u, v
        else:
            y[..., :R // 2], y[..., R // 2:R] = u, v
    return y


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


class Append:
    def __init__(self, seed, dtype, H, K, D, bs, new, ctx, R, il=False, decode=False, pad=0, mult=2.0):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, K=K, D=D, bs=bs, new=new, R=R, il=il, decode=decode)
        self.lens = [n + c for n, c in zip(new, ctx)]
        self.bt, pool = tables(self.lens, bs, g)
        rows = sum(new)
        self.total = rows + pad
        self.qkv = (torch.randn(max(self.total, 1), (H + 2 * K) * D, generator=g) * mult).to(dtype)[:self.total]
        self.codes = [torch.randint(0, 256, (pool, K, bs, D // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.randn(pool, K, bs, D // 64, 2, generator=g).half() for _ in range(2)]
        self.place, self.qs = [], [0]
        for s, (n, L) in enumerate(zip(new, self.lens)):
            self.place += [(s, t) for t in range(L - n, L)]
            self.qs.append(self.qs[-1] + n)
        top = max(self.lens + [1])
        ang = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, max(R, 2), 2) / max(R, 2))
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float() if R else None

    def run(self, query=True, in_place=False, ws=None):
        d = "cuda"
        H, K, D = self.H, self.K, self.D
        qkv = self.qkv.to(d)
        q = qkv[:, :H * D].view(-1, H, D)
        if in_place:
            q = q.contiguous()
        k, v = (qkv[:, a * D:b * D].view(-1, K, D) for a, b in ((H, H + K), (H + K, H + 2 * K)))
        self.dev = dict(codes=[c.to(d) for c in self.codes], scales=[c.to(d) for c in self.scales],
                        qo=q if in_place else torch.full((self.total, H, D), 7.0, dtype=self.dtype, device=d),
                        ko=torch.full((self.total, K, D), 7.0, dtype=self.dtype, device=d),
                        vo=torch.full((self.total, K, D), 7.0, dtype=self.dtype, device=d))
        x = self.dev
        ws = ws if ws is not None else pa.alloc_workspace(1, 1, 64, 0, 64)
        pa.pa_q4_append(*x["codes"], *x["scales"], k, v, self.bt.to(d), torch.tensor(self.lens, dtype=torch.int32, device=d),
                        ws, query=q if query else None, query_out=x["qo"] if query else None, key_out=x["ko"],
                        value_out=x["vo"], cos_sin=self.cs.to(d) if self.cs is not None else None,
                        q_start=None if self.decode else torch.tensor(self.qs, dtype=torch.int32, device=d),
                        rotary_dim=self.R, interleaved=self.il)
        assert pa.pa_read_device_status(ws) == pa.PA_OK

    def check(self, query=True):
        H, K, D, R = self.H, self.K, self.D, self.R
        rows = len(self.place)
        cs = self.cs[[t for _, t in self.place]] if self.cs is not None else None
        x = self.qkv[:rows]
        kq = x[:, H * D:(H + K) * D].view(rows, K, D)
        key = rotate(kq.float(), cs, R, self.il).to(self.dtype)
        val = x[:, (H + K) * D:].view(rows, K, D)
        names = (("ko", key), ("vo", val))
        for i, (name, want) in enumerate(names):
            codes, scales, back = quantise(want)
            ec, es = self.codes[i].clone(), self.scales[i].clone()
            for r, (s, t) in enumerate(self.place):
                p, o = int(self.bt[s, t // self.bs]), t % self.bs
                ec[p, :, o], es[p, :, o] = codes[r], scales[r]
            assert torch.equal(self.dev["codes"][i].cpu(), ec)
            assert torch.equal(self.dev["scales"][i].cpu(), es)
            got = self.dev[name].cpu()
            assert torch.equal(got[:rows], back.to(self.dtype))
            assert (got[rows:] == 7.0).all()  # padding rows
            # in 64 bits: a value is off by half a step, by what the scales' rounding to
            # f16 moves (2^-11 of the lowest value and of 15 steps), and by the key's
            # rounding to its type (which is what is coded)
            exact = rotate(kq.double(), cs, R, self.il) if name == "ko" else want.double()
            step = scales[..., 1:].double().expand(*scales.shape[:-1], 64).flatten(-2)
            lo = scales[..., :1].double().abs().expand(*scales.shape[:-1], 64).flatten(-2)
            err = (values(codes, scales) - exact).abs()
            u = torch.finfo(self.dtype).eps / 2
            assert (err <= step / 2 + 2 ** -11 * (lo + 15 * step) + 1.01 * u * exact.abs() + 2 ** -24).all()
        if query:
            q = rotate(x[:, :H * D].view(rows, H, D).float(), cs, R, self.il).to(self.dtype)
            got = self.dev["qo"].cpu()
            assert torch.equal(got[:rows], q)
            if got.data_ptr() != self.qkv.data_ptr() and len(got) > rows:
                assert (got[rows:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,K,D,bs,R,il", [
    (4, 1, 64, 8, 64, False), (8, 2, 128, 16, 128, False), (8, 2, 128, 16, 64, True), (3, 1, 256, 32, 256, True),
    (16, 4, 128, 64, 0, False), (5, 5, 64, 16, 16, False), (16, 1, 256, 8, 112, False), (8, 8, 128, 32, 96, True)])
def test_append_chunks(dtype, H, K, D, bs, R, il):
    c = Append(1, dtype, H, K, D, bs, [5, 0, 1, 33, 2], [0, 7, 15, 3, 60], R, il, pad=3)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3, 200])
def test_append_decode(B):
    rng = random.Random(B)
    c = Append(2, torch.bfloat16, 8, 2, 128, 16, [1] * B, [rng.randint(0, 90) for _ in range(B)], 128, decode=True)
    c.run()
    c.check()


@pytest.mark.gpu
def test_append_many_rows_and_in_place():
    c = Append(3, torch.bfloat16, 8, 2, 128, 16, [700, 1, 900], [5, 0, 11], 128)
    c.run(in_place=True)
    c.check()
    c = Append(4, torch.float16, 2, 1, 64, 8, [3], [9], 0)
    c.run(query=False)
    c.check(query=False)


@pytest.mark.gpu
def test_append_groups_at_the_edges():
    """Groups of one value, of infinities, of NaN, of f16's and the type's largest."""
    D, K = 64, 6
    c = Append(5, torch.bfloat16, K, K, D, 16, [1], [4], 0)
    x = c.qkv.view(3, K, D)
    x[1] = torch.randn(K, D).to(c.dtype)
    for v in (1, 2):
        x[v, 0] = 3.25                 # a step of 0
        x[v, 1, 5] = float("inf")
        x[v, 2, 7] = float("-inf")
        x[v, 3, 9] = float("nan")      # coded as the lowest
        x[v, 4] = float("nan")         # no number at all: zeros
        x[v, 5] = torch.linspace(-3e38, 3e38, D).to(c.dtype)
    c.run()
    for i, name in enumerate(("ko", "vo")):
        codes, scales = c.dev["codes"][i].cpu(), c.dev["scales"][i].cpu()
        p, o = int(c.bt[0, 0]), 4
        cd, sc = codes[p, :, o], scales[p, :, o, 0]
        got = values(cd, scales[p, :, o])
        assert torch.isfinite(sc).all() and torch.isfinite(got).all()
        assert (got[0] == 3.25).all() and sc[0, 1] == 0
        assert sc[1, 1] == 65504 and got[1, 5] >= 65504
        assert sc[2, 0] == -65504 and got[2, 7] == -65504
        src = x[1 + i, 3].double()
        fine = ~torch.isnan(src)
        assert got[3, 9] == sc[3, 0].double()
        assert (got[3][fine] - src[fine]).abs().max() <= sc[3, 1] / 2 + 1e-2
        assert (got[4] == 0).all()
        assert sc[5, 0] == -65504 and sc[5, 1] == 65504
        assert torch.equal(c.dev[name].cpu()[0], got.to(c.dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "length", "chunk", "position"])
def test_append_bad_data(what):
    c = Append(6, torch.bfloat16, 2, 1, 64, 16, [2, 3], [20, 1], 64)
    ref = [t.clone() for t in c.codes]
    # (starts 0, 4, 3: a chunk of sequence 0, and one that ends before it starts)
    own = c.bt[0, :2].long() if what != "chunk" else c.bt[1, :1].long()
    if what == "page":
        c.bt[0, 1] = 1000
    elif what == "length":
        c.lens[0] = 10 ** 6
    elif what == "chunk":
        c.qs = [0, 4, 3]
    else:
        c.cs = c.cs[:3]
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    with pytest.raises(AssertionError):
        c.run(ws=ws)
    got = c.dev["codes"][0].cpu()
    # the sequence's pages are as they were
    assert torch.equal(got[own], ref[0][own])
    assert pa.pa_read_device_status(ws) == pa.PA_OK  # (reported once)


# ---------------------------------------------------------------------------

class Attend:
    def __init__(self, seed, dtype, H, K, D, bs, lens, new=None, pad=0, qmult=1.0, vmult=1.0, offset=0.0):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, K=K, D=D, bs=bs, lens=lens, scale=1 / math.sqrt(D))
        self.new = new if new is not None else [1] * len(lens)
        self.chunks = new is not None
        self.bt, pool = tables(lens, bs, g)
        rows = sum(self.new)
        self.rows = rows
        self.q = (torch.randn(rows + pad, H, D, generator=g) * qmult).to(dtype)
        self.kc, self.ks, _ = quantise(torch.randn(pool, K, bs, D, generator=g) * 2 + offset)
        self.vc, self.vs, _ = quantise(torch.randn(pool, K, bs, D, generator=g) * vmult)
        # places that no sequence holds: anything, NaN and infinite scales too
        held = torch.zeros(pool, bs, dtype=torch.bool)
        for s, L in enumerate(lens):
            for t in range(max(L, 0)):
                held[self.bt[s, t // bs].long(), t % bs] = True
        for sc in (self.ks, self.vs):
            sc.permute(0, 2, 1, 3, 4)[~held] = float("nan")

    def reference(self):
        G = self.H // self.K
        k, v = values(self.kc, self.ks), values(self.vc, self.vs)
        out = torch.full((len(self.q), self.H, self.D), 7.0, dtype=torch.float64)
        row = 0
        for s, (n, L) in enumerate(zip(self.new, self.lens)):
            t = torch.arange(L)
            kk = k[self.bt[s, t // self.bs].long(), :, t % self.bs]
            vv = v[self.bt[s, t // self.bs].long(), :, t % self.bs]
            for i in range(n):
                m = L - n + i + 1
                for h in range(self.K):
                    q = self.q[row, h * G:(h + 1) * G].double()
                    o = torch.softmax(q @ kk[:m, h].T * self.scale, -1) @ vv[:m, h] if m > 0 else 0.0
                    out[row, h * G:(h + 1) * G] = o
                row += 1
        return out

    def device(self):
        d = "cuda"
        self.a = [t.to(d) for t in (self.q, self.kc, self.vc, self.ks, self.vs, self.bt,
                                    torch.tensor(self.lens, dtype=torch.int32))]
        qs = [0]
        for n in self.new:
            qs.append(qs[-1] + n)
        self.qs = torch.tensor(qs, dtype=torch.int32, device=d) if self.chunks else None
        self.ws = pa.alloc_q4_workspace(self.D)
        return self

    def run(self, ws=None, out=None, stream=None):
        out = torch.full_like(self.a[0], 7.0) if out is None else out
        pa.pa_q4_forward(out, *self.a, self.scale, self.ws if ws is None else ws, q_start=self.qs, stream=stream)
        return out

    def check(self, out, atol=ATOL, rtol=RTOL):
        ref = self.reference()
        err = (out.double().cpu() - ref).abs()
        assert (err <= atol + rtol * ref.abs()).all(), float((err - rtol * ref.abs()).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,K,D,bs", [(8, 1, 64, 8), (8, 2, 128, 16), (4, 4, 128, 8), (7, 1, 256, 32), (32, 2, 64, 64),
                                      (16, 1, 128, 16), (26, 2, 256, 16), (3, 1, 128, 64), (24, 2, 128, 32)])
def test_decode(dtype, H, K, D, bs):
    c = Attend(1, dtype, H, K, D, bs, [0, 1, 7, 8, 9, 31, 32, 33, 63, 64, 65, 200, 0, 517]).device()
    c.check(c.run())
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,K,D,bs", [(8, 1, 64, 8), (8, 2, 128, 16), (4, 4, 128, 8), (7, 1, 256, 32), (16, 1, 128, 64)])
def test_chunks(dtype, H, K, D, bs):
    c = Attend(2, dtype, H, K, D, bs, [5, 40, 33, 1, 300, 64], [5, 0, 3, 1, 20, 17], pad=3).device()
    c.check(c.run())  # (rows behind the last sequence stay 7)
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[20000], [9000, 3, 12000], [300] * 700])
def test_long_and_many(lens):
    """Units over hundreds of shares (joined by CTAs), and more sequences than the plan keeps."""
    c = Attend(3, torch.bfloat16, 4, 2, 64, 16, lens).device()
    c.check(c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("D,new", [(64, False), (128, False), (256, False), (128, True)])
@pytest.mark.parametrize("lens", [[1] * 900 + [7000] + [2] * 40, [33, 6000] + [5] * 200, [16] * 3, [40, 31]])
def test_short_beside_long(D, new, lens):
    """Shares that hold many whole units, parts of one, or end where a unit begins."""
    lens = lens if len(lens) < 300 or D == 64 else lens[600:]
    c = Attend(8, torch.bfloat16, 4, 2, D, 16, lens, [min(L, 3) for L in lens] if new else None).device()
    out = c.run()
    c.check(out)
    assert torch.equal(out, c.run())  # whoever takes which share


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_are_rounded_against_the_middle_code(dtype):
    """Values that are all 0, as code 7 above a lowest value of -28: weights that are off
    by 2^-11 of themselves may give what they give half a code from the middle, not seven."""
    c = Attend(9, dtype, 32, 2, 128, 16, [2, 3, 5, 40])
    c.vc[:] = 0x77
    c.vs[..., 0], c.vs[..., 1] = -28.0, 4.0
    out = c.device().run()
    # (and fp32's 2^-24 of terms up to 60, a few of them)
    assert out.double().abs().max() <= 4 * 0.5 * 2 ** -11 + 60 * 2 ** -22


@pytest.mark.gpu
def test_peaked_and_far_scores():
    """Weights that one token has alone, scores of +-1000, keys far from zero, and no
    keys' spread at all: half the weight of the type's rounding, no overflow."""
    for kw in (dict(qmult=30.0), dict(qmult=200.0), dict(offset=50.0), dict(qmult=0.0)):
        for dtype in (torch.bfloat16, torch.float16):
            c = Attend(4, dtype, 8, 2, 128, 16, [900, 40, 1], **kw).device()
            ref = c.reference()
            out = c.run().double().cpu()
            # scores of magnitude X are off by fp32's 2^-24 a term and the sum of 256:
            # X 2^-16 at most, and the output by that times the spread of the values
            X = float((c.q.double().abs().amax() * c.D * 8 + 1) * c.scale * (60 if "offset" in kw else 1))
            assert ((out - ref).abs() <= ATOL + X * 2 ** -16 * 8 + RTOL * ref.abs()).all(), kw


@pytest.mark.gpu
def test_values_of_any_magnitude():
    """Steps from f16's smallest to its largest: weights neither overflow nor vanish."""
    for mult in (1e-6, 1e-3, 1.0, 2000.0):
        for dtype in (torch.bfloat16, torch.float16):
            c = Attend(5, dtype, 8, 2, 128, 16, [700, 33], vmult=mult).device()
            # (f16's subnormal steps: the scales' own spacing, 2^-24)
            c.check(c.run(), atol=ATOL * mult + 2 ** -24, rtol=RTOL)
    # one group's steps far above another's in the same head
    c = Attend(6, torch.bfloat16, 8, 2, 128, 16, [700, 33])
    c.vs[..., 1, :] *= 1000.0
    c.device()
    ref, out = c.reference(), c.run().double().cpu()
    err = (out - ref).abs()
    assert (err[..., :64] <= ATOL + RTOL * ref[..., :64].abs()).all()
    assert (err[..., 64:] <= 1000 * ATOL + RTOL * ref[..., 64:].abs()).all()


@pytest.mark.gpu
def test_constant_values_come_back():
    """A step of 0 stands for the lowest value whatever the weights are."""
    c = Attend(7, torch.float16, 4, 1, 64, 8, [77, 1, 300])
    c.vs[..., 0], c.vs[..., 1], c.vc[:] = 1.5, 0.0, 0
    c.device()
    out = c.run()
    assert (out.float() - 1.5).abs().max() <= 2 ** -10


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["page", "length", "negative", "chunk", "rows"])
def test_bad_data(what):
    c = Attend(8, torch.bfloat16, 8, 2, 128, 16, [100, 40, 70], None if what in ("page", "length", "negative") else [3, 2, 4])
    c.device()
    ref = c.reference()
    q, kc, vc, ks, vs, bt, sl = c.a
    if what == "page":
        bt[1, 1] = 10 ** 6
    elif what == "length":
        sl[1] = 10 ** 6
    elif what == "negative":
        sl[1] = -5
    elif what == "chunk":
        c.qs = torch.tensor([0, 3, 2, 9], dtype=torch.int32, device="cuda")
    else:
        c.qs = torch.tensor([0, 3, 5, 99], dtype=torch.int32, device="cuda")
    out = c.run().double().cpu()
    assert pa.pa_read_device_status(c.ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    # (starts 0, 3, 2, 9: row 2 is sequence 0's and sequence 2's at once)
    good = [0, 2] if len(out) == 3 else [0, 1] if what == "chunk" else [0, 1, 2]
    for r in good:
        assert ((out[r] - ref[r]).abs() <= ATOL + RTOL * ref[r].abs()).all()
    if what in ("length", "negative"):
        assert (out[1] == 0).all()
    # the workspace serves the next call
    d = Attend(9, torch.bfloat16, 8, 2, 128, 16, [50]).device()
    d.check(d.run(ws=c.ws))
    assert pa.pa_read_device_status(c.ws) == pa.PA_OK


@pytest.mark.gpu
def test_graph_shared_workspace_and_streams():
    """Two captured calls of different shapes on one workspace, replayed in turn; two
    streams with a workspace each."""
    a = Attend(10, torch.bfloat16, 8, 2, 128, 16, [3000, 5, 700]).device()
    b = Attend(11, torch.bfloat16, 16, 1, 128, 8, [44, 900], [7, 3]).device()
    oa, ob = torch.zeros_like(a.a[0]), torch.zeros_like(b.a[0])
    side = torch.cuda.Stream()
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
    for _ in range(20):
        oa.fill_(0.0)
        torch.cuda.current_stream().synchronize()
        x = a.run(out=oa)
        y = b.run(stream=s2)
    torch.cuda.synchronize()
    a.check(x)
    b.check(y)


@pytest.mark.gpu
def test_far_pages():
    """Pages whose codes lie beyond 2^32 bytes and 2^31 elements."""
    D, K, bs = 128, 8, 64
    nb = 150000
    codes = [torch.empty(nb, K, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(nb, K, bs, D // 64, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
    ws = pa.alloc_q4_workspace(D)
    bt = torch.tensor([[nb - 1, 3], [nb // 2, nb - 2]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([100, 65], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(165, K, D, generator=g).bfloat16().cuda() for _ in range(2))
    qs = torch.tensor([0, 100, 165], dtype=torch.int32, device="cuda")
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pa.pa_q4_append(*codes, *scales, k, v, bt, sl, ws, key_out=ko, value_out=vo, q_start=qs)
    q = torch.randn(2, 2 * K, D, generator=g).bfloat16().cuda()
    out = torch.empty_like(q)
    pa.pa_q4_forward(out, q, *codes, *scales, bt, sl, D ** -0.5, ws)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    for s, (a, b) in enumerate(((0, 100), (100, 165))):
        kk = quantise(k[a:b].cpu())[2].double().transpose(0, 1).repeat_interleave(2, 0)
        vv = quantise(v[a:b].cpu())[2].double().transpose(0, 1).repeat_interleave(2, 0)
        x = torch.softmax(torch.einsum("hd,htd->ht", q[s].double().cpu(), kk) * D ** -0.5, -1)
        ref = torch.einsum("ht,htd->hd", x, vv)
        assert ((out[s].double().cpu() - ref).abs() <= ATOL + RTOL * ref.abs()).all()


@pytest.mark.gpu
def test_decode_loop():
    """A prompt, then tokens one by one: appended and attended to, against attention in 64
    bits over the values that the appends gave back."""
    H, K, D, bs, dt = 8, 2, 128, 16, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    prompt, steps = [37, 5], 20
    B = len(prompt)
    top = max(prompt) + steps
    width = -(-top // bs)
    kc, ks = pa.alloc_q4_cache(B * width, K, bs, D)
    vc, vs = pa.alloc_q4_cache(B * width, K, bs, D)
    bt = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    ang = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    ws = pa.alloc_q4_workspace(D)
    held = [([], []) for _ in range(B)]

    def step(new, lens, qs):
        rows = sum(new)
        qkv = torch.randn(rows, (H + 2 * K) * D, generator=g).to(dt).cuda()
        q, k, v = qkv[:, :H * D].view(rows, H, D), qkv[:, H * D:(H + K) * D].view(rows, K, D), qkv[:, (H + K) * D:].view(rows, K, D)
        qo, ko, vo = torch.empty(rows, H, D, dtype=dt, device="cuda"), torch.empty(rows, K, D, dtype=dt, device="cuda"), torch.empty(rows, K, D, dtype=dt, device="cuda")
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        pa.pa_q4_append(kc, vc, ks, vs, k, v, bt, sl, ws, query=q, query_out=qo, key_out=ko, value_out=vo, cos_sin=cs, q_start=qs)
        out = torch.empty_like(qo)
        pa.pa_q4_forward(out, qo, kc, vc, ks, vs, bt, sl, D ** -0.5, ws, q_start=qs)
        row = 0
        for s, n in enumerate(new):
            for i in range(n):
                held[s][0].append(ko[row + i].double().cpu())
                held[s][1].append(vo[row + i].double().cpu())
            kk, vv = (torch.stack(x) for x in held[s])
            for i in range(n):
                m = len(kk) - n + i + 1
                x = torch.softmax(torch.einsum("kgd,tkd->kgt", qo[row].double().cpu().view(K, H // K, D), kk[:m]) * D ** -0.5, -1)
                ref = torch.einsum("kgt,tkd->kgd", x, vv[:m]).reshape(H, D)
                # (key_out and value_out are rounded once more, to bf16: 2^-8 of a key moves a
                # score by at most 2^-8 |q||k| scale, some 0.1, and a value by 2^-8 of it)
                assert (out[row].double().cpu() - ref).abs().max() <= 0.1 * 2 + 2 ** -7
                row += 1

    step(prompt, prompt, torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32, device="cuda"))
    for t in range(1, steps + 1):
        step([1] * B, [p + t for p in prompt], None)
    assert pa.pa_read_device_status(ws) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_weights(dtype, D):
    """Weights of 2^-26 beside one of 1, every 64 keys, whose values make up for it: f16's
    smallest number is 2^-24.  A weight is off by 2^-32 of the largest at most, 63 of them
    by that times 7.5 x 4096 about the middle code.  The middle of the key of weight 1, 7.5 x
    4096 above its value of 0, goes into an fp32 sum, rounded to 2^-24 of it, and out of it by
    an MMA, whose terms are cut at 2^-23 of the largest, one each: below 2^-21 of it together."""
    c = Attend(20, dtype, 4, 1, D, 16, [640, 65, 3000])
    c.scale = 1.0
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.kc.zero_(), c.vc.fill_(0xff)
    c.ks[..., 0], c.ks[..., 1] = -18.25, 0.0
    c.vs[..., 0], c.vs[..., 1] = 0.0, 4096.0
    for s, L in enumerate(c.lens):
        for t in range(0, L, 64):
            p, o = int(c.bt[s, t // 16]), t % 16
            c.ks[p, :, o, :, 0], c.vc[p, :, o] = 0.0, 0
    ref = c.reference()
    assert (ref > 0.02).all()
    err = (c.device().run().double().cpu() - ref).abs()
    u = torch.finfo(dtype).eps / 2
    middle = 7.5 * 4096
    assert (err <= (63 * 2 ** -32 + 2 ** -21) * middle + (2 ** -11 + u + 2 ** -20) * ref).all(), float(err.max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_steps_far_below_the_heads_largest(dtype):
    """One group's steps are 2^-23.4 of another's: a weight of 1 times that is 1.5 of f16's
    smallest, and 192 of them at 2^7, half of one off."""
    c = Attend(23, dtype, 8, 2, 128, 16, [1, 1, 40, 300], qmult=0.0)
    c.vs[..., 0, 0], c.vs[..., 0, 1], c.vs[..., 1, 0], c.vs[..., 1, 1] = 0.0, 65504.0, 0.0, 1.5 * 2 ** -8
    c.vc[..., :32] = 0
    ref = c.reference()
    err = (c.device().run().double().cpu() - ref).abs()
    u = torch.finfo(dtype).eps / 2
    assert (err <= (0.5 / 190 + 2 ** -20) * 7.5 * 1.5 * 2 ** -8 + u * ref + 2 ** -24).all(), float(err.max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_negative_steps(dtype, D):
    """lowest + code step of a step below zero, in some groups, tokens or all."""
    c = Attend(24, dtype, 8, 2, D, 16, [200, 33, 1])
    g = torch.Generator().manual_seed(25)
    for sc in (c.ks, c.vs):
        sign = 1 - 2 * torch.randint(0, 2, sc.shape[:-1], generator=g)
        sign[c.bt[2, 0].long()] = -1
        sc[..., 1] *= sign
    c.check(c.device().run())


# ---------------------------------------------------------------------------
# Bounds from a case's own data, where the parity bar says little: few keys that
# carry the result, scores of +-1000, f16.

def rounding_bound(c, ref):
    """What rounding may do to c's outputs (ref, in 64 bits), by output.

    Scores: fp32 sums of terms that add up to T at most, T = scale sum |q| (|lo| + 15
    |step|): 18 additions of q a group, 16 MMAs a head of two roundings each, ten more:
    60 of 2^-24 T, so below 2^-18 T.  That moves weights against each other by a factor
    of exp(+-2 2^-18 T).  Weights times steps are rounded to f16 and meet codes about
    their middle: 2^-11 sum p |code - 7.5| step, or 2^-32 of the largest p x step a key
    where that is more (the smallest f16 against weights that start at 2^7).  Sums: fp32,
    fewer than 2^7 additions one behind another a share.  The output: half a step of its
    type."""
    u = torch.finfo(c.dtype).eps / 2
    G, NG = c.H // c.K, c.D // 64
    k, v = values(c.kc, c.ks), values(c.vc, c.vs)
    reach = (c.ks[..., 0].double().abs() + 15 * c.ks[..., 1].double().abs()).repeat_interleave(64, -1)
    step = c.vs[..., 1].double().abs()
    mid = (v - (c.vs[..., 0].double() + 7.5 * c.vs[..., 1].double()).repeat_interleave(64, -1)).abs()
    size = (c.vs[..., 0].double().abs() + 15 * step).repeat_interleave(64, -1)
    out, row = torch.zeros_like(ref), 0
    for s, (n, L) in enumerate(zip(c.new, c.lens)):
        t = torch.arange(L)
        kk, vv, rr, st, md, sz = (x[c.bt[s, t // c.bs].long(), :, t % c.bs] for x in (k, v, reach, step, mid, size))
        for i in range(n):
            m = L - n + i + 1
            if m <= 0:
                row += 1
                continue
            for h in range(c.K):
                at = slice(h * G, (h + 1) * G)
                q = c.q[row, at].double()
                p = torch.softmax(q @ kk[:m, h].T * c.scale, -1)
                T = (q.abs() @ rr[:m, h].T * abs(c.scale)).amax(-1)
                o = ref[row, at]
                spread = torch.stack([(p[g, :, None] * (vv[:m, h] - o[g]).abs()).sum(0) for g in range(G)])
                tiny = (p * st[:m, h].amax(-1)).amax(-1) * (m * 7.5 * 2 ** -32)
                e = torch.expm1(2 * 2 ** -18 * T)[:, None] * spread + 2 ** -11 * 1.01 * (p @ md[:m, h])
                out[row, at] = e + tiny[:, None] + 2 ** -16 * (p @ sz[:m, h])
            row += 1
    return out + u * (ref.abs() + out) + 2 ** -25


def lose_newest(c):
    """The case's exact outputs without each sequence's newest key."""
    d = object.__new__(Attend)
    d.__dict__.update(c.__dict__)
    d.kc, d.ks = c.kc.clone(), c.ks.clone()
    d.lens = [max(L - 1, 0) for L in c.lens]
    return d.reference()


def far_case(dtype, kind, seed=21):
    """Scores of +-1000, or keys far from zero; every other head looks for the newest key."""
    c = Attend(seed, dtype, 8, 2, 128, 16, [900, 40, 33], offset=50.0 if kind == "offset" else 0.0)
    k = values(c.kc, c.ks)
    for s, L in enumerate(c.lens):
        last = k[c.bt[s, (L - 1) // 16].long(), :, (L - 1) % 16]
        last = (last - (50.0 if kind == "offset" else 0.0)).repeat_interleave(4, 0)
        c.q[s, ::2] = last[::2].to(dtype)
    c.q = (c.q.double() * {"peaked": 30.0, "far": 200.0, "offset": 1.0}[kind]).to(dtype)
    return c


@pytest.mark.parametrize("kind", ["peaked", "far", "offset"])
def test_bounds_notice_what_is_lost(kind):
    """Zeros, and outputs without the newest key, leave the bound (an oracle's mistake)."""
    for dtype in (torch.bfloat16, torch.float16):
        c = far_case(dtype, kind)
        ref = c.reference()
        tol = rounding_bound(c, ref)
        assert (ref.abs() > tol).double().mean() > 0.75
        assert ((lose_newest(c) - ref).abs() > tol)[:, ::2].any(-1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["peaked", "far", "offset"])
def test_far_scores_within_rounding(dtype, kind):
    c = far_case(dtype, kind).device()
    ref = c.reference()
    err = (c.run().double().cpu() - ref).abs()
    assert (err <= rounding_bound(c, ref)).all(), float((err - rounding_bound(c, ref)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,K,D,bs,new", [(8, 2, 128, 16, None), (16, 1, 64, 8, None), (7, 1, 256, 32, [5, 1, 17]),
                                          (8, 1, 128, 64, [5, 1, 64])])
def test_within_rounding(dtype, H, K, D, bs, new):
    c = Attend(22, dtype, H, K, D, bs, [700, 33, 150], new).device()
    ref = c.reference()
    err = (c.run().double().cpu() - ref).abs()
    assert (err <= rounding_bound(c, ref)).all(), float((err - rounding_bound(c, ref)).max())


# ---------------------------------------------------------------------------
# Appends and attention together, captured; streams; positions of the caller's

def attend_in_64_bits(q, kc, vc, ks, vs, bt, lens, new, bs):
    """[rows, H, D]: over what the cache holds, gathered from its codes and scales."""
    k, v = values(kc.cpu(), ks.cpu()), values(vc.cpu(), vs.cpu())
    q, bt = q.double().cpu(), bt.cpu()
    K, D = k.shape[1], k.shape[3]
    out = []
    for s, (n, L) in enumerate(zip(new, lens)):
        t = torch.arange(L)
        kk, vv = (x[bt[s, t // bs].long(), :, t % bs] for x in (k, v))
        for m in range(L - n + 1, L + 1):
            x = torch.einsum("kgd,tkd->kgt", q[len(out)].view(K, -1, D), kk[:m]) * D ** -0.5
            out.append(torch.einsum("kgt,tkd->kgd", torch.softmax(x, -1), vv[:m]).reshape(-1, D))
    return torch.stack(out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_and_attend_as_graphs(dtype):
    """A prompt, then decode steps and draft chunks of which some tokens are taken back, each
    an append and the attention behind it: captured once and replayed as the lengths grow,
    beside the same calls one by one on a cache of their own.  Every output against 64 bits
    over the codes and scales that the cache then holds."""
    H, K, D, bs, B = 8, 2, 128, 16, 3
    g = torch.Generator().manual_seed(51)
    rng = random.Random(52)
    lens, width = [37, 5, 90], 9
    caches = []
    for _ in range(2):
        (kc, ks), (vc, vs) = (pa.alloc_q4_cache(B * width, K, bs, D) for _ in range(2))
        caches.append((kc, vc, ks, vs))
    bt = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    ang = torch.arange(width * bs, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    ws = pa.alloc_q4_workspace(D)

    class Step:
        def __init__(self, new, chunks):
            self.new, n = new, sum(new)
            self.qkv = torch.zeros(n, (H + 2 * K) * D, dtype=dtype, device="cuda")
            self.sl = torch.zeros(B, dtype=torch.int32, device="cuda")
            starts = [sum(new[:i]) for i in range(B + 1)]
            self.qs = torch.tensor(starts, dtype=torch.int32, device="cuda") if chunks else None
            self.qo, self.out = (torch.zeros(n, H, D, dtype=dtype, device="cuda") for _ in range(2))

        def calls(self, cache):
            n = len(self.qkv)
            q, k, v = (self.qkv[:, a * D:b * D].view(n, -1, D) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
            pa.pa_q4_append(*cache, k, v, bt, self.sl, ws, query=q, query_out=self.qo, cos_sin=cs, q_start=self.qs)
            pa.pa_q4_forward(self.out, self.qo, *cache, bt, self.sl, D ** -0.5, ws, q_start=self.qs)

        def fill(self):
            self.qkv.copy_(torch.randn(self.qkv.shape, generator=g))
            self.sl.copy_(torch.tensor(lens))

        def check(self):
            kc, vc, ks, vs = caches[0]
            ref = attend_in_64_bits(self.qo, kc, vc, ks, vs, bt, lens, self.new, bs)
            assert ((self.out.double().cpu() - ref).abs() <= ATOL + RTOL * ref.abs()).all()

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
            got = [t.clone() for t in (k.out, k.qo)]
            k.check()
            k.calls(caches[1])
            assert all(torch.equal(a, b) for a, b in zip(got, (k.out, k.qo)))
            assert all(torch.equal(a, b) for a, b in zip(*caches))
            if i % 2:  # drafts that were not right: their places are written again
                lens = [a - rng.randint(0, b - 1) for a, b in zip(lens, k.new)]
        assert pa.pa_read_device_status(ws) == pa.PA_OK


@pytest.mark.gpu
def test_two_streams_bit_by_bit():
    """A workspace each: every call gives the bits that it gives alone."""
    a = Attend(10, torch.bfloat16, 8, 2, 128, 16, [3000, 5, 700]).device()
    b = Attend(11, torch.bfloat16, 16, 1, 128, 8, [44, 900], [7, 3]).device()
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


@pytest.mark.gpu
@pytest.mark.parametrize("decode", [False, True])
def test_append_positions(decode):
    """Positions of the caller's: the keys' and queries' angles, not their places."""
    new = [1] * 4 if decode else [5, 0, 33, 2]
    c = Append(26, torch.bfloat16, 8, 2, 128, 16, new, [3, 7, 15, 60], 128, decode=decode)
    rows, top = sum(new), 500
    ang = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, 128, 2) / 128)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, top, (rows,), generator=torch.Generator().manual_seed(27)).to(torch.int32)
    d, H, K, D = "cuda", c.H, c.K, c.D
    qkv = c.qkv.to(d)
    q, k, v = (qkv[:, a * D:b * D].view(rows, -1, D) for a, b in ((0, H), (H, H + K), (H + K, H + 2 * K)))
    c.dev = dict(codes=[x.to(d) for x in c.codes], scales=[x.to(d) for x in c.scales],
                 qo=torch.empty(rows, H, D, dtype=c.dtype, device=d), ko=torch.empty(rows, K, D, dtype=c.dtype, device=d),
                 vo=torch.empty(rows, K, D, dtype=c.dtype, device=d))
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    pa.pa_q4_append(*c.dev["codes"], *c.dev["scales"], k, v, c.bt.to(d), torch.tensor(c.lens, dtype=torch.int32, device=d), ws,
                    query=q, query_out=c.dev["qo"], key_out=c.dev["ko"], value_out=c.dev["vo"], cos_sin=cs.to(d),
                    positions=pos.to(d), q_start=None if decode else torch.tensor(c.qs, dtype=torch.int32, device=d))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    x, at = c.qkv, cs[pos.long()]
    key = rotate(x[:, H * D:(H + K) * D].view(rows, K, D).float(), at, 128, False).to(c.dtype)
    assert torch.equal(c.dev["qo"].cpu(), rotate(x[:, :H * D].view(rows, H, D).float(), at, 128, False).to(c.dtype))
    for i, want in enumerate((key, x[:, (H + K) * D:].view(rows, K, D))):
        codes, scales, _ = quantise(want)
        for r, (s, t) in enumerate(c.place):
            p, o = int(c.bt[s, t // 16]), t % 16
            assert torch.equal(c.dev["codes"][i][p, :, o].cpu(), codes[r])
            assert torch.equal(c.dev["scales"][i][p, :, o].cpu(), scales[r])


@pytest.mark.gpu
def test_first_start_is_zero():
    """Rows before the first chunk are nobody's: reported, and left as they were."""
    c = Attend(28, torch.bfloat16, 8, 2, 128, 16, [100, 40], [3, 2], pad=2).device()
    ref = c.reference()
    c.qs += 2
    c.a[0].copy_(c.a[0].roll(2, 0))
    out = c.run().double().cpu()
    assert pa.pa_read_device_status(c.ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    assert (out[:2] == 7.0).all()
    assert ((out[2:7] - ref[:5]).abs() <= ATOL + RTOL * ref[:5].abs()).all()


@pytest.mark.parametrize("over", [dict(key_out=FAKE, value_out=0), dict(key_out=0, value_out=FAKE)])
def test_append_refuses_strided_rows_in_place(lib, over):
    """Rows written in place at another stride would be rows not yet read."""
    assert lib.pa_q4_append(*dict(APPEND, **over).values()) == pa.PA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("il", [False, True])
def test_append_gives_back_in_place(il):
    c = Append(29, torch.float16, 8, 2, 128, 16, [300, 1, 9], [5, 0, 11], 128, il)
    c.run()
    d, (H, K, D) = c.dev, (c.H, c.K, c.D)
    want = d["ko"].clone(), d["vo"].clone()
    k, v = (c.qkv[:, a * D:b * D].reshape(-1, K, D).cuda() for a, b in ((H, H + K), (H + K, H + 2 * K)))
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    before = [t.clone() for t in d["codes"] + d["scales"]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pa.pa_q4_append(*d["codes"], *d["scales"], k, v, c.bt.cuda(), i32(c.lens), ws, key_out=k, value_out=v,
                    cos_sin=c.cs.cuda(), q_start=i32(c.qs), interleaved=il)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert all(torch.equal(a, b) for a, b in zip(before, d["codes"] + d["scales"]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("top", [1e4, 1e7, 1e8, 1e9])
def test_weights_stay_in_range_however_far_the_scores(dtype, top):
    """Scores near `top`, rising by a few units a key, where fp32's spacing is up to 64: values
    that are all 3 come back as 3, as no weight passes f16's largest."""
    c = Attend(45, dtype, 4, 1, 64, 16, [900, 77, 2000])
    c.scale = 1.0
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 2.0 ** 12, 1.0
    c.kc.zero_()
    c.ks[..., 0], c.ks[..., 1] = 0.0, 0.0
    c.vc.fill_(0x11)
    c.vs[..., 0], c.vs[..., 1] = 2.0, 1.0
    for sign in (1.0, -1.0):
        c.scale = top / (2.0 ** 12 * 60000.0)
        for s, L in enumerate(c.lens):
            for t in range(L):
                # (the group's lowest value lifts elements 0 and 1 alike)
                c.ks[c.bt[s, t // 16].long(), :, t % 16, 0, 0] = sign * 60000.0
                c.ks[c.bt[s, t // 16].long(), :, t % 16, 0, 1] = 32.0
                c.kc[c.bt[s, t // 16].long(), :, t % 16, 0] = t * 16 // L
        out = c.device().run().double()
        assert ((out - 3.0).abs() <= 3 * (torch.finfo(dtype).eps / 2 + 2 ** -11)).all()
