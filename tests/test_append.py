"""pa_append_kv: new keys and values into the paged cache, rotated on the way,
with the pages' key bounds, against the formulas in 64 bits; its refusals (CPU)
and its reports of bad data."""
import math
import random

import pytest
import torch

import paged_decode_attention_v2_gb300 as pa

FAKE = 1 << 20  # aligned, never dereferenced by the host checks

BASE = dict(key_cache=FAKE, value_cache=FAKE, key_bounds=FAKE, query_out=FAKE, query=FAKE, key=FAKE,
            value=FAKE, query_stride=1280, key_stride=1280, value_stride=1280, cos_sin=FAKE,
            positions=FAKE, block_tables=FAKE, seq_lens=FAKE, q_start=FAKE, num_seqs=2, num_rows=5,
            num_heads=8, num_kv_heads=1, head_size=128, num_blocks=64, block_size=16,
            max_blocks_per_seq=8, max_seq_len=128, rotary_dim=128, interleaved=0, max_position=200,
            dtype=pa.PA_DTYPE_BF16, workspace=FAKE, workspace_bytes=256, stream=0)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return pa.load_library()


@pytest.mark.parametrize("over,status", [
    (dict(key_cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(value=0), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(query_out=0), pa.PA_ERR_INVALID_ARG),            # queries in, none out
    (dict(query=0), pa.PA_ERR_INVALID_ARG),
    (dict(cos_sin=0), pa.PA_ERR_INVALID_ARG),              # rotation without angles
    (dict(max_position=0), pa.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=24), pa.PA_ERR_INVALID_ARG),
    (dict(rotary_dim=144), pa.PA_ERR_INVALID_ARG),
    (dict(interleaved=2), pa.PA_ERR_INVALID_ARG),
    (dict(key=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(key_bounds=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(q_start=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 128), pa.PA_ERR_INVALID_ARG),
    (dict(key_stride=1284), pa.PA_ERR_INVALID_ARG),        # not a multiple of 16 bytes
    (dict(value_stride=120), pa.PA_ERR_INVALID_ARG),       # rows would overlap
    (dict(query_stride=1016), pa.PA_ERR_INVALID_ARG),
    (dict(query=FAKE, query_out=FAKE), pa.PA_ERR_INVALID_ARG),  # in place with another stride
    (dict(q_start=0), pa.PA_ERR_INVALID_ARG),              # one row a sequence, 5 rows for 2
    (dict(num_rows=-1), pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=9, num_kv_heads=2), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=7), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(head_size=96), pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=12, max_seq_len=96), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=17), pa.PA_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(query=0, query_out=0, workspace_bytes=255), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_refusals(lib, over, status):
    a = dict(BASE, query_out=FAKE + 4096)
    a.update(over)
    assert lib.pa_append_kv(*a.values()) == status


def test_no_rows_is_no_work(lib):
    a = dict(BASE, query_out=FAKE + 4096, num_rows=0)
    assert lib.pa_append_kv(*a.values()) == pa.PA_OK
    a.update(key=0, value=0, query=0, query_out=0, positions=0)  # empty tensors
    assert lib.pa_append_kv(*a.values()) == pa.PA_OK


def test_binding_refuses_host_tensors():
    kc = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_append_kv(kc, kc, x, x, i.view(1, 1), i, torch.zeros(256, dtype=torch.uint8))


# ---------------------------------------------------------------------------

class Case:
    """Ragged chunks (or one token a sequence) behind ragged contexts."""

    def __init__(self, seed, dtype, H, K, D, bs, new, ctx, R, interleaved=False, decode=False,
                 bounds=True, offsets=None, pad_rows=0):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, K=K, D=D, bs=bs, new=new, R=R, il=interleaved,
                             decode=decode)
        self.lens = [n + c for n, c in zip(new, ctx)]
        pages = [-(-L // bs) for L in self.lens]
        pool = sum(pages) + 3
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        self.bt = torch.full((len(new), max(pages + [1])), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(pages):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.rows = sum(new) if not decode else len(new)
        self.total = self.rows + pad_rows
        self.kc = torch.randn(pool, K, bs, D, generator=g).to(dtype)
        self.vc = torch.randn(pool, K, bs, D, generator=g).to(dtype)
        self.qkv = torch.randn(max(self.total, 1), (H + 2 * K) * D, generator=g).to(dtype)[:self.total]
        # (sequence, token, position) of every row
        self.place, self.qs = [], [0]
        for s, (n, L) in enumerate(zip(new, self.lens)):
            off = offsets[s] if offsets else 0
            self.place += [(s, t, t + off) for t in range(L - n, L)]
            self.qs.append(self.qs[-1] + n)
        self.positions = (torch.tensor([p[2] for p in self.place] + [10 ** 9] * pad_rows,
                                       dtype=torch.int32) if offsets else None)
        top = max([p[2] for p in self.place], default=0) + 1
        inv = 10000.0 ** (-torch.arange(0, max(R, 2), 2, dtype=torch.float64) / max(R, 2))
        ang = torch.arange(top, dtype=torch.float64)[:, None] * inv
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float() if R else None
        self.kb = None
        if bounds:
            self.kb = torch.randn(pool, K, 2, D, generator=g).to(dtype)
            for s, (n, L) in enumerate(zip(new, self.lens)):
                for j in range(-(-(L - n) // bs)):
                    k = self.kc[self.bt[s, j], :, :min(bs, L - n - j * bs)]
                    self.kb[self.bt[s, j], :, 0], self.kb[self.bt[s, j], :, 1] = k.amax(1), k.amin(1)

    def split(self, qkv):
        H, K, D = self.H, self.K, self.D
        n = qkv.shape[0]
        return (qkv[:, :H * D].view(n, H, D), qkv[:, H * D:(H + K) * D].view(n, K, D),
                qkv[:, (H + K) * D:].view(n, K, D))

    def rotate(self, x):
        """The formula in 64 bits, and the size of what its products add up."""
        x = x[:len(self.place)].double()
        y, size = x.clone(), x.abs()
        if not self.R:
            return y, size
        R = self.R
        cs = self.cs.double()[[p[2] for p in self.place]]
        for j in range(R // 2):
            a, b = (2 * j, 2 * j + 1) if self.il else (j, j + R // 2)
            c, s = cs[:, None, j], cs[:, None, R // 2 + j]
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
            size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
        return y, size

    def check(self, got, ref, size, what):
        # two products and a sum in fp32 (three roundings of at most 2^-24 of
        # the larger terms), one rounding to dtype (half a step; 2^-25 below
        # f16's normal range)
        fi = torch.finfo(self.dtype)
        bound = 4 * 2.0 ** -24 * size
        if self.dtype != torch.float32:
            bound = bound + fi.eps / 2 * (ref.abs() + bound) + (2.0 ** -25 if self.dtype == torch.float16 else 0)
        err = (got.double().cpu() - ref).abs()
        assert (err <= bound).all(), f"{what}: {(err - bound).max().item():.3e} over"

    def run_and_check(self, inplace=False, stream=None, calls=1):
        dev = "cuda"
        qkv = self.qkv.to(dev)
        q, k, v = self.split(qkv)
        if inplace:
            q = q.contiguous()
        qo = q if inplace else torch.full((self.total, self.H, self.D), 7.0, dtype=self.dtype, device=dev)
        kc, vc = self.kc.to(dev), self.vc.to(dev)
        kb = self.kb.to(dev) if self.kb is not None else None
        ws = pa.alloc_workspace(1, 1, 64, 0, 64)
        qs = None if self.decode else torch.tensor(self.qs, dtype=torch.int32, device=dev)
        sl = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        args = dict(query=q, query_out=qo, key_bounds=kb,
                    cos_sin=self.cs.to(dev) if self.R else None,
                    positions=self.positions.to(dev) if self.positions is not None else None,
                    q_start=qs, rotary_dim=self.R, interleaved=self.il,
                    max_seq_len=max(self.lens), stream=stream)
        torch.cuda.synchronize()
        for _ in range(calls):
            pa.pa_append_kv(kc, vc, k, v, self.bt.to(dev), sl, ws, **args)
        assert pa.pa_read_device_status(ws, stream) == pa.PA_OK
        torch.cuda.synchronize()
        hq, hk, hv = self.split(self.qkv)
        n = len(self.place)
        seq = torch.tensor([p[0] for p in self.place], dtype=torch.long)
        tok = torch.tensor([p[1] for p in self.place], dtype=torch.long)
        page = self.bt[seq, tok // self.bs].long()
        kref, ksize = self.rotate(hk)
        gk, gv = kc.cpu(), vc.cpu()
        self.check(gk[page, :, tok % self.bs], kref, ksize, "keys")
        assert torch.equal(gv[page, :, tok % self.bs], hv[:n])
        # every other slot of the caches is as it was
        gk[page, :, tok % self.bs] = self.kc[page, :, tok % self.bs]
        gv[page, :, tok % self.bs] = self.vc[page, :, tok % self.bs]
        assert torch.equal(gk, self.kc) and torch.equal(gv, self.vc)
        qref, qsize = self.rotate(hq)
        if not inplace:
            self.check(qo[:n], qref, qsize, "queries")
            assert (qo[n:] == 7.0).all()  # padding rows
        else:
            self.check(qo[:n], qref, qsize, "queries in place")
        if kb is not None:
            want = self.kb.clone()
            gk = kc.cpu()
            for s, (m, L) in enumerate(zip(self.new, self.lens)):
                for j in range((L - m) // self.bs, -(-L // self.bs)) if m else ():
                    kk = gk[self.bt[s, j], :, :min(self.bs, L - j * self.bs)]
                    want[self.bt[s, j], :, 0], want[self.bt[s, j], :, 1] = kk.amax(1), kk.amin(1)
            assert torch.equal(kb.cpu(), want)
        return kc


DTYPES = [torch.bfloat16, torch.float16, torch.float32]
ids = lambda v: str(v).replace("torch.", "")  # noqa: E731


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D,bs,R,il", [(64, 8, 64, False), (64, 64, 16, True), (128, 16, 128, False),
                                       (128, 32, 64, False), (128, 16, 128, True), (256, 32, 256, False),
                                       (256, 8, 128, True), (128, 16, 0, False)], ids=ids)
def test_chunks(dtype, D, bs, R, il):
    new, ctx = [1, 17, 0, 64, 3, 130, 1, 33], [0, 5, 9, 64, 16, 1, 77, 31]
    Case(1, dtype, 6, 2, D, bs, new, ctx, R, il).run_and_check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("B,H,K,D", [(1, 32, 4, 128), (37, 8, 8, 64), (700, 4, 1, 256), (1300, 5, 1, 64)], ids=ids)
def test_decode(dtype, B, H, K, D):
    rng = random.Random(B)
    ctx = [rng.choice([0, 1, 15, 16, 17, 40]) for _ in range(B)]
    Case(B, dtype, H, K, D, 16, [1] * B, ctx, D, decode=True).run_and_check()


@pytest.mark.gpu
def test_many_rows_of_many_lengths():
    """More rows than one row a CTA, pages that start anywhere in a tile."""
    rng = random.Random(5)
    new = [rng.choice([0, 1, 1, 2, 9, 16, 50, 200]) for _ in range(150)]
    ctx = [rng.randint(0, 40) for _ in new]
    for bs in (8, 64):
        Case(5, torch.bfloat16, 4, 2, 128, bs, new, ctx, 128).run_and_check()


@pytest.mark.gpu
def test_empty_slots_of_a_decode_batch():
    c = Case(9, torch.bfloat16, 4, 2, 64, 16, [1, 1, 1], [4, 0, 20], 64, decode=True)
    dev = "cuda"
    q, k, v = c.split(c.qkv.to(dev))
    kc, vc, kb = c.kc.to(dev), c.vc.to(dev), c.kb.to(dev)
    qo = torch.full((3, 4, 64), 7.0, dtype=c.dtype, device=dev)
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    sl = torch.tensor([5, 0, 21], dtype=torch.int32, device=dev)
    pa.pa_append_kv(kc, vc, k, v, c.bt.to(dev), sl, ws, query=q, query_out=qo, key_bounds=kb,
                    cos_sin=c.cs.to(dev))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    assert (qo[1] == 7.0).all() and not (qo[0] == 7.0).all()
    p = int(c.bt[1, 0])
    assert torch.equal(kc[p].cpu(), c.kc[p]) and torch.equal(kb[p].cpu(), c.kb[p])


@pytest.mark.gpu
def test_positions_padding_rows_and_in_place():
    new, ctx = [3, 1, 40], [10, 0, 3]
    Case(11, torch.float16, 3, 1, 128, 16, new, ctx, 64, offsets=[500, 0, 77], pad_rows=9).run_and_check()
    Case(12, torch.bfloat16, 4, 2, 128, 16, new, ctx, 128).run_and_check(inplace=True)


@pytest.mark.gpu
def test_repeated_and_on_another_stream():
    s = torch.cuda.Stream()
    c = Case(13, torch.bfloat16, 4, 2, 128, 16, [5, 30], [3, 0], 128)
    with torch.cuda.stream(s):
        c.run_and_check(stream=s, calls=2)  # the same tokens again: the same cache and bounds


@pytest.mark.gpu
def test_infinite_keys_and_nan():
    """Infinities pass through and bound their page; a NaN key is stored, its bounds skip it."""
    c = Case(14, torch.bfloat16, 2, 1, 64, 16, [4], [0], 0)
    q, k, v = c.split(c.qkv)
    k[0, 0, 3], k[1, 0, 3], k[2, 0, 5], v[0, 0, 0] = math.inf, -math.inf, math.nan, math.nan
    dev = "cuda"
    kc, vc, kb = c.kc.to(dev), c.vc.to(dev), c.kb.to(dev)
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    qkv = c.qkv.to(dev)
    _, kd, vd = c.split(qkv)
    pa.pa_append_kv(kc, vc, kd, vd, c.bt.to(dev), torch.tensor([4], dtype=torch.int32, device=dev), ws,
                    key_bounds=kb, q_start=torch.tensor([0, 4], dtype=torch.int32, device=dev))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    p = int(c.bt[0, 0])
    assert torch.equal(kc[p, :, :4].cpu().nan_to_num(9.0), k.transpose(0, 1).nan_to_num(9.0))
    assert kb[p, 0, 0, 3] == math.inf and kb[p, 0, 1, 3] == -math.inf
    rest = k[[0, 1, 3], 0, 5]
    assert kb[p, 0, 0, 5].item() == rest.max().item() and kb[p, 0, 1, 5].item() == rest.min().item()


@pytest.mark.gpu
def test_starts_that_decrease_out_of_any_rows_sight_are_reported():
    """Every row finds a chunk that holds it, but the chunks overlap."""
    c = Case(16, torch.bfloat16, 2, 1, 64, 16, [4, 3, 3], [10, 10, 10], 64, offsets=[0, 0, 0])
    dev = "cuda"
    q, k, v = c.split(c.qkv.to(dev))
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    for qs, status in (([0, 4, 7, 10], pa.PA_OK), ([0, 6, 4, 10], pa.PA_ERR_DEVICE_BAD_INPUT)):
        pa.pa_append_kv(c.kc.to(dev), c.vc.to(dev), k, v, c.bt.to(dev),
                        torch.tensor(c.lens, dtype=torch.int32, device=dev), ws, cos_sin=c.cs.to(dev),
                        q_start=torch.tensor(qs, dtype=torch.int32, device=dev))
        assert pa.pa_read_device_status(ws) == status


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["block", "length", "negative", "chunk", "position", "rows", "order"])
def test_bad_data_is_reported(what):
    """Each is found by the kernel's own checks before an address is formed; the
    other sequence's rows are appended as usual."""
    c = Case(15, torch.bfloat16, 2, 1, 64, 16, [4, 6], [3, 20], 64, offsets=[0, 0])
    dev = "cuda"
    bt, lens, qs, pos = c.bt.clone(), list(c.lens), list(c.qs), c.positions.clone()
    if what == "block":
        bt[0, 0] = c.kc.shape[0]
    elif what == "length":
        lens[0] = 10 ** 6
    elif what == "negative":
        lens[0] = -3
    elif what == "chunk":
        lens[0] = 2
    elif what == "position":
        pos[2] = c.cs.shape[0]
    elif what == "rows":
        qs = [0, 4, 11]
    elif what == "order":
        qs = [0, 12, 10]
    kc, vc, kb = c.kc.to(dev), c.vc.to(dev), c.kb.to(dev)
    q, k, v = c.split(c.qkv.to(dev))
    qo = torch.full((10, 2, 64), 7.0, dtype=c.dtype, device=dev)
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    pa.pa_append_kv(kc, vc, k, v, bt.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), ws,
                    query=q, query_out=qo, key_bounds=kb, cos_sin=c.cs.to(dev), positions=pos.to(dev),
                    q_start=torch.tensor(qs, dtype=torch.int32, device=dev), max_seq_len=32)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    p0, p1 = int(c.bt[0, 0]), int(c.bt[1, 1])
    if what in ("block", "length", "negative", "chunk"):
        assert torch.equal(kc[p0].cpu(), c.kc[p0])
    if what not in ("rows", "order"):
        ref, size = c.rotate(c.split(c.qkv)[1])
        c.check(kc[p1, :, 4:10].cpu().transpose(0, 1), ref[4:], size[4:], "the other sequence")
    if what == "position":
        assert (qo[2] == 7.0).all() and torch.equal(kc[p0, :, 5].cpu(), c.kc[p0, :, 5])


@pytest.mark.gpu
def test_captured_and_replayed_with_new_lengths():
    """One captured launch serves later steps: lengths, tables and rows are read
    from the device each time, for a batch padded to its largest size."""
    dev, D, bs, K = "cuda", 64, 16, 2
    kc = torch.zeros(8, K, bs, D, dtype=torch.bfloat16, device=dev)
    vc, kb = torch.zeros_like(kc), torch.zeros(8, K, 2, D, dtype=torch.bfloat16, device=dev)
    x = torch.zeros(6, 2 * K * D, dtype=torch.bfloat16, device=dev)
    k, v = x[:, :K * D].view(6, K, D), x[:, K * D:].view(6, K, D)
    bt = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=dev)
    sl = torch.tensor([3, 1], dtype=torch.int32, device=dev)
    qs = torch.tensor([0, 3, 4], dtype=torch.int32, device=dev)
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pa.pa_append_kv(kc, vc, k, v, bt, sl, ws, key_bounds=kb, q_start=qs)
    s.synchronize()
    with torch.cuda.graph(g):
        pa.pa_append_kv(kc, vc, k, v, bt, sl, ws, key_bounds=kb, q_start=qs)
    want = torch.zeros_like(kc)
    lens = [0, 0]
    for step, new in enumerate([(3, 1), (0, 6), (5, 0), (1, 1)]):
        gen = torch.Generator(device=dev).manual_seed(step)
        x.copy_(torch.randn(x.shape, generator=gen, device=dev))
        row = 0
        for i, n in enumerate(new):
            for _ in range(n):
                want[bt[i, lens[i] // bs], :, lens[i] % bs] = k[row]
                row, lens[i] = row + 1, lens[i] + 1
        sl.copy_(torch.tensor(lens))
        qs.copy_(torch.tensor([0, new[0], sum(new)]))
        g.replay()
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    assert torch.equal(kc, want)
    for i in range(2):
        n = min(lens[i], bs)
        page = kc[bt[i, 0].long(), :, :n]
        assert torch.equal(kb[bt[i, 0].long(), :, 0], page.amax(1))
        assert torch.equal(kb[bt[i, 0].long(), :, 1], page.amin(1))


@pytest.mark.gpu
def test_cache_beyond_32_bits():
    """Pages at the end of caches of more than 2^32 bytes."""
    c = Case(16, torch.bfloat16, 4, 4, 128, 16, [40], [9], 128)
    dev, blocks = "cuda", 300_000
    pages = c.bt[0].long()
    far = torch.arange(blocks - len(pages), blocks)
    kc = torch.empty(blocks, 4, 16, 128, dtype=c.dtype, device=dev)
    vc, kb = torch.empty_like(kc), torch.empty(blocks, 4, 2, 128, dtype=c.dtype, device=dev)
    for t, s in ((kc, c.kc), (vc, c.vc), (kb, c.kb)):
        t[far.cuda()] = s[pages].cuda()
    q, k, v = c.split(c.qkv.to(dev))
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    pa.pa_append_kv(kc, vc, k, v, far.to(torch.int32)[None].cuda(),
                    torch.tensor([49], dtype=torch.int32, device=dev), ws, key_bounds=kb,
                    cos_sin=c.cs.to(dev), q_start=torch.tensor([0, 40], dtype=torch.int32, device=dev))
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    tok = torch.arange(9, 49)
    ref, size = c.rotate(c.split(c.qkv)[1])
    got = kc[far[tok // 16].cuda(), :, (tok % 16).cuda()].cpu()
    c.check(got, ref, size, "far keys")
    assert torch.equal(vc[far[tok // 16].cuda(), :, (tok % 16).cuda()].cpu(), c.split(c.qkv)[2])
    for j, page in enumerate(far.tolist()):
        held = kc[page, :, :min(16, 49 - 16 * j)]
        assert torch.equal(kb[page, :, 0], held.amax(1)) and torch.equal(kb[page, :, 1], held.amin(1))


@pytest.mark.gpu
@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "inplace"])
@pytest.mark.parametrize("decode", [False, True], ids=["chunks", "decode"])
def test_rows_of_a_bad_page_keep_their_queries(inplace, decode):
    """Nothing of a row whose table entry is bad is written: its query too stays
    as it was, where the rotation would replace it; the other rows are as usual."""
    new, ctx = ([1] * 6, [3, 20, 40, 15, 16, 0]) if decode else ([4, 20], [3, 20])
    c = Case(15, torch.bfloat16, 6, 2, 64, 16, new, ctx, 64, decode=decode)
    dev = "cuda"
    bt = c.bt.clone()
    bt[0, 0] = c.kc.shape[0]  # of all rows of the first sequence
    bt[1, (32 if not decode else 20) // 16] = -5  # of the second's rows from token 32 on (its only one)
    kc, vc, kb = c.kc.to(dev), c.vc.to(dev), c.kb.to(dev)
    q, k, v = c.split(c.qkv.to(dev))
    q = q.contiguous()
    qo = q if inplace else torch.full_like(q, 7.0)
    was = qo.clone()
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    qs = None if decode else torch.tensor(c.qs, dtype=torch.int32, device=dev)
    pa.pa_append_kv(kc, vc, k, v, bt.to(dev), torch.tensor(c.lens, dtype=torch.int32, device=dev), ws,
                    query=q, query_out=qo, key_bounds=kb, cos_sin=c.cs.to(dev), q_start=qs)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    lost = [r for r, (s, t, _) in enumerate(c.place) if s == 0 or (s == 1 and (decode or t >= 32))]
    kept = [r for r in range(len(c.place)) if r not in lost]
    assert torch.equal(qo[lost], was[lost])
    ref, size = c.rotate(c.split(c.qkv)[0])
    c.check(qo[kept], ref[kept], size[kept], "the other rows")
    for s, t, _ in (c.place[r] for r in lost):  # their pages neither
        page = int(c.bt[s, t // 16])
        assert torch.equal(kc[page].cpu(), c.kc[page]) and torch.equal(vc[page].cpu(), c.vc[page])
        assert torch.equal(kb[page].cpu(), c.kb[page])


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [8, 16])
def test_bad_positions_leave_the_bounds_of_their_pages(bs):
    """A page whose appended rows all have bad positions keeps its bounds, a new
    page too; with one good row among them the bounds are that row's."""
    c = Case(17, torch.bfloat16, 2, 2, 64, bs, [9, 6, bs], [0, 20, 2 * bs], 64, offsets=[0, 0, 0])
    dev = "cuda"
    bad = [r for r, (s, t, _) in enumerate(c.place)
           if (s == 0 and t // bs == 0) or s == 1 or (s == 2 and t != 2 * bs + 3)]
    pos = c.positions.clone()
    pos[bad] = c.cs.shape[0]
    kc, vc, kb = c.kc.to(dev), c.vc.to(dev), c.kb.to(dev)
    _, k, v = c.split(c.qkv.to(dev))
    ws = pa.alloc_workspace(1, 1, 64, 0, 64)
    pa.pa_append_kv(kc, vc, k, v, c.bt.to(dev), torch.tensor(c.lens, dtype=torch.int32, device=dev), ws,
                    key_bounds=kb, cos_sin=c.cs.to(dev), positions=pos.to(dev),
                    q_start=torch.tensor(c.qs, dtype=torch.int32, device=dev))
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_DEVICE_BAD_INPUT
    kc, kb = kc.cpu(), kb.cpu()
    for s, j in [(0, 0)] + [(1, t // bs) for t in range(20, 26)]:
        page = int(c.bt[s, j])
        assert torch.equal(kb[page], c.kb[page]) and torch.equal(kc[page], c.kc[page])
    page = int(c.bt[2, 2])
    assert torch.equal(kb[page, :, 0], kc[page, :, 3]) and torch.equal(kb[page, :, 1], kc[page, :, 3])
    if bs == 8:  # the ninth token's page
        page = int(c.bt[0, 1])
        assert torch.equal(kb[page, :, 0], kc[page, :, 0]) and torch.equal(kb[page, :, 1], kc[page, :, 0])
