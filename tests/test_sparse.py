"""pa_select_blocks and pa_sparse_forward against their definition in 64 bits:
the selection is compared number for number, the attention over it within the
parity bar; refusals (CPU) and reports of bad data."""
import math
import random

import numpy as np
import pytest
import torch

import paged_decode_attention_v2_gb300 as pa
from gpu_helpers import assert_close

FAKE = 1 << 20  # aligned, never dereferenced by the host checks

BASE = dict(out=FAKE, selected=FAKE, query=FAKE, key_cache=FAKE, value_cache=FAKE, key_bounds=FAKE,
            block_tables=FAKE, seq_lens=FAKE, q_start=0, num_seqs=2, num_rows=2, num_heads=8,
            num_kv_heads=2, head_size=128, num_blocks=64, block_size=16, max_blocks_per_seq=8,
            max_seq_len=128, num_selected=4, sink_blocks=1, recent_blocks=1, scale=0.1,
            partition_size=512, dtype=pa.PA_DTYPE_BF16, workspace=FAKE, workspace_bytes=1 << 30,
            stream=0)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return pa.load_library()


REFUSALS = [
    (dict(query=0), pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=0), pa.PA_ERR_INVALID_ARG),
    (dict(num_rows=3), pa.PA_ERR_INVALID_ARG),
    (dict(num_seqs=0, q_start=FAKE), pa.PA_ERR_INVALID_ARG),
    (dict(num_selected=0), pa.PA_ERR_INVALID_ARG),
    (dict(recent_blocks=0), pa.PA_ERR_INVALID_ARG),
    (dict(sink_blocks=-1), pa.PA_ERR_INVALID_ARG),
    (dict(sink_blocks=2, recent_blocks=3), pa.PA_ERR_INVALID_ARG),
    (dict(query=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(key_bounds=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(selected=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=9), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(partition_size=0), pa.PA_ERR_INVALID_ARG),
    (dict(partition_size=100), pa.PA_ERR_UNSUPPORTED),
    (dict(head_size=80), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=34), pa.PA_ERR_UNSUPPORTED),
    (dict(num_selected=1 << 28), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=4096), pa.PA_ERR_WORKSPACE_TOO_SMALL),
]


@pytest.mark.parametrize("over,status", REFUSALS + [
    (dict(out=0), pa.PA_ERR_INVALID_ARG),
    (dict(key_cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(key_bounds=0, selected=0), pa.PA_ERR_INVALID_ARG),
    (dict(out=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(scale=math.inf), pa.PA_ERR_INVALID_ARG),
])
def test_sparse_refusals(lib, over, status):
    assert lib.pa_sparse_forward(*dict(BASE, **over).values()) == status


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 16, 2 ** 31 - 1])
def test_lengths_beyond_31_bit_arithmetic_are_refused(lib, n):
    """With a page added they could pass 2^31."""
    assert pa.pa_sparse_workspace_bytes(2, 8, 2, 128, 16, n, 4, 512) == 0
    a = dict(BASE, max_seq_len=n, max_blocks_per_seq=2 ** 31 - 1, workspace_bytes=1 << 50)
    assert lib.pa_sparse_forward(*a.values()) == pa.PA_ERR_UNSUPPORTED
    for name in ("out", "key_cache", "value_cache", "scale"):
        del a[name]
    assert lib.pa_select_blocks(*a.values()) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,status", REFUSALS + [
    (dict(selected=0), pa.PA_ERR_INVALID_ARG),
    (dict(key_bounds=0), pa.PA_ERR_INVALID_ARG),
])
def test_select_refusals(lib, over, status):
    a = dict(BASE, **over)
    for name in ("out", "key_cache", "value_cache", "scale"):
        del a[name]
    assert lib.pa_select_blocks(*a.values()) == status


def test_workspace_bytes(lib):
    f = pa.pa_sparse_workspace_bytes
    small = f(2, 8, 2, 128, 16, 128, 4, 512)
    assert small >= pa.pa_workspace_bytes(4, 4, 128, 64, 512) and small % 256 == 0
    assert f(0, 8, 2, 128, 16, 128, 4, 512) > 0
    assert f(2, 8, 3, 128, 16, 128, 4, 512) == 0 and f(2, 8, 2, 128, 16, 128, 0, 512) == 0
    assert lib.pa_sparse_forward(*dict(BASE, workspace_bytes=small - 1).values()) == \
        pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert lib.pa_sparse_forward(*dict(BASE, num_seqs=0, num_rows=0).values()) == pa.PA_OK
    assert lib.pa_sparse_forward(*dict(BASE, num_seqs=0, num_rows=0, query=0, out=0, seq_lens=0,
                                       block_tables=0, selected=0).values()) == pa.PA_OK


# ---------------------------------------------------------------------------

class Case:
    def __init__(self, seed, dtype, H, K, D, bs, lens, k, sinks=0, recent=1, chunks=None, P=256,
                 q_mult=1.0):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(dtype=dtype, H=H, K=K, D=D, bs=bs, lens=lens, k=k, sinks=sinks,
                             recent=recent, chunks=chunks, P=P, scale=1 / math.sqrt(D))
        pages = [-(-L // bs) for L in lens]
        pool = sum(pages) + 3
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        self.bt = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(pages):
            self.bt[s, :n] = perm[at:at + n]
            at += n
        self.rows = sum(chunks) if chunks else len(lens)
        self.q = (q_mult * torch.randn(self.rows, H, D, generator=g)).to(dtype)
        self.kc = (2 * torch.randn(pool, K, bs, D, generator=g)).to(dtype)
        self.vc = torch.randn(pool, K, bs, D, generator=g).to(dtype)
        self.set_bounds()

    def set_bounds(self):
        self.kb = torch.full((self.kc.shape[0], self.K, 2, self.D), math.nan, dtype=self.dtype)
        for s, L in enumerate(self.lens):
            for j in range(-(-L // self.bs)):
                k = self.kc[self.bt[s, j], :, :min(self.bs, L - j * self.bs)]
                self.kb[self.bt[s, j], :, 0], self.kb[self.bt[s, j], :, 1] = k.amax(1), k.amin(1)

    def row_list(self):
        if not self.chunks:
            return [(s, L) for s, L in enumerate(self.lens)]
        return [(s, L - n + i + 1) for s, (n, L) in enumerate(zip(self.chunks, self.lens))
                for i in range(n)]

    def select(self):
        """The definition, page by page, in 64 bits."""
        sel = torch.full((self.rows, self.K, self.k), -1, dtype=torch.int32)
        G = self.H // self.K
        for r, (s, vis) in enumerate(self.row_list()):
            n = -(-vis // self.bs)
            kb = self.kb[self.bt[s, :n].long()].double()
            for h in range(self.K):
                q = self.q[r, h * G:(h + 1) * G].double()[:, None]
                sc = torch.maximum(q * kb[:, h, 0], q * kb[:, h, 1]).sum((0, 2))
                wild = ~torch.isfinite(kb[:, h]).all(-1).all(-1)  # by the split sum: 0 inf is NaN
                split = (q.clamp_min(0).sum(0) * kb[:, h, 0] + q.clamp_max(0).sum(0) * kb[:, h, 1]).sum(-1)
                sc = torch.where(wild, split, sc)
                sc = torch.nan_to_num(sc, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
                order = sorted(range(n), key=lambda j: (not (j < self.sinks or j >= n - self.recent),
                                                        -float(sc[j]), j))
                got = sorted(order[:self.k])
                sel[r, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
        return sel

    def attend(self, sel):
        out = np.zeros((self.rows, self.H, self.D))
        G = self.H // self.K
        for r, (s, vis) in enumerate(self.row_list()):
            for h in range(self.K):
                j = sel[r, h][sel[r, h] >= 0].long()
                tok = (j[:, None] * self.bs + torch.arange(self.bs)).flatten()
                tok = tok[tok < vis]
                if len(tok) == 0:
                    continue
                pg = self.bt[s, tok // self.bs].long()
                k, v = self.kc[pg, h, tok % self.bs].double(), self.vc[pg, h, tok % self.bs].double()
                x = self.q[r, h * G:(h + 1) * G].double() @ k.T * self.scale
                out[r, h * G:(h + 1) * G] = (torch.softmax(x, -1) @ v).numpy()
        return out

    def device(self, max_seq_len=None, poison=True):
        dev = "cuda"
        m = max_seq_len if max_seq_len is not None else max(self.lens)
        qs = None
        if self.chunks:
            qs = torch.tensor([0] + list(np.cumsum(self.chunks)), dtype=torch.int32, device=dev)
        ws = pa.alloc_sparse_workspace(self.rows, self.H, self.K, self.D, self.bs, m, self.k, self.P)
        kc, vc = self.kc.clone(), self.vc.clone()
        if poison:  # what lies behind the last token is never used
            for s, L in enumerate(self.lens):
                if L % self.bs:
                    kc[self.bt[s, L // self.bs], :, L % self.bs:] = math.nan
                    vc[self.bt[s, L // self.bs], :, L % self.bs:] = math.nan
        return dict(q=self.q.to(dev), kc=kc.to(dev), vc=vc.to(dev), kb=self.kb.to(dev),
                    bt=self.bt.to(dev), sl=torch.tensor(self.lens, dtype=torch.int32, device=dev),
                    qs=qs, ws=ws, m=m,
                    sel=torch.full((self.rows, self.K, self.k), 99, dtype=torch.int32, device=dev),
                    out=torch.full((self.rows, self.H, self.D), math.nan, dtype=self.dtype, device=dev))

    def run(self, d, given=False, stream=None, with_sel=True):
        pa.pa_sparse_forward(d["out"], d["sel"] if with_sel else None, d["q"], d["kc"], d["vc"],
                             d["bt"], d["sl"], self.scale, self.P, d["ws"],
                             key_bounds=None if given else d["kb"], num_selected=self.k,
                             sink_blocks=self.sinks, recent_blocks=self.recent, q_start=d["qs"],
                             max_seq_len=d["m"], stream=stream)

    def check(self, calls=2, max_seq_len=None):
        d = self.device(max_seq_len)
        ref = self.select()
        want = self.attend(ref)
        for _ in range(calls):
            d["out"].fill_(math.nan)
            d["sel"].fill_(99)
            self.run(d)
            assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
            assert torch.equal(d["sel"].cpu(), ref)
            assert_close(d["out"], want, self.dtype, "selected blocks")
        # the selection alone, and the attention over it as given
        d["sel"].fill_(99)
        pa.pa_select_blocks(d["sel"], d["q"], d["kb"], d["bt"], d["sl"], self.bs, self.P, d["ws"],
                            sink_blocks=self.sinks, recent_blocks=self.recent, q_start=d["qs"],
                            max_seq_len=d["m"])
        assert torch.equal(d["sel"].cpu(), ref)
        again = d["out"].clone()
        d["out"].fill_(math.nan)
        self.run(d, given=True)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert torch.equal(d["out"], again)


DTYPES = [torch.bfloat16, torch.float16, torch.float32]
ids = lambda v: str(v).replace("torch.", "")  # noqa: E731


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D,bs,G,K,k,sinks,recent", [
    (128, 16, 8, 2, 8, 1, 2), (64, 8, 3, 2, 16, 0, 1), (256, 32, 4, 1, 5, 2, 3), (128, 64, 16, 1, 4, 0, 1),
    (64, 16, 1, 4, 33, 4, 1), (128, 16, 5, 1, 3, 1, 2)], ids=ids)
def test_decode(dtype, D, bs, G, K, k, sinks, recent):
    lens = [1, bs, bs + 1, 5 * bs - 1, 40 * bs + 3, 0, 90 * bs, 17, k * bs, k * bs + 1]
    Case(D + k, dtype, G * K, K, D, bs, lens, k, sinks, recent).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=ids)
def test_chunks_of_rows(dtype):
    Case(3, dtype, 8, 2, 128, 16, [700, 33, 5, 1500], 6, 1, 1, chunks=[4, 1, 5, 3]).check()


@pytest.mark.gpu
def test_long_sequences_cut_into_chunks():
    """Few rows: an item's pages are cut over several CTAs; more pages than the
    shared memory keeps (8192)."""
    Case(4, torch.bfloat16, 8, 2, 64, 8, [9000 * 8 - 3, 70], 40, 1, 2).check()
    Case(5, torch.float16, 4, 1, 64, 16, [33333], 100).check()


@pytest.mark.gpu
def test_many_rows():
    rng = random.Random(6)
    lens = [rng.randint(1, 600) for _ in range(400)]
    Case(6, torch.bfloat16, 4, 2, 64, 8, lens, 7, 0, 1).check(calls=1)


@pytest.mark.gpu
def test_equal_scores_go_to_the_lower_page():
    """Identical pages (equal scores, more of them than the list of pages scored
    again holds), in single-CTA and cut items; a zero query ties everything."""
    for lens, k in (([40 * 16, 9], 6), ([700 * 16 + 5], 9)):
        c = Case(7, torch.bfloat16, 4, 1, 64, 16, lens, k)
        c.kc[:] = c.kc[:1, :, :1]
        c.set_bounds()
        c.check()
        c = Case(8, torch.float16, 4, 1, 64, 16, lens, k, sinks=2, recent=2)
        c.q.zero_()
        c.check()
    # two kinds of pages, one better: ties inside each
    c = Case(9, torch.bfloat16, 2, 1, 128, 8, [300 * 8], 50)
    c.kc[:] = c.kc[:1, :, :1]
    even = c.bt[0, 0::3].long()
    c.kc[even] = c.q[0, 0].expand(1, 8, 128)
    c.set_bounds()
    c.check()


@pytest.mark.gpu
def test_scores_closer_than_fp32_can_tell():
    """Pages whose scores differ by the last bits of an fp32 key beside large
    common terms: the order is decided in 64 bits."""
    D, bs, n, k = 128, 8, 400, 60
    c = Case(10, torch.float32, 2, 1, D, bs, [n * bs], k)
    g = torch.Generator().manual_seed(11)
    base = 100 * torch.randn(D, generator=g)
    for j in range(n):
        c.kc[c.bt[0, j], 0, :] = base
        c.kc[c.bt[0, j], 0, :, 5] = base[5] * (1 + float(torch.randint(0, 1000, (1,), generator=g)) * 2.0 ** -23)
    c.set_bounds()
    sel = c.select()
    assert len(set(sel[0, 0].tolist()) & set(range(k - 1))) < k - 1  # not just the first pages
    d = c.device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert torch.equal(d["sel"].cpu(), sel)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_infinite_and_nan_bounds(value):
    """Pages with infinite bounds rank first or last, NaN scores last."""
    for lens in ([60 * 8], [900 * 8]):
        c = Case(12, torch.bfloat16, 2, 1, 64, 8, lens, 12)
        for j in (3, 17, 44):
            c.kb[c.bt[0, j], 0, 0, 7] = value
            c.kb[c.bt[0, j], 0, 1, 7] = value
        d = c.device()
        ref = c.select()
        c.run(d)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert torch.equal(d["sel"].cpu(), ref)


@pytest.mark.gpu
def test_nothing_to_see_and_rows_behind_the_last_chunk():
    c = Case(13, torch.bfloat16, 4, 2, 64, 16, [0, 0], 4)
    c.check()
    c.check(max_seq_len=0)
    c = Case(14, torch.bfloat16, 4, 2, 64, 16, [200, 90], 4, chunks=[2, 1])
    d = c.device()
    ref, want = c.select(), c.attend(c.select())
    pad = 2  # two rows more than the chunks hold
    for name in ("q", "out", "sel"):
        t = d[name]
        d[name] = torch.cat([t, t[:pad]])
    d["ws"] = pa.alloc_sparse_workspace(5, 4, 2, 64, 16, d["m"], 4, c.P)
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert torch.equal(d["sel"][:3].cpu(), ref) and (d["sel"][3:] == -1).all()
    assert_close(d["out"][:3], want, c.dtype, "rows of the chunks")
    assert (d["out"][3:] == 0).all()


@pytest.mark.gpu
def test_given_selections():
    c = Case(15, torch.bfloat16, 4, 2, 64, 16, [200, 90], 4)
    d = c.device()
    sel = torch.tensor([[[0, 3, 12, -1], [2, -1, -1, -1]], [[-1, -1, -1, -1], [0, 1, 2, 5]]], dtype=torch.int32)
    d["sel"].copy_(sel)
    c.run(d, given=True)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert_close(d["out"], c.attend(sel), c.dtype, "given blocks")
    assert torch.equal(d["sel"].cpu(), sel)
    for bad in ([3, 1, -1, -1], [2, 2, -1, -1], [0, -1, 1, -1], [0, 13, -1, -1], [-2, -1, -1, -1]):
        d["sel"].copy_(sel)
        d["sel"][0, 0] = torch.tensor(bad, dtype=torch.int32)
        c.run(d, given=True)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
        assert (d["out"][0, :2] == 0).all()
        assert_close(d["out"][1], c.attend(sel)[1], c.dtype, "the other row")


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["block", "length", "negative", "chunk", "order"])
def test_bad_data_is_reported(what):
    """Found by the kernels' own checks; the other sequence is served as usual."""
    c = Case(16, torch.bfloat16, 4, 2, 64, 16, [200, 300], 5, chunks=[2, 2])
    want = c.attend(c.select())
    d = c.device(max_seq_len=304)
    if what == "block":
        d["bt"][0, 4] = c.kc.shape[0]
    elif what == "length":
        d["sl"][0] = 305
    elif what == "negative":
        d["sl"][0] = -1
    elif what == "chunk":
        d["sl"][0] = 1
    else:
        d["qs"][0] = 1
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
    if what != "order":
        assert_close(d["out"][2:], want[2:], c.dtype, "the other sequence")
    pa.pa_workspace_init(d["ws"])


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream():
    c = Case(17, torch.bfloat16, 8, 2, 128, 16, [2000, 700, 90], 8, 1, 2)
    d = c.device(max_seq_len=2000)
    want = c.attend(c.select())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(d, stream=s, with_sel=False)
    s.synchronize()
    assert_close(d["out"], want, c.dtype, "another stream, selection not wanted")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(d)
    for lens in ([2000, 700, 90], [1600, 16, 33]):
        c2 = Case(17, torch.bfloat16, 8, 2, 128, 16, [2000, 700, 90], 8, 1, 2)
        c2.lens = lens
        c2.set_bounds()
        d["sl"].copy_(torch.tensor(lens))
        d["kb"].copy_(c2.kb)
        for _ in range(2):
            d["out"].fill_(math.nan)
            g.replay()
            assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
            assert torch.equal(d["sel"].cpu(), c2.select())
            assert_close(d["out"], c2.attend(c2.select()), c.dtype, f"replay {lens}")


@pytest.mark.gpu
def test_one_workspace_for_calls_of_many_shapes():
    """A workspace sized for the largest call, used by calls of other shapes in
    between (their layouts overlap each other's leftovers), on both the
    whole-item and the cut path."""
    cases = [Case(20, torch.bfloat16, 8, 2, 128, 16, [3000, 70, 5], 20, 1, 2),
             Case(21, torch.float16, 4, 1, 64, 8, [9000, 100, 33, 8, 700], 7),
             Case(22, torch.float32, 4, 2, 64, 16, [50], 2),
             Case(23, torch.bfloat16, 4, 2, 64, 8, [40 + i for i in range(320)], 3)]
    n = max(pa.pa_sparse_workspace_bytes(c.rows, c.H, c.K, c.D, c.bs, max(c.lens), c.k, c.P) for c in cases)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0  # the status block alone is initialised
    state = [(c, c.device(), c.select()) for c in cases]
    want = [c.attend(sel) for c, _, sel in state]
    for _ in range(2):
        for (c, d, sel), out in zip(state, want):
            d["ws"] = ws
            d["sel"].fill_(99)
            c.run(d)
            assert pa.pa_read_device_status(ws) == pa.PA_OK
            assert torch.equal(d["sel"].cpu(), sel)
            assert_close(d["out"], out, c.dtype, "shared workspace")


@pytest.mark.gpu
def test_cache_beyond_32_bits():
    """Pages at the end of caches of more than 2^32 bytes (and bounds of more
    than 2^31), where 32-bit element or byte offsets would wrap."""
    K, D, bs = 4, 128, 16
    blocks = 300_000  # 4.9 GB a cache, 0.6 GB of bounds
    c = Case(24, torch.bfloat16, 8, K, D, bs, [130], 4, 1, 1)
    d = c.device()
    pages = c.bt[0].long()
    far = torch.arange(blocks - len(pages), blocks)
    for name in ("kc", "vc", "kb"):
        t = torch.empty((blocks,) + tuple(d[name].shape[1:]), dtype=c.dtype, device="cuda")
        t[far.cuda()] = d[name][pages.cuda()]
        d[name] = t
    d["bt"] = far.to(torch.int32)[None].cuda()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    sel = c.select()
    assert torch.equal(d["sel"].cpu(), sel)
    assert_close(d["out"], c.attend(sel), c.dtype, "far pages")


@pytest.mark.gpu
def test_many_rows_with_long_ones_among_them():
    """Whole-item CTAs (enough items for every SM) whose pages exceed what a
    warp (256), the CTA's registers (1024) and its shared memory (8192) hold;
    the long rows read one another's pages, so that the caches stay small."""
    long = [9000, 8300, 4000, 1300, 1025, 700, 260]
    lens = [8 * n - 3 for n in long] + [1 + i % 90 for i in range(603)]
    c = Case(25, torch.bfloat16, 2, 1, 64, 8, [8 * long[0] - 3] + [90], 6, 1, 1)
    c.lens, c.rows = lens, len(lens)
    bt = c.bt[:1].expand(len(lens), -1).clone()
    bt[len(long):] = c.bt[1]
    c.bt = bt
    c.q = torch.randn(c.rows, 2, 64, generator=torch.Generator().manual_seed(26)).to(c.dtype)
    # a page's bounds for every row: those of all its tokens (a bound may be wide)
    k = c.kc.clone()
    c.kb = torch.stack([k.amax(2), k.amin(2)], 2)
    d = c.device(poison=False)
    ref = c.select()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert torch.equal(d["sel"].cpu(), ref)
    assert_close(d["out"], c.attend(ref), c.dtype, "long rows among many")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D,bs,G,K", [(64, 8, 3, 2), (128, 8, 8, 1), (256, 16, 2, 2)])
def test_long_tables_and_chunks_of_many_lengths(dtype, D, bs, G, K):
    """Chunks of no row, of one and of many; sequences that select every page
    beside long ones; a row that sees a page more than the one before it."""
    lens = [190 * bs + 1, 40, 140 * bs - 3, 30, 100 * bs + 8, 16, 21, 150 * bs]
    chunks = [5, 2, 19, 0, 16, 1, 20, 8]
    c = Case(30 + D, dtype, G * K, K, D, bs, lens, 9, 1, 2, chunks=chunks)
    c.check()
    c.check(calls=1, max_seq_len=190 * bs + 1)


@pytest.mark.gpu
def test_many_sequences_of_two_rows():
    lens = [2 + (i * 37) % 1023 for i in range(99)] + [1024]
    Case(31, torch.float16, 8, 4, 64, 8, lens, 7, 1, 1, chunks=[2] * 100).check(calls=1)


@pytest.mark.gpu
def test_padded_rows_and_bad_chunks():
    c = Case(32, torch.bfloat16, 4, 2, 64, 8, [1100, 900, 300], 6, 1, 1, chunks=[9, 3, 2])
    d = c.device()
    ref, want = c.select(), c.attend(c.select())
    for name in ("q", "out", "sel"):
        d[name] = torch.cat([d[name], d[name][:11]])
    d["ws"] = pa.alloc_sparse_workspace(25, 4, 2, 64, 8, d["m"], 6, c.P)
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert torch.equal(d["sel"][:14].cpu(), ref) and (d["sel"][14:] == -1).all()
    assert_close(d["out"][:14], want, c.dtype, "rows of the chunks")
    assert (d["out"][14:] == 0).all()
    good = d["qs"].clone()
    for bad in ([0, 9, 12, 99], [0, 12, 9, 14], [-4, 9, 12, 14], [3, 9, 12, 14], [9, 9, 9, 9]):
        d["qs"].copy_(torch.tensor(bad))
        c.run(d)
        if bad != [9, 9, 9, 9]:  # (rows in no chunk, as padding is)
            assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
        pa.pa_workspace_init(d["ws"])
    for n in (1101, -1, 8):
        d["qs"].copy_(good)
        d["sl"][0] = n
        c.run(d)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
        assert torch.equal(d["sel"][9:14].cpu(), ref[9:])
        assert_close(d["out"][9:14], want[9:], c.dtype, "the other sequences")
