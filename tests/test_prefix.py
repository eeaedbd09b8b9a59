"""pa_prefix_forward against the definition in 64 bits: groups of sequences
that share a prefix, every head size and 16-bit type, lengths that end anywhere
in a page, a stage or a split; refusals (CPU), reports of bad data, timeouts."""
import math
import random

import pytest
import torch

import paged_decode_attention_v2_gb300 as pa
from gpu_helpers import assert_close

FAKE = 1 << 20  # aligned, never dereferenced by the host checks

BASE = dict(out=FAKE, query=FAKE, key_cache=FAKE, value_cache=FAKE, block_tables=FAKE, seq_lens=FAKE,
            prefix_tables=FAKE, prefix_lens=FAKE, prefix_start=FAKE, num_seqs=3, num_prefixes=2,
            num_heads=8, num_kv_heads=2, head_size=128, num_blocks=64, block_size=16,
            max_blocks_per_seq=8, max_prefix_blocks=32, max_seq_len=128, max_prefix_len=512,
            scale=0.1, partition_size=512, dtype=pa.PA_DTYPE_BF16, workspace=FAKE,
            workspace_bytes=1 << 30, stream=0, opts=None)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return pa.load_library()


@pytest.mark.parametrize("over,status", [
    (dict(out=0), pa.PA_ERR_INVALID_ARG),
    (dict(query=0), pa.PA_ERR_INVALID_ARG),
    (dict(prefix_tables=0), pa.PA_ERR_INVALID_ARG),
    (dict(prefix_lens=0), pa.PA_ERR_INVALID_ARG),
    (dict(prefix_start=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(num_prefixes=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_prefix_blocks=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_prefix_len=513), pa.PA_ERR_INVALID_ARG),
    (dict(max_prefix_len=-1), pa.PA_ERR_INVALID_ARG),
    (dict(max_seq_len=129), pa.PA_ERR_INVALID_ARG),
    (dict(num_heads=9), pa.PA_ERR_INVALID_ARG),
    (dict(scale=math.nan), pa.PA_ERR_INVALID_ARG),
    (dict(query=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 64), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=pa.PA_DTYPE_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(head_size=96), pa.PA_ERR_UNSUPPORTED),
    (dict(num_heads=34), pa.PA_ERR_UNSUPPORTED),
    (dict(partition_size=96), pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=24, max_prefix_len=500), pa.PA_ERR_UNSUPPORTED),
    (dict(workspace_bytes=1000), pa.PA_ERR_WORKSPACE_TOO_SMALL),
])
def test_refusals(lib, over, status):
    assert lib.pa_prefix_forward(*dict(BASE, **over).values()) == status


def test_refused_variants(lib):
    for kw in (dict(variant=pa.PA_VARIANT_V1), dict(variant=7)):
        o = pa.pa_options_t(**kw)
        assert lib.pa_prefix_forward(*dict(BASE, opts=o).values()) == pa.PA_ERR_INVALID_ARG
    for kw in (dict(math=7), dict(num_stages=1), dict(num_stages=17)):
        o = pa.pa_options_t(**kw)
        assert lib.pa_prefix_forward(*dict(BASE, opts=o).values()) == pa.PA_ERR_INVALID_ARG
    o = pa.pa_options_t(math=pa.PA_MATH_SIMT)
    assert lib.pa_prefix_forward(*dict(BASE, opts=o).values()) == pa.PA_ERR_UNSUPPORTED


def test_more_own_partitions_than_the_count_holds(lib):
    """Items are counted below bit 30, which the prefix kernel sets."""
    for n, status in ((1 << 21, pa.PA_ERR_UNSUPPORTED), (1 << 20, pa.PA_ERR_WORKSPACE_TOO_SMALL)):
        a = dict(BASE, num_seqs=n, num_heads=8, num_kv_heads=8, max_blocks_per_seq=1 << 10, max_seq_len=1 << 14)
        assert lib.pa_prefix_forward(*a.values()) == status


def test_workspace_bytes(lib):
    f = pa.pa_prefix_workspace_bytes
    n = f(3, 2, 8, 2, 128, 128, 512, 512)
    assert n % 256 == 0 and n > pa.pa_workspace_bytes(3, 8, 128, 128, 512)
    assert lib.pa_prefix_forward(*dict(BASE, workspace_bytes=n - 1).values()) == \
        pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert lib.pa_prefix_forward(*dict(BASE, num_seqs=0).values()) == pa.PA_OK
    assert lib.pa_prefix_forward(*dict(BASE, num_seqs=0, query=0, out=0, seq_lens=0,
                                       block_tables=0).values()) == pa.PA_OK
    assert f(3, 0, 8, 2, 128, 128, 512, 512) == 0 and f(3, 1, 8, 3, 128, 128, 512, 512) == 0
    assert f(3, 1, 8, 2, 128, 0, 0, 512) > 0


def test_a_workspace_serves_every_smaller_call(lib):
    """Sized for the largest batch, prefix and own lengths, a workspace is
    refused by no call of smaller ones, whose best number of splits may be
    larger.  (Without a device a call that passes its checks ends right behind
    them.)"""
    if torch.cuda.is_available():
        pytest.skip("for the host's checks alone: the addresses are made up")
    rng = random.Random(1)
    log = lambda lo, hi: round(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    pairs = [((256, 1, 512, 32768), (224, 1, 512, 32768), 4, 8, 128)]
    for _ in range(3000):
        large = (log(1, 3000), rng.choice([1, 1, 2, 5, 30]), rng.choice([0, 64, 512, 5000]), log(64, 400_000))
        small = tuple(n if rng.random() < 0.4 else max(lo, n - rng.randint(0, n) if rng.random() < 0.5
                                                       else n - min(n, rng.randint(0, 9)))
                      for n, lo in zip(large, (1, 1, 0, 0)))
        pairs.append((large, small, rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 16]),
                      rng.choice([64, 128, 256])))
    for (B, G, own, prefix), (b, g, o, p), K, heads, D in pairs:
        P = rng.choice([64, 256, 512])
        n = pa.pa_prefix_workspace_bytes(B, G, heads * K, K, D, own, prefix, P)
        a = dict(BASE, num_seqs=b, num_prefixes=g, num_heads=heads * K, num_kv_heads=K, head_size=D,
                 max_seq_len=o, max_prefix_len=p, partition_size=P, max_blocks_per_seq=1 << 15,
                 max_prefix_blocks=1 << 15, workspace_bytes=n)
        assert n > 0 and lib.pa_prefix_forward(*a.values()) == pa.PA_ERR_CUDA, \
            (B, G, own, prefix, b, g, o, p, K, heads, D, P)


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 129, 2 ** 31 - 1])
def test_lengths_beyond_31_bit_arithmetic_are_refused(lib, n):
    """They have no size and are no call, whatever the table could hold: with a
    split added they would pass 2^31."""
    f = pa.pa_prefix_workspace_bytes
    for D in (64, 128, 256):
        for P in (64, 512, 8192):
            assert f(3, 1, 8, 2, D, 128, n, P) == f(3, 1, 8, 2, D, n, 128, P) == f(3, 1, 8, 2, D, n, n, P) == 0
    for over in (dict(max_prefix_len=n), dict(max_seq_len=n)):
        a = dict(BASE, max_prefix_blocks=2 ** 31 - 1, max_blocks_per_seq=2 ** 31 - 1,
                 workspace_bytes=1 << 40, **over)
        assert lib.pa_prefix_forward(*a.values()) == pa.PA_ERR_UNSUPPORTED
    assert 0 < f(3, 1, 8, 2, 128, 128, 2 ** 30, 512) < 1 << 24
    # as are rows whose bytes would wrap
    assert f(n, 1, n, 1, 128, 128, 512, 512) == f(n, 1, n, 1, 256, 0, 512, 64) == 0
    assert f(1 << 28, 1, 256, 256, 256, 0, 8192, 64) >> 40 > 0
    a = dict(BASE, num_seqs=1 << 27, num_heads=1 << 20, num_kv_heads=1 << 20, num_blocks=1, max_seq_len=0,
             workspace_bytes=1 << 62)
    assert lib.pa_prefix_forward(*a.values()) == pa.PA_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------

class Case:
    def __init__(self, seed, dtype, H, K, D, bs, counts, prefix, own, P=512, k_mult=2.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        B = sum(counts)
        assert len(own) == B and len(prefix) == len(counts)
        self.__dict__.update(dtype=dtype, H=H, K=K, D=D, bs=bs, counts=counts, prefix=prefix, own=own,
                             P=P, B=B, scale=1 / math.sqrt(D) if scale is None else scale)
        pages = [-(-L // bs) for L in prefix + own]
        pool = sum(pages) + 2
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        at, tabs = 0, []
        for n in pages:
            tabs.append(perm[at:at + n])
            at += n

        def table(rows):
            t = torch.full((len(rows), max([len(x) for x in rows] + [1])), -1, dtype=torch.int32)
            for i, x in enumerate(rows):
                t[i, :len(x)] = x
            return t
        self.pt, self.bt = table(tabs[:len(prefix)]), table(tabs[len(prefix):])
        self.start = [0]
        for n in counts:
            self.start.append(self.start[-1] + n)
        self.q = torch.randn(B, H, D, generator=g).to(dtype)
        self.kc = (k_mult * torch.randn(pool, K, bs, D, generator=g)).to(dtype)
        self.vc = torch.randn(pool, K, bs, D, generator=g).to(dtype)

    def rows(self, cache, table, n):
        t = torch.arange(n)
        return cache[table[t // self.bs].long(), :, t % self.bs].double().transpose(0, 1)  # [K, n, D]

    def reference(self):
        G = self.H // self.K
        out = torch.zeros(self.B, self.K, G, self.D, dtype=torch.float64)
        for g, P in enumerate(self.prefix):
            kp, vp = self.rows(self.kc, self.pt[g], P), self.rows(self.vc, self.pt[g], P)
            for s in range(self.start[g], self.start[g + 1]):
                k = torch.cat([kp, self.rows(self.kc, self.bt[s], self.own[s])], 1)
                v = torch.cat([vp, self.rows(self.vc, self.bt[s], self.own[s])], 1)
                if k.shape[1]:
                    x = self.q[s].double().view(self.K, G, self.D) @ k.transpose(1, 2) * self.scale
                    out[s] = torch.softmax(x, -1) @ v
        return out.view(self.B, self.H, self.D).numpy()

    def device(self, poison=True):
        dev = "cuda"
        kc, vc = self.kc.clone(), self.vc.clone()
        if poison:  # what lies behind the last token of a page is never used
            for t, L in zip(list(self.pt) + list(self.bt), self.prefix + self.own):
                if L % self.bs:
                    kc[t[L // self.bs], :, L % self.bs:] = math.nan
                    vc[t[L // self.bs], :, L % self.bs:] = math.inf
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        return dict(q=self.q.to(dev), kc=kc.to(dev), vc=vc.to(dev), bt=self.bt.to(dev), sl=i32(self.own),
                    pt=self.pt.to(dev), pl=i32(self.prefix), ps=i32(self.start),
                    ws=pa.alloc_prefix_workspace(self.B, len(self.prefix), self.H, self.K, self.D,
                                                 max(self.own), max(self.prefix), self.P),
                    out=torch.full((self.B, self.H, self.D), math.nan, dtype=self.dtype, device=dev))

    def run(self, d, **kw):
        pa.pa_prefix_forward(d["out"], d["q"], d["kc"], d["vc"], d["bt"], d["sl"], d["pt"], d["pl"], d["ps"],
                             self.scale, self.P, d["ws"], max_seq_len=max(self.own),
                             max_prefix_len=max(self.prefix), **kw)

    def peaky_bound(self, ref):
        """What rounding can do when few keys carry all the weight, where the
        parity bar (which counts on many rounding errors averaging out) is no
        bound.  The weights are rounded to the type, each off by at most half a
        step, u = eps / 2 of its value (f16: 2^-25 below the normal range, the
        largest weight being at least 2^-8), while their sum is not:
        |error| <= u sum p |v|; the result is rounded once more, u |out|.  The
        logits are fp32 sums of D products, off by at most
        t = (D + 2) 2^-24 scale sum |q k| each, which moves the weights by a
        factor of exp(+-2 t)."""
        u = torch.finfo(self.dtype).eps / 2
        tiny = 2.0 ** -17 if self.dtype == torch.float16 else 0.0
        G = self.H // self.K
        out = torch.zeros(self.B, self.K, G, self.D, dtype=torch.float64)
        for g, P in enumerate(self.prefix):
            kp, vp = self.rows(self.kc, self.pt[g], P), self.rows(self.vc, self.pt[g], P)
            for s in range(self.start[g], self.start[g + 1]):
                k = torch.cat([kp, self.rows(self.kc, self.bt[s], self.own[s])], 1)
                v = torch.cat([vp, self.rows(self.vc, self.bt[s], self.own[s])], 1)
                q = self.q[s].double().view(self.K, G, self.D)
                p = torch.softmax(q @ k.transpose(1, 2) * self.scale, -1)
                t = (self.D + 2) * 2.0 ** -24 * abs(self.scale) * \
                    (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
                pv = p @ v.abs()
                out[s] = (u + torch.expm1(2 * t)) * pv + tiny * v.abs().sum(1, keepdim=True)
        return out.view(self.B, self.H, self.D).numpy() * (1 + u) + u * abs(ref)

    def check(self, calls=2, peaky=False):
        d = self.device()
        ref = self.reference()
        bound = self.peaky_bound(ref) if peaky else None
        last = None
        for _ in range(calls):
            d["out"].fill_(math.nan)
            self.run(d)
            assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
            if peaky:
                err = abs(d["out"].double().cpu().numpy() - ref)
                assert (err <= bound).all(), f"{(err - bound).max():.3e} over"
            else:
                assert_close(d["out"], ref, self.dtype, "shared prefix")
            assert last is None or torch.equal(last, d["out"])  # no order of anything in the result
            last = d["out"].clone()


DTYPES = [torch.bfloat16, torch.float16]
ids = lambda v: str(v).replace("torch.", "")  # noqa: E731


@pytest.mark.gpu
def test_one_small_group():
    Case(1, torch.bfloat16, 8, 1, 128, 16, [2], [128], [5, 20]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 64])
def test_lengths(dtype, D, bs):
    """Prefixes that end inside a page, a stage, a split; own lengths from none."""
    for P in (1, 63, 64, 65, 127, 128, 129, 300, 1000):
        Case(P, dtype, 4, 2, D, bs, [3], [P], [0, 1, 40], P=256).check(calls=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D,G,K,bs", [(64, 16, 1, 16), (128, 8, 2, 16), (256, 4, 2, 32), (128, 1, 4, 8),
                                      (128, 7, 1, 32), (64, 3, 2, 64), (256, 5, 1, 16)], ids=ids)
def test_groups(dtype, D, G, K, bs):
    """Groups of none, one and many sequences, rows beyond one and two tiles."""
    rng = random.Random(D + G)
    counts = [3, 0, 1, 40, 0, 20]
    prefix = [700, 99, 0, 1500, 5, 2049]
    own = [rng.choice([0, 1, 17, 300, 600]) for _ in range(sum(counts))]
    Case(D, dtype, G * K, K, D, bs, counts, prefix, own).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_and_splits(D):
    """More items than SMs: CTAs take several, of different shapes."""
    rng = random.Random(D)
    own = [rng.randint(0, 50) for _ in range(150)]
    Case(D, torch.bfloat16, 16, 2, D, 16, [100, 50], [6001, 9000], own).check()


@pytest.mark.gpu
def test_more_groups_than_lanes():
    rng = random.Random(3)
    counts = [rng.choice([0, 1, 2, 3]) for _ in range(70)]
    prefix = [rng.choice([0, 1, 64, 200, 513]) for _ in counts]
    Case(3, torch.bfloat16, 4, 1, 128, 16, counts, prefix, [rng.randint(0, 30) for _ in range(sum(counts))]).check()


@pytest.mark.gpu
def test_nothing_at_all_gives_zeros():
    c = Case(4, torch.bfloat16, 4, 2, 64, 16, [2, 1], [0, 0], [0, 0, 0])
    d = c.device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK and (d["out"] == 0).all()


@pytest.mark.gpu
def test_long_prefix():
    Case(5, torch.bfloat16, 8, 1, 128, 16, [5], [100001], [1, 2, 3, 4, 5]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rising_maxima(D):
    """Keys that grow along the prefix: the running maximum is raised, and O
    rescaled, in most stages; large negative and zero scales too."""
    c = Case(6, torch.bfloat16, 4, 1, D, 16, [40], [1500], [9] * 40, k_mult=1.0)
    for j in range(c.pt.shape[1]):
        c.kc[c.pt[0, j]] *= 0.1 * (1 + j)
    c.check(peaky=True)
    Case(7, torch.float16, 4, 1, D, 16, [40], [700], [9] * 40, scale=-0.2).check()
    Case(8, torch.float16, 4, 1, D, 16, [2], [700], [9] * 2, scale=0.0).check()


@pytest.mark.gpu
def test_equals_the_sequences_with_the_prefix_in_their_tables():
    """A whole number of prefix pages, put in front of every sequence's own
    table: pa_v2_forward gives the same within the bar of both."""
    c = Case(9, torch.bfloat16, 32, 4, 128, 16, [30], [1024], [i * 7 for i in range(30)])
    d = c.device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    bt = torch.cat([d["pt"].expand(30, -1), d["bt"]], 1).contiguous()
    out = torch.empty_like(d["out"])
    ws = pa.alloc_workspace(30, 32, 128, bt.shape[1] * 16, 512)
    pa.pa_v2_forward(out, d["q"], d["kc"], d["vc"], bt, d["sl"] + 1024, c.scale, 512, ws)
    assert_close(d["out"], out.double().cpu().numpy(), c.dtype, "against pa_v2_forward")


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["block", "prefix_len", "own_len", "start", "end", "order"])
def test_bad_data_is_reported(what):
    """Found by the kernels' own checks before an address is formed; groups that
    are not concerned are served as usual."""
    c = Case(10, torch.bfloat16, 4, 1, 128, 16, [2, 3, 1], [300, 200, 100], [5, 50, 0, 7, 20, 1])
    ref = c.reference()
    d = c.device()
    if what == "block":
        d["pt"][0, 3] = -7
    elif what == "prefix_len":
        d["pl"][0] = 301
    elif what == "own_len":
        d["sl"][0] = 51
    elif what == "start":
        d["ps"][0] = 1
    elif what == "end":
        d["ps"][3] = 5
    else:
        d["ps"].copy_(torch.tensor([0, 5, 2, 6]))
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
    if what != "order":
        assert_close(d["out"][2:5], ref[2:5], c.dtype, "the second group")


@pytest.mark.gpu
def test_refused_depth_enqueues_nothing():
    """A ring that does not fit is refused before the prefix kernel is enqueued:
    the workspace stays as it was."""
    c = Case(13, torch.bfloat16, 4, 1, 256, 16, [3], [300], [5, 50, 20])
    d = c.device()
    d["ws"][256:] = 77
    with pytest.raises(pa.PAError):
        c.run(d, num_stages=16)
    torch.cuda.synchronize()
    assert (d["ws"][256:] == 77).all()
    c.run(d, num_stages=2)
    assert_close(d["out"], c.reference(), c.dtype, "two stages")


@pytest.mark.gpu
def test_groups_that_overlap_are_reported():
    """Starts that go up and down over many groups: no group of them is served
    twice, and the call ends as any other."""
    n = 200
    c = Case(12, torch.bfloat16, 4, 1, 64, 16, [6] + [0] * (n - 1), [300] * n, [5, 50, 0, 7, 20, 1])
    d = c.device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert_close(d["out"], c.reference(), c.dtype, "one group of many in use")
    d["ps"].copy_(torch.tensor([0, 6] * (n // 2) + [6]))
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_is_reported(D):
    """Softmax warps that never come: the bounded waits end, the kernel frees
    what it holds and reports; the next call on a fresh workspace is right."""
    c = Case(11, torch.bfloat16, 4, 1, D, 16, [3], [1000], [5, 0, 50])
    d = c.device()
    c.run(d, debug_flags=pa.PA_DEBUG_STALL_CONSUMERS, wait_limit_ns=20_000_000)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_TIMEOUT
    pa.pa_workspace_init(d["ws"])
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert_close(d["out"], c.reference(), c.dtype, "after the timeout")


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream():
    c = Case(12, torch.bfloat16, 16, 2, 128, 16, [4, 9], [777, 1300], [3 * i for i in range(13)])
    d = c.device(poison=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(d, stream=s)
    s.synchronize()
    assert_close(d["out"], c.reference(), c.dtype, "another stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(d)
    for prefix, own, start in (([777, 1300], c.own, [0, 4, 13]), ([5, 1299], [0] * 13, [0, 13, 13]),
                               ([640, 0], [i for i in range(13)], [0, 0, 13])):
        c.prefix, c.own, c.start = prefix, own, start
        d["pl"].copy_(torch.tensor(prefix))
        d["sl"].copy_(torch.tensor(own))
        d["ps"].copy_(torch.tensor(start))
        for _ in range(2):
            d["out"].fill_(math.nan)
            g.replay()
            assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
            assert_close(d["out"], c.reference(), c.dtype, f"replay {prefix} {start}")


@pytest.mark.gpu
def test_one_workspace_for_calls_of_many_shapes():
    """A workspace sized for the largest call serves calls of other shapes in
    between; only its status block is initialised."""
    cases = [Case(20, torch.bfloat16, 8, 2, 128, 16, [5, 9], [900, 1500], [7 * i for i in range(14)]),
             Case(21, torch.float16, 4, 1, 64, 8, [1], [70], [900], P=256),
             Case(22, torch.bfloat16, 4, 2, 256, 32, [30], [400], [i for i in range(30)], P=64)]
    n = max(pa.pa_prefix_workspace_bytes(c.B, len(c.prefix), c.H, c.K, c.D, max(c.own), max(c.prefix), c.P)
            for c in cases)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    state = [(c, c.device(), c.reference()) for c in cases]
    for _ in range(2):
        for c, d, ref in state:
            d["ws"] = ws
            d["out"].fill_(math.nan)
            c.run(d)
            assert pa.pa_read_device_status(ws) == pa.PA_OK
            assert_close(d["out"], ref, c.dtype, "shared workspace")


@pytest.mark.gpu
def test_cache_beyond_32_bits():
    """Pages at the end of caches of more than 2^32 bytes."""
    c = Case(23, torch.bfloat16, 8, 4, 128, 16, [3], [300], [5, 0, 33])
    d = c.device()
    blocks, pool = 300_000, c.kc.shape[0]
    for name in ("kc", "vc"):
        t = torch.empty((blocks,) + tuple(d[name].shape[1:]), dtype=c.dtype, device="cuda")
        t[blocks - pool:] = d[name]
        d[name] = t
    for name in ("bt", "pt"):
        d[name] = torch.where(d[name] >= 0, d[name] + (blocks - pool), -1).to(torch.int32)
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert_close(d["out"], c.reference(), c.dtype, "far pages")


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls with their own workspaces on two streams, overlapping."""
    a = Case(24, torch.bfloat16, 16, 2, 128, 16, [60], [3000], [i for i in range(60)])
    b = Case(25, torch.float16, 8, 1, 64, 16, [9, 30], [2000, 700], [3 * i for i in range(39)])
    state = [(c, c.device(), c.reference(), torch.cuda.Stream()) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, _, s in state:
            c.run(d, stream=s)
    torch.cuda.synchronize()
    for c, d, ref, s in state:
        assert pa.pa_read_device_status(d["ws"], s) == pa.PA_OK
        assert_close(d["out"], ref, c.dtype, "two streams")


def ramp(dtype, D, stages, v):
    """Keys whose logits step up by 4.1 to 5.4 from stage to stage of the kernel,
    another number for every row, and less than the 8 ln 2 beyond which its
    running maximum is raised in any case: weights that are no powers of two,
    and the last stage's outweighs all others.  Every value is v."""
    step = 64 if D == 256 else 128
    c = Case(30, dtype, 4, 1, D, 16, [8], [stages * step], list(range(8)), scale=1.0)
    c.q.zero_()
    c.q[..., 0] = torch.linspace(0.85, 1.1, 32).view(8, 4)
    c.kc[..., 0] = -60.0
    for j in range(stages):
        t = j * step
        c.kc[c.pt[0, t // 16], :, t % 16, 0] = max(-40.0, 4.875 * (j - stages + 1))
    c.vc.fill_(v)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("stages", [384, 383, 300])
def test_weights_sum_to_one(dtype, D, stages):
    """Values that are all alike come out as they are, whatever the weights: the
    rounded ones are what is divided by.  Sums and quotients in fp32, of at most
    200 terms each in a split and 65 splits, are off by less than 2^-14, less
    than the 2^-9 (bf16) or 2^-12 (f16) that would round to another value."""
    v = 2.0 - torch.finfo(dtype).eps
    d = (c := ramp(dtype, D, stages, v)).device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    assert (d["out"] == v).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_peaky_logits_within_the_parity_bar(dtype, D):
    """Growing keys, where few carry all the weight: the bar of every other call
    of the library holds."""
    c = Case(6, dtype, 4, 1, D, 16, [40], [1500], [9] * 40, k_mult=1.0)
    for j in range(c.pt.shape[1]):
        c.kc[c.pt[0, j]] *= 0.1 * (1 + j)
    c.check()
    c = ramp(dtype, D, 20, 0.0)
    g = torch.Generator().manual_seed(31)
    c.vc.copy_(torch.randn(c.vc.shape, generator=g))
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_f16_weights(D):
    """Weights of 2^-26 beside one of 1, every 64 keys, whose values make up for
    it: f16's smallest number is 2^-24.  A weight is off by at most 2^-32 of the
    largest, so the result by 63 x 2^-32 x 57344 = 8e-4, inside the bar."""
    c = Case(32, torch.float16, 4, 1, D, 16, [3], [640], [0, 1, 5], scale=1.0)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.kc[..., 0], c.vc[:] = -18.25, 57344.0
    for t in range(0, 640, 64):
        page = c.pt[0, t // 16]
        c.kc[page, :, t % 16, 0], c.vc[page, :, t % 16] = 0.0, 0.0
    c.check()


@pytest.mark.gpu
def test_fewer_splits_in_the_workspace_of_a_larger_batch():
    """132 sequences ask for less than 125, which would have more splits: these
    run with as many as there is room for."""
    counts = [3, 2, 90, 5, 0, 15, 0, 10]
    c = Case(33, torch.bfloat16, 64, 8, 256, 16, counts, [6000, 30, 700, 1, 5, 300, 9, 2049],
             [i % 65 for i in range(125)])
    sizes = (8, 64, 8, 256, 64, 6000, 512)
    assert pa.pa_prefix_workspace_bytes(132, *sizes) < pa.pa_prefix_workspace_bytes(125, *sizes)
    d, ref = c.device(), c.reference()
    n = pa.pa_prefix_workspace_bytes(132, *sizes)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    d["ws"] = buf[:n]
    d["ws"][:256] = 0
    for _ in range(2):
        c.run(d)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert_close(d["out"], ref, c.dtype, "the larger batch's workspace")
    assert (buf[n:] == 0xA5).all()


def marked(D, counts, prefix, H=8, K=1, bs=16, seed=40, extra=0):
    """Prefixes whose first and last tokens, those at the kernel's stage (so also
    split) edges and `extra` others, page edges among them, carry nearly all the
    weight: their keys lie along one direction that the queries share.  Values of
    random sign, so that each of the M of them moves the result by about
    0.012 a channel, more than twice the bar where the result is small, and the
    rounding of the weights by less than the bar."""
    rng = random.Random(seed)
    c = Case(seed, torch.bfloat16, H, K, D, bs, counts, prefix, [rng.randint(1, 9) for _ in range(sum(counts))],
             k_mult=0.1)
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(D, generator=g)
    u /= u.norm()
    stage = 64 if D == 256 else 128
    # logits of the marked tokens: about 9.5 above the others', alike for every row
    along = 3.1 * D ** 0.25
    c.q.copy_(0.25 * c.q.float() + along * u)
    c.marks = []
    for t, n in enumerate(prefix):
        at = {0, n - 1} | {i for i in range(n) if i % stage in (0, stage - 1)} if n else set()
        at |= {min(n - 1, rng.randint(0, n // bs) * bs + rng.choice([0, bs - 1])) for _ in range(extra)} if n else set()
        at = sorted(at)
        c.marks.append(at)
        for i in at:
            page, o = c.pt[t, i // bs], i % bs
            c.kc[page, :, o] = (c.kc[page, :, o].float() + along * u).to(c.dtype)
            c.vc[page, :, o] = (0.012 * len(at) * torch.sign(torch.randn(K, D, generator=g))).to(c.dtype)
    return c


MARKED = [(128, [5], [100001], {}), (64, [3, 2], [50001, 777], {}), (256, [2, 1], [20001, 300], dict(K=2)),
          (128, [70, 50], [6001, 9000], dict(H=16, K=2, extra=100)), (64, [150], [5000], dict(H=16, K=2, bs=8)),
          (256, [90], [4001], dict(H=16, K=2, bs=64, extra=50))]


@pytest.mark.parametrize("D,counts,prefix,kw", MARKED, ids=ids)
def test_a_lost_key_would_be_seen(D, counts, prefix, kw):
    """On the oracle: without any one marked token, without the prefix's last
    page, or with a stage counted twice, results leave the bar by half of it at
    least.  (The two calls below compare within the bar.)"""
    c = marked(D, counts, prefix, **kw)
    G, stage = c.H // c.K, 64 if D == 256 else 128
    ref = torch.from_numpy(c.reference()).view(c.B, c.K, G, D)
    for t, at in enumerate(c.marks):
        s = c.start[t]  # one sequence of the group, as every other has the same keys
        kp, vp = c.rows(c.kc, c.pt[t], prefix[t]), c.rows(c.vc, c.pt[t], prefix[t])
        k = torch.cat([kp, c.rows(c.kc, c.bt[s], c.own[s])], 1)
        p = torch.softmax(c.q[s].double().view(c.K, G, D) @ k.transpose(1, 2) * c.scale, -1)[..., :prefix[t]]
        out = ref[s]
        bar = 1.5 * (4e-3 + 1e-2 * out.abs())
        n = prefix[t]
        lost = [[i] for i in at] + [list(range((n - 1) // c.bs * c.bs, n))]
        for tok in lost:
            w = p[..., tok]
            rest = (out - w @ vp[:, tok]) / (1 - w.sum(-1, keepdim=True))
            assert ((rest - out).abs() > bar).any(), (t, tok)
        for a in range(0, n, stage):
            w = p[..., a:a + stage]
            twice = (out + w @ vp[:, a:a + stage]) / (1 + w.sum(-1, keepdim=True))
            assert ((twice - out).abs() > bar).any(), (t, a)


@pytest.mark.gpu
@pytest.mark.parametrize("D,counts,prefix,kw", MARKED, ids=ids)
def test_no_key_is_lost(D, counts, prefix, kw):
    """Every stage's and split's first and last token, the prefix's last one too,
    is in the result."""
    marked(D, counts, prefix, **kw).check(calls=1)


@pytest.mark.gpu
def test_the_count_of_items_is_left_as_other_calls_need_it():
    """One workspace in turn: the prefix call, with the own tokens beside the
    prefix or (opt-in) behind it on the other kernel, with no prefix at all,
    pa_v2_forward, and with wrong lengths: each starts from a count of zero."""
    c = Case(34, torch.bfloat16, 8, 2, 128, 16, [7, 3], [900, 300], [60 * i for i in range(10)])
    d, ref = c.device(), c.reference()
    out = torch.empty_like(d["out"])
    plain = Case(34, torch.bfloat16, 8, 2, 128, 16, [7, 3], [900, 300], [60 * i for i in range(10)])
    plain.prefix = [0, 0]
    own = plain.reference()

    def prefix(**kw):
        d["out"].fill_(math.nan)
        c.run(d, **kw)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert_close(d["out"], ref, c.dtype, str(kw))

    def decode():
        pa.pa_v2_forward(out, d["q"], d["kc"], d["vc"], d["bt"], d["sl"], c.scale, 512, d["ws"],
                         max_seq_len=max(c.own))
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert_close(out, own, c.dtype, "own tokens alone")

    for _ in range(2):
        prefix()
        decode()
        prefix(debug_flags=pa.PA_DEBUG_TCGEN05_KEYS)
        prefix()
        pa.pa_prefix_forward(out, d["q"], d["kc"], d["vc"], d["bt"], d["sl"], d["pt"], torch.zeros_like(d["pl"]),
                             d["ps"], c.scale, c.P, d["ws"], max_seq_len=max(c.own), max_prefix_len=0)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
        assert_close(out, own, c.dtype, "no prefix")
        bad = d["sl"] + 10 ** 6
        pa.pa_prefix_forward(out, d["q"], d["kc"], d["vc"], d["bt"], bad, d["pt"], d["pl"], d["ps"], c.scale, c.P,
                             d["ws"], max_seq_len=max(c.own), max_prefix_len=900)
        assert pa.pa_read_device_status(d["ws"]) == pa.PA_ERR_DEVICE_BAD_INPUT
        prefix()
        decode()
    assert (d["ws"][4:12] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heavy_first", [True, False], ids=["heavy_first", "light_first"])
def test_a_key_that_outweighs_the_others_is_exact(dtype, D, heavy_first):
    """Three stages of the last split hold a key each: one of logit 0, one 4.9 to
    5.5 above (2^7 to 2^7.9, another number for every row: a running maximum
    raised by nothing less than 2^8 would leave it rounded), one of 5/8 the
    weight of that.  Against the heaviest key the weights are 1 and 5/8, exact in
    every type, so the result is rounded once, u |ref|.  Besides, a logit is off
    by at most 2^-17 (its last bits in the key, sums of three products below 8 in
    fp32), which moves results by 2^-17 x 8 at most; fp32's part in the sums is
    smaller.  2^-12 covers both."""
    stages, step = 384, 64 if D == 256 else 128
    c = Case(35, dtype, 4, 1, D, 16, [8], [stages * step], [0] * 8, scale=1.0)
    c.q.zero_()
    c.q[..., 0] = torch.linspace(4.9, 5.49, 32).view(8, 4)
    c.q[..., 1:4] = 1.0
    c.kc.zero_()
    c.kc[..., 1] = -60.0
    c.vc.zero_()

    def key(stage, base, logit, v):
        t = stage * step
        page, o = c.pt[0, t // 16], t % 16
        hi = torch.tensor(logit, dtype=dtype)
        c.kc[page, :, o, 0] = base
        c.kc[page, :, o, 1] = hi
        c.kc[page, :, o, 2] = logit - hi.double().item()
        c.vc[page, :, o] = v

    light = math.log(5 / 8)
    key(stages - 6, 0.0, 0.0, 1.0)
    key(stages - 4, 1.0, 0.0 if heavy_first else light, 4.0 if heavy_first else -4.0)
    key(stages - 2, 1.0, light if heavy_first else 0.0, -4.0 if heavy_first else 4.0)
    ref = c.reference()
    d = c.device()
    c.run(d)
    assert pa.pa_read_device_status(d["ws"]) == pa.PA_OK
    err = abs(d["out"].double().cpu().numpy() - ref)
    bound = torch.finfo(dtype).eps / 2 * abs(ref) + 2.0 ** -12
    assert (err <= bound).all(), f"{(err - bound).max():.3e} over"
