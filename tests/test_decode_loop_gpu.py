"""The calls around the paged cache used together, as a decode loop uses them:
prompts and then tokens appended (rotated, bounds kept), attention over a shared
prefix and over selected blocks of the cache that the appends wrote, step by
step, eagerly and as one captured step replayed; every step against a plain
64-bit evaluation from the rows that went in."""
import math

import pytest
import torch

import paged_decode_attention_v2_gb300 as pa
from gpu_helpers import assert_close

pytestmark = pytest.mark.gpu

H, K, D, BS, R = 8, 2, 128, 16, 128
G = H // K
SCALE = 1 / math.sqrt(D)
PREFIX = 150                       # tokens all sequences share
PROMPTS = [1, 40, 16, 33, 7]       # own prompt of each sequence
STEPS = 21
B = len(PROMPTS)
SELECTED, SINKS, RECENT = 3, 1, 1


def _angles(n):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rotate(x, cs):
    """Half-split rotation of [rows, heads, D] in 64 bits by [rows, R] angles."""
    x, cs = x.double(), cs.double()[:, None]
    c, s = cs[..., :R // 2], cs[..., R // 2:]
    a, b = x[..., :R // 2], x[..., R // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


class Loop:
    def __init__(self, dtype, seed=3):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        own = max(PROMPTS) + STEPS
        self.width = -(-own // BS)
        npre = -(-PREFIX // BS)
        pool = npre + B * self.width + 1
        perm = torch.randperm(pool, generator=self.g).to(torch.int32)
        self.pt = perm[:npre][None].cuda()
        self.bt = perm[npre:npre + B * self.width].view(B, self.width).cuda()
        self.kc = torch.full((pool, K, BS, D), math.nan, dtype=dtype, device="cuda")
        self.vc = torch.full_like(self.kc, math.nan)
        self.kb = torch.full((pool, K, 2, D), math.nan, dtype=dtype, device="cuda")
        self.cs = _angles(PREFIX + own).cuda()
        self.lens = [0] * B
        self.max_len = self.width * BS
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.sl = i32([0] * B)
        self.pl, self.ps = i32([PREFIX]), i32([0, B])
        self.status = pa.alloc_workspace(1, 1, 64, 0, 64)
        self.ws_p = pa.alloc_prefix_workspace(B, 1, H, K, D, self.max_len, PREFIX, 128)
        self.ws_s = pa.alloc_sparse_workspace(B, H, K, D, BS, self.max_len, SELECTED, 128)
        # what went in, in 64 bits: keys (rotated, rounded) and values per sequence
        self.pre = self.append_prefix()
        self.keys = [torch.zeros(0, K, D, dtype=torch.float64) for _ in range(B)]
        self.values = [torch.zeros(0, K, D, dtype=torch.float64) for _ in range(B)]

    def rows(self, n):
        return torch.randn(n, (H + 2 * K) * D, generator=self.g).to(self.dtype)

    def split(self, x):
        n = x.shape[0]
        return (x[:, :H * D].view(n, H, D), x[:, H * D:(H + K) * D].view(n, K, D),
                x[:, (H + K) * D:].view(n, K, D))

    def append_prefix(self):
        x = self.rows(PREFIX)
        _, k, v = self.split(x.cuda())
        pa.pa_append_kv(self.kc, self.vc, k, v, self.pt, self.pl, self.status, key_bounds=self.kb,
                        cos_sin=self.cs, q_start=torch.tensor([0, PREFIX], dtype=torch.int32, device="cuda"))
        assert pa.pa_read_device_status(self.status) == pa.PA_OK
        _, k, v = self.split(x)
        return _rotate(k, self.cs.cpu()[:PREFIX]).to(self.dtype).double(), v.double()

    def note(self, x, new):
        """Record the rows of a step; returns the rotated queries in 64 bits."""
        q, k, v = self.split(x)
        pos = torch.tensor([PREFIX + L + i for L, n in zip(self.lens, new) for i in range(n)])
        cs = self.cs.cpu()[pos]
        k = _rotate(k, cs).to(self.dtype).double()
        row = 0
        for s, n in enumerate(new):
            self.keys[s] = torch.cat([self.keys[s], k[row:row + n]])
            self.values[s] = torch.cat([self.values[s], v[row:row + n].double()])
            self.lens[s] += n
            row += n
        return pos, _rotate(q, cs).to(self.dtype).double()

    def expect_prefix(self, q):
        out = torch.zeros(B, H, D, dtype=torch.float64)
        for s in range(B):
            k = torch.cat([self.pre[0], self.keys[s]]).transpose(0, 1)
            v = torch.cat([self.pre[1], self.values[s]]).transpose(0, 1)
            x = q[s].view(K, G, D) @ k.transpose(1, 2) * SCALE
            out[s] = (torch.softmax(x, -1) @ v).reshape(H, D)
        return out.numpy()

    def expect_sparse(self, q):
        out = torch.zeros(B, H, D, dtype=torch.float64)
        sel = torch.full((B, K, SELECTED), -1, dtype=torch.int32)
        for s in range(B):
            L = self.lens[s]
            n = -(-L // BS)
            for h in range(K):
                qq, kk = q[s].view(K, G, D)[h], self.keys[s][:, h]
                score = []
                for j in range(n):
                    page = kk[j * BS:(j + 1) * BS]
                    hi, lo = page.amax(0), page.amin(0)
                    forced = j < SINKS or j >= n - RECENT
                    score.append((not forced, -float(torch.maximum(qq * hi, qq * lo).sum()), j))
                got = sorted(j for _, _, j in sorted(score)[:SELECTED])
                sel[s, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
                tok = torch.cat([torch.arange(j * BS, min(L, (j + 1) * BS)) for j in got])
                w = torch.softmax(qq @ kk[tok].T * SCALE, -1)
                out[s, h * G:(h + 1) * G] = w @ self.values[s][tok, h]
        return out.numpy(), sel

    def attend(self, out_p, out_s, sel, q):
        pa.pa_prefix_forward(out_p, q, self.kc, self.vc, self.bt, self.sl, self.pt, self.pl, self.ps,
                             SCALE, 128, self.ws_p, max_seq_len=self.max_len, max_prefix_len=PREFIX)
        pa.pa_sparse_forward(out_s, sel, q, self.kc, self.vc, self.bt, self.sl, SCALE, 128, self.ws_s,
                             key_bounds=self.kb, sink_blocks=SINKS, recent_blocks=RECENT,
                             max_seq_len=self.max_len)

    def check(self, out_p, out_s, sel, q):
        for ws in (self.status, self.ws_p, self.ws_s):
            assert pa.pa_read_device_status(ws) == pa.PA_OK
        assert_close(out_p, self.expect_prefix(q), self.dtype, "shared prefix")
        want, wsel = self.expect_sparse(q)
        assert torch.equal(sel.cpu(), wsel)
        assert_close(out_s, want, self.dtype, "selected blocks")

    def prompts(self):
        x = self.rows(sum(PROMPTS))
        pos, _ = self.note(x, PROMPTS)
        starts = [0]
        for n in PROMPTS:
            starts.append(starts[-1] + n)
        _, k, v = self.split(x.cuda())
        self.sl.copy_(torch.tensor(self.lens))
        pa.pa_append_kv(self.kc, self.vc, k, v, self.bt, self.sl, self.status, key_bounds=self.kb,
                        cos_sin=self.cs, positions=pos.to(torch.int32).cuda(),
                        q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_steps(dtype):
    a = Loop(dtype)
    a.prompts()
    out_p = torch.empty(B, H, D, dtype=dtype, device="cuda")
    out_s, sel = torch.empty_like(out_p), torch.empty(B, K, SELECTED, dtype=torch.int32, device="cuda")
    rq = torch.empty_like(out_p)
    for _ in range(STEPS):
        x = a.rows(B)
        pos, q64 = a.note(x, [1] * B)
        a.sl.add_(1)
        q, k, v = a.split(x.cuda())
        pa.pa_append_kv(a.kc, a.vc, k, v, a.bt, a.sl, a.status, query=q, query_out=rq, key_bounds=a.kb,
                        cos_sin=a.cs, positions=pos.to(torch.int32).cuda())
        a.attend(out_p, out_s, sel, rq)
        a.check(out_p, out_s, sel, rq.double().cpu())
        assert (rq.double().cpu() - q64).abs().max() <= 2 ** -6  # a rounding of values below 8


def test_a_captured_step_replayed():
    """One graph holds the whole step (append, shared prefix, selected blocks);
    a second one of the same calls shares its workspaces, replayed in turn."""
    dtype = torch.bfloat16
    a = Loop(dtype, seed=4)
    a.prompts()
    x = torch.zeros(B, (H + 2 * K) * D, dtype=dtype, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = a.split(x)
    rq, out_p, out_s = (torch.empty(B, H, D, dtype=dtype, device="cuda") for _ in range(3))
    sel = torch.empty(B, K, SELECTED, dtype=torch.int32, device="cuda")

    def step():
        pa.pa_append_kv(a.kc, a.vc, k, v, a.bt, a.sl, a.status, query=q, query_out=rq, key_bounds=a.kb,
                        cos_sin=a.cs, positions=pos)
        a.attend(out_p, out_s, sel, rq)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        # every kernel once before capture; over empty rows, so that nothing is appended
        keep = a.sl.clone()
        a.sl.zero_()
        step()
        a.sl.copy_(keep)
    s.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for i in range(STEPS):
        new = a.rows(B)
        p, _ = a.note(new, [1] * B)
        x.copy_(new)
        pos.copy_(p)
        a.sl.copy_(torch.tensor(a.lens))
        graphs[i % 2].replay()
        a.check(out_p, out_s, sel, rq.double().cpu())


def test_inputs_written_right_before_the_call():
    """The lengths, the tables (with -1 for pages that a step does not have yet)
    and the cache's last row are written by the launches right before
    pa_prefix_forward, whose own tokens run beside its prefix: the bits are those
    of a run that synchronises between all of them."""
    steps = 60
    rows, outs = None, []
    for wait in (False, True):
        a = Loop(torch.bfloat16, seed=5)
        a.prompts()
        if rows is None:
            rows = [a.rows(B).cuda() for _ in range(STEPS)]
        lens = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
        pos = [lens + PREFIX + i for i in range(STEPS)]
        page = torch.arange(a.width, device="cuda")[None]
        full = a.bt.clone()
        tables = [torch.where(page <= ((lens + i) // BS)[:, None], full, -1).to(torch.int32) for i in range(STEPS)]
        rq, out = (torch.empty(B, H, D, dtype=a.dtype, device="cuda") for _ in range(2))
        got = torch.empty(steps * STEPS, B, H, D, dtype=a.dtype, device="cuda")
        sync = torch.cuda.synchronize if wait else lambda: None
        torch.cuda.synchronize()
        for j in range(steps):  # the same tokens over and over
            for i in range(STEPS):
                q, k, v = a.split(rows[i])
                a.bt.copy_(tables[i])
                torch.add(lens, i + 1, out=a.sl)
                sync()
                pa.pa_append_kv(a.kc, a.vc, k, v, a.bt, a.sl, a.status, query=q, query_out=rq, key_bounds=a.kb,
                                cos_sin=a.cs, positions=pos[i])
                sync()
                pa.pa_prefix_forward(out, rq, a.kc, a.vc, a.bt, a.sl, a.pt, a.pl, a.ps, SCALE, 128, a.ws_p,
                                     max_seq_len=a.max_len, max_prefix_len=PREFIX)
                sync()
                got[j * STEPS + i].copy_(out)
            for i in range(STEPS):  # no later round finds this one's rows
                at = (lens + i).long()
                a.kc[full.long()[torch.arange(B, device="cuda"), at // BS], :, at % BS] = math.nan
        assert pa.pa_read_device_status(a.ws_p) == pa.PA_OK and pa.pa_read_device_status(a.status) == pa.PA_OK
        outs.append(got)
    assert outs[0].isfinite().all() and torch.equal(outs[0], outs[1])
