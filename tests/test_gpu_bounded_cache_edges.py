"""The operators that bound a long context's cache in use together, and in calls at
the edges of what their documentation allows: other streams, captured and replayed
steps, workspaces in turns, failures, pools past 32-bit offsets, sequences by the
thousand, shared pages, scores at the ends of their range."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev
from test_gpu_bounded_cache import (Cache, check_evict, check_mass, check_window, compare_mass, lse_tol, mass_ref, mass_workspace, place, run_mass, run_window,  # noqa: F401
                                    window_ref, window_workspace)
from test_gpu_draft_ops import (U16, Batch, _clean_status, _lib, attention_tol, f64, head_ref, head_tol, i32, pool_rows, randn)  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- together ----------------------------------------------------------------------------

class Session:
    """A layer of a server that holds `budget` keys a sequence: prompts come in as
    chunks, then tokens one by one; keys gather weights; what outgrows the budget is
    evicted into other pages of the pool."""
    HQ, HKV, HD, PG, WINDOW, SINKS = 8, 4, 64, 64, 150, 3

    def __init__(self, rng, budget, B, pages):
        self.rng, self.budget, self.B = rng, budget, B
        self.n_pages = pages
        self.free = list(rng.permutation(pages))
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=dev())  # noqa: E731
        self.k, self.v = z(pages, self.HKV, self.PG, self.HD), z(pages, self.HKV, self.PG, self.HD)
        self.mass = z(pages, self.HKV, self.PG, dtype=torch.float32)
        self.tables = [[] for _ in range(B)]
        self.lens, self.seen = [0] * B, [0] * B         # cached slots, tokens so far

    def table(self, tables=None):
        tables = self.tables if tables is None else tables
        t = np.full((self.B, max(1, max(len(x) for x in tables))), -1, np.int32)
        for b, x in enumerate(tables):
            t[b, :len(x)] = x
        return t

    def step(self, new, stream=None):
        """New tokens of every sequence: rotated and appended, attended, weighed; each stage checked on what it was given."""
        rng, B = self.rng, self.B
        for b, n in enumerate(new):
            while len(self.tables[b]) * self.PG < self.lens[b] + n:
                self.tables[b].append(self.free.pop())
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(off[-1]) + 1
        rows = randn(rng, T, self.HQ + 2 * self.HKV, self.HD).to(dev())
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(self.seen, new)] + [[0]]).astype(np.int32)
        d = dict(page_tables=i32(self.table()), prefix_lens=i32(self.lens), offsets=i32(off))
        q = torch.zeros(T, self.HQ, self.HD, dtype=torch.bfloat16, device=dev())
        out, lse = torch.full_like(q, 7.0), torch.full((T, self.HQ), 7.0, device=dev())
        before = self.mass.cpu().numpy()
        dgp.dg_op_qk_norm_rope(rows[:, :self.HQ], None, i32(pos), q, None, stream=stream)
        dgp.dg_op_rope_kv_append(rows[:, self.HQ:self.HQ + self.HKV], rows[:, self.HQ + self.HKV:], self.k, self.v, **d, positions=i32(pos),
                                 stream=stream)
        ws = window_workspace(T, B, self.HQ, self.HKV, self.HD)
        dgp.dg_op_window_attention(q, self.k, self.v, **d, out=out, workspace=ws, window=self.WINDOW, sinks=self.SINKS, lse=lse, stream=stream)
        dgp.dg_op_key_mass(q, lse, self.k, self.mass, **d, workspace=mass_workspace(T, B, self.HQ, self.HKV, self.HD), window=self.WINDOW,
                           sinks=self.SINKS, stream=stream)
        torch.cuda.synchronize()
        dgp.dg_op_status()
        # the stages, on the values that each was given
        bt = Batch.__new__(Batch)
        bt.pre, bt.new, bt.hkv, bt.hd, bt.pg, bt.off, bt.table = list(self.lens), list(new), self.HKV, self.HD, self.PG, off, self.table()
        kp, vp = (pool_rows(x.float()) for x in (self.k, self.v))
        at = [np.arange(p + n) for p, n in zip(self.lens, new)]
        bt.keys, bt.vals = ([x[bt.table[b, j // self.PG], j % self.PG].astype(np.float64) for b, j in enumerate(at)] for x in (kp, vp))
        n = T - 1
        x, y = f64(rows), head_ref(f64(rows)[:, self.HQ:self.HQ + self.HKV], None, pos, self.HD)
        for b, m in enumerate(new):
            t = slice(off[b], off[b] + m)
            assert (np.abs(bt.keys[b][self.lens[b]:] - y[0][t]) <= head_tol(y[0][t], y[1][t])).all()
            assert np.array_equal(bt.vals[b][self.lens[b]:], x[t, self.HQ + self.HKV:])
        ref, mag, z, top = window_ref(f64(q), bt, self.WINDOW, self.SINKS, self.HD ** -0.5)
        assert (np.abs(f64(out)[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all() and (f64(out)[n:] == 7.0).all()
        assert (np.abs(f64(lse)[:n] - z[:n]) <= lse_tol(z[:n], top[:n], self.HD, 20)).all()
        compare_mass(self.mass, *mass_ref(f64(q), lse.cpu().numpy(), bt, before, self.WINDOW, self.SINKS, 0, self.HD ** -0.5), before)
        self.lens = [p + m for p, m in zip(self.lens, new)]
        self.seen = [s + m for s, m in zip(self.seen, new)]

    def evict(self):
        """Sequences past the budget move into other pages (the others' rows of the tables name their own: nothing moves)."""
        out = [[self.free.pop() for _ in range(-(-self.budget // self.PG))] if n > self.budget else list(t[:-(-n // self.PG)])
               for n, t in zip(self.lens, self.tables)]
        table, out_table = self.table(), self.table(out)
        kp, vp, mass = pool_rows(self.k.float()), pool_rows(self.v.float()), self.mass.cpu().numpy()
        out_lens = i32([9] * self.B)
        kept = torch.zeros(self.B, self.HKV, self.budget, dtype=torch.int32, device=dev())
        dgp.dg_op_cache_evict(self.k, self.v, self.mass, i32(table), i32(out_table), i32(self.lens), out_lens, self.budget, kept,
                              sinks=self.SINKS, recent=20)
        torch.cuda.synchronize()
        dgp.dg_op_status()
        k2, v2, m2 = pool_rows(self.k.float()), pool_rows(self.v.float()), self.mass.cpu().numpy()
        kept = kept.cpu().numpy()
        for b, n in enumerate(self.lens):
            m = min(n, self.budget)
            assert out_lens[b].item() == m
            for h in range(self.HKV):
                j, d = kept[b, h, :m], np.arange(m)
                assert (np.diff(j) > 0).all() and (kept[b, h, m:] == -1).all()
                old, now = (table[b, j // self.PG], j % self.PG), (out_table[b, d // self.PG], d % self.PG)
                assert np.array_equal(k2[now[0], now[1], h], kp[old[0], old[1], h]) and np.array_equal(v2[now[0], now[1], h], vp[old[0], old[1], h])
                assert np.array_equal(m2[now[0], h, now[1]], mass[old[0], h, old[1]])
                if n > self.budget:
                    w = mass[table[b, np.arange(n) // self.PG], h, np.arange(n) % self.PG].copy()
                    w[:self.SINKS] = w[n - 20:] = np.inf
                    gone = np.setdiff1d(np.arange(n), j)
                    assert w[gone].max() <= w[j].min()
            if n > self.budget:
                self.free += self.tables[b]
            self.lens[b], self.tables[b] = m, out[b]


def test_the_operators_together():
    s = Session(np.random.default_rng(71), budget=200, B=4, pages=60)
    s.step([300, 90, 0, 201])
    s.evict()
    assert s.lens == [200, 90, 0, 200]
    for _ in range(3):
        s.step([1, 1, 1, 1])
    s.step([5, 150, 2, 0])
    s.evict()
    s.step([1, 1, 1, 1])
    assert s.lens == [201, 201, 6, 201]


def test_the_operators_together_on_another_stream():
    s, st = Session(np.random.default_rng(72), budget=100, B=2, pages=40), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        s.step([130, 260], stream=st)
        s.evict()
        s.step([1, 1])


# ---- streams, captured calls, workspaces ------------------------------------------------

SHAPES = [(16, 8, 128, [5000, 30], [24, 2], 3000), (12, 4, 64, [300, 2500, 7], [500, 5, 1], 0), (8, 1, 128, [9000], [61], 0), (8, 2, 128, [0], [3000], 700),
          (32, 32, 64, [10, 700], [600, 800], 100)]


def calls_of(rng, n=len(SHAPES)):
    out = []
    for hq, hkv, hd, pre, new, window in SHAPES[:n]:
        bt = Batch(rng, pre, new, hkv, hd, 128)
        q = randn(rng, bt.T, hq, hd).to(dev())
        o, z = torch.zeros_like(q), torch.zeros(bt.T, hq, device=dev())
        run_window(bt, q, window, 4, o, z)
        mass = torch.zeros(bt.n_pages, hkv, 128, device=dev())
        run_mass(bt, q, z, mass, window, 4)
        torch.cuda.synchronize()
        dgp.dg_op_status()
        assert o[:int(bt.off[-1])].abs().sum() > 0 and mass.sum() > 0
        out.append((bt, q, window, o, z, mass))
    return out


def test_several_streams_among_other_kernels():
    calls = calls_of(np.random.default_rng(73))
    mine = [(torch.full_like(o, 7.0), torch.full_like(z, 7.0), torch.empty_like(m), torch.cuda.Stream(),
             window_workspace(bt.T, len(bt.pre), q.shape[1], bt.hkv, bt.hd, 0), mass_workspace(bt.T, len(bt.pre), q.shape[1], bt.hkv, bt.hd, 0))
            for bt, q, _, o, z, m in calls]
    a, side = torch.randn(512, 512, device=dev()), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(15):
        with torch.cuda.stream(side):
            a = torch.tanh(a @ a)
        for (bt, q, window, _, _, _), (o, z, m, st, ws, mws) in zip(calls, mine):
            with torch.cuda.stream(st):
                m.zero_()
                run_window(bt, q, window, 4, o, z, stream=st, workspace=ws)
                run_mass(bt, q, z, m, window, 4, stream=st, workspace=mws)
    torch.cuda.synchronize()
    dgp.dg_op_status()
    for (bt, _, _, o, z, m), (o2, z2, m2, _, _, _) in zip(calls, mine):
        n = int(bt.off[-1])
        assert torch.equal(o[:n], o2[:n]) and torch.equal(z[:n], z2[:n]) and torch.equal(m, m2)


def test_captured_calls_that_share_workspaces_take_turns():
    calls = calls_of(np.random.default_rng(74))
    ws = torch.full((max(dgp.dg_op_window_attention_workspace_bytes(bt.T, len(bt.pre), q.shape[1], bt.hkv, bt.hd) for bt, q, *_ in calls),), 0x5A,
                    dtype=torch.uint8, device=dev())
    mws = mass_workspace(1, 1, 1, 1, 64, 0x5A)
    st, graphs = torch.cuda.Stream(), []
    for bt, q, window, o, z, m in calls:
        o2, z2, m2, g = torch.full_like(o, 7.0), torch.full_like(z, 7.0), torch.zeros_like(m), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            m2.zero_()
            run_window(bt, q, window, 4, o2, z2, stream=st, workspace=ws)
            run_mass(bt, q, z2, m2, window, 4, stream=st, workspace=mws)
        graphs.append((g, o2, z2, m2))
    for turn in range(30):
        i = turn * 7 % len(calls)
        bt, q, window, o, z, m = calls[i]
        g, o2, z2, m2 = graphs[i]
        o2.fill_(7.0)
        m2.fill_(7.0)
        if turn % 5 == 4:
            m2.zero_()
            run_window(bt, q, window, 4, o2, z2, workspace=ws)
            run_mass(bt, q, z2, m2, window, 4, workspace=mws)
        else:
            g.replay()
        n = int(bt.off[-1])
        assert torch.equal(o[:n], o2[:n]) and torch.equal(z[:n], z2[:n]) and torch.equal(m, m2)
    dgp.dg_op_status()


def test_a_captured_step_serves_other_lengths():
    # rows for 700 tokens: prompts of other lengths are written into the same tensors
    rng = np.random.default_rng(75)
    hq, hkv, hd = 32, 16, 64
    first = Batch(rng, [300, 700, 10], [400, 100, 197], hkv, hd, 64, pad=3)
    q, o, z = randn(rng, first.T, hq, hd).to(dev()), torch.zeros(first.T, hq, hd, dtype=torch.bfloat16, device=dev()), torch.zeros(first.T, hq, device=dev())
    ws, mws = window_workspace(first.T, 3, hq, hkv, hd), mass_workspace(first.T, 3, hq, hkv, hd)
    mass = torch.zeros(first.n_pages, hkv, 64, device=dev())
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        run_window(first, q, 250, 4, o, z, stream=st, workspace=ws)
        run_mass(first, q, z, mass, 250, 4, observe=32, stream=st, workspace=mws)
    for pre, new in (([300, 700, 10], [400, 100, 197]), ([0, 0, 0], [697, 0, 0]), ([500, 3, 64], [1, 1, 1]), ([64, 700, 1], [0, 16, 600])):
        bt = Batch(rng, pre, new, hkv, hd, 64, pad=first.T - sum(new))
        assert bt.n_pages <= first.n_pages and bt.max_pages <= first.max_pages
        table = np.full(first.table.shape, -7, np.int32)
        table[:, :bt.max_pages] = bt.table
        for name, v in (("page_tables", i32(table)), ("prefix_lens", bt.d["prefix_lens"]), ("offsets", bt.d["offsets"])):
            first.d[name].copy_(v)
        first.k_pool[:bt.n_pages].copy_(bt.k_pool)
        first.v_pool[:bt.n_pages].copy_(bt.v_pool)
        q.copy_(randn(rng, first.T, hq, hd))
        before = rng.exponential(1.0, mass.shape).astype(np.float32)
        mass.copy_(torch.from_numpy(before))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        dgp.dg_op_status()
        n = sum(new)
        ref, mag, lse, top = window_ref(f64(q), bt, 250, 4, hd ** -0.5)
        assert (np.abs(f64(o)[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all() and (o[n:] == 7.0).all()
        assert (np.abs(f64(z)[:n] - lse[:n]) <= lse_tol(lse[:n], top[:n], hd, 12)).all()
        compare_mass(mass, *mass_ref(f64(q), z.cpu().numpy(), bt, before, 250, 4, 32, hd ** -0.5), before)


@pytest.mark.parametrize("hq,hkv,hd,pre,new,window", [(8, 2, 128, [4000, 4100], [61, 33], 3000), (16, 8, 128, [0, 100], [1900, 700], 500)])
def test_a_captured_window_recovers_from_a_failure(hq, hkv, hd, pre, new, window):
    # a launch that finds an earlier failure gives up; the replays after dg_op_status
    # has told of it must not take what it left in the workspace for their own
    rng = np.random.default_rng(76)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    ws = window_workspace(bt.T, len(pre), hq, hkv, hd, 0)
    q, out, z = randn(rng, bt.T, hq, hd).to(dev()), torch.empty(bt.T, hq, hd, dtype=torch.bfloat16, device=dev()), torch.empty(bt.T, hq, device=dev())
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        run_window(bt, q, window, 4, out, z, stream=st, workspace=ws)
    n = int(bt.off[-1])
    for turn in range(6):
        dgp.dg_op_wait_selftest(20_000)
        g.replay()
        torch.cuda.synchronize()
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_ETIMEOUT
        dgp.dg_op_status()                                  # cleared
        for _ in range(2):
            q.copy_(randn(rng, bt.T, hq, hd))
            want, want_z = torch.full_like(out, 7.0), torch.full_like(z, 7.0)
            run_window(bt, q, window, 4, want, want_z)      # a workspace of its own
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            dgp.dg_op_status()
            assert torch.equal(out[:n], want[:n]) and torch.equal(z[:n], want_z[:n]), turn


def test_calls_without_a_stream_take_the_current_one_and_are_captured():
    rng = np.random.default_rng(77)
    bt = Batch(rng, [500], [40], 2, 64, 64)
    q = randn(rng, bt.T, 4, 64).to(dev())
    o, z, mass = torch.zeros_like(q), torch.zeros(bt.T, 4, device=dev()), torch.zeros(bt.n_pages, 2, 64, device=dev())
    lens, kept = i32([540]), torch.zeros(1, 2, 100, dtype=torch.int32, device=dev())
    out_lens, k, v = i32([0]), bt.k_pool.clone(), bt.v_pool.clone()
    ws, mws = window_workspace(bt.T, 1, 4, 2, 64), mass_workspace(bt.T, 1, 4, 2, 64)

    def step():
        run_window(bt, q, 100, 4, o, z, workspace=ws)
        run_mass(bt, q, z, mass, 100, 4, workspace=mws)
        dgp.dg_op_cache_evict(k, v, mass, bt.d["page_tables"], bt.d["page_tables"], lens, out_lens, 100, kept)

    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        step()
    assert not o.any() and not kept.any()                   # nothing ran
    g.replay()
    torch.cuda.synchronize()
    was = [t.clone() for t in (o, z, mass, kept, out_lens, k.view(torch.int16), v.view(torch.int16))]
    assert out_lens.item() == 100 and all(bool(t.any()) for t in was)
    for t, x in ((o, 0), (z, 0), (mass, 0), (kept, 0), (out_lens, 0), (k, bt.k_pool), (v, bt.v_pool)):
        t.copy_(torch.as_tensor(x))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(1_000_000)
        step()
    torch.cuda.synchronize()
    dgp.dg_op_status()
    assert all(torch.equal(a, b) for a, b in zip(was, (o, z, mass, kept, out_lens, k.view(torch.int16), v.view(torch.int16))))


FIRST_CALL = """
import torch
import discrete_diffusion_block_gb300 as dgp
dgp.load()
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
pools = [r(40, 8, 128, 64), r(40, 8, 128, 64)]
d = dict(page_tables=i([list(range(20)), list(range(20, 40))]), prefix_lens=i([300, 700]), offsets=i([0, 1400, 2000]))
q, out, lse, mass = r(2000, 32, 64), torch.zeros(2000, 32, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2000, 32, device="cuda"), torch.zeros(40, 8, 128, device="cuda")
q1, d1 = r(2, 32, 64), dict(page_tables=d["page_tables"], prefix_lens=i([1700, 1300]), offsets=i([0, 1, 2]))
out1, lse1 = torch.zeros_like(q1), torch.zeros(2, 32, device="cuda")
lens, out_lens, kept = i([1701, 1301]), i([0, 0]), torch.zeros(2, 8, 500, dtype=torch.int32, device="cuda")
ws, ws1, mws = u8(dgp.dg_op_window_attention_workspace_bytes(2000, 2, 32, 8, 64)), u8(dgp.dg_op_window_attention_workspace_bytes(2, 2, 32, 8, 64)), u8(dgp.dg_op_key_mass_workspace_bytes(2000, 2, 32, 8, 64))
def step(st):
    dgp.dg_op_window_attention(q, *pools, **d, out=out, workspace=ws, window=400, sinks=4, lse=lse, stream=st)
    dgp.dg_op_key_mass(q, lse, pools[0], mass, **d, workspace=mws, window=400, sinks=4, stream=st)
    dgp.dg_op_window_attention(q1, *pools, **d1, out=out1, workspace=ws1, window=400, sinks=4, lse=lse1, stream=st)
    dgp.dg_op_key_mass(q1, lse1, pools[0], mass, **d1, workspace=mws, window=400, sinks=4, stream=st)
    dgp.dg_op_cache_evict(*pools, mass, d["page_tables"], d["page_tables"], lens, out_lens, 500, kept, sinks=4, recent=64, stream=st)
start = [p.clone() for p in pools]
st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=st):
    step(st)
graph.replay()
torch.cuda.synchronize()
dgp.dg_op_status()
was = [t.clone() for t in (out, lse, mass, out1, lse1, out_lens, kept, *pools)]
assert all(bool(t.any()) for t in was)
for t in (out, lse, mass, out1, lse1, out_lens, kept):
    t.zero_()
for p, s in zip(pools, start):
    p.copy_(s)
torch.cuda.synchronize()
step(None)
torch.cuda.synchronize()
dgp.dg_op_status()
assert all(torch.equal(a, b) for a, b in zip(was, (out, lse, mass, out1, lse1, out_lens, kept, *pools)))
print("the same")
"""


def test_the_first_call_of_a_process_can_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "the same" in p.stdout, p.stderr[-2000:]


# ---- chunks of many rows ---------------------------------------------------------------

CHUNKS = [(16, 16, 64, [700], [1930], 64), (16, 8, 128, [500, 0], [1000, 950], 128), (24, 8, 64, [130, 1000, 0], [1, 600, 700], 64),
          (28, 4, 64, [64], [1101], 192), (32, 4, 128, [0, 3000], [961, 40], 128), (128, 1, 64, [5, 300, 90], [200, 1, 100], 64),
          (48, 1, 64, [1000], [641], 64)]


@pytest.mark.parametrize("hq,hkv,hd,pre,new,pg", CHUNKS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (127, 130), (128, 1), (300, 0), (500, 257), (50, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_chunks_of_many_rows(hq, hkv, hd, pre, new, pg, window, sinks):
    rng = np.random.default_rng(window % 999 + hd)
    bt = Batch(rng, pre, new, hkv, hd, pg)
    assert bt.T * hq >= 120 * 256 and bt.T * hq // hkv > 128 * len(pre)        # where the kernel for chunks is taken
    check_window(bt, hq, window, sinks, rng, strided=window % 2 == 1, hidden=sinks < 2 ** 30)


def test_chunks_report_bad_pages_and_leave_other_sequences_alone():
    rng = np.random.default_rng(86)
    bt = Batch(rng, [500, 100], [1000, 950], 8, 128, 128)
    q = randn(rng, bt.T, 16, 128).to(dev())
    good, lse = torch.zeros(bt.T, 16, 128, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, 16, device=dev())
    run_window(bt, q, 300, 4, good, lse)
    for at, value in ((1, bt.n_pages), (0, -1), (11, -1)):
        bad = bt.table.copy()
        page, bad[0, at] = bad[0, at], value
        out, z = torch.zeros_like(good), torch.zeros_like(lse)
        keep, bt.d = bt.d, dict(bt.d, page_tables=i32(bad))
        run_window(bt, q, 300, 4, out, z)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_EINVAL and "page" in str(e.value)
        assert torch.equal(out[1000:1950], good[1000:1950]) and torch.equal(z[1000:1950], lse[1000:1950])
        # the keys of the bad page are hidden
        s, j = 500 + np.arange(1000)[:, None], np.arange(1500)[None]
        see = (j <= s) & ((j > s - 300) | (j < 4)) & (j // 128 != at)
        for h in (0, 15):
            k, v, x = bt.keys[0][:, h // 2], bt.vals[0][:, h // 2], f64(q)[:1000, h]
            w = np.where(see, x @ k.T * 128 ** -0.5, -np.inf)
            e_ = np.exp(w - w.max(1, keepdims=True))
            e_ /= e_.sum(1, keepdims=True)
            ref, mag = e_ @ v, e_ @ np.abs(v)
            assert (np.abs(f64(out)[:1000, h] - ref) <= attention_tol(ref, mag)).all()
    assert bool(torch.isfinite(good.float()).all())


@pytest.mark.parametrize("hq,hkv,hd,pre,new,pg", CHUNKS)
def test_chunks_without_lse_have_the_same_output(hq, hkv, hd, pre, new, pg):
    rng = np.random.default_rng(88)
    bt = Batch(rng, pre, new, hkv, hd, pg)
    q, n = randn(rng, bt.T, hq, hd).to(dev()), int(bt.off[-1])
    want, z = torch.full((bt.T, hq, hd), 7.0, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, hq, device=dev())
    out = want.clone()
    run_window(bt, q, 333, 7, want, z)
    run_window(bt, q, 333, 7, out)
    assert torch.equal(out, want) and (out[:n] != 7.0).any() and (out[n:] == 7.0).all()


@pytest.mark.parametrize("first,stride", [(0, 0), (8, 0), (0, 8), (16, 24), (8, 16)])
def test_chunks_into_rows_at_addresses_of_16_bytes(first, stride):
    rng = np.random.default_rng(91)
    bt = Batch(rng, [100], [1000], 16, 64, 64)
    q = randn(rng, bt.T, 32, 64).to(dev())
    want = torch.full((bt.T, 32, 64), 7.0, dtype=torch.bfloat16, device=dev())
    run_window(bt, q, 300, 4, want)
    store = torch.full((first + bt.T * (2048 + stride),), 7.0, dtype=torch.bfloat16, device=dev())
    out = torch.as_strided(store, (bt.T, 32, 64), (2048 + stride, 64, 1), first)
    run_window(bt, q, 300, 4, out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (store == 7.0).all()                                            # nothing between the rows was written


@pytest.mark.parametrize("new,pre", [([1], [600]), ([1000, 1], [300, 200]), ([2500, 1], [300, 200])])
def test_workspaces_of_long_chunks_serve_all_smaller_calls(new, pre):
    rng = np.random.default_rng(87)
    most = dgp.dg_op_window_attention_workspace_bytes(3000, 1, 16, 8, 128)
    for n in (1, 100, 1919, 1920, 2999):
        for seqs in (1, 30, 5000):
            assert dgp.dg_op_window_attention_workspace_bytes(n, seqs, 16, 8, 128) <= most
    bt = Batch(rng, pre, new, 8, 128, 64)
    q = randn(rng, bt.T, 16, 128).to(dev())
    ws, outs = torch.empty(most, dtype=torch.uint8, device=dev()), []
    for w in (ws, None):
        outs.append(torch.zeros_like(q))
        run_window(bt, q, 100, 4, outs[-1], workspace=w)
    n = int(bt.off[-1])
    assert torch.equal(outs[0][:n], outs[1][:n])


# ---- weights of long sequences ---------------------------------------------------------

@pytest.mark.parametrize("hq,hkv,hd,seqs,most,new,window,sinks", [
    (16, 8, 128, 30, 6000, 1, 0, 0), (12, 4, 64, 40, 5000, 1, 0, 0), (16, 8, 128, 30, 5000, 2, 1500, 200), (16, 8, 64, 30, 4000, 9, 700, 0),
    (8, 8, 128, 12, 3000, 150, 1000, 4),
])
def test_mass_of_many_long_sequences(hq, hkv, hd, seqs, most, new, window, sinks):
    # many units to a block, whose last ones have one to three key tiles: every slot and
    # buffer is used many times over, some roles have nothing to do in some units
    rng = np.random.default_rng(seqs + hd)
    pre = [int(x) for x in rng.integers(0, most, seqs)]
    check_mass(Batch(rng, pre, [int(x) for x in rng.integers(1, new + 1, seqs)], hkv, hd, 64), hq, window, sinks, 0, rng)


# ---- eviction in one launch and in two -----------------------------------------------------

@pytest.mark.parametrize("hkv,hd,pg,lens,budget", [
    (8, 128, 128, [2500, 2049, 0, 2048], 2048),             # one launch, clusters
    (4, 64, 64, [3000] * 20 + [5, 1200, 1111] * 6, 1111),   # one launch, single blocks
    (38, 64, 64, [900, 800, 700, 901], 800),                # 152 heads: the last such call
    (51, 64, 64, [900, 800, 700], 800),                     # 153: two launches
    (8, 128, 100, [5000, 4097], 4097),                      # one launch, lists of more than a block's threads
    (1, 64, 64, [8193, 300], 200),                          # slots beyond one launch's
    (8, 128, 128, [2500, 2600, 2700, 2800, 2049] + [2100] * 8, 2048),   # rows beyond one launch's
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_in_one_launch_and_in_two(hkv, hd, pg, lens, budget, in_place):
    check_evict(Cache(np.random.default_rng(hkv + budget), lens, hkv, hd, pg, budget, in_place), 3, 50)


@pytest.mark.parametrize("lens,budget", [([700, 90, 901], 300), ([20000], 9000)])
def test_evict_with_weights_at_odd_addresses(lens, budget):
    results = []
    for shift in (0, 1):
        c = Cache(np.random.default_rng(90), lens, 2, 64, 64, budget, True)
        d = c.on_gpu()
        store = torch.zeros(d["mass_pool"].numel() + shift, device=dev())
        mass = store[shift:].view(d["mass_pool"].shape)
        mass.copy_(d["mass_pool"])
        dgp.dg_op_cache_evict(d["k_pool"], d["v_pool"], mass, d["page_tables"], d["out_tables"], d["lens"], d["out_lens"], budget, d["kept"], recent=5)
        torch.cuda.synchronize()
        dgp.dg_op_status()
        results.append((d["kept"], d["out_lens"], mass, d["k_pool"].view(torch.int16), d["v_pool"].view(torch.int16)))
    assert all(torch.equal(a, b) and a.any() for a, b in zip(*results))


# ---- batches of all kinds ------------------------------------------------------------------

def shifted(bt, by):
    """The batch with its rows from row `by` on: rows before belong to no sequence."""
    bt.off = bt.off + by
    bt.T += by
    bt.d["offsets"] = i32(bt.off)
    return bt


@pytest.mark.parametrize("hq,hkv,hd,pre,new,window", [(4, 2, 64, [90, 0], [3, 70], 50), (32, 16, 64, [90, 0], [300, 700], 0)])
def test_rows_before_the_first_sequence_take_no_part(hq, hkv, hd, pre, new, window):
    rng = np.random.default_rng(81)
    bt = shifted(Batch(rng, pre, new, hkv, hd, 64), 5)
    q = randn(rng, bt.T, hq, hd)
    q[:5] = float("nan")
    q = q.to(dev())
    o, z = torch.full((bt.T, hq, hd), 7.0, dtype=torch.bfloat16, device=dev()), torch.full((bt.T, hq), 7.0, device=dev())
    run_window(bt, q, window, 2, o, z)
    x = f64(q)
    x[:5] = 0
    ref, mag, lse, top = window_ref(x, bt, window, 2, hd ** -0.5)
    live = slice(5, int(bt.off[-1]))
    assert (np.abs(f64(o)[live] - ref[live]) <= attention_tol(ref[live], mag[live])).all() and (o[:5] == 7.0).all() and (z[:5] == 7.0).all()
    z[:5] = float("nan")
    before = rng.exponential(1.0, (bt.n_pages, hkv, 64)).astype(np.float32)
    mass = torch.from_numpy(before).to(dev())
    run_mass(bt, q, z, mass, window, 2)
    compare_mass(mass, *mass_ref(x, z.cpu().numpy(), bt, before, window, 2, 0, hd ** -0.5), before)


def test_thousands_of_short_sequences():
    rng = np.random.default_rng(82)
    n = 2500
    pre, new = [int(x) for x in rng.integers(0, 100, n)], [int(x) for x in rng.integers(0, 3, n)]
    check_window(Batch(rng, pre, new, 1, 64, 64), 2, 40, 3, rng, hidden=False)
    bt = Batch(rng, pre, new, 1, 64, 64)
    check_mass(bt, 2, 40, 3, 0, rng)
    c_lens = i32([p + m for p, m in zip(pre, new)])
    out_lens, kept = torch.zeros_like(c_lens), torch.zeros(n, 1, 50, dtype=torch.int32, device=dev())
    mass = torch.rand(bt.n_pages, 1, 64, device=dev())
    table = i32(np.maximum(bt.table, 0))
    dgp.dg_op_cache_evict(bt.k_pool, bt.v_pool, mass, table, table, c_lens, out_lens, 50, kept, recent=10)
    dgp.dg_op_status()
    assert torch.equal(out_lens, c_lens.clamp(max=50))
    live = torch.arange(50, device=dev())[None, None] < out_lens[:, None, None]
    assert ((kept >= 0) == live).all()


def test_sequences_that_share_prefix_pages_read_the_same_keys():
    rng = np.random.default_rng(83)
    bt = Batch(rng, [200, 200, 10], [3, 3, 1], 2, 64, 64)
    bt.table[1, :3] = bt.table[0, :3]                       # three whole pages of a common prompt
    bt.d["page_tables"].copy_(i32(bt.table))
    for x in (bt.keys, bt.vals):
        x[1][:192] = x[0][:192]
    check_window(bt, 4, 0, 0, rng)
    check_window(bt, 4, 100, 2, rng, hidden=False)


def test_pools_past_32_bit_offsets():
    # pools of 2^31 and more elements: the results of a small pool, page for page
    rng = np.random.default_rng(84)
    n_big = 16384 + 64
    big = [torch.zeros(n_big, 8, 128, 128, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    mass_big = torch.zeros(n_big, 8, 128, device=dev())
    for pre, new, window in (([300, 40], [5, 3], 200), ([300, 40], [1100, 900], 0)):
        bt = Batch(rng, pre, new, 8, 128, 128)
        at = n_big - bt.n_pages
        q, results = randn(rng, bt.T, 16, 128).to(dev()), []
        mass = torch.rand(bt.n_pages, 8, 128, device=dev())
        for b, pool in zip(big, (bt.k_pool, bt.v_pool)):
            b[at:] = pool
        mass_big[at:] = mass
        lens, n = i32([p + m for p, m in zip(pre, new)]), int(bt.off[-1])
        for pools, weights, shift in (((bt.k_pool, bt.v_pool), mass, 0), (big, mass_big, at)):
            d = dict(page_tables=i32(np.where(bt.table < 0, bt.table, bt.table + shift)), prefix_lens=bt.d["prefix_lens"], offsets=bt.d["offsets"])
            o, z = torch.zeros(bt.T, 16, 128, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, 16, device=dev())
            dgp.dg_op_window_attention(q, *pools, **d, out=o, workspace=window_workspace(bt.T, 2, 16, 8, 128), window=window, sinks=4, lse=z)
            dgp.dg_op_key_mass(q, z, pools[0], weights, **d, workspace=mass_workspace(bt.T, 2, 16, 8, 128), window=window, sinks=4)
            out_lens, kept = torch.zeros_like(lens), torch.zeros(2, 8, 150, dtype=torch.int32, device=dev())
            dgp.dg_op_cache_evict(*pools, weights, d["page_tables"], d["page_tables"], lens, out_lens, 150, kept, sinks=2, recent=20)
            results.append((o[:n], z[:n], out_lens, kept, weights[shift:shift + bt.n_pages], *(x[shift:shift + bt.n_pages].view(torch.int16) for x in pools)))
        dgp.dg_op_status()
        for a, b in zip(*results):
            assert torch.equal(a, b) and a.any()


def test_empty_tensors_through_the_binding():
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=dev())  # noqa: E731
    f32, n32 = torch.float32, torch.int32
    pool, mass = torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16, device=dev()), torch.zeros(2, 2, 64, device=dev())
    none = dict(page_tables=i32(np.zeros((3, 1))), prefix_lens=i32([0, 0, 0]), offsets=i32([0, 0, 0, 0]))
    dgp.dg_op_window_attention(e(0, 4, 64), pool, pool, **none, out=e(0, 4, 64), workspace=None)
    dgp.dg_op_key_mass(e(0, 4, 64), e(0, 4, dtype=f32), pool, mass, **none, workspace=None)
    q = torch.ones(4, 4, 64, dtype=torch.bfloat16, device=dev())
    out, z = torch.full_like(q, 7.0), torch.zeros(4, 4, device=dev())
    ws, mws = window_workspace(4, 3, 4, 2, 64), mass_workspace(4, 3, 4, 2, 64)
    dgp.dg_op_window_attention(q, pool, pool, **none, out=out, workspace=ws)      # rows, but no sequence has any
    dgp.dg_op_key_mass(q, z, pool, mass, **none, workspace=mws)
    no_seqs = dict(page_tables=i32(np.zeros((0, 1))), prefix_lens=i32([]), offsets=i32([0]))
    dgp.dg_op_window_attention(q, pool, pool, **no_seqs, out=out, workspace=None)
    dgp.dg_op_key_mass(q, z, pool, mass, **no_seqs, workspace=None)
    dgp.dg_op_cache_evict(pool, pool.clone(), mass, e(0, 1, dtype=n32), e(0, 1, dtype=n32), e(0, dtype=n32), e(0, dtype=n32), 5, e(0, 2, 5, dtype=n32))
    lens, kept = i32([0, 0]), torch.zeros(2, 2, 5, dtype=n32, device=dev())
    out_lens = i32([3, 3])
    dgp.dg_op_cache_evict(pool, pool.clone(), mass, e(2, 0, dtype=n32), e(2, 0, dtype=n32), lens, out_lens, 5, kept)     # sequences without a slot
    dgp.dg_op_status()
    assert (out == 7.0).all() and not mass.any() and not out_lens.any() and (kept == -1).all()


# ---- scores at the ends of their range -----------------------------------------------------

@pytest.mark.parametrize("new,hq,hkv", [([4], 2, 1), ([1000, 700], 48, 24)])
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_large_and_equal_scores(new, hq, hkv, size):
    # scores of +-hundreds and +-tens of thousands: the running maximum moves over many
    # tiles; equal keys: every weight the same
    rng = np.random.default_rng(85)
    B = len(new)
    bt = Batch(rng, [900] * B, new, hkv, 64, 64)
    n = 900 + max(new)
    up = (torch.linspace(-1, 1, n)[:, None, None] * 2.0).expand(n, hkv, 64).to(torch.bfloat16)
    pool = torch.full(bt.k_pool.shape, float("nan"), dtype=torch.bfloat16)
    for b in range(B):
        m = 900 + new[b]
        place(pool, bt.table[b], np.arange(m), up[:m].contiguous())
        bt.keys[b] = f64(up[:m])
    bt.k_pool = pool.to(dev())
    q = randn(rng, bt.T, hq, 64)
    q[0], q[1], q[2] = size, -size, 0.0
    out, z = torch.zeros(bt.T, hq, 64, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, hq, device=dev())
    run_window(bt, q.to(dev()), 0, 0, out, z)
    ref, mag, lse, top = window_ref(f64(q), bt, 0, 0, 0.125)
    T = int(bt.off[-1])
    # a score of s carries 64 fp32 roundings: its exponential s 2^-18, at most a factor of e^that
    wide = np.minimum(np.expm1(top * 2.0 ** -17)[..., None], 1e9) * np.abs(bt.vals[0]).max()
    assert (np.abs(f64(out)[:T] - ref[:T]) <= attention_tol(ref[:T], mag[:T]) + wide[:T]).all()
    assert (np.abs(f64(z)[:T] - lse[:T]) <= lse_tol(lse[:T], top[:T], 64, 20)).all()
