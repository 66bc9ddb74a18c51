"""The operators over the paged cache with table entries, lengths and positions at
the ends of their types: whatever a table holds outside the pools is skipped and
reported, and what is too long is refused on the device."""
import contextlib

import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev
from test_gpu_bounded_cache import (Cache, check_evict, check_window, lse_tol, mass_case, mass_workspace, place, run_mass, run_window, same_floats, visible, window_ref,
                                    window_workspace)
from test_gpu_draft_ops import U32, Batch, _clean_status, _lib, attention_tol, f64, i32, randn, run_attention  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
OUTSIDE = [-1, -2, -3, -2 ** 31 + 1, -2 ** 31, 2 ** 31 - 1]       # entries outside any pool


# ---- pages outside the pools -------------------------------------------------------------

@contextlib.contextmanager
def entry(bt, b, at, value):
    """The batch with another entry in its page table; what the call reports is checked."""
    table = bt.table.copy()
    table[b, at] = value
    keep, bt.d = bt.d, dict(bt.d, page_tables=i32(table))
    yield
    bt.d = keep
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert e.value.code == dgp.DG_EINVAL and "page" in str(e.value)


def without_page(q, bt, at, window, sinks, head):
    """out, sum_j p_j |v_j|, lse and the largest sum of |products| of the first
    sequence's rows, in 64 bits, without the keys of its page `at`."""
    p, n, G = bt.pre[0], bt.new[0], q.shape[1] // bt.hkv
    see = visible(p, n, window, sinks) & (np.arange(p + n)[None] // bt.pg != at)
    k, v, x, scale = bt.keys[0][:, head // G], bt.vals[0][:, head // G], q[:n, head], bt.hd ** -0.5
    s = np.where(see, x @ k.T * scale, -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    z = m[:, 0] + np.log(e.sum(1))
    e /= e.sum(1, keepdims=True)
    return e @ v, e @ np.abs(v), z, (np.where(see, np.abs(x) @ np.abs(k).T * scale, 0)).max(1)


def check_without_page(bt, q, out, lse, at, window, sinks, heads):
    n, tiles = bt.new[0], (bt.pre[0] + bt.new[0]) / 128 + 2
    for h in heads:
        ref, mag, z, top = without_page(f64(q), bt, at, window, sinks, h)
        assert (np.abs(f64(out)[:n, h] - ref) <= attention_tol(ref, mag)).all(), (at, h)
        assert (np.abs(f64(lse)[:n, h] - z) <= lse_tol(z, top, bt.hd, tiles)).all(), (at, h)


CHUNK = ([500, 100], [1000, 950], 8, 128, 128)


@pytest.mark.parametrize("value", OUTSIDE)
@pytest.mark.parametrize("window,sinks", [(300, 4), (0, 0)])
def test_chunks_skip_pages_outside_the_pools(value, window, sinks):
    rng = np.random.default_rng(101)
    bt = Batch(rng, *CHUNK)
    q = randn(rng, bt.T, 16, 128).to(dev())
    good, lse = torch.zeros_like(q), torch.zeros(bt.T, 16, device=dev())
    run_window(bt, q, window, sinks, good, lse)
    for at in (0, 2, 6):
        out, z = torch.zeros_like(q), torch.zeros_like(lse)
        with entry(bt, 0, at, value):
            run_window(bt, q, window, sinks, out, z)
        check_without_page(bt, q, out, z, at, window, sinks, (0, 15))
        assert torch.equal(out[1000:1950], good[1000:1950]) and torch.equal(z[1000:1950], lse[1000:1950])


@pytest.mark.parametrize("value", OUTSIDE)
@pytest.mark.parametrize("pre,new,window", [([700, 50], [2, 3], 0), ([700, 50], [2, 3], 600), ([700, 50], [400, 3], 0)])
def test_mass_skips_and_reports_pages_outside_the_pools(value, pre, new, window):
    rng = np.random.default_rng(102)
    bt = Batch(rng, pre, new, 2, 64, 64)
    q, lse, before = mass_case(rng, bt, 4, window, 4, 0.125)
    z, good = torch.from_numpy(lse).to(dev()), torch.from_numpy(before).to(dev())
    run_mass(bt, q, z, good, window, 4)
    dgp.dg_op_status()
    for at in (0, 5, (pre[0] + new[0] - 1) // 64):         # first tokens, cached keys, new keys
        mass = torch.from_numpy(before).to(dev())
        with entry(bt, 0, at, value):
            run_mass(bt, q, z, mass, window, 4)
        want, page = good.cpu().numpy(), bt.table[0, at]
        want[page] = before[page]
        assert same_floats(mass.cpu().numpy(), want)


@pytest.mark.parametrize("value", OUTSIDE)
@pytest.mark.parametrize("window,sinks", [(300, 4), (0, 0)])
@pytest.mark.parametrize("pre,new", [([500, 50], [3, 2]), ([500, 50], [200, 3])])
def test_few_rows_skip_pages_outside_the_pools(value, window, sinks, pre, new):
    rng = np.random.default_rng(103)
    bt = Batch(rng, pre, new, 2, 64, 64)
    q = randn(rng, bt.T, 4, 64).to(dev())
    good, lse = torch.zeros_like(q), torch.zeros(bt.T, 4, device=dev())
    run_window(bt, q, window, sinks, good, lse)
    a, b = new[0], sum(new)
    for at in (0, 4, 7):
        out, z = torch.zeros_like(q), torch.zeros_like(lse)
        with entry(bt, 0, at, value):
            run_window(bt, q, window, sinks, out, z)
        check_without_page(bt, q, out, z, at, window, sinks, (0, 3))
        assert torch.equal(out[a:b], good[a:b]) and torch.equal(z[a:b], lse[a:b])


@pytest.mark.parametrize("value", OUTSIDE)
@pytest.mark.parametrize("pre,new", [([500, 50], [3, 2]), ([500, 50], [200, 3])])
def test_drafted_tokens_skip_pages_outside_the_pools(value, pre, new):
    rng = np.random.default_rng(104)
    bt = Batch(rng, pre, new, 2, 64, 64)
    q = randn(rng, bt.T, 4, 64).to(dev())
    good, a, b = torch.zeros_like(q), new[0], sum(new)
    run_attention(bt, q, None, good)
    for at in (0, 4, 7):
        out = torch.zeros_like(q)
        with entry(bt, 0, at, value):
            run_attention(bt, q, None, out)
        for h in (0, 3):
            ref, mag, _, _ = without_page(f64(q), bt, at, 0, 0, h)
            assert (np.abs(f64(out)[:a, h] - ref) <= attention_tol(ref, mag)).all()
        assert torch.equal(out[a:b], good[a:b])


# ---- warps with rows of nobody's ------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 31, 33, 64, 95, 97, 127])
@pytest.mark.parametrize("pre,window", [(0, 200), (2000, 0)])
def test_chunks_with_any_number_of_rows_in_the_last_tile(rows, pre, window):
    # one row a token: the last tile's warps are full, empty, and in between
    rng = np.random.default_rng(110 + rows)
    check_window(Batch(rng, [pre], [10 * 128 + rows], 16, 64, 64), 16, window, 2, rng)


# ---- scores that lie far apart -----------------------------------------------------------------

@pytest.mark.parametrize("new,hq,hkv", [([4, 2], 2, 1), ([1000, 700], 48, 24)])
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_rows_whose_scores_lie_far_apart(new, hq, hkv, size):
    # Keys of one number each in all 64 elements, queries likewise: a score is 64 equal
    # products of two bf16 numbers, exact in fp32 in any order, and what the exponents
    # add to it (one rounding of the factor, one of the maximum, the same for all keys of a
    # row) moves weights against each other by 2^-24 of their distance in the exponent. So
    # these rows have the tolerance of any other, and their log-sum-exps one that
    # counts the roundings of factor, ln 2 and result.
    rng = np.random.default_rng(120)
    bt = Batch(rng, [900] * len(new), new, hkv, 64, 64)
    n = 900 + max(new)
    up = (torch.linspace(-1, 1, n)[:, None, None] * 2.0).expand(n, hkv, 64).to(torch.bfloat16)
    pool = torch.full(bt.k_pool.shape, float("nan"), dtype=torch.bfloat16)
    for b, m in enumerate(new):
        place(pool, bt.table[b], np.arange(900 + m), up[:900 + m].contiguous())
        bt.keys[b] = f64(up[:900 + m])
    bt.k_pool = pool.to(dev())
    q = randn(rng, bt.T, hq, 64)
    up_rows, down_rows = bt.off[:-1].tolist(), (bt.off[:-1] + 1).tolist()
    q[up_rows], q[down_rows] = size, -size
    out, lse = torch.zeros(bt.T, hq, 64, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, hq, device=dev())
    run_window(bt, q.to(dev()), 0, 0, out, lse)
    dgp.dg_op_status()
    ref, mag, z, _ = window_ref(f64(q), bt, 0, 0, 0.125)
    rows = up_rows + down_rows
    assert (np.abs(f64(out) - ref) <= attention_tol(ref, mag))[rows].all(), np.abs(f64(out) - ref)[rows].max()
    assert (np.abs(f64(lse) - z) <= U32 * (4 * np.abs(z) + 128))[rows].all()


# ---- sequences beyond what the eviction takes --------------------------------------------

@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 31, 2 ** 31 - 32, 262144 + 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_leaves_sequences_of_too_many_slots_alone(length, in_place):
    # the table covers the length: one page of many slots, over and over
    pg, budget = 65536, 200
    rng = np.random.default_rng(105)
    table = np.zeros((3, 2 ** 31 // pg), np.int32)
    table[1, :1], table[2, :1] = 1, 2
    out = np.array([[0], [1], [2]] if in_place else [[3], [4], [5]], np.int32)
    k, v = (torch.from_numpy(rng.integers(0, 2 ** 16, (6, 1, pg, 64), dtype=np.uint16).view(np.int16)) for _ in range(2))
    mass = rng.exponential(1.0, (6, 1, pg)).astype(np.float32)
    d = [x.to(dev()).view(torch.bfloat16) for x in (k, v)] + [torch.from_numpy(mass).to(dev())]
    lens, out_lens, kept = i32([300, length, 100]), i32([7, 7, 7]), torch.full((3, 1, budget), 7, dtype=torch.int32, device=dev())
    dgp.dg_op_cache_evict(*d, i32(table), i32(out), lens, out_lens, budget, kept, sinks=2, recent=20)
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert e.value.code == dgp.DG_EINVAL and "sequence" in str(e.value)
    assert out_lens.tolist() == [200, -1, 100] and (kept[1] == -1).all()
    j = kept[0, 0].cpu().numpy()
    assert (np.diff(j) > 0).all() and j[-1] == 299
    (to0, left, to2), got = out[:, 0], [x.view(torch.int16).cpu() if x.dtype == torch.bfloat16 else x.cpu() for x in d]
    for x, was in zip(got, (k, v, torch.from_numpy(mass))):
        assert torch.equal(x[left], was[left]) and torch.equal(x[1], was[1])
    assert np.array_equal(got[2][to0, 0, :200].numpy(), mass[0, 0, j]) and np.array_equal(got[2][to2, 0, :100].numpy(), mass[2, 0, :100])


@pytest.mark.parametrize("length", [300, -1])
def test_evict_to_the_largest_budget(length):
    # the lists of kept slots are as long as the budget
    rng, budget = np.random.default_rng(106), 2 ** 31 - 1
    k, v, mass = randn(rng, 10, 1, 64, 64).to(dev()), randn(rng, 10, 1, 64, 64).to(dev()), torch.rand(10, 1, 64, device=dev())
    was = [x.clone() for x in (k, v, mass)]
    kept = torch.full((1, 1, budget), 7, dtype=torch.int32, device=dev())
    out_lens = i32([7])
    dgp.dg_op_cache_evict(k, v, mass, i32([range(5)]), i32([range(5, 10)]), i32([length]), out_lens, budget, kept, sinks=2 ** 30, recent=2 ** 30 - 1)
    if length < 0:
        with pytest.raises(dgp.DgError):
            dgp.dg_op_status()
    dgp.dg_op_status()
    n = max(length, 0)
    assert out_lens.item() == length and torch.equal(kept[0, 0, :n], torch.arange(n, dtype=torch.int32, device=dev()))
    for part in kept[0, 0, n:].split(2 ** 28):
        assert bool((part == -1).all())
    for x, w in zip((k, v, mass), was):
        flat, old = x.view(10, 1, 64, -1), w.view(10, 1, 64, -1)
        assert torch.equal(flat[:5], old[:5])
        for d in range(5):
            m = min(64, max(0, n - 64 * d))
            assert torch.equal(flat[5 + d, :, :m], old[d, :, :m]) and torch.equal(flat[5 + d, :, m:], old[5 + d, :, m:])


# ---- positions next to 2^31 ----------------------------------------------------------------

LAST = 2 ** 31 - 256        # a sequence ends at or before this slot


class Far:
    """One sequence whose new tokens end at slot `end`: of its table only the pages
    of the first tokens and of the last window are there, the rest names none."""
    HQ, HKV, HD, PG, WINDOW, SINKS = 32, 8, 64, 65536, 8000, 4

    def __init__(self, rng, end, n, most=2 ** 31):
        self.n, self.pre = n, end - n
        first = max(self.pre - self.WINDOW + 1, self.SINKS)
        self.slots = np.concatenate([np.arange(self.SINKS), np.arange(first, end)])
        table = np.full((1, most // self.PG), -9, np.int32)
        there = np.unique(self.slots // self.PG)
        table[0, there] = np.arange(len(there))
        self.table, shape = table, (len(there), self.HKV, self.PG, self.HD)
        k, v = randn(rng, len(self.slots), self.HKV, self.HD), randn(rng, len(self.slots), self.HKV, self.HD)
        self.pools = []
        for x in (k, v):
            pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            place(pool, table[0], self.slots, x)
            self.pools.append(pool.to(dev()))
        self.k, self.v = f64(k), f64(v)
        self.q = randn(rng, n, self.HQ, self.HD)
        self.d = dict(page_tables=i32(table), prefix_lens=i32([self.pre]), offsets=i32([0, n]))
        self.out, self.lse = torch.full((n, self.HQ, self.HD), 7.0, dtype=torch.bfloat16, device=dev()), torch.full((n, self.HQ), 7.0, device=dev())

    def attend(self):
        ws = window_workspace(self.n, 1, self.HQ, self.HKV, self.HD)
        dgp.dg_op_window_attention(self.q.to(dev()), *self.pools, **self.d, out=self.out, workspace=ws, window=self.WINDOW, sinks=self.SINKS,
                                   lse=self.lse)

    def weigh(self, mass, observe=0):
        dgp.dg_op_key_mass(self.q.to(dev()), self.lse, self.pools[0], mass, **self.d,
                           workspace=mass_workspace(self.n, 1, self.HQ, self.HKV, self.HD), window=self.WINDOW, sinks=self.SINKS, observe=observe)

    def scores(self, h):
        s = self.pre + np.arange(self.n)[:, None]
        see = (self.slots <= s) & ((self.slots > s - self.WINDOW) | (self.slots < self.SINKS))
        k, x = self.k[:, h // 4], f64(self.q)[:, h]
        return np.where(see, x @ k.T * self.HD ** -0.5, -np.inf), (np.abs(x) @ np.abs(k).T * self.HD ** -0.5) * see


@pytest.mark.parametrize("end,n,most", [(LAST - d, n, 2 ** 31) for d in (0, 100, 255, 256, 65000) for n in (1, 3, 200)] +
                         [(2 ** 29 - d, 700, 2 ** 29) for d in (0, 200)])        # 700 rows: the kernel for chunks
def test_far_positions(end, n, most):
    far = Far(np.random.default_rng(107), end, n, most)
    far.attend()
    dgp.dg_op_status()
    for h in (0, 3, 28) if n > 3 else range(far.HQ):
        s, mag = far.scores(h)
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        z = m[:, 0] + np.log(e.sum(1))
        e /= e.sum(1, keepdims=True)
        ref = e @ far.v[:, h // 4]
        assert (np.abs(f64(far.out)[:, h] - ref) <= attention_tol(ref, e @ np.abs(far.v[:, h // 4]))).all()
        assert (np.abs(f64(far.lse)[:, h] - z) <= lse_tol(z, mag.max(1), far.HD, 80)).all()
    page, slot = far.table[0, far.slots // far.PG], far.slots % far.PG
    for observe in (0, 1):
        before = np.random.default_rng(108).exponential(1.0, (len(far.pools[0]), far.HKV, far.PG)).astype(np.float32)
        mass = torch.from_numpy(before).to(dev())
        far.weigh(mass, observe)
        dgp.dg_op_status()
        got, rows = mass.cpu().numpy(), slice(n - observe if observe else 0, n)
        still = np.ones(got.shape, bool)
        for g in range(far.HKV):
            seen = np.isfinite(far.scores(4 * g)[0][rows]).any(0) | (far.slots >= far.pre)
            still[page[seen], g, slot[seen]] = False
            if g not in (0, 7):
                continue
            total, err = np.where(far.slots < far.pre, before[page, g, slot].astype(np.float64), 0.0), np.zeros(len(far.slots))
            for h in range(4 * g, 4 * g + 4):
                s, mag = far.scores(h)
                z = f64(far.lse)[rows, h][:, None]
                e = np.exp(s[rows] - z)
                total += e.sum(0)
                err += (e * ((far.HD + 8) * mag[rows] + 8 * np.abs(z) + 100 + n * 4 / 64)).sum(0)   # as for the other batches
            assert (np.abs(got[page, g, slot] - total) <= U32 * (err + 2 * np.abs(total)))[seen].all()
        assert np.array_equal(got.view(np.uint32)[still], before.view(np.uint32)[still])


@pytest.mark.parametrize("n", [1, 200])
def test_sequences_that_end_behind_the_last_position_are_reported(n):
    far = Far(np.random.default_rng(109), LAST, n)
    mass = torch.ones(len(far.pools[0]), far.HKV, far.PG, device=dev())
    far.d["prefix_lens"] += 1
    far.lse.fill_(1.0)
    for call in (far.attend, lambda: far.weigh(mass)):
        call()
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert "sequence" in str(e.value)
    assert (far.out == 7.0).all() and (far.lse == 1.0).all() and (mass == 1.0).all()


# ---- evictions with pages of few slots, and tables that are too short -------------------------

@pytest.mark.parametrize("pg", [1, 2, 3, 12])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_with_small_pages(pg, in_place):
    check_evict(Cache(np.random.default_rng(111), [500, 90, 1300], 3, 64, pg, 150, in_place), 4, 30)


@pytest.mark.parametrize("short", ["page_tables", "out_tables"])
def test_evict_leaves_sequences_that_tables_do_not_hold_alone(short):
    c = Cache(np.random.default_rng(112), [500, 90, 470], 2, 128, 64, 200)
    d, ref = c.on_gpu(), c.ref(2, 20)
    d[short] = d[short][:, :3 if short == "out_tables" else 7].contiguous()       # 192 slots of 200; 448 of 500 and of 470
    dgp.dg_op_cache_evict(**d, budget=200, sinks=2, recent=20)
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert e.value.code == dgp.DG_EINVAL and "sequence" in str(e.value)
    assert d["out_lens"].tolist() == [-1, 90, -1] and (d["kept"][0] == -1).all() and (d["kept"][2] == -1).all()
    assert np.array_equal(d["kept"][1].cpu().numpy(), ref[4][1])
    moved = np.zeros(c.n_pages, bool)
    moved[c.out[1, :2]] = True
    for x, was in ((d["k_pool"], c.k), (d["v_pool"], c.v)):
        assert torch.equal(x.view(torch.int16).cpu()[~moved], was[~moved])
    assert np.array_equal(d["mass_pool"].cpu().numpy()[~moved], c.mass[~moved]) and same_floats(d["mass_pool"].cpu().numpy()[moved], ref[2][moved])


# ---- sequences whose rows lie outside the call's ------------------------------------------------

@pytest.mark.parametrize("pre,new,hkv", [([300, 40, 90], [5, 3, 2], 2), ([300, 40, 90], [900, 400, 70], 16)])     # few rows, chunks
@pytest.mark.parametrize("offsets", ["behind", "before", "descending"])
def test_rows_outside_the_call_are_reported_and_left_alone(pre, new, hkv, offsets):
    rng = np.random.default_rng(113)
    bt = Batch(rng, pre, new, hkv, 64, 64)
    q = randn(rng, bt.T, 2 * hkv, 64).to(dev())
    a, b, c = new[0], new[0] + new[1], sum(new)
    # one sequence's rows outside the call's; and a batch in which it has none, whose work is shared out alike
    off, left = dict(behind=([0, a, b, bt.T + 1], [0, a, b, b]), before=([-1, a, b, c], [a, a, b, c]), descending=([0, a, b, 0], [0, a, b, b]))[offsets]
    before, results = torch.rand(bt.n_pages, hkv, 64, device=dev()), []
    lse = torch.full((bt.T, 2 * hkv), 3.0, device=dev())
    for rows in (left, off):
        out, z, mass = torch.full_like(q, 7.0), torch.full_like(lse, 7.0), before.clone()
        bt.d["offsets"] = i32(rows)
        for call in (lambda: run_window(bt, q, 200, 4, out, z), lambda: run_mass(bt, q, lse, mass, 200, 4)):
            call()
            if rows is off:
                with pytest.raises(dgp.DgError) as e:
                    dgp.dg_op_status()
                assert e.value.code == dgp.DG_EINVAL and "sequence" in str(e.value)
        dgp.dg_op_status()
        results.append((out, z, mass))
    assert all(torch.equal(x, y) for x, y in zip(*results))
    nobodys = slice(0, a) if offsets == "before" else slice(b, None)
    assert (out[nobodys] == 7.0).all() and (z[nobodys] == 7.0).all() and (out[a:b] != 7.0).any() and not torch.equal(mass, before)
