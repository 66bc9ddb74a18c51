"""The operators that serve drafted tokens (per-head norms with rotation, the
rotated append to the paged cache, tree attention, token log probabilities)
against plain numpy evaluations in 64 bits.

Tolerances.  A bf16 result is one rounding away from its fp32 value (2^-8
relative); the terms added to that are stated at each check.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24      # half a step of bf16 and fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from discrete_diffusion_block_gb300 import build
    build.build()
    dgp.load()
    torch.cuda.set_device(0)


@pytest.fixture(autouse=True)
def _clean_status():
    dgp.dg_op_status()
    yield
    dgp.dg_op_status()


def randn(rng, *shape, dtype=torch.bfloat16):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(dev())


# ---- references -------------------------------------------------------------------

def head_ref(x, gain, pos, rope, base=10000.0, eps=1e-6):
    """Norm and rotation in 64 bits: (y, |a| + |b| of the rotated pair)."""
    y = np.array(x, np.float64)
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * gain
    h = rope // 2
    mag = np.abs(y)
    if h:
        ang = np.asarray(pos, np.float64)[:, None] * base ** (-np.arange(h) * 2.0 / rope)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[..., :h].copy(), y[..., h:rope].copy()
        y[..., :h], y[..., h:rope] = a * c - b * s, b * c + a * s
        mag[..., :h] = mag[..., h:rope] = np.abs(a) + np.abs(b)
    return y, mag


def head_tol(y, mag):
    # norm: at most 21 roundings of the sum, rsqrt within 2 ulp, two products;
    # angle within 2^-25 half turns, sine and cosine within 2 ulp, two products and a sum
    return U16 * np.abs(y) + 64 * U32 * mag


def pool_rows(pool):
    """[n_pages][Hkv][pg][hd] pool tensor -> logical [n_pages][pg][Hkv][hd]
    (16-byte chunk c of slot s of a 64-wide sub-block is stored at c ^ (s % 8))."""
    x = pool.cpu().numpy() if isinstance(pool, torch.Tensor) else pool
    P, H, pg, hd = x.shape
    x = x.reshape(P, H, hd // 64, pg, 8, 8)
    at = np.arange(8)[None] ^ (np.arange(pg)[:, None] % 8)
    x = np.take_along_axis(x, np.broadcast_to(at[None, None, None, :, :, None], x.shape), axis=4)
    return x.transpose(0, 3, 1, 2, 4, 5).reshape(P, pg, H, hd)


class Batch:
    """Uneven sequences over shuffled pages: lengths, tables, pools. Slots that
    belong to no sequence hold NaN."""

    def __init__(self, rng, pre, new, hkv, hd, pg, spare=1, pad=2, fill=True):
        self.pre, self.new, self.hkv, self.hd, self.pg = list(pre), list(new), hkv, hd, pg
        need = [-(-(p + n) // pg) for p, n in zip(pre, new)]
        self.n_pages = sum(need) + spare
        perm = rng.permutation(self.n_pages)
        self.max_pages = max(max(need, default=0), 1) + 1
        self.table = np.full((len(self.pre), self.max_pages), -7, np.int32)     # entries behind a sequence are never read
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.off[-1]) + pad
        self.d = dict(page_tables=i32(self.table), prefix_lens=i32(self.pre), offsets=i32(self.off))
        shape = (self.n_pages, hkv, pg, hd)
        self.k_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.v_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.keys, self.vals = [], []
        if fill:
            for b in range(len(self.pre)):
                n = self.pre[b] + self.new[b]
                k, v = randn(rng, n, hkv, hd), randn(rng, n, hkv, hd)
                self.keys.append(f64(k))
                self.vals.append(f64(v))
                for pool, x in ((self.k_pool, k), (self.v_pool, v)):
                    self.place(pool, b, np.arange(n), x)
        self.k_pool, self.v_pool = self.k_pool.to(dev()), self.v_pool.to(dev())

    def place(self, pool, b, slots, x):
        for r, p in enumerate(slots):
            page, s = int(self.table[b, p // self.pg]), p % self.pg
            c = torch.from_numpy(np.arange(8) ^ (s % 8))
            flat = pool[page].view(self.hkv, self.hd // 64, self.pg, 8, 8)
            flat[:, :, s, c] = x[r].view(self.hkv, self.hd // 64, 8, 8)


def random_trees(rng, new, T, words=None, chain=False):
    words = words or max(1, -(-max(new, default=1) // 64))
    m = np.zeros((T, words), np.uint64)
    t0 = 0
    for n in new:
        for j in range(n):
            parent = j - 1 if chain else int(rng.integers(-1, j)) if j else -1
            if parent >= 0:
                m[t0 + j] = m[t0 + parent]
            m[t0 + j, j // 64] |= np.uint64(1 << (j % 64))
        t0 += n
    return m


def attention_ref(q, bt, mask, scale):
    """(out, sum_j p_j |v_j|) in 64 bits for the live rows; rows that see nothing are 0."""
    hq = q.shape[1]
    G = hq // bt.hkv
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        t0 = int(bt.off[b])
        for t in range(n):
            if mask is None:
                see = np.arange(n) <= t
            else:
                see = np.array([j < 64 * mask.shape[1] and bool((int(mask[t0 + t, j // 64]) >> (j % 64)) & 1) for j in range(n)], bool)
            idx = np.concatenate([np.arange(p), p + np.nonzero(see)[0]])
            if len(idx) == 0:
                continue
            k, v = bt.keys[b][idx], bt.vals[b][idx]
            for g in range(bt.hkv):
                s = q[t0 + t, g * G:(g + 1) * G] @ k[:, g].T * scale
                e = np.exp(s - s.max(1, keepdims=True))
                e /= e.sum(1, keepdims=True)
                out[t0 + t, g * G:(g + 1) * G] = e @ v[:, g]
                mag[t0 + t, g * G:(g + 1) * G] = e @ np.abs(v[:, g])
    return out, mag


def attention_tol(ref, mag):
    # the output's rounding, the probabilities' roundings to bf16 (numerator
    # and sum), and 1e-3 of that for fp32 scores and exponentials
    return U16 * np.abs(ref) + 2.002 * U16 * mag + 1e-6


# ---- norms and rotation --------------------------------------------------------------

@pytest.mark.parametrize("T,hq,hkv,hd,rope,f32,normed,packed", [
    (1, 16, 8, 128, 128, False, True, False),
    (1, 1, 1, 64, 64, True, True, False),
    (37, 16, 8, 128, 128, False, True, True),
    (37, 4, 2, 64, 32, True, True, True),
    (5, 5, 5, 64, 64, False, False, True),
    (129, 6, 3, 256, 256, False, True, False),
    (19, 3, 1, 256, 16, True, True, True),
    (33, 7, 1, 128, 0, False, True, False),
    (2048, 12, 4, 64, 64, False, True, True),
    (301, 16, 4, 128, 64, True, False, False),
    (1000, 1, 0, 128, 128, False, True, False),
    (3, 0, 2, 128, 48, False, True, False),
])
def test_qk_norm_rope(T, hq, hkv, hd, rope, f32, normed, packed):
    rng = np.random.default_rng(T + hq + hd)
    dt = torch.float32 if f32 else torch.bfloat16
    if packed:
        rows = randn(rng, T, hq + 2 * hkv + 1, hd, dtype=dt).to(dev())
        q, k = rows[:, 1:1 + hq], rows[:, 1 + hq:1 + hq + hkv]
    else:
        q, k = randn(rng, T, hq, hd, dtype=dt).to(dev()), randn(rng, T, hkv, hd, dtype=dt).to(dev())
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[0] = 0
    gains = [randn(rng, hd, dtype=torch.float32).to(dev()) if normed else None for _ in range(2)]
    outs = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device=dev()) for x in (q, k)]
    dgp.dg_op_qk_norm_rope(q if hq else None, k if hkv else None, i32(pos), outs[0] if hq else None, outs[1] if hkv else None,
                           q_gain=gains[0], k_gain=gains[1], rope_dim=rope)
    for x, g, o in zip((q, k), gains, outs):
        if not x.shape[1]:
            continue
        y, mag = head_ref(f64(x), None if g is None else f64(g), pos, rope)
        assert (np.abs(f64(o) - y) <= head_tol(y, mag)).all()


def test_qk_norm_rope_in_place_one_side_normed_and_extreme_positions():
    rng = np.random.default_rng(3)
    T, hq, hkv, hd = 17, 4, 2, 128
    rows = randn(rng, T, hq + 2 * hkv, hd).to(dev())
    was = rows.clone()
    pos = np.array([0, 1, 2 ** 31 - 1, 2 ** 30, -5] + list(range(12)), np.int32)
    gain = randn(rng, hd, dtype=torch.float32).to(dev())
    q, k = rows[:, :hq], rows[:, hq:hq + hkv]
    dgp.dg_op_qk_norm_rope(q, k, i32(pos), q, k, q_gain=gain, k_gain=None)
    for lo, hi, g in ((0, hq, f64(gain)), (hq, hq + hkv, None)):
        y, mag = head_ref(f64(was[:, lo:hi]), g, pos, hd)
        # the reference's own angle, pos * freq in 64 bits, is off by pos * 2^-53
        assert (np.abs(f64(rows[:, lo:hi]) - y) <= head_tol(y, mag) + 2.0 ** -21 * mag).all()
    assert torch.equal(rows[:, hq + hkv:], was[:, hq + hkv:])


def test_qk_norm_rope_zero_rows_and_nonfinite_heads_stay_apart():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=dev())
    x[1, 0, 5] = float("inf")
    x[2, 1, 7] = float("nan")
    o = torch.full_like(x, 3.0)
    g = torch.ones(64, device=dev())
    dgp.dg_op_qk_norm_rope(x, None, i32([0, 1, 2, 3]), o, None, q_gain=g)
    fine = torch.ones(4, 2, dtype=torch.bool)
    fine[1, 0] = fine[2, 1] = False
    assert (o.cpu()[fine] == 0).all()
    assert torch.isnan(o[2, 1]).all()
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=dev())
    dgp.dg_op_qk_norm_rope(e, None, i32([]), e.clone(), None, q_gain=g)


# ---- append ------------------------------------------------------------------------

@pytest.mark.parametrize("pre,new,hkv,hd,pg,rope,normed,own_pos", [
    ([0], [1], 2, 64, 64, 64, True, False),
    ([127], [3], 8, 128, 128, 128, True, True),
    ([5, 0, 300, 64, 0], [1, 0, 70, 64, 2], 3, 64, 64, 32, False, True),
    ([190, 191, 192, 1], [5, 5, 0, 400], 2, 256, 192, 256, True, False),
    ([10] * 70, list(range(70)), 1, 128, 128, 0, False, False),
    ([3] * 300, [1] * 300, 4, 64, 8, 64, False, False),
])
def test_rope_kv_append(pre, new, hkv, hd, pg, rope, normed, own_pos):
    rng = np.random.default_rng(sum(pre) + sum(new))
    bt = Batch(rng, pre, new, hkv, hd, pg, fill=False)
    rows = randn(rng, bt.T, 2 * hkv, hd).to(dev())
    k, v = rows[:, :hkv], rows[:, hkv:]
    gain = randn(rng, hd, dtype=torch.float32).to(dev()) if normed else None
    slots = np.concatenate([np.arange(p, p + n) for p, n in zip(pre, new)] + [[0, 0]]).astype(np.int64)
    pos = rng.integers(0, 1 << 20, bt.T) if own_pos else slots
    sentinel = 0x7FC1
    for pool in (bt.k_pool, bt.v_pool):
        pool.view(torch.int16).fill_(sentinel)
    dgp.dg_op_rope_kv_append(k, v, bt.k_pool, bt.v_pool, **bt.d, positions=i32(pos) if own_pos else None, k_gain=gain, rope_dim=rope)
    y, mag = head_ref(f64(k), None if gain is None else f64(gain), pos, rope)
    kp, vp = (pool_rows(p.view(torch.int16).cpu().numpy()) for p in (bt.k_pool, bt.v_pool))
    left = np.ones(kp.shape[:2], bool)
    for b, (p, n) in enumerate(zip(pre, new)):
        for i in range(n):
            page, s, t = bt.table[b, (p + i) // pg], (p + i) % pg, bt.off[b] + i
            left[page, s] = False
            got = (kp[page, s].view(np.uint16).astype(np.uint32) << 16).view(np.float32)
            assert (np.abs(got - y[t]) <= head_tol(y[t], mag[t])).all()
            assert np.array_equal(vp[page, s], v[t].view(torch.int16).cpu().numpy())
    assert (kp[left] == sentinel).all() and (vp[left] == sentinel).all()


def test_append_reports_slots_outside_the_table_and_bad_pages():
    rng = np.random.default_rng(5)
    bt = Batch(rng, [60, 100], [10, 6], 2, 64, 64, fill=False)
    bt.k_pool.zero_()
    bt.v_pool.zero_()
    k = randn(rng, bt.T, 2, 64).to(dev())
    bad = bt.table.copy()
    bad[0, 1] = bt.n_pages          # slots 64.. of sequence 0
    args = dict(prefix_lens=bt.d["prefix_lens"], offsets=bt.d["offsets"])
    dgp.dg_op_rope_kv_append(k, k, bt.k_pool, bt.v_pool, i32(bad), **args)
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert e.value.code == dgp.DG_EINVAL
    assert int((pool_rows(bt.v_pool.float()).reshape(-1, 2, 64) != 0).any((1, 2)).sum()) == 4 + 6
    args["prefix_lens"] = i32([10 ** 9, -4])        # behind the table; partly before it
    bt.k_pool.zero_()
    bt.v_pool.zero_()
    dgp.dg_op_rope_kv_append(k, k, bt.k_pool, bt.v_pool, bt.d["page_tables"], **args)
    with pytest.raises(dgp.DgError):
        dgp.dg_op_status()
    assert int((pool_rows(bt.v_pool.float()).reshape(-1, 2, 64) != 0).any((1, 2)).sum()) == 2


# ---- tree attention ------------------------------------------------------------------

def run_attention(bt, q, mask, out, scale=None, stream=None, workspace=None):
    n = dgp.dg_op_tree_attention_workspace_bytes(q.shape[0], len(bt.pre), q.shape[1], bt.hkv, bt.hd)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device=dev()) if workspace is None else workspace
    m = None if mask is None else torch.from_numpy(mask.view(np.int64)).to(dev())
    dgp.dg_op_tree_attention(q, bt.k_pool, bt.v_pool, **bt.d, tree_mask=m, out=out, workspace=ws, scale=scale, stream=stream)


def check_attention(bt, hq, mask, rng, scale=None, strided=False):
    if strided:
        q = randn(rng, bt.T, hq + 3, bt.hd).to(dev())[:, 1:1 + hq]
        out = torch.full((bt.T, 2 * hq, bt.hd), 7.0, dtype=torch.bfloat16, device=dev())[:, hq:]
    else:
        q = randn(rng, bt.T, hq, bt.hd).to(dev())
        out = torch.full((bt.T, hq, bt.hd), 7.0, dtype=torch.bfloat16, device=dev())
    run_attention(bt, q, mask, out, scale)
    dgp.dg_op_status()
    ref, mag = attention_ref(f64(q), bt, mask, bt.hd ** -0.5 if scale is None else scale)
    n = int(bt.off[-1])
    got = f64(out)
    assert (np.abs(got[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all(), np.abs(got[:n] - ref[:n]).max()
    assert (got[n:] == 7.0).all()           # rows behind the last sequence
    return q, out


@pytest.mark.parametrize("hq,hkv,hd,pg", [(16, 8, 128, 128), (4, 2, 64, 64), (12, 4, 64, 192), (8, 1, 128, 64), (5, 5, 64, 128), (7, 1, 128, 128)])
@pytest.mark.parametrize("pre", [0, 1, 63, 64, 65, 127, 128, 129, 700])
def test_single_token_decode(hq, hkv, hd, pg, pre):
    rng = np.random.default_rng(pre)
    check_attention(Batch(rng, [pre], [1], hkv, hd, pg), hq, None, rng)


@pytest.mark.parametrize("hq,hkv,hd,pg,pre,new", [
    (16, 8, 128, 128, [300], [17]),
    (16, 8, 128, 128, [0, 2000, 130], [64, 3, 0]),
    (12, 4, 64, 64, [100, 0, 5, 640, 0], [5, 1, 0, 33, 2]),
    (16, 4, 128, 192, [190, 191], [63, 66]),
    (32, 1, 64, 64, [70], [9]),
    (6, 2, 64, 128, [0], [200]),
    (7, 1, 128, 64, [11] * 40, [j % 5 for j in range(40)]),
    (4, 2, 64, 64, [j * 7 for j in range(200)], [1] * 200),
    (128, 1, 64, 64, [20, 64], [3, 1]),
])
@pytest.mark.parametrize("masked", [False, True])
def test_batches_of_trees(hq, hkv, hd, pg, pre, new, masked):
    rng = np.random.default_rng(len(pre) + hq)
    bt = Batch(rng, pre, new, hkv, hd, pg)
    check_attention(bt, hq, random_trees(rng, new, bt.T) if masked else None, rng, strided=masked)


def test_long_context_and_scale():
    rng = np.random.default_rng(11)
    bt = Batch(rng, [20011], [2], 2, 128, 128)
    check_attention(bt, 4, None, rng, scale=0.3)


def test_rows_that_see_nothing_short_masks_and_keys_nobody_sees():
    rng = np.random.default_rng(12)
    bt = Batch(rng, [0, 0, 40], [6, 70, 70], 2, 64, 64)
    mask = np.zeros((bt.T, 1), np.uint64)
    mask[2, 0] = 1 << 5                     # a row that sees a later key only
    mask[7, 0] = 0xFFFFFFFFFFFFFFFF         # keys past the mask's 64 bits stay hidden
    check_attention(bt, 4, mask, rng)


def test_large_and_equal_scores():
    # scores of +-hundreds: the running maximum moves over many tiles; equal
    # keys: every weight the same
    rng = np.random.default_rng(13)
    bt = Batch(rng, [900], [4], 1, 64, 64)
    q = randn(rng, bt.T, 2, 64)
    up = torch.linspace(-1, 1, 904)[:, None, None] * 2.0
    k = up.expand(904, 1, 64).to(torch.bfloat16)
    pool = torch.full(bt.k_pool.shape, float("nan"), dtype=torch.bfloat16)
    bt.place(pool, 0, np.arange(904), k)
    bt.k_pool = pool.to(dev())
    bt.keys[0] = f64(k)
    q[0], q[1], q[2] = 30.0, -30.0, 0.0
    out = torch.zeros(bt.T, 2, 64, dtype=torch.bfloat16, device=dev())
    run_attention(bt, q.to(dev()), None, out)
    ref, mag = attention_ref(f64(q), bt, None, 0.125)
    # a score of 480 carries 64 fp32 roundings: its exponential 480 * 2^-18
    assert (np.abs(f64(out)[:4] - ref[:4]) <= attention_tol(ref[:4], mag[:4]) + 480 * 2.0 ** -18 * mag[:4]).all()


def test_attention_repeats_bit_for_bit_and_ignores_the_workspace_contents():
    rng = np.random.default_rng(14)
    bt = Batch(rng, [3000, 10, 777], [20, 1, 8], 4, 128, 128)
    q = randn(rng, bt.T, 8, 128).to(dev())
    outs = []
    for fill in (0, 0xFF, 0x7F):
        n = dgp.dg_op_tree_attention_workspace_bytes(bt.T, 3, 8, 4, 128)
        ws = torch.full((max(n, 1),), fill, dtype=torch.uint8, device=dev())
        out = torch.zeros(bt.T, 8, 128, dtype=torch.bfloat16, device=dev())
        run_attention(bt, q, None, out, workspace=ws)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("hq,hkv,hd,pre,new", [
    (12, 4, 64, [100 + 37 * j for j in range(40)], [1 + j % 5 for j in range(40)]),
    (16, 8, 128, [9000, 3, 700, 0, 2500], [24, 1, 7, 13, 30]),
    (4, 1, 64, [40000], [33]),
    (8, 8, 128, [2048], [1]),
    (16, 8, 128, [2000 + 3 * j for j in range(16)], [1] * 16),
    (8, 2, 128, [4000, 4100], [61, 33]),
    (4, 1, 64, [9000, 100], [3, 40]),
    (6, 3, 64, [500, 130, 400, 1], [2, 2, 2, 2]),
])
def test_attention_replayed_many_times_repeats_bit_for_bit(hq, hkv, hd, pre, new):
    # units that span several blocks are joined between the blocks: a captured
    # call, and calls in a row on one workspace, must find its flags down
    rng = np.random.default_rng(16)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    q, out = check_attention(bt, hq, None, rng)
    n = dgp.dg_op_tree_attention_workspace_bytes(bt.T, len(pre), hq, hkv, hd)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())
    again = torch.empty_like(out)
    for _ in range(20):
        again.fill_(7.0)
        run_attention(bt, q, None, again, workspace=ws)
        assert torch.equal(again, out)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        for _ in range(3):
            run_attention(bt, q, None, again, workspace=ws, stream=st)
    for _ in range(50):
        again.fill_(7.0)
        g.replay()
        assert torch.equal(again, out)


def test_attention_reports_bad_pages_and_bad_sequences():
    rng = np.random.default_rng(15)
    bt = Batch(rng, [200, 50], [2, 3], 2, 64, 64)
    q = randn(rng, bt.T, 4, 64).to(dev())
    good = torch.zeros(bt.T, 4, 64, dtype=torch.bfloat16, device=dev())
    run_attention(bt, q, None, good)
    for entry, words in (((0, 1, bt.n_pages), "page"), ((0, 0, -1), "page")):
        bad = bt.table.copy()
        bad[entry[0], entry[1]] = entry[2]
        out = torch.zeros_like(good)
        run = dict(bt.d, page_tables=i32(bad))
        keep, bt.d = bt.d, run
        run_attention(bt, q, None, out)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_EINVAL and words in str(e.value)
        assert torch.isfinite(out.float()).all() and torch.equal(out[2:5], good[2:5])
    for change in (dict(prefix_lens=i32([10 ** 6, 50])), dict(prefix_lens=i32([-1, 50])), dict(prefix_lens=i32([2 ** 31 - 1, 50]))):
        out = torch.full_like(good, 7.0)
        keep, bt.d = bt.d, dict(bt.d, **change)
        run_attention(bt, q, None, out)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert "sequence" in str(e.value)
        assert (out[:2] == 7.0).all() and torch.equal(out[2:5], good[2:5])


# ---- log probabilities -----------------------------------------------------------------

def logprob_ref(x, tokens, k, inv_tau):
    y = (x.astype(np.float32) * np.float32(inv_tau)).astype(np.float64)
    with np.errstate(all="ignore"):
        m = y.max(1, keepdims=True)
        m0 = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(y - m0)
        S = e.sum(1, keepdims=True)
        lse = np.where(np.isneginf(m), -np.inf, m0 + np.log(np.where(S > 0, S, 1.0)))
        lp = np.where(np.isneginf(y), -np.inf, y - np.where(np.isneginf(m), 0.0, lse))
        H = -np.where(e > 0, e / np.where(S > 0, S, 1.0) * np.where(np.isneginf(y), 0.0, lp), 0.0).sum(1)
    ids = np.argsort(-x.astype(np.float64), axis=1, kind="stable")[:, :k]
    rows = np.arange(len(x))[:, None]
    given = np.where(tokens == -1, 0.0, lp[rows, np.clip(tokens, 0, None)])
    return given, H, lse[:, 0], ids, lp[rows, ids]


def run_logprobs(x, tokens, k, inv_tau=1.0, stream=None):
    T, n = tokens.shape
    f = lambda *s: torch.full(s, 9.0, dtype=torch.float32, device=dev())  # noqa: E731
    o = dict(logprobs=f(T, n), entropy=f(T), lse=f(T), top_ids=torch.full((T, k), -9, dtype=torch.int32, device=dev()), top_logprobs=f(T, k))
    dgp.dg_op_token_logprobs(x, i32(tokens), **o, inv_tau=inv_tau, stream=stream)
    return [o[n].cpu().numpy() for n in ("logprobs", "entropy", "lse", "top_ids", "top_logprobs")]


def check_logprobs(x, tokens, k, inv_tau=1.0):
    got = run_logprobs(x, tokens, k, inv_tau)
    dgp.dg_op_status()
    ref = logprob_ref(x.float().cpu().numpy(), tokens, k, inv_tau)
    V = x.shape[1]
    assert np.array_equal(got[3], ref[3])
    # sums of V exponentials in fp32, at most V / 256 + 64 roundings deep, four
    # to a step (exponential, rescale, product, sum); then the log, the
    # difference and the result's own rounding
    depth = 4 * (V / 256 + 64) * U32
    for g, r, scale in ((got[0], ref[0], 0.0), (got[1], ref[1], 1.0), (got[2], ref[2], 0.0), (got[4], ref[4], 0.0)):
        same = np.isneginf(r) | np.isneginf(g)
        assert np.array_equal(np.isneginf(r), np.isneginf(g))
        with np.errstate(invalid="ignore"):
            err = np.where(same, 0.0, np.abs(g - r))
        size = np.where(same, 0.0, np.abs(np.where(same, 0.0, r)))
        ymax = np.where(np.isfinite(ref[2]), np.abs(ref[2]), 0.0).max() + 8
        assert (err <= depth * (1 + scale * (size + 12)) + 4 * U32 * (size + ymax)).all(), err.max()


@pytest.mark.parametrize("T,V,n,k,bf16,tau", [
    (1, 1, 1, 1, False, 1.0),
    (1, 262144, 1, 8, False, 1.0),
    (3, 1000, 2, 32, False, 0.7),
    (7, 50001, 3, 5, True, 1.5),
    (300, 777, 1, 20, True, 1.0),
    (2, 31, 4, 31, False, 1.0),
    (5, 33, 0, 32, True, 1.0),
    (20, 4096, 1, 0, False, 2.0),
    (1, 131073, 1, 32, True, 1.0),
    (40, 30000, 1, 3, False, 1.0),
    (170, 20000, 1, 3, False, 1.0),
])
def test_token_logprobs(T, V, n, k, bf16, tau):
    rng = np.random.default_rng(V + T)
    x = torch.from_numpy((rng.standard_normal((T, V)) * 3).astype(np.float32))
    x = (x.to(torch.bfloat16) if bf16 else x).to(dev())
    tokens = rng.integers(0, V, (T, n))
    if n > 1:
        tokens[0, 1] = -1
    check_logprobs(x, tokens, k, 1.0 / tau)


@pytest.mark.parametrize("bf16", [False, True])
def test_logprobs_of_strided_rows_at_every_alignment(bf16):
    rng = np.random.default_rng(21)
    base = torch.from_numpy((rng.standard_normal((6, 3001)) * 4).astype(np.float32))
    base = (base.to(torch.bfloat16) if bf16 else base).to(dev())
    for lo in range(0, 9):
        for V in (1, 2, 15, 1000, 2990):
            check_logprobs(base[:, lo:lo + V], rng.integers(0, V, (6, 1)), min(V, 6))


@pytest.mark.parametrize("bf16", [False, True])
def test_logprobs_ties_order_and_masks(bf16):
    V = 5000
    rng = np.random.default_rng(22)
    rows = [np.zeros(V), np.arange(V) / 64.0, -np.arange(V) / 64.0, np.where(np.arange(V) % 2, 0.0, -0.0),
            np.full(V, -np.inf), np.where(np.arange(V) < V - 3, -np.inf, 1.0), np.full(V, -3.0e38),
            np.where(rng.random(V) < 0.9, -np.inf, rng.integers(0, 3, V) * 1.0), np.where(np.arange(V) == 4321, 80.0, -80.0)]
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    x = (x.to(torch.bfloat16) if bf16 else x).to(dev())
    tokens = rng.integers(0, V, (len(rows), 3))
    tokens[:, 1], tokens[8, 2] = V - 1, 4321
    check_logprobs(x, tokens, 32)


def test_logprobs_nan_inf_and_tokens_outside_the_vocabulary():
    V = 3000
    x = torch.zeros(4, V, device=dev())
    x[1, 77] = float("nan")
    x[2, 5] = float("inf")
    tokens = np.array([[0, -1], [0, -1], [5, -1], [V, -2]])
    lp, H, lse, ids, top = run_logprobs(x, tokens, 4)
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert e.value.code == dgp.DG_EINVAL and "token" in str(e.value)
    assert np.isfinite(lp[0]).all() and np.isnan(lp[1:3, 0]).all() and np.isnan(lp[3]).all()
    assert (lp[:3, 1] == 0).all()
    assert np.isnan(H[1:3]).all() and np.isnan(lse[1:3]).all() and np.isnan(top[1:3]).all()
    assert np.isfinite(H[[0, 3]]).all() and np.isfinite(lse[[0, 3]]).all()
    assert np.array_equal(ids[0], [0, 1, 2, 3]) and np.array_equal(ids[2], [5, 0, 1, 2])
    assert np.array_equal(ids[1], [0, 1, 2, 3])


# ---- together, on other streams, captured ---------------------------------------------------

class Step:
    """One layer of checking drafted trees: packed QKV rows -> queries normed
    and rotated, keys and values appended, attention, a vocabulary product,
    log probabilities."""
    HQ, HKV, HD, PG, V = 8, 4, 64, 64, 1500

    def __init__(self, rng, pre, new, pad):
        self.rng = rng
        self.bt = Batch(rng, pre, new, self.HKV, self.HD, self.PG, pad=pad)
        bt, H = self.bt, self.HQ + 2 * self.HKV
        self.mask = random_trees(rng, new, bt.T)
        depth = np.array([sum(bin(int(w)).count("1") for w in row) for row in self.mask]) - 1
        base = np.concatenate([np.repeat(pre, new), np.zeros(pad, np.int64)])
        self.pos = np.maximum(base + depth, 0)
        self.rows = randn(rng, bt.T, H, self.HD).to(dev())
        self.gq, self.gk = (randn(rng, self.HD, dtype=torch.float32).to(dev()) for _ in range(2))
        self.head = (randn(rng, self.HQ * self.HD, self.V, dtype=torch.float32) * 0.3).to(dev())
        self.tokens = rng.integers(0, self.V, (bt.T, 1))
        self.d = dict(pos=i32(self.pos), tokens=i32(self.tokens), mask=torch.from_numpy(self.mask.view(np.int64)).to(dev()))
        f = lambda *s: torch.zeros(*s, dtype=torch.float32, device=dev())  # noqa: E731
        T = bt.T
        self.q = torch.zeros(T, self.HQ, self.HD, dtype=torch.bfloat16, device=dev())
        self.out = torch.zeros_like(self.q)
        self.logits = f(T, self.V)
        self.lp, self.H, self.ids = f(T, 1), f(T), torch.zeros(T, 4, dtype=torch.int32, device=dev())
        n = dgp.dg_op_tree_attention_workspace_bytes(T, len(pre), self.HQ, self.HKV, self.HD)
        self.ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev())

    def run(self, stream=None):
        bt = self.bt
        dgp.dg_op_qk_norm_rope(self.rows[:, :self.HQ], None, self.d["pos"], self.q, None, q_gain=self.gq, stream=stream)
        dgp.dg_op_rope_kv_append(self.rows[:, self.HQ:self.HQ + self.HKV], self.rows[:, self.HQ + self.HKV:], bt.k_pool, bt.v_pool, **bt.d,
                                 positions=self.d["pos"], k_gain=self.gk, stream=stream)
        dgp.dg_op_tree_attention(self.q, bt.k_pool, bt.v_pool, **bt.d, tree_mask=self.d["mask"], out=self.out, workspace=self.ws, stream=stream)
        torch.mm(self.out.view(bt.T, -1).float(), self.head, out=self.logits)
        dgp.dg_op_token_logprobs(self.logits, self.d["tokens"], self.lp, self.H, None, self.ids, None, stream=stream)

    def check(self):
        bt = self.bt
        n = int(bt.off[-1])
        rows = f64(self.rows)
        q, qm = head_ref(rows[:, :self.HQ], f64(self.gq), self.pos, self.HD)
        got_q = f64(self.q)
        assert (np.abs(got_q - q) <= head_tol(q, qm)).all()
        k, km = head_ref(rows[:, self.HQ:self.HQ + self.HKV], f64(self.gk), self.pos, self.HD)
        kp, vp = pool_rows(bt.k_pool.float()), pool_rows(bt.v_pool.float())
        for b, (p, m) in enumerate(zip(bt.pre, bt.new)):
            for i in range(m):
                t, page, s = bt.off[b] + i, bt.table[b, (p + i) // self.PG], (p + i) % self.PG
                assert (np.abs(kp[page, s] - k[t]) <= head_tol(k[t], km[t])).all()
                assert np.array_equal(vp[page, s], rows[t, self.HQ + self.HKV:])
                bt.keys[b][p + i], bt.vals[b][p + i] = kp[page, s], vp[page, s]
        ref, mag = attention_ref(got_q, bt, self.mask, self.HD ** -0.5)     # each stage on the values it was given
        assert (np.abs(f64(self.out)[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all()
        lg = self.logits.cpu().numpy()
        given, H, _, ids, _ = logprob_ref(lg, self.tokens, 4, 1.0)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        assert np.abs(self.lp.cpu().numpy() - given).max() <= 1e-4 and np.abs(self.H.cpu().numpy() - H).max() <= 1e-4


def test_the_operators_together():
    rng = np.random.default_rng(31)
    s = Step(rng, [100, 0, 333, 64], [9, 1, 40, 0], pad=6)
    s.run()
    dgp.dg_op_status()
    s.check()


def test_the_operators_on_another_stream_and_two_at_once():
    rng = np.random.default_rng(32)
    steps = [Step(rng, [500, 20], [30, 3], pad=1), Step(rng, [90, 1000, 4], [1, 17, 5], pad=1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run(stream=st)
    torch.cuda.synchronize()
    dgp.dg_op_status()
    for s in steps:
        s.check()


def test_the_operators_captured_and_replayed_with_other_lengths():
    # a captured step of up to 24 packed rows serves other sequences: new
    # lengths, offsets, tables and inputs are written into the same tensors
    rng = np.random.default_rng(33)
    s = Step(rng, [900, 700, 333], [9, 1, 10], pad=4)
    s.run()
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        s.run(stream=st)
    for pre, new in (([100, 0, 333], [9, 1, 10]), ([64, 900, 1], [3, 16, 0]), ([0, 0, 0], [0, 0, 1])):
        t = Step(rng, pre, new, pad=24 - sum(new))
        assert t.bt.n_pages <= s.bt.n_pages and t.bt.max_pages <= s.bt.max_pages
        table = np.full(s.bt.table.shape, -7, np.int32)
        table[:, :t.bt.max_pages] = t.bt.table
        for name, v in (("page_tables", i32(table)), ("prefix_lens", t.bt.d["prefix_lens"]), ("offsets", t.bt.d["offsets"])):
            s.bt.d[name].copy_(v)
        for name in ("pos", "tokens", "mask"):
            s.d[name].copy_(t.d[name])
        for name in ("rows", "gq", "gk", "head"):
            getattr(s, name).copy_(getattr(t, name))
        for name in ("k_pool", "v_pool"):
            getattr(s.bt, name)[:t.bt.n_pages].copy_(getattr(t.bt, name))
        g.replay()
        torch.cuda.synchronize()
        dgp.dg_op_status()
        for name in ("q", "out", "logits", "lp", "H", "ids"):
            getattr(t, name).copy_(getattr(s, name))
        for name in ("k_pool", "v_pool"):
            getattr(t.bt, name).copy_(getattr(s.bt, name)[:t.bt.n_pages])
        t.check()


# ---- calls at the edges of what the documentation allows ----------------------------------------

@pytest.mark.parametrize("T,hq,hkv,hd,rope,f32", [
    (1, 130, 7, 64, 64, False), (3, 1, 33, 256, 256, False), (2, 40, 40, 128, 96, True), (2433, 3, 1, 64, 48, False),
    (4865, 17, 1, 128, 128, False), (5000, 2, 2, 64, 64, True), (700, 1, 9, 256, 32, True),
])
def test_qk_norm_rope_with_tokens_split_and_in_turns(T, hq, hkv, hd, rope, f32):
    # a token's heads over several warps, warps with many tokens, groups of heads partly filled
    rng = np.random.default_rng(T + 7 * hq)
    dt = torch.float32 if f32 else torch.bfloat16
    q, k = randn(rng, T, hq, hd, dtype=dt).to(dev()), randn(rng, T, hkv, hd, dtype=dt).to(dev())
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    gain = randn(rng, hd, dtype=torch.float32).to(dev())
    qo, ko = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device=dev()) for x in (q, k))
    dgp.dg_op_qk_norm_rope(q, k, i32(pos), qo, ko, q_gain=None, k_gain=gain, rope_dim=rope)
    for x, g, o in ((q, None, qo), (k, f64(gain), ko)):
        y, mag = head_ref(f64(x), g, pos, rope)
        assert (np.abs(f64(o) - y) <= head_tol(y, mag)).all()


def shifted(bt, by):
    """The batch's rows behind `by` rows that belong to no sequence."""
    bt.off = bt.off + by
    bt.T += by
    bt.d["offsets"] = i32(bt.off)
    return bt


def test_rows_before_the_first_sequence_take_no_part():
    rng = np.random.default_rng(41)
    bt = shifted(Batch(rng, [200, 70], [9, 4], 2, 64, 64), 3)
    q = randn(rng, bt.T, 4, 64).to(dev())
    out = torch.full((bt.T, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
    run_attention(bt, q, None, out)
    ref, mag = attention_ref(f64(q), bt, None, 64 ** -0.5)
    lo, hi = int(bt.off[0]), int(bt.off[-1])
    got = f64(out)
    assert (np.abs(got - ref)[lo:hi] <= attention_tol(ref[lo:hi], mag[lo:hi])).all()
    assert (got[:lo] == 7.0).all() and (got[hi:] == 7.0).all()
    rows = randn(rng, bt.T, 2, 64).to(dev())
    rows[:lo] = float("nan")
    was = bt.v_pool.clone()
    dgp.dg_op_rope_kv_append(rows, rows, bt.k_pool, bt.v_pool, **bt.d)
    dgp.dg_op_status()
    vp, old = pool_rows(bt.v_pool.float()), pool_rows(was.float())
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        for i in range(n):
            page, s = bt.table[b, (p + i) // 64], (p + i) % 64
            assert np.array_equal(vp[page, s], f64(rows)[bt.off[b] + i])
            old[page, s] = vp[page, s]
    assert np.array_equal(vp, old, equal_nan=True)


def test_thousands_of_short_sequences():
    rng = np.random.default_rng(42)
    pre, new = rng.integers(0, 5, 3000), rng.integers(0, 3, 3000)
    bt = Batch(rng, pre, new, 1, 64, 64)
    check_attention(bt, 2, None, rng)
    rows = randn(rng, bt.T, 1, 64).to(dev())
    dgp.dg_op_rope_kv_append(rows, rows, bt.k_pool, bt.v_pool, **bt.d, rope_dim=0)
    dgp.dg_op_status()
    kp, x = pool_rows(bt.k_pool.float()), f64(rows)
    for b, (p, n) in enumerate(zip(pre, new)):
        for i in range(n):
            assert np.array_equal(kp[bt.table[b, 0], p + i], x[bt.off[b] + i])


def test_pools_and_rows_past_32_bit_offsets():
    # pools of 2^31 and more elements: the results of a small pool, page for page
    rng = np.random.default_rng(43)
    bt = Batch(rng, [300, 40], [5, 3], 8, 128, 128)
    q = randn(rng, bt.T, 16, 128).to(dev())
    k = randn(rng, bt.T, 8, 128).to(dev())
    n_big = 16384 + 64
    at = n_big - bt.n_pages
    big = []
    for pool in (bt.k_pool, bt.v_pool):
        b = torch.zeros(n_big, 8, 128, 128, dtype=torch.bfloat16, device=dev())
        b[at:] = pool
        big.append(b)
    outs = []
    for pools, shift in (((bt.k_pool, bt.v_pool), 0), (big, at)):
        d = dict(bt.d, page_tables=i32(np.where(bt.table < 0, bt.table, bt.table + shift)))
        dgp.dg_op_rope_kv_append(k, k, *pools, **d)
        out = torch.zeros(bt.T, 16, 128, dtype=torch.bfloat16, device=dev())
        ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(bt.T, 2, 16, 8, 128), dtype=torch.uint8, device=dev())
        dgp.dg_op_tree_attention(q, *pools, **d, tree_mask=None, out=out, workspace=ws)
        outs.append(out)
    dgp.dg_op_status()
    assert torch.equal(outs[0], outs[1]) and outs[0].any()
    for pool, b in zip((bt.k_pool, bt.v_pool), big):
        assert torch.equal(b[at:].view(torch.int16), pool.view(torch.int16))
    # rows that lie 2^30 elements apart
    far = big[0].view(-1)
    x = far.as_strided((3, 1000), (2 ** 30, 1))
    x.copy_(randn(rng, 3, 1000).to(dev()))
    check_logprobs(x, rng.integers(0, 1000, (3, 1)), 5)
    h = far.as_strided((3, 2, 64), (2 ** 30, 64, 1))
    pos = i32([0, 9, 70000])
    a, b = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev()), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev())
    dgp.dg_op_qk_norm_rope(h.contiguous(), None, pos, a, None)
    dgp.dg_op_qk_norm_rope(h, None, pos, h, None)
    b.copy_(h)
    assert torch.equal(a, b)


def test_empty_tensors_through_the_binding():
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=dev())  # noqa: E731
    pool = torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16, device=dev())
    none = dict(page_tables=i32(np.zeros((3, 1))), prefix_lens=i32([0, 0, 0]), offsets=i32([0, 0, 0, 0]))
    dgp.dg_op_rope_kv_append(e(0, 2, 64), e(0, 2, 64), pool, pool.clone(), **none)
    dgp.dg_op_tree_attention(e(0, 4, 64), pool, pool, **none, tree_mask=None, out=e(0, 4, 64), workspace=None)
    q = torch.ones(4, 4, 64, dtype=torch.bfloat16, device=dev())
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(4, 3, 4, 2, 64), dtype=torch.uint8, device=dev())
    dgp.dg_op_tree_attention(q, pool, pool, **none, tree_mask=None, out=out, workspace=ws)     # rows, but no sequence has any
    no_seqs = dict(page_tables=i32(np.zeros((0, 1))), prefix_lens=i32([]), offsets=i32([0]))
    dgp.dg_op_tree_attention(q, pool, pool, **no_seqs, tree_mask=None, out=out, workspace=None)
    dgp.dg_op_rope_kv_append(q[:, :2], q[:, :2], pool, pool, **no_seqs)
    assert (out == 7.0).all() and not pool.any()
    dgp.dg_op_token_logprobs(e(0, 9, dtype=torch.float32), e(0, 1, dtype=torch.int32), e(0, 1, dtype=torch.float32))
    dgp.dg_op_status()


def test_captured_calls_that_share_a_workspace_take_turns():
    # two captured calls and an eager one of other shapes, one after the other on one workspace
    rng = np.random.default_rng(44)
    ws = torch.full((max(dgp.dg_op_tree_attention_workspace_bytes(200, 8, 16, 8, hd) for hd in (64, 128)),), 0x5A, dtype=torch.uint8, device=dev())
    calls, st = [], torch.cuda.Stream()
    for hq, hkv, hd, pre, new in ((16, 8, 128, [5000, 30], [24, 2]), (12, 4, 64, [3000, 2500, 7], [5, 5, 1]), (8, 1, 128, [9000], [61])):
        bt = Batch(rng, pre, new, hkv, hd, 128)
        q, ref = check_attention(bt, hq, None, rng)
        out = torch.full_like(ref, 7.0)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            run_attention(bt, q, None, out, workspace=ws, stream=st)
        calls.append((bt, q, out, ref, g))
    for turn in range(30):
        bt, q, out, ref, g = calls[turn % 3]
        out.fill_(7.0)
        if turn % 5 == 4:
            run_attention(bt, q, None, out, workspace=ws)
        else:
            g.replay()
        assert torch.equal(out, ref)


FIRST_CALL = """
import numpy as np, torch
import discrete_diffusion_block_gb300 as dgp
dgp.load()
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
rows, pools = r(9, 16, 128), [r(12, 4, 128, 128), r(12, 4, 128, 128)]
d = dict(page_tables=i([[0, 1, 2, 3, 4, 5, 6, 7], [8, 9, 10, 11, 0, 0, 0, 0]]), prefix_lens=i([1000, 300]), offsets=i([0, 5, 9]))
pos = i([1000, 1001, 1002, 1003, 1004, 300, 301, 302, 303])
q, out, logits = torch.zeros(9, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 8, 128, dtype=torch.bfloat16, device="cuda"), r(9, 40000)
ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(9, 2, 8, 4, 128), dtype=torch.uint8, device="cuda")
tok, lp, H, ids = i([[3]] * 9), torch.zeros(9, 1, device="cuda"), torch.zeros(9, device="cuda"), torch.zeros(9, 4, dtype=torch.int32, device="cuda")
def step(st):
    dgp.dg_op_qk_norm_rope(rows[:, :8], None, pos, q, None, stream=st)
    dgp.dg_op_rope_kv_append(rows[:, 8:12], rows[:, 12:], *pools, **d, stream=st)
    dgp.dg_op_tree_attention(q, *pools, **d, tree_mask=None, out=out, workspace=ws, stream=st)
    dgp.dg_op_token_logprobs(logits, tok, lp, H, None, ids, None, stream=st)
st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=st):
    step(st)
graph.replay()
torch.cuda.synchronize()
dgp.dg_op_status()
was = [t.clone() for t in (q, out, lp, H, ids, *pools)]
assert all(bool(t.any()) for t in was)
for t in (q, out, lp, H, ids):
    t.zero_()
torch.cuda.synchronize()
step(None)
torch.cuda.synchronize()
dgp.dg_op_status()
assert all(torch.equal(a, b) for a, b in zip(was, (q, out, lp, H, ids, *pools)))
print("the same")
"""


def test_the_first_call_of_a_process_can_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "the same" in p.stdout, p.stderr[-2000:]


def test_attention_on_several_streams_among_other_kernels():
    # the blocks of a call wait for one another: calls on other streams, and
    # kernels that hold some of the SMs, must not come between them
    rng = np.random.default_rng(45)
    calls = []
    for hq, hkv, hd, pre, new in ((16, 8, 128, [6000, 3000], [24, 2]), (12, 4, 64, [3000] * 20, [5] * 20), (8, 1, 128, [9000], [61])):
        bt = Batch(rng, pre, new, hkv, hd, 128)
        q, ref = check_attention(bt, hq, None, rng)
        ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(bt.T, len(pre), hq, hkv, hd), dtype=torch.uint8, device=dev())
        calls.append((bt, q, torch.full_like(ref, 7.0), ref, ws, torch.cuda.Stream()))
    a = torch.randn(512, 512, device=dev())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(side):
            a = torch.tanh(a @ a)
        for bt, q, out, _, ws, st in calls:
            run_attention(bt, q, None, out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    dgp.dg_op_status()
    for _, _, out, ref, _, _ in calls:
        assert torch.equal(out, ref)
