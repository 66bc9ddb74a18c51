"""The operators that bound a long context's cache (windowed attention with
first tokens that stay visible, attention weight per cached key, eviction)
against plain numpy evaluations in 64 bits.

Tolerances: those of the draft-serving tests for bf16 outputs; each check of an
fp32 result states the roundings it counts.
"""
import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev
from test_gpu_draft_ops import U32, Batch, _clean_status, _lib, attention_tol, f64, i32, randn  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
HEADS = [(16, 8, 128), (4, 2, 64), (12, 4, 64), (8, 1, 128), (5, 5, 64), (7, 1, 64)]


# ---- references -------------------------------------------------------------------

def visible(p, n, window, sinks):
    """[n][p + n]: the key slots that new token t, at slot p + t, sees."""
    s, j = p + np.arange(n)[:, None], np.arange(p + n)[None]
    return (j <= s) & ((j > s - window) | (j < sinks)) if window else j <= s


def place(pool, table, slots, x):
    """x [n][heads][hd] into the given slots of a sequence (16-byte chunk c of a slot's 64-wide sub-block at c ^ (slot % 8))."""
    hkv, pg, hd = pool.shape[1:]
    page, slot = torch.from_numpy(table[slots // pg]).long()[:, None], torch.from_numpy(slots % pg).long()[:, None]
    at = torch.arange(8)[None] ^ (slot % 8)
    pool.view(-1, hkv, hd // 64, pg, 8, 8)[page, :, :, slot, at] = x.view(-1, hkv, hd // 64, 8, 8).permute(0, 3, 1, 2, 4)


def hide(bt, window, sinks, first=0):
    """NaN into the keys and values that no new token from `first` on sees; pages
    that hold no other ones leave the table."""
    pools = [bt.k_pool.cpu(), bt.v_pool.cpu()]
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        if n == 0:
            continue
        seen = visible(p, n, window, sinks)[first:].any(0)
        gone = np.nonzero(~seen)[0]
        for pool in pools:
            place(pool, bt.table[b], gone, torch.full((len(gone), bt.hkv, bt.hd), float("nan"), dtype=torch.bfloat16))
        for j in range(-(-(p + n) // bt.pg)):
            if not seen[j * bt.pg:(j + 1) * bt.pg].any():
                bt.table[b, j] = -9
    for mine, pool in zip((bt.k_pool, bt.v_pool), pools):
        mine.copy_(pool)
    bt.d["page_tables"].copy_(i32(bt.table))


def window_ref(q, bt, window, sinks, scale):
    """out, sum_j p_j |v_j|, lse and the largest sum of |products| of a score, in 64 bits."""
    hq = q.shape[1]
    G = hq // bt.hkv
    out, mag, lse, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        see = visible(p, n, window, sinks)
        for t0 in range(0, n, 64):
            t1 = min(n, t0 + 64)
            j = np.nonzero(see[t0:t1].any(0))[0]
            rows = slice(bt.off[b] + t0, bt.off[b] + t1)
            for h in range(hq):
                k, v, x = bt.keys[b][j, h // G], bt.vals[b][j, h // G], q[rows, h]
                s = np.where(see[t0:t1][:, j], x @ k.T * scale, -np.inf)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                lse[rows, h] = m[:, 0] + np.log(e.sum(1))
                e /= e.sum(1, keepdims=True)
                out[rows, h], mag[rows, h] = e @ v, e @ np.abs(v)
                top[rows, h] = (np.where(see[t0:t1][:, j], np.abs(x) @ np.abs(k).T * scale, 0)).max(1)
    return out, mag, lse, top


def lse_tol(lse, top, hd, tiles):
    # scores: hd products and their sum, scaled; the sum over keys (64 of a tile's half in a
    # chain, then tile by tile and piece by piece) of exponentials within 4 ulp; the logarithm
    return U32 * ((hd + 8) * top + 8 * np.abs(lse) + 64 + tiles + 32)


def same_floats(a, b):
    return np.array_equal(np.asarray(a).view(np.uint32), np.asarray(b).view(np.uint32))


# ---- windowed attention ------------------------------------------------------------------

def window_workspace(T, B, hq, hkv, hd, fill=0xFF):
    n = dgp.dg_op_window_attention_workspace_bytes(T, B, hq, hkv, hd)
    return torch.full((max(n, 1),), fill, dtype=torch.uint8, device=dev())


def run_window(bt, q, window, sinks, out, lse=None, scale=None, stream=None, workspace=None):
    ws = window_workspace(q.shape[0], len(bt.pre), q.shape[1], bt.hkv, bt.hd) if workspace is None else workspace
    dgp.dg_op_window_attention(q, bt.k_pool, bt.v_pool, **bt.d, out=out, workspace=ws, window=window, sinks=sinks, lse=lse, scale=scale,
                               stream=stream)


def check_window(bt, hq, window, sinks, rng, scale=None, strided=False, hidden=True):
    if strided:
        q = randn(rng, bt.T, hq + 3, bt.hd).to(dev())[:, 1:1 + hq]
        out = torch.full((bt.T, 2 * hq, bt.hd), 7.0, dtype=torch.bfloat16, device=dev())[:, hq:]
    else:
        q = randn(rng, bt.T, hq, bt.hd).to(dev())
        out = torch.full((bt.T, hq, bt.hd), 7.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full((bt.T, hq), 7.0, device=dev())
    if hidden and window:
        hide(bt, window, sinks)
    run_window(bt, q, window, sinks, out, lse, scale)
    dgp.dg_op_status()
    ref, mag, z, top = window_ref(f64(q), bt, window, sinks, bt.hd ** -0.5 if scale is None else scale)
    n = int(bt.off[-1])
    got, got_z = f64(out), f64(lse)
    assert (np.abs(got[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all(), np.abs(got[:n] - ref[:n]).max()
    tiles = max((p + m for p, m in zip(bt.pre, bt.new)), default=0) / 128 + 2
    assert (np.abs(got_z[:n] - z[:n]) <= lse_tol(z[:n], top[:n], bt.hd, tiles)).all(), np.abs(got_z[:n] - z[:n]).max()
    assert (got[n:] == 7.0).all() and (got_z[n:] == 7.0).all()           # rows behind the last sequence
    return q, out, lse


@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("pre,window,sinks,pg", [
    (0, 1, 0, 128), (1, 1, 1, 64), (63, 64, 0, 64), (64, 64, 4, 128), (127, 128, 0, 192), (128, 127, 4, 128), (129, 300, 1, 64),
    (700, 1, 0, 64), (700, 64, 64, 128), (701, 65, 63, 128), (1000, 200, 65, 64), (1000, 200, 130, 192), (1000, 128, 2000, 128),
    (1999, 0, 0, 128), (1999, 2 ** 31 - 1, 2 ** 31 - 1, 128),
])
def test_window_of_single_tokens(hq, hkv, hd, pre, window, sinks, pg):
    rng = np.random.default_rng(pre + window % 1000)
    check_window(Batch(rng, [pre], [1], hkv, hd, pg), hq, window, sinks, rng)


@pytest.mark.parametrize("hq,hkv,hd,pg,pre,new", [
    (16, 8, 128, 128, [300], [17]),
    (16, 8, 128, 128, [0, 2000, 130], [64, 3, 0]),
    (12, 4, 64, 64, [100, 0, 5, 640, 0], [5, 1, 0, 133, 2]),
    (16, 4, 128, 192, [190, 191], [63, 66]),
    (32, 1, 64, 64, [70], [90]),
    (6, 2, 64, 128, [0], [500]),
    (16, 8, 128, 128, [0], [700]),
    (7, 1, 128, 64, [11] * 40, [j % 5 for j in range(40)]),
    (4, 2, 64, 64, [j * 7 for j in range(200)], [1] * 200),
    (128, 1, 64, 64, [20, 64], [30, 1]),
    (3, 1, 64, 64, [1000, 3], [333, 257]),
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (64, 4), (100, 0), (129, 130), (333, 70)])
def test_window_of_batches(hq, hkv, hd, pg, pre, new, window, sinks):
    rng = np.random.default_rng(len(pre) + hq)
    bt = Batch(rng, pre, new, hkv, hd, pg)
    check_window(bt, hq, window, sinks, rng, strided=window % 2 == 1)


@pytest.mark.parametrize("pre,new,window,sinks", [([20011], [2], 5000, 4), ([20011], [2], 0, 0), ([9000, 4], [1, 1], 8000, 200)])
def test_window_over_a_long_context_with_a_scale(pre, new, window, sinks):
    rng = np.random.default_rng(11)
    check_window(Batch(rng, pre, new, 2, 128, 128), 4, window, sinks, rng, scale=0.3)


@pytest.mark.parametrize("hq,hkv,hd,pre,new,window", [
    (16, 8, 128, [3000, 10, 777], [20, 1, 8], 2000),
    (12, 4, 64, [100 + 37 * j for j in range(40)], [1 + j % 5 for j in range(40)], 1000),
    (8, 8, 128, [8000], [1], 4096),
    (4, 1, 64, [40000], [33], 0),
    (16, 8, 128, [0], [2000], 500),
])
def test_window_repeats_bit_for_bit(hq, hkv, hd, pre, new, window):
    rng = np.random.default_rng(14)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    q = randn(rng, bt.T, hq, hd).to(dev())
    first = None
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    out, lse = torch.zeros(bt.T, hq, hd, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, hq, device=dev())
    ws = window_workspace(bt.T, len(pre), hq, hkv, hd)
    for fill in (0, 0xFF, 0x7F):
        run_window(bt, q, window, 4, out, lse, workspace=window_workspace(bt.T, len(pre), hq, hkv, hd, fill))
        if first is None:
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        for _ in range(3):
            run_window(bt, q, window, 4, out, lse, workspace=ws, stream=st)
    for _ in range(30):
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        n = int(bt.off[-1])
        assert torch.equal(out[:n], first[0][:n]) and torch.equal(lse[:n], first[1][:n])


def test_window_without_lse_and_with_all_keys_is_the_causal_attention():
    rng = np.random.default_rng(17)
    bt = Batch(rng, [300, 40], [70, 5], 4, 64, 64)
    q, out, _ = check_window(bt, 8, 0, 0, rng)
    again = torch.full_like(out, 7.0)
    run_window(bt, q, 10 ** 6, 0, again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("pre,new", [([200, 50], [2, 3]), ([200, 50], [400, 3])])
def test_window_reports_bad_pages_and_bad_sequences(pre, new):
    rng = np.random.default_rng(15)
    bt = Batch(rng, pre, new, 2, 64, 64)
    n0, n = new[0], sum(new)
    q = randn(rng, bt.T, 4, 64).to(dev())
    good, lse = torch.zeros(bt.T, 4, 64, dtype=torch.bfloat16, device=dev()), torch.zeros(bt.T, 4, device=dev())
    run_window(bt, q, 180, 4, good, lse)
    for entry in ((0, 1, bt.n_pages), (0, 0, -1)):
        bad = bt.table.copy()
        bad[entry[0], entry[1]] = entry[2]
        out, z = torch.zeros_like(good), torch.zeros_like(lse)
        keep, bt.d = bt.d, dict(bt.d, page_tables=i32(bad))
        run_window(bt, q, 180, 4, out, z)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_EINVAL and "page" in str(e.value)
        assert torch.isfinite(out.float()).all() and torch.equal(out[n0:n], good[n0:n]) and torch.equal(z[n0:n], lse[n0:n])
    for change in (dict(prefix_lens=i32([10 ** 6, 50])), dict(prefix_lens=i32([-1, 50])), dict(prefix_lens=i32([2 ** 31 - 1, 50]))):
        out = torch.full_like(good, 7.0)
        keep, bt.d = bt.d, dict(bt.d, **change)
        run_window(bt, q, 180, 4, out)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert "sequence" in str(e.value)
        assert (out[:n0] == 7.0).all() and torch.equal(out[n0:n], good[n0:n])


def test_window_rows_whose_only_keys_lie_on_a_bad_page_are_zero():
    rng = np.random.default_rng(18)
    bt = Batch(rng, [200], [1], 2, 64, 64)
    bt.table[0, 3] = bt.n_pages
    bt.d["page_tables"].copy_(i32(bt.table))
    out, lse = torch.full((bt.T, 4, 64), 7.0, dtype=torch.bfloat16, device=dev()), torch.full((bt.T, 4), 7.0, device=dev())
    run_window(bt, randn(rng, bt.T, 4, 64).to(dev()), 5, 0, out, lse)
    with pytest.raises(dgp.DgError):
        dgp.dg_op_status()
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


@pytest.mark.parametrize("pre,new,window", [([2048], [3], 0), ([40000], [3], 39000), ([10], [3], 4), ([100], [600], 300)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_window_of_a_query_that_is_not_a_number_stays_apart(pre, new, window, value):
    rng = np.random.default_rng(53)
    bt = Batch(rng, pre, new, 2, 64, 64)
    q = randn(rng, bt.T, 4, 64)
    q[1, 2, 5] = value
    out, lse = torch.full((bt.T, 4, 64), 7.0, dtype=torch.bfloat16, device=dev()), torch.full((bt.T, 4), 7.0, device=dev())
    run_window(bt, q.to(dev()), window, 1, out, lse)
    q[1, 2, 5] = 0.0
    ref, mag, z, top = window_ref(f64(q), bt, window, 1, 0.125)
    got, got_z, n = f64(out), f64(lse), int(bt.off[-1])
    assert np.isnan(got[1, 2]).all() and not np.isfinite(got_z[1, 2])
    got[1, 2], got_z[1, 2] = ref[1, 2], z[1, 2]
    assert (np.abs(got[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all()
    assert (np.abs(got_z[:n] - z[:n]) <= lse_tol(z[:n], top[:n], 64, (pre[0] + new[0]) / 128 + 2)).all()


# ---- weight that keys gather ------------------------------------------------------------

def mass_ref(q, lse, bt, mass, window, sinks, observe, scale, shared=()):
    """The weights after the call, how far fp32 may be off, and which slots must
    keep their bits, in 64 bits; q, lse, mass as the call gets them."""
    hq = q.shape[1]
    G = hq // bt.hkv
    out = mass.astype(np.float64)
    tol, still = np.zeros(out.shape), np.ones(out.shape, bool)
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        if n == 0:
            continue
        first = max(0, n - observe) if observe else 0
        see = visible(p, n, window, sinks)[first:]
        j = np.nonzero(see.any(0) | (np.arange(p + n) >= p))[0]
        page, slot = bt.table[b, j // bt.pg], j % bt.pg
        rows = slice(bt.off[b] + first, bt.off[b] + n)
        for g in range(bt.hkv):
            total, err = np.where(j < p, out[page, g, slot], 0.0), np.zeros(len(j))
            for h in range(g * G, (g + 1) * G):
                x, k = q[rows, h], np.where(see.any(0)[j][:, None], bt.keys[b][j, g], 0.0)
                z = lse[rows, h].astype(np.float64)[:, None]
                e = np.where(see[:, j], np.exp(np.where(see[:, j], x @ k.T * scale - z, 0.0)), 0.0)
                e = np.where(z == -np.inf, 0.0, e)
                total += e.sum(0)
                # scores as in lse_tol, the exponent's own roundings, sums over 128 rows and then tile by tile
                with np.errstate(invalid="ignore"):
                    err += (e * ((bt.hd + 8) * (np.abs(x) @ np.abs(k).T * scale) + 8 * np.where(np.isfinite(z), np.abs(z), 0) + 100 + n * G / 64)).sum(0)
            out[page, g, slot] = total
            tol[page, g, slot] = U32 * (err + 2 * np.abs(total))
            still[page, g, slot] = False
    return out, tol, still


def mass_workspace(T, B, hq, hkv, hd, fill=0xFF):
    return torch.full((dgp.dg_op_key_mass_workspace_bytes(T, B, hq, hkv, hd),), fill, dtype=torch.uint8, device=dev())


def run_mass(bt, q, lse, mass, window=0, sinks=0, observe=0, scale=None, stream=None, workspace=None):
    ws = mass_workspace(q.shape[0], len(bt.pre), q.shape[1], bt.hkv, bt.hd) if workspace is None else workspace
    dgp.dg_op_key_mass(q, lse, bt.k_pool, mass, **bt.d, workspace=ws, window=window, sinks=sinks, observe=observe, scale=scale, stream=stream)


def row_lse(q, bt, window, sinks, scale):
    out = np.zeros(q.shape[:2])
    G = q.shape[1] // bt.hkv
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        if n == 0:
            continue
        see = visible(p, n, window, sinks)
        rows = slice(bt.off[b], bt.off[b] + n)
        for h in range(q.shape[1]):
            s = np.where(see, q[rows, h] @ np.nan_to_num(bt.keys[b][:, h // G]).T * scale, -np.inf)
            m = s.max(1, keepdims=True)
            out[rows, h] = m[:, 0] + np.log(np.exp(s - m).sum(1))
    return out.astype(np.float32)


def mass_case(rng, bt, hq, window, sinks, scale, strided=False):
    q = randn(rng, bt.T, hq + 3, bt.hd).to(dev())[:, 1:1 + hq] if strided else randn(rng, bt.T, hq, bt.hd).to(dev())
    lse = row_lse(f64(q), bt, window, sinks, scale)
    lse[int(bt.off[-1]):] = np.nan                              # rows that belong to nobody
    mass = rng.exponential(1.0, (bt.n_pages, bt.hkv, bt.pg)).astype(np.float32)
    mass[rng.random(mass.shape) < 0.02] = np.nan
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):            # what new slots held does not matter, what cached keys hold does
        j = np.arange(p)
        mass[bt.table[b, j // bt.pg], :, j % bt.pg] = rng.exponential(1.0, (p, bt.hkv))
        j = np.arange(p, p + n)
        mass[bt.table[b, j // bt.pg], :, j % bt.pg] = np.nan
    return q, lse, mass


def compare_mass(got, ref, tol, still, before):
    got = got.cpu().numpy()
    assert np.array_equal(got.view(np.uint32)[still], before.view(np.uint32)[still])
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - ref) <= tol)[~still].all(), np.nanmax((np.abs(got - ref) - tol)[~still])


def check_mass(bt, hq, window, sinks, observe, rng, scale=None, strided=False):
    factor = bt.hd ** -0.5 if scale is None else scale
    q, lse, before = mass_case(rng, bt, hq, window, sinks, factor, strided)
    first = observe if observe else max(bt.new)
    hide_keys(bt, window, sinks, first)
    mass, z = torch.from_numpy(before).to(dev()), torch.from_numpy(lse).to(dev())
    run_mass(bt, q, z, mass, window, sinks, observe, scale)
    dgp.dg_op_status()
    compare_mass(mass, *mass_ref(f64(q), lse, bt, before, window, sinks, observe, factor), before)
    return q, z, before, mass


def hide_keys(bt, window, sinks, observe):
    """NaN into the keys that no counted row sees; pages of which none is seen and that hold no new slot leave the table."""
    pool = bt.k_pool.cpu()
    for b, (p, n) in enumerate(zip(bt.pre, bt.new)):
        if n == 0:
            continue
        seen = visible(p, n, window, sinks)[max(0, n - observe):].any(0)
        gone = np.nonzero(~seen)[0]
        place(pool, bt.table[b], gone, torch.full((len(gone), bt.hkv, bt.hd), float("nan"), dtype=torch.bfloat16))
        seen[p:] = True
        for j in range(-(-(p + n) // bt.pg)):
            if not seen[j * bt.pg:(j + 1) * bt.pg].any():
                bt.table[b, j] = bt.n_pages + 9
    bt.k_pool.copy_(pool)
    bt.d["page_tables"].copy_(i32(bt.table))


@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("pre,window,sinks,pg", [
    (0, 0, 0, 128), (1, 1, 1, 64), (63, 64, 0, 64), (255, 0, 0, 128), (256, 0, 0, 192), (300, 128, 4, 64), (1000, 200, 65, 64), (1000, 200, 130, 192),
    (1999, 600, 300, 128), (1999, 2 ** 31 - 1, 2 ** 31 - 1, 128),
])
def test_mass_of_single_tokens(hq, hkv, hd, pre, window, sinks, pg):
    rng = np.random.default_rng(pre + window % 1000)
    check_mass(Batch(rng, [pre], [1], hkv, hd, pg), hq, window, sinks, 0, rng)


@pytest.mark.parametrize("hq,hkv,hd,pg,pre,new", [
    (16, 8, 128, 128, [300], [17]),
    (16, 8, 128, 128, [0, 2000, 130], [64, 3, 0]),
    (12, 4, 64, 64, [100, 0, 5, 640, 0], [5, 1, 0, 133, 2]),
    (32, 1, 64, 64, [70], [90]),
    (6, 2, 64, 128, [0], [500]),
    (16, 8, 128, 128, [0], [700]),
    (7, 1, 128, 64, [11] * 40, [j % 5 for j in range(40)]),
    (4, 2, 64, 64, [j * 7 for j in range(200)], [1] * 200),
    (128, 1, 64, 64, [20, 64], [30, 1]),
    (3, 1, 64, 64, [1000, 3], [333, 257]),
    (16, 4, 128, 192, [3000, 0], [40, 1100]),
])
@pytest.mark.parametrize("window,sinks,observe", [(0, 0, 0), (0, 0, 1), (0, 0, 50), (1, 0, 0), (1, 3, 7), (100, 0, 0), (129, 130, 30), (333, 70, 0),
                                                  (50, 0, 1)])
def test_mass_of_batches(hq, hkv, hd, pg, pre, new, window, sinks, observe):
    rng = np.random.default_rng(len(pre) + hq)
    bt = Batch(rng, pre, new, hkv, hd, pg)
    check_mass(bt, hq, window, sinks, observe, rng, strided=window % 2 == 1)


def test_mass_with_a_scale_and_rows_that_saw_nothing_or_nan():
    rng = np.random.default_rng(21)
    bt = Batch(rng, [700, 300], [5, 2], 2, 64, 64)
    q, lse, before = mass_case(rng, bt, 4, 0, 0, 0.3)
    lse[1] = -np.inf
    z, mass = torch.from_numpy(lse).to(dev()), torch.from_numpy(before).to(dev())
    run_mass(bt, q, z, mass, scale=0.3)
    compare_mass(mass, *mass_ref(f64(q), lse, bt, before, 0, 0, 0, 0.3), before)
    lse[6, 2] = np.nan                                  # the second sequence's last token, KV head 1
    z, mass = torch.from_numpy(lse).to(dev()), torch.from_numpy(before).to(dev())
    run_mass(bt, q, z, mass, scale=0.3)
    got = mass.cpu().numpy()
    j = np.arange(302)
    assert np.isnan(got[bt.table[1, j // 64], 1, j % 64]).all()
    ref, tol, still = mass_ref(f64(q), np.where(np.isnan(lse), 0, lse), bt, before, 0, 0, 0, 0.3)
    still[bt.table[1, j // 64], 1, j % 64] = True
    assert (np.abs(got - ref) <= tol)[~still].all()


@pytest.mark.parametrize("hq,hkv,hd,pre,new,window,sinks,observe", [
    (16, 8, 128, [3000, 10, 777], [20, 1, 8], 0, 0, 0),
    (8, 2, 128, [0], [3000], 500, 4, 0),                # the first tokens' keys are seen by all rows: many pieces
    (4, 1, 64, [20000], [600], 0, 0, 0),
    (12, 4, 64, [100 + 37 * j for j in range(40)], [1 + j % 5 for j in range(40)], 0, 0, 0),
])
def test_mass_repeats_bit_for_bit(hq, hkv, hd, pre, new, window, sinks, observe):
    rng = np.random.default_rng(22)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    q, z, before, first = check_mass(bt, hq, window, sinks, observe, rng)
    ws = mass_workspace(bt.T, len(pre), hq, hkv, hd)
    old, mass = torch.from_numpy(before).to(dev()), torch.empty_like(first)
    bits = lambda t: t.view(torch.int32)  # noqa: E731
    for fill in (0, 0x7F, 0xFF, None, None):
        if fill is not None:
            ws.fill_(fill)
        mass.copy_(old)
        run_mass(bt, q, z, mass, window, sinks, observe, workspace=ws)
        assert torch.equal(bits(mass), bits(first))
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        mass.copy_(old)
        run_mass(bt, q, z, mass, window, sinks, observe, workspace=ws, stream=st)
    for _ in range(30):
        mass.zero_()
        g.replay()
        assert torch.equal(bits(mass), bits(first))
    # the second step adds to the first's
    run_mass(bt, q, z, mass, window, sinks, observe, workspace=ws)
    after = first.cpu().numpy()
    compare_mass(mass, *mass_ref(f64(q), z.cpu().numpy(), bt, after, window, sinks, observe, hd ** -0.5), after)


def test_mass_reports_bad_pages_and_bad_sequences():
    rng = np.random.default_rng(23)
    bt = Batch(rng, [200, 50], [2, 3], 2, 64, 64)
    q, lse, before = mass_case(rng, bt, 4, 0, 0, 0.125)
    z, good = torch.from_numpy(lse).to(dev()), torch.from_numpy(before).to(dev())
    run_mass(bt, q, z, good)
    good = good.cpu().numpy()
    for value in (bt.n_pages, -1):
        bad = bt.table.copy()
        page, bad[0, 1] = bad[0, 1], value
        mass = torch.from_numpy(before).to(dev())
        keep, bt.d = bt.d, dict(bt.d, page_tables=i32(bad))
        run_mass(bt, q, z, mass)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_EINVAL and "page" in str(e.value)
        want = good.copy()
        want[page] = before[page]
        assert same_floats(mass.cpu().numpy(), want)
    for change in (dict(prefix_lens=i32([10 ** 6, 50])), dict(prefix_lens=i32([-1, 50])), dict(prefix_lens=i32([2 ** 31 - 1, 50]))):
        mass = torch.from_numpy(before).to(dev())
        keep, bt.d = bt.d, dict(bt.d, **change)
        run_mass(bt, q, z, mass)
        bt.d = keep
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert "sequence" in str(e.value)
        want = good.copy()
        pages = bt.table[0, :4]
        want[pages] = before[pages]
        assert same_floats(mass.cpu().numpy(), want)


@pytest.mark.parametrize("hq,hkv,hd,pre,new", [(8, 2, 128, [0], [3000]), (4, 1, 64, [20000], [600])])
def test_a_captured_mass_recovers_from_a_failure(hq, hkv, hd, pre, new):
    # a launch that finds an earlier failure gives up and may leave counts of arrivals behind
    rng = np.random.default_rng(24)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    q, z, before, first = check_mass(bt, hq, 0, 0, 0, rng)
    ws, old, mass = mass_workspace(bt.T, 1, hq, hkv, hd), torch.from_numpy(before).to(dev()), torch.empty_like(first)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        run_mass(bt, q, z, mass, workspace=ws, stream=st)
    for turn in range(8):
        dgp.dg_op_wait_selftest(20_000)
        g.replay()
        torch.cuda.synchronize()
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_ETIMEOUT
        dgp.dg_op_status()                                  # cleared
        for _ in range(3):
            mass.copy_(old)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            dgp.dg_op_status()
            assert torch.equal(mass.view(torch.int32), first.view(torch.int32)), turn


# ---- eviction ----------------------------------------------------------------------------

class Cache:
    """Sequences over shuffled pages with a weight per slot and KV head, and other
    pages (or the same) for what stays. Pages are shared between the first two
    sequences where `shared`."""

    def __init__(self, rng, lens, hkv, hd, pg, budget, in_place=False, shared=0, weights=None, dtype=torch.bfloat16):
        self.lens, self.hkv, self.hd, self.pg, self.budget = list(lens), hkv, hd, pg, budget
        need = [-(-n // pg) for n in lens]
        kept = [-(-min(n, budget) // pg) for n in lens]
        self.n_pages = sum(need) + (0 if in_place else sum(kept)) + 1
        perm = list(rng.permutation(self.n_pages))
        self.table = np.full((len(lens), max(need) + 1), -5, np.int32)
        self.out = np.full((len(lens), max(kept) + 1), -5, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = [perm.pop() for _ in range(m)]
        if shared:
            self.table[1, :shared] = self.table[0, :shared]
        for b, m in enumerate(kept):
            self.out[b, :m] = self.table[b, :m] if in_place else [perm.pop() for _ in range(m)]
        shape = (self.n_pages, hkv, pg, hd)
        self.k, self.v = (torch.from_numpy(rng.integers(0, 2 ** 16, shape, dtype=np.uint16).view(np.int16)) for _ in range(2))    # any bits
        self.mass = (np.exp(2 * rng.standard_normal(shape[:3])) if weights is None else weights(shape[:3])).astype(np.float32)

    def ref(self, sinks, recent):
        """Pools in slot order, weights, lengths and kept slots after the eviction."""
        order = [pool_view(x) for x in (self.k, self.v)]
        k, v, mass = (np.array(x) for x in (*order, self.mass))
        kept = np.full((len(self.lens), self.hkv, self.budget), -1, np.int32)
        for b, n in enumerate(self.lens):
            for h in range(self.hkv):
                j = np.arange(n)
                if n > self.budget:
                    mid = j[sinks:n - recent]
                    w = self.mass[self.table[b, mid // self.pg], h, mid % self.pg].astype(np.float64)
                    best = sorted(range(len(mid)), key=lambda i: (np.isnan(w[i]), 0.0 if np.isnan(w[i]) else -w[i], i))
                    j = np.concatenate([j[:sinks], np.sort(mid[best[:self.budget - sinks - recent]]), j[n - recent:]])
                kept[b, h, :len(j)] = j
                d = np.arange(len(j))
                dst, src = (self.out[b, d // self.pg], d % self.pg), (self.table[b, j // self.pg], j % self.pg)
                for x, old in ((k, order[0]), (v, order[1])):
                    x[dst[0], dst[1], h] = old[src[0], src[1], h]
                mass[dst[0], h, dst[1]] = self.mass[src[0], h, src[1]]
        return k, v, mass, np.minimum(self.lens, self.budget), kept

    def on_gpu(self):
        d = dict(k_pool=self.k.to(dev()).view(torch.bfloat16), v_pool=self.v.to(dev()).view(torch.bfloat16),
                 mass_pool=torch.from_numpy(self.mass).to(dev()), page_tables=i32(self.table), lens=i32(self.lens),
                 out_lens=i32([7] * len(self.lens)), kept=torch.full((len(self.lens), self.hkv, self.budget), 7, dtype=torch.int32, device=dev()))
        d["out_tables"] = i32(self.out)
        return d


def pool_view(pool):
    """The pool's bits in slot order: [n_pages][pg][heads][hd] int16."""
    from test_gpu_draft_ops import pool_rows
    return pool_rows(pool.view(torch.int16) if isinstance(pool, torch.Tensor) else pool)


def check_evict(c, sinks, recent, **call):
    d = c.on_gpu()
    dgp.dg_op_cache_evict(**d, budget=c.budget, sinks=sinks, recent=recent, **call)
    torch.cuda.synchronize()
    dgp.dg_op_status()
    compare_evict(d, c.ref(sinks, recent))
    return d


def compare_evict(d, ref):
    k, v, mass, lens, kept = ref
    assert np.array_equal(d["out_lens"].cpu().numpy(), lens)
    assert np.array_equal(d["kept"].cpu().numpy(), kept)
    assert np.array_equal(pool_view(d["k_pool"]), k) and np.array_equal(pool_view(d["v_pool"]), v)
    assert same_floats(d["mass_pool"].cpu().numpy(), mass)


@pytest.mark.parametrize("lens,hkv,hd,pg,budget,sinks,recent", [
    ([2], 1, 64, 64, 1, 0, 0),
    ([2, 1, 0], 2, 128, 64, 1, 1, 0),
    ([300], 1, 128, 128, 299, 4, 64),
    ([300, 77, 0, 301], 3, 64, 64, 300, 0, 0),
    ([1000, 5, 999], 2, 128, 192, 100, 4, 96),
    ([1000, 5, 999], 2, 128, 7, 100, 3, 90),
    ([700] * 30, 2, 64, 64, 333, 1, 100),
    ([2176], 8, 128, 128, 2048, 4, 256),
    ([9000], 1, 128, 128, 8000, 0, 0),
    ([40000], 2, 64, 128, 5000, 10, 1000),
    ([70000, 33000], 1, 64, 128, 65000, 0, 300),
    ([500], 2, 64, 64, 64, 64, 0),
    ([500], 2, 64, 64, 64, 0, 64),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(lens, hkv, hd, pg, budget, sinks, recent, in_place):
    rng = np.random.default_rng(len(lens) + pg)
    check_evict(Cache(rng, lens, hkv, hd, pg, budget, in_place), sinks, recent)


@pytest.mark.parametrize("weights", ["equal", "few", "nan", "signs", "ends"])
@pytest.mark.parametrize("budget,sinks,recent", [(500, 0, 0), (900, 4, 77), (31, 3, 0)])
def test_evict_weights_of_all_kinds(weights, budget, sinks, recent):
    rng = np.random.default_rng(3)
    kinds = dict(
        equal=lambda s: np.zeros(s), few=lambda s: rng.integers(0, 3, s) * 0.5,
        nan=lambda s: np.where(rng.random(s) < 0.6, np.nan, rng.standard_normal(s)),
        signs=lambda s: np.where(rng.random(s) < 0.3, rng.choice([0.0, -0.0], s), rng.integers(-2, 3, s) * 1e-3),
        ends=lambda s: rng.choice([np.inf, -np.inf, 3e38, -3e38, 1e-45, -1e-45, 1.0, 1.0000001], s))
    for in_place in (False, True):
        check_evict(Cache(rng, [1000, 1300], 2, 64, 64, budget, in_place, weights=kinds[weights]), sinks, recent)


def test_evict_leaves_shared_pages_whole():
    rng = np.random.default_rng(5)
    c = Cache(rng, [800, 700, 30], 2, 64, 64, 200, shared=6)
    before = c.table[0, :6]
    d = check_evict(c, 2, 20)
    for name, was in (("k_pool", c.k), ("v_pool", c.v)):
        assert torch.equal(d[name].view(torch.int16).cpu()[before], was[before])


def test_evict_some_in_place_and_some_elsewhere():
    rng = np.random.default_rng(6)
    c = Cache(rng, [800, 90, 1000, 40], 2, 128, 64, 200)
    for b in (0, 3):
        m = -(-min(c.lens[b], 200) // 64)
        c.out[b, :m] = c.table[b, :m]
    check_evict(c, 2, 20)


def test_evict_repeats_and_is_captured():
    rng = np.random.default_rng(7)
    c = Cache(rng, [5000, 3000, 12], 4, 128, 128, 1500)
    ref = c.ref(4, 300)
    d = c.on_gpu()
    dgp.dg_op_cache_evict(**d, budget=1500, sinks=4, recent=300)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        dgp.dg_op_cache_evict(**d, budget=1500, sinks=4, recent=300, stream=st)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    compare_evict(d, ref)
    # other lengths and weights in the same tensors: the captured call takes them
    e = Cache(rng, [4000, 100, 1800], 4, 128, 128, 1500)
    e.table, e.out, e.n_pages = c.table, c.out, c.n_pages
    e.k, e.v, e.mass = e.k.new_zeros(c.k.shape), e.v.new_zeros(c.v.shape), rng.random(c.mass.shape).astype(np.float32)
    e.lens = [4000, 100, 12]
    for name, x in e.on_gpu().items():
        d[name].copy_(x)
    g.replay()
    torch.cuda.synchronize()
    compare_evict(d, e.ref(4, 300))


def test_evict_reports_bad_sequences_and_pages():
    rng = np.random.default_rng(8)
    for change, words in ((dict(lens=-1), "sequence"), (dict(lens=10 ** 6), "sequence"), (dict(lens=2 ** 31 - 1), "sequence"),
                          (dict(table=-1), "page"), (dict(table="n"), "page"), (dict(out="n"), "page")):
        c = Cache(rng, [500, 400, 300], 2, 64, 64, 200)
        good = Cache.ref(c, 2, 20)
        d = c.on_gpu()
        for what, value in change.items():
            if what == "lens":
                d["lens"][1] = value
            else:
                d["page_tables" if what == "table" else "out_tables"][1, 2] = c.n_pages if value == "n" else value
        dgp.dg_op_cache_evict(**d, budget=200, sinks=2, recent=20)
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_EINVAL and words in str(e.value)
        # the sequence is left as it is, the others are moved
        assert d["out_lens"].tolist() == [200, -1, 200] and (d["kept"][1] == -1).all()
        left = c.out[1, :4]
        for name, was, want in (("k_pool", c.k, good[0]), ("v_pool", c.v, good[1])):
            assert torch.equal(d[name].view(torch.int16).cpu()[left], was[left])
            got = pool_view(d[name])
            assert np.array_equal(got[c.out[0, :4]], want[c.out[0, :4]]) and np.array_equal(got[c.out[2, :4]], want[c.out[2, :4]])


def test_evict_of_more_slots_than_are_taken_is_reported():
    rng = np.random.default_rng(9)
    n = 262144 + 64
    c = Cache(rng, [64, 64], 1, 64, 64, 10)
    d = c.on_gpu()
    d["lens"][0] = n
    d["page_tables"] = i32(np.tile(c.table[:, :1], (1, n // 64)))
    dgp.dg_op_cache_evict(**d, budget=10)
    with pytest.raises(dgp.DgError) as e:
        dgp.dg_op_status()
    assert "sequence" in str(e.value) and d["out_lens"].tolist() == [-1, 10]
