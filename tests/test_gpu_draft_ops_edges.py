"""The operators that serve drafted tokens after failures, on values at the ends
of their types and in calls that other tests do not make, against the plain numpy
evaluations of test_gpu_draft_ops."""
import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev
from test_draft_ops_host import packed
from test_gpu_draft_ops import (U32, Batch, Step, _clean_status, _lib, attention_ref, attention_tol,  # noqa: F401  (fixtures)
                                check_logprobs, f64, i32, randn, run_attention, run_logprobs)

pytestmark = pytest.mark.gpu


# ---- after a failure ------------------------------------------------------------------

@pytest.mark.parametrize("hq,hkv,hd,pre,new", [
    (16, 8, 128, [9000, 3, 700, 0, 2500], [24, 1, 7, 13, 30]),
    (4, 1, 64, [40000], [33]),
    (8, 8, 128, [2048], [1]),
    (8, 2, 128, [4000, 4100], [61, 33]),
])
def test_a_captured_attention_recovers_from_a_failure(hq, hkv, hd, pre, new):
    # A launch that finds the record of an earlier failure set gives up and leaves
    # flags of its pieces up in the workspace; the replays after dg_op_status has
    # told of it must not take them for their own.  Each turn has queries of its
    # own: pieces of another turn would show.
    rng = np.random.default_rng(51)
    bt = Batch(rng, pre, new, hkv, hd, 128)
    n = dgp.dg_op_tree_attention_workspace_bytes(bt.T, len(pre), hq, hkv, hd)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev())
    q, out = randn(rng, bt.T, hq, hd).to(dev()), torch.empty(bt.T, hq, hd, dtype=torch.bfloat16, device=dev())
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        run_attention(bt, q, None, out, workspace=ws, stream=st)
    for turn in range(12):
        dgp.dg_op_wait_selftest(20_000)
        g.replay()
        torch.cuda.synchronize()
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_status()
        assert e.value.code == dgp.DG_ETIMEOUT
        dgp.dg_op_status()                                  # cleared
        for _ in range(3):
            q.copy_(randn(rng, bt.T, hq, hd))
            want = torch.full_like(out, 7.0)
            run_attention(bt, q, None, want)                # a workspace of its own
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            dgp.dg_op_status()
            assert torch.equal(out, want), turn


# ---- values at the ends of their types --------------------------------------------------

@pytest.mark.parametrize("hq,hkv,hd,pre,new", [
    (8, 8, 128, [2048], [3]),                     # a unit in a few pieces
    (4, 1, 64, [40000], [3]),                     # in many
    (4, 2, 64, [10], [3]),                        # in one
])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_a_number_gives_nan_and_stays_apart(hq, hkv, hd, pre, new, value):
    rng = np.random.default_rng(53)
    bt = Batch(rng, pre, new, hkv, hd, 64)
    q = randn(rng, bt.T, hq, hd)
    q[1, 2, 5] = value
    out = torch.full((bt.T, hq, hd), 7.0, dtype=torch.bfloat16, device=dev())
    run_attention(bt, q.to(dev()), None, out)
    q[1, 2, 5] = 0.0
    ref, mag = attention_ref(f64(q), bt, None, hd ** -0.5)
    got, n = f64(out), int(bt.off[-1])
    assert np.isnan(got[1, 2]).all()
    got[1, 2] = ref[1, 2]
    assert (np.abs(got[:n] - ref[:n]) <= attention_tol(ref[:n], mag[:n])).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [700, 131072])
def test_logprobs_of_rows_that_overflow_downwards(V, bf16):
    low = float(torch.finfo(torch.bfloat16 if bf16 else torch.float32).min)
    x = np.full((4, V), low, np.float32)
    x[1, V // 3] = 2.0
    x[2, V - 1] = low / 2
    x[3, 5], x[3, 6] = low / 2, -np.inf
    x = torch.from_numpy(x)
    x = (x.to(torch.bfloat16) if bf16 else x).to(dev())
    tokens = np.array([[0, V - 1], [V // 3, 0], [V - 1, 0], [5, 6]])
    for tau in (0.7, 0.3, 1.0, 2.0):
        for r in range(4):                           # (tolerances go by the largest value of a call)
            with np.errstate(over="ignore"):         # (the reference's products)
                check_logprobs(x[r:r + 1], tokens[r:r + 1], 20, 1.0 / tau)


# ---- refusals of the binding ---------------------------------------------------------------

def test_an_empty_mask_is_refused():
    rng = np.random.default_rng(54)
    bt = Batch(rng, [100], [4], 2, 64, 64)
    q = randn(rng, bt.T, 4, 64).to(dev())
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(bt.T, 1, 4, 2, 64), dtype=torch.uint8, device=dev())
    for shape in ((bt.T, 0), (bt.T,), (1, bt.T), (bt.T, 1, 1)):
        mask = torch.zeros(shape, dtype=torch.int64, device=dev())
        with pytest.raises(dgp.DgError) as e:
            dgp.dg_op_tree_attention(q, bt.k_pool, bt.v_pool, **bt.d, tree_mask=mask, out=out, workspace=ws)
        assert e.value.code == dgp.DG_EINVAL and "tree_mask" in str(e.value)
    assert (out == 7.0).all()


# ---- torch's current stream ----------------------------------------------------------------

def test_calls_without_a_stream_take_the_current_one():
    rng = np.random.default_rng(55)
    s = Step(rng, [500, 20], [30, 3], pad=1)
    s.run()                                          # (a kernel's first launch may wait for the GPU)
    rows, st = s.rows.clone(), torch.cuda.Stream()
    s.rows.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)                # some ms in which the rows are not there yet
        s.rows.copy_(rows)
        s.run()
    torch.cuda.synchronize()
    dgp.dg_op_status()
    s.check()


def test_calls_without_a_stream_are_captured():
    rng = np.random.default_rng(56)
    s = Step(rng, [500, 20], [30, 3], pad=1)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    s.rows.copy_(randn(rng, *s.rows.shape))
    for t in (s.q, s.out, s.logits, s.lp, s.H, s.ids):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    dgp.dg_op_status()
    s.check()


def test_status_without_a_stream_waits_for_the_current_one():
    x = torch.zeros(1, 100, device=dev())
    lp, tok = torch.zeros(1, 1, device=dev()), i32([[100]])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        dgp.dg_op_token_logprobs(x, tok, lp, stream=st)
        with pytest.raises(dgp.DgError):
            dgp.dg_op_status()
    torch.cuda.synchronize()


# ---- log probabilities of rows split over several blocks, and of many given tokens ------------

@pytest.mark.parametrize("bf16", [False, True])
def test_logprobs_of_split_rows_ties_order_and_masks(bf16):
    # 16 rows and fewer of 131072 and more entries are split over several blocks
    V = 131072
    rng = np.random.default_rng(61)
    at = np.arange(V)
    rows = [np.zeros(V), at // 512, -(at // 512), np.where(at < V - 3, -np.inf, 1.0), np.where(at < 5, 1.0, -np.inf), np.full(V, -np.inf),
            np.where(at // 8192 % 2, -np.inf, rng.integers(0, 3, V)), np.where(rng.random(V) < 0.999, -np.inf, rng.integers(0, 3, V)),
            np.where(at % 8192 == 0, 3.0, 0.0), np.where(at == 77777, 80.0, -80.0)]
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    x = (x.to(torch.bfloat16) if bf16 else x).to(dev())
    tokens = rng.integers(0, V, (len(rows), 3))
    tokens[:, 1], tokens[9, 2] = V - 1, 77777
    check_logprobs(x, tokens, 32)
    check_logprobs(x[3:5], tokens[3:5], 7)
    check_logprobs(x[6:7, :V - 5], tokens[6:7, :1] // 2, 32, 0.5)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("at", [0, 60000, 131071])
def test_logprobs_of_split_rows_with_one_bad_entry(bf16, at):
    V = 131072
    x = torch.zeros(4, V, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    x[1, at], x[2, at], x[3, at] = float("nan"), float("inf"), float("-inf")
    lp, H, lse, ids, top = run_logprobs(x, np.array([[at], [at], [at], [(at + 1) % V]]), 4)
    dgp.dg_op_status()
    for r in (1, 2):
        assert np.isnan(lp[r]).all() and np.isnan(H[r]) and np.isnan(lse[r]) and np.isnan(top[r]).all()
    first = [i for i in range(5) if i != at][:4]
    assert np.array_equal(ids[0], range(4)) and np.array_equal(ids[1], first) and np.array_equal(ids[3], first)
    assert np.array_equal(ids[2], [at] + [i for i in range(4) if i != at][:3])
    # V or V - 1 equal entries: sums of equal terms, then the log's and the subtraction's roundings
    tol = 4 * (V / 256 + 64) * U32
    for r, n in ((0, V), (3, V - 1)):
        assert abs(lp[r, 0] + np.log(n)) <= tol and abs(lse[r] - np.log(n)) <= tol and abs(H[r] - np.log(n)) <= 13 * tol


@pytest.mark.parametrize("T,V", [(3, 900), (2, 131072)])
def test_logprobs_of_many_given_tokens(T, V):
    rng = np.random.default_rng(62)
    x = torch.from_numpy((rng.standard_normal((T, V)) * 3).astype(np.float32)).to(dev())
    tokens = rng.integers(0, V, (T, 1300))
    tokens[:, 511:514], tokens[:, 1299] = [-1, V - 1, -1], 0
    check_logprobs(x, tokens, 3)


# ---- the packed-argument form -----------------------------------------------------------------

def test_packed_calls_do_what_the_calls_do():
    # every argument of a full call through both entries
    L = dgp.load()
    rng = np.random.default_rng(63)
    bt = Batch(rng, [200, 70], [9, 4], 2, 64, 64)
    T = bt.T
    rows = randn(rng, T, 10, 64).to(dev())
    gq, gk = (randn(rng, 64, dtype=torch.float32).to(dev()) for _ in range(2))
    pos = i32(rng.integers(0, 1000, T))
    mask = torch.from_numpy(rng.integers(0, 1 << 40, (T, 2))).to(dev())
    ws = torch.zeros(dgp.dg_op_tree_attention_workspace_bytes(T, 2, 4, 2, 64), dtype=torch.uint8, device=dev())
    logits = (randn(rng, T, 603, dtype=torch.float32) * 4).to(dev())
    tok = i32(rng.integers(0, 600, (T, 2)))
    d, row = bt.d, rows.stride(0)

    def both(which, name, out, args):
        got = []
        for go in (lambda a: getattr(L, name)(*a), lambda a: L.dg_op_packed(which, packed(a))):
            for o, init in out:
                o.copy_(init)
            assert go([a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]) == dgp.DG_OK
            got.append([o.clone() for o, _ in out])
        dgp.dg_op_status()
        for a, b, (o, init) in zip(*got, out):
            bits = torch.int16 if a.dtype is torch.bfloat16 else a.dtype
            assert torch.equal(a.view(bits), b.view(bits)) and not torch.equal(a.view(bits), init.view(bits))

    fill = lambda *s, dtype=torch.bfloat16: (torch.empty(*s, dtype=dtype, device=dev()), torch.full(s, 7, dtype=dtype, device=dev()))  # noqa: E731
    q, k = fill(T, 4, 64), fill(T, 3, 64)
    both(0, "dg_op_qk_norm_rope", [q, k], [rows, rows[:, 4:], 0, row, row, pos, T, 4, 2, 64, 32, 500.0, gq, gk, 1e-3, q[0], 256, k[0], 192, None])
    pools = [(p, p.clone()) for p in (bt.k_pool, bt.v_pool)]
    both(1, "dg_op_rope_kv_append", pools, [rows[:, 4:], rows[:, 7:], row, row, pos, d["prefix_lens"], d["offsets"], d["page_tables"], bt.max_pages, 2,
                                            T, 2, 64, 48, 700.0, gk, 1e-2, bt.k_pool, bt.v_pool, bt.n_pages, 64, None])
    o = fill(T, 5, 64)
    both(2, "dg_op_tree_attention", [o], [rows, row, bt.k_pool, bt.v_pool, d["page_tables"], bt.max_pages, d["prefix_lens"], d["offsets"], mask, 2, 2, T,
                                          4, 2, 64, 64, bt.n_pages, 0.2, o[0], 320, ws, ws.numel(), None])
    f = lambda *s: fill(*s, dtype=torch.float32)  # noqa: E731
    lp, H, lse, ids, top = f(T, 2), f(T), f(T), fill(T, 5, dtype=torch.int32), f(T, 5)
    both(3, "dg_op_token_logprobs", [lp, H, lse, ids, top], [logits, 0, 603, T, 600, 0.8, tok, 2, lp[0], H[0], lse[0], 5, ids[0], top[0], None])
