"""The operators that serve drafted tokens after failures, on values at the ends
of their types and in calls that other tests do not make, against the plain numpy
evaluations of test_gpu_draft_ops."""
import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from gpu_util import dev
from test_gpu_draft_ops import (Batch, Step, _clean_status, _lib, attention_ref, attention_tol,  # noqa: F401  (fixtures)
                                check_logprobs, f64, i32, randn, run_attention)

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
