"""Refusals of the calls that bound a long context's cache: argument checks run
on the host before any CUDA call, so the addresses here are never read."""
import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from test_draft_ops_host import A, INF, L, call, packed  # noqa: F401  (L: a fixture)

WA = dict(q=A, qs=2048, k_pool=A, v_pool=A, tables=A, max_pages=4, prefix=A, offsets=A, window=100, sinks=4, n_seqs=2, n_tok=5, hq=16, hkv=8,
          hd=128, pg=128, n_pages=9, scale=0.1, out=2 * A, os=2048, lse=A, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(out=None), dict(out=A), dict(q=A + 8), dict(qs=2047), dict(os=1024), dict(k_pool=None), dict(v_pool=A + 8),
    dict(tables=None), dict(prefix=None), dict(offsets=None), dict(window=-1), dict(sinks=-1), dict(n_seqs=-1), dict(n_tok=-1), dict(hq=15),
    dict(hq=0), dict(hkv=0), dict(hq=1032), dict(hd=256), dict(pg=32), dict(pg=100), dict(n_pages=0), dict(scale=0.0), dict(scale=INF),
    dict(scale=float("nan")), dict(scale=float(np.finfo(np.float32).max)), dict(max_pages=-1), dict(n_tok=1 << 28), dict(lse=A + 2),
])
def test_window_attention_refuses(L, change):  # noqa: F811
    assert call(L.dg_op_window_attention, WA, **change) == dgp.DG_EINVAL
    assert L.dg_last_error()


def test_window_attention_checks_its_workspace(L):  # noqa: F811
    need = L.dg_op_window_attention_workspace_bytes(5, 2, 16, 8, 128)
    assert need > 0
    assert call(L.dg_op_window_attention, WA, ws_bytes=need - 1) == dgp.DG_EINVAL
    assert call(L.dg_op_window_attention, WA, ws=None) == dgp.DG_EINVAL
    assert call(L.dg_op_window_attention, WA, ws=A + 4) == dgp.DG_EINVAL
    assert L.dg_op_window_attention_workspace_bytes(5, 2, 16, 0, 128) == 0


KM = dict(q=A, qs=2048, lse=A, k_pool=A, mass=A, tables=A, max_pages=4, prefix=A, offsets=A, window=100, sinks=4, observe=0, n_seqs=2, n_tok=5,
          hq=16, hkv=8, hd=128, pg=128, n_pages=9, scale=0.1, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(lse=None), dict(k_pool=None), dict(mass=None), dict(q=A + 8), dict(lse=A + 2), dict(mass=A + 1), dict(k_pool=A + 8),
    dict(qs=2047), dict(qs=1024), dict(tables=None), dict(prefix=None), dict(offsets=None), dict(window=-1), dict(sinks=-1), dict(observe=-1),
    dict(n_seqs=-1), dict(n_tok=-1), dict(hq=15), dict(hkv=0), dict(hq=1032), dict(hd=256), dict(pg=32), dict(pg=100), dict(n_pages=0),
    dict(scale=0.0), dict(scale=INF), dict(scale=float("nan")), dict(max_pages=-1), dict(n_tok=1 << 28), dict(qs=1 << 40), dict(scale=1e-31),
])
def test_key_mass_refuses(L, change):  # noqa: F811
    assert call(L.dg_op_key_mass, KM, **change) == dgp.DG_EINVAL
    assert L.dg_last_error()


def test_key_mass_checks_its_workspace(L):  # noqa: F811
    need = L.dg_op_key_mass_workspace_bytes(5, 2, 16, 8, 128)
    assert need > 0
    assert call(L.dg_op_key_mass, KM, ws_bytes=need - 1) == dgp.DG_EINVAL
    assert call(L.dg_op_key_mass, KM, ws=None) == dgp.DG_EINVAL
    assert call(L.dg_op_key_mass, KM, ws=A + 4) == dgp.DG_EINVAL
    assert L.dg_op_key_mass_workspace_bytes(5, 2, 16, 0, 128) == 0


EV = dict(k_pool=A, v_pool=A, mass=A, tables=A, max_pages=4, out_tables=2 * A, out_max=4, lens=A, n_seqs=2, hkv=8, hd=128, pg=128, n_pages=9,
          budget=200, sinks=4, recent=30, out_lens=2 * A, kept=A, stream=None)


@pytest.mark.parametrize("change", [
    dict(k_pool=None), dict(v_pool=None), dict(mass=None), dict(k_pool=A + 8), dict(mass=A + 2), dict(tables=None), dict(out_tables=None),
    dict(lens=None), dict(out_lens=None), dict(out_lens=A), dict(kept=None), dict(max_pages=-1), dict(out_max=-1), dict(n_seqs=-1), dict(hkv=0), dict(hd=96),
    dict(hd=256), dict(pg=0), dict(n_pages=0), dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=100, recent=101),
    dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(n_seqs=1 << 30),
])
def test_cache_evict_refuses(L, change):  # noqa: F811
    assert call(L.dg_op_cache_evict, EV, **change) == dgp.DG_EINVAL
    assert L.dg_last_error()


CALLS = [("dg_op_window_attention", 8, WA, dict(n_tok=0), dict(scale=-1.0), "n_pages"),
         ("dg_op_key_mass", 9, KM, dict(n_tok=0), dict(observe=-1), "sinks"),
         ("dg_op_cache_evict", 10, EV, dict(n_seqs=0), dict(budget=0), "recent")]


@pytest.mark.parametrize("name,which,base,empty,bad,wide", CALLS)
def test_empty_calls_succeed_and_packed_ones_answer_as_the_calls(L, name, which, base, empty, bad, wide):  # noqa: F811
    assert call(getattr(L, name), base, **empty) == dgp.DG_OK
    assert call(getattr(L, name), base, **{**empty, "n_seqs": 0}) == dgp.DG_OK
    assert L.dg_op_packed(which, packed({**base, **empty}.values())) == dgp.DG_OK
    assert call(getattr(L, name), base, **bad) == dgp.DG_EINVAL
    message = L.dg_last_error()
    assert L.dg_op_packed(which, packed({**base, **bad}.values())) == dgp.DG_EINVAL
    assert L.dg_last_error() == message
    assert L.dg_op_packed(which, packed({**base, wide: 1 << 33}.values())) == dgp.DG_EINVAL
    assert b"range" in L.dg_last_error()


def test_binding_refuses_tensors_that_are_not_on_the_device():
    t, i = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(2, 4, 64, 64, dtype=torch.bfloat16)
    calls = [lambda: dgp.dg_op_window_attention(t, pool, pool, i[:, None], i, torch.zeros(3, dtype=torch.int32), t.clone(), None),
             lambda: dgp.dg_op_key_mass(t, torch.zeros(2, 4), pool, torch.zeros(2, 4, 64), i[:, None], i, torch.zeros(3, dtype=torch.int32), None),
             lambda: dgp.dg_op_cache_evict(pool, pool, torch.zeros(2, 4, 64), i[:, None], i[:, None], i, i.clone(), 5, torch.zeros(2, 4, 5, dtype=torch.int32))]
    for c in calls:
        with pytest.raises(dgp.DgError) as e:
            c()
        assert e.value.code == dgp.DG_EINVAL
