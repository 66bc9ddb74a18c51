"""Refusals of the draft-serving entry points: argument checks run on the host
before any CUDA call, so the addresses here are never read."""
import numpy as np
import pytest
import torch

import discrete_diffusion_block_gb300 as dgp
from discrete_diffusion_block_gb300 import build

A = 4096                     # an aligned address that nothing reads
INF = float("inf")


@pytest.fixture(scope="module")
def L():
    build.build()
    return dgp.load()


def call(fn, base, **change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return fn(*args.values())


QK = dict(q=A, k=A, in_f32=0, q_stride=2048, k_stride=1024, positions=A, n_tok=3, hq=16, hkv=8, hd=128, rope_dim=128, rope_base=1e4, q_gain=A,
          k_gain=A, eps=1e-6, q_out=2 * A, qo_stride=2048, k_out=2 * A, ko_stride=1024, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(k_out=None), dict(q=A + 2), dict(k_out=A + 8), dict(q_stride=2040), dict(q_stride=2052), dict(ko_stride=1016),
    dict(positions=None), dict(n_tok=-1), dict(hq=-1), dict(hd=96), dict(hd=32), dict(rope_dim=136), dict(rope_dim=24), dict(rope_dim=-16),
    dict(rope_base=0.5), dict(rope_base=INF), dict(rope_base=float("nan")), dict(eps=0.0), dict(eps=float("nan")), dict(q_gain=A + 4),
    dict(q_out=A, qo_stride=4096), dict(in_f32=1, q_out=A), dict(in_f32=1, q_stride=2050),
])
def test_qk_norm_rope_refuses(L, change):
    assert call(L.dg_op_qk_norm_rope, QK, **change) == dgp.DG_EINVAL
    assert L.dg_last_error()


AP = dict(k=A, v=A, ks=1024, vs=1024, positions=None, prefix=A, offsets=A, tables=A, max_pages=4, n_seqs=2, n_tok=5, hkv=8, hd=128,
          rope_dim=128, rope_base=1e4, k_gain=None, eps=0.0, k_pool=A, v_pool=A, n_pages=9, pg=128, stream=None)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=A + 2), dict(ks=1000), dict(vs=1028), dict(prefix=None), dict(offsets=None), dict(tables=None), dict(max_pages=-1),
    dict(n_seqs=-1), dict(n_tok=-1), dict(hkv=0), dict(hd=80), dict(rope_dim=256), dict(k_gain=A), dict(k_gain=A + 4, eps=1e-6),
    dict(k_pool=None), dict(v_pool=A + 8), dict(n_pages=0), dict(pg=0),
])
def test_append_refuses(L, change):
    assert call(L.dg_op_rope_kv_append, AP, **change) == dgp.DG_EINVAL


AT = dict(q=A, qs=2048, k_pool=A, v_pool=A, tables=A, max_pages=4, prefix=A, offsets=A, mask=A, words=1, n_seqs=2, n_tok=5, hq=16, hkv=8,
          hd=128, pg=128, n_pages=9, scale=0.1, out=2 * A, os=2048, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(out=None), dict(out=A), dict(q=A + 8), dict(qs=2047), dict(os=1024), dict(k_pool=None), dict(tables=None),
    dict(prefix=None), dict(offsets=None), dict(words=0), dict(mask=None), dict(n_seqs=-1), dict(n_tok=-1), dict(hq=15), dict(hq=0),
    dict(hkv=0), dict(hq=1032), dict(hd=256), dict(pg=32), dict(pg=100), dict(n_pages=0), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=INF), dict(scale=float("nan")), dict(max_pages=-1),
    dict(n_tok=1 << 28),
])
def test_tree_attention_refuses(L, change):
    assert call(L.dg_op_tree_attention, AT, **change) == dgp.DG_EINVAL


def test_tree_attention_checks_its_workspace(L):
    need = L.dg_op_tree_attention_workspace_bytes(5, 2, 16, 8, 128)
    if need:
        assert call(L.dg_op_tree_attention, AT, ws_bytes=need - 1) == dgp.DG_EINVAL
        assert call(L.dg_op_tree_attention, AT, ws=None) == dgp.DG_EINVAL
        assert call(L.dg_op_tree_attention, AT, ws=A + 4) == dgp.DG_EINVAL
    assert L.dg_op_tree_attention_workspace_bytes(0, 0, 16, 8, 128) >= 0
    assert L.dg_op_tree_attention_workspace_bytes(5, 2, 16, 0, 128) == 0


LP = dict(logits=A, bf16=0, stride=1000, rows=4, V=1000, inv_tau=1.0, tokens=A, n_given=1, logprobs=A, entropy=A, lse=A, top_k=8, top_ids=A,
          top_logprobs=A, stream=None)


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(logits=A + 2), dict(logits=A + 1, bf16=1), dict(stride=999), dict(rows=-1), dict(V=0), dict(inv_tau=0.0),
    dict(inv_tau=INF), dict(inv_tau=float("nan")), dict(tokens=None), dict(logprobs=None), dict(n_given=-1), dict(top_k=33), dict(top_k=-1),
    dict(top_ids=None), dict(V=7, top_k=8),
])
def test_token_logprobs_refuses(L, change):
    assert call(L.dg_op_token_logprobs, LP, **change) == dgp.DG_EINVAL


def test_empty_calls_succeed_without_a_gpu(L):
    assert call(L.dg_op_qk_norm_rope, QK, n_tok=0, q=None, positions=None) == dgp.DG_OK
    assert call(L.dg_op_qk_norm_rope, QK, hq=0, hkv=0) == dgp.DG_OK
    assert call(L.dg_op_rope_kv_append, AP, n_tok=0, k=None) == dgp.DG_OK
    assert call(L.dg_op_rope_kv_append, AP, n_seqs=0, prefix=None) == dgp.DG_OK
    assert call(L.dg_op_tree_attention, AT, n_tok=0) == dgp.DG_OK
    assert call(L.dg_op_token_logprobs, LP, rows=0, logits=None) == dgp.DG_OK


def packed(args):
    import struct
    return struct.pack("=" + "".join("d" if isinstance(a, float) else "q" for a in args), *[0 if a is None else a for a in args])


@pytest.mark.parametrize("which,base,change", [
    (0, QK, dict(hd=96)), (0, QK, dict(ko_stride=1016)), (1, AP, dict(n_pages=0)), (1, AP, dict(eps=0.0, k_gain=A)), (2, AT, dict(scale=-1.0)),
    (2, AT, dict(pg=100)), (3, LP, dict(top_k=33)), (3, LP, dict(top_ids=None)),
])
def test_packed_calls_give_the_answers_of_the_calls(L, which, base, change):
    # (an empty call is accepted, a bad one refused with the same message)
    names = ("dg_op_qk_norm_rope", "dg_op_rope_kv_append", "dg_op_tree_attention", "dg_op_token_logprobs")
    empty = dict(rows=0) if which == 3 else dict(n_tok=0)
    assert L.dg_op_packed(which, packed({**base, **empty}.values())) == dgp.DG_OK
    assert call(getattr(L, names[which]), base, **change) == dgp.DG_EINVAL
    message = L.dg_last_error()
    assert L.dg_op_packed(which, packed({**base, **change}.values())) == dgp.DG_EINVAL
    assert L.dg_last_error() == message


def test_packed_calls_refuse_unknown_calls_and_wide_integers(L):
    assert L.dg_op_packed(4, packed(QK.values())) == dgp.DG_EINVAL
    assert L.dg_op_packed(0, None) == dgp.DG_EINVAL
    for which, base, name in ((0, QK, "n_tok"), (1, AP, "max_pages"), (2, AT, "n_pages"), (3, LP, "V")):
        assert L.dg_op_packed(which, packed({**base, name: 1 << 33}.values())) == dgp.DG_EINVAL
        assert b"range" in L.dg_last_error()


def test_binding_refuses_tensors_that_are_not_on_the_device():
    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(2, 4, 64, 64, dtype=torch.bfloat16)
    f = torch.zeros(2, 100)
    calls = [lambda: dgp.dg_op_qk_norm_rope(t, None, i, t, None),
             lambda: dgp.dg_op_rope_kv_append(t, t, pool, pool, i[:, None], i, torch.zeros(3, dtype=torch.int32)),
             lambda: dgp.dg_op_tree_attention(t, pool, pool, i[:, None], i, torch.zeros(3, dtype=torch.int32), None, t.clone(), None),
             lambda: dgp.dg_op_token_logprobs(f, None, None, top_ids=torch.zeros(2, 3, dtype=torch.int32)),
             lambda: dgp.dg_op_qk_norm_rope(None, None, i, None, None)]
    for c in calls:
        with pytest.raises(dgp.DgError) as e:
            c()
        assert e.value.code == dgp.DG_EINVAL


def test_pool_order_of_the_reference_in_use():
    # the swizzle that the operators' tests undo is the documented one: 16-byte
    # chunk c of slot s at chunk position c ^ (s % 8)
    from test_gpu_draft_ops import pool_rows
    pg, hd = 64, 128
    logical = np.arange(pg * hd).reshape(pg, hd)
    stored = np.zeros((1, 1, pg, hd), np.int64)
    flat = stored.reshape(hd // 64, pg, 64)
    for s in range(pg):
        for f in range(hd):
            flat[f // 64, s, 8 * (((f % 64) // 8) ^ (s % 8)) + f % 8] = logical[s, f]
    assert np.array_equal(pool_rows(stored)[0, :, 0], logical)
