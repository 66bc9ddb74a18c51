"""Measured cases of the operators that serve drafted tokens over the paged KV cache.

Four operators run one after the other when a decoder checks drafted tokens
(or decodes one token per sequence): the query and key heads of the new tokens
are normalised and rotated to their positions, keys and values are appended to
the cache's pages with the rotation applied on the way, the new tokens attend
to their sequence's prefix and to their ancestors in the draft tree, and the
logits give each drafted token's log probability with the distribution's
entropy and its top alternatives.

`own` False: plain torch operations in fp32 (angles in fp64); True: the
library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False
PAD = 3           # rows behind the last sequence (a batch padded for a captured step)
EPS = 1e-6
BASE = 10000.0


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # the step of one sequence that decodes one token: latency only
        dict(name="qk 1 token", op="qk", tokens=1, hq=16, hkv=8, hd=128, rope=128, f32=False, packed=True, norm=True, far=2048),
        # queries and keys of a small model's fp32 projections, odd row count, half of each head rotated
        dict(name="qk 777 fp32 rows", op="qk", tokens=777, hq=4, hkv=2, hd=64, rope=32, f32=True, packed=False, norm=True, far=100000),
        # prompt encoding: the rows of one large chunk, taken out of the packed QKV rows
        dict(name="qk 16384 tokens", op="qk", tokens=16384, hq=16, hkv=8, hd=128, rope=128, f32=False, packed=True, norm=True, far=16384),
        # a batch of drafts: a few tokens for each of 37 sequences, starting anywhere in a page
        dict(name="append 37 drafts", op="append", seqs=37, new=16, prefix=900, hkv=8, hd=128, rope=128, page=128, norm=True, tree=True, ragged=5),
        # prompt chunks of five sequences written to the cache
        dict(name="append 5 prompts", op="append", seqs=5, new=6000, prefix=500, hkv=8, hd=128, rope=128, page=128, norm=False, tree=False, ragged=6),
        # one sequence, one token: the plain decoding step
        dict(name="attend 1 x 1 over 2k", op="attend", seqs=1, new=1, prefix=2048, hq=16, hkv=8, hd=128, page=128, tree=False, ragged=0),
        # one sequence, a tree of 61 drafted tokens over a long context
        dict(name="attend 1 x 61 over 32k", op="attend", seqs=1, new=61, prefix=32700, hq=16, hkv=8, hd=128, page=128, tree=True, ragged=0),
        # a serving batch of uneven contexts, small heads, chains of a few drafted tokens
        dict(name="attend 40 x 5 ragged", op="attend", seqs=40, new=5, prefix=3000, hq=12, hkv=4, hd=64, page=64, tree=False, ragged=8),
        # a large serving batch of trees over contexts of up to 16k tokens
        dict(name="attend 64 x 24 over 16k", op="attend", seqs=64, new=24, prefix=16384, hq=16, hkv=8, hd=128, page=128, tree=True, ragged=9),
        # the next token of one sequence, full vocabulary
        dict(name="logprobs 1 x 262144", op="logprobs", rows=1, vocab=262144, given=1, top=8, f32=True, masked=False, tau=1.0),
        # the drafted tokens of a batch, an odd vocabulary, bf16 logits with some entries masked out
        dict(name="logprobs 301 x 50001 bf16", op="logprobs", rows=301, vocab=50001, given=3, top=5, f32=False, masked=True, tau=0.7),
        # scoring a text: a chunk of rows over the full vocabulary
        dict(name="logprobs 1024 x 262144", op="logprobs", rows=1024, vocab=262144, given=1, top=20, f32=True, masked=False, tau=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "append", "attend", "attend", "logprobs"])
    if op == "qk":
        hq, hkv, hd = rng.choice([(16, 8, 128), (16, 4, 128), (4, 2, 64), (12, 4, 64), (8, 1, 128), (5, 5, 64), (8, 2, 256), (6, 3, 256)])
        rope = rng.choice([hd, hd, hd // 2])
        return dict(op=op, tokens=_log_int(rng, 1, 16384 * 24 * 128 // ((hq + hkv) * hd * 2)), hq=hq, hkv=hkv, hd=hd, rope=rope,
                    f32=rng.random() < 0.3, packed=rng.random() < 0.6, norm=rng.random() < 0.8, far=_log_int(rng, 64, 1000000))
    if op == "append":
        hkv, hd = rng.choice([(8, 128), (4, 128), (2, 64), (1, 128), (3, 64), (2, 256)])
        seqs = _log_int(rng, 1, 200)
        new = _log_int(rng, 1, max(1, 24000 // seqs))
        return dict(op=op, seqs=seqs, new=new, prefix=_log_int(rng, 1, max(2, 16000 // seqs)), hkv=hkv, hd=hd, rope=rng.choice([hd, hd // 2]),
                    page=rng.choice([64, 128, 192]), norm=rng.random() < 0.6, tree=new <= 64 and rng.random() < 0.5, ragged=rng.randrange(1, 1 << 20))
    if op == "attend":
        hq, hkv, hd = rng.choice([(16, 8, 128), (16, 8, 128), (16, 4, 128), (4, 2, 64), (12, 4, 64), (8, 1, 128), (5, 5, 64), (7, 1, 64)])
        seqs, new = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        room = 400000 * 8 * 128 // (hkv * hd) // seqs // (1 + new * (hq // hkv) // 48)
        return dict(op=op, seqs=seqs, new=new, prefix=_log_int(rng, 1, max(2, min(32768, room))), hq=hq, hkv=hkv, hd=hd,
                    page=rng.choice([64, 128, 128, 192]), tree=rng.random() < 0.7, ragged=rng.randrange(1, 1 << 20))
    vocab = rng.choice([262144, _log_int(rng, 1000, 262144)])
    return dict(op=op, rows=_log_int(rng, 1, 1024), vocab=vocab, given=rng.randrange(1, 9), top=rng.randrange(1, 33),
                f32=rng.random() < 0.5, masked=rng.random() < 0.4, tau=rng.choice([1.0, 1.0, 0.7, 1.5]))


def _lens(case):
    """(cached tokens, new tokens) of each sequence, from the case alone: the
    case's own figures where "ragged" is 0, else spread below them, a few
    sequences with nothing cached and a few with nothing new."""
    if not case["ragged"]:
        return [case["prefix"]] * case["seqs"], [case["new"]] * case["seqs"]
    r = random.Random(case["ragged"])
    pre = [0 if r.random() < 0.05 else r.randint(1, case["prefix"]) for _ in range(case["seqs"])]
    new = [0 if r.random() < 0.05 else r.randint(1, case["new"]) for _ in range(case["seqs"])]
    pre[0], new[0] = case["prefix"], case["new"]
    return pre, new


def work(case):
    if case["op"] == "qk":
        e = case["tokens"] * (case["hq"] + case["hkv"]) * case["hd"]
        return {"bytes": e * ((4 if case["f32"] else 2) + 2) + 4 * case["tokens"], "flops": 8 * e}
    if case["op"] == "append":
        n = sum(_lens(case)[1])
        return {"bytes": n * case["hkv"] * case["hd"] * 8 + 4 * n, "flops": 8 * n * case["hkv"] * case["hd"]}
    if case["op"] == "attend":
        pre, new = _lens(case)
        keys = sum(p + n for p, n in zip(pre, new) if n)
        rows = sum(new) * case["hq"] * case["hd"]
        pairs = sum(n * (p + n) for p, n in zip(pre, new))
        return {"bytes": keys * case["hkv"] * case["hd"] * 4 + rows * 4, "flops": 4 * pairs * case["hq"] * case["hd"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["f32"] else 2) + case["rows"] * 8 * (1 + case["given"] + case["top"]), "flops": 6 * n}


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _trees(new, seed, tree):
    """Ancestor masks (bit j of a token's words: it sees drafted token j of its
    sequence, itself among them) and depths of one random tree per sequence;
    chains without `tree`."""
    r = np.random.default_rng(seed)
    words = max(1, -(-max(new) // 64))
    mask, depth = np.zeros((sum(new) + PAD, words), np.uint64), np.zeros(sum(new) + PAD, np.int64)
    t0 = 0
    for n in new:
        for j in range(n):
            parent = j - 1 if not tree else int(r.integers(-1, j)) if j else -1
            if parent >= 0:
                mask[t0 + j] = mask[t0 + parent]
                depth[t0 + j] = depth[t0 + parent] + 1
            mask[t0 + j, j // 64] |= np.uint64(1 << (j % 64))
        t0 += n
    return mask, depth


def _paged(case, seed, pre, new):
    """Page tables over shuffled pages, sequence offsets and cached lengths."""
    pg = case["page"]
    need = [-(-(p + n) // pg) for p, n in zip(pre, new)]
    n_pages = sum(need) + 2
    perm = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
    table = np.zeros((len(pre), max(max(need), 1)), np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return dict(table=_i32(table), pre=_i32(pre), offsets=_i32(np.concatenate([[0], np.cumsum(new)])), n_pages=n_pages)


def prepare(case, seed):
    g = _gen(seed)
    r = np.random.default_rng(seed)
    randn = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(dtype)  # noqa: E731
    if case["op"] == "qk":
        T, hq, hkv, hd = case["tokens"], case["hq"], case["hkv"], case["hd"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        if case["packed"]:                      # q and k are columns of the projection's packed rows
            rows = randn(T, hq + 2 * hkv, hd, dtype=dt)
            q, k = rows[:, :hq], rows[:, hq:hq + hkv]
        else:
            q, k = randn(T, hq, hd, dtype=dt), randn(T, hkv, hd, dtype=dt)
        s = dict(q=q, k=k, positions=_i32(r.integers(0, case["far"], T)),
                 q_out=torch.zeros(T, hq, hd, dtype=torch.bfloat16, device="cuda"), k_out=torch.zeros(T, hkv, hd, dtype=torch.bfloat16, device="cuda"))
        s["q_gain"], s["k_gain"] = [1.0 + 0.2 * randn(hd, dtype=torch.float32) if case["norm"] else None for _ in range(2)]
    elif case["op"] == "append":
        pre, new = _lens(case)
        hkv, hd, n = case["hkv"], case["hd"], sum(new) + PAD
        s = _paged(case, seed, pre, new)
        depth = _trees(new, seed, True)[1] if case["tree"] else np.concatenate([np.arange(m) for m in new] + [np.zeros(PAD, np.int64)])
        rows = randn(n, 2 * hkv, hd)            # the projection's K and V columns
        s.update(k=rows[:, :hkv], v=rows[:, hkv:], positions=_i32(depth + np.concatenate([np.repeat(pre, new), np.zeros(PAD, np.int64)])),
                 k_gain=1.0 + 0.2 * randn(hd, dtype=torch.float32) if case["norm"] else None,
                 k_pool=randn(s["n_pages"], hkv, case["page"], hd), v_pool=randn(s["n_pages"], hkv, case["page"], hd))
    elif case["op"] == "attend":
        pre, new = _lens(case)
        hq, hkv, hd, n = case["hq"], case["hkv"], case["hd"], sum(new) + PAD
        s = _paged(case, seed, pre, new)
        s.update(q=randn(n, hq, hd), out=torch.zeros(n, hq, hd, dtype=torch.bfloat16, device="cuda"),
                 k_pool=randn(s["n_pages"], hkv, case["page"], hd), v_pool=randn(s["n_pages"], hkv, case["page"], hd))
        s["mask"] = torch.from_numpy(_trees(new, seed, case["tree"])[0].view(np.int64)).cuda() if case["tree"] else None
        s["max_keys"], s["max_new"] = max(p + m for p, m in zip(pre, new)), max(new)
    else:
        T, V = case["rows"], case["vocab"]
        logits = torch.randn(T, V, generator=g, device="cuda", dtype=torch.float32).mul_(3.0)
        peak = torch.randint(0, V, (T, 4), generator=g, device="cuda")
        logits.scatter_add_(1, peak, torch.rand(T, 4, generator=g, device="cuda") * 14.0)     # a few likely tokens
        if case["masked"]:                      # a grammar or a token filter leaves a part of the vocabulary
            logits.masked_fill_(torch.rand(T, V, generator=g, device="cuda") < 0.3, -math.inf)
        if not case["f32"]:
            logits = logits.to(torch.bfloat16)
        tokens = torch.randint(0, V, (T, case["given"]), generator=g, device="cuda", dtype=torch.int32)
        tokens[:, 0] = peak[:, 0].to(torch.int32)
        f = lambda *sh: torch.zeros(*sh, dtype=torch.float32, device="cuda")  # noqa: E731
        s = dict(logits=logits, tokens=tokens, logprobs=f(T, case["given"]), entropy=f(T), lse=f(T), top_logprobs=f(T, case["top"]),
                 top_ids=torch.zeros(T, case["top"], dtype=torch.int32, device="cuda"))
    s["case"] = case
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _own_qk(s):
    import discrete_diffusion_block_gb300 as dgp
    dgp.dg_op_qk_norm_rope(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS,
                           rope_base=BASE, rope_dim=s["case"]["rope"])
    return s["q_out"], s["k_out"]


def _own_append(s):
    import discrete_diffusion_block_gb300 as dgp
    dgp.dg_op_rope_kv_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["pre"], s["offsets"], positions=s["positions"],
                             k_gain=s["k_gain"], eps=EPS, rope_base=BASE, rope_dim=s["case"]["rope"])
    return s["k_pool"], s["v_pool"]


def _own_attend(s):
    import discrete_diffusion_block_gb300 as dgp
    if "workspace" not in s:
        c = s["case"]
        n = dgp.dg_op_tree_attention_workspace_bytes(s["q"].shape[0], c["seqs"], c["hq"], c["hkv"], c["hd"])
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    dgp.dg_op_tree_attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["pre"], s["offsets"], s["mask"], s["out"], s["workspace"])
    return s["out"]


def _own_logprobs(s):
    import discrete_diffusion_block_gb300 as dgp
    dgp.dg_op_token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["entropy"], s["lse"], s["top_ids"], s["top_logprobs"],
                             inv_tau=1.0 / s["case"]["tau"])
    return s["logprobs"], s["entropy"], s["lse"], s["top_ids"], s["top_logprobs"]


def _norm_rope(x, gain, positions, rope):
    """RMSNorm of each head (where it has a gain), then the rotation of the
    pairs (j, j + rope / 2) by position * base^(-2 j / rope), rounded once."""
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
    half = rope // 2
    inv = BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = positions.double()[:, None] * inv
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    lo, hi, rest = x[..., :half], x[..., half:rope], x[..., rope:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, rest], -1).to(torch.bfloat16)


def _plain_qk(s):
    rope = s["case"]["rope"]
    return _norm_rope(s["q"], s["q_gain"], s["positions"], rope), _norm_rope(s["k"], s["k_gain"], s["positions"], rope)


def _chunks(rows, hd):
    """Pool order of 8-element chunks inside a slot's hd / 64 sub-blocks: chunk c at position c ^ (slot % 8)."""
    return torch.arange(8, device=rows.device)[None, :] ^ (rows[:, None] % 8)


def _plain_append(s):
    c = s["case"]
    hkv, hd, pg = c["hkv"], c["hd"], c["page"]
    off = s["offsets"].long()
    n = s["k"].shape[0]
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(off, t, right=True) - 1
    live = (b < c["seqs"]).nonzero()[:, 0]
    t, b = t[live], b[live]
    p = s["pre"].long()[b] + t - off[b]
    page, slot = s["table"].long()[b, p // pg], p % pg
    k, v = _norm_rope(s["k"], s["k_gain"], s["positions"], c["rope"])[t], s["v"][t]
    order = _chunks(slot, hd)
    for pool, x in ((s["k_pool"], k), (s["v_pool"], v)):
        x = x.reshape(-1, hkv, hd // 64, 8, 8)
        x = x.gather(3, order[:, None, None, :, None].expand(x.shape))
        pool.view(-1, hkv, hd // 64, pg, 64)[page, :, :, slot] = x.reshape(-1, hkv, hd // 64, 64)
    return s["k_pool"], s["v_pool"]


def _plain_attend(s):
    c = s["case"]
    B, hq, hkv, hd, pg, N = c["seqs"], c["hq"], c["hkv"], c["hd"], c["page"], s["max_new"]
    off, pre = s["offsets"].long(), s["pre"].long()
    n = off[1:] - off[:-1]
    p = torch.arange(s["max_keys"], device="cuda")
    page = s["table"].long()[:, (p // pg).clamp(max=s["table"].shape[1] - 1)]
    order = _chunks(p % pg, hd)

    def cached(pool):                                                      # [B][hkv][keys][hd] fp32
        x = pool.view(-1, hkv, hd // 64, pg, 64)[page, :, :, (p % pg)[None]].view(B, -1, hkv, hd // 64, 8, 8)
        x = x.gather(4, order[None, :, None, None, :, None].expand(x.shape))
        return x.reshape(B, -1, hkv, hd).float().transpose(1, 2)

    j = torch.arange(N, device="cuda")
    rows = (off[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)             # [B][N]
    q = s["q"][rows].float().view(B, N, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, hd)
    d = p[None] - pre[:, None]                                             # [B][keys]: drafted index, < 0 in the prefix
    dn = d.clamp(0, N - 1)
    if s["mask"] is None:
        sees = dn[:, None] <= j[None, :, None]
    else:
        words = s["mask"][rows]                                            # [B][N][words]
        sees = (words.gather(2, (dn // 64)[:, None].expand(-1, N, -1)) >> (dn % 64)[:, None]) & 1 == 1
    sees = torch.where((d < 0)[:, None], True, sees & (d < n[:, None])[:, None])
    x = torch.matmul(q, cached(s["k_pool"]).transpose(2, 3)) * (1.0 / math.sqrt(hd))
    x = x.view(B, hkv, hq // hkv, N, -1).masked_fill(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(x.view(B, hkv, -1, x.shape[-1]), cached(s["v_pool"])).view(B, hkv, hq // hkv, N, hd)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, hq, hd).to(torch.bfloat16)
    out = torch.zeros_like(s["q"])
    live = j[None] < n[:, None]
    out[rows[live]] = o[live]
    return out


def _plain_logprobs(s):
    x = s["logits"].float() * (1.0 / s["case"]["tau"])
    lse = x.max(1, keepdim=True)[0]
    lse = lse + (x - lse).exp().double().sum(1, keepdim=True).log().float()
    lp = x - lse
    entropy = -torch.where(lp == -math.inf, 0.0, lp.exp() * lp).double().sum(1).float()
    # descending value, lowest index first among equals: one integer key
    bits = s["logits"].float().add(0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (s["logits"].shape[1] - 1 - torch.arange(x.shape[1], device=x.device))
    ids = key.topk(s["case"]["top"], dim=1)[1]
    return lp.gather(1, s["tokens"].long()), entropy, lse[:, 0], ids.to(torch.int32), lp.gather(1, ids)


_plain = dict(qk=_plain_qk, append=_plain_append, attend=_plain_attend, logprobs=_plain_logprobs)
_own = dict(qk=_own_qk, append=_own_append, attend=_own_attend, logprobs=_own_logprobs)


# ---- the definition, in 64 bits ------------------------------------------------

def _exact_head(x, gain, positions, rope):
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS) * gain.double()
    # the rotation as a product of complex numbers
    half = rope // 2
    freq = torch.exp(torch.arange(half, device=x.device, dtype=torch.float64) * (-2.0 * math.log(BASE) / rope))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), positions.double()[:, None, None] * freq)
    z = torch.complex(y[..., :half], y[..., half:rope]) * turn
    y = y.clone()
    y[..., :half], y[..., half:rope] = z.real, z.imag
    return y


def _slots(pool, page, slot, hd):
    """Index of each element of (page, slot) rows in a flat pool: [rows][heads][hd]."""
    hkv, pg = pool.shape[1], pool.shape[2]
    f = torch.arange(hd, device=pool.device)
    inner = (f // 64)[None] * pg * 64 + slot[:, None] * 64 + ((f % 64 // 8)[None] ^ (slot[:, None] % 8)) * 8 + f[None] % 8
    return ((page[:, None] * hkv + torch.arange(hkv, device=pool.device)[None]) * pg * hd)[:, :, None] + inner[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return tuple(_exact_head(s[x], s[x + "_gain"], s["positions"], case["rope"]) for x in "qk")
    if case["op"] == "logprobs":
        lp, ent, lse, tops = [], [], [], []
        for r in range(case["rows"]):
            y = s["logits"][r].double() / case["tau"]
            z = torch.logsumexp(y, 0)
            p = torch.exp(y - z)
            lp.append(y[s["tokens"][r].long()] - z)
            ent.append(z - (p * y.clamp(min=-1e300)).sum())
            lse.append(z)
            tops.append(torch.sort(y, descending=True, stable=True)[0][:case["top"]] - z)
        return torch.stack(lp), torch.stack(ent), torch.stack(lse), None, torch.stack(tops)
    pre, new = _lens(case)
    hd, pg = case["hd"], case["page"]
    t0 = 0
    if case["op"] == "append":
        k = _exact_head(s["k"], s["k_gain"], s["positions"], case["rope"])
        pools = [s["k_pool"].double(), s["v_pool"].double()]
        for b, (p, m) in enumerate(zip(pre, new)):
            at = torch.arange(p, p + m, device="cuda")
            i = _slots(s["k_pool"], s["table"][b, at // pg].long(), at % pg, hd)
            for pool, x in zip(pools, (k, s["v"].double())):
                pool.view(-1)[i] = x[t0:t0 + m]
            t0 += m
        return tuple(pools)
    out = s["out"].double()
    grp = case["hq"] // case["hkv"]
    for b, (p, m) in enumerate(zip(pre, new)):
        if not m:
            continue
        at = torch.arange(p + m, device="cuda")
        i = _slots(s["k_pool"], s["table"][b, at // pg].long(), at % pg, hd)
        k, v = (s[x].view(-1)[i].double().repeat_interleave(grp, 1) for x in ("k_pool", "v_pool"))
        see = torch.ones(m, p + m, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            see[:, p:] = torch.ones(m, m, device="cuda").tril().bool()
        else:
            w = s["mask"][t0:t0 + m].cpu().numpy().view(np.uint8).reshape(m, -1)
            see[:, p:] = torch.from_numpy(np.unpackbits(w, axis=1, bitorder="little")[:, :m].astype(bool)).cuda()
        a = torch.einsum("thd,khd->htk", s["q"][t0:t0 + m].double(), k) / math.sqrt(hd)
        a = torch.softmax(a.masked_fill(~see[None], -math.inf), -1)
        out[t0:t0 + m] = torch.einsum("htk,khd->thd", a, v)
        t0 += m
    return out
