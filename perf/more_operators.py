"""Measured cases of the operators that keep a long context's KV cache bounded.

Three operators work together on the paged cache when contexts grow past what
a server wants to hold: new tokens (a prompt's chunk, or one token per
sequence) attend to a sliding window of their sequence and to its first tokens,
which stay visible, and leave the log-sum-exp of their scores; from that each
cached key's attention weight is summed up over the rows that saw it; and the
keys that gathered the least are evicted, what stays being moved together into
other pages.

`own` False: plain torch operations in fp32; True: the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False
PAD = 2           # rows behind the last sequence (a batch padded for a captured step)
BLOCK = 512       # rows that the plain form scores at once


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one sequence that decodes one token of a long context: latency only
        dict(name="window 1 x 1 of 4k", op="window", seqs=1, new=1, prefix=9000, hq=16, hkv=8, hd=128, page=128, window=4096, sinks=4, ragged=0),
        # a serving batch of single tokens over contexts of up to 32k tokens, windows of 4k
        dict(name="window 64 x 1 of 4k", op="window", seqs=64, new=1, prefix=32768, hq=16, hkv=8, hd=128, page=128, window=4096, sinks=4, ragged=3),
        # chunks of uneven prompts, small heads, short windows at odd places, sinks past one page
        dict(name="window 21 x 201 of 333", op="window", seqs=21, new=201, prefix=2500, hq=12, hkv=4, hd=64, page=64, window=333, sinks=70, ragged=8),
        # a long prompt encoded in one call
        dict(name="window 16384 of 1k", op="window", seqs=1, new=16384, prefix=0, hq=16, hkv=8, hd=128, page=128, window=1024, sinks=4, ragged=0),
        # a prompt's chunk over all of a long context (a layer without a window)
        dict(name="window 2048 over 30k", op="window", seqs=1, new=2048, prefix=30000, hq=16, hkv=8, hd=128, page=128, window=0, sinks=0, ragged=0),
        # the weights of one decoded token
        dict(name="mass 1 x 1 over 8k", op="mass", seqs=1, new=1, prefix=8191, hq=16, hkv=8, hd=128, page=128, window=0, sinks=0, observe=0, ragged=0),
        # the weights of a batch's step, uneven contexts of up to 16k tokens
        dict(name="mass 48 x 1 over 16k", op="mass", seqs=48, new=1, prefix=16384, hq=16, hkv=8, hd=128, page=128, window=0, sinks=0, observe=0, ragged=5),
        # prompts of which the last 64 tokens tell what is worth keeping
        dict(name="mass 6 x 3900, last 64", op="mass", seqs=6, new=3900, prefix=0, hq=12, hkv=4, hd=64, page=64, window=0, sinks=0, observe=64, ragged=6),
        # all rows of a long prompt
        dict(name="mass 8192", op="mass", seqs=1, new=8192, prefix=0, hq=16, hkv=8, hd=128, page=128, window=0, sinks=0, observe=0, ragged=0),
        # one sequence a page over its budget
        dict(name="evict 1 x 2176 to 2048", op="evict", seqs=1, length=2176, hkv=8, hd=128, page=128, budget=2048, sinks=4, recent=256, ragged=0),
        # uneven sequences, some of them within the budget, small heads and pages
        dict(name="evict 29 x 2900 to 1111", op="evict", seqs=29, length=2900, hkv=4, hd=64, page=64, budget=1111, sinks=1, recent=100, ragged=4),
        # prompts cut down to a fraction before decoding begins
        dict(name="evict 12 x 32k to 8k", op="evict", seqs=12, length=32768, hkv=8, hd=128, page=128, budget=8192, sinks=16, recent=512, ragged=7),
    ]


HEADS = [(16, 8, 128), (16, 8, 128), (16, 4, 128), (4, 2, 64), (12, 4, 64), (8, 1, 128), (5, 5, 64), (7, 1, 64)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "mass", "evict"])
    hq, hkv, hd = rng.choice(HEADS)
    page = rng.choice([64, 128, 128, 192])
    ragged = rng.choice([0, rng.randrange(1, 1 << 20)])
    if op == "evict":
        seqs = _log_int(rng, 1, 64)
        length = _log_int(rng, 8, max(16, min(65536, 12 * 32768 * 8 * 128 // (seqs * hkv * hd))))
        budget = max(2, int(length * rng.uniform(0.1, 0.97)))
        sinks = rng.choice([0, 1, 4, rng.randrange(0, 200)])
        sinks = min(sinks, budget // 2)
        return dict(op=op, seqs=seqs, length=length, hkv=hkv, hd=hd, page=page, budget=budget, sinks=sinks,
                    recent=rng.randrange(0, budget - sinks + 1), ragged=ragged)
    seqs = _log_int(rng, 1, 64)
    new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(2, min(4096, 16384 // seqs)))
    window = 0 if rng.random() < 0.4 else _log_int(rng, 1, 8192)
    sinks = rng.choice([0, 4, rng.randrange(0, 200)]) if window else 0
    room = min(32768, 32 * 8192 * 8 * 128 // (seqs * hkv * hd), 30000000 * 16 * 128 // (seqs * new * hq * hd))
    case = dict(op=op, seqs=seqs, new=new, prefix=_log_int(rng, 1, max(2, room)) if rng.random() < 0.9 else 0, hq=hq, hkv=hkv, hd=hd,
                page=page, window=window, sinks=sinks, ragged=ragged)
    if op == "mass":
        case["observe"] = rng.choice([0, _log_int(rng, 1, 256)])
    return case


def _lens(case):
    """(cached tokens, new tokens) of each sequence, from the case alone: the
    case's own figures where "ragged" is 0, else spread below them, a few
    sequences with nothing cached and a few with nothing new."""
    if not case["ragged"]:
        return [case["prefix"]] * case["seqs"], [case["new"]] * case["seqs"]
    r = random.Random(case["ragged"])
    pre = [0 if r.random() < 0.05 else r.randint(min(1, case["prefix"]), case["prefix"]) for _ in range(case["seqs"])]
    new = [0 if r.random() < 0.05 else r.randint(1, case["new"]) for _ in range(case["seqs"])]
    pre[0], new[0] = case["prefix"], case["new"]
    return pre, new


def _lengths(case):
    """Cached tokens of each sequence before an eviction."""
    if not case["ragged"]:
        return [case["length"]] * case["seqs"]
    r = random.Random(case["ragged"])
    return [case["length"]] + [0 if r.random() < 0.05 else r.randint(1, case["length"]) for _ in range(case["seqs"] - 1)]


def _first(case, m):
    """First of m new tokens whose weights count."""
    return max(0, m - case["observe"]) if case.get("observe") else 0


def _seen(case, p, m):
    """(pairs of rows and keys, keys that some row sees) of a sequence, the
    rows those that count."""
    w, s = case["window"], case["sinks"]
    t0 = _first(case, m)
    if m == 0:
        return 0, 0
    if not w:
        return sum(range(p + t0 + 1, p + m + 1)), p + m
    slots = range(p + t0, p + m)
    low = max(0, p + t0 - w + 1)
    return sum(min(t + 1, w) + min(s, max(0, t - w + 1)) for t in slots), p + m - low + min(s, low)


def work(case):
    if case["op"] == "evict":
        row = case["hkv"] * (4 * case["hd"] + 4)
        lens = _lengths(case)
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": sum(lens) * case["hkv"] * 4 + 2 * kept * row + case["seqs"] * case["hkv"] * case["budget"] * 4,
                "flops": sum(lens) * case["hkv"]}
    pre, new = _lens(case)
    seen = [_seen(case, p, m) for p, m in zip(pre, new)]
    pairs, keys = sum(a for a, _ in seen), sum(b for _, b in seen)
    rows = sum(m - _first(case, m) for m in new) * case["hq"]
    if case["op"] == "window":
        return {"bytes": keys * case["hkv"] * case["hd"] * 4 + rows * (case["hd"] * 4 + 4), "flops": 4 * pairs * case["hq"] * case["hd"]}
    return {"bytes": keys * case["hkv"] * (case["hd"] * 2 + 8) + rows * (case["hd"] * 2 + 4), "flops": 2 * pairs * case["hq"] * case["hd"]}


# ---- inputs ------------------------------------------------------------------

def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _tables(perm, lens, page, width=None):
    """Page tables that take their pages from `perm` in turn, and how many."""
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(max(need), 1) if width is None else width), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    hkv, hd, pg = case["hkv"], case["hd"], case["page"]
    # keys of uneven weight: a few of them gather most of the attention
    keys = lambda n: (randn(n, hkv, pg, hd).to(torch.bfloat16) * torch.exp(0.4 * randn(n, hkv, pg, 1)).to(torch.bfloat16))  # noqa: E731
    if case["op"] == "evict":
        lens = _lengths(case)
        kept = [min(n, case["budget"]) for n in lens]
        n_pages = sum(-(-n // pg) for n in lens) + sum(-(-n // pg) for n in kept) + 2
        perm = r.permutation(n_pages).astype(np.int32)
        table, at = _tables(perm, lens, pg)
        out_table, _ = _tables(perm[at:], kept, pg)
        # weights spread over orders of magnitude, many keys that nothing looked at, equal ones among them
        mass = torch.exp(2.0 * randn(n_pages, hkv, pg)).mul_(64.0).round_().div_(64.0)
        return dict(case=case, k_pool=keys(n_pages), v_pool=randn(n_pages, hkv, pg, hd).to(torch.bfloat16), mass_pool=mass, table=_i32(table),
                    out_table=_i32(out_table), lens=_i32(lens), out_lens=_i32(np.zeros(len(lens))),
                    kept=torch.full((len(lens), hkv, case["budget"]), -1, dtype=torch.int32, device="cuda"), longest=max(lens))
    pre, new = _lens(case)
    hq, n = case["hq"], sum(new) + PAD
    n_pages = sum(-(-(p + m) // pg) for p, m in zip(pre, new)) + 2
    table, _ = _tables(r.permutation(n_pages).astype(np.int32), [p + m for p, m in zip(pre, new)], pg)
    if case["window"]:
        for b, p in enumerate(pre):             # pages that no window reaches any more went back to the pool
            table[b, -(-case["sinks"] // pg):max(0, p - case["window"] + 1) // pg] = -1
    s = dict(case=case, pre=pre, new=new, table=_i32(table), prefix_lens=_i32(pre), offsets=_i32(np.concatenate([[0], np.cumsum(new)])),
             q=randn(n, hq, hd).to(torch.bfloat16), k_pool=keys(n_pages))
    if case["op"] == "window":
        s.update(v_pool=randn(n_pages, hkv, pg, hd).to(torch.bfloat16), out=torch.zeros(n, hq, hd, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(n, hq, dtype=torch.float32, device="cuda"))
    else:
        s["mass_pool"] = torch.exp(randn(n_pages, hkv, pg))
        s["lse"] = torch.zeros(n, hq, dtype=torch.float32, device="cuda")
        for rows, _, _, x in _scores(s):
            s["lse"][rows] = torch.logsumexp(x.view(hkv, -1, rows.stop - rows.start, x.shape[-1]), -1).permute(2, 0, 1).reshape(-1, hq)
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _workspace(s, bytes_of):
    if "workspace" not in s:
        c = s["case"]
        s["workspace"] = torch.empty(max(bytes_of(s["q"].shape[0], c["seqs"], c["hq"], c["hkv"], c["hd"]), 1), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_window(s):
    import discrete_diffusion_block_gb300 as dgp
    c = s["case"]
    dgp.dg_op_window_attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["prefix_lens"], s["offsets"], s["out"],
                               _workspace(s, dgp.dg_op_window_attention_workspace_bytes), window=c["window"], sinks=c["sinks"], lse=s["lse"])
    return s["out"], s["lse"]


def _own_mass(s):
    import discrete_diffusion_block_gb300 as dgp
    c = s["case"]
    dgp.dg_op_key_mass(s["q"], s["lse"], s["k_pool"], s["mass_pool"], s["table"], s["prefix_lens"], s["offsets"],
                       _workspace(s, dgp.dg_op_key_mass_workspace_bytes), window=c["window"], sinks=c["sinks"], observe=c["observe"])
    return s["mass_pool"]


def _own_evict(s):
    import discrete_diffusion_block_gb300 as dgp
    c = s["case"]
    dgp.dg_op_cache_evict(s["k_pool"], s["v_pool"], s["mass_pool"], s["table"], s["out_table"], s["lens"], s["out_lens"], c["budget"],
                          sinks=c["sinks"], recent=c["recent"], kept=s["kept"])
    return s["k_pool"], s["v_pool"], s["mass_pool"], s["out_lens"], s["kept"]


def _rows_of(pool, page, slot):
    """[...][heads][hd] rows of (page, slot): the pool keeps 16-byte chunk c of
    a slot's 64-wide sub-block at chunk position c ^ (slot % 8)."""
    hkv, pg, hd = pool.shape[1:]
    x = pool.view(-1, hkv, hd // 64, pg, 64)[page, :, :, slot]
    order = torch.arange(8, device=pool.device) ^ (slot[..., None] % 8)
    x = x.view(*page.shape, hkv, hd // 64, 8, 8)
    return x.gather(-2, order[..., None, None, :, None].expand(x.shape)).view(*page.shape, hkv, hd)


def _scores(s):
    """The scaled scores of the rows that count, a block of one sequence's rows
    at a time: (rows, sequence, key slots, [hkv][G rows][keys] fp32 with -inf
    where a row does not see a key)."""
    c = s["case"]
    hq, hkv, hd, pg = c["hq"], c["hkv"], c["hd"], c["page"]
    first = 0
    for b, (p, m) in enumerate(zip(s["pre"], s["new"])):
        for t0 in range(_first(c, m), m, BLOCK):
            t1 = min(m, t0 + BLOCK)
            lo = max(0, p + t0 - c["window"] + 1) if c["window"] else 0
            j = torch.arange(lo, p + t1, device="cuda")
            if c["sinks"]:
                j = torch.cat([torch.arange(min(lo, c["sinks"]), device="cuda"), j])
            k = _rows_of(s["k_pool"], s["table"][b].long()[j // pg], j % pg).float()
            rows = slice(first + t0, first + t1)
            q = s["q"][rows].float().view(t1 - t0, hkv, hq // hkv, hd).permute(1, 2, 0, 3).reshape(hkv, -1, hd)
            x = torch.matmul(q, k.permute(1, 2, 0)) * (1.0 / math.sqrt(hd))
            at = torch.arange(p + t0, p + t1, device="cuda")[:, None]
            sees = j[None] <= at
            if c["window"]:
                sees &= (j[None] > at - c["window"]) | (j[None] < c["sinks"])
            yield rows, b, j, x.view(hkv, hq // hkv, t1 - t0, -1).masked_fill(~sees, -math.inf).view(x.shape)
        first += m


def _plain_window(s):
    c = s["case"]
    hq, hkv, hd, pg = c["hq"], c["hkv"], c["hd"], c["page"]
    out, lse = torch.zeros_like(s["q"]), torch.zeros_like(s["lse"])
    for rows, b, j, x in _scores(s):
        n = rows.stop - rows.start
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top)
        total = e.sum(-1, keepdim=True)
        v = _rows_of(s["v_pool"], s["table"][b].long()[j // pg], j % pg).float()
        o = torch.matmul(e / total, v.transpose(0, 1))
        out[rows] = o.view(hkv, hq // hkv, n, hd).permute(2, 0, 1, 3).reshape(n, hq, hd).to(torch.bfloat16)
        lse[rows] = (top + total.log()).view(hkv, hq // hkv, n).permute(2, 0, 1).reshape(n, hq)
    return out, lse


def _plain_mass(s):
    c = s["case"]
    hq, hkv, pg = c["hq"], c["hkv"], c["page"]
    # the new tokens' own keys begin at 0
    for b, (p, m) in enumerate(zip(s["pre"], s["new"])):
        j = torch.arange(p, p + m, device="cuda")
        s["mass_pool"][s["table"][b].long()[j // pg], :, j % pg] = 0.0
    for rows, b, j, x in _scores(s):
        n = rows.stop - rows.start
        lse = s["lse"][rows].view(n, hkv, hq // hkv).permute(1, 2, 0).reshape(hkv, -1, 1)
        s["mass_pool"][s["table"][b].long()[j // pg], :, j % pg] += torch.exp(x - lse).sum(1).T
    return s["mass_pool"]


def _plain_evict(s):
    c = s["case"]
    hkv, hd, pg, budget = c["hkv"], c["hd"], c["page"], c["budget"]
    n = s["lens"].long()[:, None]                                       # [B][1]
    j = torch.arange(s["longest"], device="cuda")
    page = s["table"].long()[:, j // pg].clamp(min=0)
    mass = s["mass_pool"][page, :, (j % pg)[None]].transpose(1, 2)      # [B][hkv][longest]
    # one integer key: descending weight, lowest slot first among equals; what always stays above, what is not there below
    bits = mass.add(0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 31) - j
    stays = (j[None] < c["sinks"]) | (j[None] >= n - c["recent"])
    key = torch.where(stays[:, None], (1 << 62) - j, key)
    key = torch.where((j[None] < n)[:, None], key, -(1 << 62) - j)
    k = min(budget, s["longest"])
    kept = key.topk(k, dim=2)[1]
    d = torch.arange(k, device="cuda")
    live = (d[None] < n)[:, None].expand(kept.shape)
    kept = torch.where(live, kept, s["longest"]).sort(dim=2)[0]
    s["kept"].fill_(-1)
    s["kept"][:, :, :k] = torch.where(live, kept, -1).to(torch.int32)
    b, h, i = live.nonzero(as_tuple=True)
    src = kept[b, h, i]
    sp, ss, dp, ds = s["table"].long()[b, src // pg], src % pg, s["out_table"].long()[b, i // pg], i % pg
    e = torch.arange(hd, device="cuda")
    at = lambda page, slot: (((page * hkv + h) * pg * hd)[:, None] + (e // 64) * (pg * 64) + (slot * 64)[:, None]  # noqa: E731
                             + ((e % 64 // 8)[None] ^ (slot % 8)[:, None]) * 8 + e % 8)
    for pool in (s["k_pool"], s["v_pool"]):
        flat = pool.view(-1)
        flat[at(dp, ds)] = flat[at(sp, ss)]
    s["mass_pool"][dp, h, ds] = s["mass_pool"][sp, h, ss]
    s["out_lens"].copy_(n[:, 0].clamp(max=budget))
    return s["k_pool"], s["v_pool"], s["mass_pool"], s["out_lens"], s["kept"]


_plain = dict(window=_plain_window, mass=_plain_mass, evict=_plain_evict)
_own = dict(window=_own_window, mass=_own_mass, evict=_own_evict)


# ---- the definition, in 64 bits ------------------------------------------------

def _logical(pool, table, slots):
    """Rows [slots][heads][hd] of one sequence in 64 bits, out of the flat pool."""
    hkv, pg, hd = pool.shape[1:]
    slots = slots.to(pool.device)
    page, slot = table[slots // pg].long()[:, None, None], (slots % pg)[:, None, None]
    h = torch.arange(hkv, device=pool.device)[None, :, None]
    f = torch.arange(hd, device=pool.device)[None, None, :]
    i = ((page * hkv + h) * (hd // 64) + f // 64) * pg * 64 + slot * 64 + ((f // 8 % 8) ^ (slot % 8)) * 8 + f % 8
    return pool.reshape(-1)[i].double()


def _visible(case, p, t0, t1, slots):
    """Which key slots the new tokens t0 .. t1 - 1 see."""
    back = (p + torch.arange(t0, t1, device=slots.device))[:, None] - slots[None]
    see = back >= 0
    return see & ((back < case["window"]) | (slots < case["sinks"])[None]) if case["window"] else see


def _exact_evict(case, s):
    pools = [s["k_pool"].double(), s["v_pool"].double(), s["mass_pool"].double()]
    old = [x.clone() for x in pools]
    pg, hd = case["page"], case["hd"]
    table, out = s["table"].cpu().numpy(), s["out_table"].cpu().numpy()
    mass, lens = s["mass_pool"].cpu().numpy(), s["lens"].cpu().numpy()
    kept = np.full(tuple(s["kept"].shape), -1, np.int64)
    f = torch.arange(hd, device="cuda")

    def cell(page, slot, h):
        return (((page * case["hkv"] + h) * (hd // 64))[:, None] + f // 64) * pg * 64 + (slot * 64)[:, None] \
            + ((f // 8 % 8) ^ (slot % 8)[:, None]) * 8 + f % 8

    for b, n in enumerate(lens):
        j = np.arange(n)
        for h in range(case["hkv"]):
            stay = j
            if n > case["budget"]:
                middle = j[case["sinks"]:n - case["recent"]]
                order = np.argsort(-mass[table[b, middle // pg], h, middle % pg].astype(np.float64), kind="stable")
                best = middle[order[:case["budget"] - case["sinks"] - case["recent"]]]
                stay = np.sort(np.concatenate([j[:case["sinks"]], best, j[n - case["recent"]:]]))
            kept[b, h, :len(stay)] = stay
            d = np.arange(len(stay))
            to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).long().cuda()  # noqa: E731
            src, dst = (to(table[b, stay // pg]), to(stay % pg)), (to(out[b, d // pg]), to(d % pg))
            for x, y in zip(pools[:2], old[:2]):
                x.view(-1)[cell(*dst, h)] = y.view(-1)[cell(*src, h)]
            pools[2][dst[0], h, dst[1]] = old[2][src[0], h, src[1]]
    return (*pools, torch.from_numpy(np.minimum(lens, case["budget"])).cuda(), torch.from_numpy(kept).cuda())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    hq, hd, pg = case["hq"], case["hd"], case["page"]
    grp = hq // case["hkv"]
    if case["op"] == "window":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        mass = s["mass_pool"].double()
    row = 0
    for b, (p, m) in enumerate(zip(s["pre"], s["new"])):
        slots = torch.arange(p + m, device="cuda")
        if case["op"] == "mass":
            own_slots = slots[p:]
            mass[s["table"][b, own_slots // pg].long(), :, own_slots % pg] = 0.0
        for t0 in range(_first(case, m), m, 256):
            t1 = min(m, t0 + 256)
            see = _visible(case, p, t0, t1, slots)
            some = see.any(0).nonzero()[:, 0]                 # keys that a row of the block sees
            see = see[:, some]
            k = _logical(s["k_pool"], s["table"][b], some)
            q = s["q"][row + t0:row + t1].double()
            a = torch.einsum("thd,khd->htk", q, k.repeat_interleave(grp, 1)) / math.sqrt(hd)
            a = a.masked_fill(~see[None], -math.inf)
            if case["op"] == "window":
                z = torch.logsumexp(a, -1)
                v = _logical(s["v_pool"], s["table"][b], some).repeat_interleave(grp, 1)
                out[row + t0:row + t1] = torch.einsum("htk,khd->thd", torch.exp(a - z[..., None]), v)
                lse[row + t0:row + t1] = z.T
            else:
                e = torch.exp(a - s["lse"][row + t0:row + t1].double().T[..., None]).sum(1)          # [hq][keys]
                mass[s["table"][b, some // pg].long(), :, some % pg] += e.view(-1, grp, len(some)).sum(1).T
        row += m
    return (out, lse) if case["op"] == "window" else mass
