"""Cases of the serving operators: attention over an 8-bit key/value cache, the appends that write the
caches, and the block tables and slot maps that place new tokens.

Every case is a dict of plain values with an "op":
  decode8   attention of the newest Nq tokens of every sequence over an E4M3 cache with one float32 factor
            per block of tokens and KV head (page_size 0: contiguous cache, blocks of 128 tokens; else pages)
  append8   new keys and values quantised into such a cache (paged or contiguous)
  append16  new keys and values copied into a 16-bit paged cache through a slot map
  tables    pages of a free list given to the requests' new tokens: block table, slot map, new lengths

`own` false: the plain forms, elementary torch operations in 32 bits. `own` true: the calls of
exact_tiled_attention_36_b200.binding.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # the smallest block factor is 2^MIN_EXP (a block of zeros)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short conversation answered token by token: latency decides
        dict(name="decode8_one_short", op="decode8", B=1, Hq=8, Hkv=2, Nq=1, cap=512, d=128, dtype="bf16",
             causal=False, page=64, min_len=300, max_len=300, len_seed=1),
        # a full batch of 8192-key contiguous caches, grouped heads: the memory-bound ordinary step
        dict(name="decode8_batch_contiguous", op="decode8", B=32, Hq=32, Hkv=8, Nq=1, cap=8192, d=128, dtype="bf16",
             causal=False, page=0, min_len=8192, max_len=8192, len_seed=0),
        # continuous batching: every sequence at its own length, 64-token pages
        dict(name="decode8_paged_ragged", op="decode8", B=32, Hq=32, Hkv=8, Nq=1, cap=8192, d=128, dtype="bf16",
             causal=False, page=64, min_len=1, max_len=8192, len_seed=7),
        # speculative decoding: four drafted tokens a sequence, causal among themselves
        dict(name="decode8_speculative", op="decode8", B=32, Hq=32, Hkv=8, Nq=4, cap=8192, d=128, dtype="bf16",
             causal=True, page=128, min_len=5000, max_len=8191, len_seed=8),
        # small heads in fp16 with small pages
        dict(name="decode8_d64_small_pages", op="decode8", B=48, Hq=32, Hkv=8, Nq=1, cap=4096, d=64, dtype="fp16",
             causal=False, page=16, min_len=1000, max_len=4095, len_seed=9),
        # two very long documents: the keys of a few sequences spread over the whole GPU
        dict(name="decode8_long_context", op="decode8", B=2, Hq=32, Hkv=4, Nq=1, cap=131072, d=128, dtype="bf16",
             causal=False, page=256, min_len=100001, max_len=131072, len_seed=10),
        # one decode step's write: one token a sequence, most pages partly filled
        dict(name="append8_decode_step", op="append8", B=64, Hkv=8, cap=4096, d=128, dtype="bf16", page=64,
             max_old=4000, min_new=1, max_new=1, len_seed=11),
        # prompts of different lengths written in one go
        dict(name="append8_prompts", op="append8", B=12, Hkv=8, cap=8192, d=128, dtype="bf16", page=64,
             max_old=0, min_new=100, max_new=3000, len_seed=12),
        # chunks of prompts continued in contiguous fp16 caches
        dict(name="append8_contiguous_chunks", op="append8", B=16, Hkv=4, cap=4096, d=64, dtype="fp16", page=0,
             max_old=3000, min_new=0, max_new=700, len_seed=13),
        # prompts written to the 16-bit paged cache, keys and values as views of one packed projection
        dict(name="append16_prompts", op="append16", B=12, Hkv=8, cap=8192, d=128, dtype="bf16", page=16,
             max_old=1000, min_new=100, max_new=3000, len_seed=14),
        # one decode step of a large batch: few requests need a page
        dict(name="tables_decode_step", op="tables", B=256, cap=8192, page=64, max_old=8000, min_new=1, max_new=1,
             len_seed=15),
        # prompts arriving next to running requests
        dict(name="tables_prompts", op="tables", B=96, cap=8192, page=16, max_old=4000, min_new=0, max_new=4000,
             len_seed=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode8", "decode8", "decode8", "append8", "append8", "append16", "tables"])
    seed = rng.randrange(1 << 20)
    if op == "decode8":
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 4, 5, 8])
        Nq = rng.choice([1, 1, 1, 2, 4, 7])
        B = _log(rng, 1, 128)
        most = max(64, 32 * 8192 * 8 * 128 // (B * Hkv * d))
        hi = _log(rng, 30, min(131072, most))
        page = rng.choice([0, 16, 32, 64, 128, 256])
        unit = page or 1  # a contiguous cache ends anywhere
        return dict(op=op, B=B, Hq=group * Hkv, Hkv=Hkv, Nq=Nq, cap=-(-hi // unit) * unit, d=d,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), causal=rng.random() < 0.5, page=page,
                    min_len=rng.choice([1, hi // 2 + 1, hi]), max_len=hi, len_seed=seed)
    if op in ("append8", "append16"):
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, 18000 // B))
        old = rng.choice([0, 17, 1000, 4000])
        page = rng.choice([16, 32, 64, 128, 256])
        if op == "append8":
            page = rng.choice([0, 16, 32, 64, 128, 256])
        unit = page or 128
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 3, 4, 8]), cap=-(-(old + hi) // unit) * unit,
                    d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]), page=page, max_old=old,
                    min_new=rng.choice([0, 1, hi]), max_new=hi, len_seed=seed)
    B = _log(rng, 1, 1024)
    hi = _log(rng, 1, max(2, 180000 // B))
    old = rng.choice([0, 100, 5000])
    page = rng.choice([16, 32, 64, 128, 256])
    return dict(op=op, B=B, cap=-(-(old + hi) // page) * page, page=page, max_old=old,
                min_new=rng.choice([0, 1, hi]), max_new=hi, len_seed=seed)


def _lengths(case):
    """Host lengths of a case: keys of a sequence (decode8), or (keys before, new tokens)."""
    r = random.Random(case["len_seed"])
    B = case["B"]
    if case["op"] == "decode8":
        return [r.randint(case["min_len"], case["max_len"]) for _ in range(B)]
    olds = [r.randint(0, case["max_old"]) for _ in range(B)]
    news = [r.randint(case["min_new"], case["max_new"]) for _ in range(B)]
    if sum(news) == 0:
        news[0] = 1
    return olds, news


def work(case):
    op = case["op"]
    if op == "decode8":
        lens = _lengths(case)
        B, Hq, Hkv, Nq, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "d"))
        unit = case["page"] or 128
        keys = sum(lens)
        blocks = sum(-(-n // unit) for n in lens)
        by = 2 * keys * Hkv * d + 2 * 4 * blocks * Hkv + 4 * B + (4 * blocks if case["page"] else 0)
        by += 2 * 2 * B * Nq * Hq * d + 4 * B * Hq * Nq
        return {"bytes": by, "flops": 4 * keys * Hq * Nq * d}
    olds, news = _lengths(case)
    B, total, page = case["B"], sum(news), case["page"]
    if op == "append8":
        unit = page or 128
        row = case["Hkv"] * case["d"]
        touched = sum((o + n - 1) // unit - o // unit + 1 for o, n in zip(olds, news) if n > 0)
        kept = sum(1 for o, n in zip(olds, news) if n > 0 and o % unit)
        by = 2 * total * row * (2 + 1) + 2 * 4 * (touched + kept) * case["Hkv"] + 4 * (3 * B + 1)
        return {"bytes": by + (4 * touched if page else 0), "flops": 4 * total * row}
    if op == "append16":
        return {"bytes": 2 * total * case["Hkv"] * case["d"] * 2 * 2 + 4 * total, "flops": 0}
    fresh = sum(-(-(o + n) // page) - -(-o // page) for o, n in zip(olds, news))
    return {"bytes": 4 * (2 * B + 2 * fresh + total + (B + 1) + B + 1) + 4 * B, "flops": 0}


# ---------------------------------------------------------------------------------------- prepare
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _codes(g, shape):
    """E4M3 codes of normal values times 64 (the largest of millions stays below 448)."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device="cuda").mul_(64.0).clamp_(-E4M3_MAX, E4M3_MAX)
        flat[i:i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _factors(g, shape):
    """Block factors 2^-7, 2^-6 or 2^-5: blocks whose values have a standard deviation of 1/2, 1 or 2."""
    return torch.exp2(torch.randint(-7, -4, shape, generator=g, device="cuda").float())


def _tables(g, B, per_seq, spare=3):
    """A block table with every page used once, in random order, and the number of pages."""
    pages = B * per_seq + spare
    order = torch.randperm(pages, generator=g, device="cuda")[:B * per_seq]
    return order.to(torch.int32).view(B, per_seq).contiguous(), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["B"]
    st = {"case": case}
    if op == "decode8":
        Hq, Hkv, Nq, d, cap, page = (case[n] for n in ("Hq", "Hkv", "Nq", "d", "cap", "page"))
        lens = _lengths(case)
        dt = TYPES[case["dtype"]]
        st["q"] = torch.randn(B, Nq, Hq, d, generator=g, device="cuda").to(dt)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(B, Hq, Nq, device="cuda")
        # a batch of full contiguous caches gives no lengths
        st["lens"] = None if not page and min(lens) == cap else _i32(lens)
        if page:
            st["table"], n = _tables(g, B, cap // page)
            st["k"], st["v"] = _codes(g, (n, page, Hkv, d)), _codes(g, (n, page, Hkv, d))
            st["ks"], st["vs"] = _factors(g, (n, Hkv)), _factors(g, (n, Hkv))
        else:
            st["table"] = None
            st["k"], st["v"] = _codes(g, (B, cap, Hkv, d)), _codes(g, (B, cap, Hkv, d))
            st["ks"], st["vs"] = _factors(g, (B, Hkv, -(-cap // 128))), _factors(g, (B, Hkv, -(-cap // 128)))
            for b, n in enumerate(lens):  # rows past a sequence's length hold anything, NaN codes too
                st["k"][b, n:] |= 0x7F
                st["v"][b, n:] |= 0x7F
        return st
    olds, news = _lengths(case)
    total = sum(news)
    st["olds"], st["news"] = _i32(olds), _i32(news)
    st["lens"] = _i32([o + n for o, n in zip(olds, news)])
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    st["cu"], st["total"], st["max_new"] = _i32(cu), total, max(news)
    cap, page = case["cap"], case["page"]
    if op == "tables":
        st["table0"], n = _tables(g, B, cap // page)
        have = (st["olds"].long() + page - 1) // page
        used = torch.arange(cap // page, device="cuda")[None, :] < have[:, None]
        st["num_pages"] = n
        st["free"] = st["table0"][~used].contiguous()  # the pages no request holds
        if st["free"].numel() == 0:
            st["free"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["free"] = st["free"][torch.randperm(st["free"].numel(), generator=g, device="cuda")].contiguous()
        st["table"] = torch.where(used, st["table0"], torch.full_like(st["table0"], -1))
        st["slots"] = torch.empty(total, dtype=torch.int32, device="cuda")
        st["cu_out"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        st["lens_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["used"] = torch.empty(1, dtype=torch.int32, device="cuda")
        return st
    Hkv, d, dt = case["Hkv"], case["d"], TYPES[case["dtype"]]
    # keys and values as views of one packed projection [total, 2, Hkv, d]
    kv = torch.randn(total, 2, Hkv, d, generator=g, device="cuda")
    kv = kv * torch.exp2(torch.randint(-2, 3, (total, 2, Hkv, 1), generator=g, device="cuda").float())
    st["kv"] = kv.to(dt)
    st["knew"], st["vnew"] = st["kv"][:, 0], st["kv"][:, 1]
    if op == "append16":
        st["table"], n = _tables(g, B, cap // page)
        # one page more than the pool, for what the plain form must not write
        st["k"] = torch.zeros(n, page, Hkv, d, dtype=dt, device="cuda")
        st["v"] = torch.zeros(n, page, Hkv, d, dtype=dt, device="cuda")
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), st["news"].long())
        pos = torch.arange(total, device="cuda") - st["cu"].long()[b] + st["olds"].long()[b]
        st["slots"] = (st["table"][b, pos // page] * page + (pos % page)).to(torch.int32)
        return st
    unit = page or 128
    per = cap // unit
    if page:
        st["table"], n = _tables(g, B, per)
        blocks = st["table"].long()
    else:
        st["table"], n = None, B * per
        blocks = torch.arange(n, device="cuda").view(B, per)
    st["blocks"] = blocks  # block of token position p of sequence b: blocks[b, p // unit]
    # one block more than the cache, where the plain form writes what belongs nowhere
    st["kfull"], st["vfull"] = _codes(g, (n + 1, unit, Hkv, d)), _codes(g, (n + 1, unit, Hkv, d))
    st["k"], st["v"] = st["kfull"][:n], st["vfull"][:n]
    st["ks"], st["vs"] = _factors(g, (n, Hkv)), _factors(g, (n, Hkv))
    if not page:
        st["k"], st["v"] = st["k"].view(B, cap, Hkv, d), st["v"].view(B, cap, Hkv, d)
        st["ks"] = st["ks"].view(B, per, Hkv).transpose(1, 2).contiguous()
        st["vs"] = st["vs"].view(B, per, Hkv).transpose(1, 2).contiguous()
    return st


# -------------------------------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    return {"decode8": _plain_decode, "append8": _plain_append8, "append16": _plain_append16,
            "tables": _plain_tables}[op](st)


def _own(st, op):
    from exact_tiled_attention_36_b200 import binding as fb
    c = st["case"]
    if op == "decode8":
        if "ws" not in st:  # the workspace a program keeps for its decode steps
            n = fb.fa_decode_fp8_workspace_size(c["B"], c["Hq"], c["Hkv"], c["Nq"], c["d"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return fb.attention_decode_fp8(st["q"], st["k"], st["v"], st["ks"], st["vs"], st["lens"],
                                       causal=c["causal"], block_table=st["table"], workspace=st["ws"],
                                       out=st["out"], lse=st["lse"])
    if op == "append8":
        fb.cache_append_fp8(st["knew"], st["vnew"], st["k"], st["v"], st["ks"], st["vs"], st["cu"], st["olds"],
                            st["lens"], st["max_new"], block_table=st["table"])
        f8 = torch.float8_e4m3fn
        return st["k"].view(f8), st["v"].view(f8), st["ks"], st["vs"]
    if op == "append16":
        fb.cache_append_paged(st["knew"], st["vnew"], st["k"], st["v"], st["slots"])
        return st["k"], st["v"]
    fb.build_block_tables(st["olds"], st["news"], st["free"], st["table"], c["page"], st["num_pages"], st["total"],
                          slot_map=st["slots"], cu_new=st["cu_out"], new_seqlens=st["lens_out"],
                          pages_used=st["used"])
    return st["table"], st["slots"], st["cu_out"], st["lens_out"], st["used"]


def _values(codes, factors):
    return codes.view(torch.float8_e4m3fn).float() * factors


def _plain_decode(st):
    c, q = st["case"], st["q"]
    B, Hq, Hkv, Nq, d, cap, page = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "cap", "page"))
    if page:
        t = st["table"].long()
        k = _values(st["k"][t], st["ks"][t][:, :, None, :, None]).reshape(B, cap, Hkv, d)
        v = _values(st["v"][t], st["vs"][t][:, :, None, :, None]).reshape(B, cap, Hkv, d)
    else:
        ks = st["ks"].transpose(1, 2).repeat_interleave(128, 1)[:, :cap, :, None]
        vs = st["vs"].transpose(1, 2).repeat_interleave(128, 1)[:, :cap, :, None]
        k, v = _values(st["k"], ks), _values(st["v"], vs)
    n = st["lens"].long() if st["lens"] is not None else torch.full((B,), cap, device=q.device)
    j = torch.arange(cap, device=q.device)
    inside = j[None, :] < n[:, None]
    v = torch.where(inside[:, :, None, None], v, torch.zeros((), device=q.device))
    # rows of a KV head: its heads' queries of every new token
    qg = q.float().view(B, Nq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, Nq, cap) * d ** -0.5
    seen = inside[:, None, :].expand(B, Nq, cap)
    if c["causal"]:
        last = torch.arange(Nq, device=q.device)[None, :] + (n - Nq)[:, None]
        seen = seen & (j[None, None, :] <= last[:, :, None])
    s = torch.where(seen[:, None, None], s, torch.full((), -math.inf, device=q.device))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul((p / torch.where(l > 0, l, torch.ones_like(l))).view(B, Hkv, -1, cap), v.permute(0, 2, 1, 3))
    o = o.view(B, Hkv, Hq // Hkv, Nq, d).permute(0, 3, 1, 2, 4).reshape(B, Nq, Hq, d)
    lse = (m + torch.log(l)).view(B, Hq, Nq)
    return o.to(q.dtype), lse


def _factor_of(amax):
    """The smallest power of two f with amax <= 448 f, at least 2^MIN_EXP."""
    frac, ex = torch.frexp(amax)  # amax = frac 2^ex, frac in [1/2, 1)
    e = torch.where(frac <= E4M3_MAX / 512, ex - 9, ex - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append8(st):
    c = st["case"]
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    unit = page or 128
    blocks, total = st["blocks"], st["total"]
    scratch = st["kfull"].shape[0] - 1
    olds, news = st["olds"].long(), st["news"].long()
    b = torch.searchsorted(st["cu"][1:].long(), torch.arange(total, device="cuda"), right=True)
    pos = torch.arange(total, device="cuda") - st["cu"].long()[b] + olds[b]
    blk = blocks[b, pos // unit]
    # the block a sequence had begun, and its rows
    per = blocks.shape[1]
    first = torch.where(news > 0, blocks.gather(1, (olds // unit).clamp(max=per - 1)[:, None])[:, 0],
                        torch.full_like(olds, scratch))
    kept = torch.arange(unit, device="cuda")[None, :, None, None] < (olds % unit)[:, None, None, None]
    for x, pool, name in ((st["knew"], st["kfull"], "ks"), (st["vnew"], st["vfull"], "vs")):
        sc = st[name] if page else st[name].transpose(1, 2).reshape(-1, Hkv)
        x = x.float()
        a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
        top = torch.zeros(scratch + 1, Hkv, device="cuda").scatter_reduce(0, blk[:, None].expand(-1, Hkv), a, "amax")
        need = _factor_of(top)
        old = torch.zeros_like(need)
        go_on = first[:, None] * torch.ones(1, Hkv, dtype=torch.long, device="cuda")
        was = torch.where((olds % unit > 0)[:, None], torch.cat([sc, sc[:1]])[first], torch.zeros_like(need[first]))
        old = old.scatter(0, go_on, was)
        new = torch.maximum(need, old)
        ratio = (was / new[first])[:, None, :, None]
        codes = pool[first].view(torch.float8_e4m3fn)
        again = (codes.float() * ratio).to(torch.float8_e4m3fn)
        pool[first] = torch.where(kept & (ratio < 1), again.view(torch.uint8), codes.view(torch.uint8))
        y = (x / new[blk][:, :, None]).to(torch.float8_e4m3fn)
        y = torch.where(torch.isfinite(x), y.view(torch.uint8), torch.full((), 0x7F, dtype=torch.uint8, device="cuda"))
        pool[blk, pos % unit] = y
        touched = torch.zeros(scratch + 1, 1, dtype=torch.bool, device="cuda")
        touched[blk] = True
        sc = torch.where(touched[:-1], new[:-1], sc)
        st[name].copy_(sc if page else sc.view(B, per, Hkv).transpose(1, 2))
    f8 = torch.float8_e4m3fn
    return st["k"].view(f8), st["v"].view(f8), st["ks"], st["vs"]


def _plain_append16(st):
    slots = st["slots"].long()
    for x, pool in ((st["knew"], st["k"]), (st["vnew"], st["v"])):
        pool.view(-1, *pool.shape[2:])[slots] = x
    return st["k"], st["v"]


def _plain_tables(st):
    c = st["case"]
    page, total, per = c["page"], st["total"], st["table"].shape[1]
    olds, news, free = st["olds"].long(), st["news"].long(), st["free"].long()
    have = (olds + page - 1) // page
    need = (olds + news + page - 1) // page - have
    upto = torch.cumsum(need, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(news, 0)])
    # column j of request b is its page of rank j - have[b] among the new ones
    rank = torch.arange(per, device="cuda")[None, :] - have[:, None]
    is_new = (rank >= 0) & (rank < need[:, None])
    at = ((upto - need)[:, None] + rank).clamp(0, free.numel() - 1)
    table = torch.where(is_new, free[at], st["table"].long())
    b = torch.searchsorted(cu[1:], torch.arange(total, device="cuda"), right=True)
    pos = torch.arange(total, device="cuda") - cu[b] + olds[b]
    slots = table[b, pos // page] * page + pos % page
    st["table"].copy_(table)
    i32 = torch.int32
    return st["table"], slots.to(i32), cu.to(i32), (olds + news).to(i32), upto[-1:].to(i32)


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"decode8": _exact_decode, "append8": _exact_append8, "append16": _exact_append16,
            "tables": _exact_tables}[case["op"]](case, st)


def _e4m3_values():
    """The 256 values of the format: sign, 4 exponent bits of bias 7, 3 mantissa bits, 0x7F NaN."""
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_decode(case, st):
    B, Hq, Hkv, Nq, d, page = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "page"))
    lut, lens, g = _e4m3_values(), _lengths(case), Hq // Hkv
    o = torch.zeros(B, Nq, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        p = torch.arange(n, device="cuda")
        if page:
            pg = st["table"][b].long()[p // page]
            kc, vc, kf, vf = st["k"][pg, p % page], st["v"][pg, p % page], st["ks"][pg], st["vs"][pg]
        else:
            kc, vc, kf, vf = st["k"][b, :n], st["v"][b, :n], st["ks"][b].T[p // 128], st["vs"][b].T[p // 128]
        for h in range(Hkv):
            k = lut[kc[:, h].long()] * kf[:, h, None].double()
            v = lut[vc[:, h].long()] * vf[:, h, None].double()
            s = torch.einsum("tgd,nd->gtn", st["q"][b, :, h * g:(h + 1) * g].double(), k) / math.sqrt(d)
            if case["causal"]:
                t = torch.arange(Nq, device="cuda")
                s = s.masked_fill(p[None, :] > (t + n - Nq)[:, None], -math.inf)
            L = torch.logsumexp(s, -1)
            w = torch.exp(s - L[:, :, None]).masked_fill(torch.isinf(L)[:, :, None], 0.0)
            o[b, :, h * g:(h + 1) * g] = torch.einsum("gtn,nd->tgd", w, v)
            lse[b, h * g:(h + 1) * g] = L
    return o, lse


def _exact_append8(case, st):
    """Block by block: the codes as the values they stand for, and the factors."""
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    unit = page or 128
    lut = _e4m3_values()
    grid = lut[:127]  # the finite non-negative values, ascending
    olds, news = _lengths(case)

    def nearest(x):
        """The nearest E4M3 value, ties to the even code."""
        a = x.abs()
        hi = torch.searchsorted(grid, a).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = a - grid[lo], grid[hi] - a
        code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        return torch.copysign(grid[code], x)

    out, facs = [], []
    for x, codes, fac in ((st["knew"], st["k"], st["ks"]), (st["vnew"], st["v"], st["vs"])):
        flat = codes.view(-1, unit, *codes.shape[-2:])
        val = torch.empty(flat.shape, dtype=torch.float64, device="cuda")
        for i in range(0, flat.shape[0], 4096):
            val[i:i + 4096] = lut[flat[i:i + 4096].long()]
        fac = fac.double().clone()
        at = 0
        for b, (o, n) in enumerate(zip(olds, news)):
            p = o
            while p < o + n:
                blk = int(st["blocks"][b, p // unit])
                m = min(unit - p % unit, o + n - p)
                r = p % unit
                y = x[at + p - o:at + p - o + m].double()
                a = y.abs().amax((0, 2))
                e = torch.ceil(torch.log2(a / E4M3_MAX).clamp(min=MIN_EXP))
                e = torch.where(a <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=MIN_EXP)
                f = torch.exp2(torch.where(a > E4M3_MAX * torch.exp2(e), e + 1, e))
                row = fac[blk] if page else fac[b, :, p // unit]
                if r:
                    f = torch.maximum(f, row)
                    scaled = nearest(val[blk, :r] * (row / f)[None, :, None])
                    val[blk, :r] = torch.where((row < f)[None, :, None], scaled, val[blk, :r])
                val[blk, r:r + m] = nearest(y / f[None, :, None])
                if page:
                    fac[blk] = f
                else:
                    fac[b, :, p // unit] = f
                p += m
            at += n
        out.append(val.view(codes.shape))
        facs.append(fac)
    return out[0], out[1], facs[0], facs[1]


def _exact_append16(case, st):
    out = []
    for x, pool in ((st["knew"], st["k"]), (st["vnew"], st["v"])):
        y = pool.double()
        y.view(-1, *pool.shape[2:]).index_copy_(0, st["slots"].long(), x.double())
        out.append(y)
    return out[0], out[1]


def _exact_tables(case, st):
    return None  # whole numbers: equal to the plain form's
