"""Plain references of the serving operators in Python integers and 64-bit floats (test
infrastructure only; nothing of the CUDA path)."""
import numpy as np

import oracle

E4M3 = oracle.e4m3_decode(np.arange(127, dtype=np.uint8))  # the finite values >= 0, ascending


def e4m3_encode(x):
    """Codes of the nearest E4M3 values (ties to the even code; |x| <= 448); not finite: 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.minimum(np.searchsorted(E4M3, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def factor_of(amax):
    """The smallest power of two f with amax <= 448 f, at least 2^-100."""
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_fp8(x, codes, factors, place, cu, olds, news, unit):
    """x [T, Hkv, d] into `codes` (uint8 [blocks, unit, Hkv, d]) and `factors` (float64 [blocks,
    Hkv]) in place; place[b][i] is the block that holds tokens i * unit .. of sequence b."""
    x = np.asarray(x, dtype=np.float64)
    for b in range(len(olds)):
        p = olds[b]
        while p < news[b]:
            blk, r = place[b][p // unit], p % unit
            n = min(unit - r, news[b] - p)
            y = x[cu[b] + p - olds[b]:][:n]
            for h in range(x.shape[1]):
                v = np.abs(y[:, h])
                f = factor_of(float(np.where(np.isfinite(v), v, 0.0).max()))
                if r > 0:
                    old = factors[blk, h]
                    if f > old:
                        codes[blk, :r, h] = e4m3_encode(oracle.e4m3_decode(codes[blk, :r, h]) * (old / f))
                    f = max(f, old)
                codes[blk, r:r + n, h] = e4m3_encode(y[:, h] / f)
                factors[blk, h] = f
            p += n


def tables(olds, news, free, table, page, num_pages, total):
    """(block table, slot map, cu_new, new lengths, pages used) by the definition."""
    table = [list(map(int, row)) for row in table]
    width = len(table[0])
    slots, cu, lens, used, at = [-1] * total, [0], [], 0, 0
    page_sum = 0
    for b, (n, c) in enumerate(zip(olds, news)):
        ok = n >= 0 and c >= 0 and n + c <= width * page
        c = max(c, 0)
        have, need = -(-n // page), 0
        if ok:
            need = -(-(n + c) // page) - have
        page_sum += need
        if need and page_sum > len(free):
            ok = False
        if at + c > total:
            ok = False
        if ok:
            for i in range(need):
                table[b][have + i] = int(free[page_sum - need + i])
            if need:
                used = page_sum
            for t in range(c):
                pg = table[b][(n + t) // page]
                if 0 <= pg < num_pages:
                    slots[at + t] = pg * page + (n + t) % page
        lens.append(n + c if ok else n)
        at += c
        cu.append(min(at, total))
    return table, slots, cu, lens, used


def decode_fp8(q, k, v, k_fac, v_fac, lens, scale, causal, unit, table=None):
    """O, L and sum_j p_j |v_j| (what the rounding of P is bounded by) of attention over E4M3
    caches: k, v uint8 [B, Nk, Hkv, d] with factors [B, Hkv, blocks], or pages with [pages, Hkv]
    and table [B, max_pages] (a page outside the pool holds zeros)."""
    B, Nq, Hq, d = q.shape
    Hkv = k.shape[2]
    o, w = np.zeros((B, Nq, Hq, d)), np.zeros((B, Nq, Hq, d))
    lse = np.full((B, Hq, Nq), -np.inf)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        p = np.arange(n)
        if table is not None:
            pg = np.asarray(table[b])[p // unit]
            ok = ((pg >= 0) & (pg < k.shape[0]))[:, None]
            at = np.where(ok[:, 0], pg, 0)
            kk = oracle.e4m3_decode(np.where(ok[..., None], k[at, p % unit], 0)) * np.where(ok, k_fac[at], 0)[..., None]
            vv = oracle.e4m3_decode(np.where(ok[..., None], v[at, p % unit], 0)) * np.where(ok, v_fac[at], 0)[..., None]
        else:
            kk = oracle.e4m3_decode(k[b, :n]) * k_fac[b].T[p // unit][..., None]
            vv = oracle.e4m3_decode(v[b, :n]) * v_fac[b].T[p // unit][..., None]
        ob, lb = oracle.attn_fwd(q[b:b + 1], kk[None], vv[None], scale, causal)
        wb, _ = oracle.attn_fwd(q[b:b + 1], kk[None], np.abs(vv)[None], scale, causal)
        o[b], lse[b], w[b] = ob[0], lb[0], wb[0]
    return o, lse, w
