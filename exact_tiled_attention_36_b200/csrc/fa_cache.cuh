// fa_cache.cuh: what writes the key/value caches of the decode on sm_100a: block
// tables and slot maps from the requests' lengths, and the appends of new keys and
// values to 16-bit and E4M3 caches.
#pragma once

#include "fa_host.h"
#include "sm100.cuh"

namespace fa {

// ------------------------------------------------------------------ block tables
// With n_b tokens cached and c_b new ones, request b needs
//     need_b = ceil((n_b + c_b) / ps) - ceil(n_b / ps)
// pages; two exclusive prefix sums over b give the first of its pages in the free
// list and the first of its tokens in the packed order. Every CTA takes the whole
// scan itself (B integers, a few block scans), then writes its share of the new table
// entries and its slice of the slot map, finding the request of an entry or token in
// the scanned sums by bisection: one launch, no CTA waits for another, and a request's
// pages are spread over the threads however many they are (a warp per request, one
// request after the other, took 11.8 us for 256 requests). What bounds it is latency:
// one read of the lengths, the scan, one dependent page read, one write.
struct TableArgs {
    const int* seqlens;    // [B] or null (0)
    const int* new_lens;   // [B]
    const int* free_pages;  // [num_free]
    int* block_table;      // [B, max_pages]
    int* slot_map;         // [total_new]
    int* cu_new;           // [B + 1]
    int* new_seqlens;      // [B]
    int* pages_used;       // [1]
    int B, num_free, num_pages, page_size, max_pages, total_new;
    int* err;
};

constexpr int kTableThreads = 256;
constexpr int kTableRun = 4;  // consecutive tokens of a thread
constexpr int kTableSlice = kTableThreads * kTableRun;  // tokens of the slot map a CTA writes

// The last entry of the ascending sums[0 .. n) that is at most x (sums[0] <= x): of equal
// ones that is the only request with anything of its own there.
__device__ __forceinline__ int table_find(const int* sums, int n, int x) {
    int l = 0, r = n - 1;
    while (l < r) {
        const int m = (l + r + 1) >> 1;
        if (sums[m] <= x) l = m;
        else r = m - 1;
    }
    return l;
}

__global__ void __launch_bounds__(kTableThreads) fa_block_tables_kernel(const TableArgs a) {
    constexpr int kWarps = kTableThreads / 32;
    __shared__ long long w_tok[kWarps], w_page[kWarps];
    __shared__ int s_tok[kTableThreads + 1];   // first packed token of the chunk's requests
    __shared__ int s_page[kTableThreads];      // their first page in the free list
    __shared__ int s_old[kTableThreads];       // tokens cached; -1: the request gets nothing
    const int tid = static_cast<int>(threadIdx.x), lane = lane_id(), warp = warp_id();
    const int cta = static_cast<int>(blockIdx.x), G = static_cast<int>(gridDim.x);
    const uint32_t ps = static_cast<uint32_t>(a.page_size);
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;  // < 2^31
    const int t_lo = cta * kTableSlice;  // < total_new + 2^10
    const int t_hi = static_cast<int>(min(static_cast<long long>(t_lo) + kTableSlice, static_cast<long long>(a.total_new)));
    const bool aligned = (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0;
    auto pages_of = [ps](int n) { return static_cast<int>((static_cast<uint32_t>(n) + ps - 1) / ps); };
    long long tok = 0, page = 0;  // packed tokens and pages of the chunks before
    bool bad = false;
    int used = 0;  // pages of the requests this thread accepted, counted from the list's start
    for (int base = 0, chunk = 0; base < a.B; base += kTableThreads, ++chunk) {
        const int b = base + tid;
        int n = 0, c = 0;
        if (b < a.B) {
            n = a.seqlens ? a.seqlens[b] : 0;
            c = a.new_lens[b];
        }
        bool ok = n >= 0 && c >= 0 && static_cast<long long>(n) + c <= cap;
        c = max(c, 0);
        const int need = ok ? pages_of(n + c) - pages_of(n) : 0;
        long long it = c, ip = need;  // inclusive sums over the warp, then the block
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, it, off), y = __shfl_up_sync(0xffffffffu, ip, off);
            if (lane >= off) {
                it += x;
                ip += y;
            }
        }
        if (lane == 31) {
            w_tok[warp] = it;
            w_page[warp] = ip;
        }
        __syncthreads();
        long long bt = tok, bp = page, tt = 0, tp = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                bt += w_tok[w];
                bp += w_page[w];
            }
            tt += w_tok[w];
            tp += w_page[w];
        }
        const long long tok0 = bt + it - c, page0 = bp + ip - need;
        // A request is taken as a whole or not at all; where the free list or the slot
        // map ends, every later request that needs more of it is refused too.
        ok = ok && tok0 + c <= a.total_new && (need == 0 || page0 + need <= a.num_free);
        s_tok[tid] = static_cast<int>(min(tok0, static_cast<long long>(a.total_new)));
        s_page[tid] = static_cast<int>(min(page0, static_cast<long long>(a.num_free)));
        s_old[tid] = ok ? n : -1;
        tok += tt;
        page += tp;
        if (tid == 0) s_tok[kTableThreads] = static_cast<int>(min(tok, static_cast<long long>(a.total_new)));
        __syncthreads();
        if (b < a.B) {
            bad |= !ok;
            if (ok && need > 0) used = static_cast<int>(page0) + need;
            if (chunk % G == cta) {
                a.cu_new[b] = s_tok[tid];
                a.new_seqlens[b] = ok ? n + c : n;
            }
        }
        const int here = min(kTableThreads, a.B - base);
        // New table entries: entry i of the free list belongs to the request whose pages start
        // at or before it.
        const int p_end = static_cast<int>(min(page, static_cast<long long>(a.num_free)));
        for (long long i = static_cast<long long>(s_page[0]) + cta * kTableThreads + tid; i < p_end;
             i += static_cast<long long>(G) * kTableThreads) {
            const int pg = a.free_pages[i];
            const int l = table_find(s_page, here, static_cast<int>(i));
            if (s_old[l] >= 0)
                a.block_table[static_cast<size_t>(base + l) * a.max_pages + pages_of(s_old[l]) + (i - s_page[l])] = pg;
        }
        // Slots of the tokens of this CTA's slice that belong to the chunk's requests, runs
        // of consecutive tokens a thread: their request and page change seldom.
        const int lo = max(t_lo, s_tok[0]), hi = min(t_hi, s_tok[here]);
        const int t0 = t_lo + tid * kTableRun;
        if (t0 < hi && t0 + kTableRun > lo) {
            int slot[kTableRun];
            int l = table_find(s_tok, here, max(t0, lo));
            int at = -1, pg = -1;  // the page's place in the request's row, the page
#pragma unroll
            for (int k = 0; k < kTableRun; ++k) {
                const int t = t0 + k;
                slot[k] = -1;
                if (t < lo || t >= hi) continue;
                while (l + 1 < here && s_tok[l + 1] <= t) {
                    ++l;
                    at = -1;
                }
                const int old = s_old[l];
                if (old < 0) continue;
                const int pos = old + (t - s_tok[l]);
                const int j = static_cast<int>(static_cast<uint32_t>(pos) / ps);
                if (j != at) {
                    const int have = pages_of(old);
                    pg = j < have ? a.block_table[static_cast<size_t>(base + l) * a.max_pages + j]
                                  : a.free_pages[s_page[l] + (j - have)];
                    at = j;
                }
                if (pg >= 0 && pg < a.num_pages) slot[k] = pg * a.page_size + (pos - j * a.page_size);
                else bad = true;
            }
            if (aligned && t0 >= lo && t0 + kTableRun <= hi) {
                *reinterpret_cast<int4*>(a.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            } else {
#pragma unroll
                for (int k = 0; k < kTableRun; ++k)
                    if (t0 + k >= lo && t0 + k < hi) a.slot_map[t0 + k] = slot[k];
            }
        }
        if (base + kTableThreads < a.B) __syncthreads();  // the sums are written again
    }
    // Tokens of no request.
    for (long long t = max(static_cast<long long>(t_lo), min(tok, static_cast<long long>(a.total_new))) + tid; t < t_hi;
         t += kTableThreads)
        a.slot_map[t] = -1;
    if (bad) atomicCAS(a.err, 0, kErrCacheRange);
    if (cta != 0) return;
    // The accepted requests that take pages are a prefix of those that need any, so the
    // largest count is the number of pages taken.
    used = __reduce_max_sync(0xffffffffu, used);
    __syncthreads();
    if (lane == 0) w_page[warp] = used;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) used = max(used, static_cast<int>(w_page[w]));
        a.pages_used[0] = used;
        a.cu_new[a.B] = static_cast<int>(min(tok, static_cast<long long>(a.total_new)));
    }
}

// ------------------------------------------------------------------ 16-bit append
// Row t of k and v goes to row slot_map[t] of the page pools (a slot outside the pool
// is skipped: -1 marks a token of no request). A copy: one thread moves 16 bytes of a
// key row and of a value row, both loads in flight before either store.
struct Append16Args {
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* kp;
    uint16_t* vp;
    const int* slot_map;
    long long kst, ksh, vst, vsh;  // token and head strides (elements)
    long long chunks;              // 16-byte chunks of all rows: total_new * Hkv * d / 8
    int row_chunks, head_chunks;   // of one row (Hkv d / 8) and of one head (d / 8)
    int slots;                     // rows of the pool
};

__global__ void __launch_bounds__(256) fa_append16_kernel(const Append16Args a) {
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.chunks; i += step) {
        const long long t = i / a.row_chunks;
        const int c = static_cast<int>(i - t * a.row_chunks);
        const int slot = a.slot_map[t];
        if (slot < 0 || slot >= a.slots) continue;
        const int h = c / a.head_chunks, w = c % a.head_chunks;
        const uint4 x = *reinterpret_cast<const uint4*>(a.k + t * a.kst + h * a.ksh + w * 8);
        const uint4 y = *reinterpret_cast<const uint4*>(a.v + t * a.vst + h * a.vsh + w * 8);
        const size_t at = static_cast<size_t>(slot) * a.row_chunks + c;
        reinterpret_cast<uint4*>(a.kp)[at] = x;
        reinterpret_cast<uint4*>(a.vp)[at] = y;
    }
}

// ------------------------------------------------------------------ 8-bit append
// A block (128 tokens of a contiguous cache, or a page) of one KV head has one float32
// factor f; its E4M3 codes stand for code * f. For the new tokens x of a block
//     f_new = the smallest power of two with max |x| <= 448 f_new, at least 2^-100,
// and a block that held tokens before keeps f = max(f_old, f_new): when it grows, the
// rows below the first new one are rescaled, code -> e4m3(code f_old / f_new). A power
// of two costs E4M3 nothing in precision (the format floats) and makes both the
// division and the rescale of a normal code exact; only codes that fall below 2^-6 are
// rounded again. Infinities and NaN count for no factor and are stored as NaN.
//
// One group of TG threads takes one (block, KV head, key or value): it reads the new
// rows once, holding them (16 bytes a chunk, kHold chunks a thread) for the maximum and
// the codes. TG is the smallest of 32, 64, 128 and 256 whose threads hold the rows a
// block can get, so that every thread has kHold copies in flight (when that was chosen,
// 17,000 tokens of 8 heads took 31 us so, and 45 us with 256 threads for 64-row blocks, four
// loads each; now 24.7 us, 64 % of the copy rate). They go to shared memory, each thread
// reading back its own. The maximum is taken of the 16-bit patterns,
// two at a time, and the test for infinities and NaN once per group, not per value: with
// both in fp32 the kernel was bound by issuing instructions. Groups of a warp share CTAs
// of eight.
struct Append8Args {
    const uint16_t* x[2];  // k, v
    uint8_t* codes[2];
    float* factors[2];
    long long st[2], sh[2];  // token and head strides (elements)
    const int* cu_new;       // [B + 1]
    const int* seqlens;      // [B] tokens cached before
    const int* new_seqlens;  // [B] and after
    const int* block_table;  // [B, max_pages], null: contiguous
    int B, Hkv, total_new, max_new;
    int unit;                // tokens of a block
    int cap;                 // tokens a sequence can hold
    int per_seq;             // blocks of a sequence (contiguous: ceil(cap / 128); paged: max_pages)
    int num_pages;
    int touched;             // blocks of one sequence that max_new tokens can touch
    long long groups;
    int* err;
};

constexpr int kHold = 8;
constexpr int kMinFactorExp = -100;

// The exponent e of the smallest power of two with amax <= 448 * 2^e (amax finite, >= 0).
__device__ __forceinline__ int e4m3_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = m 2^x with m in [1, 2) (a subnormal counts as x = -127: both are below the
    // smallest factor); 448 = 1.75 * 2^8.
    const int x = static_cast<int>(u >> 23) - 127;
    const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
    return max(e, kMinFactorExp);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = unpack_lo<BF16>(w[i]);
        f[2 * i + 1] = unpack_hi<BF16>(w[i]);
    }
}

// The larger of two pairs of 16-bit magnitudes, with those of `u` (a pair of values);
// `finite`: infinities and NaN count as 0.
template <bool BF16>
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t m, uint32_t u, bool finite) {
    constexpr uint32_t kInf2 = BF16 ? 0x7f807f80u : 0x7c007c00u;
    u &= 0x7fff7fffu;
    if (finite) u &= __vcmpltu2(u, kInf2);
    return __vmaxu2(m, u);
}

// Four E4M3 codes times `ratio`, rounded to E4M3 again.
__device__ __forceinline__ uint32_t rescale4_e4m3(uint32_t c, float ratio) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    return pack4_e4m3(unpack_lo<false>(lo) * ratio, unpack_hi<false>(lo) * ratio, unpack_lo<false>(hi) * ratio,
                      unpack_hi<false>(hi) * ratio);
}

template <bool BF16, int D, int TG>
__global__ void __launch_bounds__(TG == 32 ? 256 : TG, TG == 32 ? 4 : 1024 / TG) fa_append8_kernel(const Append8Args a) {
    constexpr int kChunks = D / 8;            // 16-byte chunks of a row
    constexpr int kRows = TG / kChunks;       // rows a group reads at a time
    __shared__ uint32_t red[2][8];
    __shared__ uint4 held[kHold][TG == 32 ? 256 : TG];
    const int lane = lane_id(), warp = warp_id();
    const long long grp = TG == 32 ? static_cast<long long>(blockIdx.x) * 8 + warp : blockIdx.x;
    if (grp >= a.groups) return;  // uniform over the group
    const int tg = TG == 32 ? lane : static_cast<int>(threadIdx.x);
    // Heads fastest (a row's heads lie together), then key / value, block, sequence.
    const int h = static_cast<int>(grp % a.Hkv);
    const int kv = static_cast<int>((grp / a.Hkv) & 1);
    const long long bb = grp / (2 * a.Hkv);
    const int i_blk = static_cast<int>(bb % a.touched), b = static_cast<int>(bb / a.touched);
    const int old = a.seqlens[b], t0 = a.cu_new[b], t1 = a.cu_new[b + 1];
    long long count = static_cast<long long>(a.new_seqlens[b]) - old;
    const bool bad = old < 0 || count < 0 || count > a.max_new || old + count > a.cap || t0 < 0 || static_cast<long long>(t1) - t0 < count ||
                     t0 + count > a.total_new;
    if (bad) {  // lengths that do not fit the cache or the packed tokens: the sequence is left out
        if (i_blk == 0 && h == 0 && kv == 0 && tg == 0) atomicCAS(a.err, 0, kErrCacheRange);
        return;
    }
    const int blk = old / a.unit + i_blk;
    const long long p0 = max(static_cast<long long>(blk) * a.unit, static_cast<long long>(old));
    const long long p1 = min((static_cast<long long>(blk) + 1) * a.unit, old + count);
    if (p0 >= p1) return;
    const int r0 = static_cast<int>(p0 - static_cast<long long>(blk) * a.unit);  // first new row of the block
    const int rows = static_cast<int>(p1 - p0);
    // The rows are on their way before the block's place is looked up.
    const uint16_t* src = a.x[kv] + (t0 + p0 - old) * a.st[kv] + h * a.sh[kv];
    const int c = tg % kChunks, r_first = tg / kChunks;
    uint4* mine = &held[0][threadIdx.x];
    constexpr int kStride = TG == 32 ? 256 : TG;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int r = r_first + i * kRows;
        if (r < rows)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(mine + i * kStride)),
                         "l"(src + r * a.st[kv] + c * 8)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int per_row = a.Hkv * D;
    uint8_t* dst;  // row 0 of the block, this head
    float* fac;
    if (a.block_table) {
        const int pg = a.block_table[static_cast<size_t>(b) * a.per_seq + blk];
        if (pg < 0 || pg >= a.num_pages) {
            if (h == 0 && kv == 0 && tg == 0) atomicCAS(a.err, 0, kErrCacheRange);
            asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives its CTA's shared memory
            return;
        }
        dst = a.codes[kv] + static_cast<size_t>(pg) * a.unit * per_row + h * D;
        fac = a.factors[kv] + static_cast<size_t>(pg) * a.Hkv + h;
    } else {
        dst = a.codes[kv] + (static_cast<size_t>(b) * a.cap + static_cast<size_t>(blk) * a.unit) * per_row + h * D;
        fac = a.factors[kv] + (static_cast<size_t>(b) * a.Hkv + h) * a.per_seq + blk;
    }
    const float f_old = r0 > 0 ? *fac : 0.f;
    constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
    // The largest magnitude's bits over the group; with infinities or NaN among them the
    // finite ones are looked at once more, alone.
    uint32_t top = 0;
    bool odd = false;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        uint32_t m = 0;
        auto take = [&](const uint4& u) {
            m = max_magnitude2<BF16>(m, u.x, odd);
            m = max_magnitude2<BF16>(m, u.y, odd);
            m = max_magnitude2<BF16>(m, u.z, odd);
            m = max_magnitude2<BF16>(m, u.w, odd);
        };
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (r_first + i * kRows < rows) take(mine[i * kStride]);
        // Blocks of more rows than are held (pages of more than kHold * kRows): read again.
        for (int r = r_first + kHold * kRows; r < rows; r += kRows)
            take(*reinterpret_cast<const uint4*>(src + r * a.st[kv] + c * 8));
        top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        if constexpr (TG > 32) {
            if (lane == 0) red[pass][warp] = top;
            __syncthreads();  // every thread has read the old factor too
#pragma unroll
            for (int w = 0; w < TG / 32; ++w) top = max(top, red[pass][w]);
        }
        if (odd || top < kInf) break;
        odd = true;
    }
    const int e = e4m3_exponent(unpack_lo<BF16>(top));
    const float f_new = fmaxf(exp2_int(e), f_old);
    if (tg == 0) *fac = f_new;
    // The division by a factor the caller brought along need not be exact; by a power of
    // two the product with its inverse is.
    const bool pow2 = (__float_as_uint(f_new) & 0x7fffffu) == 0;
    const bool plain = pow2 && !odd;
    const float inv = 1.f / f_new;
    auto put = [&](int r, const uint4& u) {
        float f[8];
        unpack8<BF16>(u, f);
        if (plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= inv;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = !(fabsf(f[i]) < INFINITY) ? __uint_as_float(0x7fffffffu) : pow2 ? f[i] * inv : f[i] / f_new;
        }
        *reinterpret_cast<uint2*>(dst + static_cast<size_t>(r0 + r) * per_row + c * 8) =
            make_uint2(pack4_e4m3(f[0], f[1], f[2], f[3]), pack4_e4m3(f[4], f[5], f[6], f[7]));
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (r_first + i * kRows < rows) put(r_first + i * kRows, mine[i * kStride]);
    for (int r = r_first + kHold * kRows; r < rows; r += kRows)
        put(r, *reinterpret_cast<const uint4*>(src + r * a.st[kv] + c * 8));
    const float ratio = f_old / f_new;
    if (r0 > 0 && ratio < 1.f) {
        for (int i = tg; i < r0 * (D / 16); i += TG) {
            uint4* q = reinterpret_cast<uint4*>(dst + static_cast<size_t>(i / (D / 16)) * per_row + i % (D / 16) * 16);
            uint4 u = *q;
            u.x = rescale4_e4m3(u.x, ratio);
            u.y = rescale4_e4m3(u.y, ratio);
            u.z = rescale4_e4m3(u.z, ratio);
            u.w = rescale4_e4m3(u.w, ratio);
            *q = u;
        }
    }
}

}  // namespace fa
