// fa_cache.cuh: what writes the key/value caches of the decode on sm_100a: block
// tables and slot maps from the requests' lengths, and the appends of new keys and
// values to 16-bit and E4M3 caches.
#pragma once

#include "sm100.cuh"

namespace fa {

// ------------------------------------------------------------------ block tables
// With n_b tokens cached and c_b new ones, request b needs
//     need_b = ceil((n_b + c_b) / ps) - ceil(n_b / ps)
// pages; two exclusive prefix sums over b give the first of its pages in the free
// list and the first of its tokens in the packed order. Every CTA takes the whole
// scan itself (B integers, a few block scans), then writes its own slice of the slot
// map and the table rows of its own requests: one launch, no CTA waits for another.
// What bounds it is latency (one read of the lengths, the scan, one dependent page
// read, one write).
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
constexpr int kTableSlice = 1024;  // tokens of the slot map a CTA writes

// The page of rank j (0-based) of a request: one it holds already, or one of the free
// list from `first` on.
__device__ __forceinline__ int table_page(const TableArgs& a, int b, int j, int have, long long first) {
    return j < have ? a.block_table[static_cast<size_t>(b) * a.max_pages + j] : a.free_pages[first + (j - have)];
}

__global__ void __launch_bounds__(kTableThreads) fa_block_tables_kernel(const TableArgs a) {
    constexpr int kWarps = kTableThreads / 32;
    __shared__ long long w_tok[kWarps], w_page[kWarps];
    __shared__ int s_tok[kTableThreads + 1];    // first packed token of the chunk's requests
    __shared__ int s_old[kTableThreads];        // tokens cached; -1: the request gets nothing
    __shared__ long long s_first[kTableThreads];  // its first page in the free list
    const int tid = static_cast<int>(threadIdx.x), lane = lane_id(), warp = warp_id();
    const int cta = static_cast<int>(blockIdx.x);
    const long long t_lo = static_cast<long long>(cta) * kTableSlice;
    const long long t_hi = min(t_lo + kTableSlice, static_cast<long long>(a.total_new));
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    long long tok = 0, page = 0;  // packed tokens and pages of the chunks before
    int chunk = 0;
    bool bad = false;
    long long used = 0;  // pages of the requests this thread accepted, counted from the list's start
    for (int base = 0; base < a.B; base += kTableThreads, ++chunk) {
        const int b = base + tid;
        long long n = 0, c = 0;
        if (b < a.B) {
            n = a.seqlens ? a.seqlens[b] : 0;
            c = a.new_lens[b];
        }
        bool ok = n >= 0 && c >= 0 && n + c <= cap;
        c = max(c, 0LL);
        const int have = ok ? static_cast<int>((n + a.page_size - 1) / a.page_size) : 0;
        const int need = ok ? static_cast<int>((n + c + a.page_size - 1) / a.page_size) - have : 0;
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
        s_old[tid] = ok ? static_cast<int>(n) : -1;
        s_first[tid] = page0;
        if (b < a.B) {
            bad |= !ok;
            if (ok && need > 0) used = page0 + need;
            if (chunk % static_cast<int>(gridDim.x) == cta) {
                a.cu_new[b] = s_tok[tid];
                a.new_seqlens[b] = static_cast<int>(ok ? n + c : n);
            }
        }
        tok += tt;
        page += tp;
        if (tid == 0) s_tok[kTableThreads] = static_cast<int>(min(tok, static_cast<long long>(a.total_new)));
        __syncthreads();
        // Table rows of this CTA's requests: a warp for each, its lanes over the new pages.
        const int here = min(kTableThreads, a.B - base);
        if (chunk % static_cast<int>(gridDim.x) == cta) {
            for (int i = warp; i < here; i += kWarps) {
                if (s_old[i] < 0) continue;
                const int old = s_old[i];
                const int count = s_tok[i + 1] - s_tok[i];
                const int h0 = (old + a.page_size - 1) / a.page_size;
                const int h1 = static_cast<int>((static_cast<long long>(old) + count + a.page_size - 1) / a.page_size);
                for (int j = h0 + lane; j < h1; j += 32)
                    a.block_table[static_cast<size_t>(base + i) * a.max_pages + j] = a.free_pages[s_first[i] + j - h0];
            }
        }
        // Slots of the tokens of this CTA's slice that belong to the chunk's requests.
        const int lo = static_cast<int>(max(t_lo, static_cast<long long>(s_tok[0])));
        const int hi = static_cast<int>(min(t_hi, static_cast<long long>(s_tok[here])));
        for (int t = lo + tid; t < hi; t += kTableThreads) {
            int l = 0, r = here - 1;  // the last request that starts at or before t (not an empty one)
            while (l < r) {
                const int m = (l + r + 1) / 2;
                if (s_tok[m] <= t) l = m;
                else r = m - 1;
            }
            int slot = -1;
            if (s_old[l] >= 0) {
                const int old = s_old[l];
                const int pos = old + (t - s_tok[l]);
                const int have_l = (old + a.page_size - 1) / a.page_size;
                const int pg = table_page(a, base + l, pos / a.page_size, have_l, s_first[l]);
                if (pg >= 0 && pg < a.num_pages) slot = pg * a.page_size + pos % a.page_size;
                else bad = true;
            }
            a.slot_map[t] = slot;
        }
        __syncthreads();
    }
    // Tokens of no request.
    for (long long t = max(t_lo, min(tok, static_cast<long long>(a.total_new))) + tid; t < t_hi; t += kTableThreads)
        a.slot_map[t] = -1;
    // The accepted requests that take pages are a prefix of those that need any, so the
    // largest count is the number of pages taken.
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) used = max(used, __shfl_xor_sync(0xffffffffu, used, off));
    if (lane == 0) w_page[warp] = used;
    __syncthreads();
    if (cta == 0 && tid == 0) {
        for (int w = 1; w < kWarps; ++w) used = max(used, w_page[w]);
        a.pages_used[0] = static_cast<int>(used);
        a.cu_new[a.B] = static_cast<int>(min(tok, static_cast<long long>(a.total_new)));
    }
    if (bad) atomicCAS(a.err, 0, kErrCacheRange);
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
// rows once, holding them in registers (16 bytes a chunk, kHold chunks a thread) for
// the maximum and the codes. TG = 32 where a block's new rows fit a warp's registers
// (eight groups share a CTA, no block barrier), else 256.
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

// Eight values times `inv` (a power of two) as E4M3 codes; what is not finite becomes NaN.
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float inv) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = (__float_as_uint(f[i]) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : f[i] * inv;
    return make_uint2(pack4_e4m3(y[0], y[1], y[2], y[3]), pack4_e4m3(y[4], y[5], y[6], y[7]));
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
__global__ void __launch_bounds__(256) fa_append8_kernel(const Append8Args a) {
    constexpr int kChunks = D / 8;            // 16-byte chunks of a row
    constexpr int kRows = TG / kChunks;       // rows a group reads at a time
    __shared__ float red[8];
    const int lane = lane_id(), warp = warp_id();
    const long long grp = static_cast<long long>(blockIdx.x) * (256 / TG) + (TG == 32 ? warp : 0);
    if (grp >= a.groups) return;  // TG = 256: uniform over the CTA
    const int tg = TG == 32 ? lane : static_cast<int>(threadIdx.x);
    // Heads fastest (a row's heads lie together), then key / value, block, sequence.
    const int h = static_cast<int>(grp % a.Hkv);
    const int kv = static_cast<int>((grp / a.Hkv) & 1);
    const long long bb = grp / (2 * a.Hkv);
    const int i_blk = static_cast<int>(bb % a.touched), b = static_cast<int>(bb / a.touched);
    const int old = a.seqlens[b], t0 = a.cu_new[b], t1 = a.cu_new[b + 1];
    long long count = static_cast<long long>(a.new_seqlens[b]) - old;
    const bool bad = old < 0 || count < 0 || count > a.max_new || old + count > a.cap || t0 < 0 || t1 - t0 < count ||
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
    const int per_row = a.Hkv * D;
    uint8_t* dst;  // row 0 of the block, this head
    float* fac;
    if (a.block_table) {
        const int pg = a.block_table[static_cast<size_t>(b) * a.per_seq + blk];
        if (pg < 0 || pg >= a.num_pages) {
            if (h == 0 && kv == 0 && tg == 0) atomicCAS(a.err, 0, kErrCacheRange);
            return;
        }
        dst = a.codes[kv] + static_cast<size_t>(pg) * a.unit * per_row + h * D;
        fac = a.factors[kv] + static_cast<size_t>(pg) * a.Hkv + h;
    } else {
        dst = a.codes[kv] + (static_cast<size_t>(b) * a.cap + static_cast<size_t>(blk) * a.unit) * per_row + h * D;
        fac = a.factors[kv] + (static_cast<size_t>(b) * a.Hkv + h) * a.per_seq + blk;
    }
    const uint16_t* src = a.x[kv] + (t0 + p0 - old) * a.st[kv] + h * a.sh[kv];
    const int c = tg % kChunks, r_first = tg / kChunks;
    const float f_old = r0 > 0 ? *fac : 0.f;
    uint4 held[kHold];
    float amax = 0.f;
    auto take = [&](const uint4& u) {
        float f[8];
        unpack8<BF16>(u, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = fabsf(f[i]);
            amax = fmaxf(amax, x < INFINITY ? x : 0.f);
        }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int r = r_first + i * kRows;
        if (r < rows) held[i] = *reinterpret_cast<const uint4*>(src + r * a.st[kv] + c * 8);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (r_first + i * kRows < rows) take(held[i]);
    // Blocks past the registers' reach (pages of more than kHold * kRows rows): read twice.
    for (int r = r_first + kHold * kRows; r < rows; r += kRows)
        take(*reinterpret_cast<const uint4*>(src + r * a.st[kv] + c * 8));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if constexpr (TG == 256) {
        if (lane == 0) red[warp] = amax;
        __syncthreads();  // every thread has read the old factor too
#pragma unroll
        for (int w = 0; w < 8; ++w) amax = fmaxf(amax, red[w]);
    }
    const int e = e4m3_exponent(amax);
    const float f_new = fmaxf(exp2_int(e), f_old);
    if (tg == 0) *fac = f_new;
    // The division by a factor the caller brought along need not be exact; by a power of
    // two the product with its inverse is.
    const bool pow2 = (__float_as_uint(f_new) & 0x7fffffu) == 0;
    const float inv = pow2 ? 1.f / f_new : 0.f;
    auto put = [&](int r, const uint4& u) {
        float f[8];
        unpack8<BF16>(u, f);
        if (!pow2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (fabsf(f[i]) < INFINITY) f[i] = f[i] / f_new;
        }
        *reinterpret_cast<uint2*>(dst + static_cast<size_t>(r0 + r) * per_row + c * 8) = quantise8(f, pow2 ? inv : 1.f);
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (r_first + i * kRows < rows) put(r_first + i * kRows, held[i]);
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
