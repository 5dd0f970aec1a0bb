// fa_decode_fp8.cuh: attention of a few query tokens per sequence over an E4M3 key/value
// cache with one float32 factor per block of tokens and KV head, on sm_100a.
//
//     s_j = scale k_f(j) (q . k8_j),   O = sum_j softmax(s)_j v_f(j) v8_j
//
// What bounds it is the cache: 2 d bytes a key and KV head, read once. The codes must
// therefore go from HBM to the tensor core as they are (expanding them to 16 bits in the
// SM would cost more shared-memory traffic than the products), while the queries and the
// weights have 8 or more significant bits that E4M3's four do not hold. Both are split
// into terms: x = t1 + t2 / 16 (+ t3 / 256) with t1 = e4m3(x), t2 = e4m3(16 (x - t1)), ...
// Rounding to four significant bits leaves a remainder of four fewer, so two terms hold a
// bf16 value and three an fp16 value exactly (within E4M3's range: x is scaled by a power
// of two so that its largest magnitude is below 448). The terms are further rows of the
// same product, so they cost no further pass over the codes.
//
// Products, with keys along the tensor core's M = 128 as in the 16-bit narrow kernel:
//     S^T = K8 Q^T      (M = 128 keys, N = rows x terms, K = d)
//     O_t^T = V8^T P^T  (M = d,        N = rows x terms, K = 128 keys)
// Unlike there, P of a tile carries its block's V factor and is taken relative to the row's
// largest such product in the TILE: with u_j = v_f(j) / v_max(tile),
//     w_j = 2^(s_j + log2 u_j - m_tile),   m_tile = max over the row's keys of s_j + log2 u_j,
// and O_t = V8^T w is a product of its own, added to the running output in registers with
//     f = 2^(m_tile - m_run) v_max(tile) / 256
// per row; the sum of weights takes w_j / u_j. E4M3 spans 2^17: with a reference that stays
// at the running maximum the small weights of a long tail behind one large key would all
// round to zero, and so would those beside a block with a large factor to which the row gives
// no weight (or that it must not see), were the factor taken into account after the maximum.
// It also frees the accumulation from rescaling in TMEM. u_j counts as at least 2^-64.
//
// Work split: an item is (sequence, KV head, chunk of RC query rows); d = 64: two adjacent
// KV heads, whose code rows form one 128-byte row (S^T of each is a product over its own 64
// bytes, O^T lanes 64 k .. hold head k). TS neighbouring items of a sequence form a group
// and are walked in step by a team of TS CTAs, one item each: a token's codes of all heads
// lie together, and 128 bytes of each 1 KB at a time, by CTAs at different places, cost
// DRAM its page hits (8192 keys x 8 heads x 32 sequences: 100 us; in step 86 us). Chunks of
// one head in a team meet in the L2. The groups' key tiles, laid end to end, are split
// evenly over the teams (stream-K) as fa_decode.cuh splits items over CTAs, with the same
// segments and merge.
//
// Two CTAs share an SM, so one's softmax overlaps the other's products and loads. Warp
// roles: warp 0 TMA producer (its lanes issue the boxes of a tile), warp 1 TMEM and the
// MMA thread, warp 2 block factors, warp 3 the queries' terms and NaN among the new tokens'
// values, then NW softmax warpgroups, each with RT / NW of the rows (thread l: key l of
// every tile, then d index l of O).
// With all 16 rows in one warpgroup the loop was bound by instruction fetch (2.2 warps
// waiting for instructions per issue) and by its own latency; two halve its length.
#pragma once

#include "fa_cache.cuh"
#include "notice_ring.h"
#include "segment_range.h"
#include "sm100.cuh"

namespace fa {

struct Decode8Args {
    const uint16_t* q;       // [B, Nq, Hq, d] 16-bit
    const float* k_scale;    // [B, Hkv, per_seq] or [num_pages, Hkv]
    const float* v_scale;
    uint16_t* o;             // [B, Nq, Hq, d] 16-bit
    float* lse;              // [B, Hq, Nq]
    float* o_part;           // [slots, RT, d] normalised partial outputs
    float* lse_part;         // [slots, RT], log2
    int2* meta;              // [items]: the teams that hold an item's first and last tile
    const int* seqlens;      // [B] or null (every sequence has cap keys)
    const int* block_table;  // [B, per_seq]; null: contiguous
    int B, Hq, Hkv, group, Nq, R;
    int cap, per_seq, num_pages;       // keys a sequence can hold, its blocks, pages of the pool
    int page_size, page_box;           // rows of a page and of one TMA box (contiguous: 128)
    int HV, nch, RC;         // items of a sequence = heads (or pairs) x chunks of RC rows
    int RT, heads;           // rows of an item's partial results, heads of an item (2: RT / 2 rows each)
    int TS, HG;              // items of a group, groups of a sequence (HV = TS HG)
    int teams;               // CTAs of the split kernel: teams x TS
    float scale_log2;
    int* err;
};

constexpr int kDec8Ctas = 2;       // per SM
// Units of a segment's fixed work (see kDecItemCost). 0, 1 and 2: ragged pages 47.6, 46.8 and 46.8
// us, speculative 85.1, 84.7 and 85.3, small heads on 16-row pages 34.9, 35.1 and 36.5.
constexpr int kDec8ItemCost = 1;

template <bool BF16, bool PAIR, int RT>
struct Dec8Cfg {
    static constexpr int NW = RT == 4 ? 1 : 2;                    // softmax warpgroups
    static constexpr int RW = RT / NW;                            // rows of one
    static constexpr int kThreads = 128 + 128 * NW;
    static constexpr int NT = BF16 ? 2 : 3;                       // terms of a query and of a weight
    static constexpr int N = (NT * RT + 15) / 16 * 16;            // rows of P
    static constexpr int RH = PAIR ? RT / 2 : RT;                 // rows of one KV head
    static constexpr int NH = (NT * RH + 15) / 16 * 16;           // rows of Q of one KV head
    static constexpr int NQ = PAIR ? 2 * NH : NH;
    static constexpr int kRowPieces = PAIR ? 8 : 16;              // 8-value pieces of a query row
    static constexpr int kQPieces = RT * kRowPieces;
    static constexpr int kTile = 128 * 128;                       // one K or V tile
    static constexpr int kUnits = 5;                              // ring of tiles: K, V, K, V, ...
    static constexpr int kQB = 2;                                 // query buffers
    static constexpr int kScSlots = 4;                            // tiles of block factors
    static constexpr int kQOff = 0;
    static constexpr int kPOff = kQOff + kQB * NQ * 128;
    static constexpr int kRingOff = kPOff + 2 * N * 128;
    static constexpr int kBarOff = kRingOff + kUnits * kTile;
    static constexpr int kNumBars = 2 * kUnits + 2 * kQB + 2 * kScSlots + 8 + 3 * NW + 2 * kNotices;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;       // 224 bytes: dec8_locate
    static constexpr int kScOff = (kMiscOff + 224 + 15) / 16 * 16;  // float [slots][kScSlot]
    static constexpr int kScSlot = 52;
    static constexpr int kQfOff = kScOff + kScSlots * kScSlot * 4;  // float [2][RT]: scale of a query row
    // A warpgroup's share of each: its RW rows.
    static constexpr int kRedOff = kQfOff + 2 * RT * 4;           // float [NW][2][4][RW]: warps' maxima
    static constexpr int kRowOff = kRedOff + 8 * RT * 4;          // float [NW][4][5][RW]: a warp's row values
    static constexpr int kSumOff = kRowOff + 20 * RT * 4;         // float [NW][4][RW]: warps' sums
    static constexpr int kLenOff = kSumOff + 4 * RT * 4;          // int [kLens]: lengths of the first sequences
    static constexpr int kLens = 256;
    static constexpr int kNanOff = kLenOff + kLens * 4;           // uint8 [3][128]: see dec8_hide_nan
    static constexpr int kSmemBytes = kNanOff + 3 * 128;
    static constexpr uint32_t kColO = 2 * NQ;                     // S^T buffers at 0 and NQ
    static constexpr uint32_t kCols = 2 * NQ + 2 * N;
    static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : (kCols <= 128 ? 128 : 256);
    static_assert(kQPieces <= 128 * NW && kQPieces % 32 == 0, "one piece a softmax thread, whole warps");
    static_assert(kCols <= 256, "two CTAs share the SM's 512 columns");
    static_assert(kNotices >= ring_values(kUnits), "a notice barrier per value tile the ring holds");
    static_assert(kRingOff % 1024 == 0 && kPOff % 1024 == 0, "swizzle atoms");
    static_assert(kSmemBytes <= 115712, "two CTAs share the SM's shared memory");
};

// ------------------------------------------------------------------- work split
// One CTA's item: group hg of sequence b, and in it the CTA's place hl of the team, which
// is item vh = hg TS + hl: chunk ch of the rows of KV head (d = 64: pair of heads) hh.
struct Dec8Item {
    int b, hg, hh, ch, len, ntk, cost;
    long long P;  // first unit of its group's cost
};

__device__ __forceinline__ int dec8_len(const Decode8Args& a, int b) {
    return a.seqlens ? min(max(a.seqlens[b], 0), a.cap) : a.cap;
}

__device__ __forceinline__ Dec8Item dec8_item(const Decode8Args& a, int b, int hg, int hl, int len, long long P) {
    Dec8Item it;
    it.b = b;
    it.hg = hg;
    const int vh = hg * a.TS + hl;
    it.hh = vh;
    it.ch = 0;
    if (a.nch > 1) {  // (a division costs as much as a small tile's softmax row)
        it.hh = vh / a.nch;
        it.ch = vh - it.hh * a.nch;
    }
    it.len = len;
    it.ntk = (len + 127) / 128;
    it.cost = it.ntk > 0 ? it.ntk + kDec8ItemCost : 0;
    it.P = P;
    return it;
}

// a b / c and a / b, in 32 bits where the operands allow it (64-bit divisions are calls).
__device__ __forceinline__ long long dec8_muldiv(int a, long long b, int c) {
    if (b < (1 << 20) && a <= 2048) return static_cast<uint32_t>(a) * static_cast<uint32_t>(b) / static_cast<uint32_t>(c);
    return a * b / c;
}
__device__ __forceinline__ int dec8_div(long long a, long long b) {
    if (a < (1LL << 31) && b < (1LL << 31)) return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return static_cast<int>(a / b);
}

struct Dec8Range {
    long long T, lo, hi;
    int team, hl;
    const int* lens;  // shared memory: the first n_lens sequences' lengths (a load from global memory
    int n_lens;       // takes a microsecond or more while the caches stream)
    Dec8Item first;
};

// This CTA's item of the group after that of `it`; past the last one P = T.
__device__ __forceinline__ Dec8Item dec8_next(const Decode8Args& a, const Dec8Range& rg, const Dec8Item& it) {
    if (it.hg + 1 < a.HG) return dec8_item(a, it.b, it.hg + 1, rg.hl, it.len, it.P + it.cost);
    if (it.b + 1 < a.B) {
        const int len = it.b + 1 < rg.n_lens ? rg.lens[it.b + 1] : dec8_len(a, it.b + 1);
        return dec8_item(a, it.b + 1, 0, rg.hl, len, it.P + it.cost);
    }
    Dec8Item e = it;
    e.P = rg.T;
    e.ntk = e.cost = 0;
    return e;
}

// Slot of a team's segment of item (hg, hl) of sequence b (the team's segments are of
// ascending groups, and its last group is at most the next team's first: team + group is
// unique).
__device__ __forceinline__ size_t dec8_slot(const Decode8Args& a, int team, int b, int hg, int hl) {
    return (static_cast<size_t>(team) + static_cast<size_t>(b) * a.HG + hg) * a.TS + hl;
}

// The key tiles [j0, j0 + n) of an item in the CTA's range (false: none).
__device__ __forceinline__ bool dec8_segment(const Dec8Range& rg, const Dec8Item& it, int& j0, int& n) {
    const long long r0 = it.P + kDec8ItemCost;
    const long long lo = max(rg.lo, r0), hi = min(rg.hi, it.P + it.cost);
    if (lo >= hi) return false;
    j0 = static_cast<int>(lo - r0);
    n = static_cast<int>(hi - lo);
    return true;
}

// The team's range of the T units and the item of the group that holds its first one;
// called by every thread (it synchronises the CTA). False, for every thread, when the team
// has none: only min(teams, T) share the units, so each of those has one at least. Uses misc + 8 .. 223.
template <int THREADS, int LENS = THREADS>
__device__ __forceinline__ bool dec8_locate(const Decode8Args& a, uint8_t* misc, int* lens, Dec8Range& rg) {
    const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = lane_id();
    rg.team = static_cast<int>(blockIdx.x) / a.TS;
    rg.hl = static_cast<int>(blockIdx.x) - rg.team * a.TS;
    constexpr int kWarps = THREADS / 32;
    auto range = [&] {
        const int n = static_cast<int>(min(static_cast<long long>(a.teams), rg.T));
        if (rg.team >= n) return false;
        rg.lo = dec8_muldiv(rg.team, rg.T, n);
        rg.hi = dec8_muldiv(rg.team + 1, rg.T, n);
        return true;
    };
    int b0;
    long long P0;
    rg.lens = lens;
    rg.n_lens = 0;
    if (a.seqlens) {
        int* found = reinterpret_cast<int*>(misc + 8);
        int* sh_b0 = reinterpret_cast<int*>(misc + 12);
        long long* sh_P0 = reinterpret_cast<long long*>(misc + 16);
        long long* ws = reinterpret_cast<long long*>(misc + 32);  // sums of the scanned sequences
        long long* wr = ws + kWarps;                              // sums of the rest
        auto units_of = [&](int b) -> long long {
            if (b >= a.B) return 0;
            const int len = dec8_len(a, b);
            if (b < LENS) lens[b] = len;
            const int ntk = (len + 127) / 128;
            return ntk > 0 ? static_cast<long long>(a.HG) * (ntk + kDec8ItemCost) : 0;
        };
        // The first THREADS sequences are scanned while the others are only summed; a CTA whose
        // range starts further on scans on from there.
        rg.n_lens = min(a.B, LENS);
        long long x = units_of(tid), rest = 0;
        for (int b = tid + THREADS; b < a.B; b += THREADS) rest += units_of(b);
        long long incl = x, run = 0;
        if (tid == 0) *found = 0;
        for (int base = 0;; base += THREADS) {
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            if (lane == 31) ws[warp] = incl;
            if (base == 0) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
                if (lane == 0) wr[warp] = rest;
            }
            __syncthreads();
            long long before = 0, total = 0, others = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const long long y = ws[w];
                if (w < warp) before += y;
                total += y;
                others += wr[w];
            }
            if (base == 0) {
                rg.T = total + others;
                if (!range()) return false;
            }
            const long long excl = run + before + incl - x;
            if (x > 0 && excl <= rg.lo && rg.lo < excl + x) {  // one thread at most
                *sh_b0 = base + tid;
                *sh_P0 = excl;
                *found = 1;
            }
            __syncthreads();
            if (*found) break;
            run += total;
            if (base + THREADS >= a.B) return false;  // cannot happen: lo < T
            x = incl = units_of(base + THREADS + tid);
        }
        b0 = *sh_b0;
        P0 = *sh_P0;
    } else {
        const int ntk = (a.cap + 127) / 128;
        const long long per_b = ntk > 0 ? static_cast<long long>(a.HG) * (ntk + kDec8ItemCost) : 0;
        rg.T = per_b * a.B;
        if (!range()) return false;
        b0 = dec8_div(rg.lo, per_b);
        P0 = b0 * per_b;
    }
    const int len = b0 < rg.n_lens ? lens[b0] : dec8_len(a, b0);
    const int cost = (len + 127) / 128 + kDec8ItemCost;
    const int hg = dec8_div(rg.lo - P0, cost);
    rg.first = dec8_item(a, b0, hg, rg.hl, len, P0 + static_cast<long long>(hg) * cost);
    return true;
}

// ------------------------------------------------------------------- primitives
// Descriptor of an unswizzled K-major operand: 8-row x 16-byte pieces of 128 contiguous
// bytes, `k` bytes apart along K and `mn` bytes apart along the rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t k, uint32_t mn) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((k >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((mn >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46);
}

// N columns of this thread's TMEM lane. The values may be used after tmem_ld_done and a
// tie (which keeps the compiler from moving their uses above it).
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t addr, uint32_t* r) {
    if constexpr (N == 2) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
    } else if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : FA_R8(r, 0)
                     : "r"(addr)
                     : "memory");
    } else {
        static_assert(N == 16, "columns of one load");
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : FA_R8(r, 0), FA_R8(r, 8)
            : "r"(addr)
            : "memory");
    }
}
__device__ __forceinline__ void tmem_ld_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void tie(uint32_t* r) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// Largest value over the warp (NaN counts only where every lane has it).
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// A pair of fp16 values as a pair of E4M3 codes (low half: low byte) and back (exact).
__device__ __forceinline__ uint32_t e4m3x2_of_h2(uint32_t h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    return c;
}
__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return h;
}
// x - t of a pair, t being x rounded to E4M3, or 16 times that: both exact.
template <bool SCALE>
__device__ __forceinline__ uint32_t h2_rest(uint32_t x, uint32_t t) {
    uint32_t d, r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(t));
    if constexpr (!SCALE) return d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(d), "r"(0x4c004c00u));
    return r;
}
// The NT terms of a pair of values (fp16), each a pair of codes; SCALE: term i times 16^i.
template <int NT, bool SCALE = true>
__device__ __forceinline__ void e4m3_terms(uint32_t x, uint32_t (&c)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        c[i] = e4m3x2_of_h2(x);
        if (i + 1 < NT) x = h2_rest<SCALE>(x, h2_of_e4m3x2(c[i]));
    }
}

// The queries' terms: piece i of a tile's RT rows is 8 values, consecutive pieces (and
// lanes) one row's. dec8_query_load reads it (zeros where the row is none of the item's),
// dec8_query_put scales the row by a power of two so that its largest magnitude is below
// 448, writes the piece's terms and the row's scale. Whole warps call them.
template <typename C, bool PAIR, int RT>
__device__ __forceinline__ uint4 dec8_query_load(const Decode8Args& a, const Dec8Item& it, int i) {
    const int r = i / C::kRowPieces, c = i % C::kRowPieces;
    const int hd = PAIR ? r / C::RH : 0, rr = PAIR ? r % C::RH : r;
    const int gr = it.ch * a.RC + rr, head = PAIR ? 2 * it.hh + hd : it.hh;
    if (rr >= a.RC || gr >= a.R || head >= a.Hkv) return make_uint4(0, 0, 0, 0);
    const size_t row = (static_cast<size_t>(it.b) * a.Nq + gr / a.group) * a.Hq + static_cast<size_t>(head) * a.group +
                       gr % a.group;
    return *reinterpret_cast<const uint4*>(a.q + (row * C::kRowPieces + c) * 8);
}
// One piece of a row that LANES neighbouring lanes hold: its NT terms to at(term), 8 bytes
// each. Returns the row's power of two.
template <bool BF16, int LANES, int NT, bool SCALE, typename At>
__device__ __forceinline__ float dec8_piece_put(const uint4& raw, At at) {
    float v[8];
    unpack8<BF16>(raw, v);
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]) < INFINITY ? fabsf(v[k]) : 0.f);
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const int e = e4m3_exponent(top);
    const float inv = exp2_int(-e);
    uint32_t t4[4][NT];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fabsf(v[k]) < INFINITY ? v[k] * inv : __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int k = 0; k < 4; ++k) e4m3_terms<NT, SCALE>(pack2<false>(v[2 * k], v[2 * k + 1]), t4[k]);
#pragma unroll
    for (int t = 0; t < NT; ++t)
        *reinterpret_cast<uint2*>(at(t)) = make_uint2(t4[0][t] | (t4[1][t] << 16), t4[2][t] | (t4[3][t] << 16));
    return exp2_int(e);
}
template <typename C, bool BF16, bool PAIR, int RT>
__device__ __forceinline__ void dec8_query_put(const Decode8Args& a, const uint4& raw, int i, uint8_t* dst, float* qf) {
    const int r = i / C::kRowPieces, c = i % C::kRowPieces;
    const int hd = PAIR ? r / C::RH : 0, rr = PAIR ? r % C::RH : r;
    const int col = hd * 64 + c * 8;  // the piece's first byte of the tile's row
    const float scale = dec8_piece_put<BF16, C::kRowPieces, C::NT, true>(raw, [&](int t) {
        const int row = hd * C::NH + t * C::RH + rr;
        return dst + row * 128 + (((col >> 4) ^ (row & 7)) << 4) + (col & 15);
    });
    if (c == 0) qf[r] = a.scale_log2 * scale;
}

// The new tokens are seen by some rows only (causal, Nq > 1), and NaN among their values must
// not reach the others as 0 x NaN. A warp of its own (within the softmax's loop the search cost
// 3 %, here 1 %; who tells whom of which tile: notice_ring.h) looks through those rows of a V tile
// in shared memory before the products read it: NaN codes become zeros, and `first` keeps, per
// byte of the tile's rows (lane: four of them), the first such key, counted from `first_part` (the
// first key not seen by all; 255: none). The rows that see that key get their NaN with the result.
__device__ __forceinline__ void dec8_hide_nan(uint8_t* tile, int key0, int first_part, int len, uint32_t& first) {
    const int lane = lane_id();
#pragma unroll 1
    for (int k = max(first_part - key0, 0); k < min(len - key0, 128); ++k) {
        uint32_t* w = reinterpret_cast<uint32_t*>(tile + k * 128 + (((lane >> 2) ^ (k & 7)) << 4) + (lane & 3) * 4);
        const uint32_t x = *w, bad = __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (bad != 0) {
            first = __vminu4(first, static_cast<uint32_t>(key0 + k - first_part) * 0x01010101u | ~bad);
            *w = x & ~bad;
        }
    }
}

// A block's V factor as a share of a reference 2^ref: its log2 (which joins the scores) and its
// inverse (which takes it out of their sum). Shares below 2^-64 (also 0, of a page outside the pool,
// whose codes are zeros) count as 2^-64, so that a sum of inverses stays in fp32's range; NaN stays.
// Exact for powers of two. (With divisions and log2f, which are code of their own, the loops waited for
// instructions: ragged pages 50.5 us against 45.7, 128 rows of a head 165 against 148.)
__device__ __forceinline__ float lg2_approx(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float dec8_share(float v, float ref) {
    const float lg = lg2_approx(v) - ref;
    return lg < -64.f ? -64.f : lg;
}

// ------------------------------------------------------------------- split kernel
template <bool BF16, bool PAIR, bool PAGED, int RT>
__global__ void __launch_bounds__(Dec8Cfg<BF16, PAIR, RT>::kThreads, kDec8Ctas)
    fa_decode8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const Decode8Args args, const int causal) {
    using C = Dec8Cfg<BF16, PAIR, RT>;
    constexpr int NT = C::NT, U = C::kUnits, QB = C::kQB, SC = C::kScSlots, RH = C::RH;
    constexpr int NW = C::NW, RW = C::RW, THREADS = C::kThreads;
    constexpr int D = PAIR ? 64 : 128;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (!smem_base_ok(smem, args.err)) return;
    const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = lane_id();
    uint8_t* misc = smem + C::kMiscOff;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc);
    int* abort_flag = reinterpret_cast<int*>(misc + 4);
    uint8_t* sQ = smem + C::kQOff;
    uint8_t* sP = smem + C::kPOff;
    uint8_t* ring = smem + C::kRingOff;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [U] tiles, unit 2 g: K of tile g, 2 g + 1: V
    uint64_t* empty = full + U;
    uint64_t* q_full = empty + U;      // [QB] a segment's queries
    uint64_t* q_empty = q_full + QB;
    uint64_t* sc_full = q_empty + QB;  // [SC] a tile's block factors
    uint64_t* sc_empty = sc_full + SC;
    uint64_t* s_full = sc_empty + SC;  // [2] S^T of tile g in buffer g & 1
    uint64_t* p_full = s_full + 2;     // [2] P of the tile written, S^T read, O_t of tile g - 2 read
    uint64_t* pv_done = p_full + 2;    // [2] O_t of the tile complete
    uint64_t* mma_done = pv_done + 2;
    uint64_t* sm_done = mma_done + 1;
    uint64_t* meet_bar = sm_done + 1;  // [NW][3]: a warpgroup's warps, per tile parity and per segment
    uint64_t* v_seen = meet_bar + 3 * NW;  // [kNotices] a tile's values looked through by dec8_hide_nan
    uint64_t* v_due = v_seen + kNotices;   // [kNotices] the load of such a tile has begun
    float* sc = reinterpret_cast<float*>(smem + C::kScOff);
    float* qf = reinterpret_cast<float*>(smem + C::kQfOff);
    const bool part_seen = causal && args.Nq > 1;  // not every row sees the new tokens

    // Rows of P past the terms are zeros (those of Q are never looked at: their columns
    // of S^T are not read, but they must hold codes that are there).
    for (int i = tid; i < (C::kRingOff - C::kQOff) / 16; i += THREADS)
        reinterpret_cast<uint4*>(smem + C::kQOff)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (tid == 0) {
        for (int i = 0; i < U; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < QB; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1 + 4 * NW);  // the last S^T product, and each softmax warp's last use of the scales
        }
        for (int i = 0; i < SC; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], 4 * NW);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128 * NW);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 3 * NW; ++i) mbar_init(&meet_bar[i], 4);
        for (int i = 0; i < kNotices; ++i) {
            mbar_init(&v_seen[i], 1);
            mbar_init(&v_due[i], 1);
        }
        mbar_init(mma_done, 1);
        mbar_init(sm_done, 128 * NW);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // Launched as a programmatic dependent of whatever ran before on the stream: what
    // follows reads that kernel's results (and overwrites the workspace).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The merge may be scheduled now; it waits for this grid in turn.
    asm volatile("griddepcontrol.launch_dependents;");
    // TMEM first: the SM starts its second CTA only after the first gave up the permit to
    // allocate (measured: 0.35 us after it, wherever in the kernel that is).
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::kTmemCols);
        tmem_relinquish();
    }
    Dec8Range rg;
    const bool work = dec8_locate<THREADS, C::kLens>(args, misc, reinterpret_cast<int*>(smem + C::kLenOff), rg);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!work) {
        if (warp == 1) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(tmem_holder), C::kTmemCols);
        return;
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    const WaitCtx wc{abort_flag, args.err};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // Lane x issues box x of every tile: rows x * page_box .. of the 128 keys, from the
        // page that holds them (a page outside the pool: zeros). Boxes past the sequence's
        // end are not loaded.
        const int pb = args.page_box;
        int u = 0, n_due = 0;
        bool ok = true;
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            if (lane == 0) {
                int2* m = args.meta + (static_cast<size_t>(it.b) * args.HG + it.hg) * args.TS + rg.hl;
                if (j0 == 0) m->x = rg.team;
                if (j0 + n == it.ntk) m->y = rg.team;
            }
            const int x0 = it.hh * 128;  // the head's (or pair's) first byte of a row
            const int* bt = PAGED ? args.block_table + static_cast<size_t>(it.b) * args.per_seq : nullptr;
            auto page_of = [&](int kt) {
                const int key = kt * 128 + lane * pb;
                return PAGED && lane * pb < 128 && key < it.len ? bt[key / args.page_size] : 0;
            };
            int page = page_of(j0);
            const int kt_part = part_seen ? max(it.len - args.Nq + 1, 0) / 128 : it.ntk;  // first tile of v_due
            for (int j = 0; ok && j < n; ++j) {
                const int kt = j0 + j;
                const int boxes = PAGED ? (min(128, it.len - kt * 128) + pb - 1) / pb : 1;
                const int next = j + 1 < n ? page_of(kt + 1) : 0;  // in flight while this tile's buffers come free
                for (int kv = 0; kv < 2; ++kv, ++u) {
                    const int st = u % U;
                    if (!(ok = warp_all(mbar_wait(&empty[st], ((u / U) & 1) ^ 1u, wc, 120)))) break;
                    uint8_t* dst = ring + st * C::kTile;
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(PAGED ? boxes * pb * 128 : C::kTile));
                    if (kv && kt >= kt_part) {
                        if (lane == 0) mbar_arrive(&v_due[notice_bar(n_due)]);
                        ++n_due;
                    }
                    __syncwarp();
                    const CUtensorMap* m = kv ? &tm_v : &tm_k;
                    if (PAGED) {
                        if (lane < boxes)
                            tma_load_4d(dst + lane * pb * 128, m, &full[st], x0, (kt * 128 + lane * pb) % args.page_size, page, 0);
                    } else if (lane == 0) {
                        tma_load_4d(dst, m, &full[st], x0, kt * 128, it.b, 0);
                    }
                }
                page = next;
            }
        }
        // Leave no load in flight: wait for the last one issued into every buffer.
        for (int st = 0; st < U && st < u; ++st) mbar_wait_drain(&full[st], ((u - 1 - st) / U) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_e4m3(128, C::NH, false, false);
            constexpr uint32_t id_pv = idesc_e4m3(128, C::N, true, false);
            uint32_t q_addr = smem_u32(sQ);
            auto issue_s = [&](int gg) {
                const uint32_t k_addr = smem_u32(ring + ((2 * gg) % U) * C::kTile);
                const uint32_t d_col = tmem + static_cast<uint32_t>((gg & 1) * C::NQ);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int hd = PAIR ? kk >> 1 : 0;  // d = 64: head hd's 64 bytes are two steps
                    mma_ss_f8(d_col + hd * C::NH, sdesc_sw128(k_addr + kk * 32, 16, 1024),
                              sdesc_sw128(q_addr + hd * C::NH * 128 + kk * 32, 16, 1024), id_s,
                              (PAIR ? kk & 1 : kk) > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[gg & 1]);
                tc_commit(&empty[(2 * gg) % U]);
            };
            int gk = 0, nq = 0, n_seen = 0;
            bool ok = true;
            for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
                int j0, n;
                if (!dec8_segment(rg, it, j0, n)) continue;
                const int j_part = part_seen ? max(it.len - args.Nq + 1, 0) / 128 - j0 : n;  // first tile of v_seen
                const int qb = nq % QB;
                q_addr = smem_u32(sQ + qb * C::NQ * 128);
                if (!(ok = mbar_wait(&q_full[qb], (nq / QB) & 1, wc, 121))) break;
                for (int j = 0; ok && j < min(n, 2); ++j) {
                    const int gg = gk + j;
                    if (!(ok = mbar_wait(&full[(2 * gg) % U], ((2 * gg) / U) & 1, wc, 122))) break;
                    tc_fence_after();
                    issue_s(gg);
                }
                if (!ok) break;
                if (n <= 2) tc_commit(&q_empty[qb]);
                for (int j = 0; ok && j < n; ++j) {
                    const int gg = gk + j, b = gg & 1, uv = 2 * gg + 1;
                    if (!(ok = mbar_wait(&full[uv % U], (uv / U) & 1, wc, 123))) break;
                    if (j >= j_part) {
                        if (!(ok = mbar_wait(&v_seen[notice_bar(n_seen)], notice_parity(n_seen), wc, 135))) break;
                        ++n_seen;
                    }
                    if (!(ok = mbar_wait(&p_full[b], (gg >> 1) & 1, wc, 124))) break;
                    tc_fence_after();
                    const uint32_t v_addr = smem_u32(ring + (uv % U) * C::kTile);
                    const uint32_t p_addr = smem_u32(sP + b * C::N * 128);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss_f8(tmem + C::kColO + static_cast<uint32_t>(b * C::N), sdesc_sw128(v_addr + kk * 4096, C::kTile, 1024),
                                  sdesc_plain(p_addr + kk * 256, 128, 1024), id_pv, kk > 0 ? 1u : 0u);
                    tc_commit(&pv_done[b]);
                    tc_commit(&empty[uv % U]);
                    if (j + 2 < n) {  // S^T of tile gg + 2 into the buffer that p_full says was read
                        const int u2 = 2 * (gg + 2);
                        if (!(ok = mbar_wait(&full[u2 % U], (u2 / U) & 1, wc, 125))) break;
                        tc_fence_after();
                        issue_s(gg + 2);
                        if (j + 3 == n) tc_commit(&q_empty[qb]);
                    }
                }
                gk += n;
                ++nq;
            }
            tc_commit(mma_done);
            mbar_wait_drain(mma_done, 0);
            const uint32_t a = smem_u32(sm_done);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < 4000000000ull) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    } else if (warp == 2) {
        // ------------------------------------------------------------ block factors
        // Lane x + 8 kv + 16 h: box x of a tile, key or value factor, head h of the pair. A
        // slot holds, [h][box], 16 key factors, log2 of 16 value shares u = v / v_max and 16 inverses
        // 1 / (256 u), and v_max / 256 [h].
        const int x = lane & 7, kv = (lane >> 3) & 1, h = lane >> 4;
        const int pb = args.page_box;
        int gk = 0;
        bool ok = true;
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            const int head = PAIR ? 2 * it.hh + h : it.hh;
            const bool mine = (PAIR || h == 0) && head < args.Hkv;
            const float* f = kv ? args.v_scale : args.k_scale;
            auto read = [&](int kt) -> float {
                const int key = kt * 128 + x * pb;
                if (!mine || x * pb >= 128 || key >= it.len) return 0.f;
                if constexpr (PAGED) {
                    const int pg = args.block_table[static_cast<size_t>(it.b) * args.per_seq + key / args.page_size];
                    return pg >= 0 && pg < args.num_pages ? f[static_cast<size_t>(pg) * args.Hkv + head] : 0.f;
                } else {
                    return f[(static_cast<size_t>(it.b) * args.Hkv + head) * args.per_seq + kt];
                }
            };
            float v = read(j0);
            for (int j = 0; j < n; ++j) {
                const int gg = gk + j, slot = gg % SC;
                const float next = j + 1 < n ? read(j0 + j + 1) : 0.f;
                float top = v;
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                if (!(ok = warp_all(mbar_wait(&sc_empty[slot], ((gg / SC) & 1) ^ 1u, wc, 126)))) break;
                float* s = sc + slot * C::kScSlot;
                const float lg = dec8_share(v, top > 0.f ? lg2_approx(top) : 0.f);
                s[kv * 16 + h * 8 + x] = kv ? lg : v;
                if (kv) s[32 + h * 8 + x] = ex2_approx(-8.f - lg);
                if (kv && x == 0) s[48 + h] = top * (1.f / 256.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[slot]);
                v = next;
            }
            gk += n;
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ query terms, NaN of new tokens
        // The next segment's queries first, then NaN in the segment before: its last tiles may still
        // be on their way, and the next products would wait for their queries meanwhile.
        int gk = 0, n_told = 0;
        int p_len = 0, p_j0 = 0, p_n = 0;  // the segment before
        bool ok = true, more = true;
        Dec8Item it = rg.first;
        for (int nq = 0; ok && more; ++nq) {
            int j0 = 0, n = 0;
            while (it.P < rg.hi && !dec8_segment(rg, it, j0, n)) it = dec8_next(args, rg, it);
            more = it.P < rg.hi;
            if (more && nq > 0) {  // the first segment's: the softmax warps
                const int qb = nq % QB;
                uint4 raw = dec8_query_load<C, PAIR, RT>(args, it, lane);
                if (!(ok = warp_all(mbar_wait(&q_empty[qb], ((nq / QB) & 1) ^ 1u, wc, 127)))) break;
#pragma unroll 1
                for (int i = lane; i < C::kQPieces; i += 32) {
                    const uint4 next = i + 32 < C::kQPieces ? dec8_query_load<C, PAIR, RT>(args, it, i + 32) : raw;
                    dec8_query_put<C, BF16, PAIR, RT>(args, raw, i, sQ + qb * C::NQ * 128, qf + (nq & 1) * RT);
                    raw = next;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[qb]);
            }
            const int first_part = p_len - args.Nq + 1;
            if (nq > 0 && part_seen && (p_j0 + p_n) * 128 > first_part) {
                // Segment nq - 4, the last to use this part of the notes, has been read: the queries'
                // buffer of segment nq - 3 came free after it.
                uint32_t* noted = reinterpret_cast<uint32_t*>(smem + C::kNanOff + (nq - 1) % 3 * 128) + lane;
                uint32_t first = 0xffffffffu;
                for (int j = max(first_part / 128 - p_j0, 0); j < p_n; ++j) {
                    const int key0 = (p_j0 + j) * 128, uv = 2 * (gk + j) + 1;
                    if (!(ok = warp_all(mbar_wait(&v_due[notice_bar(n_told)], notice_parity(n_told), wc, 137)))) break;
                    if (!(ok = warp_all(mbar_wait(&full[uv % U], (uv / U) & 1, wc, 136)))) break;
                    dec8_hide_nan(ring + (uv % U) * C::kTile, key0, first_part, p_len, first);
                    *noted = first;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_seen[notice_bar(n_told)]);
                    ++n_told;
                }
            }
            gk += p_n;
            p_len = it.len;
            p_j0 = j0;
            p_n = n;
            if (more) it = dec8_next(args, rg, it);
        }
    } else {
        // ------------------------------------------------------------ softmax, output
        const int wg = (warp - 4) >> 2, w4 = warp & 3;  // warp % 4 is the TMEM lane quarter it reaches
        constexpr bool kMixed = PAIR && RW > RH;         // one warpgroup holds both heads' rows
        const int first = wg * RW;                       // its first row of the tile
        const int wg_hd = PAIR && !kMixed ? first / RH : 0;
        const int l_idx = w4 * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
        float* red = reinterpret_cast<float*>(smem + C::kRedOff) + wg * 8 * RW;  // [2][4][RW]
        float* row_m = reinterpret_cast<float*>(smem + C::kRowOff) + (wg * 4 + w4) * 5 * RW;  // this warp's row values
        float* row_f = row_m + RW;      // [2]: 2^(m_tile - m_run), times the tile's V factor from the second use on
        float* row_a = row_f + 2 * RW;  // 2^(m_run before - m_run)
        int* row_hi = reinterpret_cast<int*>(row_a + RW);  // keys a row sees
        uint64_t* meets = meet_bar + 3 * wg;
        const int box = l_idx / args.page_box;
        // Row `lane` of the warpgroup: its head of the pair, its place among that head's rows.
        const int my_r = first + (lane < RW ? lane : 0);
        const int my_hd = PAIR ? my_r / RH : 0, my_rr = PAIR ? my_r % RH : my_r;
        float* sums = reinterpret_cast<float*>(smem + C::kSumOff) + wg * 4 * RW;  // [4][RW], once per segment
        Dec8Item first_item = rg.first;  // the one of the CTA's first segment
        {
            int j0, n;
            while (first_item.P < rg.hi && !dec8_segment(rg, first_item, j0, n))
                first_item = dec8_next(args, rg, first_item);
        }
        int gk = 0, nq = 0;
        bool ok = true;
        auto meet = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            return warp_all(mbar_wait(bar, parity, wc, site));
        };
        // The first segment's queries, a piece a thread (one warp taking them piece after piece
        // would keep the first product waiting).
        {
            const int i = wg * 128 + l_idx;
            if (i < C::kQPieces)
                dec8_query_put<C, BF16, PAIR, RT>(args, dec8_query_load<C, PAIR, RT>(args, first_item, i), i, sQ, qf);
            fence_proxy_async_smem();
            named_bar_sync(1, 128 * NW);
            if (wg == 0 && l_idx == 0) mbar_arrive(&q_full[0]);
        }
        auto rows4 = [](const float* p, int r) { return *reinterpret_cast<const float4*>(p + r); };
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            const int my_gr = it.ch * args.RC + my_rr;  // this lane's row in its head's group
            __syncwarp();
            if (lane < RW) {
                const int t = causal && args.Nq > 1 ? my_gr / args.group : 0;
                row_hi[lane] = causal ? min(it.len, t + it.len - args.Nq + 1) : it.len;
            }
            __syncwarp();
            const int all_hi = causal ? it.len - args.Nq + 1 : it.len;  // keys below it are seen by every row
            ok = warp_all(mbar_wait(&q_full[nq % QB], (nq / QB) & 1, wc, 128));
            if (!ok) break;
            const float* my_qf = qf + (nq & 1) * RT + first;
            float acc[RW], l[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) acc[r] = l[r] = 0.f;
            float m_run = -INFINITY;  // of row `lane`
            // acc += f O_t of tile gg, whose factors sit in row_f of its parity.
            auto drain = [&](int gg) -> bool {
                const int b = gg & 1;
                if (!warp_all(mbar_wait(&pv_done[b], (gg >> 1) & 1, wc, 129))) return false;
                tc_fence_after();
                uint32_t o[NT][RW];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    tmem_ldn<RW>(lane_base + C::kColO + static_cast<uint32_t>(b * C::N + t * RT + first), o[t]);
                tmem_ld_done();
#pragma unroll
                for (int t = 0; t < NT; ++t) tie<RW>(o[t]);
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 f4 = rows4(row_f + b * RW, r);
                    const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = __uint_as_float(o[NT - 1][r + i]);
#pragma unroll
                        for (int t = NT - 2; t >= 0; --t) v = fmaf(v, 0.0625f, __uint_as_float(o[t][r + i]));
                        acc[r + i] = fmaf(v, f[i], acc[r + i]);
                    }
                }
                return true;
            };
            for (int j = 0; j < n; ++j) {
                const int gg = gk + j, par = gg & 1, slot = gg % SC;
                ok = warp_all(mbar_wait(&sc_full[slot], (gg / SC) & 1, wc, 130));
                if (!ok) break;
                const float* s_sc = sc + slot * C::kScSlot;
                const float kf0 = s_sc[8 * wg_hd + box], kf1 = kMixed ? s_sc[8 + box] : 0.f;
                const float vl0 = s_sc[16 + 8 * wg_hd + box], vl1 = kMixed ? s_sc[24 + box] : 0.f;
                const float vi0 = s_sc[32 + 8 * wg_hd + box], vi1 = kMixed ? s_sc[40 + box] : 0.f;
                const float my_vm = s_sc[48 + my_hd];
                ok = warp_all(mbar_wait(&s_full[par], (gg >> 1) & 1, wc, 131));
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_empty[slot]);
                tc_fence_after();
                float x[RW];
                {
                    uint32_t s[NT][RW];
                    const uint32_t s_addr = lane_base + static_cast<uint32_t>(
                        par * C::NQ + (PAIR ? first / RH * C::NH + first % RH : first));
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        tmem_ldn<kMixed ? RH : RW>(s_addr + t * RH, s[t]);
                        if constexpr (kMixed) tmem_ldn<RH>(s_addr + C::NH + t * RH, s[t] + RH);
                    }
                    tmem_ld_done();
#pragma unroll
                    for (int t = 0; t < NT; ++t) tie<RW>(s[t]);
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 f4 = rows4(my_qf, r);
                        const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {  // (packed pairs further on cost registers: slower)
                            auto two = [&](int t) {
                                return f2_pack(__uint_as_float(s[t][r + i]), __uint_as_float(s[t][r + i + 1]));
                            };
                            const float kf = kMixed && r + i >= RH ? kf1 : kf0, vl = kMixed && r + i >= RH ? vl1 : vl0;
                            uint64_t v = two(NT - 1);
#pragma unroll
                            for (int t = NT - 2; t >= 0; --t) v = f2_fma(v, f2_pack(0.0625f, 0.0625f), two(t));
                            f2_unpack(f2_fma(f2_mul(v, f2_pack(f[i], f[i + 1])), f2_pack(kf, kf), f2_pack(vl, vl)), x[r + i], x[r + i + 1]);
                        }
                    }
                }
                if (j == n - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_empty[nq % QB]);
                }
                const int key = (j0 + j) * 128 + l_idx;
                if ((j0 + j + 1) * 128 > all_hi) {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (key >= row_hi[r]) x[r] = -INFINITY;
                }
                // Every row's largest product of weight and V factor in the tile (log2): over the warp,
                // then the four warps.
                float* rd = red + par * 4 * RW;
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 v = make_float4(warp_max(x[r]), warp_max(x[r + 1]), warp_max(x[r + 2]), warp_max(x[r + 3]));
                    if (lane == 0) *reinterpret_cast<float4*>(rd + w4 * RW + r) = v;
                }
                ok = meet(&meets[par], (gg >> 1) & 1, 132);
                if (!ok) break;
                // Lane r takes row r's running values.
                bool moved = false;
                if (lane < RW) {
                    const float mt = fmaxf(fmaxf(rd[lane], rd[RW + lane]), fmaxf(rd[2 * RW + lane], rd[3 * RW + lane]));
                    float alpha = 1.f;
                    if (mt > m_run + kRescaleThreshold) {
                        alpha = ex2_approx(m_run - mt);  // 0 for the first keys
                        m_run = mt;
                        moved = true;
                    }
                    const bool none = mt == -INFINITY;
                    const float f = none ? 0.f : ex2_approx(mt - m_run);
                    row_m[lane] = none ? 0.f : 8.f - mt;
                    row_f[par * RW + lane] = f;
                    row_a[lane] = alpha;
                }
                moved = __any_sync(0xffffffffu, moved);
                __syncwarp();
                // w = 256 2^(x - m_tile), the weights' sum in the running scale, and the terms of w.
                // Row n, key l in the unswizzled layout: rows at constant offsets from the key's place
                // (the 128-byte swizzle would cost an address of its own for every row).
                uint8_t* pb = sP + par * C::N * 128 + (first >> 3) * 1024 + (first & 7) * 16 + (l_idx >> 4) * 128 + (l_idx & 15);
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 m4 = rows4(row_m, r), f4 = rows4(row_f + par * RW, r);
                    const float mm[4] = {m4.x, m4.y, m4.z, m4.w}, ff[4] = {f4.x, f4.y, f4.z, f4.w};
                    if (moved) {
                        const float4 a4 = rows4(row_a, r);
                        l[r] *= a4.x;
                        l[r + 1] *= a4.y;
                        l[r + 2] *= a4.z;
                        l[r + 3] *= a4.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float p0 = ex2_approx(x[r + i] + mm[i]), p1 = ex2_approx(x[r + i + 1] + mm[i + 1]);
                        const float vi = kMixed && r + i >= RH ? vi1 : vi0;  // (pairs of rows are of one head)
                        l[r + i] = fmaf(p0 * vi, ff[i], l[r + i]);
                        l[r + i + 1] = fmaf(p1 * vi, ff[i + 1], l[r + i + 1]);
                        uint32_t c[NT];
                        e4m3_terms<NT>(pack2<false>(p0, p1), c);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const int n0 = t * RT + r + i, n1 = n0 + 1;  // past the warpgroup's first row
                            pb[(n0 >> 3) * 1024 + (n0 & 7) * 16] = static_cast<uint8_t>(c[t]);
                            pb[(n1 >> 3) * 1024 + (n1 & 7) * 16] = static_cast<uint8_t>(c[t] >> 8);
                        }
                    }
                }
                // The sequence's last tile: rows of V past its end may hold anything (0 x NaN
                // would reach O); they are zeroed before the product reads them.
                if (j0 + j == it.ntk - 1 && (it.len & 127) != 0) {
                    const int uv = 2 * gg + 1;
                    ok = warp_all(mbar_wait(&full[uv % U], (uv / U) & 1, wc, 133));
                    if (!ok) break;
                    const int v0 = it.len & 127;
                    uint4* vt = reinterpret_cast<uint4*>(ring + (uv % U) * C::kTile + v0 * 128);
                    for (int i = wg * 128 + l_idx; i < (128 - v0) * 8; i += 128 * NW) vt[i] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[par]);
                // While this tile's product runs: the previous one's output.
                if (j > 0 && !(ok = drain(gg - 1))) break;
                if (moved) {
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 a4 = rows4(row_a, r);
                        acc[r] *= a4.x;
                        acc[r + 1] *= a4.y;
                        acc[r + 2] *= a4.z;
                        acc[r + 3] *= a4.w;
                    }
                }
                // The factor of O_t carries the tile's V factor too.
                __syncwarp();
                if (lane < RW) row_f[par * RW + lane] *= my_vm;
                __syncwarp();
            }
            if (!ok) break;
            ok = drain(gk + n - 1);
            if (!ok) break;
            // Row sums over the 128 keys' threads (written again a segment later, after
            // every warp has met at a tile in between). Each step of the sum over the warp
            // halves the rows a lane keeps; lane RW-group g ends with row g.
#pragma unroll
            for (int off = 16, m = RW; off > 0; off >>= 1) {
                if (m > 1) {
                    m >>= 1;
                    const bool up = (lane & off) != 0;
#pragma unroll
                    for (int r = 0; r < m; ++r) {
                        const float keep = up ? l[r + m] : l[r], give = up ? l[r] : l[r + m];
                        l[r] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                } else {
                    l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
                }
            }
            if (lane % (32 / RW) == 0) sums[w4 * RW + lane / (32 / RW)] = l[0];
            ok = meet(&meets[2], nq & 1, 134);
            if (!ok) break;
            if (part_seen && (j0 + n) * 128 > all_hi) {
                const int noted = smem[C::kNanOff + nq % 3 * 128 + l_idx];
#pragma unroll
                for (int r = 0; r < RW; ++r)
                    if (row_hi[r] > all_hi + noted) acc[r] = __uint_as_float(0x7fffffffu);
            }
            const size_t slot = dec8_slot(args, rg.team, it.b, it.hg, rg.hl);
            const int rows = min(args.RC, args.R - it.ch * args.RC);  // of each head
            auto valid = [&](int rt) {
                return (PAIR ? rt % RH : rt) < rows && (PAIR ? 2 * it.hh + rt / RH : it.hh) < args.Hkv;
            };
            if (lane < RW) {
                const float lt = sums[lane] + sums[RW + lane] + sums[2 * RW + lane] + sums[3 * RW + lane];
                row_a[lane] = lt == 0.f ? 0.f : __fdividef(1.f, lt);  // no key: 0; NaN stays NaN
                float lg;
                asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(lt));
                if (w4 == 0 && valid(my_r)) args.lse_part[slot * RT + my_r] = lt == 0.f ? -INFINITY : m_run + lg;
            }
            __syncwarp();
            float* op = args.o_part + (slot * RT + first) * D + (PAIR ? l_idx & 63 : l_idx);
#pragma unroll
            for (int r = 0; r < RW; r += 4) {
                const float4 f4 = rows4(row_a, r);
                const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (valid(first + r + i) && (!PAIR || (l_idx >> 6) == (first + r + i) / RH))
                        op[(r + i) * D] = acc[r + i] * f[i];
            }
            gk += n;
            ++nq;
        }
        tc_fence_before();
        mbar_arrive(sm_done);
    }
}

// Merge of the segments of each output row of [B, Nq, Hq]. WIDE: one block of eight warps
// per row (warp w takes every eighth segment), for items split over many teams; else one
// warp per row. A lane holds four values.
constexpr int kDec8WideWarps = 8;
template <int D, bool BF16, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 32 * kDec8WideWarps : 128) fa_decode8_combine(const Decode8Args a, const int rows) {
    constexpr int W = WIDE ? kDec8WideWarps : 1;
    __shared__ float4 part[W][D / 4];
    const int lane = lane_id(), warp = WIDE ? warp_id() : 0;
    const int row = WIDE ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * 4 + warp_id();
    if (row >= rows) return;
    const int h = row % a.Hq, bt = row / a.Hq;
    const int t = bt % a.Nq, b = bt / a.Nq;
    const int hk = h / a.group, gr = t * a.group + h % a.group;
    const int vh = hk / a.heads * a.nch + gr / a.RC;
    const int r = hk % a.heads * (a.RT / 2) + gr % a.RC;
    const size_t item = static_cast<size_t>(b) * a.HV + vh;
    // Launched as a programmatic dependent of the split kernel: what that wrote may be read
    // from here on.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int2 cc = a.meta[item];
    const SegmentRange seg = segment_range(cc.x, cc.y, dec8_len(a, b), a.teams);
    const int c0 = seg.first, c1 = seg.last;
    // The segment of team c lies c TS RT rows further.
    const size_t s0 = dec8_slot(a, 0, b, vh / a.TS, vh % a.TS) * a.RT + r, step = static_cast<size_t>(a.TS) * a.RT;
    const float* lp = a.lse_part + s0;
    const float4* op = reinterpret_cast<const float4*>(a.o_part + s0 * D) + lane;
    float Lm = -INFINITY, wsum = 0.f;
    bool nan = false;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4& x) {
        acc.x = fmaf(w, x.x, acc.x);
        acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z);
        acc.w = fmaf(w, x.w, acc.w);
    };
    constexpr int kFew = WIDE ? 6 : 4;
    const bool mine = lane < D / 4;
    if (!WIDE && c1 - c0 < kFew) {
        // Every load in flight at once, every lane with all the weights.
        float L[kFew];
        float4 x[kFew];
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            L[i] = c0 + i <= c1 ? lp[(c0 + i) * step] : -INFINITY;
            x[i] = c0 + i <= c1 && mine ? op[(c0 + i) * step * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            Lm = fmaxf(Lm, L[i]);
            nan |= L[i] != L[i];
        }
        const float ref = Lm == -INFINITY ? 0.f : Lm;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            const float w = ex2_approx(L[i] - ref);
            wsum += w;
            add(w, x[i]);
        }
    } else {
        float4 x[kFew];  // of the warp's first segments, on their way before the weights are known
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            const int c = c0 + warp + i * W;
            x[i] = c <= c1 && mine ? op[c * step * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int c = c0 + lane; c <= c1; c += 32) {
            const float L = lp[c * step];
            Lm = fmaxf(Lm, L);
            nan |= L != L;
        }
        Lm = warp_max(Lm);
        nan = __any_sync(0xffffffffu, nan);
        const float ref = Lm == -INFINITY ? 0.f : Lm;
        for (int c = c0 + lane; c <= c1; c += 32) wsum += ex2_approx(lp[c * step] - ref);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            const int c = c0 + warp + i * W;
            if (c <= c1) add(ex2_approx(lp[c * step] - ref), x[i]);
        }
        if (mine)
            for (int c = c0 + warp + kFew * W; c <= c1; c += W) add(ex2_approx(lp[c * step] - ref), op[c * step * (D / 4)]);
        if (WIDE && mine) part[warp][lane] = acc;
    }
    if constexpr (WIDE) {
        __syncthreads();
        if (warp != 0) return;
        if (lane < D / 4) {
#pragma unroll
            for (int w = 1; w < W; ++w) {
                const float4 y = part[w][lane];
                acc.x += y.x;
                acc.y += y.y;
                acc.z += y.z;
                acc.w += y.w;
            }
        }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    if (mine)
        *reinterpret_cast<uint2*>(a.o + static_cast<size_t>(row) * D + lane * 4) =
            make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
    if (lane == 0)
        a.lse[(static_cast<size_t>(b) * a.Hq + h) * a.Nq + t] =
            nan ? __uint_as_float(0x7fffffffu) : (wsum == 0.f ? -INFINITY : (Lm + log2f(wsum)) * kLn2);
}

}  // namespace fa
