// fa_decode_fp8_rows.cuh: the decode over an E4M3 cache for many query rows per KV head
// (more than 32, for d = 64 more than 24, to 128: several tokens of many heads, or many
// heads on one KV head).
//
// With so many rows the transposed products of fa_decode_fp8.cuh are bound by their softmax
// (maxima across threads, weights written byte by byte, 16 rows at a time: 347 us for 128
// rows of 16 x 8192 keys x 8 heads). Here the rows lie along the tensor core's M = 128,
// as in the 16-bit kernel of fa_decode.cuh, with two softmax threads a row:
//     S = Q K^T   (M = 128 rows, N = 128 keys),   O += P V   (M = 128 rows, N = d)
// with P going through TMEM and O rescaled there when a row's maximum grows by more than
// 2^8. S is taken from the codes as they are, a product for each of the queries' E4M3 terms
// into the same columns (unscaled terms: exact where a value is within 2^-10 of the row's
// largest, else to 2^-18 of that). P needs a wide exponent range, which E4M3 terms do not
// have when a row keeps one reference: it is rounded to fp16, and four warps expand V's codes
// to fp16 in shared memory (exact). The keys' block factors join each score, and so does log2 of
// the values', as their share u of a power of two v_ref near the largest one met so far:
//     w = 2^(s + log2 u - m),   m at most 8 below the row's largest s + log2 u so far,
// so a block to which the row gives no weight, or that it must not see, costs the other weights
// nothing, whatever its factor. The sum of weights takes w / u; O is in units of v_ref 2^m, and
// when v_ref grows, m falls by as much and the products stay as they are. u counts as at least 2^-64.
//
// Work split, segments, teams and merge: fa_decode_fp8.cuh, with one item per KV head. For
// d = 64 a tile still loads the 128 bytes of two heads (the neighbouring CTA of the team
// takes the other from the L2) and uses one.
//
// Warps: 0 TMA producer, 1 TMEM and the MMA thread, 2 block factors, 3 NaN among the new
// tokens' values, 4-7 and 8-11 softmax (a row's first and second 64 keys of every tile, then
// half of its outputs; the two threads exchange their maxima), 12-15 the expansion of V and
// each segment's queries. One CTA an SM: two fp16 V tiles, a ring of six code tiles, Q's
// terms.
//
// Measured (16 x 8192 keys, 8 KV heads, d = 128, bf16): 118 us for 64 rows, 136 us for 128
// (178 and 347 us in chunks of 16 rows); d = 64: 103 and 114 us. A tile takes 2,900 cycles, of
// which the pipe of the exponentials and conversions is busy for 2,050 (two softmax warps and
// one of the expansion on an SM sub-partition). K expanded too: 146 and 168 us (when the codes'
// S took 119 and 138). From 33 rows on (d = 64: 25) the 16-bit decode of the same shape is faster:
// 105 and 122 us; d = 64: 89 and 103.
#pragma once

#include "fa_decode_fp8.cuh"

namespace fa {

template <bool BF16, int D>
struct Dec8RowsCfg {
    static constexpr int kThreads = 512;
    static constexpr int NT = BF16 ? 2 : 3;                // terms of a query
    static constexpr int kSlab = 128 * 128;                // 128 rows x 64 fp16 columns
    static constexpr int kTile = D / 64 * kSlab;           // an fp16 V tile
    static constexpr int kRaw = 128 * 128;                 // a tile of codes, or of one term of Q
    static constexpr int kUnits = 6;                       // ring of code tiles: K, V, K, V, ...
    static constexpr int kScSlots = 4;
    static constexpr int kQOff = 0;
    static constexpr int kVOff = kQOff + NT * kRaw;
    static constexpr int kRawOff = kVOff + 2 * kTile;
    static constexpr int kBarOff = kRawOff + kUnits * kRaw;
    static constexpr int kNumBars = 2 * kUnits + 4 + 2 + 2 * kScSlots + 4 + 3 + 2 + 16 + 2 * kNotices;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;       // 288 bytes: dec8_locate
    static constexpr int kScOff = (kMiscOff + 288 + 15) / 16 * 16;  // float [slots][kScSlot]
    static constexpr int kScSlot = 28;
    static constexpr int kQfOff = kScOff + kScSlots * kScSlot * 4;     // float [128]: scale of a query row
    static constexpr int kExOff = kQfOff + 128 * 4;               // float [3][2][128]: a row's halves (two tiles' maxima, sums)
    static constexpr int kLenOff = kExOff + 6 * 128 * 4;          // int [256]
    static constexpr int kLens = 256;
    static constexpr int kNanOff = kLenOff + kLens * 4;           // uint8 [8][128]: see dec8_hide_nan
    static constexpr int kSmemBytes = kNanOff + 8 * 128;
    static constexpr uint32_t kColO = 256;                        // S / P at 0 and 128
    static_assert(kUnits % 2 == 0, "a slot of the ring holds always K or always V");
    static_assert(kNotices >= ring_values(kUnits), "a notice barrier per value tile the ring holds");
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <bool BF16, int D, bool PAGED>
__global__ void __launch_bounds__(Dec8RowsCfg<BF16, D>::kThreads, 1)
    fa_decode8_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const Decode8Args args, const int causal) {
    using C = Dec8RowsCfg<BF16, D>;
    constexpr int U = C::kUnits, SC = C::kScSlots, NT = C::NT;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (!smem_base_ok(smem, args.err)) return;
    const int tid = static_cast<int>(threadIdx.x), warp = warp_id(), lane = lane_id();
    uint8_t* misc = smem + C::kMiscOff;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc);
    int* abort_flag = reinterpret_cast<int*>(misc + 4);
    uint8_t* sQ = smem + C::kQOff;
    uint8_t* sV = smem + C::kVOff;
    uint8_t* raw = smem + C::kRawOff;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [U] code tiles, unit 2 g: K of tile g, 2 g + 1: V
    uint64_t* empty = full + U;
    uint64_t* v_full = empty + U;     // [2] expanded V of tile g in buffer g & 1
    uint64_t* v_empty = v_full + 2;
    uint64_t* q_full = v_empty + 2;   // a segment's queries
    uint64_t* q_empty = q_full + 1;
    uint64_t* sc_full = q_empty + 1;  // [SC] a tile's block factors
    uint64_t* sc_empty = sc_full + SC;
    uint64_t* s_full = sc_empty + SC;  // [2]
    uint64_t* p_full = s_full + 2;     // [2]
    uint64_t* pv_done = p_full + 2;    // one completion per O += P V
    uint64_t* o_ready = pv_done + 1;   // the segment's products are complete
    uint64_t* o_free = o_ready + 1;    // O has been read
    uint64_t* mma_done = o_free + 1;
    uint64_t* sm_done = mma_done + 1;
    uint64_t* pair = sm_done + 1;      // [4][4] the two warps of 32 rows: per tile parity, per segment, per step of v_ref
    uint64_t* v_seen = pair + 16;      // [kNotices] a tile's values looked through by dec8_hide_nan
    uint64_t* v_due = v_seen + kNotices;  // [kNotices] the load of such a tile has begun
    float* sc = reinterpret_cast<float*>(smem + C::kScOff);
    float* qf = reinterpret_cast<float*>(smem + C::kQfOff);
    const bool part_seen = causal && args.Nq > 1;  // not every row sees the new tokens
    const int n_warps = (args.R + 31) / 32, n_act = 64 * n_warps;  // softmax warps of a half and threads that hold rows

    // Rows of Q past R are zeros: their scores are looked at by no one but must be there.
    for (int i = tid; i < NT * C::kRaw / 16; i += C::kThreads)
        if ((i % (C::kRaw / 16)) / 8 >= args.R) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (tid == 0) {
        for (int i = 0; i < U; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], i & 1 ? 4 : 1);  // V: the expansion's warps, K: the S product
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 128);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], n_act);
        }
        mbar_init(q_full, 128);
        mbar_init(q_empty, 1 + 2 * n_warps);  // the last S product, and each softmax warp's reading of the scales
        for (int i = 0; i < SC; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], 2 * n_warps);
        }
        mbar_init(pv_done, 1);
        mbar_init(o_ready, 1);
        mbar_init(o_free, n_act);
        for (int i = 0; i < kNotices; ++i) {
            mbar_init(&v_seen[i], 1);
            mbar_init(&v_due[i], 1);
        }
        mbar_init(mma_done, 1);
        mbar_init(sm_done, n_act);
        for (int i = 0; i < 16; ++i) mbar_init(&pair[i], 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // As fa_decode8_kernel: what follows reads the previous kernel's results.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    Dec8Range rg;
    const bool work = dec8_locate<C::kThreads, C::kLens>(args, misc, reinterpret_cast<int*>(smem + C::kLenOff), rg);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    if (!work) {
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }
    const WaitCtx wc{abort_flag, args.err};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
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
            const int x0 = (D == 64 ? it.hh / 2 : it.hh) * 128;  // first byte of the tile's columns
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
                const int next = j + 1 < n ? page_of(kt + 1) : 0;
                for (int kv = 0; kv < 2; ++kv, ++u) {
                    const int st = u % U;
                    if (!(ok = warp_all(mbar_wait(&empty[st], ((u / U) & 1) ^ 1u, wc, 140)))) break;
                    uint8_t* dst = raw + st * C::kRaw;
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(PAGED ? boxes * pb * 128 : C::kRaw));
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
            constexpr uint32_t id_s = idesc_e4m3(128, 128, false, false);
            constexpr uint32_t id_pv = idesc_f16(128, D, false, false, true);
            const uint32_t q_addr = smem_u32(sQ);
            // S of tile gg; col0: the head's first byte in the code rows.
            auto issue_s = [&](int gg, uint32_t col0) {
                const int st = (2 * gg) % U;
                const uint32_t k_addr = smem_u32(raw + st * C::kRaw) + col0;
#pragma unroll
                for (int i = 0; i < NT * (D / 32); ++i) {
                    const int t = i / (D / 32), kk = i % (D / 32);
                    mma_ss_f8(tmem + 128 * (gg & 1), sdesc_sw128(q_addr + t * C::kRaw + kk * 32, 16, 1024),
                              sdesc_sw128(k_addr + kk * 32, 16, 1024), id_s, i > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[gg & 1]);
                tc_commit(&empty[st]);
            };
            int gk = 0, nq = 0;
            bool ok = true;
            for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
                int j0, n;
                if (!dec8_segment(rg, it, j0, n)) continue;
                const uint32_t col0 = D == 64 ? (it.hh & 1) * 64 : 0;
                if (!(ok = mbar_wait(q_full, nq & 1, wc, 141))) break;
                for (int j = 0; ok && j < min(n, 2); ++j) {
                    const int gg = gk + j, u = 2 * gg;
                    if (!(ok = mbar_wait(&full[u % U], (u / U) & 1, wc, 142))) break;
                    tc_fence_after();
                    issue_s(gg, col0);
                }
                if (!ok) break;
                if (n <= 2) tc_commit(q_empty);
                for (int j = 0; ok && j < n; ++j) {
                    const int gg = gk + j, b = gg & 1;
                    if (!(ok = mbar_wait(&v_full[b], (gg >> 1) & 1, wc, 143))) break;
                    // O is overwritten by the segment's first P V: the previous segment's
                    // epilogue must have read it.
                    if (j == 0 && nq > 0 && !(ok = mbar_wait(o_free, (nq - 1) & 1, wc, 144))) break;
                    if (!(ok = mbar_wait(&p_full[b], (gg >> 1) & 1, wc, 145))) break;
                    tc_fence_after();
                    const uint32_t v_addr = smem_u32(sV + b * C::kTile);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::kColO, tmem + 128 * b + kk * 8, sdesc_sw128(v_addr + kk * 2048, C::kSlab, 1024),
                               id_pv, (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(pv_done);
                    tc_commit(&v_empty[b]);
                    // S of tile gg + 2 into the columns P was just read from: one thread's
                    // tcgen05.mma operations execute in issue order.
                    if (j + 2 < n) {
                        const int u2 = 2 * (gg + 2);
                        if (!(ok = mbar_wait(&full[u2 % U], (u2 / U) & 1, wc, 146))) break;
                        tc_fence_after();
                        issue_s(gg + 2, col0);
                        if (j + 3 == n) tc_commit(q_empty);
                    }
                }
                tc_commit(o_ready);
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
        tmem_dealloc(tmem, 512);
    } else if (warp == 2) {
        // ------------------------------------------------------------ block factors
        // Lane x + 8 kv: keys 16 x .. of a tile, key or value factor. A slot holds the 8 key
        // factors, log2 and inverse of the 8 value factors as shares of v_ref, that power of two (the
        // segment's largest factor so far, rounded down; 0: none yet) and log2 of its step.
        const int x = lane & 7, kv = (lane >> 3) & 1;
        int gk = 0;
        bool ok = true;
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            const float* f = kv ? args.v_scale : args.k_scale;
            auto read = [&](int kt) -> float {
                const int key = kt * 128 + x * 16;
                if (lane >= 16 || key >= it.len) return 0.f;
                if constexpr (PAGED) {
                    const int pg = args.block_table[static_cast<size_t>(it.b) * args.per_seq + key / args.page_size];
                    return pg >= 0 && pg < args.num_pages ? f[static_cast<size_t>(pg) * args.Hkv + it.hh] : 0.f;
                } else {
                    return f[(static_cast<size_t>(it.b) * args.Hkv + it.hh) * args.per_seq + kt];
                }
            };
            float v = read(j0), v_ref = 0.f, e_ref = 0.f;  // v_ref = 2^e_ref, or 0
            for (int j = 0; j < n; ++j) {
                const int gg = gk + j, slot = gg % SC;
                const float next = j + 1 < n ? read(j0 + j + 1) : 0.f;
                float top = v, step = 0.f;
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                top = __shfl_sync(0xffffffffu, top, 8);
                const int e = max(static_cast<int>(__float_as_uint(top) >> 23), 1) - 127;
                if (top > 0.f && (v_ref == 0.f || static_cast<float>(e) > e_ref)) {
                    if (v_ref > 0.f) step = static_cast<float>(e) - e_ref;
                    v_ref = exp2_int(e);
                    e_ref = static_cast<float>(e);
                }
                const float lg = dec8_share(v, e_ref);
                if (!(ok = warp_all(mbar_wait(&sc_empty[slot], ((gg / SC) & 1) ^ 1u, wc, 147)))) break;
                float* s = sc + slot * C::kScSlot;
                // Keys without a block (past the end, pages outside the pool) have zero codes or
                // are masked: any key factor does, but -inf times it has to stay -inf.
                if (lane < 16) s[kv * 8 + x] = kv ? lg : (v == 0.f ? 1.f : v);
                if (lane < 16 && kv) s[16 + x] = ex2_approx(-lg);
                if (lane == 8) *reinterpret_cast<float2*>(s + 24) = make_float2(v_ref, step);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[slot]);
                v = next;
            }
            gk += n;
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ NaN of new tokens
        int gk = 0, nq = 0, n_told = 0;
        bool ok = true;
        for (Dec8Item it = rg.first; ok && part_seen && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            const int first_part = it.len - args.Nq + 1;
            // Segment nq - 8, the last to use this part of the notes, has been read: the ring holds V
            // of three tiles and the products run at most two behind, so with V of tile g here the
            // scores of tile g - 5 have been read, and the results of tiles before it.
            uint32_t* noted = reinterpret_cast<uint32_t*>(smem + C::kNanOff + (nq & 7) * 128) + lane;
            uint32_t first = 0xffffffffu;
            for (int j = max(first_part / 128 - j0, 0); j < n; ++j) {
                const int key0 = (j0 + j) * 128, u = 2 * (gk + j) + 1, st = u % U;
                if (!(ok = warp_all(mbar_wait(&v_due[notice_bar(n_told)], notice_parity(n_told), wc, 161)))) break;
                if (!(ok = warp_all(mbar_wait(&full[st], (u / U) & 1, wc, 159)))) break;
                dec8_hide_nan(raw + st * C::kRaw, key0, first_part, it.len, first);
                *noted = first;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_seen[notice_bar(n_told)]);
                ++n_told;
            }
            gk += n;
            ++nq;
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ expansion
        const int t = tid - 384;
        int gk = 0, nq = 0, n_seen = 0;
        bool ok = true;
        // 16 codes (a 16-byte piece) to 16 fp16 values.
        auto expand = [](uint32_t w, uint32_t& lo, uint32_t& hi) {
            lo = h2_of_e4m3x2(w & 0xffffu);
            hi = h2_of_e4m3x2(w >> 16);
        };
        // Code tile of ring unit u into the 16-bit tile `dst`, rows from `rows` on as zeros.
        auto tile = [&](int u, uint8_t* dst, int rows, int col0) -> bool {
            const int st = u % U;
            if (!warp_all(mbar_wait(&full[st], (u / U) & 1, wc, 148))) return false;
            const uint8_t* src = raw + st * C::kRaw;
            constexpr int P = D / 16;  // pieces of a row
#pragma unroll 4
            for (int i = t; i < 128 * P; i += 128) {
                const int r = i / P, c = i % P;
                uint4 w = *reinterpret_cast<const uint4*>(src + r * 128 + (((c + col0) ^ (r & 7)) << 4));
                if (r >= rows) w = make_uint4(0, 0, 0, 0);
                uint4 a, b;
                expand(w.x, a.x, a.y);
                expand(w.y, a.z, a.w);
                expand(w.z, b.x, b.y);
                expand(w.w, b.z, b.w);
                // Values 16 c .. + 7 and + 8 ..: two 16-byte pieces of the slab's row. The lanes of the
                // second slab store theirs in the other order (the slabs share banks).
                uint8_t* row = dst + (c >> 2) * C::kSlab + r * 128;
                const int p0 = 2 * (c & 3), flip = (c >> 2) & 1;
                *reinterpret_cast<uint4*>(row + (((p0 + flip) ^ (r & 7)) << 4)) = flip ? b : a;
                *reinterpret_cast<uint4*>(row + (((p0 + 1 - flip) ^ (r & 7)) << 4)) = flip ? a : b;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            return true;
        };
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            // The queries' terms: eight lanes (d = 64) or sixteen take a row, 8 values each.
            if (!(ok = warp_all(mbar_wait(q_empty, (nq & 1) ^ 1u, wc, 149)))) break;
            constexpr int QP = D / 8;
#pragma unroll 1
            for (int i = t; i < 128 * QP; i += 128) {
                const int r = i / QP, c = i % QP;
                if (r - (lane / QP) >= args.R) break;  // uniform over the warp: its first row
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < args.R) {
                    const size_t row = (static_cast<size_t>(it.b) * args.Nq + r / args.group) * args.Hq +
                                       static_cast<size_t>(it.hh) * args.group + r % args.group;
                    w = *reinterpret_cast<const uint4*>(args.q + row * D + c * 8);
                }
                const float scale = dec8_piece_put<BF16, QP, NT, false>(
                    w, [&](int k) { return sQ + k * C::kRaw + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8; });
                if (c == 0) qf[r] = args.scale_log2 * scale;
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
            const int j_part = part_seen ? max(it.len - args.Nq + 1, 0) / 128 - j0 : n;  // first tile of v_seen
            for (int j = 0; ok && j < n; ++j) {
                const int gg = gk + j, b = gg & 1;
                // Rows past the sequence's end may hold anything (0 x NaN would reach O).
                const int rows = min(128, it.len - (j0 + j) * 128);
                if (j >= j_part) {
                    if (!(ok = warp_all(mbar_wait(&v_seen[notice_bar(n_seen)], notice_parity(n_seen), wc, 160)))) break;
                    ++n_seen;
                }
                if (!(ok = warp_all(mbar_wait(&v_empty[b], ((gg >> 1) & 1) ^ 1u, wc, 151)))) break;
                if (!(ok = tile(2 * gg + 1, sV + b * C::kTile, rows, D == 64 ? (it.hh & 1) * 4 : 0))) break;
                fence_proxy_async_smem();
                mbar_arrive(&v_full[b]);
            }
            gk += n;
            ++nq;
        }
    } else if (warp >= 4 && (warp & 3) < n_warps) {
        // ------------------------------------------------------------ softmax, output
        const int w4 = warp & 3, half = (warp - 4) >> 2, r = w4 * 32 + lane;  // r: TMEM lane and query row
        const bool live = r < args.R;
        const int tok = live ? r / args.group : 0;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
        const uint32_t o_addr = lane_base + C::kColO + half * (D / 2);  // this thread's outputs
        float* ex = reinterpret_cast<float*>(smem + C::kExOff);
        uint64_t* meets = pair + 4 * w4;
        auto meet = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            return warp_all(mbar_wait(bar, parity, wc, site));
        };
        int gk = 0, nq = 0, n_steps = 0;
        bool ok = true;
        for (Dec8Item it = rg.first; ok && it.P < rg.hi; it = dec8_next(args, rg, it)) {
            int j0, n;
            if (!dec8_segment(rg, it, j0, n)) continue;
            const int key_hi = causal ? min(it.len, tok + it.len - args.Nq + 1) : it.len;
            const int all_hi = it.len - args.Nq + 1;  // (causal) keys below it are seen by every row
            const int rel_hi = key_hi - j0 * 128;
            ok = warp_all(mbar_wait(q_full, nq & 1, wc, 152));
            if (!ok) break;
            const float my_qf = live ? qf[r] : 1.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty);
            float m = -INFINITY, l = 0.f, v_ref = 0.f;
            for (int j = 0; j < n; ++j) {
                const int gg = gk + j, b = gg & 1, slot = gg % SC;
                ok = warp_all(mbar_wait(&sc_full[slot], (gg / SC) & 1, wc, 153));
                if (!ok) break;
                const float* s_sc = sc + slot * C::kScSlot + 4 * half;
                const float2 ref = *reinterpret_cast<const float2*>(sc + slot * C::kScSlot + 24);
                v_ref = ref.x;
                ok = warp_all(mbar_wait(&s_full[b], (gg >> 1) & 1, wc, 154));
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_addr = lane_base + 128 * b;
                const int lim = rel_hi - j * 128 - 64 * half;  // this half's columns >= lim are masked
                uint32_t sv[2][32];
                tmem_ld32(s_addr + 64 * half, sv[0]);
                tmem_ld32(s_addr + 64 * half + 32, sv[1]);
                const float4 f4 = *reinterpret_cast<const float4*>(s_sc);
                const float4 g4 = *reinterpret_cast<const float4*>(s_sc + 8);
                const float vl[4] = {g4.x, g4.y, g4.z, g4.w};
                // Masked scores are -inf before they are scaled and have to stay so: a product below
                // fp32's range (a zero row over a block of zeros: 2^-200) counts as the smallest
                // normal value instead, with which any raw score is below 2^-100.
                auto scaled = [my_qf](float f) { return f * my_qf == 0.f ? 1.17549435e-38f : f * my_qf; };
                const float kf[4] = {scaled(f4.x), scaled(f4.y), scaled(f4.z), scaled(f4.w)};
                float alpha = 1.f;
                bool resc = false;
                if (ref.y > 0.f) {
                    // v_ref 2^step: m falls by the step, O stays, the sum of weights 2^(s - m) grows. Past
                    // 2^80 of that sum (of both halves) O is scaled down instead: 2^72 a key still to come
                    // leaves fp32's range to more keys than a sequence has.
                    ex[(4 + half) * 128 + r] = l;
                    ok = meet(&meets[3], n_steps++ & 1, 162);
                    if (!ok) break;
                    const float both = l + ex[(5 - half) * 128 + r];
                    const int room = min(max(80 - (static_cast<int>(__float_as_uint(both) >> 23) - 127), 0), 120);
                    const float down = fminf(ref.y, static_cast<float>(room));
                    m -= down;
                    l *= exp2_int(static_cast<int>(down));
                    alpha = ex2_approx(down - ref.y);
                    resc = down < ref.y;
                }
                tmem_ld_wait(sv[0]);
                tmem_ld_wait(sv[1]);
                if (__any_sync(0xffffffffu, lim < 64)) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (i >= lim) sv[i >> 5][i & 31] = __float_as_uint(-INFINITY);
                }
                // The largest scaled score with its V share: a block's largest raw one is scaled.
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(sv[g >> 1][16 * (g & 1) + i]);
                    const float a = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8]));
                    const float c = fmax3(fmax3(x[9], x[10], x[11]), fmax3(x[12], x[13], x[14]), x[15]);
                    mx = fmaxf(mx, fmaf(fmaxf(a, c), kf[g], vl[g]));
                }
                // The row's other half (and both have read the scores' columns from here on).
                tc_fence_before();
                ex[(b * 2 + half) * 128 + r] = mx;
                ok = meet(&meets[b], (gg >> 1) & 1, 157);
                if (!ok) break;
                tc_fence_after();
                mx = fmaxf(mx, ex[(b * 2 + 1 - half) * 128 + r]);
                if (mx > m + kRescaleThreshold) {
                    if (m != -INFINITY) {
                        const float a = ex2_approx(m - mx);
                        alpha *= a;
                        l *= a;
                        resc = true;
                    }
                    m = mx;
                }
                const float neg_m = m == -INFINITY ? 0.f : -m;
                uint32_t pk[16];
                // (The shares once more: kept over the maximum they cost registers, 126 against 117 us.)
                const float4 h4 = *reinterpret_cast<const float4*>(s_sc + 8);
                const float4 i4 = *reinterpret_cast<const float4*>(s_sc + 16);
                const float vm[4] = {h4.x + neg_m, h4.y + neg_m, h4.z + neg_m, h4.w + neg_m}, vi[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint64_t c2 = f2_pack(kf[g], kf[g]), m2 = f2_pack(vm[g], vm[g]);
                    uint64_t sum = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 16 * (g & 1) + 2 * i;
                        float y0, y1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[g >> 1][k]), __uint_as_float(sv[g >> 1][k + 1])), c2, m2), y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        sum = f2_add(sum, f2_pack(p0, p1));
                        pk[8 * (g & 1) + i] = pack2<false>(p0, p1);
                    }
                    l = fmaf(f2_sum(sum), vi[g], l);
                    if (g & 1) tmem_st16(s_addr + 32 * half + 8 * (g - 1), pk);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_empty[slot]);
                // Rescale O once the previous tile's P V is complete.
                if (j > 0 && __any_sync(0xffffffffu, resc)) {
                    ok = warp_all(mbar_wait(pv_done, (gg - 1) & 1, wc, 155));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < D / 2; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32(o_addr + c0, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st32(o_addr + c0, ov);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[b]);
            }
            if (!ok) break;
            ex[(4 + half) * 128 + r] = l;
            ok = meet(&meets[2], nq & 1, 158);
            if (!ok) break;
            l += ex[(5 - half) * 128 + r];
            ok = warp_all(mbar_wait(o_ready, nq & 1, wc, 156));
            if (!ok) break;
            tc_fence_after();
            const size_t row = dec8_slot(args, rg.team, it.b, it.hg, rg.hl) * args.RT + (live ? r : 0);
            const float inv = l == 0.f ? 0.f : __fdividef(v_ref, l);  // no key: 0; NaN stays NaN
            float* dst = args.o_part + row * D + half * (D / 2);
#pragma unroll
            for (int c0 = 0; c0 < D / 2; c0 += 32) {
                uint32_t ov[32];
                tmem_ld32(o_addr + c0, ov);
                tmem_ld_wait(ov);
                if (part_seen && (j0 + n) * 128 > all_hi) {
                    const uint8_t* noted = smem + C::kNanOff + (nq & 7) * 128 + (D == 64 ? (it.hh & 1) * 64 : 0) + half * (D / 2) + c0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (key_hi > all_hi + noted[i]) ov[i] = 0x7fffffffu;
                }
                if (live) {
                    float4* d4 = reinterpret_cast<float4*>(dst + c0);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d4[i] = make_float4(__uint_as_float(ov[4 * i]) * inv, __uint_as_float(ov[4 * i + 1]) * inv,
                                            __uint_as_float(ov[4 * i + 2]) * inv, __uint_as_float(ov[4 * i + 3]) * inv);
                }
            }
            tc_fence_before();
            mbar_arrive(o_free);
            if (live && half == 0) {
                float lg;
                asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(l));
                args.lse_part[row] = l == 0.f ? -INFINITY : m + lg;
            }
            gk += n;
            ++nq;
        }
        tc_fence_before();
        mbar_arrive(sm_done);
    }
}

}  // namespace fa
