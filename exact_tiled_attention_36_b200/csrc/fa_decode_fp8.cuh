// fa_decode_fp8.cuh: attention of a few query tokens per sequence over an E4M3 key/value
// cache with one float32 factor per block of tokens and KV head, on sm_100a.
//
//     s_j = scale k_f(j) (q . k8_j),  O = sum_j softmax(s)_j v_f(j) v8_j
#pragma once

#include "sm100.cuh"

namespace fa {

struct Decode8Args {
    const void* q;           // [B, Nq, Hq, d] 16-bit
    const uint8_t* k;        // [B, Nk, Hkv, d] or [num_pages, page_size, Hkv, d]
    const uint8_t* v;
    const float* k_scale;    // [B, Hkv, per_seq] or [num_pages, Hkv]
    const float* v_scale;
    void* o;                 // [B, Nq, Hq, d] 16-bit
    float* lse;              // [B, Hq, Nq]
    const int* seqlens;      // [B] or null (every sequence has cap keys)
    const int* block_table;  // [B, per_seq]; null: contiguous
    int B, Hq, Hkv, group, Nq;
    int cap, unit, per_seq, num_pages;  // keys a sequence can hold, keys of a block, blocks of a sequence
    float scale_log2;
};

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(byte));
    return unpack_lo<false>(h);
}

// One CTA per query row: its four warps take every fourth key, a lane d / 32 values,
// each warp with an online softmax of its own; the four are merged at the end.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_decode8_rows_kernel(const Decode8Args a, const int causal) {
    constexpr int E = D / 32;
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    const int lane = lane_id(), warp = warp_id();
    const int h = static_cast<int>(blockIdx.x % a.Hq);
    const int t = static_cast<int>(blockIdx.x / a.Hq % a.Nq), b = static_cast<int>(blockIdx.x / a.Hq / a.Nq);
    const int hk = h / a.group;
    const int len = a.seqlens ? min(max(a.seqlens[b], 0), a.cap) : a.cap;
    const int hi = causal ? min(len, t + len - a.Nq + 1) : len;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((static_cast<size_t>(b) * a.Nq + t) * a.Hq + h) * D + lane * E;
    float qv[E], acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        qv[i] = unpack_lo<BF16>(q[i]);
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < hi; j += 4) {
        const int blk = j / a.unit;
        size_t row;
        float kf = 0.f, vf = 0.f;
        bool in = true;
        if (a.block_table) {
            const int pg = a.block_table[static_cast<size_t>(b) * a.per_seq + blk];
            in = pg >= 0 && pg < a.num_pages;  // a page outside the pool reads zeros
            row = static_cast<size_t>(in ? pg : 0) * a.unit + j % a.unit;
            if (in) {
                kf = a.k_scale[static_cast<size_t>(pg) * a.Hkv + hk];
                vf = a.v_scale[static_cast<size_t>(pg) * a.Hkv + hk];
            }
        } else {
            row = static_cast<size_t>(b) * a.cap + j;
            const size_t f = (static_cast<size_t>(b) * a.Hkv + hk) * a.per_seq + blk;
            kf = a.k_scale[f];
            vf = a.v_scale[f];
        }
        const size_t at = (row * a.Hkv + hk) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += in ? qv[i] * e4m3_to_float(a.k[at + i]) : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2 * kf;
        const float m_new = fmaxf(m, s);
        const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
        const float p = ex2_approx(s - m_new);
        m = m_new;
        l = l * alpha + p;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = acc[i] * alpha + (in ? p * vf * e4m3_to_float(a.v[at + i]) : 0.f);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = acc[i];
    __syncthreads();
    const float mx = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float w[4], lt = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = s_m[i] == -INFINITY ? 0.f : ex2_approx(s_m[i] - mx);
        lt += w[i] * s_l[i];
    }
    const int c = static_cast<int>(threadIdx.x);
    if (c < D) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x += w[i] * s_o[i][c];
        const uint32_t u = pack2<BF16>(lt > 0.f ? x / lt : (lt == 0.f ? 0.f : lt), 0.f);
        static_cast<uint16_t*>(a.o)[((static_cast<size_t>(b) * a.Nq + t) * a.Hq + h) * D + c] =
            static_cast<uint16_t>(u & 0xffffu);
    }
    if (c == 0) a.lse[(static_cast<size_t>(b) * a.Hq + h) * a.Nq + t] = lt == 0.f ? -INFINITY : (mx + log2f(lt)) * kLn2;
}

}  // namespace fa
