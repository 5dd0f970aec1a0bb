// fa_serve.cu: the serving entry points of libfa.so (declared in include/fa.h): decode
// over an E4M3 cache, the cache appends, and block tables with slot maps. Host side
// only: argument validation and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "per_device.h"
#include "fa_cache.cuh"
#include "fa_decode_fp8.cuh"
#include "fa_decode_fp8_rows.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634074f;

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

cudaStream_t cu(fa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// {token, head} strides of a [T, Hkv, d] tensor (null: contiguous).
fa_status row_strides(const long long* p, int Hkv, int d, long long& st, long long& sh) {
    st = p ? p[0] : static_cast<long long>(Hkv) * d;
    sh = p ? p[1] : d;
    if (st <= 0 || sh <= 0) return FA_ERR_INVALID_ARG;
    return st % 8 || sh % 8 ? FA_ERR_MISALIGNED : FA_OK;
}

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || (ps > 0 && ps % 64 == 0); }

fa_status append_checks(const void* k, const void* v, const void* kc, const void* vc, int total_new, int Hkv, int d,
                        fa_dtype dtype) {
    if (total_new < 0 || Hkv < 1) return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (Hkv > 65535) return FA_ERR_UNSUPPORTED;
    if (total_new > 0 && (!k || !v || !kc || !vc)) return FA_ERR_INVALID_ARG;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(kc, 16) || misaligned(vc, 16)) return FA_ERR_MISALIGNED;
    return FA_OK;
}

// `chunks`: pieces of 8 values that a block's new rows of one head can have.
template <bool BF16, int D>
fa_status launch_append8(const fa::Append8Args& a, long long chunks, cudaStream_t s) {
    const bool warps = chunks <= 32 * fa::kHold;
    const long long ctas = warps ? (a.groups + 7) / 8 : a.groups;
    if (ctas > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(ctas);
    if (warps) fa::fa_append8_kernel<BF16, D, 32><<<grid, 256, 0, s>>>(a);
    else if (chunks <= 64 * fa::kHold) fa::fa_append8_kernel<BF16, D, 64><<<grid, 64, 0, s>>>(a);
    else if (chunks <= 128 * fa::kHold) fa::fa_append8_kernel<BF16, D, 128><<<grid, 128, 0, s>>>(a);
    else fa::fa_append8_kernel<BF16, D, 256><<<grid, 256, 0, s>>>(a);
    return launched();
}

// fa_cache_append_fp8 (block_table null: caches [B, Nk, Hkv, d], cap = Nk) and
// fa_cache_append_paged_fp8 (page pools).
fa_status append8(const void* k, const void* v, const long long* k_strides, const long long* v_strides,
                  void* kc, void* vc, float* k_scale, float* v_scale, const int* cu_new, const int* seqlens,
                  const int* new_seqlens, const int* block_table, bool paged, int B, int total_new, int max_new,
                  int Hkv, int num_pages, int unit, int per_seq, int cap, int d, fa_dtype dtype, fa_stream_t stream) {
    if (B < 1 || max_new < 0) return FA_ERR_INVALID_ARG;
    fa_status st = append_checks(k, v, kc, vc, total_new, Hkv, d, dtype);
    if (st != FA_OK) return st;
    if (!cu_new || !seqlens || !new_seqlens || !k_scale || !v_scale || (paged && !block_table))
        return FA_ERR_INVALID_ARG;
    if (misaligned(cu_new, 4) || misaligned(seqlens, 4) || misaligned(new_seqlens, 4) || misaligned(block_table, 4) ||
        misaligned(k_scale, 4) || misaligned(v_scale, 4))
        return FA_ERR_MISALIGNED;
    fa::Append8Args a{};
    if ((st = row_strides(k_strides, Hkv, d, a.st[0], a.sh[0])) != FA_OK) return st;
    if ((st = row_strides(v_strides, Hkv, d, a.st[1], a.sh[1])) != FA_OK) return st;
    if (total_new == 0 || max_new == 0 || cap == 0) return FA_OK;
    a.x[0] = static_cast<const uint16_t*>(k);
    a.x[1] = static_cast<const uint16_t*>(v);
    a.codes[0] = static_cast<uint8_t*>(kc);
    a.codes[1] = static_cast<uint8_t*>(vc);
    a.factors[0] = k_scale;
    a.factors[1] = v_scale;
    a.cu_new = cu_new;
    a.seqlens = seqlens;
    a.new_seqlens = new_seqlens;
    a.block_table = paged ? block_table : nullptr;
    a.B = B;
    a.Hkv = Hkv;
    a.total_new = total_new;
    a.max_new = max_new < total_new ? max_new : total_new;
    a.unit = unit;
    a.cap = cap;
    a.per_seq = per_seq;
    a.num_pages = num_pages;
    // max_new consecutive tokens touch at most 1 + ceil((max_new - 1) / unit) blocks.
    const long long touched = 1 + (a.max_new - 1LL + unit - 1) / unit;
    a.touched = touched < per_seq ? static_cast<int>(touched) : per_seq;
    a.groups = static_cast<long long>(B) * a.touched * Hkv * 2;
    a.err = fa_host::error_word();
    if (!a.err) return FA_ERR_CUDA;
    const long long chunks = static_cast<long long>(a.max_new < unit ? a.max_new : unit) * (d / 8);
    const cudaStream_t s = cu(stream);
    if (dtype == FA_BF16) return d == 64 ? launch_append8<true, 64>(a, chunks, s) : launch_append8<true, 128>(a, chunks, s);
    return d == 64 ? launch_append8<false, 64>(a, chunks, s) : launch_append8<false, 128>(a, chunks, s);
}

// More rows of a KV head than this take the form with the rows along M. Measured, 16 x 8192 keys
// and 8 KV heads, in chunks (of 16 rows; d = 64: 8) against it: d = 128, 32 rows 96 us against 111,
// 40 rows 138 against 108; d = 64, 24 rows 86 us against 98, 32 rows 109 against 98.
int dec8_many_rows(int d) { return d == 64 ? 24 : 32; }

// How a call's rows become items, and its workspace: meta (each item's first and last team), the
// partial L and O (fp32) of slots = teams x TS + items, RT rows each.
struct Dec8Plan {
    bool rows;    // the form with the rows along M (fa_decode8_rows_kernel)
    int rt;       // rows of a tile: the smallest of 4, 8, 16 that holds a head's (d = 64: two heads') rows
    int heads;    // KV heads of an item
    int nch, RC;  // chunks a head's rows are cut into, and rows of a chunk
    int HV, TS;   // items of a sequence, items of a group (a team of CTAs)
    long long items, teams;
    size_t meta, lse, total;
};

bool dec8_plan(int B, int Hq, int Hkv, int Nq, int d, Dec8Plan& p) {
    const int sms = fa_host::sm_count();
    if (sms <= 0) return false;
    const int R = Hq / Hkv * (Nq > 0 ? Nq : 1);
    p.rows = R > dec8_many_rows(d);
    if (p.rows) {
        p.rt = p.RC = R;
        p.heads = p.nch = 1;
    } else {
        p.heads = d == 64 ? 2 : 1;
        p.rt = p.heads * R <= 4 ? 4 : p.heads * R <= 8 ? 8 : 16;
        const int most = p.rt / p.heads;
        p.nch = (R + most - 1) / most;
        p.RC = (R + p.nch - 1) / p.nch;
    }
    p.HV = (Hkv + p.heads - 1) / p.heads * p.nch;
    p.items = static_cast<long long>(B) * p.HV;
    // A team walks 8 items in step, or as many as divide a sequence's items evenly: 8 heads' codes
    // are 1 KB of a token, and 296 CTAs make 37 teams of 8.
    p.TS = 1;
    for (int n = 2; n <= 16 && n <= p.HV; ++n)
        if (p.HV % n == 0 && (n <= 8 || p.TS == 1)) p.TS = n;
    p.teams = static_cast<long long>(sms) * (p.rows ? 1 : fa::kDec8Ctas) / p.TS;
    if (p.teams < 1) p.teams = 1;
    const size_t slots = static_cast<size_t>(p.items + p.teams * p.TS) * p.rt;
    auto round = [](size_t x) { return (x + 255) & ~size_t(255); };
    p.meta = round(p.items * sizeof(int2));
    p.lse = round(slots * sizeof(float));
    p.total = p.meta + p.lse + round(slots * d * sizeof(float));
    return true;
}

// Codes [outer, rows, row bytes]: boxes of `box` rows x 128 bytes.
fa_status code_map(CUtensorMap* m, const void* base, int64_t row, int64_t rows, int64_t outer, int box) {
    return fa_host::make_map_box(m, base, static_cast<int>(row), static_cast<int>(rows), outer, 1, false, row,
                                 row * rows, row * rows * outer, box, 1, false, 1);
}

template <auto Kern>
bool kernel_ready(int smem) {
    static fa::PerDevice<int> done;
    int n = 0;
    return done.get(fa_host::current_device(), [smem](int& v) {
        v = 1;
        return cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
    }, &n);
}

// The split kernel and the merge, each launched as a programmatic dependent of the kernel before
// it on the stream: the launch and the part before its griddepcontrol.wait overlap that one's end.
template <auto Kern, bool BF16, int D>
fa_status launch_dec8_k(int threads, int smem, const CUtensorMap& mk, const CUtensorMap& mv, const fa::Decode8Args& a,
                        int causal, bool run_split, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (run_split) {
        if (!kernel_ready<Kern>(smem)) return FA_ERR_CUDA;
        cfg.gridDim = dim3(a.teams * a.TS);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        if (cudaLaunchKernelEx(&cfg, Kern, mk, mv, a, causal) != cudaSuccess) return FA_ERR_CUDA;
    }
    // A row's segments: about teams / groups, one or two more where ranges cross.
    const int rows = a.B * a.Hq * a.Nq;
    const bool wide = a.teams > 6LL * a.B * a.HG;
    cfg.gridDim = dim3(wide ? rows : (rows + 3) / 4);
    cfg.blockDim = dim3(wide ? 32 * fa::kDec8WideWarps : 128);
    cfg.dynamicSmemBytes = 0;
    if ((wide ? cudaLaunchKernelEx(&cfg, fa::fa_decode8_combine<D, BF16, true>, a, rows)
              : cudaLaunchKernelEx(&cfg, fa::fa_decode8_combine<D, BF16, false>, a, rows)) != cudaSuccess)
        return FA_ERR_CUDA;
    return launched();
}

template <bool BF16, int D, bool PAGED, int RT>
fa_status launch_dec8_t(const CUtensorMap& mk, const CUtensorMap& mv, const fa::Decode8Args& a, int causal,
                        bool run_split, cudaStream_t s) {
    using C = fa::Dec8Cfg<BF16, D == 64, RT>;
    return launch_dec8_k<fa::fa_decode8_kernel<BF16, D == 64, PAGED, RT>, BF16, D>(C::kThreads, C::kSmemBytes, mk, mv, a,
                                                                                 causal, run_split, s);
}

// rt: rows of a tile (0: the form with the rows along M).
template <bool BF16, int D, bool PAGED>
fa_status launch_dec8_r(int rt, const CUtensorMap& mk, const CUtensorMap& mv, const fa::Decode8Args& a, int causal,
                        bool run_split, cudaStream_t s) {
    if (rt == 4) return launch_dec8_t<BF16, D, PAGED, 4>(mk, mv, a, causal, run_split, s);
    if (rt == 8) return launch_dec8_t<BF16, D, PAGED, 8>(mk, mv, a, causal, run_split, s);
    if (rt == 16) return launch_dec8_t<BF16, D, PAGED, 16>(mk, mv, a, causal, run_split, s);
    using C = fa::Dec8RowsCfg<BF16, D>;
    return launch_dec8_k<fa::fa_decode8_rows_kernel<BF16, D, PAGED>, BF16, D>(C::kThreads, C::kSmemBytes, mk, mv, a,
                                                                            causal, run_split, s);
}

template <bool BF16>
fa_status launch_dec8(int rt, int d, bool paged, const CUtensorMap& mk, const CUtensorMap& mv,
                      const fa::Decode8Args& a, int causal, bool run_split, cudaStream_t s) {
    if (d == 64) return paged ? launch_dec8_r<BF16, 64, true>(rt, mk, mv, a, causal, run_split, s)
                              : launch_dec8_r<BF16, 64, false>(rt, mk, mv, a, causal, run_split, s);
    return paged ? launch_dec8_r<BF16, 128, true>(rt, mk, mv, a, causal, run_split, s)
                 : launch_dec8_r<BF16, 128, false>(rt, mk, mv, a, causal, run_split, s);
}

fa_status decode8(const void* q, const void* k, const void* v, const float* k_scale, const float* v_scale, void* o,
                  float* lse, const int* seqlens, const int* block_table, void* workspace, int B, int Hq, int Hkv,
                  int Nq, int Nk, bool paged, int num_pages, int page_size, int max_pages, int d, float scale,
                  int causal, fa_dtype dtype, fa_stream_t stream) {
    if (B < 1 || Nq < 0 || Nk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (paged) {
        if (!seqlens || !block_table || num_pages < 1 || max_pages < 1 || page_size < 16) return FA_ERR_INVALID_ARG;
        if (!page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
        if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    }
    const int cap = paged ? max_pages * page_size : Nk;
    if (cap > 0x7fffffff - 8192) return FA_ERR_UNSUPPORTED;  // key indices of a tile and its boxes stay below 2^31
    if (Nq > 0 && (!q || !o || !lse || !workspace)) return FA_ERR_INVALID_ARG;
    if (cap > 0 && (!k || !v || !k_scale || !v_scale)) return FA_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(lse, 16) ||
        misaligned(workspace, 16) || misaligned(k_scale, 4) || misaligned(v_scale, 4) || misaligned(seqlens, 4) ||
        misaligned(block_table, 4))
        return FA_ERR_MISALIGNED;
    fa_status st = FA_OK;
    const int g = Hq / Hkv;
    if (static_cast<long long>(g) * Nq > 128) return FA_ERR_UNSUPPORTED;
    if (Hq > 65535 || B > 65535 || static_cast<long long>(B) * Hq * Nq > 0x7ffffff0LL) return FA_ERR_UNSUPPORTED;
    if (Nq == 0) return FA_OK;
    Dec8Plan pl;
    if (!dec8_plan(B, Hq, Hkv, Nq, d, pl)) return FA_ERR_CUDA;
    const long long tiles = pl.items * ((static_cast<long long>(cap) + 127) / 128);
    if (pl.items > 0x7fffffffLL || tiles > (1LL << 40)) return FA_ERR_UNSUPPORTED;
    fa::Decode8Args a{};
    a.err = fa_host::error_word();
    if (!a.err) return FA_ERR_CUDA;
    const int box = !paged ? 128 : page_size % 128 == 0 ? 128 : page_size < 64 ? page_size : 64;
    CUtensorMap mk{}, mv{};
    if (cap > 0) {
        // One row of codes as Hkv d columns: a box takes 128 of them (a head, or two of 64; past
        // an odd number of small heads it reads zeros).
        const int64_t row = static_cast<int64_t>(Hkv) * d;
        const int64_t rows = paged ? page_size : Nk, outer = paged ? num_pages : B;
        if ((st = code_map(&mk, k, row, rows, outer, box)) != FA_OK ||
            (st = code_map(&mv, v, row, rows, outer, box)) != FA_OK)
            return st;
    }
    a.q = static_cast<const uint16_t*>(q);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.o = static_cast<uint16_t*>(o);
    a.lse = lse;
    a.meta = static_cast<int2*>(workspace);
    a.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.meta);
    a.o_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.meta + pl.lse);
    a.seqlens = seqlens;
    a.block_table = paged ? block_table : nullptr;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = g;
    a.Nq = Nq;
    a.R = g * Nq;
    a.cap = cap;
    a.per_seq = paged ? max_pages : static_cast<int>((Nk + 127LL) / 128);
    a.num_pages = num_pages;
    a.page_size = paged ? page_size : 128;
    a.page_box = box;
    a.HV = pl.HV;
    a.nch = pl.nch;
    a.RC = pl.RC;
    a.RT = pl.rt;
    a.heads = pl.heads;
    a.TS = pl.TS;
    a.HG = pl.HV / pl.TS;
    const long long group_tiles = tiles / pl.TS;
    a.teams = static_cast<int>(group_tiles < pl.teams ? (group_tiles > 0 ? group_tiles : 1) : pl.teams);
    a.scale_log2 = scale * kLog2e;
    const cudaStream_t s = cu(stream);
    if (dtype == FA_BF16) return launch_dec8<true>(pl.rows ? 0 : pl.rt, d, paged, mk, mv, a, causal, tiles > 0, s);
    return launch_dec8<false>(pl.rows ? 0 : pl.rt, d, paged, mk, mv, a, causal, tiles > 0, s);
}

}  // namespace

extern "C" {

fa_status fa_build_block_tables(const int* cache_seqlens, const int* new_lens, const int* free_pages,
                                int* block_table, int* slot_map, int* cu_new, int* new_seqlens, int* pages_used,
                                int B, int num_free, int num_pages, int page_size, int max_pages, int total_new,
                                fa_stream_t stream) {
    if (B < 1 || num_free < 0 || num_pages < 0 || page_size < 1 || max_pages < 1 || total_new < 0)
        return FA_ERR_INVALID_ARG;
    if (!new_lens || !block_table || !cu_new || !new_seqlens || !pages_used || (num_free > 0 && !free_pages) ||
        (total_new > 0 && !slot_map))
        return FA_ERR_INVALID_ARG;
    if (new_seqlens == cache_seqlens || new_seqlens == new_lens) return FA_ERR_INVALID_ARG;
    if (misaligned(cache_seqlens, 4) || misaligned(new_lens, 4) || misaligned(free_pages, 4) ||
        misaligned(block_table, 4) || misaligned(slot_map, 4) || misaligned(cu_new, 4) ||
        misaligned(new_seqlens, 4) || misaligned(pages_used, 4))
        return FA_ERR_MISALIGNED;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL ||
        static_cast<long long>(max_pages) * page_size > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;  // a slot is an int32
    if (total_new > 0x7fffffff - 2 * fa::kTableSlice) return FA_ERR_UNSUPPORTED;
    fa::TableArgs a{};
    a.seqlens = cache_seqlens;
    a.new_lens = new_lens;
    a.free_pages = free_pages;
    a.block_table = block_table;
    a.slot_map = slot_map;
    a.cu_new = cu_new;
    a.new_seqlens = new_seqlens;
    a.pages_used = pages_used;
    a.B = B;
    a.num_free = num_free;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.total_new = total_new;
    a.err = fa_host::error_word();
    if (!a.err) return FA_ERR_CUDA;
    const int grid = total_new > fa::kTableSlice ? (total_new + fa::kTableSlice - 1) / fa::kTableSlice : 1;
    fa::fa_block_tables_kernel<<<grid, fa::kTableThreads, 0, cu(stream)>>>(a);
    return launched();
}

fa_status fa_cache_append_paged(const void* k, const void* v, const long long* k_strides, const long long* v_strides,
                                void* k_pages, void* v_pages, const int* slot_map, int total_new, int Hkv,
                                int num_pages, int page_size, int d, fa_dtype dtype, fa_stream_t stream) {
    fa_status st = append_checks(k, v, k_pages, v_pages, total_new, Hkv, d, dtype);
    if (st != FA_OK) return st;
    if (num_pages < 1 || page_size < 1 || (total_new > 0 && !slot_map)) return FA_ERR_INVALID_ARG;
    if (misaligned(slot_map, 4)) return FA_ERR_MISALIGNED;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    fa::Append16Args a{};
    if ((st = row_strides(k_strides, Hkv, d, a.kst, a.ksh)) != FA_OK) return st;
    if ((st = row_strides(v_strides, Hkv, d, a.vst, a.vsh)) != FA_OK) return st;
    if (total_new == 0) return FA_OK;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.kp = static_cast<uint16_t*>(k_pages);
    a.vp = static_cast<uint16_t*>(v_pages);
    a.slot_map = slot_map;
    a.head_chunks = d / 8;
    a.row_chunks = Hkv * (d / 8);
    a.chunks = static_cast<long long>(total_new) * a.row_chunks;
    a.slots = num_pages * page_size;
    const long long want = (a.chunks + 255) / 256;
    const long long most = 16LL * fa_host::sm_count();
    if (most <= 0) return FA_ERR_CUDA;
    fa::fa_append16_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, cu(stream)>>>(a);
    return launched();
}

fa_status fa_cache_append_fp8(const void* k, const void* v, const long long* k_strides, const long long* v_strides,
                              void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int* cu_new,
                              const int* cache_seqlens, const int* new_seqlens, int B, int total_new, int max_new,
                              int Hkv, int Nk, int d, fa_dtype dtype, fa_stream_t stream) {
    if (Nk < 0) return FA_ERR_INVALID_ARG;
    return append8(k, v, k_strides, v_strides, k_cache, v_cache, k_scale, v_scale, cu_new, cache_seqlens, new_seqlens,
                   nullptr, false, B, total_new, max_new, Hkv, 0, 128, static_cast<int>((Nk + 127LL) / 128), Nk, d, dtype, stream);
}

fa_status fa_cache_append_paged_fp8(const void* k, const void* v, const long long* k_strides,
                                    const long long* v_strides, void* k_pages, void* v_pages, float* k_scale,
                                    float* v_scale, const int* cu_new, const int* cache_seqlens,
                                    const int* new_seqlens, const int* block_table, int B, int total_new,
                                    int max_new, int Hkv, int num_pages, int page_size, int max_pages, int d,
                                    fa_dtype dtype, fa_stream_t stream) {
    if (num_pages < 1 || page_size < 16 || max_pages < 1) return FA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
    if (static_cast<long long>(max_pages) * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    return append8(k, v, k_strides, v_strides, k_pages, v_pages, k_scale, v_scale, cu_new, cache_seqlens, new_seqlens,
                   block_table, true, B, total_new, max_new, Hkv, num_pages, page_size, max_pages,
                   max_pages * page_size, d, dtype, stream);
}

size_t fa_decode_fp8_workspace_size(int B, int Hq, int Hkv, int Nq, int d) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 0 || (d != 64 && d != 128)) return 0;
    if (static_cast<long long>(Hq / Hkv) * Nq > 128) return 0;
    Dec8Plan p;
    return dec8_plan(B, Hq, Hkv, Nq, d, p) ? p.total : 0;
}

fa_status fa_decode_fp8(const void* q, const void* k, const void* v, const float* k_scale, const float* v_scale,
                        void* o, float* lse, const int* cache_seqlens, void* workspace, int B, int Hq, int Hkv,
                        int Nq, int Nk, int d, float scale, int causal, fa_dtype dtype, fa_stream_t stream) {
    return decode8(q, k, v, k_scale, v_scale, o, lse, cache_seqlens, nullptr, workspace, B, Hq, Hkv, Nq, Nk, false, 0,
                   0, 0, d, scale, causal, dtype, stream);
}

fa_status fa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                              const float* v_scale, void* o, float* lse, const int* cache_seqlens,
                              const int* block_table, void* workspace, int B, int Hq, int Hkv, int Nq, int num_pages,
                              int page_size, int max_pages, int d, float scale, int causal, fa_dtype dtype,
                              fa_stream_t stream) {
    return decode8(q, k_pages, v_pages, k_scale, v_scale, o, lse, cache_seqlens, block_table, workspace, B, Hq, Hkv,
                   Nq, 0, true, num_pages, page_size, max_pages, d, scale, causal, dtype, stream);
}

}  // extern "C"
