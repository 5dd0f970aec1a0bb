// fa_host.h: host-side services of the library shared between its sources (defined in
// fa_api.cu): the current device's error word and SM count, and tensor maps.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fa.h"

namespace fa {
// Device error word (beside the codes of sm100.cuh): a serving call met lengths, pages or
// free pages that do not fit its cache; it left those tokens out.
enum : int { kErrCacheRange = 0x4000 };
}  // namespace fa

namespace fa_host {

int* error_word();     // device address of the current device's error word (null: lookup failed)
int sm_count();        // SMs of the current device (0: query failed)
int current_device();  // index of the current device (-1: query failed)

// Tensor map of a [batches, rows, H, d] tensor, box = box_rows rows x box_h heads x 128 bytes
// of columns, 128-byte swizzle (cached per host thread).
fa_status make_map_box(CUtensorMap* m, const void* base, int d, int H, int64_t rows, int64_t batches, bool bf16,
                       int64_t sh, int64_t ss, int64_t sb, int box_h, int box_rows, bool promote_256,
                       int elem_bytes);

}  // namespace fa_host
