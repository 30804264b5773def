// sv_paged.hpp -- what the paged-cache kernels share: the cache's geometry, the
// page lookup, and conversions between fp32 and the cache's element types.
//
// A cache is pages [num_pages][kv_heads][page_size][head_dim] for K and one
// such array for V: the rows of one head in one page are consecutive (4 KB for
// 16 slots of 128 bf16 values), so the attention of a (request, head) streams
// whole runs.  A page size is a power of two of at least 16, so 16 consecutive
// slots that start at a multiple of 16 lie in one page and a wave looks its
// pages up once per 16 slots, in scalar registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.hpp"

namespace sv {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two floats rounded to nearest even bf16, the first in the low half.
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
}
// Four floats rounded to nearest even e4m3, the first in the low byte.
__device__ __forceinline__ unsigned pack_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return static_cast<unsigned>(w);
}
// Two of a word's four e4m3 values as bf16 (exact), the first in the low half.
template <bool HI>
__device__ __forceinline__ unsigned e4m3_to_bf16(unsigned w) {
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Rows a request has in its window: counts[b] clipped to [0, N], or N.
__device__ __forceinline__ int window_rows(const int32_t *__restrict__ counts, int b, int N) {
    if (!counts) return N;
    const int c = counts[b];
    return c < 0 ? 0 : (c > N ? N : c);
}

}  // namespace sv
