// Device pieces of attention over the paged NVFP4 cache for gfx950: cached codes to f16 MFMA operands,
// query rows to f16, cross-lane reductions, and the work split that the kernels share.
//
// Arithmetic. level * E4M3(scale) has at most 2 + 4 significant bits and lies in 2^-10 .. 2688, so
// it is exact in f16: K and V enter the products as f16 without error and the global scales S_k and
// S_v multiply the logits and the outputs. E4M3 code c as f16 times 2^-8 is the bit pattern c << 7
// (same mantissa field, subnormals included); the up-conversion of the 4-bit codes supplies 2^8. A
// scale byte is masked to 7 bits, so no byte of the cache gives an infinity or NaN, and a weight of
// zero cancels whatever lies behind a sequence. A query row is scaled by a power of two that brings its
// largest value into [2^14, 2^15): bf16 values are then exact in f16 down to 2^-28 of the largest, and
// off by at most 2^-39 of it below; f32 values are split into two f16 halves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_formats.h"
#include "kv_cache.h"

namespace nvfp4 {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

union Half8 {
    half8v v;
    half2v p[4];
    uint32_t u[4];
};

__device__ __forceinline__ half2v as_half2(uint32_t u) { return __builtin_bit_cast(half2v, u); }

// The two values of byte SEL of w, times 2^8 and a pair of scales that carry 2^-8.
template <int SEL>
__device__ __forceinline__ half2v dequant2(uint32_t w, half2v scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, SEL) * scale;
}

// Scale byte B of `bytes` (masked), twice; and the pair of bytes (0, 1) or (2, 3): f16 times 2^-8.
template <int B>
__device__ __forceinline__ half2v scale_twice(uint32_t bytes) {
    constexpr uint32_t sel = 0x0C000C00u | (uint32_t)B | ((uint32_t)B << 16);
    return as_half2(__builtin_amdgcn_perm(0u, bytes, sel) << 7);
}
template <int HIGH>
__device__ __forceinline__ half2v scale_pair(uint32_t bytes) {
    constexpr uint32_t sel = HIGH ? 0x0C030C02u : 0x0C010C00u;
    return as_half2(__builtin_amdgcn_perm(0u, bytes, sel) << 7);
}

// (bits of a where the mask is set) | (bits of b elsewhere)
__device__ __forceinline__ uint32_t select_bits(uint32_t mask, uint32_t a, uint32_t b) {
    return (a & mask) | (b & ~mask);
}

// Maximum (sum) over the four 16-lane groups of a wave, in every lane.
__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// Exponent k that brings a row's largest |value| into [2^14, 2^15), at most 126.
__device__ __forceinline__ int row_exponent(float top) {
    if (!(top > 0.0f)) return 0;
    return min(15 - __builtin_amdgcn_frexp_expf(top), 126);
}

// One rounding to bf16, to nearest even, of finite values.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const auto r = [](float v) {
        const uint32_t u = __float_as_uint(v);
        return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    };
    return r(a) | (r(b) << 16);
}

// Work split: the (item, head) pairs' query rows in tiles, the visible positions of a tile in chunks.
// Rows of an item and head: (token j, query head of the group), row = j * group + head.
struct KvPlan {
    int32_t tile_rows;       // query rows of a workgroup
    int32_t tiles;           // row tiles of the largest item
    int32_t splits;          // chunks of the largest span
    int32_t chunk;           // positions of a chunk, a multiple of 32
    uint64_t page_magic;     // division of a 16-token unit by the units of a page
    uint32_t page_shift;
};

// What one tile of an item sees: positions begin .. end - 1 (begin a multiple of 32).
struct KvRange {
    int32_t begin, end;
};

__device__ __forceinline__ KvRange tile_range(const KvAttention& a, int len, int rows_new, int group,
                                              int row0, int rows) {
    KvRange r;
    r.begin = 0;
    r.end = min(len, a.max_kv);
    const int first = len - rows_new + row0 / group;
    if (a.causal) r.end = min(r.end, len - rows_new + (row0 + rows - 1) / group + 1);
    if (a.window > 0) r.begin = max(0, first - a.window + 1) & ~31;
    r.end = max(r.end, r.begin);
    return r;
}

}  // namespace nvfp4
