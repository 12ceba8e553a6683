// Device pieces of the products with NVFP4 matrices for gfx950: codes to bf16 MFMA operands, activations
// and their slopes, and the search for a workgroup's rows.
//
// Arithmetic. level * E4M3(scale) has at most 2 + 4 significant bits and lies in 2^-10 .. 2880, so it is
// exact in bf16, and its product with a bf16 value is exact in binary32: the MFMA's sums are the only
// roundings before the global scale S, which multiplies the sum. A scale byte is masked to 7 bits; the
// codes of groups past the matrix's edge are multiplied by a scale of zero. f16 operands take half the
// instructions, but bf16 rows fit f16's range only after a scaling: the kernel for few rows, which has a row's values in
// registers, does that by itself; the others would need a pass over the rows before them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_formats.h"
#include "kv_cache.h"
#include "product.h"

namespace nvfp4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Rows of codes start at multiples of 8 bytes, rows of scale bytes anywhere.
typedef u32x4 u32x4_at8 __attribute__((aligned(8)));
typedef u32x2 u32x2_at8 __attribute__((aligned(8)));
typedef uint16_t u16_at1 __attribute__((aligned(1)));

enum ProductAct { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4 };

// Scale byte B of `bytes` as binary32.
template <int B>
__device__ __forceinline__ float scale_value(uint32_t bytes) {
    return __builtin_amdgcn_cvt_f32_fp8(bytes & 0x7F7F7F7Fu, B);
}

// Values of the two codes in byte B of w.
template <int B>
__device__ __forceinline__ void code_values(uint32_t w, float scale, float& x, float& y) {
    const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
    x = v[0] * scale;
    y = v[1] * scale;
}

// Eight codes times their scale as bf16, exact.
__device__ __forceinline__ u32x4 dequant8(uint32_t w, float scale) {
    float x[8];
    code_values<0>(w, scale, x[0], x[1]);
    code_values<1>(w, scale, x[2], x[3]);
    code_values<2>(w, scale, x[4], x[5]);
    code_values<3>(w, scale, x[6], x[7]);
    return u32x4{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
}

// act(z). bf16 outputs use the hardware's exponential and reciprocal (a few binary32 steps off, far
// below 2^-9); binary32 ones the library's functions and IEEE division.
template <bool F32>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (F32) return 1.0f / (1.0f + expf(-z));
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
// 0.5 (1 + tanh v) is sigmoid(2 v), v = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh_arg(float z) {
    return 1.5957691216057308f * z * __builtin_fmaf(0.044715f * z, z, 1.0f);
}

template <bool F32>
__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case kActSilu: return z * sigmoid<F32>(z);
        case kActGelu: return 0.5f * z * erfcf(-0.7071067811865476f * z);
        case kActGeluTanh: return z * sigmoid<F32>(gelu_tanh_arg(z));
        case kActRelu: return z > 0.0f ? z : (z == z ? 0.0f : z);
        default: return z;
    }
}

// act(z) and act'(z).
template <bool F32>
__device__ __forceinline__ void act_slope(int act, float z, float& a, float& slope) {
    switch (act) {
        case kActSilu: {
            const float p = sigmoid<F32>(z);
            a = z * p;
            slope = __builtin_fmaf(a, 1.0f - p, p);
            return;
        }
        case kActGelu: {
            const float cdf = 0.5f * erfcf(-0.7071067811865476f * z);
            a = z * cdf;
            slope = __builtin_fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), cdf);
            return;
        }
        case kActGeluTanh: {
            const float p = sigmoid<F32>(gelu_tanh_arg(z));
            const float c = fminf(fmaxf(z, -32.0f), 32.0f);     // beyond, p is 0 or 1 and z^3 may overflow
            a = z * p;
            slope = __builtin_fmaf(c * p * (1.0f - p), 1.5957691216057308f * __builtin_fmaf(0.134145f * c, c, 1.0f), p);
            return;
        }
        case kActRelu:
            a = act_value<F32>(act, z);
            slope = z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
            return;
        default:
            a = z;
            slope = 1.0f;
    }
}

__device__ __forceinline__ float load_value(const void* p, int64_t i, bool f32) {
    if (f32) return static_cast<const float*>(p)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ uint16_t bf16_bits(float x) { return (uint16_t)bf16_pair(x, 0.0f); }
__device__ __forceinline__ void store_value(void* p, int64_t i, float x, bool f32) {
    if (f32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = bf16_bits(x);
}

// The value that a product's columns make: z of a linear layer, g and u of a gated pair.
__device__ __forceinline__ void product_linear(const Product& p, int64_t t, int64_t n, float z, bool f32) {
    if (p.pre[0]) store_value(p.pre[0], t * p.ldpre[0] + n, z, f32);
    float y = f32 ? act_value<true>(p.act, z) : act_value<false>(p.act, z);
    if (p.residual) y += load_value(p.residual, t * p.ldr + n, f32);
    store_value(p.y, t * p.ldy + n, y, f32);
}
__device__ __forceinline__ void product_gated(const Product& p, int64_t t, int64_t n, float g, float u, bool f32) {
    if (p.pre[0]) {
        store_value(p.pre[0], t * p.ldpre[0] + n, g, f32);
        store_value(p.pre[1], t * p.ldpre[1] + n, u, f32);
    }
    store_value(p.y, t * p.ldy + n, (f32 ? act_value<true>(p.act, g) : act_value<false>(p.act, g)) * u, f32);
}

// Columns of a product's partial sums: whole pieces of 8 (a gated pair's u behind its g).
__device__ __forceinline__ int64_t partial_cols(int64_t N) { return (N + 7) & ~(int64_t)7; }

// Values c .. c + 7 of a row, zeros from `cols`; `wide`: rows are laid out for 16-byte accesses.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t row, int64_t c, int64_t cols, bool wide, float (&x)[8]) {
    if (wide && c + 8 <= cols) {
        if constexpr (F32) {
            const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + c);
            const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + c + 4);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + row + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = bf16_lo(a[k]);
                x[2 * k + 1] = bf16_hi(a[k]);
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = c + k < cols ? load_value(p, row + c + k, F32) : 0.0f;
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t row, int64_t c, int64_t cols, bool wide, const float (&x)[8]) {
    if (wide && c + 8 <= cols) {
        if constexpr (F32) {
            float* to = static_cast<float*>(p) + row + c;
            *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + row + c) =
                u32x4{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < cols) store_value(p, row + c + k, x[k], F32);
}

// Columns n .. n + 7 (a multiple of 8) of row t, which is matrix e's: a share's sums (of several) to the workspace,
// else what the product makes of them. v: sums times S; gated, u: the second matrix's.
template <bool GATED, bool F32>
__device__ __forceinline__ void product_out8(const Product& p, int splits, int split, int64_t e, int64_t t, int64_t n,
                                             int64_t N, float (&v)[8], float (&u)[8]) {
    if (splits > 1) {
        const int64_t cols = partial_cols(N);
        float* to = p.partial + ((int64_t)split * p.rows.tokens + t) * (GATED ? 2 * cols : cols) + n;
        reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
        if constexpr (GATED) {
            reinterpret_cast<float4*>(to + cols)[0] = make_float4(u[0], u[1], u[2], u[3]);
            reinterpret_cast<float4*>(to + cols)[1] = make_float4(u[4], u[5], u[6], u[7]);
        }
        return;
    }
    if constexpr (GATED) {
        if (p.pre[0]) {
            store8<F32>(p.pre[0], t * p.ldpre[0], n, N, p.wide, v);
            store8<F32>(p.pre[1], t * p.ldpre[1], n, N, p.wide, u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act_value<F32>(p.act, v[k]) * u[k];
    } else if (!p.backward) {
        if (p.bias) {
            float b[8];
            load8<F32>(p.bias, e * N, n, N, p.wide, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += b[k];
        }
        if (p.pre[0]) store8<F32>(p.pre[0], t * p.ldpre[0], n, N, p.wide, v);
        if (p.act != kActNone) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = act_value<F32>(p.act, v[k]);
        }
        if (p.residual) {
            float r[8];
            load8<F32>(p.residual, t * p.ldr, n, N, p.wide, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += r[k];
        }
    }
    store8<F32>(p.y, t * p.ldy, n, N, p.wide, v);
}

typedef __attribute__((address_space(1))) const void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;

// 16 (4) bytes a lane from global memory to lds + 16 (4) * lane (lds uniform).
__device__ __forceinline__ void copy16(const void* src, void* lds) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)lds, 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void* src, void* lds) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)lds, 4, 0, 0);
}

// Loads through a buffer descriptor over `bytes` from p, from a lane's offset plus a uniform one: an offset of
// kNowhere reads zeros.
constexpr uint32_t kReach = 0x80000000u, kNowhere = 0xC0000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* p, uint32_t bytes = kReach) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
// `at` where in, else kNowhere; by a select (the compiler would make two loads and a branch of it).
__device__ __forceinline__ uint32_t offset_if(bool in, uint32_t at) {
    uint32_t v = in ? at : kNowhere;
    asm("" : "+v"(v));
    return v;
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t plus = 0) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, plus, 0));
}
__device__ __forceinline__ u32x2 load8(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t plus = 0) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at, plus, 0));
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t plus = 0) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, at, plus, 0);
}
__device__ __forceinline__ uint32_t load2(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t plus = 0) {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, plus, 0);
}
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t plus = 0) {
    return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, at, plus, 0);
}

// copy16, from a uniform address plus a lane's offset, that the compiler does not see as one: it would wait for all
// copies under way before the next write to LDS, whichever part of it they are for. The caller waits, by wait_copies.
__device__ __forceinline__ void copy16_unseen(const void* src, uint32_t at, void* lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(at), "s"(src), "s"((uint32_t)(uintptr_t)(LdsPtr)lds)
                 : "memory", "m0");
}

// Waits until at most N of the wave's loads and copies are under way, and for its LDS accesses.
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
}
// The bare barrier: the waits that it needs are explicit (__syncthreads would wait for every copy under way).
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

// Rows of matrix e, inside the tokens whatever the offsets hold.
__device__ __forceinline__ void segment(const ProductRows& r, int e, int64_t& lo, int64_t& hi) {
    lo = min(max(r.seg[e], (int64_t)0), r.tokens);
    hi = min(max(r.seg[e + 1], lo), r.tokens);
}

// First row that belongs to no matrix.
__device__ __forceinline__ int64_t rows_end(const ProductRows& r) {
    return r.seg ? min(max(r.seg[r.batch], (int64_t)0), r.tokens) : r.tokens;
}

// v of the lane whose number differs in bit 1.
__device__ __forceinline__ uint32_t swap_pairs(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);
}

// A value that is the same in every lane, for the compiler to keep it in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
                     ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32));
}

// A workgroup's rows: tile `tile` of the matrices' rows in tiles of `size`, numbered matrix by matrix; false past the
// last. Uniform. A few matrices each wave searches by itself, 64 at a time; for many there is a map.
__device__ __forceinline__ bool find_rows(const ProductRows& r, int tile, int size, RowTile& t) {
    t = RowTile{0, 0, 0};
    if (r.batch <= 1) {
        int64_t lo = 0, hi = r.tokens;
        if (r.seg) segment(r, 0, lo, hi);
        t.first = lo + (int64_t)tile * size;
        t.rows = (int32_t)min(max(hi - t.first, (int64_t)0), (int64_t)size);
    } else if (r.batch > kMapped) {
        t = r.map[tile];
    } else {
        const int lane = threadIdx.x & 63;
        int before = 0;
        for (int base = 0; base < r.batch; base += 64) {
            int64_t lo = 0, hi = 0;
            if (base + lane < r.batch) segment(r, base + lane, lo, hi);
            const int n = (int)((hi - lo + size - 1) / size);
            int upto = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_up(upto, d, 64);
                if (lane >= d) upto += v;
            }
            const uint64_t in = __ballot(before + upto > tile);
            if (in) {
                const int at = __builtin_ctzll(in);
                const int k = tile - before - (upto - n);            // of the matrix's own tiles
                const int64_t first = lo + (int64_t)k * size;
                t.e = base + at;
                t.rows = __builtin_amdgcn_readlane(k >= 0 && k < n ? (int)min((int64_t)size, hi - first) : 0, at);
                t.first = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)first, at) |
                                    ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(first >> 32), at) << 32));
                break;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
        }
    }
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.first = uniform(t.first);
    return t.rows > 0;
}

}  // namespace nvfp4
