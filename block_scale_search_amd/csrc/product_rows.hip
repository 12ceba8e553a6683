// Products of few rows with NVFP4 matrices for gfx950, forward and gated: a token's or a small batch's pass,
// bound by reading the codes.
//
// A wave owns a slice of the reduction, 1024 columns, and keeps the rows' values of that slice in registers, as operands
// of MFMA 16x16x32; the codes stream past. The 16 lanes that give the MFMA 16 rows of its left operand
// hold 4 rows of the matrix by 4 pieces of the slice, the right operand's 16 columns 4 rows of X by the same 4
// pieces: of the 16 x 16 sums the quarter where the pieces are the same is wanted. What that wastes of the matrix units
// is idle here anyway, and it lets four neighbouring lanes read neighbouring bytes of a row (16 rows side by
// side, a lane each, took 1.5 to 2 times as long: the loads' addresses were the bound). A lane converts 64
// codes of 4 groups a step. The slices' sums meet in LDS, in a fixed order.
//
// Operands. bf16 rows enter as f16 ones, a row's slice times a power of two, since f16 weights (level * E4M3 is exact in
// them too) take half the instructions of bf16 ones: 2 to 8% of the whole. f16 holds a value's bits down to 2^-31
// of the largest of its slice; a wave that meets values below that, or an infinity or a NaN, takes that slice as bf16
// instead (looking costs 1 to 2% of 4096 x 14336, nothing of larger ones). So do the parts of f32 rows enter.
//
// Measured: gate and up of 2 x 28672 x 8192, one row, 52.3 us = 5.0 TB/s, a large copy's rate; 8192 x 28672 29 us (4.6);
// 4096 x 14336, 256 workgroups of 14 waves, 11.4 us (2.9), bound by launch and first codes.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int kSlice = 1024;
constexpr int kRows = 4;             // rows of X of a workgroup
template <bool F32>
constexpr int kWaves = F32 ? 8 : 16; // at most (registers)
constexpr int kDepth = 4;            // groups of 4 matrix rows in flight

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

template <bool HALF>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (!HALF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a), __builtin_bit_cast(half8v, b),
                                                      c, 0, 0, 0);
}

// Scale byte B (masked) times 2^-8 as f16, twice: E4M3's fields are f16's upper ones.
template <int B>
__device__ __forceinline__ half2v scale_half(uint32_t bytes) {
    return __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0u, bytes, 0x0C000C00u | B | B << 16) << 7);
}
// Eight codes times their scale (as scale_half gives it) as f16, exact.
__device__ __forceinline__ u32x4 dequant8_half(uint32_t w, half2v scale) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 0) * scale),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 1) * scale),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 2) * scale),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, 3) * scale)};
}

// Makes bf16 values f16 ones times 2^k, the largest magnitude of the row's slice (that of the 16 lanes with the same
// n4) coming to 2^14 .. 2^15; k to `raised`. Where a value of the wave would lose bits (f16's last bit is 2^-24, a bf16
// value has eight) or is no number, false, and all stay as they are.
__device__ __forceinline__ bool to_half(u32x4 (&x)[8], int& raised) {
    ushort2v most = {0, 0}, least = {0xFFFF, 0xFFFF};
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const ushort2v a = __builtin_bit_cast(ushort2v, x[s][j] & 0x7FFF7FFFu);
            most = __builtin_elementwise_max(most, a);
            least = __builtin_elementwise_min(least, a);
        }
    int m = max((int)most[0], (int)most[1]);
    m = max(m, __builtin_amdgcn_update_dpp(0, m, 0xB1, 0xF, 0xF, true));
    m = max(m, __builtin_amdgcn_update_dpp(0, m, 0x4E, 0xF, 0xF, true));
    m = max(m, __shfl_xor(m, 16, 64));
    m = max(m, __shfl_xor(m, 32, 64));
    const int e = m >> 7;
    int low = min((int)least[0], (int)least[1]) >> 7;
    if (__ballot(low < e - 31)) {                        // zeros, most often: the least of the others
        least = ushort2v{0xFFFF, 0xFFFF};
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                least = __builtin_elementwise_min(
                    least, (ushort2v)(__builtin_bit_cast(ushort2v, x[s][j] & 0x7FFF7FFFu) - (ushort2v){1, 1}));
        low = (min((int)least[0], (int)least[1]) + 1) >> 7;
    }
    raised = 141 - max(e, 1);
    if (__ballot(e == 255 || low < e - 31)) return false;
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[s][j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(__builtin_amdgcn_ldexpf(bf16_lo(x[s][j]), raised),
                                                                              __builtin_amdgcn_ldexpf(bf16_hi(x[s][j]), raised)));
    return true;
}

// Sum over four neighbouring lanes, in each of them.
__device__ __forceinline__ float sum_quad(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));
}

// A lane's 64 codes of a group of 4 matrix rows, and their scale bytes.
struct Codes {
    u32x4 code[2];
    uint32_t scale;
};

// Up to kRows rows of X, `block` rows of each matrix (a multiple of 16). WHOLE: in is a multiple of 64, so a lane's 64
// columns are all inside the matrix or all outside.
template <bool GATED, bool F32, bool WHOLE>
__global__ __launch_bounds__(64 * kWaves<F32>) void k_product_rows(Product p, int nn, int block) {
    constexpr int P = F32 ? 3 : 1;                       // parts of a value
    extern __shared__ float sums[];                      // [wave][group][64]
    const int lane = threadIdx.x & 63, seg = lane & 3, n4 = lane >> 2 & 3, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int tile = (int)(blockIdx.x / (uint32_t)nn), tn = (int)(blockIdx.x - (uint32_t)tile * (uint32_t)nn);
    RowTile rows;
    if (!find_rows(p.rows, tile, kRows, rows)) return;
    const int n0 = tn * block, N = (int)p.out, K = (int)p.in;
    const int slices = (K + kSlice - 1) / kSlice;
    const int half = block / 4, groups = GATED ? 2 * half : half;

    __amdgpu_buffer_rsrc_t codes[GATED ? 2 : 1], scales[GATED ? 2 : 1];
#pragma unroll
    for (int m = 0; m < (GATED ? 2 : 1); ++m) {
        const int64_t at = rows.e * p.w[m].stride + (int64_t)n0 * K;
        codes[m] = window(p.w[m].packed + at / 2);
        scales[m] = window(p.w[m].scales + at / 16);
    }

    for (int slice = wave; slice < slices; slice += waves) {
        const int k = slice * kSlice + kg * 256 + seg * 64;          // the lane's 64 columns
        // its values of row n4
        u32x4 x[P][8];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const __amdgpu_buffer_rsrc_t from = window(p.a[0].p + i * p.plane + rows.first * p.a[0].ld);
            const uint32_t at = (uint32_t)(n4 * p.a[0].ld + k) * 2;
#pragma unroll
            for (int s = 0; s < 8; ++s) x[i][s] = load16(from, n4 < rows.rows && k + 8 * s < K ? at + 16 * s : kNowhere);
        }
        const uint32_t first = (uint32_t)n4 * (uint32_t)(K / 16) + (uint32_t)(k / 16);   // in groups of 16 weights
        const auto load = [&](Codes& b, int g) {
            const int j = GATED && g >= half ? g - half : g;
            const bool second = GATED && g >= half;
            const uint32_t at = first + (uint32_t)j * 4u * (uint32_t)(K / 16);
            const bool live = n0 + 4 * j + n4 < N && g < groups;
            const __amdgpu_buffer_rsrc_t c = GATED && second ? codes[GATED ? 1 : 0] : codes[0];
            const __amdgpu_buffer_rsrc_t e = GATED && second ? scales[GATED ? 1 : 0] : scales[0];
            if constexpr (WHOLE) {
                const bool in = live && k < K;
                b.code[0] = load16(c, in ? at * 8 : kNowhere);
                b.code[1] = load16(c, in ? at * 8 + 16 : kNowhere);
                b.scale = load4(e, in ? at : kNowhere);
            } else {
                u32x2 w[4];
                b.scale = 0;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const bool in = live && k + 16 * s < K;
                    w[s] = load8(c, in ? at * 8 + 8 * s : kNowhere);
                    b.scale |= load1(e, in ? at + s : kNowhere) << (8 * s);
                }
                b.code[0] = u32x4{w[0][0], w[0][1], w[1][0], w[1][1]};
                b.code[1] = u32x4{w[2][0], w[2][1], w[3][0], w[3][1]};
            }
        };
        constexpr int kFirst = F32 ? kDepth : kDepth / 2;            // under way while the operands are made
        Codes buf[kDepth];
#pragma unroll
        for (int d = 0; d < kFirst; ++d) {
            load(buf[d], d);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the slice's sums of all the workgroup's matrix rows; bf16 operands of a bf16 row, a rare case, with half as many codes
        // in flight (registers)
        const auto multiply_all = [&](auto half_operands, int raised) {
            constexpr bool HALF = decltype(half_operands)::value;
            constexpr int kAhead = HALF || F32 ? kDepth : kFirst;
#pragma unroll
            for (int d = kFirst; d < kAhead; ++d) {
                load(buf[d], d);
                __builtin_amdgcn_sched_barrier(0);
            }
            for (int g0 = 0; g0 < groups; g0 += kAhead) {
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    Codes& b = buf[d];
                    f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
                    const auto multiply = [&](const auto (&e)[4]) {
#pragma unroll
                        for (int s = 0; s < 8; ++s) {
                            u32x4 w;
                            if constexpr (HALF) w = dequant8_half(b.code[s >> 2][s & 3], e[s >> 1]);
                            else w = dequant8(b.code[s >> 2][s & 3], e[s >> 1]);
#pragma unroll
                            for (int i = 0; i < P; ++i) acc[s & 1] = mfma<HALF>(w, x[i][s], acc[s & 1]);
                        }
                    };
                    if constexpr (!HALF) {
                        const float e[4] = {scale_value<0>(b.scale), scale_value<1>(b.scale), scale_value<2>(b.scale),
                                            scale_value<3>(b.scale)};
                        multiply(e);
                    } else {
                        const uint32_t bytes = b.scale & 0x7F7F7F7Fu;
                        const half2v e[4] = {scale_half<0>(bytes), scale_half<1>(bytes), scale_half<2>(bytes),
                                             scale_half<3>(bytes)};
                        multiply(e);
                    }
                    load(b, g0 + d + kAhead);
                    // register r of a lane holds piece r of matrix row kg; the lane's own piece is seg
                    const f32x4 a = acc[0] + acc[1];
                    float v = sum_quad(seg < 2 ? (seg == 0 ? a[0] : a[1]) : (seg == 2 ? a[2] : a[3]));
                    if constexpr (HALF) v = __builtin_amdgcn_ldexpf(v, -raised);
                    float* to = sums + (wave * groups + g0 + d) * 64 + lane;
                    *to = slice == wave ? v : *to + v;
                    __builtin_amdgcn_sched_barrier(0);       // else all loads are issued together, and waited for together
                }
            }
        };
        int raised = 0;
        if constexpr (F32) multiply_all(std::false_type{}, 0);
        else if (to_half(x[0], raised)) multiply_all(std::true_type{}, raised);
        else multiply_all(std::false_type{}, 0);
    }
    __syncthreads();

    const int used = min(waves, slices);
    const float S0 = p.w[0].S[rows.e], S1 = GATED ? p.w[1].S[rows.e] : 0.0f;
    const auto total = [&](int g, int at) {
        float s = 0.0f;
        for (int w = 0; w < used; ++w) s += sums[(w * groups + g) * 64 + at];
        return s;
    };
    for (int o = threadIdx.x; o < block * rows.rows; o += blockDim.x) {
        const int row = o / block, c = o - row * block;
        const int64_t n = n0 + c, t = rows.first + row;
        if (n >= N) continue;
        const int g = c >> 2, at = (c & 3) * 16 + row * 4;
        if constexpr (GATED) {
            const float gate = total(g, at) * S0, up = total(g + half, at) * S1;
            product_gated(p, t, n, gate, up, F32);
        } else {
            const float bias = p.bias ? load_value(p.bias, rows.e * (int64_t)N + n, F32) : 0.0f;
            product_linear(p, t, n, __builtin_fmaf(total(g, at), S0, bias), F32);
        }
    }
}

template <bool GATED, bool F32>
void launch(const Product& p, hipStream_t stream) {
    const int64_t slices = (p.in + kSlice - 1) / kSlice;
    const int waves = (int)(slices < kWaves<F32> ? slices : kWaves<F32>);
    // As many matrix rows a workgroup, 16 to 128, as leave each compute unit the waves of one full workgroup, gated two:
    // fewer start and end (one row, 8192 x 28672: 32 rows 30 us, 16 35.5, 64 no better than 32; 4096 x 14336: 16 rows 11.2,
    // 32 15.9; rows of 128 gated experts 2 x 768 x 2048: 64 rows 65 us, 16 72; of 64 of 4096 x 1024: 128 rows 41.5, 16
    // and 32 46; gated with one: 1 x 2 x 28672 x 8192 64 rows 56 us, 32 and 16 52.7)
    const int64_t tiles = product_row_tiles(p.rows.tokens, p.rows.batch, kRows);
    int block = 16;
    while (block < 128 && waves * 2 * block * (GATED ? 2 : 1) <= 1024 &&
           tiles * ((p.out + 2 * block - 1) / (2 * block)) * waves >= (GATED ? 512 : 256) * kWaves<F32>)
        block *= 2;
    const int64_t nn = (p.out + block - 1) / block;
    const dim3 grid((uint32_t)(tiles * nn)), threads(64 * waves);
    const size_t lds = (size_t)waves * (GATED ? 2 : 1) * block * 64;
    if (p.in % 64 == 0)
        hipLaunchKernelGGL((k_product_rows<GATED, F32, true>), grid, threads, lds, stream, p, (int)nn, block);
    else
        hipLaunchKernelGGL((k_product_rows<GATED, F32, false>), grid, threads, lds, stream, p, (int)nn, block);
}

}  // namespace

void launch_product_rows(const Product& p, hipStream_t stream) {
    if (p.matrices == 2) {
        if (p.f32) launch<true, true>(p, stream);
        else launch<true, false>(p, stream);
    } else {
        if (p.f32) launch<false, true>(p, stream);
        else launch<false, false>(p, stream);
    }
}

}  // namespace nvfp4
