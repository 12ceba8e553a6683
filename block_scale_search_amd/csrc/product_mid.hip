// Products of some tens of rows with NVFP4 matrices for gfx950, forward and gated: a serving batch's pass.
//
// A workgroup owns BM rows and 128 rows of the matrix, 32 a wave, over a share of the reduction, in steps of 128. A
// step's values of X, codes and scale bytes go from global memory straight into LDS, kStages - 1 steps ahead. A
// wave converts the codes of its own matrix rows in registers (level * E4M3 is exact in bf16): they are the operands
// of MFMA 32x32x16 as they lie, 32 codes a lane, the reduction being taken in that order on both sides; so
// the converted weights never pass through LDS. Gated: a wave's 32 matrix rows are 16 of the gate and the same 16 of
// the other matrix, and the two meet by a lane exchange.
//
// Bound by the conversion first (16 instructions for 8 weights: vector units 57 to 77% busy, matrix units 33%), then by
// LDS and copies. 64 rows by 8192 x 28672 49 us (2.8 TB/s) and 5 for the shares' sums; 16384 rows of 128 experts
// 2048 x 768 99 us. Two stages: with three, tiles of 64 rows are no faster and fewer workgroups fit a compute unit.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int kStep = 128, kWaves = 4, kThreads = 64 * kWaves, kCols = 32 * kWaves;

template <int BM>
struct Stage {
    uint16_t a[BM][kStep];
    uint8_t code[kCols][kStep / 2];
    uint8_t scale[kCols][kStep / 16];
};

// 16-byte pieces of a row are permuted by the row, so that 8 lanes that read a piece of 8 rows use all banks.
__device__ __forceinline__ int a_piece(int row, int c) { return c ^ (row & 15); }
__device__ __forceinline__ int code_piece(int row, int c) { return c ^ (row >> 1 & 3); }

template <int BM, int STAGES, bool GATED>
__global__ __launch_bounds__(kThreads) void k_product_mid(Product p, int nn, int splits, int each) {
    constexpr int TM = BM / 32;
    __shared__ __align__(1024) Stage<BM> stage[STAGES];
    const int lane = threadIdx.x & 63, n32 = lane & 31, kg = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t of = blockIdx.x / (uint32_t)splits;
    const int split = (int)(blockIdx.x - of * (uint32_t)splits);
    const int tile = (int)(of / (uint32_t)nn), tn = (int)(of - (uint32_t)tile * (uint32_t)nn);
    RowTile rows;
    if (!find_rows(p.rows, tile, BM, rows)) return;
    constexpr int kOut = GATED ? kCols / 2 : kCols;
    const int n0 = tn * kOut, N = (int)p.out, K = (int)p.in;
    const int first = split * each, last = min(first + each, (K + kStep - 1) / kStep);

    // copies of a step: X, 16 lanes a row; codes and scale bytes of the wave's own matrix rows, 4 and 2 lanes a row
    const auto matrix_row = [&](int r) -> int64_t {      // r: 0 .. 31 of the wave
        const int c = GATED ? wave * 16 + (r & 15) : wave * 32 + r;
        return min(n0 + c, N - 1);
    };
    constexpr int kLoads = BM * (kStep / 8) / kThreads;
    const uint16_t* xs[kLoads];
    int xk[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = (i * kThreads + (int)threadIdx.x) >> 4;
        xk[i] = a_piece(row, threadIdx.x & 15) * 8;
        xs[i] = p.a[0].p + (rows.first + min(row, rows.rows - 1)) * p.a[0].ld;
    }
    const uint8_t* cs[2];
    int ck[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 16 * i + (lane >> 2);
        const ProductMatrix& w = p.w[GATED && r >= 16 ? 1 : 0];
        ck[i] = code_piece(r, lane & 3) * 32;
        cs[i] = w.packed + (rows.e * w.stride + matrix_row(r) * K) / 2;
    }
    const ProductMatrix& ws = p.w[GATED && lane >= 32 ? 1 : 0];
    const uint8_t* ss = ws.scales + (rows.e * ws.stride + matrix_row(lane >> 1) * K) / 16;
    const int sk = (lane & 1) * 64;
    const auto copy = [&](Stage<BM>& st, int s) {
        // pieces past the edge come from the rows' first columns: they meet weights of zero
        const int k0 = s * kStep;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int k = k0 + xk[i];
            copy16(xs[i] + (k < K ? k : 0), &st.a[(i * kThreads + 64 * wave) >> 4][0]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = k0 + ck[i];
            copy16(cs[i] + (k < K ? k : 0) / 2, &st.code[32 * wave + 16 * i][0]);
        }
        const int k = k0 + sk;
        copy4(ss + (k < K ? k : 0) / 16, &st.scale[32 * wave][0]);
    };

    f32x16 acc[TM];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (first + s < last) copy(stage[s], first + s);
    int at = 0;
    for (int s = first; s < last; ++s) {
        // the copies of step s are done; those of the steps after it may be under way
        if (STAGES >= 4 && s + 2 < last) wait_copies<2 * (kLoads + 3)>();
        else if (STAGES >= 3 && s + 1 < last) wait_copies<kLoads + 3>();
        else wait_copies<0>();
        barrier();
        const Stage<BM>& st = stage[at];
        if (s + STAGES - 1 < last) copy(stage[at == 0 ? STAGES - 1 : at - 1], s + STAGES - 1);
        at = at + 1 == STAGES ? 0 : at + 1;
        // 8 slices of 16: half h's codes are 64 h + 32 kg .. + 31. Operands are read kAhead slices before their use.
        constexpr int kAhead = 4;
        const int row = 32 * wave + n32, left = K - s * kStep;
        u32x4 code[2];
        uint32_t sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            code[h] = *reinterpret_cast<const u32x4*>(&st.code[row][code_piece(n32, 2 * h + kg) * 16]);
            sc[h] = *reinterpret_cast<const uint16_t*>(&st.scale[row][4 * h + 2 * kg]);
        }
        bf16x8 x[8][TM];
        const auto read = [&](int z) {
#pragma unroll
            for (int a = 0; a < TM; ++a) {
                const int r = 32 * a + n32;
                x[z][a] = *reinterpret_cast<const bf16x8*>(&st.a[r][a_piece(r, 8 * (z >> 2) + 4 * kg + (z & 3)) * 8]);
            }
        };
#pragma unroll
        for (int z = 0; z < kAhead; ++z) read(z);
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[h] = 64 * h + 32 * kg < left ? sc[h] : 0;
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            const float e = (z & 2) ? scale_value<1>(sc[z >> 2]) : scale_value<0>(sc[z >> 2]);
            const u32x4 w = dequant8(code[z >> 2][z & 3], e);
            if (z + kAhead < 8) read(z + kAhead);
#pragma unroll
            for (int a = 0; a < TM; ++a)
                acc[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[z][a], __builtin_bit_cast(bf16x8, w), acc[a], 0, 0, 0);
        }
    }

    // a lane holds rows 8 (e / 4) + 4 kg + e % 4 of matrix row n32; by way of LDS it gets 8 columns of a row
    const float S = p.w[GATED && n32 >= 16 ? 1 : 0].S[rows.e];
    constexpr int kWide = kCols + 4, kLanes = kOut / 8;
    static_assert(sizeof(float) * 32 * kWide <= sizeof(stage), "LDS of the outputs");
    float* out = reinterpret_cast<float*>(stage);
    const int column = GATED ? (n32 >> 4) * kOut + wave * 16 + (n32 & 15) : wave * 32 + n32;
#pragma unroll
    for (int a = 0; a < TM; ++a) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) out[((e >> 2) * 8 + kg * 4 + (e & 3)) * kWide + column] = acc[a][e] * S;
        __syncthreads();
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += kThreads / kLanes) {
            const int r = r0 + (int)threadIdx.x / kLanes, c = (int)threadIdx.x % kLanes * 8, row = 32 * a + r;
            const float* from = out + r * kWide + c;
            float v[8], u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = from[k];
                u[k] = GATED ? from[kOut + k] : 0.0f;
            }
            if (row < rows.rows && n0 + c < N)
                product_out8<GATED, false>(p, splits, split, rows.e, rows.first + row, n0 + c, N, v, u);
        }
    }
}

template <int BM, int STAGES, bool GATED>
void launch(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    const int64_t cols = GATED ? kCols / 2 : kCols, nn = (p.out + cols - 1) / cols;
    const int64_t steps = (p.in + kStep - 1) / kStep, each = (steps + plan.splits - 1) / plan.splits;
    const dim3 grid((uint32_t)(product_row_tiles(p.rows.tokens, p.rows.batch, BM) * nn * plan.splits));
    hipLaunchKernelGGL((k_product_mid<BM, STAGES, GATED>), grid, dim3(kThreads), 0, stream, p, (int)nn, plan.splits,
                       (int)each);
}

template <bool GATED>
void launch(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    if (plan.tile_rows == 32) launch<32, 3, GATED>(p, plan, stream);
    else if (plan.tile_rows == 64) launch<64, 2, GATED>(p, plan, stream);
    else launch<96, 2, GATED>(p, plan, stream);
}

}  // namespace

void launch_product_mid(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    if (p.matrices == 2) launch<true>(p, plan, stream);
    else launch<false>(p, plan, stream);
}

}  // namespace nvfp4
