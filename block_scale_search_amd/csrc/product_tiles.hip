// Products of many rows with NVFP4 matrices for gfx950, by tiles: forward, gated and backward.
//
// A workgroup owns a tile of rows and columns and walks the reduction in steps of 64. The rows' side
// goes from global memory straight into LDS; the codes of the next step are loaded into registers while
// the current one is multiplied, converted there (level * E4M3 is exact in bf16) and written to LDS as
// [column][64], the same in both directions: backward, a thread converts four rows of the matrix by eight columns
// and pairs the rows in the conversion to bf16, which is the transposition. The 16-byte pieces of an
// LDS row are permuted by the row so that the reads of MFMA operands and the writes use all banks.
// Gated: the columns of a tile are 32 of the gate, the same 32 of the other matrix, and so on, so that
// both values of an output are in the same lane.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int BK = 64;
enum Mode { kLinear = 0, kGated = 1, kBackward = 2 };

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;     // MFMA tiles of a wave
    static constexpr int kLoads = BM * (BK / 8) / kThreads;        // 16-byte pieces of A a thread
    static_assert(BN * BK / kThreads == 32, "a thread converts 32 weights a step");
};

// Piece c (8 values) of LDS row r sits at c ^ swizzle(r).
__device__ __forceinline__ int swizzle(int r) { return (r ^ (r >> 3)) & 7; }

// A thread's codes of one step. Forward: 32 columns of one row, two scale bytes. Backward: 8 columns of
// four rows, their scale bytes.
struct Raw {
    u32x4 code;
    uint32_t scale;
};

// Where in the reduction a step lies: step `kt` of plane `plane` of matrix `m`.
struct Cursor {
    int kt = 0, plane = 0, m = 0;
    __device__ __forceinline__ void at(int step, int nk, int planes) {
        kt = step % nk;
        plane = step / nk % planes;
        m = step / nk / planes;
    }
    __device__ __forceinline__ void next(int nk, int planes) {
        if (++kt == nk) {
            kt = 0;
            if (++plane == planes) {
                plane = 0;
                ++m;
            }
        }
    }
};

template <int M_, int N_, int WM_, int WN_, int MODE, bool F32>
__global__ __launch_bounds__(64 * WM_ * WN_) void k_product_tiles(Product p, int nn, int splits, int each) {
    typedef Shape<M_, N_, WM_, WN_> S;
    constexpr int BM = S::BM, BN = S::BN, TM = S::TM, TN = S::TN;
    __shared__ __align__(1024) uint16_t lds_a[2][BM][BK];
    __shared__ __align__(1024) uint16_t lds_b[2][BN][BK];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const uint32_t of = blockIdx.x / (uint32_t)splits;
    const int split = (int)(blockIdx.x - of * (uint32_t)splits);
    const int tile = (int)(of / (uint32_t)nn), tn = (int)(of - (uint32_t)tile * (uint32_t)nn);
    RowTile rows;
    if (!find_rows(p.rows, tile, BM, rows)) return;

    constexpr int kCols = MODE == kGated ? BN / 2 : BN;            // output columns of a tile
    const int64_t n0 = (int64_t)tn * kCols;
    const int64_t N = MODE == kBackward ? p.in : p.out;
    const int64_t K = MODE == kBackward ? p.out : p.in;
    const int64_t k_pad = (K + 7) / 8 * 8;
    const int nk = (int)((K + BK - 1) / BK);
    const int matrices = MODE == kBackward ? p.matrices : 1;
    const int begin = split * each, steps = min(each, nk * p.planes * matrices - begin);

    const auto load_a = [&](int buf, const Cursor& c) {
        const ProductOperand& a = p.a[MODE == kBackward ? c.m : 0];
        const uint16_t* base = a.p + c.plane * p.plane;
        const int64_t k0 = (int64_t)c.kt * BK;
#pragma unroll
        for (int r = 0; r < S::kLoads; ++r) {
            const int id = tid + S::kThreads * r, row = id >> 3;
            const int64_t k = k0 + ((id & 7) ^ swizzle(row)) * 8;
            // rows past the tile read its last row, pieces past the edge the row's first: both meet
            // columns that are not stored or weights of zero
            const uint16_t* from = base + (rows.first + min(row, rows.rows - 1)) * a.ld + (k < k_pad ? k : 0);
            copy16(from, &lds_a[buf][(S::kThreads * r + 64 * wave) >> 3][0]);
        }
    };

    // forward: row b_row of lds_b, half b_half of its 64 values
    const int b_row = tid >> 1, b_half = tid & 1;
    // backward: columns 8 b_block .. + 7, values 8 b_octet + 4 b_half .. + 3
    const int b_block = (tid >> 1) % (BN / 8), b_octet = (tid >> 1) / (BN / 8);
    const auto load_b = [&](Raw& raw, const Cursor& c) {
        const int64_t k0 = (int64_t)c.kt * BK;
        if constexpr (MODE == kBackward) {
            const ProductMatrix& w = p.w[c.m];
            const int64_t col = min(n0 + b_block * 8, N - 8);
            raw.scale = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t o = k0 + b_octet * 8 + b_half * 4 + r;
                const int64_t at = rows.e * w.stride + min(o, K - 1) * p.in + col;
                raw.code[r] = *reinterpret_cast<const uint32_t*>(w.packed + at / 2);
                const uint32_t s = w.scales[at / 16];
                raw.scale |= (o < K ? s : 0u) << (8 * r);
            }
        } else {
            const int second = MODE == kGated ? (b_row >> 5) & 1 : 0;
            const int c32 = MODE == kGated ? (b_row >> 6) * 32 + (b_row & 31) : b_row;
            const ProductMatrix& w = p.w[second];
            const int64_t k = k0 + b_half * 32;
            const int64_t at = rows.e * w.stride + min(n0 + c32, N - 1) * K + k;
            if (k + 32 <= K) {
                raw.code = *reinterpret_cast<const u32x4_at8*>(w.packed + at / 2);
                raw.scale = *reinterpret_cast<const u16_at1*>(w.scales + at / 16);
            } else {
                raw.code = u32x4{0u, 0u, 0u, 0u};
                raw.scale = 0;
                if (k + 16 <= K) {
                    const u32x2 half = *reinterpret_cast<const u32x2_at8*>(w.packed + at / 2);
                    raw.code[0] = half[0];
                    raw.code[1] = half[1];
                    raw.scale = w.scales[at / 16];
                }
            }
        }
    };
    const auto store_b = [&](int buf, const Raw& raw) {
        if constexpr (MODE == kBackward) {
            float x[4][8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float s = r == 0 ? scale_value<0>(raw.scale) : r == 1 ? scale_value<1>(raw.scale)
                              : r == 2 ? scale_value<2>(raw.scale) : scale_value<3>(raw.scale);
                code_values<0>(raw.code[r], s, x[r][0], x[r][1]);
                code_values<1>(raw.code[r], s, x[r][2], x[r][3]);
                code_values<2>(raw.code[r], s, x[r][4], x[r][5]);
                code_values<3>(raw.code[r], s, x[r][6], x[r][7]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = b_block * 8 + j;
                *reinterpret_cast<u32x2*>(&lds_b[buf][row][(b_octet ^ swizzle(row)) * 8 + b_half * 4]) =
                    u32x2{bf16_pair(x[0][j], x[1][j]), bf16_pair(x[2][j], x[3][j])};
            }
        } else {
            const float s0 = scale_value<0>(raw.scale), s1 = scale_value<1>(raw.scale);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<u32x4*>(&lds_b[buf][b_row][((b_half * 4 + j) ^ swizzle(b_row)) * 8]) =
                    dequant8(raw.code[j], j < 2 ? s0 : s1);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;

    const int r32 = lane & 31, kg = lane >> 5;
    Cursor ca, cb;
    cb.at(begin, nk, p.planes);
    ca = cb;
    const int to_switch = nk * p.planes - begin;         // the step at which the second matrix begins
    Raw raw;
    load_b(raw, cb);
    load_a(0, ca);
    store_b(0, raw);
    ca.next(nk, p.planes);
    cb.next(nk, p.planes);
    if (steps > 1) load_b(raw, cb);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        const int buf = s & 1;
        if (s + 1 < steps) load_a(buf ^ 1, ca);
        const Raw now = raw;
        cb.next(nk, p.planes);
        ca.next(nk, p.planes);
        if (s + 2 < steps) load_b(raw, cb);
        if constexpr (MODE == kBackward) {
            if (s == to_switch && s > 0) {                      // the second matrix's sums carry its S
                const float f = p.w[0].S[rows.e] / p.w[1].S[rows.e];
#pragma unroll
                for (int a = 0; a < TM; ++a)
#pragma unroll
                    for (int b = 0; b < TN; ++b)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[a][b][e] *= f;
            }
        }
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
            bf16x8 fa[TM], fb[TN];
            const int c = 2 * ks + kg;
#pragma unroll
            for (int a = 0; a < TM; ++a) {
                const int row = (wm * TM + a) * 32 + r32;
                fa[a] = *reinterpret_cast<const bf16x8*>(&lds_a[buf][row][(c ^ swizzle(row)) * 8]);
            }
#pragma unroll
            for (int b = 0; b < TN; ++b) {
                const int row = (wn * TN + b) * 32 + r32;
                fb[b] = *reinterpret_cast<const bf16x8*>(&lds_b[buf][row][(c ^ swizzle(row)) * 8]);
            }
#pragma unroll
            for (int a = 0; a < TM; ++a)
#pragma unroll
                for (int b = 0; b < TN; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
        }
        if (s + 1 < steps) store_b(buf ^ 1, now);
        __syncthreads();
    }

    // a lane holds rows 8 (e / 4) + 4 kg + e % 4 of column r32 of each 32 x 32 tile; backward, the sums are over the
    // S of the last matrix met
    const int at = MODE == kBackward && to_switch < steps ? 1 : 0;
    const float S0 = p.w[at].S[rows.e];
    const float S1 = MODE == kGated ? p.w[1].S[rows.e] : 0.0f;
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; b += MODE == kGated ? 2 : 1) {
            const int64_t n = n0 + (MODE == kGated ? (wn * TN + b) * 16 : (wn * TN + b) * 32) + r32;
            if (n >= N) continue;
            const float bias = MODE == kLinear && p.bias ? load_value(p.bias, rows.e * N + n, F32) : 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = (wm * TM + a) * 32 + (e >> 2) * 8 + kg * 4 + (e & 3);
                if (row >= rows.rows) continue;
                const int64_t t = rows.first + row;
                const float v = acc[a][b][e] * S0;
                if constexpr (MODE == kGated) {
                    const float u = acc[a][b + 1][e] * S1;
                    if (splits > 1) {
                        product_partial(p, split, t, n, 2 * N) = v;
                        product_partial(p, split, t, N + n, 2 * N) = u;
                    } else {
                        product_gated(p, t, n, v, u, F32);
                    }
                } else if (splits > 1) {
                    product_partial(p, split, t, n, N) = v;
                } else if constexpr (MODE == kBackward) {
                    store_value(p.y, t * p.ldy + n, v, F32);
                } else {
                    product_linear(p, t, n, v + bias, F32);
                }
            }
        }
}

typedef Shape<128, 128, 2, 2> Small;

template <typename S, int MODE>
void launch(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    const int64_t N = MODE == kBackward ? p.in : p.out, K = MODE == kBackward ? p.out : p.in;
    const int64_t cols = MODE == kGated ? S::BN / 2 : S::BN, nn = (N + cols - 1) / cols;
    const int64_t steps = (K + BK - 1) / BK * p.planes * (MODE == kBackward ? p.matrices : 1);
    const int64_t each = (steps + plan.splits - 1) / plan.splits;
    const dim3 grid((uint32_t)(product_row_tiles(p.rows.tokens, p.rows.batch, S::BM) * nn * plan.splits));
    if (p.f32)
        hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, true>), grid, dim3(S::kThreads), 0,
                           stream, p, (int)nn, plan.splits, (int)each);
    else
        hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, false>), grid, dim3(S::kThreads), 0,
                           stream, p, (int)nn, plan.splits, (int)each);
}

}  // namespace

void launch_product_tiles(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    if (p.backward) launch<Small, kBackward>(p, plan, stream);
    else if (p.matrices == 2) launch<Small, kGated>(p, plan, stream);
    else launch<Small, kLinear>(p, plan, stream);
}

}  // namespace nvfp4
