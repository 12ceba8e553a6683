// What runs before a product with NVFP4 matrices for gfx950: binary32 rows (and bf16 rows that are not laid out
// for 16-byte loads) as bf16 parts, gradients before an activation, and a bias's gradient.
//
// Parts. A binary32 value is the sum of three bf16 values, each the truncation of what the earlier ones leave
// (8 + 8 + 8 bits: exact, but for what lies below 2^-133); an infinity or NaN is its first part. Each part's
// product with a weight is exact in binary32, as that of a bf16 value is.
// Slopes. dZ, dG and dU are rounded once, to the outputs' type, and the product reads those: dX is the product of what
// the caller gets, as in a program of separate calls. So bf16 dX of a pair is off by 2.3e-3 of its norm; from unrounded
// values, as two bf16 parts and thus by twice the product, it would be 1.7e-3, its own rounding. A bias's gradient sums
// the unrounded.
// All of these kernels read and write once: they are bound by memory (dG and dU of 4096 x 14336 from three such tensors 94 us,
// 6.2 TB/s with what the cache still holds) or, small, by their chain of loads (333 x 1003 in binary32 with a bias 12 us).
#include <hip/hip_runtime.h>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void split(float x, uint32_t (&part)[3]) {
    const bool finite = fabsf(x) < __builtin_inff();
    const uint32_t u = __float_as_uint(x) & 0xFFFF0000u;
    const float r = finite ? x - __uint_as_float(u) : 0.0f;
    const uint32_t v = __float_as_uint(r) & 0xFFFF0000u;
    part[0] = (x == x ? u : 0x7FC00000u) >> 16;
    part[1] = v >> 16;
    part[2] = __float_as_uint(r - __uint_as_float(v)) >> 16;
}

__device__ __forceinline__ u32x4 pack8(const uint32_t (&x)[8]) {
    return u32x4{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16};
}

// The parts of values 8 piece .. + 7 of row t.
template <bool F32>
__device__ __forceinline__ void store_parts(const float (&x)[8], uint16_t* parts, int64_t at, int64_t plane) {
    uint32_t b[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (F32) {
            uint32_t s[3];
            split(x[i], s);
            b[0][i] = s[0];
            b[1][i] = s[1];
            b[2][i] = s[2];
        } else {
            b[0][i] = bf16_bits(x[i]);
        }
    }
#pragma unroll
    for (int k = 0; k < (F32 ? 3 : 1); ++k)
        *reinterpret_cast<u32x4*>(parts + k * plane + at) = pack8(b[k]);
}

// One thread per piece of 8 values, `pieces` a row.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_product_parts(const void* X, int64_t cols, int64_t ldx, bool wide,
                                                            int64_t pieces, int64_t total, uint16_t* parts,
                                                            int64_t ld, int64_t plane) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / pieces, c = (i - t * pieces) * 8;
    float x[8];
    load8<F32>(X, t * ldx, c, cols, wide, x);
    store_parts<F32>(x, parts, t * ld + c, plane);
}

// Bias gradients. A workgroup sums COLS columns over a share of a matrix's rows; its lanes take COLS columns by 64 / COLS
// rows, eight rows' loads at a time, and their sums are added in binary64. Up to kWhole rows a matrix (on average)
// there is one share, and 16 columns a workgroup, so that no second launch is needed; else 64 columns, and a second
// kernel adds the shares' sums in binary64. The order is fixed.
constexpr int kWhole = 512;
constexpr int kShareRows = 32;       // rows of a share at least
struct Bias {
    float* to;                       // dbias, or the shares' sums
    int32_t shares, blocks, groups;  // workgroups, and those of a share of a matrix
    bool narrow;
};
Bias bias_of(int64_t tokens, int64_t batch, int64_t cols) {
    Bias b{nullptr, 1, 0, 0, batch < 1 || (tokens <= kWhole * batch && batch * cols <= 1 << 24)};
    b.groups = (int32_t)((cols + (b.narrow ? 15 : 63)) / (b.narrow ? 16 : 64));
    if (!b.narrow) {
        const int64_t groups = batch * b.groups;
        const int64_t want = (2048 + groups - 1) / groups, most = (tokens / batch + kShareRows - 1) / kShareRows;
        const int64_t shares = want < most ? want : most;
        b.shares = (int32_t)(shares < 1 ? 1 : shares < 64 ? shares : 64);   // with fewer rows than matrices too: zeros
    }
    b.blocks = (int32_t)(b.groups * batch * b.shares);
    return b;
}

template <bool F32, int COLS>
__device__ __forceinline__ void bias_sums(const ProductSlopes& p, const Bias& b, int block) {
    constexpr int kRows = 64 / COLS * (kThreads / 64);   // rows side by side
    __shared__ float sums[kRows][COLS];
    const int column = threadIdx.x % COLS, row = threadIdx.x / COLS;
    const int group = block % b.groups, share = block / b.groups % b.shares;
    const int64_t e = block / b.groups / b.shares, n = (int64_t)group * COLS + column;
    int64_t lo = 0, hi = p.rows.tokens;
    if (p.rows.seg) segment(p.rows, (int)e, lo, hi);
    const int64_t each = (hi - lo + b.shares - 1) / b.shares, first = lo + each * share;
    const int64_t last = min(first + each, hi);
    float sum = 0.0f;
    if (n < p.cols) {
        for (int64_t t0 = first + row; t0 < last; t0 += 8 * kRows) {  // 8 rows summed by themselves
            float d[8], z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t t = min(t0 + kRows * k, last - 1);
                d[k] = load_value(p.dY, t * p.lddy + n, F32);
                z[k] = p.Z ? load_value(p.Z, t * p.ldz + n, F32) : 0.0f;
            }
            float part = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float a, slope = 1.0f;
                if (p.Z) act_slope<F32>(p.act, z[k], a, slope);
                part += t0 + kRows * k < last ? d[k] * slope : 0.0f;
            }
            sum += part;
        }
    }
    sums[row][column] = sum;
    __syncthreads();
    if (row == 0 && n < p.cols) {
        double s = 0.0;
#pragma unroll
        for (int k = 0; k < kRows; ++k) s += (double)sums[k][column];
        b.to[(e * b.shares + share) * p.cols + n] = (float)s;
    }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void k_product_bias(ProductSlopes p, Bias b) {
    if (b.narrow) bias_sums<F32, 16>(p, b, blockIdx.x);
    else bias_sums<F32, 64>(p, b, blockIdx.x);
}

struct Wide {
    bool dY, Z, U, d[2];
};

// One thread per piece of 8 values. The first workgroups make the bias gradient (b.blocks, none if it is not asked for).
template <bool F32, bool GATED>
__global__ __launch_bounds__(kThreads) void k_product_slopes(ProductSlopes p, Wide w, int64_t pieces, int64_t total, Bias b) {
    if constexpr (!GATED) {
        if (blockIdx.x < (uint32_t)b.blocks) {
            if (b.narrow) bias_sums<F32, 16>(p, b, blockIdx.x);
            else bias_sums<F32, 64>(p, b, blockIdx.x);
            return;
        }
    }
    const int64_t i = ((int64_t)blockIdx.x - b.blocks) * kThreads + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / pieces, c = (i - t * pieces) * 8;
    if (t >= rows_end(p.rows)) return;
    float dy[8], z[8], d1[8];
    load8<F32>(p.dY, t * p.lddy, c, p.cols, w.dY, dy);
    if (p.Z) load8<F32>(p.Z, t * p.ldz, c, p.cols, w.Z, z);
    if constexpr (GATED) {
        float u[8], d2[8];
        load8<F32>(p.U, t * p.ldu, c, p.cols, w.U, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, slope;
            act_slope<F32>(p.act, z[k], a, slope);
            d1[k] = dy[k] * u[k] * slope;
            d2[k] = dy[k] * a;
        }
        if (p.d[1]) store8<F32>(p.d[1], t * p.ldd[1], c, p.cols, w.d[1], d2);
        if (p.parts[1]) store_parts<F32>(d2, p.parts[1], t * p.ld + c, p.plane);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, slope = 1.0f;
            if (p.Z) act_slope<F32>(p.act, z[k], a, slope);
            d1[k] = dy[k] * slope;
        }
    }
    if (p.d[0]) store8<F32>(p.d[0], t * p.ldd[0], c, p.cols, w.d[0], d1);
    if (p.parts[0]) store_parts<F32>(d1, p.parts[0], t * p.ld + c, p.plane);
}

bool wide(const void* p, int64_t ld, bool f32) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % (f32 ? 4 : 8) == 0;
}

__global__ __launch_bounds__(kThreads) void k_product_bias_join(const float* partial, int64_t cols, int64_t total,
                                                                int shares, float* dbias) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const int64_t e = i / cols, n = i - e * cols;
    double s = 0.0;
    for (int k = 0; k < shares; ++k) s += (double)partial[(e * shares + k) * cols + n];
    dbias[i] = (float)s;
}

}  // namespace

hipError_t launch_product_parts(const void* X, bool f32, int64_t tokens, int64_t cols, int64_t ldx,
                                uint16_t* parts, int64_t ld, int64_t plane, hipStream_t stream) {
    const int64_t pieces = ld / 8, total = tokens * pieces;
    const dim3 grid((uint32_t)((total + kThreads - 1) / kThreads));
    const bool w = wide(X, ldx, f32);
    if (f32)
        hipLaunchKernelGGL(k_product_parts<true>, grid, dim3(kThreads), 0, stream, X, cols, ldx, w, pieces, total,
                           parts, ld, plane);
    else
        hipLaunchKernelGGL(k_product_parts<false>, grid, dim3(kThreads), 0, stream, X, cols, ldx, w, pieces, total,
                           parts, ld, plane);
    return hipGetLastError();
}

size_t product_bias_workspace_bytes(int64_t tokens, int64_t batch, int64_t cols) {
    const Bias b = bias_of(tokens, batch, cols);
    return batch > 0 ? (size_t)(batch * b.shares * cols) * 4 : 0;
}

hipError_t launch_product_slopes(const ProductSlopes& p, bool slopes, float* dbias, void* workspace, hipStream_t stream) {
    const int64_t pieces = (p.cols + 7) / 8, total = slopes ? p.rows.tokens * pieces : 0;
    Bias b{};
    if (dbias) {
        b = bias_of(p.rows.tokens, p.rows.batch, p.cols);
        b.to = b.shares > 1 ? static_cast<float*>(workspace) : dbias;
    }
    if (total > 0 && b.blocks > ((((int64_t)1 << 32) - 256) - total) / kThreads) {   // a launch has fewer than 2^32 threads
        const hipError_t e = launch_product_slopes(p, false, dbias, workspace, stream);
        return e == hipSuccess ? launch_product_slopes(p, true, nullptr, nullptr, stream) : e;
    }
    const dim3 grid((uint32_t)(b.blocks + (total + kThreads - 1) / kThreads));
    const Wide w{wide(p.dY, p.lddy, p.f32), wide(p.Z, p.ldz, p.f32), wide(p.U, p.ldu, p.f32),
                 {wide(p.d[0], p.ldd[0], p.f32), wide(p.d[1], p.ldd[1], p.f32)}};
    const auto launch = [&](auto* kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, w, pieces, total, b);
    };
    if (p.U) {
        if (p.f32) launch(k_product_slopes<true, true>);
        else launch(k_product_slopes<false, true>);
    } else if (slopes) {
        if (p.f32) launch(k_product_slopes<true, false>);
        else launch(k_product_slopes<false, false>);
    } else if (p.f32) {
        hipLaunchKernelGGL(k_product_bias<true>, grid, dim3(kThreads), 0, stream, p, b);
    } else {
        hipLaunchKernelGGL(k_product_bias<false>, grid, dim3(kThreads), 0, stream, p, b);
    }
    if (b.shares > 1) {
        const int64_t all = p.rows.batch * p.cols;
        hipLaunchKernelGGL(k_product_bias_join, dim3((uint32_t)((all + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           stream, b.to, p.cols, all, b.shares, dbias);
    }
    return hipGetLastError();
}

}  // namespace nvfp4
