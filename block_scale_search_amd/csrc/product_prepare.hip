// What runs before a product with NVFP4 matrices for gfx950: binary32 rows (and bf16 rows that are not laid out
// for 16-byte loads) as bf16 parts, gradients before an activation, and a bias's gradient.
//
// Parts. A binary32 value is the sum of three bf16 values, each the truncation of what the earlier ones leave
// (8 + 8 + 8 bits: exact, but for what lies below 2^-133); an infinity or NaN is its first part. Each part's
// product with a weight is exact in binary32, as that of a bf16 value is.
// All of these kernels read and write once: they are bound by memory.
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

struct Wide {
    bool dY, Z, U, d[2];
};

template <bool F32, bool GATED>
__global__ __launch_bounds__(kThreads) void k_product_slopes(ProductSlopes p, Wide w, int64_t pieces, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
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

// Bias gradients. A workgroup sums 64 columns over a share of a matrix's rows, each of its four waves every
// fourth row, eight rows' loads at a time; the shares' sums are added in binary64 by a second kernel. The order is fixed.
constexpr int kShareRows = 32;       // rows of a share at least
int64_t bias_shares(int64_t tokens, int64_t batch, int64_t cols) {
    if (batch < 1) return 1;
    const int64_t groups = batch * ((cols + 63) / 64);
    const int64_t want = (2048 + groups - 1) / groups, most = (tokens / batch + kShareRows - 1) / kShareRows;
    int64_t n = want < most ? want : most;
    if (n > 64) n = 64;
    return n < 1 ? 1 : n;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void k_product_bias(ProductSlopes p, int shares, float* partial) {
    __shared__ float sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    const int64_t e = blockIdx.y;
    int64_t lo = 0, hi = p.rows.tokens;
    if (p.rows.seg) segment(p.rows, (int)e, lo, hi);
    const int64_t each = (hi - lo + shares - 1) / shares, first = lo + each * blockIdx.z;
    const int64_t last = min(first + each, hi);
    float sum = 0.0f;
    if (n < p.cols) {
        for (int64_t t0 = first + wave; t0 < last; t0 += 32) {        // 8 rows summed by themselves
            float d[8], z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t t = min(t0 + 4 * k, last - 1);
                d[k] = load_value(p.dY, t * p.lddy + n, F32);
                z[k] = p.Z ? load_value(p.Z, t * p.ldz + n, F32) : 0.0f;
            }
            float part = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float a, slope = 1.0f;
                if (p.Z) act_slope<F32>(p.act, z[k], a, slope);
                part += t0 + 4 * k < last ? d[k] * slope : 0.0f;
            }
            sum += part;
        }
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && n < p.cols)
        partial[(e * shares + blockIdx.z) * p.cols + n] =
            (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
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

hipError_t launch_product_slopes(const ProductSlopes& p, hipStream_t stream) {
    const int64_t pieces = (p.cols + 7) / 8, total = p.rows.tokens * pieces;
    const dim3 grid((uint32_t)((total + kThreads - 1) / kThreads));
    const Wide w{wide(p.dY, p.lddy, p.f32), wide(p.Z, p.ldz, p.f32), wide(p.U, p.ldu, p.f32),
                 {wide(p.d[0], p.ldd[0], p.f32), wide(p.d[1], p.ldd[1], p.f32)}};
    if (p.U) {
        if (p.f32)
            hipLaunchKernelGGL((k_product_slopes<true, true>), grid, dim3(kThreads), 0, stream, p, w, pieces, total);
        else
            hipLaunchKernelGGL((k_product_slopes<false, true>), grid, dim3(kThreads), 0, stream, p, w, pieces, total);
    } else {
        if (p.f32)
            hipLaunchKernelGGL((k_product_slopes<true, false>), grid, dim3(kThreads), 0, stream, p, w, pieces, total);
        else
            hipLaunchKernelGGL((k_product_slopes<false, false>), grid, dim3(kThreads), 0, stream, p, w, pieces, total);
    }
    return hipGetLastError();
}

size_t product_bias_workspace_bytes(int64_t tokens, int64_t batch, int64_t cols) {
    return (size_t)(batch * bias_shares(tokens, batch, cols) * cols) * 4;
}

hipError_t launch_product_bias(const ProductSlopes& p, float* dbias, void* workspace, hipStream_t stream) {
    const int64_t shares = bias_shares(p.rows.tokens, p.rows.batch, p.cols);
    float* partial = static_cast<float*>(workspace);
    const dim3 grid((uint32_t)((p.cols + 63) / 64), (uint32_t)p.rows.batch, (uint32_t)shares);
    if (p.f32)
        hipLaunchKernelGGL(k_product_bias<true>, grid, dim3(kThreads), 0, stream, p, (int)shares, partial);
    else
        hipLaunchKernelGGL(k_product_bias<false>, grid, dim3(kThreads), 0, stream, p, (int)shares, partial);
    const int64_t total = p.rows.batch * p.cols;
    hipLaunchKernelGGL(k_product_bias_join, dim3((uint32_t)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       stream, partial, p.cols, total, (int)shares, dbias);
    return hipGetLastError();
}

}  // namespace nvfp4
