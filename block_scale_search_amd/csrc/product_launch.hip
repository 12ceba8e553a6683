// Products with NVFP4 matrices for gfx950: which kernel computes one, in how many shares of the reduction, and the
// kernel that adds the shares.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// One thread per 8 output columns of a row: the shares' sums (each times S already) in order, then what the
// product's own kernel does with whole sums.
template <bool GATED, bool F32>
__global__ __launch_bounds__(kThreads) void k_product_join(Product p, int splits, int64_t N, int64_t pieces, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / pieces, n = (i - t * pieces) * 8;
    if (t >= rows_end(p.rows)) return;
    const int64_t cols = partial_cols(N), stride = p.rows.tokens * (GATED ? 2 * cols : cols);
    const float* from = p.partial + t * (GATED ? 2 * cols : cols) + n;
    const auto sum = [&](const float* q, float (&s)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < splits; ++k, q += stride) {
            const float4 a = reinterpret_cast<const float4*>(q)[0], b = reinterpret_cast<const float4*>(q)[1];
            s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
            s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
        }
    };
    float v[8], u[8];
    sum(from, v);
    if constexpr (GATED) sum(from + cols, u);
    int e = 0;
    if (p.bias && p.rows.seg) {                          // the last matrix whose rows start at or before t
        int hi = p.rows.batch;
        while (hi - e > 1) {
            const int mid = (e + hi) >> 1;
            if (p.rows.seg[mid] <= t) e = mid;
            else hi = mid;
        }
    }
    product_out8<GATED, F32>(p, 1, 0, e, t, n, N, v, u);
}

// What each of `tiles` tiles of rows is. One thread a tile; a workgroup takes the matrices 256 at a time, sums their
// tiles and lets those of its threads whose tile is among them search the sums.
__global__ __launch_bounds__(kThreads) void k_product_map(ProductRows r, int size, int tiles) {
    __shared__ int upto[kThreads], waves[kThreads / 64];
    __shared__ int64_t from[kThreads], to[kThreads];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tile = blockIdx.x * kThreads + threadIdx.x;
    RowTile mine{0, 0, 0};
    int before = 0;
    for (int base = 0; base < r.batch; base += kThreads) {
        int64_t lo = 0, hi = 0;
        if (base + (int)threadIdx.x < r.batch) segment(r, base + threadIdx.x, lo, hi);
        int sum = (int)((hi - lo + size - 1) / size);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d, 64);
            if (lane >= d) sum += v;
        }
        if (lane == 63) waves[wave] = sum;
        __syncthreads();
        int all = before;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w == wave) sum += all;
            all += waves[w];
        }
        upto[threadIdx.x] = sum;
        from[threadIdx.x] = lo;
        to[threadIdx.x] = hi;
        __syncthreads();
        if (tile >= before && tile < all) {
            int at = 0;                                  // the first whose sum is above the tile
#pragma unroll
            for (int d = kThreads / 2; d > 0; d >>= 1)
                if (upto[at + d - 1] <= tile) at += d;
            const int k = tile - (at ? upto[at - 1] : before);
            mine.e = base + at;
            mine.first = from[at] + (int64_t)k * size;
            mine.rows = k >= 0 ? (int32_t)min((int64_t)size, to[at] - mine.first) : 0;
        }
        before = all;
        __syncthreads();
    }
    if (tile < tiles) r.map[tile] = mine;
}

}  // namespace

ProductPlan product_plan(int64_t tokens, int64_t batch, int64_t out, int64_t in, int32_t matrices,
                         bool backward, bool f32) {
    ProductPlan plan;
    const int64_t N = backward ? in : out, K = backward ? out : in;
    const int64_t each = batch > 0 ? (tokens + batch - 1) / batch : 0;
    int64_t steps, tiles;
    // rows of a matrix (on average): up to 4 of them pass through the kernel that keeps them in registers (8192 x 28672:
    // 37.6 us at 4 rows, by tiles of 32 rows 46; twice 4 take 48.3 and 47, of 2 x 14336 x 4096 34 and 28.7), up to 96
    // through tiles whose weights are converted where they are used (96 rows 70 us, 128 rows 106; by tiles through LDS 88 and 93)
    if (!backward && each <= 4) {
        plan.kernel = ProductKernel::kRows;
        plan.tile_rows = 4;
        plan.tile_cols = 16;
        plan.splits = 1;
        const int64_t slices = (K + 1023) / 1024, most = f32 ? 8 : 16;
        plan.threads = product_row_tiles(tokens, batch, 4) * ((out + 15) / 16) * 64 * (slices < most ? slices : most);
        return plan;
    }
    // Several matrices leave part of a tile empty each, which costs the kernel of smaller tiles less: 128 rows on average
    // of 128 matrices of 2048 x 768 119 us and 150, 256 rows 210 and 259, of 8 matrices of 2 x 14336 x 4096 701 and 821;
    // but 192 rows of 8 of 4096 x 14336 317 and 282, and from some 400 rows on it is the slower one. Tiles of 64
    // rows, since three workgroups share a compute unit then (64 rows on average of 128 matrices of 2048 x 768 79
    // us, by tiles of 96 rows 95); for one matrix, whose rows fill it, one of 96 (80 rows by 8192 x 28672 71.5 us, by two
    // of 64 96.6).
    if (!backward && !f32 && in % 64 == 0 && each <= (batch <= 1 ? 96 : in <= 4096 ? 256 : 128)) {
        plan.kernel = ProductKernel::kMid;
        plan.tile_rows = each <= 32 ? 32 : each <= 64 || batch > 1 ? 64 : 96;
        plan.tile_cols = 128;
        steps = (K + 127) / 128;
        tiles = product_row_tiles(tokens, batch, plan.tile_rows) * ((N * matrices + 127) / 128);
    } else {
        plan.kernel = ProductKernel::kTiles;
        steps = (K + 127) / 128 * 2 * (f32 ? 3 : 1) * (backward ? matrices : 1);
        const int64_t cols = N * (backward ? 1 : matrices);
        // tiles of 256 x 256 where they have work of 32 steps a compute unit at least (512 rows by 8192 x 8192 89 us, by
        // tiles of 128 x 128 96; 1024 by 4096 x 4096 63 and 56; 4096 by 4096 x 14336 400 and 560)
        const int64_t big = product_tile_rows(tokens, batch, 256) * ((cols + 255) / 256);
        // and where their last round, one tile a compute unit, is not left too empty (of one matrix; of several it is not known
        // how many there are): 272 tiles 205 us, by tiles of 128 x 128 188; 544 324 and 337
        const bool even = batch > 1 || big <= 256 || 2 * ((big + 255) / 256 * 256) <= 3 * big;
        const int side = each >= 256 && big * steps >= 256 * 32 && even ? 256 : 128;
        plan.tile_rows = plan.tile_cols = side;
        tiles = side == 256 ? big : product_tile_rows(tokens, batch, 128) * ((cols + 127) / 128);
    }
    // shares: about two workgroups a compute unit, of at least 4 steps each (64 rows by 8192 x 28672 in 8 shares 59.7 us,
    // in 4 69.2, in 12 64.0)
    const int64_t unit = plan.kernel == ProductKernel::kTiles ? 4 : 1;
    const int64_t want = plan.kernel == ProductKernel::kTiles && plan.tile_rows == 256 ? 256 : 512;
    int64_t splits = tiles > 0 ? want / tiles : 1;
    if (plan.kernel == ProductKernel::kTiles && tiles >= 256) splits = 1;       // 1024 rows by 4096 x 4096 50 us, in 2 shares 56
    if (splits > steps / (2 * unit)) splits = steps / (2 * unit);
    if (splits > 32) splits = 32;
    if (splits < 1) splits = 1;
    const int64_t share = ((steps + splits - 1) / splits + unit - 1) / unit * unit;
    splits = (steps + share - 1) / share;                // none empty
    plan.splits = (int32_t)splits;
    plan.threads = tiles * splits * (plan.tile_rows == 256 ? 512 : 256);
    return plan;
}

size_t product_partial_bytes(const ProductPlan& plan, int64_t tokens, int64_t out, int64_t in,
                             int32_t matrices, bool backward) {
    if (plan.splits <= 1) return 0;
    const int64_t N = backward ? in : out;
    return (size_t)(plan.splits * tokens * ((N + 7) / 8 * 8) * (backward ? 1 : matrices)) * 4;
}

size_t product_map_bytes(const ProductPlan& plan, int64_t tokens, int64_t batch) {
    return batch > kMapped ? (size_t)product_tile_rows(tokens, batch, plan.tile_rows) * sizeof(RowTile) : 0;
}

hipError_t launch_product(const Product& given, hipStream_t stream) {
    Product p = given;
    const auto wide = [&](const void* q, int64_t ld) {
        return q == nullptr || ((reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld % (p.f32 ? 4 : 8) == 0);
    };
    p.wide = wide(p.y, p.ldy) && wide(p.pre[0], p.ldpre[0]) && wide(p.pre[1], p.ldpre[1]) &&
             wide(p.residual, p.ldr) && wide(p.bias, p.out);
    ProductPlan plan = product_plan(p.rows.tokens, p.rows.batch, p.out, p.in, p.matrices, p.backward, p.f32);
    // the tile kernel asks for less alignment than the copies of codes and scale bytes into LDS
    const auto at = [](const void* q, uintptr_t to) { return (reinterpret_cast<uintptr_t>(q) & (to - 1)) == 0; };
    bool fits = true;
    for (int m = 0; plan.kernel == ProductKernel::kMid && m < p.matrices; ++m)
        fits = fits && at(p.w[m].packed, 16) && at(p.w[m].scales, 4) && p.w[m].stride % 64 == 0;
    if (!fits) plan = ProductPlan{ProductKernel::kTiles, 128, 128, 1, 0};   // no smaller tiles: no larger map
    if (p.rows.batch > kMapped) {
        const int tiles = (int)product_tile_rows(p.rows.tokens, p.rows.batch, plan.tile_rows);   // all that a grid has
        hipLaunchKernelGGL(k_product_map, dim3((uint32_t)((tiles + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                           stream, p.rows, plan.tile_rows, tiles);
    }
    if (plan.kernel == ProductKernel::kRows) {
        launch_product_rows(p, stream);
        return hipGetLastError();
    }
    if (plan.kernel == ProductKernel::kMid) {
        launch_product_mid(p, plan, stream);
    } else {
        launch_product_tiles(p, plan, stream);
    }
    if (plan.splits > 1) {
        const int64_t N = p.backward ? p.in : p.out, pieces = (N + 7) / 8, total = p.rows.tokens * pieces;
        const dim3 grid((uint32_t)((total + kThreads - 1) / kThreads));
        const bool gated = !p.backward && p.matrices == 2;
        if (gated && p.f32)
            hipLaunchKernelGGL((k_product_join<true, true>), grid, dim3(kThreads), 0, stream, p, plan.splits, N, pieces, total);
        else if (gated)
            hipLaunchKernelGGL((k_product_join<true, false>), grid, dim3(kThreads), 0, stream, p, plan.splits, N, pieces, total);
        else if (p.f32)
            hipLaunchKernelGGL((k_product_join<false, true>), grid, dim3(kThreads), 0, stream, p, plan.splits, N, pieces, total);
        else
            hipLaunchKernelGGL((k_product_join<false, false>), grid, dim3(kThreads), 0, stream, p, plan.splits, N, pieces, total);
    }
    return hipGetLastError();
}

}  // namespace nvfp4
