// Products with NVFP4 matrices: the views that the C-ABI layer (product_api.hip) makes of its checked
// arguments, and the launchers of the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// Matrices [out, in] of codes and scale bytes, `stride` weights apart, and their global scales.
struct ProductMatrix {
    const uint8_t* packed;
    const uint8_t* scales;
    const float* S;
    int64_t stride;
};

// Which rows meet which matrix: rows seg[e] .. seg[e+1] - 1 matrix e; no seg: all rows matrix 0.
// map: with more than kMapped matrices, what each tile of rows is, filled by a kernel of its own (some 2 us); else not
// used, and each workgroup searches the offsets, 64 at a time. Gradients are as fast either way at 128 matrices, forward products
// at some 256, and in between each loses 4% at most by the other's limit. Us without a map and with it, of 4 rows a matrix by
// gate and up of 768 x 2048, 64 by 512 x 768, and 64 back through 2 x 512 x 1024: 128 matrices 63.3 and 66.3, 28.2 and 29.7,
// 87.7 and 87.8; 256 matrices 110.6 and 114.4, 48.1 and 47.5, 164.6 and 158.6; 512 matrices 245 and 235, 93.5 and 83.9, 351
// and 319.
constexpr int kMapped = 128;
struct RowTile {
    int32_t e, rows;         // rows 0: none
    int64_t first;
};
struct ProductRows {
    const int64_t* seg;
    int64_t tokens;
    int32_t batch;
    RowTile* map;
};

// The activations' side, bf16 rows: `planes` parts of a value (1: bf16 itself, 3: the parts of a
// binary32 value), `plane` elements apart. Columns past `k` up to the next multiple of 8 are zero.
struct ProductOperand {
    const uint16_t* p;
    int64_t ld;
};

// One product. Forward: rows [in] times matrices' rows, out columns; gated: two matrices, out columns
// each. Backward: rows [out] times matrices' columns, in columns; two matrices: their sum.
struct Product {
    ProductMatrix w[2];
    int32_t matrices;
    bool backward;
    bool f32;                // outputs, bias and residual are binary32, else bf16
    int64_t out, in;
    ProductRows rows;
    ProductOperand a[2];     // forward: a[0] only
    int32_t planes;
    int64_t plane;
    // forward: y = act(z + bias) + residual, or act(g) * u; pre: z, or g and u. backward: y only.
    int32_t act;
    const void* bias;        // [batch, out] or null
    const void* residual;    // or null
    int64_t ldr;
    void* pre[2];            // or null
    int64_t ldpre[2];
    void* y;
    int64_t ldy;
    bool wide;               // rows of y, pre, residual and bias are whole 16-byte pieces
    float* partial;          // [splits][tokens][columns up to a multiple of 8, gated: twice], where there are splits
};

// Tiles of `size` rows that the matrices' rows make at most.
inline int64_t product_row_tiles(int64_t tokens, int64_t batch, int64_t size) {
    if (batch <= 1) return (tokens + size - 1) / size;
    return tokens / size + (batch < tokens ? batch : tokens);
}

// Rows of tiles in the tile kernel's grid: with many of several matrices, whole turns of the 8 XCDs.
constexpr int kManyRowTiles = 64;
inline int64_t product_tile_rows(int64_t tokens, int64_t batch, int64_t size) {
    const int64_t n = product_row_tiles(tokens, batch, size);
    return batch > 1 && n >= kManyRowTiles ? (n + 7) / 8 * 8 : n;
}

// Which kernel computes a product, and in how many shares of its reduction (more than one: their sums go to the
// workspace, and a second kernel adds them). A function of the sizes alone, since the workspace's size is.
enum class ProductKernel { kRows, kMid, kTiles };
struct ProductPlan {
    ProductKernel kernel;
    int32_t tile_rows;       // rows of X a workgroup
    int32_t tile_cols;       // matrix rows (backward: columns) a workgroup
    int32_t splits;
    int64_t threads;         // of all workgroups
};
ProductPlan product_plan(int64_t tokens, int64_t batch, int64_t out, int64_t in, int32_t matrices,
                         bool backward, bool f32);
size_t product_partial_bytes(const ProductPlan& plan, int64_t tokens, int64_t out, int64_t in,
                             int32_t matrices, bool backward);

// p.partial: a workspace of product_partial_bytes; p.rows.map, with several matrices: of product_map_bytes.
size_t product_map_bytes(const ProductPlan& plan, int64_t tokens, int64_t batch);
hipError_t launch_product(const Product& p, hipStream_t stream);

// The kernels' launchers.
void launch_product_rows(const Product& p, hipStream_t stream);
void launch_product_mid(const Product& p, const ProductPlan& plan, hipStream_t stream);
void launch_product_tiles(const Product& p, const ProductPlan& plan, hipStream_t stream);

// bf16 parts of rows [tokens, cols] of dtype, padded with zeros to ld columns (a multiple of 8).
hipError_t launch_product_parts(const void* X, bool f32, int64_t tokens, int64_t cols, int64_t ldx,
                                uint16_t* parts, int64_t ld, int64_t plane, hipStream_t stream);

// Gradients before a product's activation: dZ = dY act'(Z), or (U given) dG = dY U act'(G) and
// dU = dY act(G), written to d1 (and d2) where given, and as parts where given. Rows of
// no matrix are left alone.
struct ProductSlopes {
    ProductRows rows;
    bool f32;
    int64_t cols;
    int32_t act;
    const void* dY;
    int64_t lddy;
    const void* Z;           // null for no activation
    int64_t ldz;
    const void* U;
    int64_t ldu;
    void* d[2];
    int64_t ldd[2];
    uint16_t* parts[2];
    int64_t ld, plane;
};
// With dbias: dbias[e] = sum of dY act'(Z) over matrix e's rows, [batch, cols], in the same launch; without `slopes`
// only that.
size_t product_bias_workspace_bytes(int64_t tokens, int64_t batch, int64_t cols);
hipError_t launch_product_slopes(const ProductSlopes& p, bool slopes, float* dbias, void* workspace, hipStream_t stream);

}  // namespace nvfp4
