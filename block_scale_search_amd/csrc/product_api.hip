// C ABI of the products with NVFP4 matrices (include/nvfp4.h): argument validation on the host, then
// kernel launches on the caller's stream. Every check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include "../../include/nvfp4.h"
#include "product.h"

namespace {

constexpr int64_t kInt32 = (int64_t)1 << 31;
constexpr int64_t kMaxSide = (int64_t)1 << 22;     // 32-bit offsets inside a tile
constexpr int64_t kMaxSpan = (int64_t)1 << 56;
constexpr int64_t kMaxBiases = (int64_t)1 << 29;   // gradients of biases: 4 threads each, matrices rounded up to 256
constexpr int64_t kThreads32 = ((int64_t)1 << 32) - 256;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool span_ok(int64_t n, int64_t stride) {
    return stride <= kMaxSpan && (n <= 1 || stride <= kMaxSpan / n);
}
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int elem_size(int dtype) {
    if (dtype == NVFP4_DTYPE_F32) return 4;
    if (dtype == NVFP4_DTYPE_BF16) return 2;
    return 0;
}

bool sizes_ok(int64_t tokens, int64_t batch, int64_t out, int64_t in) {
    return tokens >= 0 && tokens < kInt32 && batch >= 0 && batch <= 65535 && out >= 1 && in >= 16 &&
           in % 16 == 0 && in < kMaxSide && out < kMaxSide && out * (in / 16) < kInt32;
}

nvfp4_status check_matrix(const nvfp4_matrix* m) {
    if (m == nullptr) return NVFP4_ERR_NULL;
    if (!sizes_ok(0, m->batch, m->out, m->in)) return NVFP4_ERR_SHAPE;
    if (m->batch > 1 && (m->stride < m->out * m->in || !span_ok(m->batch, m->stride))) return NVFP4_ERR_SHAPE;
    if (m->batch == 0) return NVFP4_OK;
    if (m->packed == nullptr || m->scales == nullptr || m->S == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(m->packed, 8) || !aligned(m->S, 4) || (m->batch > 1 && m->stride % 16 != 0))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// What every call needs: the type, one or two matrices of one shape, the activation, the rows.
nvfp4_status check_call(int dtype, const nvfp4_matrix* w, const nvfp4_matrix* w2, bool two, int activation,
                        int64_t tokens, const int64_t* seg, bool backward) {
    if (elem_size(dtype) == 0) return NVFP4_ERR_DTYPE;
    nvfp4_status st = check_matrix(w);
    if (st != NVFP4_OK) return st;
    if (two) {
        st = check_matrix(w2);
        if (st != NVFP4_OK) return st;
        if (w->batch != w2->batch || w->out != w2->out || w->in != w2->in) return NVFP4_ERR_SHAPE;
    }
    if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_RELU) return NVFP4_ERR_ARG;
    if (!sizes_ok(tokens, w->batch, w->out, w->in)) return NVFP4_ERR_SHAPE;
    // a launch has fewer than 2^32 threads: one per 8 values of a row or per bias, and the product's own
    const int64_t pieces = ((w->out > w->in ? w->out : w->in) + 7) / 8;
    if (tokens * pieces > kThreads32 || w->batch * w->out > kThreads32 ||
        nvfp4::product_plan(tokens, w->batch, w->out, w->in, two ? 2 : 1, backward,
                            dtype == NVFP4_DTYPE_F32).threads > kThreads32)
        return NVFP4_ERR_SHAPE;
    if (seg == nullptr && w->batch != 1) return NVFP4_ERR_NULL;
    if (!aligned(seg, 8)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Rows [tokens, cols] of row stride ld; `to`: the bytes that rows are aligned to (16: a product reads them as they are).
nvfp4_status check_rows(const void* p, int esz, int64_t tokens, int64_t cols, int64_t ld, int64_t to) {
    if (ld < cols || !span_ok(tokens, ld) || (to == 16 && ld >= kMaxSide)) return NVFP4_ERR_SHAPE;
    if (p == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(p, to) || (tokens > 1 && ld * esz % to != 0)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4_status hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

nvfp4::ProductMatrix view_of(const nvfp4_matrix* m) {
    return nvfp4::ProductMatrix{m->packed, m->scales, m->S, m->batch > 1 ? m->stride : 0};
}

// Workspace: the operands' parts, where the rows given are not bf16 rows of whole 16-byte pieces, the sums of the
// shares of a product's reduction, the map of its tiles of rows, and the sums of a bias gradient.
struct Space {
    bool parts;
    int planes;
    int64_t ld, plane;       // elements
    size_t operand;          // bytes of one operand
    size_t partial, map, bias;
    size_t total;
};
Space space_of(int dtype, int64_t tokens, int64_t batch, int64_t out, int64_t in, int32_t matrices, bool backward,
               bool with_bias) {
    Space s;
    const int64_t cols = backward ? out : in;
    const bool f32 = dtype == NVFP4_DTYPE_F32;
    s.planes = f32 ? 3 : 1;
    s.parts = f32 || cols % 8 != 0;
    s.ld = up(cols, 8);
    s.plane = tokens * s.ld;
    s.operand = s.parts ? (size_t)up(s.planes * s.plane * 2, 256) : 0;
    const nvfp4::ProductPlan plan = nvfp4::product_plan(tokens, batch, out, in, matrices, backward, f32);
    s.partial = (size_t)up((int64_t)nvfp4::product_partial_bytes(plan, tokens, out, in, matrices, backward), 256);
    s.map = (size_t)up((int64_t)nvfp4::product_map_bytes(plan, tokens, batch), 256);
    s.bias = with_bias ? nvfp4::product_bias_workspace_bytes(tokens, batch, out) : 0;
    s.total = s.operand * (backward ? matrices : 1) + s.partial + s.map + s.bias;
    return s;
}

nvfp4_status check_workspace(size_t need, const void* ws, size_t bytes) {
    if (need > 0 && (ws == nullptr || bytes < need)) return NVFP4_ERR_WORKSPACE;
    return aligned(ws, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// The product's own part of the workspace, behind the operands.
void place_sums(nvfp4::Product& p, const Space& s, uint8_t* at) {
    p.partial = reinterpret_cast<float*>(at);
    p.rows.map = reinterpret_cast<nvfp4::RowTile*>(at + s.partial);
}

// The rows' side of a forward product: X itself, or its parts.
hipError_t forward_operand(nvfp4::Product& p, const Space& s, const void* X, int64_t ldx, void* workspace,
                           hipStream_t stream) {
    p.planes = s.planes;
    p.plane = s.plane;
    p.a[0] = nvfp4::ProductOperand{static_cast<const uint16_t*>(X), ldx};
    place_sums(p, s, static_cast<uint8_t*>(workspace) + s.operand);
    if (!s.parts) return hipSuccess;
    uint16_t* parts = static_cast<uint16_t*>(workspace);
    p.a[0] = nvfp4::ProductOperand{parts, s.ld};
    return nvfp4::launch_product_parts(X, p.f32, p.rows.tokens, p.in, ldx, parts, s.ld, s.plane, stream);
}

nvfp4::Product product_of(const nvfp4_matrix* w, const nvfp4_matrix* w2, bool backward, int dtype,
                          int64_t tokens, const int64_t* seg, int activation) {
    nvfp4::Product p = {};
    p.w[0] = view_of(w);
    if (w2) p.w[1] = view_of(w2);
    p.matrices = w2 ? 2 : 1;
    p.backward = backward;
    p.f32 = dtype == NVFP4_DTYPE_F32;
    p.out = w->out;
    p.in = w->in;
    p.rows = nvfp4::ProductRows{seg, tokens, (int32_t)w->batch, nullptr};
    p.act = activation;
    return p;
}

// Gradients of two or one matrices' outputs: the element-wise pass where it is needed, then the product.
nvfp4_status backward(nvfp4::Product& p, nvfp4::ProductSlopes& g, float* dbias, const Space& s, void* workspace,
                      hipStream_t stream) {
    p.planes = s.planes;
    p.plane = s.plane;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    place_sums(p, s, ws + p.matrices * s.operand);
    for (int m = 0; m < p.matrices; ++m) {
        if (s.parts) {
            g.parts[m] = reinterpret_cast<uint16_t*>(ws + m * s.operand);
            p.a[m] = nvfp4::ProductOperand{g.parts[m], s.ld};
        } else {
            const bool as_given = g.Z == nullptr;
            p.a[m] = nvfp4::ProductOperand{static_cast<const uint16_t*>(as_given ? g.dY : g.d[m]),
                                           as_given ? g.lddy : g.ldd[m]};
        }
    }
    g.ld = s.ld;
    g.plane = s.plane;
    const bool slopes = p.rows.tokens > 0 && (s.parts || g.Z);
    if (slopes || dbias) {
        void* sums = ws + p.matrices * s.operand + s.partial + s.map;
        if (nvfp4::launch_product_slopes(g, slopes, dbias, sums, stream) != hipSuccess) return NVFP4_ERR_HIP;
    }
    return p.rows.tokens > 0 ? hip_status(nvfp4::launch_product(p, stream)) : NVFP4_OK;
}

}  // namespace

extern "C" {

size_t nvfp4_linear_workspace_size(int dtype, int64_t tokens, int64_t batch, int64_t out, int64_t in) {
    if (elem_size(dtype) == 0 || !sizes_ok(tokens, batch, out, in)) return 0;
    return space_of(dtype, tokens, batch, out, in, 1, false, false).total;
}

nvfp4_status nvfp4_linear(const nvfp4_matrix* W, const void* X, int dtype, int64_t tokens, int64_t ldx,
                          const int64_t* seg_offsets, const void* bias, int activation,
                          const void* residual, int64_t ldr, void* Z, int64_t ldz, void* Y, int64_t ldy,
                          void* workspace, size_t workspace_bytes, void* stream) {
    nvfp4_status st = check_call(dtype, W, nullptr, false, activation, tokens, seg_offsets, false);
    if (st != NVFP4_OK) return st;
    if (tokens == 0 || W->batch == 0) return NVFP4_OK;
    const int esz = elem_size(dtype);
    st = check_rows(X, esz, tokens, W->in, ldx, 16);
    if (st == NVFP4_OK && residual) st = check_rows(residual, esz, tokens, W->out, ldr, esz);
    if (st == NVFP4_OK && Z) st = check_rows(Z, esz, tokens, W->out, ldz, esz);
    if (st == NVFP4_OK) st = check_rows(Y, esz, tokens, W->out, ldy, esz);
    if (st != NVFP4_OK) return st;
    if (!aligned(bias, esz)) return NVFP4_ERR_ALIGN;
    const Space s = space_of(dtype, tokens, W->batch, W->out, W->in, 1, false, false);
    st = check_workspace(s.total, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    nvfp4::Product p = product_of(W, nullptr, false, dtype, tokens, seg_offsets, activation);
    p.bias = bias;
    p.residual = residual;
    p.ldr = ldr;
    p.pre[0] = Z;
    p.ldpre[0] = ldz;
    p.y = Y;
    p.ldy = ldy;
    const hipStream_t on = static_cast<hipStream_t>(stream);
    if (forward_operand(p, s, X, ldx, workspace, on) != hipSuccess) return NVFP4_ERR_HIP;
    return hip_status(nvfp4::launch_product(p, on));
}

size_t nvfp4_gated_workspace_size(int dtype, int64_t tokens, int64_t batch, int64_t out, int64_t in) {
    if (elem_size(dtype) == 0 || !sizes_ok(tokens, batch, out, in)) return 0;
    return space_of(dtype, tokens, batch, out, in, 2, false, false).total;
}

nvfp4_status nvfp4_gated(const nvfp4_matrix* W_gate, const nvfp4_matrix* W_up, const void* X, int dtype,
                         int64_t tokens, int64_t ldx, const int64_t* seg_offsets, int activation, void* G,
                         int64_t ldg, void* U, int64_t ldu, void* H, int64_t ldh, void* workspace,
                         size_t workspace_bytes, void* stream) {
    nvfp4_status st = check_call(dtype, W_gate, W_up, true, activation, tokens, seg_offsets, false);
    if (st != NVFP4_OK) return st;
    if ((G == nullptr) != (U == nullptr)) return NVFP4_ERR_NULL;
    if (tokens == 0 || W_gate->batch == 0) return NVFP4_OK;
    const int esz = elem_size(dtype);
    const int64_t out = W_gate->out;
    st = check_rows(X, esz, tokens, W_gate->in, ldx, 16);
    if (st == NVFP4_OK && G) st = check_rows(G, esz, tokens, out, ldg, esz);
    if (st == NVFP4_OK && U) st = check_rows(U, esz, tokens, out, ldu, esz);
    if (st == NVFP4_OK) st = check_rows(H, esz, tokens, out, ldh, esz);
    if (st != NVFP4_OK) return st;
    const Space s = space_of(dtype, tokens, W_gate->batch, out, W_gate->in, 2, false, false);
    st = check_workspace(s.total, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    nvfp4::Product p = product_of(W_gate, W_up, false, dtype, tokens, seg_offsets, activation);
    p.pre[0] = G;
    p.ldpre[0] = ldg;
    p.pre[1] = U;
    p.ldpre[1] = ldu;
    p.y = H;
    p.ldy = ldh;
    const hipStream_t on = static_cast<hipStream_t>(stream);
    if (forward_operand(p, s, X, ldx, workspace, on) != hipSuccess) return NVFP4_ERR_HIP;
    return hip_status(nvfp4::launch_product(p, on));
}

size_t nvfp4_linear_backward_workspace_size(int dtype, int64_t tokens, int64_t batch, int64_t out,
                                            int64_t in, int with_bias) {
    if (elem_size(dtype) == 0 || !sizes_ok(tokens, batch, out, in)) return 0;
    return space_of(dtype, tokens, batch, out, in, 1, true, with_bias != 0).total;
}

nvfp4_status nvfp4_linear_backward(const nvfp4_matrix* W, const void* dY, int dtype, int64_t tokens,
                                   int64_t lddy, const int64_t* seg_offsets, int activation,
                                   const void* Z, int64_t ldz, void* dZ, int64_t lddz, float* dbias,
                                   void* dX, int64_t lddx, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    nvfp4_status st = check_call(dtype, W, nullptr, false, activation, tokens, seg_offsets, true);
    if (st != NVFP4_OK) return st;
    if (W->batch == 0) return NVFP4_OK;
    const int esz = elem_size(dtype);
    const bool act = activation != NVFP4_ACT_NONE;
    const Space s = space_of(dtype, tokens, W->batch, W->out, W->in, 1, true, dbias != nullptr);
    if (tokens > 0) {
        // the product reads dY, or dZ, as they are where no parts are made
        st = check_rows(dY, esz, tokens, W->out, lddy, !act && !s.parts ? 16 : esz);
        if (st == NVFP4_OK && act) st = check_rows(Z, esz, tokens, W->out, ldz, esz);
        if (st == NVFP4_OK && act) st = check_rows(dZ, esz, tokens, W->out, lddz, s.parts ? esz : 16);
        if (st == NVFP4_OK) st = check_rows(dX, esz, tokens, W->in, lddx, esz);
        if (st != NVFP4_OK) return st;
    }
    if (!aligned(dbias, 4)) return NVFP4_ERR_ALIGN;
    if (dbias && W->batch * W->out > kMaxBiases) return NVFP4_ERR_SHAPE;
    st = check_workspace(s.total, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    nvfp4::ProductSlopes g = {};
    g.rows = nvfp4::ProductRows{seg_offsets, tokens, (int32_t)W->batch, nullptr};
    g.f32 = dtype == NVFP4_DTYPE_F32;
    g.cols = W->out;
    g.act = activation;
    g.dY = dY;
    g.lddy = lddy;
    g.Z = act ? Z : nullptr;
    g.ldz = ldz;
    g.d[0] = act ? dZ : nullptr;
    g.ldd[0] = lddz;
    nvfp4::Product p = product_of(W, nullptr, true, dtype, tokens, seg_offsets, NVFP4_ACT_NONE);
    p.y = dX;
    p.ldy = lddx;
    return backward(p, g, dbias, s, workspace, static_cast<hipStream_t>(stream));
}

size_t nvfp4_gated_backward_workspace_size(int dtype, int64_t tokens, int64_t batch, int64_t out,
                                           int64_t in) {
    if (elem_size(dtype) == 0 || !sizes_ok(tokens, batch, out, in)) return 0;
    return space_of(dtype, tokens, batch, out, in, 2, true, false).total;
}

nvfp4_status nvfp4_gated_backward(const nvfp4_matrix* W_gate, const nvfp4_matrix* W_up, const void* dH,
                                  int dtype, int64_t tokens, int64_t lddh, const int64_t* seg_offsets,
                                  int activation, const void* G, int64_t ldg, const void* U, int64_t ldu,
                                  void* dG, int64_t lddg, void* dU, int64_t lddu, void* dX, int64_t lddx,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    nvfp4_status st = check_call(dtype, W_gate, W_up, true, activation, tokens, seg_offsets, true);
    if (st != NVFP4_OK) return st;
    if (tokens == 0 || W_gate->batch == 0) return NVFP4_OK;
    const int esz = elem_size(dtype);
    const int64_t out = W_gate->out;
    const Space s = space_of(dtype, tokens, W_gate->batch, out, W_gate->in, 2, true, false);
    const int64_t to = s.parts ? esz : 16;               // the product reads dG and dU where no parts are made
    st = check_rows(dH, esz, tokens, out, lddh, esz);
    if (st == NVFP4_OK) st = check_rows(G, esz, tokens, out, ldg, esz);
    if (st == NVFP4_OK) st = check_rows(U, esz, tokens, out, ldu, esz);
    if (st == NVFP4_OK) st = check_rows(dG, esz, tokens, out, lddg, to);
    if (st == NVFP4_OK) st = check_rows(dU, esz, tokens, out, lddu, to);
    if (st == NVFP4_OK) st = check_rows(dX, esz, tokens, W_gate->in, lddx, esz);
    if (st != NVFP4_OK) return st;
    if (!s.parts && lddg != lddu) return NVFP4_ERR_SHAPE;
    st = check_workspace(s.total, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    nvfp4::ProductSlopes g = {};
    g.rows = nvfp4::ProductRows{seg_offsets, tokens, (int32_t)W_gate->batch, nullptr};
    g.f32 = dtype == NVFP4_DTYPE_F32;
    g.cols = out;
    g.act = activation;
    g.dY = dH;
    g.lddy = lddh;
    g.Z = G;
    g.ldz = ldg;
    g.U = U;
    g.ldu = ldu;
    g.d[0] = dG;
    g.ldd[0] = lddg;
    g.d[1] = dU;
    g.ldd[1] = lddu;
    nvfp4::Product p = product_of(W_gate, W_up, true, dtype, tokens, seg_offsets, NVFP4_ACT_NONE);
    p.y = dX;
    p.ldy = lddx;
    return backward(p, g, nullptr, s, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
