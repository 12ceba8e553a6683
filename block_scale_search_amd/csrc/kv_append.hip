// Tokens into and out of the paged NVFP4 key/value cache for gfx950.
//
// Append: the group search of search_device.h (MSE, a window around the max-abs code) on each
// group of 16 values, one lane a group, a workgroup within one head of K or V so that S and the
// code table in LDS are the workgroup's own. Read: the inverse, value = S * (level * E4M3), one lane
// a group. Both move one group's codes as 8 bytes: contiguous in the K region, as 16 / (D/16) pieces
// in the V region, where four tokens' pieces of the same values lie side by side.
//
// What bounds append is vector arithmetic: 11 candidates a value. 4106 rows of 8 heads, 128 wide, bf16:
// 20.8 us, 4.0e11 values/s (1.0 TB/s of rows read and codes written); one row of each of 128 slots 6.9 us,
// a launch and the chain offset, length, page, store. Read has that chain too, 4.2 us for 128 rows, and then its
// bytes, in one round of workgroups: 8.8 us for 4108 rows, 2.4 TB/s.
#include <hip/hip_runtime.h>

#include "device_formats.h"
#include "kv_cache.h"
#include "search_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

// A lane's group: token row t, position in the cache, group of the head. `page` < 0: none.
struct Place {
    int64_t t;
    int32_t page, row;       // page of the cache, row in the page
    int g;
    bool valid;              // t is a row of the batch
};

// Flat group index -> token row and position. GPH = dim / 16 groups a head row. The rows of a wave are
// few (64 / GPH), so their items come from one search and a window of the next 64 offsets.
template <int GPH>
__device__ __forceinline__ Place place_of(const KvView& kv, const KvBatch& b) {
    constexpr int ROWS = 64 / GPH;
    const int lane = threadIdx.x & 63;
    const int64_t flat = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t0 = ((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~63)) / GPH;
    Place p;
    p.t = flat / GPH;
    p.g = (int)(flat % GPH);
    const int64_t total = min((int64_t)b.cu[b.seqs], b.tokens);
    p.valid = p.t < total;
    p.page = -1;
    p.row = 0;
    if (t0 >= total) return p;               // the whole wave
    const int first = kv_find_item(b.cu, b.seqs, t0);
    const int64_t next = b.cu[min(first + 1 + lane, b.seqs)];
    int item = first;
    for (int r = 0; r < ROWS; ++r) {
        const int64_t t = t0 + r;
        int at = first + __popcll(__ballot(first + 1 + lane < b.seqs && next <= t));
        if (at == first + 64) at = kv_find_item(b.cu, b.seqs, t);   // uniform: at is the wave's
        if (p.t == t) item = at;
    }
    const KvItem it = kv_item(kv, b, item);
    const int64_t pos = (int64_t)it.len - ((int64_t)b.cu[item + 1] - p.t);
    if (p.valid && pos >= 0 && pos < it.len) {
        const int col = (int)pos / kv.page;
        p.page = kv_page(kv, it.slot, col);
        p.row = (int)pos - col * kv.page;
    }
    return p;
}

// Piece i of a group's 8 code bytes in the V region: PIECE = dim / 32 bytes each, for n = g * NP + i.
template <int GPH>
struct VPiece {
    static constexpr int bytes = GPH / 2, count = 16 / GPH;
};

template <int GPH>
__device__ __forceinline__ int64_t v_offset(const KvView& kv, int head, int row, int n) {
    return (((int64_t)head * (kv.page >> 2) + (row >> 2)) * 16 + n) * (4 * VPiece<GPH>::bytes) +
           (row & 3) * VPiece<GPH>::bytes;
}

template <int GPH>
__device__ __forceinline__ void store_v(uint8_t* v, const KvView& kv, int head, int row, int g,
                                        uint32_t lo, uint32_t hi) {
    constexpr int NP = VPiece<GPH>::count;
    if constexpr (GPH == 16) {
        *reinterpret_cast<uint2*>(v + v_offset<GPH>(kv, head, row, g)) = make_uint2(lo, hi);
    } else if constexpr (GPH == 8) {
        *reinterpret_cast<uint32_t*>(v + v_offset<GPH>(kv, head, row, g * NP)) = lo;
        *reinterpret_cast<uint32_t*>(v + v_offset<GPH>(kv, head, row, g * NP + 1)) = hi;
    } else {
        const uint32_t w[2] = {lo, hi};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint16_t*>(v + v_offset<GPH>(kv, head, row, g * NP + i)) =
                (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

template <int GPH>
__device__ __forceinline__ uint2 load_v(const uint8_t* v, const KvView& kv, int head, int row,
                                        int g) {
    constexpr int NP = VPiece<GPH>::count;
    if constexpr (GPH == 16) {
        return *reinterpret_cast<const uint2*>(v + v_offset<GPH>(kv, head, row, g));
    } else if constexpr (GPH == 8) {
        return make_uint2(
            *reinterpret_cast<const uint32_t*>(v + v_offset<GPH>(kv, head, row, g * NP)),
            *reinterpret_cast<const uint32_t*>(v + v_offset<GPH>(kv, head, row, g * NP + 1)));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint16_t*>(v + v_offset<GPH>(kv, head, row, g * NP + i));
        return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
}

// Address of the scale byte of group g in a record's scale region (V: four tokens together).
template <int GPH>
__device__ __forceinline__ int64_t scale_offset(const KvView& kv, bool is_v, int head, int row,
                                                int g) {
    const int64_t r = (int64_t)head * kv.page + row;
    return is_v ? ((r >> 2) * GPH + g) * 4 + (r & 3) : r * GPH + g;
}

template <bool BF16, int GPH, int NWIN>
__global__ __launch_bounds__(kThreads) void k_kv_append(KvView kv, KvTokens K, KvTokens V,
                                                        KvBatch b, int lo, int hi) {
    __shared__ float2 tab[128];
    __shared__ int flag;
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const Place p = place_of<GPH>(kv, b);
    const KvTokens x = is_v ? V : K;
    float w[16], h[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = h[j] = 0.0f;
    if (p.valid) {
        const uint8_t* src = static_cast<const uint8_t*>(x.p) + p.t * x.stride_t +
                             head * x.stride_h + p.g * (BF16 ? 32 : 64);
        if constexpr (BF16) {
            const uint4 a = reinterpret_cast<const uint4*>(src)[0];
            const uint4 c = reinterpret_cast<const uint4*>(src)[1];
            const uint32_t d[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[2 * i] = bf16_lo(d[i]);
                w[2 * i + 1] = bf16_hi(d[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = reinterpret_cast<const float4*>(src)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    }
    const float S = (is_v ? kv.S_v : kv.S_k)[head];
    const bool octave_ok = build_table(S, tab, &flag);
    const int base = base_code(w, S);
    const bool live = p.page >= 0 && base > 0;
    float best = __builtin_inff();
    int code = min(max(base + lo, 1), 126);
    search_window<false, NWIN>(w, h, tab, octave_ok, live, base + lo, hi - lo + 1, best, code);
    if (p.page < 0) return;
    if (!live) code = 0;
    const float r = tab[code].y;             // 0 for code 0: signed zero codes
    uint32_t c0 = 0u, c1 = 0u;
    c0 = e2m1_pack2<0>(c0, w[0] * r, w[1] * r);
    c0 = e2m1_pack2<1>(c0, w[2] * r, w[3] * r);
    c0 = e2m1_pack2<2>(c0, w[4] * r, w[5] * r);
    c0 = e2m1_pack2<3>(c0, w[6] * r, w[7] * r);
    c1 = e2m1_pack2<0>(c1, w[8] * r, w[9] * r);
    c1 = e2m1_pack2<1>(c1, w[10] * r, w[11] * r);
    c1 = e2m1_pack2<2>(c1, w[12] * r, w[13] * r);
    c1 = e2m1_pack2<3>(c1, w[14] * r, w[15] * r);
    const int64_t half = kv_code_bytes(kv);
    uint8_t* rec = kv.pages + (int64_t)p.page * kv.page_stride;
    if (is_v) {
        store_v<GPH>(rec + half, kv, head, p.row, p.g, c0, c1);
    } else {
        reinterpret_cast<uint2*>(rec + ((int64_t)head * kv.page + p.row) * (8 * GPH))[p.g] =
            make_uint2(c0, c1);
    }
    rec[2 * half + (is_v ? half >> 3 : 0) + scale_offset<GPH>(kv, is_v, head, p.row, p.g)] =
        (uint8_t)code;
}

template <bool BF16, int GPH>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvView kv, uint8_t* __restrict__ K,
                                                      uint8_t* __restrict__ V, KvBatch b) {
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const float S_head = (is_v ? kv.S_v : kv.S_k)[head];  // beside the look-up, not behind it
    const Place p = place_of<GPH>(kv, b);
    if (!p.valid) return;
    uint2 c = make_uint2(0u, 0u);
    float e = 0.0f;
    if (p.page >= 0) {
        const int64_t half = kv_code_bytes(kv);
        const uint8_t* rec = kv.pages + (int64_t)p.page * kv.page_stride;
        c = is_v ? load_v<GPH>(rec + half, kv, head, p.row, p.g)
                 : reinterpret_cast<const uint2*>(
                       rec + ((int64_t)head * kv.page + p.row) * (8 * GPH))[p.g];
        const int s = rec[2 * half + (is_v ? half >> 3 : 0) +
                          scale_offset<GPH>(kv, is_v, head, p.row, p.g)];
        e = e4m3_value(s & 127);
    }
    const float S = p.page >= 0 ? S_head : 0.0f;         // zeros where nothing is cached, whatever S is
    float v[16];
    e2m1_levels2<0>(c.x, v[0], v[1]);
    e2m1_levels2<1>(c.x, v[2], v[3]);
    e2m1_levels2<2>(c.x, v[4], v[5]);
    e2m1_levels2<3>(c.x, v[6], v[7]);
    e2m1_levels2<0>(c.y, v[8], v[9]);
    e2m1_levels2<1>(c.y, v[10], v[11]);
    e2m1_levels2<2>(c.y, v[12], v[13]);
    e2m1_levels2<3>(c.y, v[14], v[15]);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = (v[j] * e) * S;
    uint8_t* dst = (is_v ? V : K) +
                   ((p.t * kv.heads + head) * GPH + p.g) * (int64_t)(BF16 ? 32 : 64);
    if constexpr (BF16) {
        uint32_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(d[0], d[1], d[2], d[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(d[4], d[5], d[6], d[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(dst)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

dim3 grid_of(const KvView& kv, const KvBatch& b) {
    const int64_t groups = b.tokens * (kv.dim / 16);
    return dim3((uint32_t)((groups + kThreads - 1) / kThreads), (uint32_t)kv.heads, 2);
}

template <bool BF16, int GPH>
void append(const KvView& kv, const KvTokens& K, const KvTokens& V, const KvBatch& b, int lo, int hi,
            hipStream_t stream) {
    // the window of 11 codes (offsets -3 .. 7) is unrolled, as the search's own launches do
    if (hi - lo + 1 == 11)
        hipLaunchKernelGGL((k_kv_append<BF16, GPH, 11>), grid_of(kv, b), dim3(kThreads), 0, stream,
                           kv, K, V, b, lo, hi);
    else
        hipLaunchKernelGGL((k_kv_append<BF16, GPH, 0>), grid_of(kv, b), dim3(kThreads), 0, stream, kv,
                           K, V, b, lo, hi);
}

template <bool BF16>
void append_dim(const KvView& kv, const KvTokens& K, const KvTokens& V, const KvBatch& b, int lo,
                int hi, hipStream_t stream) {
    if (kv.dim == 64) append<BF16, 4>(kv, K, V, b, lo, hi, stream);
    else if (kv.dim == 128) append<BF16, 8>(kv, K, V, b, lo, hi, stream);
    else append<BF16, 16>(kv, K, V, b, lo, hi, stream);
}

template <bool BF16>
void read_dim(const KvView& kv, uint8_t* K, uint8_t* V, const KvBatch& b, hipStream_t stream) {
    const dim3 grid = grid_of(kv, b);
    if (kv.dim == 64)
        hipLaunchKernelGGL((k_kv_read<BF16, 4>), grid, dim3(kThreads), 0, stream, kv, K, V, b);
    else if (kv.dim == 128)
        hipLaunchKernelGGL((k_kv_read<BF16, 8>), grid, dim3(kThreads), 0, stream, kv, K, V, b);
    else
        hipLaunchKernelGGL((k_kv_read<BF16, 16>), grid, dim3(kThreads), 0, stream, kv, K, V, b);
}

}  // namespace

hipError_t launch_kv_append(const KvView& kv, const KvTokens& K, const KvTokens& V, bool bf16,
                            const KvBatch& b, int lo, int hi, hipStream_t stream) {
    if (bf16) append_dim<true>(kv, K, V, b, lo, hi, stream);
    else append_dim<false>(kv, K, V, b, lo, hi, stream);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvView& kv, void* K, void* V, bool bf16, const KvBatch& b,
                          hipStream_t stream) {
    uint8_t* k = static_cast<uint8_t*>(K);
    uint8_t* v = static_cast<uint8_t*>(V);
    if (bf16) read_dim<true>(kv, k, v, b, stream);
    else read_dim<false>(kv, k, v, b, stream);
    return hipGetLastError();
}

}  // namespace nvfp4
