// Attention over the paged NVFP4 key/value cache for gfx950: one wave per (token row, query head),
// 64 positions at a time with a running maximum and sum. Each lane scores one position; the
// weighted values are then summed with each lane owning dim / 64 columns.
#include <hip/hip_runtime.h>

#include "device_formats.h"
#include "kv_cache.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const float m = (c & 7u) < 2u ? 0.5f * (float)(c & 7u)
                                  : (1.0f + 0.5f * (float)(c & 1u)) * (float)(1u << (((c >> 1) & 3u) - 1u));
    return (c & 8u) ? -m : m;
}

template <bool BF16>
__device__ __forceinline__ float load_element(const uint8_t* p, int d) {
    if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(p)[d]);
    else return reinterpret_cast<const float*>(p)[d];
}

template <bool BF16, int D>
__global__ __launch_bounds__(64) void k_kv_attention(KvAttention a) {
    __shared__ float q[D], prob[64];
    __shared__ int where[64];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int head_q = blockIdx.y;
    const KvView& kv = a.kv;
    const int head = head_q / (a.q_heads / kv.heads);
    if (t >= min((int64_t)a.b.cu[a.b.seqs], a.b.tokens)) return;
    const int item = kv_find_item(a.b.cu, a.b.seqs, t);
    const KvItem it = kv_item(kv, a.b, item);
    if (t - a.b.cu[item] >= a.max_q) return;
    const int64_t pos = (int64_t)it.len - ((int64_t)a.b.cu[item + 1] - t);
    int64_t end = min(it.len, a.max_kv);
    if (a.causal) end = min(end, pos + 1);
    const int64_t begin = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
    const uint8_t* qp = static_cast<const uint8_t*>(a.q.p) + t * a.q.stride_t + head_q * a.q.stride_h;
    for (int d = lane; d < D; d += 64) q[d] = load_element<BF16>(qp, d);
    __syncthreads();
    const int64_t half = kv_code_bytes(kv);
    float m = -__builtin_inff(), l = 0.0f, acc[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) acc[i] = 0.0f;
    const float f = a.scale * kv.S_k[head];
    for (int64_t p0 = begin; p0 < end; p0 += 64) {
        const int64_t p = p0 + lane;
        int page = -1, row = 0;
        float s = -__builtin_inff();
        if (p < end) {
            page = kv_page(kv, it.slot, (int)(p / kv.page));
            row = (int)(p % kv.page);
        }
        if (page >= 0) {
            const uint8_t* rec = kv.pages + (int64_t)page * kv.page_stride;
            const uint8_t* code = rec + ((int64_t)head * kv.page + row) * (D / 2);
            const uint8_t* sc = rec + 2 * half + ((int64_t)head * kv.page + row) * (D / 16);
            float dot = 0.0f;
            for (int g = 0; g < D / 16; ++g) {
                const float e = e4m3_value(sc[g] & 127);
                for (int d = 16 * g; d < 16 * g + 16; ++d) {
                    const uint32_t c = (code[d >> 1] >> (4 * (d & 1))) & 15u;
                    dot = __builtin_fmaf(q[d], e2m1_value(c) * e, dot);
                }
            }
            s = dot * f;
        }
        float top = s;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        if (top == -__builtin_inff()) continue;
        const float mn = fmaxf(m, top);
        const float al = __expf(m - mn), pr = __expf(s - mn);
        float sum = pr;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
        l = l * al + sum;
        m = mn;
        __syncthreads();
        prob[lane] = pr;
        where[lane] = page;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < D / 64; ++i) acc[i] *= al;
        for (int j = 0; j < 64; ++j) {
            if (where[j] < 0) continue;
            const uint8_t* rec = kv.pages + (int64_t)where[j] * kv.page_stride;
            const int64_t r = (int64_t)head * kv.page + (p0 + j) % kv.page;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int d = lane + 64 * i, n = d / (D / 16), e = d % (D / 16);
                const uint32_t b = rec[half + (((r >> 2) * 16 + n) * 4 + (r & 3)) * (D / 32) + (e >> 1)];
                const float sc = e4m3_value(rec[2 * half + (half >> 3) +
                                                ((r >> 2) * (D / 16) + d / 16) * 4 + (r & 3)] & 127);
                acc[i] = __builtin_fmaf(prob[j], e2m1_value((b >> (4 * (e & 1))) & 15u) * sc, acc[i]);
            }
        }
    }
    const float inv = l > 0.0f ? kv.S_v[head] / l : 0.0f;
    uint8_t* o = static_cast<uint8_t*>(a.out) + t * a.out_stride_t + head_q * a.out_stride_h;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const float v = acc[i] * inv;
        const int d = lane + 64 * i;
        if constexpr (BF16) {
            const uint32_t u = __float_as_uint(v);
            reinterpret_cast<uint16_t*>(o)[d] = (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
        } else {
            reinterpret_cast<float*>(o)[d] = v;
        }
    }
    if (a.lse && lane == 0) a.lse[t * a.q_heads + head_q] = m + __logf(l);
}

template <bool BF16>
void launch(const KvAttention& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.b.tokens, (uint32_t)a.q_heads);
    if (a.kv.dim == 64)
        hipLaunchKernelGGL((k_kv_attention<BF16, 64>), grid, dim3(64), 0, stream, a);
    else if (a.kv.dim == 128)
        hipLaunchKernelGGL((k_kv_attention<BF16, 128>), grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL((k_kv_attention<BF16, 256>), grid, dim3(64), 0, stream, a);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t, int64_t, bool, int64_t, int64_t, int64_t, int64_t,
                                    int64_t) {
    return 0;
}

hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream) {
    if (a.bf16) launch<true>(a, stream);
    else launch<false>(a, stream);
    return hipGetLastError();
}

}  // namespace nvfp4
