// The paged NVFP4 key/value cache as the kernels see it: one layer's records, the page table, and
// where a position's codes and scale bytes lie (layout in include/nvfp4.h). Launchers of the
// cache's calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

struct KvView {
    uint8_t* pages;          // the layer's records
    int64_t page_stride;
    int32_t num_pages;
    int32_t heads, dim, page;
    int32_t max_slots, max_pages;
    const int32_t* table;
    const int32_t* lens;
    const float* S_k;        // [heads] of the layer
    const float* S_v;
};

inline int64_t kv_record_bytes(int64_t heads, int64_t dim, int64_t page) {
    return heads * page * dim * 9 / 8;
}

// The token tensors' split into items: rows cu[i] .. cu[i+1] - 1 of slot slots[i] (or i).
struct KvBatch {
    const int32_t* cu;
    const int32_t* slots;
    int32_t seqs;
    int64_t tokens;
};

struct KvTokens {            // [tokens, heads, dim] with byte strides
    const void* p;
    int64_t stride_t, stride_h;
};

hipError_t launch_kv_append(const KvView& kv, const KvTokens& K, const KvTokens& V, bool bf16,
                            const KvBatch& b, int lo, int hi, hipStream_t stream);
hipError_t launch_kv_read(const KvView& kv, void* K, void* V, bool bf16, const KvBatch& b,
                          hipStream_t stream);

struct KvAttention {
    KvView kv;
    KvBatch b;
    KvTokens q;
    bool bf16;
    int32_t q_heads;
    int32_t max_q, max_kv;
    float scale;
    bool causal;
    int32_t window;          // 0: none
    void* out;
    int64_t out_stride_t, out_stride_h;   // bytes
    float* lse;              // or null
    void* workspace;
};
// Whether such a batch fits one launch.
bool kv_attention_fits(int64_t heads, int64_t dim, int64_t tokens, int64_t q_heads, int64_t seqs,
                       int64_t max_q, int64_t max_kv);
size_t kv_attention_workspace_bytes(int64_t heads, int64_t dim, int64_t tokens, int64_t q_heads,
                                    int64_t seqs, int64_t max_q, int64_t max_kv);
hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream);

struct KvPool {              // all layers, for the page calls
    uint8_t* pages;
    int64_t layers, layer_stride, page_stride, record;
    int32_t num_pages, page, max_slots, max_pages;
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
};
size_t kv_pages_workspace_bytes(int64_t num_pages, int64_t n);
hipError_t launch_kv_reserve(const KvPool& p, const int32_t* slots, const int32_t* counts,
                             int32_t n, int32_t* status, void* workspace, hipStream_t stream);
hipError_t launch_kv_fork(const KvPool& p, const int32_t* parents, const int32_t* children,
                          int32_t n, int32_t* status, void* workspace, hipStream_t stream);
hipError_t launch_kv_free(const KvPool& p, const int32_t* slots, int32_t n, int32_t* status,
                          hipStream_t stream);
hipError_t launch_kv_compact(const KvPool& p, int32_t* used, void* workspace, hipStream_t stream);

#ifdef __HIPCC__

// Byte offsets of the V region and of the two scale regions in a record.
__device__ __forceinline__ int64_t kv_code_bytes(const KvView& kv) {
    return (int64_t)kv.heads * kv.page * (kv.dim >> 1);
}

// Slot of item i and its length, clamped to what the table can hold; 0 for a slot outside it and for a
// cache without pages.
struct KvItem {
    int32_t slot, len;
};
__device__ __forceinline__ KvItem kv_item(const KvView& kv, const KvBatch& b, int i) {
    KvItem it;
    it.slot = b.slots ? b.slots[i] : i;
    const bool ok = (uint32_t)it.slot < (uint32_t)kv.max_slots && kv.num_pages > 0;
    it.slot = ok ? it.slot : 0;
    const int32_t cap = kv.max_pages * kv.page;
    it.len = ok ? min(max(kv.lens[it.slot], 0), cap) : 0;
    return it;
}

// Page of a position (pos in 0 .. len - 1), -1 if the table names none.
__device__ __forceinline__ int kv_page(const KvView& kv, int slot, int col) {
    const int p = kv.table[(int64_t)slot * kv.max_pages + col];
    return (uint32_t)p < (uint32_t)kv.num_pages ? p : -1;
}

// The item of token row t: the largest i with cu[i] <= t, found by the whole wave for one t (64 probes
// a round). Terminates whatever cu holds.
__device__ __forceinline__ int kv_find_item(const int32_t* __restrict__ cu, int seqs, int64_t t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int64_t k = lo + (int64_t)(lane + 1) * step;
        const bool below = k < hi && (int64_t)cu[k] <= t;
        const int cnt = __popcll(__ballot(below));
        lo += cnt * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Two values rounded to bf16, to nearest even, a in the low half; NaN of any bits stays NaN. The hardware's
// conversion: for all 2^32 values the bits of rounding by integer steps (NaN aside), which takes several
// instructions a value (a read of 4108 rows 9.6 us, with the conversion 8.8).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef float f32_pair __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16_pair_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32_pair{a, b}), bf16_pair_t));
}

#endif  // __HIPCC__

}  // namespace nvfp4
