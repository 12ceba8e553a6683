// Page bookkeeping of the paged key/value cache for gfx950: reserve, fork, free and compact change the
// page table, the lengths and the reference counts on the device.
//
// The bookkeeping of reserve, fork and free is one workgroup: it checks every item before it changes
// anything (slots listed twice are found in a bit map in LDS), ranks the pages the items need with a
// prefix sum, collects that many free pages in ascending order, and hands them out one wave per
// item. Fork's partly filled pages are then copied by a second launch. Compact needs the whole of
// refs: workgroups of kChunk pages count, then rank, then move, in three launches. Reference counts
// change by integer atomics, whose result does not depend on their order.
#include <hip/hip_runtime.h>

#include "../../include/nvfp4.h"
#include "kv_cache.h"

namespace nvfp4 {
namespace {

constexpr int kBook = 1024;          // threads of the bookkeeping workgroup
constexpr int kWaves = kBook / 64;
constexpr int kSlotWords = 65536 / 32;
constexpr int kChunk = 4096;         // pages per workgroup of compact's counting
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;        // 16-byte loads in flight per lane
constexpr int kPart = kCopyThreads * kCopyLoads * 16;   // bytes of a record per step

__device__ __forceinline__ int wave_inclusive(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// Exclusive prefix sum of v over a workgroup of WAVES waves; total gets the sum. `sums` holds WAVES + 1
// words; the caller's threads may call it again at once.
template <int WAVES>
__device__ __forceinline__ int block_exclusive(int v, int* sums, int& total) {
    const int incl = wave_inclusive(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
        const int s = sums[q];
        before += q < (int)(threadIdx.x >> 6) ? s : 0;
        total += s;
    }
    return before + incl - v;
}

__device__ __forceinline__ int pages_of(int64_t len, int page) {
    return (int)((len + page - 1) / page);
}

// A slot's length, clamped to what the table can hold.
__device__ __forceinline__ int length_of(const KvPool& p, int slot) {
    return min(max(p.lens[slot], 0), p.max_pages * p.page);
}

// Adds the items' slots to the bit map; true (for this thread) if one is outside the table or listed
// twice.
__device__ __forceinline__ bool mark_slots(const KvPool& p, const int32_t* slots, int n,
                                           uint32_t* map) {
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += kBook) {
        const int s = slots[i];
        if ((uint32_t)s >= (uint32_t)p.max_slots) {
            bad = true;
        } else {
            const uint32_t bit = 1u << (s & 31);
            bad |= (atomicOr(&map[s >> 5], bit) & bit) != 0;
        }
    }
    return bad;
}

// The lowest `need` free pages in ascending order into list[]; returns how many were found (at most
// need).
__device__ __forceinline__ int take_free(const KvPool& p, int need, int32_t* list, int* sums) {
    int found = 0;
    for (int p0 = 0; p0 < p.num_pages && found < need; p0 += 4 * kBook) {
        const int q = p0 + 4 * (int)threadIdx.x;
        int r[4], free = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = q + i < p.num_pages ? p.refs[q + i] : 1;
            free += r[i] <= 0;
        }
        int total;
        int k = found + block_exclusive<kWaves>(free, sums, total);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (r[i] <= 0) {
                if (k < need) list[k] = q + i;
                ++k;
            }
        }
        found += total;
    }
    return min(found, need);
}

// Workspace of reserve and fork: first[n] (an item's first rank among the pages taken), list[]
// (the pages taken), and for fork src[n], dst[n].
__global__ __launch_bounds__(kBook) void k_kv_reserve(KvPool p, const int32_t* __restrict__ slots,
                                                      const int32_t* __restrict__ counts, int n,
                                                      int32_t* status, int32_t* first,
                                                      int32_t* list) {
    __shared__ uint32_t map[kSlotWords];
    __shared__ int sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSlotWords; i += kBook) map[i] = 0u;
    __syncthreads();
    if (__syncthreads_or(mark_slots(p, slots, n, map))) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_SLOT;
        return;
    }
    bool bad = false;
    int64_t need = 0;
    for (int i0 = 0; i0 < n; i0 += kBook) {
        const int i = i0 + threadIdx.x;
        int add = 0;
        if (i < n) {
            const int old = length_of(p, slots[i]);
            const int64_t now = (int64_t)old + counts[i];
            if (counts[i] < 0 || now > (int64_t)p.max_pages * p.page) bad = true;
            else add = pages_of(now, p.page) - pages_of(old, p.page);
        }
        int total;
        const int before = block_exclusive<kWaves>(add, sums, total);
        // beyond num_pages the call fails anyway: ranks are kept inside int32
        if (i < n) first[i] = (int)min(need + before, (int64_t)p.num_pages + 1);
        need += total;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_LENGTH;
        return;
    }
    if (need > p.num_pages || take_free(p, (int)need, list, sums) < (int)need) {
        if (threadIdx.x == 0) *status = NVFP4_KV_NO_PAGES;
        return;
    }
    __syncthreads();
    for (int i = wave; i < n; i += kWaves) {
        const int s = slots[i];
        const int old = length_of(p, s);
        const int now = old + counts[i];
        const int have = pages_of(old, p.page), add = pages_of(now, p.page) - have;
        for (int k = lane; k < add; k += 64) {
            const int page = list[first[i] + k];
            p.table[(int64_t)s * p.max_pages + have + k] = page;
            p.refs[page] = 1;
        }
        if (lane == 0) p.lens[s] = now;
    }
    if (threadIdx.x == 0) *status = NVFP4_KV_DONE;
}

__global__ __launch_bounds__(kBook) void k_kv_fork(KvPool p, const int32_t* __restrict__ parents,
                                                   const int32_t* __restrict__ children, int n,
                                                   int32_t* status, int32_t* first, int32_t* list,
                                                   int32_t* src, int32_t* dst) {
    __shared__ uint32_t map[kSlotWords];
    __shared__ int sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSlotWords; i += kBook) map[i] = 0u;
    for (int i = threadIdx.x; i < n; i += kBook) src[i] = -1;      // nothing to copy yet
    __syncthreads();
    bool bad = mark_slots(p, children, n, map);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBook) {
        const int a = parents[i], c = children[i];
        if ((uint32_t)a >= (uint32_t)p.max_slots) bad = true;
        else bad |= ((map[a >> 5] >> (a & 31)) & 1u) != 0;
        if ((uint32_t)c < (uint32_t)p.max_slots) bad |= p.lens[c] != 0;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_SLOT;
        return;
    }
    int need = 0;                                                  // at most n <= 65,536
    for (int i0 = 0; i0 < n; i0 += kBook) {
        const int i = i0 + threadIdx.x;
        const int part = i < n && length_of(p, parents[i]) % p.page != 0;
        int total;
        const int before = block_exclusive<kWaves>(part, sums, total);
        if (i < n) first[i] = need + before;
        need += total;
    }
    if (take_free(p, need, list, sums) < need) {
        if (threadIdx.x == 0) *status = NVFP4_KV_NO_PAGES;
        return;
    }
    __syncthreads();
    for (int i = wave; i < n; i += kWaves) {
        const int len = length_of(p, parents[i]);
        const int full = len / p.page;
        const int32_t* from = p.table + (int64_t)parents[i] * p.max_pages;
        int32_t* to = p.table + (int64_t)children[i] * p.max_pages;
        for (int k = lane; k < full; k += 64) {
            const int page = from[k];
            to[k] = page;
            if ((uint32_t)page < (uint32_t)p.num_pages) atomicAdd(&p.refs[page], 1);
        }
        if (lane == 0) {
            if (len % p.page != 0) {
                const int page = list[first[i]];
                to[full] = page;
                p.refs[page] = 1;
                dst[i] = page;
                src[i] = (uint32_t)from[full] < (uint32_t)p.num_pages ? from[full] : -1;
            }
            p.lens[children[i]] = len;
        }
    }
    if (threadIdx.x == 0) *status = NVFP4_KV_DONE;
}

__global__ __launch_bounds__(kBook) void k_kv_free(KvPool p, const int32_t* __restrict__ slots,
                                                   int n, int32_t* status) {
    __shared__ uint32_t map[kSlotWords];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSlotWords; i += kBook) map[i] = 0u;
    __syncthreads();
    if (__syncthreads_or(mark_slots(p, slots, n, map))) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_SLOT;
        return;
    }
    for (int i = wave; i < n; i += kWaves) {
        const int s = slots[i];
        const int held = pages_of(length_of(p, s), p.page);
        int32_t* row = p.table + (int64_t)s * p.max_pages;
        for (int k = lane; k < held; k += 64) {
            const int page = row[k];
            row[k] = -1;
            if ((uint32_t)page < (uint32_t)p.num_pages) atomicSub(&p.refs[page], 1);
        }
        if (lane == 0) p.lens[s] = 0;
    }
    if (threadIdx.x == 0) *status = NVFP4_KV_DONE;
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// kPart bytes of a record from byte `at` (records are multiples of 16 bytes).
__device__ __forceinline__ void copy_part(const uint8_t* __restrict__ s, uint8_t* __restrict__ d,
                                          int64_t at, int64_t record) {
    u32x4 v[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int64_t o = at + ((int64_t)k * kCopyThreads + threadIdx.x) * 16;
        if (o < record) v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(s + o));
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int64_t o = at + ((int64_t)k * kCopyThreads + threadIdx.x) * 16;
        if (o < record) __builtin_nontemporal_store(v[k], reinterpret_cast<u32x4*>(d + o));
    }
}

// Fork's copies: item blockIdx.y, layer blockIdx.z, the record's parts over blockIdx.x.
__global__ __launch_bounds__(kCopyThreads) void k_kv_copy(KvPool p, const int32_t* __restrict__ src,
                                                          const int32_t* __restrict__ dst) {
    const int a = src[blockIdx.y];
    if (a < 0) return;
    uint8_t* base = p.pages + (int64_t)blockIdx.z * p.layer_stride;
    copy_part(base + (int64_t)a * p.page_stride, base + (int64_t)dst[blockIdx.y] * p.page_stride,
              (int64_t)blockIdx.x * kPart, p.record);
}

// Compact's workspace: head[2] = (used pages, pages to move), counts[chunks], src[], dst[] by rank,
// rank[] of a page that moves (-1 for others).
struct CompactSpace {
    int32_t* head;
    int32_t* counts;
    int32_t* src;
    int32_t* dst;
    int32_t* rank;
};

constexpr int kCountThreads = 256;

// Used pages of a chunk.
__device__ __forceinline__ int used_in(const KvPool& p, int begin, int end, int* sums) {
    int used = 0;
    for (int q = begin + threadIdx.x; q < end; q += kCountThreads) used += p.refs[q] > 0;
    int total;
    block_exclusive<kCountThreads / 64>(used, sums, total);
    return total;
}

__global__ __launch_bounds__(kCountThreads) void k_kv_count(KvPool p, CompactSpace w) {
    __shared__ int sums[kCountThreads / 64];
    const int begin = blockIdx.x * kChunk;
    const int total = used_in(p, begin, min(begin + kChunk, p.num_pages), sums);
    if (threadIdx.x == 0) w.counts[blockIdx.x] = total;
}

__global__ __launch_bounds__(kCountThreads) void k_kv_rank(KvPool p, CompactSpace w, int chunks) {
    __shared__ int sums[kCountThreads / 64];
    constexpr int W = kCountThreads / 64;
    // used pages in all chunks, before this chunk, and before the chunk that holds page U
    int all = 0, mine = 0;
    for (int c = threadIdx.x; c < chunks; c += kCountThreads) {
        const int v = w.counts[c];
        all += v;
        mine += c < (int)blockIdx.x ? v : 0;
    }
    int U, before;
    block_exclusive<W>(all, sums, U);
    block_exclusive<W>(mine, sums, before);
    const int cu = min(U / kChunk, chunks - 1);
    int low = 0;
    for (int c = threadIdx.x; c < cu; c += kCountThreads) low += w.counts[c];
    int below;                                    // used pages below U
    block_exclusive<W>(low, sums, below);
    below += used_in(p, cu * kChunk, min(U, p.num_pages), sums);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        w.head[0] = U;
        w.head[1] = U - below;
    }
    const int begin = blockIdx.x * kChunk, end = min(begin + kChunk, p.num_pages);
    for (int q0 = begin; q0 < end; q0 += kCountThreads) {
        const int q = q0 + threadIdx.x;
        const int used = q < end && p.refs[q] > 0;
        int total;
        const int k = before + block_exclusive<W>(used, sums, total);   // used pages before q
        if (q < end) {
            int r = -1;
            if (used && q >= U) {
                r = k - below;
                w.src[r] = q;
            } else if (!used && q < U) {
                w.dst[q - k] = q;
            }
            w.rank[q] = r;
        }
        before += total;
    }
}

// Moves the records, and (first workgroups) rewrites table and refs.
__global__ __launch_bounds__(kCopyThreads) void k_kv_move(KvPool p, CompactSpace w, int parts,
                                                          int32_t* used_out) {
    const int m = w.head[1];
    const int64_t tid = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * kCopyThreads;
    if (tid == 0) *used_out = w.head[0];
    for (int64_t k = tid; k < m; k += threads) {
        const int a = w.src[k], d = w.dst[k];
        p.refs[d] = p.refs[a];
        p.refs[a] = 0;
    }
    const int64_t entries = (int64_t)p.max_slots * p.max_pages;
    for (int64_t k = tid; k < entries; k += threads) {
        const int e = p.table[k];
        if ((uint32_t)e < (uint32_t)p.num_pages) {
            const int r = w.rank[e];
            if (r >= 0) p.table[k] = w.dst[r];
        }
    }
    const int64_t items = (int64_t)m * p.layers * parts;
    for (int64_t k = blockIdx.x; k < items; k += gridDim.x) {
        const int64_t page = k / parts;
        const int64_t layer = page / m;
        const int64_t i = page - layer * m;
        uint8_t* base = p.pages + layer * p.layer_stride;
        copy_part(base + (int64_t)w.src[i] * p.page_stride, base + (int64_t)w.dst[i] * p.page_stride,
                  (k - page * parts) * kPart, p.record);
    }
}

int64_t parts_of(const KvPool& p) { return (p.record + kPart - 1) / kPart; }
int64_t words(int64_t n) { return (n + 3) / 4 * 4; }
int64_t chunks_of(int64_t num_pages) { return num_pages > 0 ? (num_pages + kChunk - 1) / kChunk : 1; }

}  // namespace

size_t kv_pages_workspace_bytes(int64_t num_pages, int64_t n) {
    // reserve: first[n], list[num_pages]; fork: first, src, dst [n], list[n]; compact: head,
    // counts[chunks], src, dst, rank [num_pages]
    const int64_t a = words(n) + words(num_pages), b = 4 * words(n);
    const int64_t c = 4 + words(chunks_of(num_pages)) + 3 * words(num_pages);
    return (size_t)(n > 0 ? (a > b ? a : b) : c) * 4;
}

hipError_t launch_kv_reserve(const KvPool& p, const int32_t* slots, const int32_t* counts,
                             int32_t n, int32_t* status, void* workspace, hipStream_t stream) {
    int32_t* first = static_cast<int32_t*>(workspace);
    hipLaunchKernelGGL(k_kv_reserve, dim3(1), dim3(kBook), 0, stream, p, slots, counts, n, status,
                       first, first + words(n));
    return hipGetLastError();
}

hipError_t launch_kv_fork(const KvPool& p, const int32_t* parents, const int32_t* children,
                          int32_t n, int32_t* status, void* workspace, hipStream_t stream) {
    int32_t* first = static_cast<int32_t*>(workspace);
    int32_t *src = first + words(n), *dst = src + words(n), *list = dst + words(n);
    hipLaunchKernelGGL(k_kv_fork, dim3(1), dim3(kBook), 0, stream, p, parents, children, n, status,
                       first, list, src, dst);
    if (n > 0 && p.layers > 0 && p.record > 0)
        hipLaunchKernelGGL(k_kv_copy, dim3((uint32_t)parts_of(p), (uint32_t)n, (uint32_t)p.layers),
                           dim3(kCopyThreads), 0, stream, p, src, dst);
    return hipGetLastError();
}

hipError_t launch_kv_free(const KvPool& p, const int32_t* slots, int32_t n, int32_t* status,
                          hipStream_t stream) {
    hipLaunchKernelGGL(k_kv_free, dim3(1), dim3(kBook), 0, stream, p, slots, n, status);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvPool& p, int32_t* used, void* workspace, hipStream_t stream) {
    const int chunks = (int)chunks_of(p.num_pages);
    CompactSpace w;
    w.head = static_cast<int32_t*>(workspace);
    w.counts = w.head + 4;
    w.src = w.counts + words(chunks);
    w.dst = w.src + words(p.num_pages);
    w.rank = w.dst + words(p.num_pages);
    hipLaunchKernelGGL(k_kv_count, dim3(chunks), dim3(kCountThreads), 0, stream, p, w);
    hipLaunchKernelGGL(k_kv_rank, dim3(chunks), dim3(kCountThreads), 0, stream, p, w, chunks);
    // the number of moves is known on the device only: a grid that fills the chip strides over them
    const int64_t most = (int64_t)(p.num_pages / 2) * p.layers * parts_of(p);
    const uint32_t grid = (uint32_t)(most < 2048 ? (most > 16 ? most : 16) : 2048);
    hipLaunchKernelGGL(k_kv_move, dim3(grid), dim3(kCopyThreads), 0, stream, p, w, (int)parts_of(p),
                       used);
    return hipGetLastError();
}

}  // namespace nvfp4
