// Page bookkeeping of the paged key/value cache for gfx950: reserve, fork, free and compact change the
// page table, the lengths and the reference counts on the device.
//
// The bookkeeping of reserve and fork is one workgroup: it checks every item before it changes
// anything (slots listed twice are found in a bit map in LDS), ranks the pages the items need with a
// prefix sum, collects that many free pages in ascending order, and hands them out. What bounds it is
// the chain of dependent loads (slot, length, table entry), so every step is made for all items at
// once and the first reference counts are on their way from the start. Fork's rows and partly filled
// pages are copied by a second launch. Compact ranks all pages in one workgroup, or, beyond kOne
// pages, in workgroups of kChunk that count and then rank, and moves the records in a last launch, at
// the rate of a copy. Reference counts change by integer atomics, whose result does not depend on
// their order.
//
// 16 slots of up to 500 positions (pages of 16): free 2.5 us, fork 4.9 and its copies 3.6, reserve 4.4.
// 256 slots of up to 4000 (pages of 64, 4 layers, 8 heads, 128 wide): 3.9, 5.5 and 8.4 (37 MB, 4.4 TB/s), 5.7.
// Compact of 192 slots of up to 3000: 6.5 us to rank, 140 to move 785 MB (5.6 TB/s read and written).
#include <hip/hip_runtime.h>

#include "../../include/nvfp4.h"
#include "kv_cache.h"

namespace nvfp4 {
namespace {

constexpr int kBook = 1024;          // threads of the bookkeeping workgroup
constexpr int kWaves = kBook / 64;
constexpr int kSlotWords = 65536 / 32;
constexpr int kFirst = 4;            // reference counts a thread loads ahead
constexpr int kFreeRows = 16;        // slots a workgroup of free empties, one a wave, where there are few
constexpr int kFreeMost = 64;        // its workgroups (65,536 slots: kBook each)
constexpr int kOne = 16 * kBook;     // pages that one workgroup ranks for compact
constexpr int kChunk = 1024;         // pages per workgroup of compact's counting
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

// Exclusive prefix sum of v over a workgroup of WAVES waves; total gets the sum. `sums` holds WAVES
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

__device__ __forceinline__ void clear_map(const KvPool& p, uint32_t* map) {
    for (int i = threadIdx.x; i < (p.max_slots + 31) / 32; i += kBook) map[i] = 0u;
    __syncthreads();
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

// Reference counts of the pages q .. q + 3 (`none` at or beyond end) in one load: counts one by one would
// touch a line again and again, and a touch of a line that is still on its way waits for it (256 slots:
// fork 5.5 us, reserve 5.7; with eight counts a thread one by one 7.6 and 7.8).
typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ i32x4 counts_of(const KvPool& p, int q, int end, int none) {
    if (q + 4 <= end) return *reinterpret_cast<const i32x4*>(p.refs + q);
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = q + i < end ? p.refs[q + i] : none;
    return r;
}

// Which of the thread's kFirst pages from page p0 on are free, as bits; of kFirst kBook pages in all.
__device__ __forceinline__ uint32_t free_bits(const KvPool& p, int p0) {
    const i32x4 r = counts_of(p, p0 + kFirst * (int)threadIdx.x, p.num_pages, 1);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kFirst; ++i) bits |= r[i] <= 0 ? 1u << i : 0u;
    return bits;
}

// The lowest `need` free pages in ascending order into list[]; returns how many were found (at most
// need). bits: free_bits(p, 0), loaded ahead, as every round's are by the one before.
__device__ __forceinline__ int take_free(const KvPool& p, int need, uint32_t bits, int32_t* list,
                                         int* sums) {
    int found = 0;
    for (int64_t p0 = 0; p0 < p.num_pages && found < need; p0 += kFirst * kBook) {
        const bool more = p0 + kFirst * kBook < p.num_pages;
        const uint32_t next = more ? free_bits(p, (int)p0 + kFirst * kBook) : 0u;
        int total;
        int k = found + block_exclusive<kWaves>(__popc(bits), sums, total);
        for (uint32_t left = bits; left != 0 && k < need; left &= left - 1)
            list[k++] = (int)p0 + kFirst * (int)threadIdx.x + __builtin_ctz(left);
        found += total;
        bits = next;
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
    const uint32_t bits = free_bits(p, 0);
    clear_map(p, map);
    if (__syncthreads_or(mark_slots(p, slots, n, map))) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_SLOT;
        return;
    }
    bool bad = false, many = false;
    int need = 0;                        // the slots are distinct, so all their pages are < 2^31
    // the thread's item of the last batch, kept for the common call of one batch
    int slot = 0, have = 0, add = 0, now = 0, rank = 0;
    for (int i0 = 0; i0 < n; i0 += kBook) {
        const int i = i0 + threadIdx.x;
        add = 0;
        if (i < n) {
            slot = slots[i];
            const int count = counts[i], old = length_of(p, slot);
            const int64_t len = (int64_t)old + count;
            if (count < 0 || len > (int64_t)p.max_pages * p.page) {
                bad = true;
            } else {
                now = (int)len;
                have = pages_of(old, p.page);
                add = pages_of(now, p.page) - have;
            }
        }
        many |= add > 1;
        int total;
        rank = need + block_exclusive<kWaves>(add, sums, total);
        if (i < n) first[i] = rank;
        need += total;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) *status = NVFP4_KV_BAD_LENGTH;
        return;
    }
    if (need > p.num_pages || take_free(p, need, bits, list, sums) < need) {
        if (threadIdx.x == 0) *status = NVFP4_KV_NO_PAGES;
        return;
    }
    // an item's first page by its thread; the others, where an item takes more, one wave an item.
    // Lengths are written when every item's old one has been used.
    const bool any_many = __syncthreads_or(many);
    if (n <= kBook && !any_many) {
        if ((int)threadIdx.x < n) {
            if (add > 0) {
                const int page = list[rank];
                p.table[(int64_t)slot * p.max_pages + have] = page;
                p.refs[page] = 1;
            }
            p.lens[slot] = now;
        }
        if (threadIdx.x == 0) *status = NVFP4_KV_DONE;
        return;
    }
    for (int i = threadIdx.x; i < n; i += kBook) {
        const int s = slots[i], old = length_of(p, s), now = old + counts[i];
        const int held = pages_of(old, p.page);
        if (pages_of(now, p.page) > held) {
            const int page = list[first[i]];
            p.table[(int64_t)s * p.max_pages + held] = page;
            p.refs[page] = 1;
        }
        if (!any_many) p.lens[s] = now;
    }
    if (any_many) {
        for (int i = wave; i < n; i += kWaves) {
            const int s = slots[i], old = length_of(p, s), now = old + counts[i];
            const int held = pages_of(old, p.page), more = pages_of(now, p.page) - held;
            for (int k = lane + 1; k < more; k += 64) {
                const int page = list[first[i] + k];
                p.table[(int64_t)s * p.max_pages + held + k] = page;
                p.refs[page] = 1;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kBook) {
            const int s = slots[i];
            p.lens[s] = length_of(p, s) + counts[i];
        }
    }
    if (threadIdx.x == 0) *status = NVFP4_KV_DONE;
}

// Checks a fork and gives every item the record to copy: src[i] its page (kRowOnly: none), kNothing
// for all where the fork is refused, and dst[i].
constexpr int kRowOnly = -1, kNothing = -2;

__global__ __launch_bounds__(kBook) void k_kv_fork(KvPool p, const int32_t* __restrict__ parents,
                                                   const int32_t* __restrict__ children, int n,
                                                   int32_t* status, int32_t* first, int32_t* list,
                                                   int32_t* src, int32_t* dst) {
    __shared__ uint32_t map[kSlotWords];
    __shared__ int sums[kWaves];
    const uint32_t bits = free_bits(p, 0);
    clear_map(p, map);
    bool bad = mark_slots(p, children, n, map);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBook) {
        const int a = parents[i], c = children[i];
        if ((uint32_t)a >= (uint32_t)p.max_slots) bad = true;
        else bad |= ((map[a >> 5] >> (a & 31)) & 1u) != 0;
        if ((uint32_t)c < (uint32_t)p.max_slots) bad |= p.lens[c] != 0;
    }
    int reason = __syncthreads_or(bad) ? NVFP4_KV_BAD_SLOT : NVFP4_KV_DONE;
    int need = 0;                                                  // at most n <= 65,536
    if (reason == NVFP4_KV_DONE) {
        for (int i0 = 0; i0 < n; i0 += kBook) {
            const int i = i0 + threadIdx.x;
            const int part = i < n && length_of(p, parents[i]) % p.page != 0;
            int total;
            const int before = block_exclusive<kWaves>(part, sums, total);
            if (i < n) first[i] = need + before;
            need += total;
        }
        if (take_free(p, need, bits, list, sums) < need) reason = NVFP4_KV_NO_PAGES;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBook) {
        int from = kNothing;
        if (reason == NVFP4_KV_DONE) {
            const int len = length_of(p, parents[i]), full = len / p.page;
            from = kRowOnly;
            if (len % p.page != 0) {
                const int old = p.table[(int64_t)parents[i] * p.max_pages + full];
                const int page = list[first[i]];
                dst[i] = page;
                p.refs[page] = 1;
                p.table[(int64_t)children[i] * p.max_pages + full] = page;
                from = (uint32_t)old < (uint32_t)p.num_pages ? old : kRowOnly;
            }
            p.lens[children[i]] = len;
        }
        src[i] = from;
    }
    if (threadIdx.x == 0) *status = reason;
}

// Every workgroup checks all slots and empties its share of them: the changes of reference counts are
// scattered atomics, which one compute unit issues an address at a time (256 slots of up to 63 pages 9.0 us
// in one workgroup, 3.9 in sixteen).
__global__ __launch_bounds__(kBook) void k_kv_free(KvPool p, const int32_t* __restrict__ slots,
                                                   int n, int32_t* status) {
    __shared__ uint32_t map[kSlotWords];
    __shared__ int slot[kBook], held[kBook];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    clear_map(p, map);
    if (__syncthreads_or(mark_slots(p, slots, n, map))) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *status = NVFP4_KV_BAD_SLOT;
        return;
    }
    const int share = (n + (int)gridDim.x - 1) / (int)gridDim.x;        // at most kBook
    const int i0 = (int)blockIdx.x * share, m = min(share, n - i0);
    if ((int)threadIdx.x < m) {
        const int s = slots[i0 + threadIdx.x];
        slot[threadIdx.x] = s;
        held[threadIdx.x] = pages_of(length_of(p, s), p.page);
        p.lens[s] = 0;
    }
    __syncthreads();
    for (int j = wave; j < m; j += kWaves) {             // a row of a wave at a time
        int32_t* row = p.table + (int64_t)slot[j] * p.max_pages;
        for (int k = lane; k < held[j]; k += 64) {
            const int page = row[k];
            row[k] = -1;
            if ((uint32_t)page < (uint32_t)p.num_pages) atomicSub(&p.refs[page], 1);
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = NVFP4_KV_DONE;
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

// Fork's copies: item blockIdx.x, the parts of its record over blockIdx.y, layer blockIdx.z; the first
// workgroup of an item also copies its table row of full pages.
__global__ __launch_bounds__(kCopyThreads) void k_kv_copy(KvPool p, const int32_t* __restrict__ parents,
                                                          const int32_t* __restrict__ children,
                                                          const int32_t* __restrict__ src,
                                                          const int32_t* __restrict__ dst, int parts) {
    const int i = blockIdx.x;
    const int a = src[i];
    if (a == kNothing) return;
    if (blockIdx.y == 0 && blockIdx.z == 0) {
        const int full = length_of(p, parents[i]) / p.page;
        const int32_t* from = p.table + (int64_t)parents[i] * p.max_pages;
        int32_t* to = p.table + (int64_t)children[i] * p.max_pages;
        for (int k = threadIdx.x; k < full; k += kCopyThreads) {
            const int page = from[k];
            to[k] = page;
            if ((uint32_t)page < (uint32_t)p.num_pages) atomicAdd(&p.refs[page], 1);
        }
    }
    if (a < 0) return;
    uint8_t* base = p.pages + (int64_t)blockIdx.z * p.layer_stride;
    for (int64_t part = blockIdx.y; part < parts; part += gridDim.y)
        copy_part(base + (int64_t)a * p.page_stride, base + (int64_t)dst[i] * p.page_stride,
                  part * kPart, p.record);
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
constexpr int kEach = kChunk / kCountThreads;            // consecutive pages of a thread

// Which of N consecutive pages from q on (below end) are used, as bits.
template <int N>
__device__ __forceinline__ uint32_t used_bits(const KvPool& p, int q, int end) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const i32x4 r = counts_of(p, q + i, end, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) bits |= r[j] > 0 ? 1u << (i + j) : 0u;
    }
    return bits;
}

// Ranks N consecutive pages from q on, `before` used ones before them, U used in all, `below` of them
// below page U: used pages at or above U move to the free pages below it, in order.
template <int N>
__device__ __forceinline__ void rank_pages(const KvPool& p, const CompactSpace& w, int q, uint32_t bits,
                                           int before, int U, int below) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (q + i >= p.num_pages) break;
        const bool used = (bits >> i) & 1u;
        int r = -1;
        if (used && q + i >= U) {
            r = before - below;
            w.src[r] = q + i;
        } else if (!used && q + i < U) {
            w.dst[q + i - before] = q + i;
        }
        w.rank[q + i] = r;
        before += used;
    }
}

// All of at most kOne pages.
__global__ __launch_bounds__(kBook) void k_kv_rank_all(KvPool p, CompactSpace w) {
    constexpr int N = kOne / kBook;
    __shared__ int sums[kWaves];
    const int q = N * (int)threadIdx.x;
    const uint32_t bits = used_bits<N>(p, q, p.num_pages);
    int U, below;
    const int before = block_exclusive<kWaves>(__popc(bits), sums, U);
    const int inside = min(max(U - q, 0), N);            // pages of the thread below U
    block_exclusive<kWaves>(__popc(bits & ((1u << inside) - 1u)), sums, below);
    if (threadIdx.x == 0) {
        w.head[0] = U;
        w.head[1] = U - below;
    }
    rank_pages<N>(p, w, q, bits, before, U, below);
}

__global__ __launch_bounds__(kCountThreads) void k_kv_count(KvPool p, CompactSpace w) {
    __shared__ int sums[kCountThreads / 64];
    const int q = blockIdx.x * kChunk + kEach * (int)threadIdx.x;
    int total;
    block_exclusive<kCountThreads / 64>(__popc(used_bits<kEach>(p, q, p.num_pages)), sums, total);
    if (threadIdx.x == 0) w.counts[blockIdx.x] = total;
}

__global__ __launch_bounds__(kCountThreads) void k_kv_rank(KvPool p, CompactSpace w, int chunks) {
    __shared__ int sums[kCountThreads / 64];
    constexpr int W = kCountThreads / 64;
    const int q = blockIdx.x * kChunk + kEach * (int)threadIdx.x;
    const uint32_t bits = used_bits<kEach>(p, q, p.num_pages);
    // used pages in all chunks, before this chunk, and before the chunk that holds page U
    int all = 0, mine = 0;
    for (int c = threadIdx.x; c < chunks; c += kCountThreads) {
        const int v = w.counts[c];
        all += v;
        mine += c < (int)blockIdx.x ? v : 0;
    }
    int U, before, below, in_chunk, ahead;
    block_exclusive<W>(all, sums, U);
    block_exclusive<W>(mine, sums, before);
    const int cu = min(U / kChunk, chunks - 1);
    int low = 0;
    for (int c = threadIdx.x; c < cu; c += kCountThreads) low += w.counts[c];
    low += __popc(used_bits<kEach>(p, cu * kChunk + kEach * (int)threadIdx.x, min(U, p.num_pages)));
    block_exclusive<W>(low, sums, below);                // used pages below U
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        w.head[0] = U;
        w.head[1] = U - below;
    }
    ahead = block_exclusive<W>(__popc(bits), sums, in_chunk);
    rank_pages<kEach>(p, w, q, bits, before + ahead, U, below);
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
    const int64_t parts = parts_of(p);
    if (n > 0)
        hipLaunchKernelGGL(k_kv_copy, dim3((uint32_t)n, (uint32_t)(parts < 64 ? parts : 64), (uint32_t)p.layers),
                           dim3(kCopyThreads), 0, stream, p, parents, children, src, dst,
                           (int)parts);
    return hipGetLastError();
}

hipError_t launch_kv_free(const KvPool& p, const int32_t* slots, int32_t n, int32_t* status,
                          hipStream_t stream) {
    const int wanted = (n + kFreeRows - 1) / kFreeRows;
    const int groups = wanted < 1 ? 1 : wanted < kFreeMost ? wanted : kFreeMost;
    hipLaunchKernelGGL(k_kv_free, dim3(groups), dim3(kBook), 0, stream, p, slots, n, status);
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
    if (p.num_pages <= kOne) {
        hipLaunchKernelGGL(k_kv_rank_all, dim3(1), dim3(kBook), 0, stream, p, w);
    } else {
        hipLaunchKernelGGL(k_kv_count, dim3(chunks), dim3(kCountThreads), 0, stream, p, w);
        hipLaunchKernelGGL(k_kv_rank, dim3(chunks), dim3(kCountThreads), 0, stream, p, w, chunks);
    }
    // the number of moves is known on the device only: a grid that fills the chip strides over them
    const int64_t most = (int64_t)(p.num_pages / 2) * p.layers * parts_of(p);
    const uint32_t grid = (uint32_t)(most < 2048 ? (most > 16 ? most : 16) : 2048);
    hipLaunchKernelGGL(k_kv_move, dim3(grid), dim3(kCopyThreads), 0, stream, p, w, (int)parts_of(p),
                       used);
    return hipGetLastError();
}

}  // namespace nvfp4
