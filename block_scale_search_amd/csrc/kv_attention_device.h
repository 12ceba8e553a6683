// Device pieces of attention over the paged NVFP4 cache for gfx950: cached codes to f16 MFMA operands,
// query rows to f16, cross-lane reductions, and the work split that the kernels share.
//
// Arithmetic. level * E4M3(scale) has at most 2 + 4 significant bits and lies in 2^-10 .. 2688, so
// it is exact in f16: K and V enter the products as f16 without error and the global scales S_k and
// S_v multiply the logits and the outputs. E4M3 code c as f16 times 2^-8 is the bit pattern c << 7
// (same mantissa field, subnormals included); the up-conversion of the 4-bit codes supplies 2^8. A
// scale byte is masked to 7 bits, so no byte of the cache gives an infinity or NaN, and a weight of
// zero cancels whatever lies behind a sequence. A query row is scaled by a power of two that brings its
// largest value into [2^14, 2^15): bf16 values are then exact in f16 down to 2^-28 of the largest, and
// off by at most 2^-39 of it below; f32 values are split into two f16 halves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_formats.h"
#include "kv_cache.h"

namespace nvfp4 {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

union Half8 {
    half8v v;
    half2v p[4];
    uint32_t u[4];
};

__device__ __forceinline__ half2v as_half2(uint32_t u) { return __builtin_bit_cast(half2v, u); }

// The two values of byte SEL of w, times 2^8 and a pair of scales that carry 2^-8.
template <int SEL>
__device__ __forceinline__ half2v dequant2(uint32_t w, half2v scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, SEL) * scale;
}

// Scale byte B of `bytes` (masked), twice; and the pair of bytes (0, 1) or (2, 3): f16 times 2^-8.
template <int B>
__device__ __forceinline__ half2v scale_twice(uint32_t bytes) {
    constexpr uint32_t sel = 0x0C000C00u | (uint32_t)B | ((uint32_t)B << 16);
    return as_half2(__builtin_amdgcn_perm(0u, bytes, sel) << 7);
}
template <int HIGH>
__device__ __forceinline__ half2v scale_pair(uint32_t bytes) {
    constexpr uint32_t sel = HIGH ? 0x0C030C02u : 0x0C010C00u;
    return as_half2(__builtin_amdgcn_perm(0u, bytes, sel) << 7);
}

// (bits of a where the mask is set) | (bits of b elsewhere)
__device__ __forceinline__ uint32_t select_bits(uint32_t mask, uint32_t a, uint32_t b) {
    return (a & mask) | (b & ~mask);
}

// Maximum (sum) over the four 16-lane groups of a wave, in every lane.
__device__ __forceinline__ float max_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// Exponent k that brings a row's largest |value| into [2^14, 2^15), at most 126.
__device__ __forceinline__ int row_exponent(float top) {
    if (!(top > 0.0f)) return 0;
    return min(15 - __builtin_amdgcn_frexp_expf(top), 126);
}

// What the row's values are multiplied by: 2^k, or NaN for a row with an infinity and where S_k is NaN or
// infinite. Such logits are infinite or NaN, their softmax is NaN whatever they are, and logits of -infinity
// would look like positions that are masked.
__device__ __forceinline__ float row_factor(int k, float top, float S) {
    return top < __builtin_inff() && S < __builtin_inff() ? __builtin_ldexpf(1.0f, k)
                                                          : __builtin_nanf("");
}

// Weights enter the second product as f16, for f32 outputs in two halves (22 bits), for bf16 in one: an error of at
// most 2^-11 of each weight, independent of the others, below the 2^-8 of the output's own rounding. Their sum
// is taken in binary32, unrounded, for lse's sake. Error against 64 bits of 64 rows over up to 8192 positions:
// 1.692e-3 with one half, 1.686e-3 with two, which take 55.9 us instead of 54.2 (one row over 1023 positions
// 11.4 and 10.7, 32 drafts of 5 over up to 4096 36.3 and 32.9, two prompts of 8192 rows 1505 and 1138).
constexpr float kUp = 8.0f;          // log2 of the weights' scale
constexpr float kSlack = 7.0f;       // how far a logit may exceed the maximum in use, log2

// Raises a row's maximum in use m (and sub, what its logits are shifted by) to `top`, the row's largest logit, if
// that passes the slack; returns the factor of the row's sums so far. The wave comes here when one of its rows
// has to; another keeps its m, so that its bits are the same whatever the wave's other rows hold.
__device__ __forceinline__ float raise_row(float& m, float& sub, float top, float slack) {
    const bool up = top > m + slack;
    const float al = up ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
    m = up ? top : m;
    sub = up ? kUp - top : sub;
    return al;
}

// A lane's bytes of 16 tokens (a unit). K: D/4 values of its token and their scale bytes. V:
// D/16 values of 4 tokens, and those tokens' scale bytes.
template <int D>
struct HalfTile {
    static constexpr int W = D / 32;          // code words
    uint32_t k[W], v[W], ks, vs;
};

// K operand of step s: values 8 s .. 8 s + 7 of the lane's D/4.
template <int S, int W>
__device__ __forceinline__ half8v k_operand(const uint32_t (&w)[W], uint32_t scales) {
    Half8 r;
    const half2v e = scale_twice<S / 2>(scales);
    r.p[0] = dequant2<0>(w[S], e);
    r.p[1] = dequant2<1>(w[S], e);
    r.p[2] = dequant2<2>(w[S], e);
    r.p[3] = dequant2<3>(w[S], e);
    return r.v;
}

// V's codes with two tokens' values of one column in a byte: pair[q][c] byte b holds column
// 8 (c / 2) + 2 b + c % 2 of tokens 2 q (low nibble) and 2 q + 1.
template <int D>
struct VPairs {
    static constexpr int C = D == 64 ? 2 : D / 64;      // words per pair of tokens
    uint32_t w[2][C];
    half2v e[2];
};

template <int D>
__device__ __forceinline__ void pair_tokens(VPairs<D>& r, const uint32_t (&v)[D / 32], uint32_t scales) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        constexpr int X = D == 64 ? 1 : D / 128;        // words of a token
#pragma unroll
        for (int x = 0; x < X; ++x) {
            uint32_t a, b;
            if constexpr (D == 64) {
                a = v[q];
                b = v[q] >> 16;
            } else {
                a = v[2 * q * X + x];
                b = v[(2 * q + 1) * X + x];
            }
            r.w[q][2 * x] = select_bits(0x0F0F0F0Fu, a, b << 4);
            r.w[q][2 * x + 1] = select_bits(0x0F0F0F0Fu, a >> 4, b);
        }
    }
    scales &= 0x7F7F7F7Fu;
    r.e[0] = scale_pair<0>(scales);
    r.e[1] = scale_pair<1>(scales);
}

template <int N, typename F, int I = 0>
__device__ __forceinline__ void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, F, I + 1>(static_cast<F&&>(f));
    }
}

// Row row of the item's (token, query head) rows: its byte offset in Q or O, and in lse.
struct RowAt {
    int64_t token;
    int32_t head;
};
__device__ __forceinline__ RowAt row_at(int64_t first, int head, int group, int row) {
    const int j = row / group;
    return RowAt{first + j, head * group + row - j * group};
}

// lse of a row from its maximum (log2, the weights' scale of 2^kUp apart) and sum; a sum of zero is a row
// that sees nothing, a NaN (of a query) stays one.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.0f ? -__builtin_inff() : (m - kUp + __builtin_amdgcn_logf(l)) * kLn2;
}

// Work split. Rows of an item and head: (token j, query head of the group), row = j * group + head,
// in tiles; the positions a tile sees in chunks. Lengths are known on the device only, and in a batch
// they differ widely, so each workgroup finds its task itself: a wave sums the positions of all
// tiles, which gives the chunk size that makes about `target` tasks a head (as many as run at once),
// and then finds its own in the prefix sum of the items' tasks. (A grid made for the longest item left most
// workgroups without work and the others unevenly spread: 4 sequences of up to 131072 positions took 81 us
// that way and 57 us so.)
constexpr int kUnit = 128;       // positions by which chunks are cut
constexpr int kMaxScan = 1024;   // items up to which scanning them to find a task is worth its time

struct KvPlan {
    int32_t tile_rows;       // query rows of a workgroup
    int32_t tiles;           // row tiles of the largest item
    int32_t target;          // tasks a head aimed at; 0: no splitting
    int32_t scan;            // tasks are numbered without gaps; else task = item * tiles + tile
    int32_t tasks;           // tasks a head at most
    int32_t fit;             // tasks a head that run at once
    int32_t least;           // units of a chunk at least
    int32_t alone;           // few rows: at most a workgroup for each compute unit, and much for each to do
    int32_t by_item;         // join: workgroups by (item, row of max_q) instead of by token row
    uint64_t page_magic;     // division of a 16-token unit by the units of a page
    uint32_t page_shift;
};

constexpr int kPrefillRows = 128;   // of a workgroup of kv_prefill.hip
void launch_kv_prefill(const KvAttention& a, const KvPlan& p, hipStream_t stream);

// What one tile of an item sees: positions begin .. end - 1 (begin a multiple of 32).
struct KvRange {
    int32_t begin, end;
};

__device__ __forceinline__ KvRange tile_range(const KvAttention& a, int len, int rows_new, int group,
                                              int row0, int rows) {
    KvRange r;
    r.begin = 0;
    r.end = min(len, a.max_kv);
    const int first = len - rows_new + row0 / group;
    if (a.causal) r.end = min(r.end, len - rows_new + (row0 + rows - 1) / group + 1);
    if (a.window > 0) r.begin = (int)max((int64_t)0, (int64_t)first - a.window + 1) & ~31;
    r.end = max(r.end, r.begin);
    return r;
}

__device__ __forceinline__ int units_of(const KvRange& r) {
    return (int)(((int64_t)r.end - r.begin + kUnit - 1) / kUnit);
}

// An item as the kernels use it: its first row and its rows (all of them, and those that exist and are
// asked for), query rows, slot and length.
struct KvWork {
    int32_t first, all_new, rows, slot, len;
};

__device__ __forceinline__ KvWork work_of(const KvAttention& a, int i, int group) {
    KvWork w{0, 0, 0, 0, 0};
    if (i >= a.b.seqs) return w;
    const int32_t total = (int32_t)min((int64_t)a.b.cu[a.b.seqs], a.b.tokens);
    const int32_t next = a.b.cu[i + 1];
    w.first = a.b.cu[i];
    w.all_new = (int32_t)((uint32_t)next - (uint32_t)w.first);
    const KvItem it = kv_item(a.kv, a.b, i);
    w.slot = it.slot;
    w.len = it.len;
    const int32_t last = min(next, total);
    w.rows = w.first < 0 || last <= w.first ? 0 : min(last - w.first, a.max_q) * group;
    return w;
}

// Inclusive prefix sum over the wave's lanes by lane shifts inside rows of 16, then across them.
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {
    static_assert(sizeof(T) == 4, "one register");
    const auto shifted = [](T x, auto control, auto rows) {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(
            0, __builtin_bit_cast(int, x), decltype(control)::value, decltype(rows)::value, 0xF, false));
    };
    using I = std::integral_constant<int, 0xF>;
    v += shifted(v, std::integral_constant<int, 0x111>{}, I{});     // row_shr:1
    v += shifted(v, std::integral_constant<int, 0x112>{}, I{});
    v += shifted(v, std::integral_constant<int, 0x114>{}, I{});
    v += shifted(v, std::integral_constant<int, 0x118>{}, I{});
    v += shifted(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row_bcast:15
    v += shifted(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row_bcast:31
    return v;
}

template <typename T>
__device__ __forceinline__ T last_lane(T v) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

struct KvTask {
    KvWork work;
    int32_t item, tile, chunk, chunks;
    int32_t base;            // the item's first task
    int32_t row0, rows;      // of the tile
    int32_t begin, end;      // positions of the chunk
};

__device__ __forceinline__ int chunks_of(int units, int chunk) {
    return max(1, (int)(((uint32_t)units + (uint32_t)chunk - 1u) / (uint32_t)chunk));
}

// The task of number w (uniform), found by the whole wave; false if there is none.
__device__ __forceinline__ bool find_task(const KvAttention& a, const KvPlan& p, int w, KvTask& t) {
    const int lane = threadIdx.x & 63;
    const int group = a.q_heads / a.kv.heads;
    KvWork mine;
    int inside;
    if (!p.scan) {
        t.item = w / p.tiles;
        mine = work_of(a, t.item, group);
        t.work = mine;
        inside = w - t.item * p.tiles;
        t.base = t.item * p.tiles;
        t.chunks = 1;
    } else {
        float sum = 0.0f;
        int units = 0, tiles = 0;
        for (int i0 = 0; i0 < a.b.seqs; i0 += 64) {
            mine = work_of(a, i0 + lane, group);
            tiles = (mine.rows + p.tile_rows - 1) / p.tile_rows;
            units = mine.rows > 0 ? units_of(tile_range(a, mine.len, mine.all_new, group, 0, mine.rows)) : 0;
            sum += (float)units * (float)tiles;
        }
        // units a chunk: above sum / target whatever binary32 rounded, so that no item has more than
        // `target` chunks and all have at most `target` more than their tiles
        const float share = last_lane(wave_prefix(sum)) / (float)max(p.target, 1);
        int chunk = p.target > 0 ? max((int)min(share * 1.001f, 1e9f) + 1, p.least) : 0x7FFFFFFF;
        if (p.target > 0 && a.b.seqs <= 64) {
            if (p.tiles > 1) {
                // prompts: the longest item in k chunks, k such that the rounds of workgroups times a chunk's
                // length (and a unit's worth of start) is least (8 items of up to 1000 rows over up to 8000
                // positions, 4 heads of 4, 256 wide: 261 us; with `target` tasks, whatever their rounds, 318)
                int longest = units;
#pragma unroll
                for (int o = 32; o >= 1; o >>= 1) longest = max(longest, __shfl_xor(longest, o, 64));
                float best = __builtin_inff();
                for (int k = 1; k <= 16; ++k) {
                    const int size = max((longest + k - 1) / k, p.least);
                    const int all = last_lane(wave_prefix(tiles * chunks_of(units, size)));
                    if (all > p.tasks) break;
                    const float cost = (float)((all + p.fit - 1) / p.fit) * (float)(size + 1);
                    if (cost < best) {
                        best = cost;
                        chunk = size;
                    }
                    if (size == p.least) break;
                }
            } else if (last_lane(wave_prefix(tiles)) < p.fit) {
                // every item's chunks are rounded up: larger ones until all tasks run at once, if they can
                for (int i = 0; i < 16; ++i) {
                    const int all = last_lane(wave_prefix(tiles * chunks_of(units, chunk)));
                    if (all <= p.fit) break;
                    chunk += max(1, chunk >> 3);
                }
            }
        }
        int before = 0;
        bool found = false;
        for (int i0 = 0; i0 < a.b.seqs && !found; i0 += 64) {
            if (a.b.seqs > 64) {
                mine = work_of(a, i0 + lane, group);
                tiles = (mine.rows + p.tile_rows - 1) / p.tile_rows;
                units = mine.rows > 0 ? units_of(tile_range(a, mine.len, mine.all_new, group, 0, mine.rows)) : 0;
            }
            const int chunks = chunks_of(units, chunk);
            const int tasks = tiles * chunks;
            const int incl = wave_prefix(tasks);
            const uint64_t past = __ballot(before + incl > w);
            if (past != 0) {
                const int src = __builtin_ctzll(past);
                found = true;
                t.item = i0 + src;
                t.base = before + __builtin_amdgcn_readlane(incl - tasks, src);
                t.chunks = __builtin_amdgcn_readlane(chunks, src);
                t.work.first = __builtin_amdgcn_readlane(mine.first, src);
                t.work.all_new = __builtin_amdgcn_readlane(mine.all_new, src);
                t.work.rows = __builtin_amdgcn_readlane(mine.rows, src);
                t.work.slot = __builtin_amdgcn_readlane(mine.slot, src);
                t.work.len = __builtin_amdgcn_readlane(mine.len, src);
            }
            before += last_lane(incl);
        }
        if (!found) return false;
        inside = w - t.base;
    }
    // the last tile of a causal item sees the most: it comes first
    const int tiles = (t.work.rows + p.tile_rows - 1) / p.tile_rows;
    t.chunk = tiles > 0 ? inside / tiles : 0;
    t.tile = tiles - 1 - (inside - t.chunk * tiles);
    if (t.tile < 0 || t.chunk >= t.chunks) return false;
    t.row0 = t.tile * p.tile_rows;
    t.rows = min(p.tile_rows, t.work.rows - t.row0);
    const KvRange r = tile_range(a, t.work.len, t.work.all_new, group, t.row0, t.rows);
    const int64_t units = units_of(r);
    t.begin = r.begin + (int)(units * t.chunk / t.chunks) * kUnit;
    t.end = t.chunk + 1 == t.chunks ? r.end
                                    : min(r.end, r.begin + (int)(units * (t.chunk + 1) / t.chunks) * kUnit);
    return true;
}

// Workspace of a split batch: (first task, chunks) of every item; then for every task and head the tile's
// (maximum, sum) of each row, and its outputs (binary32, scaled like the weights).
__device__ __forceinline__ int2* item_info(const KvAttention& a) {
    return static_cast<int2*>(a.workspace);
}
__device__ __forceinline__ float2* part_stat(const KvAttention& a, const KvPlan& p, int task, int head) {
    return reinterpret_cast<float2*>(static_cast<int2*>(a.workspace) + (a.b.seqs + 1) / 2 * 2) +
           ((int64_t)task * a.kv.heads + head) * p.tile_rows;
}
__device__ __forceinline__ float* part_out(const KvAttention& a, const KvPlan& p, int task, int head) {
    float* out = reinterpret_cast<float*>(part_stat(a, p, p.tasks, 0));
    return out + ((int64_t)task * a.kv.heads + head) * p.tile_rows * a.kv.dim;
}

}  // namespace nvfp4
