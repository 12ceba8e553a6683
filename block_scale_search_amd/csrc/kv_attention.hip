// Attention over the paged NVFP4 key/value cache for gfx950.
//
// Few rows per (item, key/value head) - decode steps and drafts: k_kv_decode. A wave owns tiles of 32
// positions and 16 RT query rows. S^T = K Q^T puts a query row in a lane column: the f16 MFMA 16x16x32
// gives lane (n, g) = (lane % 16, lane / 16) the logits of row n at positions 4g .. 4g + 3 of each half
// tile. O^T = V^T P^T needs, in that same lane, the weights of row n at 8 positions: any 8, as long as
// V's operand uses the same ones, so the logits' registers are the weights' registers and no lane
// exchanges anything. V's operand then holds, for lane (n, g), the positions 4g .. 4g + 3 of both half
// tiles and the values d = n D/16 + j of tile j: the record layout keeps exactly those codes together,
// 4 tokens x D/16 values in one load.
// A row's running maximum is only raised when a logit exceeds it by more than 2^7 (weights are
// scaled by 2^8 and stay below 2^15), so most tiles need no cross-lane step and no rescaling.
// The waves of a workgroup take tiles in turn and are joined in LDS; the chunks of a long
// sequence are joined by k_kv_join.
//
// What bounds it is HBM, and before that the loads' order: read from the pages in the operands' order, a tile
// touches each 128-byte line several times, and a touch of a line that is still on its way waits for it. So a
// wave copies whole tiles into its own ring in LDS, each line once and one tile ahead, and reads operands
// there. 64 rows of 4 heads over up to 8192 positions, 8 key/value heads, 128 wide (247.5 MB): 54 us
// (4.6 TB/s; straight from the pages 72) and the join 5; 4 rows of 8 over up to 131072 (238 MB): 45
// (5.3 TB/s) and 5. A large copy runs at 5.0 TB/s. Few short sequences are bound by what one compute unit
// can have on its way (about 28 GB/s) and by the chain of launch, task, length, page and tile: one row over
// 1023 positions 12 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "internal.h"
#include "kv_attention_device.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kUnits = 256;          // compute units
constexpr int kMaxSplits = 1024;     // chunks of a row
constexpr int64_t kMaxGrid = (int64_t)1 << 24;   // workgroups: 2^32 threads a launch
// Rows up to which k_kv_decode takes an item (in tiles of 16 or 32). Above, kv_prefill.hip shares the
// conversion of a tile: 46 items of 112 rows over up to 10596 positions, 2 heads, 54 us (here 74), of 40
// rows 42 (here 42).
constexpr int kFewRows = 32;
// The join gives a row a workgroup below this many rows, a wave above: 256 rows of 17 chunks 55.9 us in all
// (a wave each 56.7), 1920 rows of few chunks 17.5 (a workgroup each 21).
constexpr int kWideJoin = 1024;

// A tile of 32 positions in LDS, as it is copied from the pages: the codes of [K half 0][K half 1]
// [V half 0][V half 1], then their scale bytes in the same order. In K's rows the 16-byte pieces
// are permuted (piece c of row n at c ^ f(n)), so that 16 lanes reading one piece of 16 rows use all
// banks; the copy's source addresses carry the permutation.
template <int D>
struct TileLds {
    static constexpr int kHalf = 8 * D;                  // code bytes of a half
    static constexpr int kScales = 4 * kHalf;
    static constexpr int kBytes = kScales + 4 * D;
    static constexpr int kCodeLoads = kScales / 1024;    // 64 lanes x 16 bytes each
    static constexpr int kLoads = kCodeLoads + 1;
    static constexpr int kPieces = D / 32;               // of a row of K
    static constexpr int kShift = D == 64 ? 3 : D == 128 ? 2 : 1;
    static __device__ __forceinline__ int f(int n) { return (n >> kShift) & (kPieces - 1); }
};

// A lane's source offsets in the records: load j of a tile's codes, and the scales (lane < D / 4).
template <int D>
struct CopyOffsets {
    uint32_t code[TileLds<D>::kCodeLoads], scale;
};

template <int D>
__device__ __forceinline__ CopyOffsets<D> copy_offsets(const KvView& kv, int head, int lane) {
    using T = TileLds<D>;
    const uint32_t region = (uint32_t)kv_code_bytes(kv);
    CopyOffsets<D> o;
#pragma unroll
    for (int j = 0; j < T::kCodeLoads; ++j) {
        const uint32_t at = 1024 * j + 16 * lane, part = at / T::kHalf;
        uint32_t in = at % T::kHalf;
        if (part < 2) {                                  // K: the piece that belongs at this place
            const uint32_t n = in / (D / 2), c = in % (D / 2) / 16;
            in = n * (D / 2) + (c ^ T::f(n)) * 16;
        }
        o.code[j] = (uint32_t)head * kv.page * (D / 2) + in + (part < 2 ? 0 : region);
    }
    const uint32_t at = 16 * lane, part = at / D;
    o.scale = 2 * region + (uint32_t)head * kv.page * (D / 16) + at % D +
              (part < 2 ? 0 : region >> 3);
    return o;
}

typedef __attribute__((address_space(1))) const void* GlobalPtr;
typedef __attribute__((address_space(3))) void* LdsPtr;

// 16 bytes a lane from global memory to lds + 16 * lane (lds uniform).
__device__ __forceinline__ void copy16(const uint8_t* src, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)lds, 16, 0, 0);
}

// Copies a tile: rec[u] and row[u] are the record and first row of half u (uniform).
template <int D>
__device__ __forceinline__ void copy_tile(uint8_t* lds, const uint8_t* rec0, int row0,
                                          const uint8_t* rec1, int row1, const CopyOffsets<D>& o,
                                          int lane) {
    using T = TileLds<D>;
    const uint8_t* c0 = rec0 + (int64_t)row0 * (D / 2);
    const uint8_t* c1 = rec1 + (int64_t)row1 * (D / 2);
#pragma unroll
    for (int j = 0; j < T::kCodeLoads; ++j) {
        const bool second = D == 64 ? lane >= 32 : (1024 * j / T::kHalf) & 1;
        copy16((second ? c1 : c0) + o.code[j], lds + 1024 * j);
    }
    const uint8_t* s0 = rec0 + (int64_t)row0 * (D / 16);
    const uint8_t* s1 = rec1 + (int64_t)row1 * (D / 16);
    if (lane < D / 4) copy16(((16 * lane / D) & 1 ? s1 : s0) + o.scale, lds + T::kScales);
}

// A lane's LDS addresses in a tile, for lane (n, g).
struct ReadOffsets {
    uint32_t k[2], v, ks, vs;
};

template <int D>
__device__ __forceinline__ ReadOffsets read_offsets(int n, int g) {
    using T = TileLds<D>;
    ReadOffsets r;
    if constexpr (D == 64) {
        r.k[0] = r.k[1] = n * 32 + ((g >> 1) ^ T::f(n)) * 16 + (g & 1) * 8;
    } else if constexpr (D == 128) {
        r.k[0] = r.k[1] = n * 64 + (g ^ T::f(n)) * 16;
    } else {
        r.k[0] = n * 128 + ((2 * g) ^ T::f(n)) * 16;
        r.k[1] = n * 128 + ((2 * g + 1) ^ T::f(n)) * 16;
    }
    r.v = 2 * T::kHalf + (g * 16 + n) * (D / 8);
    r.ks = T::kScales + n * (D / 16) + g * (D / 64);
    r.vs = T::kScales + 2 * D + (g * (D / 16) + n * D / 256) * 4;
    return r;
}

// Reads a tile into registers. The reads and their wait are one block: the copies into other tiles of
// the ring stay in flight, which the compiler's own waits for LDS reads would not allow.
template <int D>
__device__ __forceinline__ void read_tile(HalfTile<D> (&h)[2], uint32_t base, const ReadOffsets& o) {
    constexpr int H = TileLds<D>::kHalf;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t k = base + o.k[0], v = base + o.v, ks = base + o.ks, vs = base + o.vs;
    if constexpr (D == 64) {
        u32x2 k0, k1, v0, v1;
        asm volatile(
            "ds_read_b64 %0, %8\n ds_read_b64 %1, %8 offset:%c12\n"
            "ds_read_b64 %2, %9\n ds_read_b64 %3, %9 offset:%c12\n"
            "ds_read_u8 %4, %10\n ds_read_u8 %5, %10 offset:%c13\n"
            "ds_read_b32 %6, %11\n ds_read_b32 %7, %11 offset:%c13\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(k0), "=&v"(k1), "=&v"(v0), "=&v"(v1), "=&v"(h[0].ks), "=&v"(h[1].ks),
              "=&v"(h[0].vs), "=&v"(h[1].vs)
            : "v"(k), "v"(v), "v"(ks), "v"(vs), "n"(H), "n"(D)
            : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[0].k[i] = k0[i]; h[1].k[i] = k1[i]; h[0].v[i] = v0[i]; h[1].v[i] = v1[i];
        }
    } else if constexpr (D == 128) {
        u32x4 k0, k1, v0, v1;
        asm volatile(
            "ds_read_b128 %0, %8\n ds_read_b128 %1, %8 offset:%c12\n"
            "ds_read_u16 %4, %10\n ds_read_u16 %5, %10 offset:%c13\n"
            "ds_read_b128 %2, %9\n ds_read_b128 %3, %9 offset:%c12\n"
            "ds_read_b32 %6, %11\n ds_read_b32 %7, %11 offset:%c13\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(k0), "=&v"(k1), "=&v"(v0), "=&v"(v1), "=&v"(h[0].ks), "=&v"(h[1].ks),
              "=&v"(h[0].vs), "=&v"(h[1].vs)
            : "v"(k), "v"(v), "v"(ks), "v"(vs), "n"(H), "n"(D)
            : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[0].k[i] = k0[i]; h[1].k[i] = k1[i]; h[0].v[i] = v0[i]; h[1].v[i] = v1[i];
        }
    } else {
        u32x4 k0, k1, k2, k3, v0, v1, v2, v3;
        const uint32_t kb = base + o.k[1];
        asm volatile(
            "ds_read_b128 %0, %12\n ds_read_b128 %1, %13\n"
            "ds_read_b128 %2, %12 offset:%c17\n ds_read_b128 %3, %13 offset:%c17\n"
            "ds_read_b32 %8, %15\n ds_read_b32 %9, %15 offset:%c18\n"
            "ds_read_b128 %4, %14\n ds_read_b128 %5, %14 offset:16\n"
            "ds_read_b128 %6, %14 offset:%c17\n ds_read_b128 %7, %14 offset:%c19\n"
            "ds_read_b32 %10, %16\n ds_read_b32 %11, %16 offset:%c18\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(k0), "=&v"(k1), "=&v"(k2), "=&v"(k3), "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3),
              "=&v"(h[0].ks), "=&v"(h[1].ks), "=&v"(h[0].vs), "=&v"(h[1].vs)
            : "v"(k), "v"(kb), "v"(v), "v"(ks), "v"(vs), "n"(H), "n"(D), "n"(H + 16)
            : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[0].k[i] = k0[i]; h[0].k[4 + i] = k1[i]; h[1].k[i] = k2[i]; h[1].k[4 + i] = k3[i];
            h[0].v[i] = v0[i]; h[0].v[4 + i] = v1[i]; h[1].v[i] = v2[i]; h[1].v[4 + i] = v3[i];
        }
    }
}

template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%c0)" ::"n"(N) : "memory");
}
// Waits until at most `behind` tiles (0 .. N) of L copies each are in flight.
template <int L, int N>
__device__ __forceinline__ void wait_behind(int behind) {
    if constexpr (N == 0) {
        wait_copies<0>();
    } else if (behind == N) {
        wait_copies<N * L>();
    } else {
        wait_behind<L, N - 1>(behind);
    }
}

// V operand of output tile J: column J of the lane's D/16, tokens 4g .. 4g + 3 of both half tiles.
template <int D, int J>
__device__ __forceinline__ half8v v_operand(const VPairs<D> (&h)[2]) {
    constexpr int c = 2 * (J / 8) + (J & 1), b = (J & 7) >> 1;
    Half8 r;
    r.p[0] = dequant2<b>(h[0].w[0][c], h[0].e[0]);
    r.p[1] = dequant2<b>(h[0].w[1][c], h[0].e[1]);
    r.p[2] = dequant2<b>(h[1].w[0][c], h[1].e[0]);
    r.p[3] = dequant2<b>(h[1].w[1][c], h[1].e[1]);
    return r.v;
}

__device__ __forceinline__ f32x4 mfma(half8v a, half8v b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A lane's query values as f16 operands: row n of row tile rt, values g D/4 + 8 s .. + 7 of step s.
template <int D, bool BF16>
struct QRow {
    half8v hi[D / 32];
    half8v lo[BF16 ? 1 : D / 32];
    float f;                 // logit (log2) of a product
};

// A lane's query values as they lie in memory (zeros for no row).
template <int D, bool BF16>
struct RawQuery {
    static constexpr int W = BF16 ? D / 32 : D / 16;
    uint4 w[W];
};

template <int D, bool BF16>
__device__ __forceinline__ void load_query(RawQuery<D, BF16>& r, const uint8_t* p, bool live, int g) {
    constexpr int W = RawQuery<D, BF16>::W;
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[g * W + i];
    }
}

template <int D, bool BF16>
__device__ __forceinline__ void convert_query(QRow<D, BF16>& q, const RawQuery<D, BF16>& r, float scale,
                                              float S) {
    float x[D / 4];
#pragma unroll
    for (int i = 0; i < RawQuery<D, BF16>::W; ++i) {
        const uint32_t d[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BF16) {
                x[8 * i + 2 * k] = bf16_lo(d[k]);
                x[8 * i + 2 * k + 1] = bf16_hi(d[k]);
            } else {
                x[4 * i + k] = __uint_as_float(d[k]);
            }
        }
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
    top = max_groups(top);
    const int k = row_exponent(top);
    const float up = row_factor(k, top, S);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = x[8 * s + j] * up;
            const _Float16 h = (_Float16)v;
            q.hi[s][j] = h;
            if constexpr (!BF16) q.lo[s][j] = (_Float16)(v - (float)h);
        }
    }
    // at least the smallest normal number: a masked logit of -infinity times it stays -infinity
    q.f = fmaxf(__builtin_ldexpf(scale, -k) * (S * kLog2e), 0x1p-126f);
}

// Waves a SIMD should hold: as many as the accumulators and two tiles in flight leave room for. (f32 queries take
// more: at 32 rows 21 registers are spilled 64 wide, 36 at 256.)
template <int D, int RT>
constexpr int kOccupancy = D * RT <= 128 ? 4 : D * RT <= 256 ? 2 : 1;

// Waves of a workgroup and tiles of a wave in LDS. Four waves with two tiles, so that a compute unit holds
// as many waves as its registers (three tiles: 64 rows over up to 8192 positions 70 us, not 63). A
// workgroup that has a compute unit to itself (`ALONE`) takes its whole LDS: eight waves and what fits
// (one row over 1023 positions 12.2 us, with four and two 13.0; up to 512 positions and 256 wide they are
// no slower).
template <int D, bool ALONE>
struct Shape {
    static constexpr int kWaves = ALONE ? 8 : 4;
    static constexpr int kDepth = ALONE ? 4096 / D / kWaves : 2;
};

template <int D, bool BF16, int RT, bool ALONE>
__global__ __launch_bounds__((64 * Shape<D, ALONE>::kWaves), (ALONE ? 2 : kOccupancy<D, RT>))
void k_kv_decode(KvAttention a, KvPlan plan) {
    constexpr int kWaves = Shape<D, ALONE>::kWaves, kThreads = 64 * kWaves;
    constexpr int kDepth = Shape<D, ALONE>::kDepth;
    constexpr int R = 16 * RT, NJ = D / 16, NS = D / 32;
    constexpr int JC = NJ < 8 ? NJ : 8;                  // output tiles joined at a time
    using T = TileLds<D>;
    constexpr int kRing = kDepth * T::kBytes;            // a wave's tiles; later the joined outputs
    constexpr int kRow = JC * 16 + 4;
    constexpr int kJoin = 16 * kRow * 4;
    __shared__ __align__(16) uint8_t space[kWaves * (kRing > kJoin ? kRing : kJoin)];
    float(*joined)[16][kRow] = reinterpret_cast<float(*)[16][kRow]>(space);
    __shared__ float2 stat[kWaves][R];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvView& kv = a.kv;

    // work of this workgroup: head fastest
    const int task = (int)(blockIdx.x / (uint32_t)kv.heads);
    const int head = (int)(blockIdx.x - (uint32_t)task * (uint32_t)kv.heads);
    const int group = a.q_heads / kv.heads;
    KvTask job;
    if (!find_task(a, plan, task, job)) return;
    const int64_t first = job.work.first;
    const int all_new = job.work.all_new, row0 = job.row0, rows = job.rows;
    const int begin = job.begin, end = job.end;
    const bool whole = job.chunks <= 1;
    if (plan.target > 0 && head == 0 && job.chunk == 0 && job.tile == 0 && threadIdx.x == 0)
        item_info(a)[job.item] = make_int2(job.base, job.chunks);

    RawQuery<D, BF16> raw[RT];
    int low[RT], lim[RT];                                // the lane's row sees low .. lim - 1
    int low_all = 0, lim_all = end;                      // and so does every row
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const bool live = 16 * rt + n < rows;
        const RowAt of = row_at(first, head, group, live ? row0 + 16 * rt + n : row0);
        load_query<D, BF16>(raw[rt], static_cast<const uint8_t*>(a.q.p) + of.token * a.q.stride_t +
                                         of.head * a.q.stride_h, live, g);
        const int pos = job.work.len - all_new + (int)(of.token - first);
        low[rt] = a.window > 0 ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
        lim[rt] = a.causal ? min(end, pos + 1) : end;
    }
    {
        const int p0 = job.work.len - all_new + row0 / group;
        const int p1 = job.work.len - all_new + (row0 + rows - 1) / group;
        if (a.causal) lim_all = min(end, p0 + 1);
        if (a.window > 0) low_all = (int)max((int64_t)p1 - a.window + 1, (int64_t)0);
    }

    f32x4 o[RT][NJ];
    float m[RT], sub[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -__builtin_inff();
        sub[rt] = 0.0f;
        l[rt] = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[rt][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    constexpr int kStep = 32 * kWaves;
    const CopyOffsets<D> from = copy_offsets<D>(kv, head, lane);
    const ReadOffsets at = read_offsets<D>(n, g);
    uint8_t* ring = space + wave * kRing;
    const uint32_t ring_at = (uint32_t)(uintptr_t)(LdsPtr)ring;
    const int32_t* table = kv.table + (int64_t)job.work.slot * kv.max_pages;
    const int32_t units = kv.page >> 4;
    const int t0 = begin + 32 * wave;
    const int tiles = t0 < end ? (end - t0 + kStep - 1) / kStep : 0;    // of this wave
    // Where the wave's next 64 tiles lie, lane i the i-th: page (-1: the table names none) and first row
    // of each half tile. One vector load of the table every 64 tiles instead of a dependent scalar
    // load in front of every tile's copies.
    int32_t page[2], row[2];
    uint32_t named = 0;                                  // two bits a tile, the latest lowest
    const auto copy = [&](int i) {
        if ((i & 63) == 0) {
            const int64_t t = t0 + (int64_t)(i + lane) * kStep;
            const bool in = t < end;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int unit = in ? (int)(t >> 4) + u : 0;
                const int col = (int)div_gpr((uint32_t)unit, plan.page_magic, plan.page_shift);
                row[u] = (unit - col * units) << 4;
                page[u] = in && col < kv.max_pages ? table[col] : -1;
            }
        }
        const uint8_t* rec[2];
        int r[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pg = __builtin_amdgcn_readlane(page[u], i & 63);
            const bool ok = (uint32_t)pg < (uint32_t)kv.num_pages;
            named = named << 1 | (ok ? 1u : 0u);
            rec[u] = kv.pages + (int64_t)(ok ? pg : 0) * kv.page_stride;
            r[u] = __builtin_amdgcn_readlane(row[u], i & 63);
        }
        copy_tile<D>(ring + i % kDepth * T::kBytes, rec[0], r[0], rec[1], r[1], from, lane);
    };
    struct Tile {
        HalfTile<D> h[2];
        bool ok[2];
    };
    for (int i = 0; i < kDepth - 1 && i < tiles; ++i) copy(i);
    QRow<D, BF16> q[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) convert_query<D, BF16>(q[rt], raw[rt], a.scale, kv.S_k[head]);
    const auto process = [&](int t, const Tile& x) {
        f32x4 s[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t scales = x.h[u].ks & 0x7F7F7F7Fu;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            unroll<NS>([&](auto step) {
                constexpr int S = decltype(step)::value;
                const half8v k = k_operand<S>(x.h[u].k, scales);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s[rt][u] = mfma(k, q[rt].hi[S], s[rt][u]);
                    if constexpr (!BF16) s[rt][u] = mfma(k, q[rt].lo[S], s[rt][u]);
                }
            });
        }
        if (!(x.ok[0] && x.ok[1] && t >= low_all && t + 32 <= lim_all)) {
            asm volatile("");                            // a branch, not selects in every tile
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = t + 16 * u + 4 * g + i;
                        if (!(x.ok[u] && p >= low[rt] && p < lim[rt]))
                            s[rt][u][i] = -__builtin_inff();
                    }
        }
        __builtin_amdgcn_sched_barrier(0);
        Half8 hi[RT], lo[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = fmaxf(fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3])),
                              fmaxf(fmaxf(s[rt][1][0], s[rt][1][1]), fmaxf(s[rt][1][2], s[rt][1][3])));
            top *= q[rt].f;
            if (__any(top > m[rt] + kSlack)) {
                const float al = raise_row(m[rt], sub[rt], max_groups(top), kSlack);
                l[rt] *= al;
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[rt][j] *= al;
            }
            float pr[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                pr[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i >> 2][i & 3], q[rt].f, sub[rt]));
            l[rt] += ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[rt].p[i] = half2v{(_Float16)pr[2 * i], (_Float16)pr[2 * i + 1]};
                if constexpr (!BF16)
                    lo[rt].p[i] = half2v{(_Float16)(pr[2 * i] - (float)hi[rt].p[i][0]),
                                         (_Float16)(pr[2 * i + 1] - (float)hi[rt].p[i][1])};
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        VPairs<D> vp[2];
        pair_tokens<D>(vp[0], x.h[0].v, x.h[0].vs);
        pair_tokens<D>(vp[1], x.h[1].v, x.h[1].vs);
        unroll<NJ>([&](auto tile_j) {
            constexpr int J = decltype(tile_j)::value;
            const half8v v = v_operand<D, J>(vp);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                o[rt][J] = mfma(v, hi[rt].v, o[rt][J]);
                if constexpr (!BF16) o[rt][J] = mfma(v, lo[rt].v, o[rt][J]);
            }
        });
    };
    // a ring of kDepth tiles a wave: tile i is processed while the next ones are copied
    for (int i = 0; i < tiles; ++i) {
        Tile x;
        const int behind = min(kDepth - 1, tiles - 1 - i);   // tiles in flight after this one
        if (i + kDepth - 1 < tiles) copy(i + kDepth - 1);    // its place was read an iteration ago
        wait_behind<T::kLoads, kDepth - 1>(behind);
        x.ok[0] = (named >> (2 * behind + 1)) & 1u;
        x.ok[1] = (named >> (2 * behind)) & 1u;
        read_tile<D>(x.h, ring_at + i % kDepth * T::kBytes, at);
        process(t0 + i * kStep, x);
    }
    __syncthreads();                                     // the rings become the joined outputs

    // join the waves: the rows' maxima and sums, then the outputs scaled to the joint maximum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = sum_groups(l[rt]);
        if (g == 0) stat[wave][16 * rt + n] = make_float2(m[rt], l[rt]);
    }
    __syncthreads();
    const float S_v = kv.S_v[head];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        float mm = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < kWaves; ++k) mm = fmaxf(mm, stat[k][16 * rt + n].x);
        const float f = m[rt] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[rt] - mm);
#pragma unroll
        for (int jc = 0; jc < NJ / JC; ++jc) {
            if (rt + jc > 0) __syncthreads();
            // value d = (4 g + i) NJ + j of row n; this pass holds j in jc JC .. + JC - 1 as column
            // (4 g + i) JC + j % JC
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < JC; j += 4) {
                    const int J = jc * JC + j;
                    *reinterpret_cast<float4*>(&joined[wave][n][(4 * g + i) * JC + j]) =
                        make_float4(o[rt][J][i] * f, o[rt][J + 1][i] * f, o[rt][J + 2][i] * f,
                                    o[rt][J + 3][i] * f);
                }
            __syncthreads();
            // 4 columns a thread and step: the row's joint statistics, then the sum of the waves
            for (int e = threadIdx.x; e < 16 * JC * 4; e += kThreads) {
                const int r = e / (JC * 4), c = (e - r * (JC * 4)) * 4;
                if (16 * rt + r >= rows) continue;
                float rm = -__builtin_inff(), rl = 0.0f;
#pragma unroll
                for (int k = 0; k < kWaves; ++k) rm = fmaxf(rm, stat[k][16 * rt + r].x);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kWaves; ++k) {
                    const float2 sk = stat[k][16 * rt + r];
                    if (sk.y != 0.0f) rl += sk.y * __builtin_amdgcn_exp2f(sk.x - rm);
                    const float4 x = *reinterpret_cast<const float4*>(&joined[k][r][c]);
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                }
                const int d = (c / JC) * NJ + jc * JC + c % JC;
                const RowAt of = row_at(first, head, group, row0 + 16 * rt + r);
                if (whole) {
                    const int64_t row = of.token * a.q_heads + of.head;
                    const float z = rl == 0.0f ? 0.0f : S_v / rl;
                    uint8_t* dst = static_cast<uint8_t*>(a.out) + of.token * a.out_stride_t +
                                   of.head * a.out_stride_h;
                    if constexpr (BF16)
                        *reinterpret_cast<uint2*>(dst + 2 * d) =
                            make_uint2(bf16_pair(v.x * z, v.y * z), bf16_pair(v.z * z, v.w * z));
                    else
                        *reinterpret_cast<float4*>(dst + 4 * d) =
                            make_float4(v.x * z, v.y * z, v.z * z, v.w * z);
                    if (a.lse && d == 0) a.lse[row] = row_lse(rm, rl);
                } else {
                    *reinterpret_cast<float4*>(part_out(a, plan, task, head) + (16 * rt + r) * D + d) = v;
                    if (d == 0) part_stat(a, plan, task, head)[16 * rt + r] = make_float2(rm, rl);
                }
            }
        }
    }
}

// What joins a row's chunks: where its outputs go, its chunks' statistics and outputs (chunk s at
// s * stat_step and s * stat_step * D).
struct JoinRow {
    int64_t row;
    uint8_t* dst;
    const float2* stat;
    const float* part;
    int64_t stat_step;
    int head, chunks;
};

// Number `index` of the rows to join (uniform); false if there is none or it has one chunk, which is
// already its output.
__device__ __forceinline__ bool find_row(const KvAttention& a, const KvPlan& plan, uint32_t index,
                                         JoinRow& r) {
    const KvView& kv = a.kv;
    const int64_t at = index / (uint32_t)a.q_heads;
    const int hq = (int)(index - (uint32_t)at * (uint32_t)a.q_heads);
    const int group = a.q_heads / kv.heads;
    r.head = hq / group;
    const int64_t total = min((int64_t)a.b.cu[a.b.seqs], a.b.tokens);
    int item;
    int64_t j;
    if (plan.by_item) {
        item = (int)(at / a.max_q);
        if (item >= a.b.seqs) return false;
        j = at - (int64_t)item * a.max_q;
    } else {
        if (at >= total) return false;
        item = kv_find_item(a.b.cu, a.b.seqs, at);
        j = at - a.b.cu[item];
    }
    const int2 info = item_info(a)[item];
    const int64_t first = a.b.cu[item];
    const int64_t last = min((int64_t)a.b.cu[item + 1], total);
    if (first < 0 || last <= first) return false;
    const int n_new = (int)(last - first);
    if (j < 0 || j >= min(n_new, a.max_q)) return false;
    const int64_t token = first + j;
    r.row = token * a.q_heads + hq;
    r.dst = static_cast<uint8_t*>(a.out) + token * a.out_stride_t + hq * a.out_stride_h;
    const int q = (int)j * group + hq - r.head * group;
    const int tile = q / plan.tile_rows, inside = q - tile * plan.tile_rows;
    const int tiles = (min(n_new, a.max_q) * group + plan.tile_rows - 1) / plan.tile_rows;
    // chunk s of this row's tile: task info.x + s * tiles + (tiles - 1 - tile)
    const int task0 = info.x + tiles - 1 - tile;
    r.chunks = min(min(info.y, kMaxSplits), (plan.tasks - task0 + tiles - 1) / tiles);
    if (task0 < 0 || r.chunks <= 1) return false;        // (offsets that overlap: no task may have said)
    r.stat_step = (int64_t)tiles * kv.heads * plan.tile_rows;
    r.stat = part_stat(a, plan, task0, r.head) + inside;
    r.part = part_out(a, plan, task0, r.head) + inside * kv.dim;
    return true;
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 fma4(float4 a, float f, float4 b) {
    return make_float4(__builtin_fmaf(a.x, f, b.x), __builtin_fmaf(a.y, f, b.y),
                       __builtin_fmaf(a.z, f, b.z), __builtin_fmaf(a.w, f, b.w));
}

template <bool BF16>
__device__ __forceinline__ void store_row(const KvAttention& a, const JoinRow& r, int c, float4 v, float m,
                                          float l) {
    const float z = l == 0.0f ? 0.0f : a.kv.S_v[r.head] / l;
    if constexpr (BF16)
        reinterpret_cast<uint2*>(r.dst)[c] =
            make_uint2(bf16_pair(v.x * z, v.y * z), bf16_pair(v.z * z, v.w * z));
    else
        reinterpret_cast<float4*>(r.dst)[c] = make_float4(v.x * z, v.y * z, v.z * z, v.w * z);
    if (a.lse && c == 0) a.lse[r.row] = row_lse(m, l);
}

// Joins the chunks of a row. WIDE: one workgroup a row, for few rows of many chunks; else one wave a row. Its
// lanes own D / 4 columns, (lanes) / (D / 4) chunks at a time, four loads in flight each, and the first
// chunks' outputs are on their way while the factors are made.
template <int D, bool BF16, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_kv_join(KvAttention a, KvPlan plan) {
    constexpr int C = D / 4, P = (WIDE ? kThreads : 64) / C;   // column lanes, chunks at a time
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    JoinRow r;
    if (!find_row(a, plan, WIDE ? blockIdx.x : blockIdx.x * kWaves + wave, r)) return;
    const int c = (WIDE ? (int)threadIdx.x : lane) % C, p = (WIDE ? (int)threadIdx.x : lane) / C;
    const float4* part = reinterpret_cast<const float4*>(r.part) + c;
    const int64_t step = r.stat_step * C;
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 x[4], v = none;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = p + k * P < r.chunks ? part[(p + k * P) * step] : none;
    if constexpr (WIDE) {
        __shared__ float factor[kMaxSplits], red[kWaves], sums[kWaves];
        __shared__ float4 acc[P][C];
        float mm = -__builtin_inff(), l = 0.0f;
        for (int s = threadIdx.x; s < r.chunks; s += kThreads) mm = fmaxf(mm, r.stat[s * r.stat_step].x);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o, 64));
        if (lane == 0) red[wave] = mm;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWaves; ++k) mm = fmaxf(mm, red[k]);
        for (int s = threadIdx.x; s < r.chunks; s += kThreads) {
            const float2 st = r.stat[s * r.stat_step];
            const float f = st.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(st.x - mm);
            factor[s] = f;
            l = __builtin_fmaf(st.y, f, l);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, 64);
        if (lane == 0) sums[wave] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) l += sums[k];
        for (int s = p; s < r.chunks; s += 4 * P) {
            if (s > p) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = s + k * P < r.chunks ? part[(s + k * P) * step] : none;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v = fma4(x[k], s + k * P < r.chunks ? factor[s + k * P] : 0.0f, v);
        }
        acc[p][c] = v;
        __syncthreads();
        if (p > 0) return;
        v = acc[0][c];
#pragma unroll
        for (int k = 1; k < P; ++k) v = add4(v, acc[k][c]);
        store_row<BF16>(a, r, c, v, mm, l);
    } else {
        // 64 chunks a round, a lane's statistics in registers
        float m = -__builtin_inff(), l = 0.0f;
        for (int s0 = 0; s0 < r.chunks; s0 += 64) {
            const float2 st = s0 + lane < r.chunks ? r.stat[(s0 + lane) * r.stat_step]
                                                   : make_float2(-__builtin_inff(), 0.0f);
            float mn = st.x;
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) mn = fmaxf(mn, __shfl_xor(mn, o, 64));
            mn = fmaxf(m, mn);
            const float al = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - mn);
            const float f = st.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(st.x - mn);
            m = mn;
            l = __builtin_fmaf(l, al, st.y * f);
            v = make_float4(v.x * al, v.y * al, v.z * al, v.w * al);
            const int n = min(64, r.chunks - s0);
            for (int s1 = 0; s1 < n; s1 += 4 * P) {          // uniform: every lane joins each shuffle
                const int s = s1 + p;
                if (s0 + s1 > 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = s + k * P < n ? part[(s0 + s + k * P) * step] : none;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float w = __shfl(f, (s + k * P) & 63, 64);
                    v = fma4(x[k], s + k * P < n ? w : 0.0f, v);
                }
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, 64);
#pragma unroll
        for (int o = C; o < 64; o <<= 1)
            v = add4(v, make_float4(__shfl_xor(v.x, o, 64), __shfl_xor(v.y, o, 64),
                                    __shfl_xor(v.z, o, 64), __shfl_xor(v.w, o, 64)));
        if (p == 0) store_row<BF16>(a, r, c, v, m, l);
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a batch is split: row tiles of 16, 32 or (prompts) 128 rows, and where these alone do not fill the
// chip, chunks of positions. span: the most positions a row tile sees. Splitting costs the join, about 5 us:
// a decode batch is split where its tiles leave workgroup slots empty and a tile may have more than 10
// units of work, or more the more tiles there are: those load the chip without it, unless lengths differ
// (8 heads of 4: 16 rows over 1400 positions 19 us, not split 16; 64 over 1400 33 and 25, over up to 8192,
// ragged, 63 and 83; 8 heads of 8: 4 over up to 131072 56 and 642). A prompt's tiles are 128 rows whose
// partial outputs outweigh a few hundred positions: it is split below 256 tiles and from 6 units on, into
// at least 2 units each (4 items of 200 rows over up to 2088 positions 26 us, not split 55).
// Batches whose tiles fill the slots, or of more than kMaxScan items, are never split, however uneven: their
// time is the longest item's in one workgroup a head (8 heads of 4, 127 slots of 2048 positions and one of
// 131072: 867 us, where the bytes take 91).
KvPlan plan_of(int64_t heads, int64_t dim, int64_t tokens, int64_t q_heads, int64_t seqs, int64_t max_q,
               int64_t span) {
    const int64_t group = q_heads / heads, rows = max_q * group;
    KvPlan p{};
    p.tile_rows = rows <= 16 ? 16 : rows <= kFewRows ? 32 : kPrefillRows;
    p.tiles = (int32_t)ceil_div(rows, p.tile_rows);
    p.tiles = p.tiles > 0 ? p.tiles : 1;
    const bool prefill = p.tile_rows == kPrefillRows;
    // workgroups that 256 compute units are taken to hold at once; 64 wide the registers would let them hold
    // three of prompts and six of few rows (bf16; f32 five of 16 rows)
    const int64_t slots = kUnits * (prefill ? (dim <= 128 ? 2 : 1)
                                 : dim * p.tile_rows <= 128 * 16 ? 4 : dim * p.tile_rows <= 256 * 16 ? 2 : 1);
    p.least = prefill ? 2 : 1;
    // tiles of all items, a head: numbered by item and tile, or without gaps where bounds that are too wide
    // would leave most of those numbers empty, or have more of them than a launch
    int64_t most = seqs * p.tiles;
    const int64_t by_rows = seqs + ceil_div(tokens * group, p.tile_rows);
    p.scan = by_rows < most && (most >= kMaxGrid / heads || (seqs <= kMaxScan && by_rows < most / 2));
    if (p.scan || seqs <= kMaxScan) most = most < by_rows ? most : by_rows;
    if (seqs <= kMaxScan) {
        const int64_t all = most * heads;
        if (prefill ? all < kUnits && span > 6 * kUnit
                    : all < slots && span > (10 + all / 24) * (dim <= 128 ? kUnit : kUnit / 2)) {
            // few rows: as many tasks as run at once; two to a compute unit where one would do for the tiles
            const int64_t now = !prefill && all <= kUnits && slots > 2 * kUnits ? 2 * kUnits : slots;
            const int64_t target = (prefill ? 512 : now) / heads, fit = now / heads;
            p.target = (int32_t)(target < 1 ? 1 : target < kMaxSplits ? target : kMaxSplits);
            p.scan = 1;
            p.fit = (int32_t)(fit < 1 ? 1 : fit);
        }
    }
    int64_t tasks = p.scan ? most : seqs * p.tiles;
    if (p.target > 0) {
        // no tile has more chunks than its units allow
        const int64_t chunks = ceil_div(ceil_div(span, kUnit), p.least);
        tasks = most + p.target < most * chunks ? most + p.target : most * chunks;
        p.by_item = seqs * max_q <= 2 * tokens;
    }
    p.tasks = tasks < kMaxGrid / heads ? (int32_t)tasks : -1;
    p.alone = !prefill && dim <= 128 && tasks * heads <= kUnits && span > 4 * kUnit;
    return p;
}

size_t space_of(const KvPlan& p, int64_t heads, int64_t dim, int64_t seqs) {
    if (p.target == 0) return 0;
    return (size_t)((seqs + 1) / 2 * 2) * 8 +
           (size_t)p.tasks * (size_t)heads * (size_t)p.tile_rows * (size_t)(8 + 4 * dim);
}

template <int D, bool BF16, int RT>
void launch_decode(const KvAttention& a, const KvPlan& p, dim3 grid, hipStream_t stream) {
    if constexpr (D <= 128) {
        if (p.alone) {
            hipLaunchKernelGGL((k_kv_decode<D, BF16, RT, true>), grid, dim3(64 * Shape<D, true>::kWaves), 0,
                               stream, a, p);
            return;
        }
    }
    hipLaunchKernelGGL((k_kv_decode<D, BF16, RT, false>), grid, dim3(64 * Shape<D, false>::kWaves), 0,
                       stream, a, p);
}

template <int D, bool BF16>
hipError_t launch(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.kv.heads * p.tasks));
    if (p.tile_rows == 16)
        launch_decode<D, BF16, 1>(a, p, grid, stream);
    else if (p.tile_rows == 32)
        launch_decode<D, BF16, 2>(a, p, grid, stream);
    else
        launch_kv_prefill(a, p, stream);
    if (p.target > 0) {
        const int64_t rows = (p.by_item ? (int64_t)a.b.seqs * a.max_q : a.b.tokens) * a.q_heads;
        if (rows < kWideJoin)
            hipLaunchKernelGGL((k_kv_join<D, BF16, true>), dim3((uint32_t)rows), dim3(kThreads), 0, stream,
                               a, p);
        else
            hipLaunchKernelGGL((k_kv_join<D, BF16, false>), dim3((uint32_t)ceil_div(rows, kWaves)),
                               dim3(kThreads), 0, stream, a, p);
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dim(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    if (a.kv.dim == 64) return launch<64, BF16>(a, p, stream);
    if (a.kv.dim == 128) return launch<128, BF16>(a, p, stream);
    return launch<256, BF16>(a, p, stream);
}

}  // namespace

bool kv_attention_fits(int64_t heads, int64_t dim, int64_t tokens, int64_t q_heads, int64_t seqs,
                       int64_t max_q, int64_t max_kv) {
    return plan_of(heads, dim, tokens, q_heads, seqs, max_q, max_kv).tasks >= 0;
}

size_t kv_attention_workspace_bytes(int64_t heads, int64_t dim, int64_t tokens, int64_t q_heads,
                                    int64_t seqs, int64_t max_q, int64_t max_kv) {
    return space_of(plan_of(heads, dim, tokens, q_heads, seqs, max_q, max_kv), heads, dim, seqs);
}

hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream) {
    // a window bounds what a tile sees; the workspace is sized without it and so never too small
    int64_t span = a.max_kv;
    if (a.window > 0 && (int64_t)a.window + a.max_q + 31 < span) span = (int64_t)a.window + a.max_q + 31;
    KvPlan p = plan_of(a.kv.heads, a.kv.dim, a.b.tokens, a.q_heads, a.b.seqs, a.max_q, span);
    gpr_divisor(a.kv.page / 16, p.page_magic, p.page_shift);
    return a.bf16 ? launch_dim<true>(a, p, stream) : launch_dim<false>(a, p, stream);
}

}  // namespace nvfp4
