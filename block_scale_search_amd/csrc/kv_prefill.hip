// Attention over the paged NVFP4 cache for gfx950, many query rows per (item, key/value head): prompts
// and chunks of prompts.
//
// A workgroup owns 128 rows, a wave 32 of them, and all walk the positions in tiles of 64. What costs
// here is vector arithmetic (the exponentials and the conversion of the codes), so the codes of a
// tile are converted once for all four waves: a wave loads one page unit of 16 tokens (contiguous
// lanes, the next tile's loads in flight while the current one is used), converts it to f16 and
// writes K as [token][d] and V as [d][token] to LDS, double-buffered, one barrier a tile. The products
// are S^T = K Q^T and O^T = V^T P^T on f16 MFMA 32x32x16: lane (n, h) = (lane % 32, lane / 32) gets
// the logits of row n at positions 8 i + 4 h .. + 3, and those registers are P^T's operand as they
// are, once V's positions are stored in that order (V's row holds, for each 16 positions, the blocks
// of four 0, 2 for h = 0 and 1, 3 for h = 1).
// Both LDS tiles permute the 16-byte pieces of a row so that 16 lanes that read a piece, and 8 that write
// pieces of K, use all banks (4 heads of 4, 256 wide, two prompts of 4096 rows over 8192 positions: 1027 us,
// with a permutation that only the reads need 1088).
//
// Rates (one MI355X): two prompts of 8192 rows, 8 heads of 4, 128 wide, bf16: 1.10 to 1.17 ms with the
// clock, 940 to 1000 TFLOP/s of the pairs that causal rows see. Two prompts of 4096 rows over 8192 positions, 4
// heads of 4: 128 wide 455 us, the matrix units busy 46% of the cycles, vector arithmetic 61%, one or the
// other 82%; 64 wide, where the exponentials weigh twice as much against the products, 309 us (33%, 73%,
// 85%); 256 wide 1011 us (34%, 45%, 67%): a wave has a SIMD for itself (registers and LDS), so its waits are
// not covered; making a tile's logits while the previous tile's become weights gave nothing there (1059 us
// against 1027) nor 128 wide. f32 has two products an operand: 64, 128 and 256 wide 452, 751 and 1742 us (the
// last spills 36 registers).
#include <hip/hip_runtime.h>

#include "internal.h"
#include "kv_attention_device.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 64;            // positions of a tile: one 16-token unit a wave

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(half8v a, half8v b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <int D>
struct Lds {
    static constexpr int kK = kTile * D * 2;             // bytes of K; V has as many
    static constexpr int kBuffer = 2 * kK;
    // K: piece c (8 values) of token t
    static __device__ __forceinline__ int k(int t, int c) {
        constexpr int P = D / 8;
        const int f = D == 64 ? ((t >> 1) & 7) ^ (t & 1) : t & 15;
        return (t * P + (c ^ f ^ (c >> 3 << 1))) * 16;
    }
    // V: piece c (8 positions) of row r
    static __device__ __forceinline__ int v(int r, int c) {
        return kK + (r * (kTile / 8) + (c ^ ((r >> 1) & 7))) * 16;
    }
};

// Lane offsets of a unit's codes and scales in a record, without its first row: token lane / 4 and a
// quarter of its values for K; for V, values of column lane % 16 of 4 tokens, block value_block(lane): the
// blocks 0 and 2, whose 8 bytes lie side by side in LDS, in the lower half of the wave.
__device__ __forceinline__ int value_block(int lane) { return (lane >> 5) | ((lane >> 3) & 2); }

struct UnitOffsets {
    uint32_t k, v, ks, vs;
};

template <int D>
__device__ __forceinline__ UnitOffsets unit_offsets(const KvView& kv, int head, int lane) {
    const uint32_t region = (uint32_t)kv_code_bytes(kv);
    const uint32_t codes = (uint32_t)head * kv.page * (D / 2), scales = (uint32_t)head * kv.page * (D / 16);
    UnitOffsets o;
    o.k = codes + lane * (D / 8);
    const int block = value_block(lane), n = lane & 15;
    o.v = codes + region + (block * 16 + n) * (D / 8);
    o.ks = 2 * region + scales + lane * (D / 64);
    o.vs = 2 * region + (region >> 3) + scales + (block * (D / 16) + n * D / 256) * 4;
    return o;
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
        const u32x2 t = *reinterpret_cast<const u32x2*>(p);
        w[0] = t[0]; w[1] = t[1];
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const u32x4 t = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * i + k] = t[k];
        }
    }
}

// rec: record, row: the unit's first row (both uniform).
template <int D>
__device__ __forceinline__ void load_unit(HalfTile<D>& u, const uint8_t* rec, int row,
                                          const UnitOffsets& o) {
    const uint8_t* codes = rec + (int64_t)row * (D / 2);
    const uint8_t* scales = rec + (int64_t)row * (D / 16);
    load_words<D / 32>(codes + o.k, u.k);
    load_words<D / 32>(codes + o.v, u.v);
    if constexpr (D == 64) u.ks = scales[o.ks];
    else if constexpr (D == 128) u.ks = *reinterpret_cast<const uint16_t*>(scales + o.ks);
    else u.ks = *reinterpret_cast<const uint32_t*>(scales + o.ks);
    u.vs = *reinterpret_cast<const uint32_t*>(scales + o.vs);
}

// Conversion of a wave's unit (number `wave` of the tile) into a buffer, in kPieces pieces that the
// caller spreads between matrix instructions: D/32 pieces of K (8 values of a token), then D/16 of V (4
// tokens of a value).
template <int D>
struct UnitStore {
    static constexpr int kPieces = D / 32 + D / 16;
    uint8_t* buf;
    const HalfTile<D>& u;
    VPairs<D> v;
    uint32_t scales;
    int t, first, n, c, high;

    __device__ __forceinline__ UnitStore(uint8_t* to, const HalfTile<D>& unit, int wave, int lane)
        : buf(to), u(unit) {
        scales = unit.ks & 0x7F7F7F7Fu;
        pair_tokens<D>(v, unit.v, unit.vs);
        t = 16 * wave + (lane >> 2);
        first = (lane & 3) * (D / 32);
        n = lane & 15;
        c = 2 * wave + (value_block(lane) & 1);
        high = (value_block(lane) >> 1) * 8;
    }
    template <int I>
    __device__ __forceinline__ void piece() {
        if constexpr (I < D / 32) {
            *reinterpret_cast<half8v*>(buf + Lds<D>::k(t, first + I)) = k_operand<I>(u.k, scales);
        } else {
            constexpr int J = I - D / 32, w = 2 * (J / 8) + (J & 1), b = (J & 7) >> 1;
            const half2v x = dequant2<b>(v.w[0][w], v.e[0]), y = dequant2<b>(v.w[1][w], v.e[1]);
            *reinterpret_cast<u32x2*>(buf + Lds<D>::v(J * 16 + n, c) + high) =
                u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
        }
    }
    __device__ __forceinline__ void all() {
        unroll<kPieces>([&](auto i) { piece<decltype(i)::value>(); });
    }
};

// Values 16 s + 8 h .. + 7 of a row as f16 operands, and the logit (log2) of a product.
template <int D, bool BF16>
struct Query {
    half8v hi[D / 16];
    half8v lo[BF16 ? 1 : D / 16];
    float f;
};

template <int D, bool BF16>
__device__ __forceinline__ void load_query(Query<D, BF16>& q, const uint8_t* p, bool live, int h,
                                           float scale, float S) {
    constexpr int N = D / 16;
    float x[N][8];
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if constexpr (BF16) {
            u32x4 t = {0u, 0u, 0u, 0u};
            if (live) t = *reinterpret_cast<const u32x4*>(p + (16 * s + 8 * h) * 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[s][2 * k] = bf16_lo(t[k]);
                x[s][2 * k + 1] = bf16_hi(t[k]);
            }
        } else {
            f32x4 t[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            if (live) {
                t[0] = reinterpret_cast<const f32x4*>(p + (16 * s + 8 * h) * 4)[0];
                t[1] = reinterpret_cast<const f32x4*>(p + (16 * s + 8 * h) * 4)[1];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) x[s][k] = t[k >> 2][k & 3];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[s][k]));
    }
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int e = row_exponent(top);
    const float up = row_factor(e, top, S);
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float v = x[s][k] * up;
            const _Float16 r = (_Float16)v;
            q.hi[s][k] = r;
            if constexpr (!BF16) q.lo[s][k] = (_Float16)(v - (float)r);
        }
    q.f = fmaxf(__builtin_ldexpf(scale, -e) * (S * kLog2e), 0x1p-126f);
}

template <int D>
constexpr int kOccupancy = D <= 128 ? 2 : 1;

// A wave rescales its outputs at the tiles where one of its 32 rows passes the slack, each row at a tile of its
// own: 12.5 of 64 tiles for normal logits. Where every row's maximum follows the largest logit it has seen, at
// the wave's tiles 4, 16, 64, ..., they are 7.7 (8 items of up to 1000 rows over up to 8000 positions, 4 heads of
// 4, 256 wide: 252.3 us, without 259.6; two prompts of 8192 rows, 8 heads of 4, 128 wide: 1126 and 1129). 64 wide
// rescaling is cheap, and the register that this takes is the 169th: two workgroups fit a compute unit instead
// of three (two prompts of up to 4096 rows over up to 8192, 4 heads of 4: 198 us, without 180).
template <int D>
constexpr bool kFollow = D >= 128;
__device__ __forceinline__ bool follow_tile(int i) { return (i & (i - 1)) == 0 && (i & 0x55555554) != 0; }

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads, kOccupancy<D>) void k_kv_prefill(KvAttention a, KvPlan plan) {
    constexpr int NS = D / 16, NJ = D / 32;
    __shared__ __align__(16) uint8_t space[2 * Lds<D>::kBuffer];
    const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvView& kv = a.kv;
    const int task = (int)(blockIdx.x / (uint32_t)kv.heads);
    const int head = (int)(blockIdx.x - (uint32_t)task * (uint32_t)kv.heads);
    const int group = a.q_heads / kv.heads;
    KvTask job;
    if (!find_task(a, plan, task, job)) return;
    const bool whole = job.chunks <= 1;
    if (plan.target > 0 && head == 0 && job.chunk == 0 && job.tile == 0 && threadIdx.x == 0)
        item_info(a)[job.item] = make_int2(job.base, job.chunks);
    const int begin = job.begin, end = job.end;
    const int tiles = (end - begin + kTile - 1) / kTile;

    // pages of the next 64 tiles, lane i the i-th: the tile's four units
    const int32_t* table = kv.table + (int64_t)job.work.slot * kv.max_pages;
    const int32_t units = kv.page >> 4;
    int32_t page[kWaves], row = 0;
    const auto look_up = [&](int i) {
        const int64_t t = begin + (int64_t)(i + lane) * kTile;
        const bool in = t < end;
#pragma unroll
        for (int u = 0; u < kWaves; ++u) {
            const int unit = in ? (int)(t >> 4) + u : 0;
            const int col = (int)div_gpr((uint32_t)unit, plan.page_magic, plan.page_shift);
            page[u] = in && col < kv.max_pages ? table[col] : -1;
            row = u == wave ? (unit - col * units) << 4 : row;
        }
    };
    const UnitOffsets from = unit_offsets<D>(kv, head, lane);
    HalfTile<D> raw;
    uint32_t named = 0;                                  // four bits a tile, the latest lowest
    const auto load = [&](int i) {
        if ((i & 63) == 0) look_up(i);
        int mine = 0;
#pragma unroll
        for (int u = 0; u < kWaves; ++u) {
            const int pg = __builtin_amdgcn_readlane(page[u], i & 63);
            const bool ok = (uint32_t)pg < (uint32_t)kv.num_pages;
            named = named << 1 | (ok ? 1u : 0u);
            mine = u == wave && ok ? pg : mine;
        }
        load_unit<D>(raw, kv.pages + (int64_t)mine * kv.page_stride,
                     __builtin_amdgcn_readlane(row, i & 63), from);
    };
    if (tiles > 0) load(0);

    // the wave's rows
    const int row_first = 32 * wave;
    const int rows = min(32, job.rows - row_first);      // may be none
    const int at_row = job.row0 + row_first;
    const bool live = n < rows;
    const RowAt of = row_at(job.work.first, head, group, live ? at_row + n : job.row0);
    Query<D, BF16> q;
    load_query<D, BF16>(q, static_cast<const uint8_t*>(a.q.p) + of.token * a.q.stride_t + of.head * a.q.stride_h,
                        live, h, a.scale, kv.S_k[head]);
    const int pos = job.work.len - job.work.all_new + (int)(of.token - job.work.first);
    const int low = a.window > 0 ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
    const int lim = a.causal ? min(end, pos + 1) : end;
    // every row of the wave sees low_all .. lim_all - 1, none anything outside low_any .. lim_any - 1
    int low_all = 0, lim_all = end, low_any = 0, lim_any = rows > 0 ? end : begin;
    if (rows > 0) {
        const int p0 = job.work.len - job.work.all_new + at_row / group;
        const int p1 = job.work.len - job.work.all_new + (at_row + rows - 1) / group;
        if (a.causal) {
            lim_all = min(end, p0 + 1);
            lim_any = min(end, p1 + 1);
        }
        if (a.window > 0) {
            low_all = (int)max((int64_t)p1 - a.window + 1, (int64_t)0);
            low_any = (int)max((int64_t)p0 - a.window + 1, (int64_t)0);
        }
    }

    f32x16 o[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
    float m = -__builtin_inff(), sub = 0.0f, l = 0.0f, seen = m;

    if (tiles > 0) UnitStore<D>(space, raw, wave, lane).all();
    uint32_t ok = named & 15u;
    if (tiles > 1) load(1);
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const uint8_t* buf = space + (i & 1) * Lds<D>::kBuffer;
        uint8_t* other = space + (~i & 1) * Lds<D>::kBuffer;   // of tile i + 1; after the last one unused
        const uint32_t next = named & 15u;
        const int t = begin + i * kTile;
        if (t < lim_any && t + kTile > low_any) {        // the wave sees something of the tile
            // the first products of this tile, and in their shadow the conversion of the next: three
            // pieces to four steps. The operands are read kAhead steps ahead of their use.
            constexpr int kSteps = 2 * NS, kAhead = kSteps < 4 ? kSteps : 4;
            UnitStore<D> store(other, raw, wave, lane);
            half8v k[kSteps];
            const auto read_k = [&](int z) {
                k[z] = *reinterpret_cast<const half8v*>(buf + Lds<D>::k(32 * (z & 1) + n, 2 * (z >> 1) + h));
            };
            f32x16 s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
            for (int z = 0; z < kAhead; ++z) read_k(z);
            unroll<kSteps>([&](auto step) {
                constexpr int Z = decltype(step)::value;
                s[Z & 1] = mfma(k[Z], q.hi[Z >> 1], s[Z & 1]);
                if constexpr (!BF16) s[Z & 1] = mfma(k[Z], q.lo[Z >> 1], s[Z & 1]);
                if constexpr (Z + kAhead < kSteps) read_k(Z + kAhead);
                if constexpr (Z % 4 != 3) store.template piece<Z / 4 * 3 + Z % 4>();
                __builtin_amdgcn_sched_barrier(0);
            });
            if (!(ok == 15u && t >= low_all && t + kTile <= lim_all)) {
                asm volatile("");                        // a branch, not selects in every tile
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int p = 32 * u + 8 * (k >> 2) + 4 * h + (k & 3);   // in the tile
                        const bool here = (ok >> (3 - (2 * u + (k >> 3)))) & 1u;
                        if (!(here && t + p >= low && t + p < lim)) s[u][k] = -__builtin_inff();
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int k = 1; k < 32; ++k) top = fmaxf(top, s[k >> 4][k & 15]);
            top *= q.f;
            if constexpr (kFollow<D>) top = seen = fmaxf(seen, top);
            const float slack = kFollow<D> && follow_tile(i) ? 0.0f : kSlack;
            if (__any(top > m + slack)) {
                const float al = raise_row(m, sub, fmaxf(top, __shfl_xor(top, 32, 64)), slack);
                l *= al;
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[j] *= al;
            }
            if (i + 2 < tiles) load(i + 2);
            Half8 hi[4], lo[4];
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = __builtin_amdgcn_exp2f(
                        __builtin_fmaf(s[u >> 1][8 * (u & 1) + 2 * k], q.f, sub));
                    const float y = __builtin_amdgcn_exp2f(
                        __builtin_fmaf(s[u >> 1][8 * (u & 1) + 2 * k + 1], q.f, sub));
                    sum += x + y;
                    hi[u].p[k] = half2v{(_Float16)x, (_Float16)y};
                    if constexpr (!BF16)
                        lo[u].p[k] = half2v{(_Float16)(x - (float)hi[u].p[k][0]),
                                            (_Float16)(y - (float)hi[u].p[k][1])};
                }
            }
            l += sum;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const half8v v = *reinterpret_cast<const half8v*>(
                        buf + Lds<D>::v(32 * j + n, 2 * u + h));
                    o[j] = mfma(v, hi[u].v, o[j]);
                    if constexpr (!BF16) o[j] = mfma(v, lo[u].v, o[j]);
                }
            // order of the block above: four LDS reads ahead, then one with each step's products
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int z = 0; z < 4 * NJ; ++z) {
                __builtin_amdgcn_sched_group_barrier(0x8, BF16 ? 1 : 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        } else {
            UnitStore<D>(other, raw, wave, lane).all();
            if (i + 2 < tiles) load(i + 2);
        }
        ok = next;
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    // o[j][i]: V's row 32 j + 8 (i / 4) + 4 h + i % 4 = 16 e + c, the value d = c D/16 + e: for each of the
    // lane's eight c, D/16 values in a row
    const float z = whole ? (l == 0.0f ? 0.0f : kv.S_v[head] / l) : 1.0f;
    uint8_t* dst = static_cast<uint8_t*>(a.out) + of.token * a.out_stride_t + of.head * a.out_stride_h;
    float* part = whole ? nullptr : part_out(a, plan, task, head) + (row_first + n) * D;
    if (h == 0) {
        if (!whole)
            part_stat(a, plan, task, head)[row_first + n] = make_float2(m, l);
        else if (a.lse)
            a.lse[of.token * a.q_heads + of.head] = row_lse(m, l);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = 8 * k + 4 * h + r;
            float x[D / 16];
#pragma unroll
            for (int e = 0; e < D / 16; ++e) x[e] = o[e / 2][8 * (e & 1) + 4 * k + r] * z;
#pragma unroll
            for (int e = 0; e < D / 16; e += 4) {
                const int d = c * (D / 16) + e;
                if (!whole)
                    *reinterpret_cast<f32x4*>(part + d) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
                else if constexpr (BF16)
                    *reinterpret_cast<u32x2*>(dst + 2 * d) =
                        u32x2{bf16_pair(x[e], x[e + 1]), bf16_pair(x[e + 2], x[e + 3])};
                else
                    *reinterpret_cast<f32x4*>(dst + 4 * d) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
            }
        }
}

template <int D>
void launch(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.kv.heads * p.tasks));
    if (a.bf16)
        hipLaunchKernelGGL((k_kv_prefill<D, true>), grid, dim3(kThreads), 0, stream, a, p);
    else
        hipLaunchKernelGGL((k_kv_prefill<D, false>), grid, dim3(kThreads), 0, stream, a, p);
}

}  // namespace

void launch_kv_prefill(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    if (a.kv.dim == 64) launch<64>(a, p, stream);
    else if (a.kv.dim == 128) launch<128>(a, p, stream);
    else launch<256>(a, p, stream);
}

}  // namespace nvfp4
