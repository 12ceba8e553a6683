// Attention over the paged NVFP4 key/value cache for gfx950.
//
// Few rows per (item, key/value head) - decode steps and drafts: k_kv_decode. A wave owns tiles of 32
// positions and 16 RT query rows, with everything in registers. S^T = K Q^T puts a query row in a
// lane column: the f16 MFMA 16x16x32 gives lane (n, g) = (lane % 16, lane / 16) the logits of row n
// at positions 4g .. 4g + 3 of each half tile. O^T = V^T P^T needs, in that same lane, the weights of row n
// at 8 positions: any 8, as long as V's operand uses the same ones, so the logits' registers are the
// weights' registers and no lane exchanges anything. V's operand then holds, for lane (n, g), the
// positions 4g .. 4g + 3 of both half tiles and the values d = n D/16 + j of tile j: the record
// layout keeps exactly those codes together, 4 tokens x D/16 values in one load.
// A row's running maximum is only raised when a logit exceeds it by more than 2^7 (weights are
// scaled by 2^8 and stay below 2^15), so most tiles need no cross-lane step and no rescaling.
// The waves of a workgroup take tiles in turn and are joined in LDS; the chunks of a long
// sequence are joined by k_kv_join.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "internal.h"
#include "kv_attention_device.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kUp = 8.0f;          // log2 of the weights' scale
constexpr float kSlack = 7.0f;       // how far a logit may exceed the maximum in use, log2

// A lane's bytes of one 16-token half tile. K: D/4 values of its token and their scale bytes. V:
// D/16 values of 4 tokens, and those tokens' scale bytes.
template <int D>
struct HalfTile {
    static constexpr int W = D / 32;          // code words
    uint32_t k[W], v[W], ks, vs;
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        w[0] = t.x; w[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 t = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
        }
    }
}

// Offsets of a lane's bytes in a record, without the part that depends on the tile's first row.
struct LaneOffsets {
    uint32_t k, ks, v, vs;
};

template <int D>
__device__ __forceinline__ LaneOffsets lane_offsets(const KvView& kv, int head, int n, int g) {
    const uint32_t half = (uint32_t)kv_code_bytes(kv);
    const uint32_t row = (uint32_t)head * kv.page;
    LaneOffsets o;
    o.k = (row + n) * (D / 2) + g * (D / 8);
    o.ks = 2 * half + (row + n) * (D / 16) + g * (D / 64);
    o.v = half + (((row >> 2) + g) * 16 + n) * (D / 8);
    o.vs = 2 * half + (half >> 3) + (((row >> 2) + g) * (D / 16) + n * D / 256) * 4;
    return o;
}

// rec: the page's record; row: the half tile's first row in it (both uniform).
template <int D>
__device__ __forceinline__ void load_half(HalfTile<D>& t, const uint8_t* rec, int row,
                                          const LaneOffsets& o) {
    load_words<D / 32>(rec + o.k + row * (D / 2), t.k);
    const uint8_t* s = rec + o.ks + row * (D / 16);
    if constexpr (D == 64) t.ks = *s;
    else if constexpr (D == 128) t.ks = *reinterpret_cast<const uint16_t*>(s);
    else t.ks = *reinterpret_cast<const uint32_t*>(s);
    load_words<D / 32>(rec + o.v + row * (D / 2), t.v);
    t.vs = *reinterpret_cast<const uint32_t*>(rec + o.vs + row * (D / 16));
}

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

template <int N, typename F, int I = 0>
__device__ __forceinline__ void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, F, I + 1>(static_cast<F&&>(f));
    }
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

template <int D, bool BF16>
__device__ __forceinline__ void load_query(QRow<D, BF16>& q, const uint8_t* p, int g, float scale,
                                           float S) {
    float x[D / 4];
#pragma unroll
    for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
    if (p) {
        if constexpr (BF16) {
            const uint4* s = reinterpret_cast<const uint4*>(p + g * (D / 2));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 t = s[i];
                const uint32_t d[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[8 * i + 2 * k] = bf16_lo(d[k]);
                    x[8 * i + 2 * k + 1] = bf16_hi(d[k]);
                }
            }
        } else {
            const float4* s = reinterpret_cast<const float4*>(p + g * D);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float4 t = s[i];
                x[4 * i] = t.x; x[4 * i + 1] = t.y; x[4 * i + 2] = t.z; x[4 * i + 3] = t.w;
            }
        }
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
    const int k = row_exponent(max_groups(top));
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = __builtin_ldexpf(x[8 * s + j], k);
            const _Float16 h = (_Float16)v;
            q.hi[s][j] = h;
            if constexpr (!BF16) q.lo[s][j] = (_Float16)(v - (float)h);
        }
    }
    // at least the smallest normal number: a masked logit of -infinity times it stays -infinity
    q.f = fmaxf(__builtin_ldexpf(scale, -k) * (S * kLog2e), 0x1p-126f);
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

// Workspace of split sequences: O (binary32, scaled like the weights) of every row and chunk, then
// (maximum, sum) of every row and chunk.
__device__ __forceinline__ float* part_out(const KvAttention& a, int splits, int64_t row, int s, int D) {
    return static_cast<float*>(a.workspace) + (row * splits + s) * D;
}
__device__ __forceinline__ float2* part_stat(const KvAttention& a, int splits, int64_t row, int s,
                                             int D) {
    float* end = static_cast<float*>(a.workspace) + a.b.tokens * a.q_heads * (int64_t)splits * D;
    return reinterpret_cast<float2*>(end) + row * splits + s;
}

// lse of a row from its maximum (log2, the weights' scale of 2^kUp apart) and sum.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l > 0.0f ? (m - kUp + __builtin_amdgcn_logf(l)) * kLn2 : -__builtin_inff();
}

template <int D, bool BF16, int RT>
__global__ __launch_bounds__(kThreads) void k_kv_decode(KvAttention a, KvPlan plan) {
    constexpr int R = 16 * RT, NJ = D / 16, NS = D / 32;
    constexpr int JC = NJ < 8 ? NJ : 8;                  // output tiles joined at a time
    __shared__ float joined[kWaves][16][JC * 16 + 4];
    __shared__ float2 stat[kWaves][R];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvView& kv = a.kv;

    // work of this workgroup: head fastest, then item, row tile, chunk
    uint32_t w = blockIdx.x;
    const int head = w % (uint32_t)kv.heads;
    w /= (uint32_t)kv.heads;
    const int item = w % (uint32_t)a.b.seqs;
    w /= (uint32_t)a.b.seqs;
    const int tile = w % (uint32_t)plan.tiles, split = w / (uint32_t)plan.tiles;
    const int group = a.q_heads / kv.heads;
    const int64_t total = min((int64_t)a.b.cu[a.b.seqs], a.b.tokens);
    const int64_t first = a.b.cu[item];
    const int n_new = (int)min((int64_t)a.b.cu[item + 1], total) - (int)first;
    const int all_new = a.b.cu[item + 1] - (int)first;
    const int row0 = tile * R;
    const int rows = min(R, min(n_new, a.max_q) * group - row0);
    if (first < 0 || rows <= 0) return;
    const KvItem it = kv_item(kv, a.b, item);
    const KvRange range = tile_range(a, it.len, all_new, group, row0, rows);
    const int chunks = (range.end - range.begin + plan.chunk - 1) / plan.chunk;
    if (split > 0 && split >= chunks) return;
    const int begin = range.begin + split * plan.chunk;
    const int end = min(range.end, begin + plan.chunk);

    QRow<D, BF16> q[RT];
    int low[RT], lim[RT];                                // the lane's row sees low .. lim - 1
    int low_all = 0, lim_all = end;                      // and so does every row
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + 16 * rt + n;
        const bool live = 16 * rt + n < rows;
        const RowAt at = row_at(first, head, group, live ? row : row0);
        const uint8_t* p = static_cast<const uint8_t*>(a.q.p) + at.token * a.q.stride_t +
                           at.head * a.q.stride_h;
        load_query<D, BF16>(q[rt], live ? p : nullptr, g, a.scale, kv.S_k[head]);
        const int pos = it.len - all_new + (int)(at.token - first);
        low[rt] = a.window > 0 ? pos - a.window + 1 : 0;
        lim[rt] = a.causal ? min(end, pos + 1) : end;
    }
    {
        const int p0 = it.len - all_new + row0 / group;
        const int p1 = it.len - all_new + (row0 + rows - 1) / group;
        if (a.causal) lim_all = min(end, p0 + 1);
        if (a.window > 0) low_all = p1 - a.window + 1;
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

    const LaneOffsets off = lane_offsets<D>(kv, head, n, g);
    const int32_t* table = kv.table + (int64_t)it.slot * kv.max_pages;
    const uint32_t units = (uint32_t)kv.page >> 4;
    // page (clamped to a valid one) and first row of 16-token unit u; ok: the table names a page
    const auto locate = [&](int u, bool& ok, int& row) {
        const uint32_t col = div_gpr((uint32_t)u, plan.page_magic, plan.page_shift);
        row = ((uint32_t)u - col * units) << 4;
        const int page = (int)col < kv.max_pages ? table[col] : -1;
        ok = (uint32_t)page < (uint32_t)kv.num_pages;
        return kv.pages + (int64_t)(ok ? page : 0) * kv.page_stride;
    };
    constexpr int kStep = 32 * kWaves;
    HalfTile<D> now[2], next[2];
    bool ok[2], ok_next[2];
    const auto fetch = [&](int t, HalfTile<D> (&h)[2], bool (&good)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            int row;
            const uint8_t* rec = locate((t >> 4) + u, good[u], row);
            load_half<D>(h[u], rec, row, off);
        }
    };
    int t = begin + 32 * wave;
    if (t < end) fetch(t, now, ok);
    for (; t < end; t += kStep) {
        const bool more = t + kStep < end;
        if (more) fetch(t + kStep, next, ok_next);

        f32x4 s[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t scales = now[u].ks & 0x7F7F7F7Fu;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            unroll<NS>([&](auto step) {
                constexpr int S = decltype(step)::value;
                const half8v k = k_operand<S>(now[u].k, scales);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s[rt][u] = mfma(k, q[rt].hi[S], s[rt][u]);
                    if constexpr (!BF16) s[rt][u] = mfma(k, q[rt].lo[S], s[rt][u]);
                }
            });
        }
        if (!(ok[0] && ok[1] && t >= low_all && t + 32 <= lim_all)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = t + 16 * u + 4 * g + i;
                        if (!(ok[u] && p >= low[rt] && p < lim[rt])) s[rt][u][i] = -__builtin_inff();
                    }
        }
        Half8 hi[RT], lo[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float top = fmaxf(fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3])),
                              fmaxf(fmaxf(s[rt][1][0], s[rt][1][1]), fmaxf(s[rt][1][2], s[rt][1][3])));
            top *= q[rt].f;
            if (__any(top > m[rt] + kSlack)) {
                const float mn = fmaxf(m[rt], max_groups(top));
                const bool none = mn == -__builtin_inff();
                const float al = none ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
                m[rt] = mn;
                sub[rt] = none ? 0.0f : kUp - mn;
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
        VPairs<D> vp[2];
        pair_tokens<D>(vp[0], now[0].v, now[0].vs);
        pair_tokens<D>(vp[1], now[1].v, now[1].vs);
        unroll<NJ>([&](auto tile_j) {
            constexpr int J = decltype(tile_j)::value;
            const half8v v = v_operand<D, J>(vp);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                o[rt][J] = mfma(v, hi[rt].v, o[rt][J]);
                if constexpr (!BF16) o[rt][J] = mfma(v, lo[rt].v, o[rt][J]);
            }
        });
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            now[u] = next[u];
            ok[u] = ok_next[u];
        }
    }

    // join the waves: the rows' maxima and sums, then the outputs scaled to the joint maximum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = sum_groups(l[rt]);
        if (g == 0) stat[wave][16 * rt + n] = make_float2(m[rt], l[rt]);
    }
    __syncthreads();
    const float S_v = kv.S_v[head];
    const bool whole = chunks <= 1;
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
                    if (sk.x != -__builtin_inff()) rl += sk.y * __builtin_amdgcn_exp2f(sk.x - rm);
                    const float4 x = *reinterpret_cast<const float4*>(&joined[k][r][c]);
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                }
                const int d = (c / JC) * NJ + jc * JC + c % JC;
                const RowAt at = row_at(first, head, group, row0 + 16 * rt + r);
                const int64_t row = at.token * a.q_heads + at.head;
                if (whole) {
                    const float z = rl > 0.0f ? S_v / rl : 0.0f;
                    uint8_t* dst = static_cast<uint8_t*>(a.out) + at.token * a.out_stride_t +
                                   at.head * a.out_stride_h;
                    if constexpr (BF16)
                        *reinterpret_cast<uint2*>(dst + 2 * d) =
                            make_uint2(bf16_pair(v.x * z, v.y * z), bf16_pair(v.z * z, v.w * z));
                    else
                        *reinterpret_cast<float4*>(dst + 4 * d) =
                            make_float4(v.x * z, v.y * z, v.z * z, v.w * z);
                    if (a.lse && d == 0) a.lse[row] = row_lse(rm, rl);
                } else {
                    *reinterpret_cast<float4*>(part_out(a, plan.splits, row, split, D) + d) = v;
                    if (d == 0) *part_stat(a, plan.splits, row, split, D) = make_float2(rm, rl);
                }
            }
        }
    }
}

// Joins the chunks of a row: one workgroup per (token row, query head), its waves over the chunks.
template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void k_kv_join(KvAttention a, KvPlan plan) {
    constexpr int E = D / 64;
    __shared__ float acc[kWaves][D];
    const KvView& kv = a.kv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const int64_t token = row / a.q_heads;
    const int hq = (int)(row - token * a.q_heads);
    const int group = a.q_heads / kv.heads, head = hq / group;
    const int64_t total = min((int64_t)a.b.cu[a.b.seqs], a.b.tokens);
    if (token >= total) return;
    const int item = kv_find_item(a.b.cu, a.b.seqs, token);
    const int64_t first = a.b.cu[item];
    const int64_t j = token - first;
    if (j < 0 || j >= a.max_q) return;
    const int all_new = a.b.cu[item + 1] - (int)first;
    const int n_new = (int)min((int64_t)a.b.cu[item + 1], total) - (int)first;
    const KvItem it = kv_item(kv, a.b, item);
    const int r = (int)j * group + hq - head * group;
    const int row0 = r / plan.tile_rows * plan.tile_rows;
    const int rows = min(plan.tile_rows, min(n_new, a.max_q) * group - row0);
    const KvRange range = tile_range(a, it.len, all_new, group, row0, rows);
    const int chunks = (range.end - range.begin + plan.chunk - 1) / plan.chunk;
    if (chunks <= 1) return;                              // already written
    float mm = -__builtin_inff();
    for (int s = lane; s < chunks; s += 64) mm = fmaxf(mm, part_stat(a, plan.splits, row, s, D)->x);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o, 64));
    float l = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
    for (int s = wave; s < chunks; s += kWaves) {
        const float2 st = *part_stat(a, plan.splits, row, s, D);
        const float f = st.x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(st.x - mm);
        const float* p = part_out(a, plan.splits, row, s, D) + lane * E;
        l += st.y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __builtin_fmaf(p[e], f, v[e]);
    }
    __shared__ float sums[kWaves];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[wave][lane * E + e] = v[e];
    if (lane == 0) sums[wave] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) l += sums[k];
    const float z = l > 0.0f ? kv.S_v[head] / l : 0.0f;
    uint8_t* dst = static_cast<uint8_t*>(a.out) + token * a.out_stride_t + hq * a.out_stride_h;
    for (int d = threadIdx.x; d < D / 2; d += kThreads) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            x += acc[k][2 * d];
            y += acc[k][2 * d + 1];
        }
        if constexpr (BF16) reinterpret_cast<uint32_t*>(dst)[d] = bf16_pair(x * z, y * z);
        else reinterpret_cast<float2*>(dst)[d] = make_float2(x * z, y * z);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = row_lse(mm, l);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of 16 or 32 rows; chunks so that about 1024 workgroups (four on each compute unit) share
// the positions.
KvPlan plan_of(int64_t heads, int64_t q_heads, int64_t seqs, int64_t max_q, int64_t max_kv) {
    const int64_t rows = max_q * (q_heads / heads);
    KvPlan p{};
    p.tile_rows = rows <= 16 ? 16 : 32;
    p.tiles = (int32_t)ceil_div(rows, p.tile_rows);
    const int64_t base = seqs * heads * p.tiles;
    const int64_t want = ceil_div(1024, base > 0 ? base : 1);
    int64_t chunk = ceil_div(ceil_div(max_kv > 0 ? max_kv : 1, want), 32 * kWaves) * 32 * kWaves;
    p.chunk = (int32_t)(chunk < ((int64_t)1 << 30) ? chunk : (int64_t)1 << 30);
    p.splits = (int32_t)ceil_div(max_kv > 0 ? max_kv : 1, p.chunk);
    return p;
}

template <int D, bool BF16>
hipError_t launch(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.kv.heads * a.b.seqs * p.tiles * p.splits;
    if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 grid((uint32_t)blocks);
    if (p.tile_rows == 16)
        hipLaunchKernelGGL((k_kv_decode<D, BF16, 1>), grid, dim3(kThreads), 0, stream, a, p);
    else
        hipLaunchKernelGGL((k_kv_decode<D, BF16, 2>), grid, dim3(kThreads), 0, stream, a, p);
    if (p.splits > 1)
        hipLaunchKernelGGL((k_kv_join<D, BF16>), dim3((uint32_t)(a.b.tokens * a.q_heads)),
                           dim3(kThreads), 0, stream, a, p);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dim(const KvAttention& a, const KvPlan& p, hipStream_t stream) {
    if (a.kv.dim == 64) return launch<64, BF16>(a, p, stream);
    if (a.kv.dim == 128) return launch<128, BF16>(a, p, stream);
    return launch<256, BF16>(a, p, stream);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t heads, int64_t dim, bool bf16, int64_t tokens,
                                    int64_t q_heads, int64_t seqs, int64_t max_q, int64_t max_kv) {
    (void)bf16;
    const KvPlan p = plan_of(heads, q_heads, seqs, max_q, max_kv);
    if (p.splits <= 1) return 0;
    return (size_t)(tokens * q_heads * (int64_t)p.splits) * (dim * 4 + 8);
}

hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream) {
    KvPlan p = plan_of(a.kv.heads, a.q_heads, a.b.seqs, a.max_q, a.max_kv);
    gpr_divisor(a.kv.page / 16, p.page_magic, p.page_shift);
    return a.bf16 ? launch_dim<true>(a, p, stream) : launch_dim<false>(a, p, stream);
}

}  // namespace nvfp4
