// Products of many rows with NVFP4 matrices for gfx950, by tiles: forward, gated and backward.
//
// A workgroup owns a tile of rows and columns and walks the reduction in steps of 64. The rows' side
// goes from global memory straight into LDS; the codes of the next step are loaded into registers while
// the current one is multiplied, converted there (level * E4M3 is exact in bf16) and written to LDS as
// [column][64], the same in both directions: backward, a thread converts four rows of the matrix by eight columns
// and pairs the rows in the conversion to bf16, which is the transposition. The 16-byte pieces of an
// LDS row are permuted by the row so that the reads of MFMA operands and the writes use all banks.
// Gated: the columns of a tile are 32 of the gate, the same 32 of the other matrix, and so on, so that
// both values of an output are in the same lane.
//
// What bounds it. Tiles of 256 x 256: the matrix units, 67 to 69% busy forward and 56 to 59% backward at the clock that the
// power limit leaves (1.8 GHz); their LDS traffic (192 KB read, 64 KB written a step) takes as long as they do, and runs
// beside them. 8192 rows by 2 x 14336 x 4096 1560 us (1.23 PFLOP/s), of which the matrix instructions alone take 1217 to
// 1254, LDS, conversion and barriers 150, copies of the rows 130, loads of codes 150. Tiles of 128 x 128: latencies of
// short reductions (two workgroups a compute unit); gradients of 16384 rows of 128 experts 2 x 768 x 2048 255 us (0.4
// PFLOP/s), matrix units 30% busy, vector units 41%, neither 43%.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "internal.h"
#include "product_device.h"

namespace nvfp4 {
namespace {

constexpr int BK = 64;
enum Mode { kLinear = 0, kGated = 1, kBackward = 2 };

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;     // MFMA tiles of a wave
    static constexpr int kLoads = BM * (BK / 8) / kThreads;        // 16-byte pieces of A a thread
    static_assert(BN * BK / kThreads == 32, "a thread converts 32 weights a step");
};

// Piece c (8 values) of LDS row r sits at c ^ swizzle(r).
__device__ __forceinline__ int swizzle(int r) { return (r ^ (r >> 3)) & 7; }

// A thread's codes of two steps, as loaded and, once exchanged, by step. Forward: 32 columns, two scale bytes (in one
// or two words). Backward: 8 columns of four rows, four scale bytes (as loaded in four words of the first row, then
// packed in the first word of each).
struct Raw {
    uint32_t code[2][4], scale[2][4];
};

template <typename F>
__device__ __forceinline__ void unroll4(F&& f) {
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
}

// Where in the reduction a step lies: step `kt` of plane `plane` of matrix `m`.
struct Cursor {
    int kt = 0, plane = 0, m = 0;
    __device__ __forceinline__ void at(int step, int nk, int planes) {
        kt = step % nk;
        plane = step / nk % planes;
        m = step / nk / planes;
    }
    __device__ __forceinline__ void next(bool really, int nk, int planes) {
        const int k = kt + (really ? 1 : 0), q = plane + (k == nk ? 1 : 0);
        kt = k == nk ? 0 : k;
        plane = q == planes ? 0 : q;
        m += q == planes ? 1 : 0;
    }
};

// Workgroup -> tile. Workgroups go to the 8 XCDs in turn. One matrix: XCD x takes a run of tiles, and a run walks down 4
// row tiles before the next column tile, so that the 32 workgroups on an XCD read 4 row tiles and 8 column tiles together.
// Several: how many row tiles there are is not known here, and rows of different matrices share nothing but their own
// column tiles. From kManyRowTiles on XCD x takes every eighth row tile (with runs, 2048 x 768 by 128 rows each of 128
// matrices left half of the XCDs without work, 165 us); fewer would leave XCDs without work that way, so a run walks down all
// row tiles before the next column tile (gradients of 512 rows by 2 of 2 x 14336 x 4096 224 us, by every eighth
// row tile 378; 48 row tiles 74.6 and 79; 64 150 and 137).
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t nm, uint32_t nn, bool several, int& tm, int& tn) {
    const uint32_t xcd = id & 7, j = id >> 3;
    if (several && nm >= (uint32_t)kManyRowTiles) {
        tm = (int)(j / nn * 8 + xcd);
        tn = (int)(j % nn);
        return;
    }
    const uint32_t blocks = nm * nn, rest = blocks & 7;
    const uint32_t q = xcd * (blocks >> 3) + min(xcd, rest) + j;
    const uint32_t down = several ? nm : 4;
    const uint32_t group = q / (down * nn), l = q - group * down * nn;
    const uint32_t high = min(down, nm - down * group);
    tn = (int)(l / high);
    tm = (int)(down * group + l - (uint32_t)tn * high);
}

// WHOLE (forward): in is a multiple of 32, so a thread's 32 columns are all inside the matrix or all outside.
template <int M_, int N_, int WM_, int WN_, int MODE, bool F32, bool WHOLE>
__global__ __launch_bounds__(64 * WM_ * WN_) void k_product_tiles(Product p, int nm, int nn, int splits, int each) {
    typedef Shape<M_, N_, WM_, WN_> S;
    constexpr int BM = S::BM, BN = S::BN, TM = S::TM, TN = S::TN;
    __shared__ __align__(1024) uint16_t lds[2 * (BM + BN) * BK];
    uint16_t (&lds_a)[2][BM][BK] = *reinterpret_cast<uint16_t (*)[2][BM][BK]>(lds);
    uint16_t (&lds_b)[2][BN][BK] = *reinterpret_cast<uint16_t (*)[2][BN][BK]>(lds + 2 * BM * BK);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const uint32_t of = blockIdx.x / (uint32_t)splits;
    const int split = (int)(blockIdx.x - of * (uint32_t)splits);
    int tile, tn;
    tile_of(of, (uint32_t)nm, (uint32_t)nn, p.rows.batch > 1, tile, tn);
    RowTile rows;
    if (!find_rows(p.rows, tile, BM, rows)) return;

    constexpr int kCols = MODE == kGated ? BN / 2 : BN;            // output columns of a tile
    const int64_t n0 = (int64_t)tn * kCols;
    const int64_t N = MODE == kBackward ? p.in : p.out;
    const int K = (int)(MODE == kBackward ? p.out : p.in);
    const int k_pad = (K + 7) & ~7;
    const int nk = (K + 2 * BK - 1) / (2 * BK) * 2;      // steps go in pairs: the last one may be empty
    const int matrices = MODE == kBackward ? p.matrices : 1;
    const int begin = split * each, steps = min(each, nk * p.planes * matrices - begin);
    const int to_switch = nk * p.planes - begin;         // the step at which the next matrix begins
    // Of two matrices the one of the smaller S goes first, so that the quotient of the S by which its sums go over to the
    // other's is at most 1: the sums of two matrices do not overflow where dX does not.
    int swapped = 0;
    if constexpr (MODE == kBackward)
        swapped = __builtin_amdgcn_readfirstlane(matrices == 2 && p.w[0].S[rows.e] > p.w[1].S[rows.e]);

    // copies of the rows' side: a thread's piece is the same in each of its rows
    const uint16_t* const a0 = p.a[0].p + rows.first * p.a[0].ld;
    const uint16_t* const a1 = p.a[1].p + rows.first * p.a[1].ld;
    uint32_t xrow[S::kLoads];
#pragma unroll
    for (int r = 0; r < S::kLoads; ++r)                  // rows past the tile read its last row: they are not stored
        xrow[r] = (uint32_t)min((tid + S::kThreads * r) >> 3, rows.rows - 1) * (uint32_t)p.a[0].ld * 2;
    // rows 32 apart differ in bit 2 of the swizzle, rows 64 apart have the same
    constexpr int kPieces = S::kThreads == 256 ? 2 : 1;
    static_assert(S::kThreads == 256 || S::kThreads == 512, "32 or 64 rows a turn");
    const int xpiece = ((tid & 7) ^ swizzle(tid >> 3)) * 16;
    struct Source {
        const uint16_t* p;
        uint32_t at[kPieces];
    };
    const auto source = [&](const Cursor& c) {
        // pieces past the edge read the row's last: they meet weights of zero
        const uint16_t* base = MODE == kBackward && (c.m ^ swapped) ? a1 : a0;
        const int kt = min(c.kt, (K - 1) / BK);
        base += c.plane * p.plane + kt * BK;
        const int last = (k_pad - kt * BK) * 2 - 16;
        Source s;
        s.p = reinterpret_cast<const uint16_t*>(uniform(reinterpret_cast<int64_t>(base)));
#pragma unroll
        for (int k = 0; k < kPieces; ++k) s.at[k] = (uint32_t)min(xpiece ^ (64 * k), last);
        return s;
    };
    const auto load_a = [&](int buf, const Source& from, int r) {
        copy16_unseen(from.p, xrow[r] + from.at[r % kPieces], &lds_a[buf][(S::kThreads * r + 64 * wave) >> 3][0]);
    };

    // The codes of two steps are loaded together and lanes two apart exchange half of theirs, so that each has its
    // share of either step: half as many loads, of twice the length. (64 bytes of a row by four lanes instead of 32
    // by two took 4 to 8% off the whole.)
    const bool b_high = lane & 2;
    // forward: a lane loads a quarter of 128 columns of row lane / 4 of the wave's 32 and of the row 16 behind; it has
    // half b_half of row b_row of lds_b
    const int b_row = 32 * wave + (lane >> 2) + (b_high ? 16 : 0), b_half = lane & 1;
    // backward: a lane loads 16 columns of 4 rows of one of the steps; it has columns 8 b_block .. + 7, values
    // 8 b_octet + 4 b_quad .. + 3
    const int b_block = (tid >> 2) % (BN / 16) * 2 + (b_high ? 1 : 0), b_octet = (tid >> 2) / (BN / 16), b_quad = tid & 1;
    const int b_first = (b_high ? BK : 0) + b_octet * 8 + b_quad * 4;
    uint32_t b_code[2], b_scale[2];                      // of the thread's first codes: bytes from the windows' start
    const uint8_t *codes, *scales;                       // forward: from row n0 (of the wave's matrix)
    if constexpr (MODE == kBackward) {
        const uint32_t at = (uint32_t)b_first * (uint32_t)N + (uint32_t)min(n0 + (b_block >> 1) * 16, N - 16);
        b_code[0] = at / 2;
        b_scale[0] = at / 16;
    } else {
        const ProductMatrix& w = p.w[MODE == kGated ? wave & 1 : 0];   // a wave's 32 rows are of one matrix
        const int64_t at = rows.e * w.stride + n0 * K;
        codes = w.packed + at / 2;
        scales = w.scales + at / 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c32 = (MODE == kGated ? (wave >> 1) * 32 : wave * 32) + (lane >> 2) + 16 * h;
            b_scale[h] = (uint32_t)(min(n0 + c32, N - 1) - n0) * (uint32_t)(K / 16) + 2 * (lane & 3);
            b_code[h] = b_scale[h] * 8;
        }
    }
    const auto load_b = [&](Raw& raw, const Cursor& c, int step) {
        const int left = K - c.kt * BK;                  // of the reduction
        const uint32_t reach = step < steps ? kReach : 0;              // no codes past the last step
        if constexpr (MODE == kBackward) {
            const ProductMatrix& w = p.w[c.m ^ swapped];
            const int64_t at = rows.e * w.stride + (int64_t)c.kt * BK * N;
            const __amdgpu_buffer_rsrc_t from = window(w.packed + at / 2, reach), bytes = window(w.scales + at / 16, reach);
            const int mine = left - b_first;
#pragma unroll
            for (int r = 0; r < 4; ++r) {                // N / 2 and N / 16 are whole
                const u32x2 w2 = load8(from, offset_if(r < mine, b_code[0]), (uint32_t)r * (uint32_t)(N / 2));
                raw.code[0][r] = w2[0];
                raw.code[1][r] = w2[1];
                raw.scale[0][r] = load1(bytes, offset_if(r < mine, b_scale[0]), (uint32_t)r * (uint32_t)(N / 16));
            }
        } else {
            const __amdgpu_buffer_rsrc_t from = window(codes, reach), bytes = window(scales, reach);
            const uint32_t k = (uint32_t)c.kt * (BK / 16);
            const bool in = (lane & 3) * 32 < left, in2 = (lane & 3) * 32 + 16 < left;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 w;
                if constexpr (WHOLE) {
                    w = load16(from, offset_if(in, b_code[h]), k * 8);
                    raw.scale[h][0] = load2(bytes, offset_if(in, b_scale[h]), k);
                } else {
                    const u32x2 lo = load8(from, offset_if(in, b_code[h]), k * 8);
                    const u32x2 hi = load8(from, offset_if(in2, b_code[h] + 8), k * 8);
                    w = u32x4{lo[0], lo[1], hi[0], hi[1]};
                    raw.scale[h][0] = load1(bytes, offset_if(in, b_scale[h]), k);
                    raw.scale[h][1] = load1(bytes, offset_if(in2, b_scale[h] + 1), k);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) raw.code[h][j] = w[j];
            }
        }
    };
    const auto exchange = [&](uint32_t& a, uint32_t& b) {
        const uint32_t got = swap_pairs(b_high ? a : b);
        a = b_high ? got : a;
        b = b_high ? b : got;
    };
    // a quarter of a thread's weights of the even or odd step of two, converted and written: piece 0 .. 3; the even
    // step's come first and make the exchange
    const auto store_b = [&](int buf, Raw& raw, auto odd, auto which) {
        constexpr int I = decltype(which)::value, ODD = decltype(odd)::value;
        if constexpr (MODE == kBackward) {
            if constexpr (ODD == 0 && I == 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r) exchange(raw.code[0][r], raw.code[1][r]);
                const uint32_t mine = raw.scale[0][0] | raw.scale[0][1] << 8 | raw.scale[0][2] << 16 | raw.scale[0][3] << 24;
                const uint32_t other = swap_pairs(mine);
                raw.scale[0][0] = b_high ? other : mine;
                raw.scale[1][0] = b_high ? mine : other;
            }
            const uint32_t bytes = raw.scale[ODD][0];
            const float s[4] = {scale_value<0>(bytes), scale_value<1>(bytes), scale_value<2>(bytes), scale_value<3>(bytes)};
            float x[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) code_values<I>(raw.code[ODD][r], s[r], x[r][0], x[r][1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = b_block * 8 + 2 * I + j;
                *reinterpret_cast<u32x2*>(&lds_b[buf][row][(b_octet ^ swizzle(row)) * 8 + b_quad * 4]) =
                    u32x2{bf16_pair(x[0][j], x[1][j]), bf16_pair(x[2][j], x[3][j])};
            }
        } else {
            if constexpr (ODD == 0) {
                exchange(raw.code[0][I], raw.code[1][I]);
                if constexpr (I == 0) exchange(raw.scale[0][0], raw.scale[1][0]);
                if constexpr (!WHOLE && I == 2) exchange(raw.scale[0][1], raw.scale[1][1]);
            }
            const float s = I < 2 ? scale_value<0>(raw.scale[ODD][0]) : WHOLE ? scale_value<1>(raw.scale[ODD][0])
                                                                              : scale_value<0>(raw.scale[ODD][1]);
            *reinterpret_cast<u32x4*>(&lds_b[buf][b_row][((b_half * 4 + I) ^ swizzle(b_row)) * 8]) =
                dequant8(raw.code[ODD][I], s);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;

    // operands of one slice of 16: a lane holds values 8 kg .. + 7 of row r32 of each 32-row block
    struct Frag {
        bf16x8 a[TM], b[TN];
    };
    const int r32 = lane & 31, kg = lane >> 5;
    const auto read = [&](Frag& f, int buf, int slice) {
        const int c = 2 * slice + kg;
#pragma unroll
        for (int b = 0; b < TN; ++b) {
            const int row = (wn * TN + b) * 32 + r32;
            f.b[b] = *reinterpret_cast<const bf16x8*>(&lds_b[buf][row][(c ^ swizzle(row)) * 8]);
        }
#pragma unroll
        for (int a = 0; a < TM; ++a) {
            const int row = (wm * TM + a) * 32 + r32;
            f.a[a] = *reinterpret_cast<const bf16x8*>(&lds_a[buf][row][(c ^ swizzle(row)) * 8]);
        }
    };
    const auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int b = 0; b < TN; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[a], f.b[b], acc[a][b], 0, 0, 0);
    };
    // the order of a slice: its matrix instructions with the next slice's reads and a quarter of the conversion between
    const auto interleave = [&]() {
#pragma unroll
        for (int i = 0; i < TM * TN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, (24 + TM * TN - 1) / (TM * TN), 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // Step s is multiplied from one half of LDS while step s + 1 is made in the other: its rows are copied, its
    // codes converted from registers, and the codes of the steps after it loaded. A step's one barrier stands before
    // its last slice, whose operands are in registers by then: behind it the first half is free, and the last
    // slice's matrix instructions cover the reads of step s + 1's first operands. Steps go in fours: past the last,
    // copies are of the last step again and codes zeros (more ways out of the loop would cost registers).
    Cursor ca, cb;
    cb.at(begin, nk, p.planes);
    ca = cb;
    Raw raw[2];
    int loaded = 0;
    const auto load_next = [&](Raw& r) {
        load_b(r, cb, loaded);
        cb.next(++loaded < steps, nk, p.planes);
        cb.next(++loaded < steps, nk, p.planes);
    };
    int copied = 0;
    const auto source_next = [&]() {
        const Source from = source(ca);
        ca.next(++copied < steps, nk, p.planes);
        return from;
    };
    const auto load_all = [&](int buf) {
        const Source from = source_next();
#pragma unroll
        for (int r = 0; r < S::kLoads; ++r) load_a(buf, from, r);
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    load_next(raw[0]);
    load_all(0);
    load_next(raw[1]);
    load_all(1);
    unroll4([&](auto i) { store_b(0, raw[0], even, i); });
    wait_copies<0>();
    barrier();
    Frag f[2];
    read(f[0], 0, 0);
    store_b(1, raw[0], odd, even);
    __builtin_amdgcn_sched_barrier(0);
    const auto step = [&](int s, auto which) {
        constexpr int J = decltype(which)::value, buf = J & 1;
        // where step s + 1's codes are, and step s + 2's
        constexpr int X = ((J + 1) >> 1) & 1, Y = ((J + 2) >> 1) & 1;
        const std::integral_constant<int, (J + 1) & 1> x_odd;
        const std::integral_constant<int, J & 1> y_odd;
        if constexpr (MODE == kBackward) {
            if (s == to_switch && s > 0 && s < steps) {  // the sums carry the S of the matrix met last
                const float r = p.w[swapped].S[rows.e] / p.w[1 - swapped].S[rows.e];
#pragma unroll
                for (int a = 0; a < TM; ++a)
#pragma unroll
                    for (int b = 0; b < TN; ++b)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[a][b][e] *= r;
            }
        }
        read(f[1], buf, 1);
        multiply(f[0]);
        store_b(buf ^ 1, raw[X], x_odd, std::integral_constant<int, 1>{});
        interleave();
        read(f[0], buf, 2);
        multiply(f[1]);
        store_b(buf ^ 1, raw[X], x_odd, std::integral_constant<int, 2>{});
        interleave();
        read(f[1], buf, 3);
        multiply(f[0]);
        store_b(buf ^ 1, raw[X], x_odd, std::integral_constant<int, 3>{});
        interleave();
        const Source from = source_next();
        wait_copies<0>();                                // step s + 1's rows and step s + 2's codes
        barrier();
        // the last slice: its matrix instructions in TM groups, with the copies between
        read(f[0], buf ^ 1, 0);
#pragma unroll
        for (int a = 0; a < TM; ++a) {
#pragma unroll
            for (int b = 0; b < TN; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[1].a[a], f[1].b[b], acc[a][b], 0, 0, 0);
#pragma unroll
            for (int r = a * S::kLoads / TM; r < (a + 1) * S::kLoads / TM; ++r) load_a(buf, from, r);
            if (a == TM - 1) {
                if constexpr (J % 2 == 0) load_next(raw[X]);           // it has been used up
                store_b(buf, raw[Y], y_odd, even);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    for (int s = 0; s < steps; s += 4) {
        step(s, std::integral_constant<int, 0>{});
        step(s + 1, std::integral_constant<int, 1>{});
        step(s + 2, std::integral_constant<int, 2>{});
        step(s + 3, std::integral_constant<int, 3>{});
    }
    wait_copies<0>();
    barrier();

    // a lane holds rows 8 (e / 4) + 4 kg + e % 4 of column r32 of each 32 x 32 tile; backward, the sums are over the
    // S of the last matrix met
    const int at = swapped ^ (MODE == kBackward && to_switch < steps ? 1 : 0);
    const float S0 = p.w[at].S[rows.e];
    const float S1 = MODE == kGated ? p.w[1].S[rows.e] : 0.0f;
    // 32 rows at a time by way of the wave's own part of LDS, so that a lane has 8 columns of a row
    constexpr int kWide = TN * 32 + 4, kLanes = (MODE == kGated ? TN * 16 : TN * 32) / 8;
    static_assert(sizeof(float) * 32 * kWide * S::WM * S::WN <= sizeof(lds_a) + sizeof(lds_b), "LDS of the outputs");
    float* mine = reinterpret_cast<float*>(lds) + wave * 32 * kWide;
    const int64_t n_wave = n0 + wn * (MODE == kGated ? TN * 16 : TN * 32);
#pragma unroll
    for (int a = 0; a < TM; ++a) {
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                mine[((e >> 2) * 8 + kg * 4 + (e & 3)) * kWide + b * 32 + r32] =
                    acc[a][b][e] * (MODE == kGated && b % 2 ? S1 : S0);
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 64 / kLanes) {
            const int r = r0 + lane / kLanes, c = lane % kLanes * 8, row = (wm * TM + a) * 32 + r;
            // gated: 8 of the 32 columns of a pair of MFMA tiles
            const float* from = mine + r * kWide + (MODE == kGated ? c / 32 * 64 + c % 32 : c);
            float v[8], u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = from[k];
                u[k] = MODE == kGated ? from[32 + k] : 0.0f;
            }
            if (row < rows.rows && n_wave + c < N)
                product_out8<MODE == kGated, F32>(p, splits, split, rows.e, rows.first + row, n_wave + c, N, v, u);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

typedef Shape<128, 128, 2, 2> Small;
typedef Shape<256, 256, 2, 4> Big;

template <typename S, int MODE>
void launch(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    const int64_t N = MODE == kBackward ? p.in : p.out, K = MODE == kBackward ? p.out : p.in;
    const int64_t cols = MODE == kGated ? S::BN / 2 : S::BN, nn = (N + cols - 1) / cols;
    const int64_t steps = (K + 2 * BK - 1) / (2 * BK) * 2 * p.planes * (MODE == kBackward ? p.matrices : 1);
    const int64_t each = ((steps + plan.splits - 1) / plan.splits + 3) / 4 * 4;
    const int64_t nm = product_tile_rows(p.rows.tokens, p.rows.batch, S::BM);
    const dim3 grid((uint32_t)(nm * nn * plan.splits)), threads(S::kThreads);
    const bool whole = MODE == kBackward || p.in % 32 == 0;
    if (p.f32 && whole)
        hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, true, true>), grid, threads, 0, stream, p,
                           (int)nm, (int)nn, plan.splits, (int)each);
    else if (whole)
        hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, false, true>), grid, threads, 0, stream, p,
                           (int)nm, (int)nn, plan.splits, (int)each);
    else if constexpr (MODE != kBackward) {
        if (p.f32)
            hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, true, false>), grid, threads, 0,
                               stream, p, (int)nm, (int)nn, plan.splits, (int)each);
        else
            hipLaunchKernelGGL((k_product_tiles<S::BM, S::BN, S::WM, S::WN, MODE, false, false>), grid, threads, 0,
                               stream, p, (int)nm, (int)nn, plan.splits, (int)each);
    }
}

template <typename S>
void launch(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    if (p.backward) launch<S, kBackward>(p, plan, stream);
    else if (p.matrices == 2) launch<S, kGated>(p, plan, stream);
    else launch<S, kLinear>(p, plan, stream);
}

}  // namespace

void launch_product_tiles(const Product& p, const ProductPlan& plan, hipStream_t stream) {
    if (plan.tile_cols == 128) launch<Small>(p, plan, stream);
    else launch<Big>(p, plan, stream);
}

}  // namespace nvfp4
