// Grouped matrix product over the receive segments with its epilogue:
// out[r] = act(x[r] W[e]^T + b[e]) + residual[r] for the rows r of segment e.
//
// A workgroup computes one tile of BM rows by BN columns (gated activations:
// BN / 2 gate and the matching up columns, so that the activation needs no
// second pass).  Both operands pass through LDS in K steps of 128 bytes per
// row (64 bf16 or 128 fp8 channels), copied there without registers.
//
// The weights are the matrix instruction's first operand, so four accumulators
// of a lane are four consecutive columns of one row.  The sums change lanes in
// LDS once, so that bias, residual, codes and output move in whole lines.
//
// LDS rows are 8 chunks of 16 bytes, chunk c of row r in slot c ^ (r/2 & 7):
// the 16 rows x 16 bytes a quarter wave reads lie in 16 different slots of the
// 256-byte bank line.  Weights that lie [k, n] (transposed) are staged as 64
// rows of 256 columns and read by the transposing LDS read.
#include <algorithm>

#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kBN = 256;

struct LinearK {
    SegmentRows seg;
    const uint8_t *x;
    const uint8_t *x_scales;
    const uint8_t *w;
    const uint8_t *w_scales;
    const uint16_t *bias;
    const uint16_t *residual;
    uint16_t *out;
    uint8_t *ckpt;
    uint8_t *ckpt_scales;
    int n, k, m;          // weight rows, contraction, output columns
    int kind;             // activation function
    int col_tiles;
};

// Four consecutive scale bytes of a row from step s on, as far as the row has them.
__device__ __forceinline__ int scales4(const uint8_t *row, int s, int groups) {
    int v = 0;
    if (s + 4 <= groups) {
        __builtin_memcpy(&v, row + s, 4);
    } else {
        for (int i = 0; s + i < groups; ++i) v |= (int)row[s + i] << (8 * i);
    }
    return v;
}

// What a kernel multiplies: bf16 rows; fp8 rows by the fp8 instruction; fp8 rows
// turned to bf16 on the way, for a checkpoint.
enum { kBf16, kFp8, kFp8Exact };

// The fp8 matrix instruction with one scale byte (SB of four) per operand row.
// It adds into fp32, but the products of 8 consecutive channels are first
// aligned to the largest of them and cut off below 2^-13 of it: a loss around
// 1e-5 of sum |x w|, well inside the result's bf16 rounding, for twice the bf16
// instruction's rate.  A checkpoint is taken from the sums themselves, and there it
// showed: one code in 1000 was not the nearest one (one in 10^5 of the bf16
// products' sums).  So with a checkpoint the operands become bf16 values, which is
// exact (a code has four significant bits, the scales are powers of two; the value
// stays a normal number from 2^-126 to 2^127), and the bf16 instruction multiplies
// them: 8 experts, 32768 rows of 7168 to 4096, swiglu, 1.71 ms, between the 0.82 of
// the fp8 instruction and bf16 rows' 1.51 with the same checkpoint.  (Converted in
// front of the instruction that needs it, or once for all four parts of a step, with
// the copies' offsets spilled: 3.5 to 4.2 ms.)
template <int SB>
__device__ __forceinline__ ep_f32x4 mfma_fp8(const ep_u32x4 *a, const ep_u32x4 *b, ep_f32x4 c,
                                             int sa, int sb) {
    // a lane's 32 channels are chunks q and q + 4 of the row, alike in both
    // operands; one scale covers all 128
    ep_i32x8 x, y;
    x.lo = __builtin_bit_cast(ep_i32x4, a[0]);
    x.hi = __builtin_bit_cast(ep_i32x4, a[1]);
    y.lo = __builtin_bit_cast(ep_i32x4, b[0]);
    y.hi = __builtin_bit_cast(ep_i32x4, b[1]);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, SB, sa, SB, sb);
}

// Codes 8 P to 8 P + 7 of a lane's 32 (chunks q and q + 4), times the row's power
// of two, as a bf16 operand.  Which channels a piece holds does not matter: they
// are the same of both operands.
template <int P>
__device__ __forceinline__ ep_u32x4 piece_of(const ep_u32x4 *codes, float scale) {
    const uint32_t lo = codes[P >> 1][(P & 1) * 2], hi = codes[P >> 1][(P & 1) * 2 + 1];
    ep_u32x4 v;
    v.x = fp8_pair_bf16<false>(lo, scale);
    v.y = fp8_pair_bf16<true>(lo, scale);
    v.z = fp8_pair_bf16<false>(hi, scale);
    v.w = fp8_pair_bf16<true>(hi, scale);
    return v;
}

// The power of two of byte SB of four scale bytes.
template <int SB>
__device__ __forceinline__ float scale_byte(int bytes) {
    return ue8m0_value((uint32_t)bytes >> (8 * SB) & 0xFF);
}

// Bias, checkpoint, activation, residual and output of a wave's accumulators: NT
// tiles of 16 columns of z (gated: the first half gates, the second their ups)
// by MT of 16 rows, STRIDE apart from row `first` of the segment on, `live_rows`
// of the segment's rows left there;
// c0 is the first column of out.  Accumulator j of tile (t, i) is column 16 t + 4
// q + j, row 16 i + lane % 16.  The sums go through the wave's part of the LDS in
// batches of BT row tiles, fp32, 16-byte chunk c of row r in place c ^ (r & 15),
// and come back as 8 consecutive columns of one row per lane: the arithmetic is
// a short loop over rows (unrolled over the registers it would not fit the
// instruction cache), and residual, output and codes move in whole lines.
// The residual of the first batch may be on its way since before the product.
template <int NT, int BT, int STRIDE, bool GATED>
struct Output {
    static constexpr int COLS = NT * 16, OUT = GATED ? COLS / 2 : COLS;
    static constexpr int LANES = OUT / 8;              // lanes of a row
    static constexpr int RPI = 64 / LANES;             // rows of an iteration
    static constexpr int IT = BT * 16 / RPI;           // iterations of a batch
    ep_u32x4 res[IT];

    // first row of iteration i of a batch
    static __device__ __forceinline__ constexpr int row_of(int batch, int i) {
        return (batch * BT + i * RPI / 16) * STRIDE + i * RPI % 16;
    }
    __device__ __forceinline__ void load(const LinearK &a, const TileAt &at, int first,
                                         int live_rows, int c0, int batch) {
        if (!a.residual) return;
        const int lane = threadIdx.x & 63, lc = lane % LANES, lr = lane / LANES;
        const uint16_t *p = a.residual + ((int64_t)at.row0 + first + lr) * a.m + c0 + lc * 8;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = row_of(batch, i);
            res[i] = ep_u32x4{0, 0, 0, 0};
            if (c0 + lc * 8 < a.m && r + lr < live_rows) res[i] = *(const ep_u32x4 *)(p + (int64_t)r * a.m);
        }
    }
};

template <int KIND, int NT, int MT, int BT, int STRIDE, bool GATED>
__device__ __forceinline__ void epilogue_of(const LinearK &a, const TileAt &at, uint8_t *lds,
                                            int first, int live_rows, int c0,
                                            ep_f32x4 (*acc)[MT],
                                            Output<NT, BT, STRIDE, GATED> &now) {
    typedef Output<NT, BT, STRIDE, GATED> O;
    constexpr int COLS = O::COLS, OUT = O::OUT, LANES = O::LANES, RPI = O::RPI, IT = O::IT;
    constexpr int NK = GATED ? 2 : 1;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int lc = lane % LANES, lr = lane / LANES;
    const int N = a.n, m = a.m;
    const int col = c0 + lc * 8;
    const bool there = col < m;                        // n is a multiple of 8 (m too)
    const int64_t row0 = (int64_t)at.row0 + first + lr;
    float b[NK][8];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        ep_u32x4 v = {0, 0, 0, 0};
        if (a.bias && there) v = *(const ep_u32x4 *)(a.bias + (int64_t)at.e * N + k * m + col);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b[k][2 * j] = bf16_lo(v[j]);
            b[k][2 * j + 1] = bf16_hi(v[j]);
        }
    }
    each<MT / BT>([&](auto bb) __attribute__((always_inline)) {
        constexpr int batch = decltype(bb)::value;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < BT; ++i) {
                ep_f32x4 s = acc[t][batch * BT + i];
                pin(s);
                *(ep_f32x4 *)(lds + (i * 16 + l16) * COLS * 4 + ((t * 4 + q) ^ l16) * 16) = s;
            }
        O next;
        if (batch + 1 < MT / BT) next.load(a, at, first, live_rows, c0, batch + 1);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int at_row = O::row_of(batch, i);
            const int r = i * RPI + lr;
            const bool live = there && at_row + lr < live_rows;
            const int64_t row = row0 + at_row;
            float z[NK][8];
#pragma unroll
            for (int k = 0; k < NK; ++k) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = k * (OUT / 4) + lc * 2 + h;
                    const ep_f32x4 v = *(const ep_f32x4 *)(lds + r * COLS * 4 + (c ^ (r & 15)) * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[k][4 * h + j] = v[j] + b[k][4 * h + j];
                }
                if (a.ckpt) {
                    // 32 channels, four lanes, to e4m3 codes under a power of
                    // two: the format of ep_cast_fp8 with UE8M0 scales, taken
                    // from the fp32 sums.  (n is a multiple of the group: its
                    // channels are all there or none is.)
                    float big = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(z[k][j]));
                    big = fminf(group_max(big, 4), 3.0e38f);
                    const uint32_t e = ue8m0_of(pow2_ceil(scale_of(big)));
                    const float inv = __uint_as_float((254u - e) << 23);
                    ep_u32x2 codes;
                    codes.x = pack4_e4m3(z[k][0] * inv, z[k][1] * inv, z[k][2] * inv, z[k][3] * inv);
                    codes.y = pack4_e4m3(z[k][4] * inv, z[k][5] * inv, z[k][6] * inv, z[k][7] * inv);
                    if (live) {
                        const int64_t o = row * N + k * m + col;
                        *(ep_u32x2 *)(a.ckpt + o) = codes;
                        if ((lane & 3) == 0) a.ckpt_scales[o >> 5] = (uint8_t)e;
                    }
                }
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = act_value<KIND>(z[0][j]);
                if (GATED) y[j] *= z[NK - 1][j];
            }
            if (a.residual) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t v = now.res[i][j >> 1];
                    y[j] += (j & 1) ? bf16_hi(v) : bf16_lo(v);
                }
            }
            if (live)
                *(ep_u32x4 *)(a.out + row * m + col) =
                    ep_u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                             pack_bf16(y[6], y[7])};
        }
        if (batch + 1 < MT / BT) now = next;
    });
}

template <int NT, int MT, int BT, int STRIDE, bool GATED>
__device__ __forceinline__ void epilogue(const LinearK &a, const TileAt &at, uint8_t *lds, int first,
                                         int live_rows, int c0, ep_f32x4 (*acc)[MT],
                                         Output<NT, BT, STRIDE, GATED> &o) {
    if (a.kind == 1) epilogue_of<1, NT, MT, BT, STRIDE, GATED>(a, at, lds, first, live_rows, c0, acc, o);
    else if (a.kind == 2) epilogue_of<2, NT, MT, BT, STRIDE, GATED>(a, at, lds, first, live_rows, c0, acc, o);
    else if (!GATED) epilogue_of<0, NT, MT, BT, STRIDE, GATED>(a, at, lds, first, live_rows, c0, acc, o);
}

// Tiles of 128 or 192 rows by 256 columns, for experts of few rows: bound by
// reading the weights (256 experts of 7168 x 4096, 128 rows each, swiglu: 3.1 ms,
// 5.0 TB/s); tiles of 64 by 64 for small products, bound by the latency
// of a step.
// The ring of NS stages keeps NS - 1 steps in flight; row tiles that hold no row
// are not multiplied.
template <int BM, int WM, int WN, int NS, int IN, bool WT, bool GATED>
__global__ __launch_bounds__(64 * WN * WM, 2) void expert_linear_kernel(LinearK a) {
    constexpr bool FP8 = IN != kBf16, EXACT = IN == kFp8Exact;
    constexpr int kWaves = WN * WM;
    constexpr int BN = 64 * WN;
    static_assert(!WT || BN == 256, "transposed weights lie in rows of 256 columns");
    constexpr int MT = BM / WM / 16;               // 16-row tiles of a wave
    constexpr int kWStage = BN * 128, kXStage = BM * 128;
    constexpr int kStage = kWStage + kXStage;
    constexpr int WL = kWStage / 1024 / kWaves;    // copies of a wave per step
    constexpr int XL = kXStage / 1024 / kWaves;
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int BK = 128 / ES;
    __shared__ __align__(1024) uint8_t lds[NS * kStage];
    __shared__ int red[16];

    TileAt at;
    if (!find_tile<64 * kWaves>(a.seg, BM, a.col_tiles, blockIdx.x, red, &at)) return;

    const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    const int K = a.k, N = a.n;
    const int half = N >> 1;
    const int row0 = at.mt * BM;                       // in the segment
    const int rows = min(BM, at.rows - row0);

    // copies: source offsets of this lane
    const uint32_t ld_bytes = (uint32_t)K * ES;
    const ep_i32x4 xb = buffer_of(a.x + ((int64_t)at.row0 + row0) * ld_bytes,
                                  (uint32_t)rows * ld_bytes);
    const uint32_t w_bytes = (uint32_t)N * ld_bytes;
    const ep_i32x4 wb = buffer_of(a.w + (int64_t)at.e * w_bytes, w_bytes);
    const int chunk = (lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7);
    uint32_t xoff[XL], woff[WL];
    int wk[WT ? WL : 1];                               // transposed: the k row of each copy
    for (int j = 0; j < XL; ++j) xoff[j] = (uint32_t)((j * kWaves + wave) * 8 + (lane >> 3)) * ld_bytes + chunk * 16;
    // column of the weights at place r of the tile: gated tiles hold,
    // per wave, 32 gate columns and the 32 up columns that go with them
    auto column = [&](int r) {
        if (!GATED) return at.nt * BN + r;
        const int c = at.nt * (BN / 2) + (r >> 6) * 32 + (r & 31);
        return (r & 32) ? half + c : c;
    };
    for (int j = 0; j < WL; ++j) {
        if (!WT) {
            const int r = (j * kWaves + wave) * 8 + (lane >> 3);
            const int c = column(r);
            woff[j] = (uint32_t)c * ld_bytes + chunk * 16;
            // a gated tile's columns past the halves lie in the other half or
            // behind the matrix: their products are not stored
            if (c >= N) woff[j] = kOutOfRange;
        } else {
            const int kr = (j * kWaves + wave) * 2 + (lane >> 5);
            const int c16 = lane & 31;
            const int c = column(((c16 >> 1) ^ granule_of(kr)) * 16 + (c16 & 1) * 8);
            wk[j] = kr;
            woff[j] = (uint32_t)kr * (uint32_t)N * 2 + (uint32_t)c * 2;
            if (c >= N) woff[j] = kOutOfRange;
        }
    }
    const uint32_t lds0 = lds_offset(lds);
    const int steps = (K + BK - 1) / BK;
    // copies of x that hold a row, of this wave's: the others are left out, and
    // the rows behind the segment are what the LDS holds (they go nowhere)
    const int xl = max(0, min(XL, ((rows + 7) / 8 - wave + kWaves - 1) / kWaves));
    auto copy = [&](int s, int stage) {
        const uint32_t base = lds0 + stage * kStage + wave * 1024;
        const bool tail = !FP8 && (s + 1) * BK > K;
        if (tail) {
            // channels at or past K become zeros in both operands
            const uint32_t out = s * BK + chunk * 8 >= K ? kOutOfRange : 0;
            for (int j = 0; j < WL; ++j) {
                const uint32_t wo = WT ? (s * BK + wk[WT ? j : 0] >= K ? kOutOfRange : 0) : out;
                dma16(wb, base + j * kWaves * 1024, woff[j] | wo,
                      WT ? (uint32_t)s * BK * (uint32_t)N * 2 : s * 128);
            }
            for (int j = 0; j < XL; ++j)
                if (j < xl) dma16(xb, base + kWStage + j * kWaves * 1024, xoff[j] | out, s * 128);
        } else {
            for (int j = 0; j < WL; ++j)
                dma16(wb, base + j * kWaves * 1024, woff[j],
                      WT ? (uint32_t)s * BK * (uint32_t)N * 2 : s * 128);
            for (int j = 0; j < XL; ++j)
                if (j < xl) dma16(xb, base + kWStage + j * kWaves * 1024, xoff[j], s * 128);
        }
    };

    ep_f32x4 acc[4][MT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = ep_f32x4{0, 0, 0, 0};

    int xs[FP8 ? MT : 1], ws[FP8 ? 4 : 1];             // fp8: scale bytes of four steps
    auto scales = [&](int s) {
        const int groups = K / kFp8Group;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = min((i * WM + wm) * 16 + l16, rows - 1);
            xs[FP8 ? i : 0] = scales4(a.x_scales + ((int64_t)at.row0 + row0 + r) * groups, s, groups);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int c = min(column(wn * 64 + t * 16) + l16, N - 1);
            ws[FP8 ? t : 0] = scales4(a.w_scales + ((int64_t)at.e * N + c) * groups, s, groups);
        }
    };

    // row tiles of this wave that hold a row: the waves take them in turn
    const int live = ((rows + 15) / 16 - wm + WM - 1) / WM;
    const int slot = l16 * 128 + (q ^ (l16 >> 1)) * 16;
    auto compute = [&](int stage, auto sb) {
        if (live <= 0) return;
        const uint8_t *wl = lds + stage * kStage;
        const uint8_t *xl = wl + kWStage + wm * 2048;
        ep_u32x4 wf[4][2], xf[MT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                wf[t][h] = WT ? transposed_operand<512>(wl, wn * 4 + t, h)
                              : *(const ep_u32x4 *)(wl + (wn * 4 + t) * 2048 + (slot ^ (h * 64)));
        auto read_x = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                xf[i][h] = *(const ep_u32x4 *)(xl + i * WM * 2048 + (slot ^ (h * 64)));
        };
        read_x(0);
        // all reads before the first product: with few registers in use the
        // compiler would wait for each by itself
        __builtin_amdgcn_sched_barrier(0);
        constexpr int SB = decltype(sb)::value;
        ep_u32x4 wp[EXACT ? 4 : 1][4];                 // [tile][piece]
        if (EXACT) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                each<4>([&](auto p) __attribute__((always_inline)) {
                    wp[EXACT ? t : 0][p] = piece_of<p>(wf[t], scale_byte<SB>(ws[FP8 ? t : 0]));
                });
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (i >= live) break;
            if (i > 0) read_x(i);
            if (EXACT) {
                each<4>([&](auto p) __attribute__((always_inline)) {
                    const ep_u32x4 v = piece_of<p>(xf[i], scale_byte<SB>(xs[FP8 ? i : 0]));
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t][i] = mfma_bf16(wp[EXACT ? t : 0][p], v, acc[t][i]);
                });
                continue;
            }
#pragma unroll
            for (int h = 0; h < (FP8 ? 1 : 2); ++h)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (FP8)
                        acc[t][i] = mfma_fp8<SB>(wf[t], xf[i], acc[t][i], ws[FP8 ? t : 0], xs[FP8 ? i : 0]);
                    else
                        acc[t][i] = mfma_bf16(wf[t][h], xf[i][h], acc[t][i]);
                }
        }
    };

    for (int s = 0; s < NS - 1; ++s)
        if (s < steps) copy(s, s);
    int stage = 0;
    auto step = [&](int s, auto sb) {
        // stage s has landed once at most the copies of the steps after it
        // are in flight; near the end there are none, and all are waited for
        if (s + NS - 2 < steps)
            each<XL + 1>([&](auto n) __attribute__((always_inline)) {
                if (xl == decltype(n)::value) dma_wait<(NS - 2) * (WL + decltype(n)::value)>();
            });
        else dma_wait<0>();
        barrier_only();
        const int next = stage == 0 ? NS - 1 : stage - 1;
        if (s + NS - 1 < steps) copy(s + NS - 1, next);
        compute(stage, sb);
        stage = stage + 1 == NS ? 0 : stage + 1;
    };
    if (FP8) {
        for (int s = 0; s < steps; s += 4) {
            scales(s);
            step(s, std::integral_constant<int, 0>{});
            if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
            if (s + 2 < steps) step(s + 2, std::integral_constant<int, 2>{});
            if (s + 3 < steps) step(s + 3, std::integral_constant<int, 3>{});
        }
    } else {
        for (int s = 0; s < steps; ++s) step(s, std::integral_constant<int, 0>{});
    }
    dma_wait<0>();
    barrier_only();                                    // the stages are the epilogue's now
    constexpr int BT = MT > 4 ? MT / 2 : MT;           // row tiles of an epilogue batch
    static_assert(kWaves * BT * 4096 <= NS * kStage && MT % BT == 0, "a batch must fit the stages");
    Output<4, BT, WM * 16, GATED> o;
    o.load(a, at, row0 + wm * 16, rows - wm * 16, column(wn * 64), 0);
    epilogue<4, MT, BT, WM * 16, GATED>(a, at, lds + wave * BT * 4096, row0 + wm * 16,
                                        rows - wm * 16, column(wn * 64), acc, o);
}

// Tiles of 256 rows, bound by the matrix instructions.  Four waves of 128 x 128:
// a K step then reads 128 KB of LDS for 2048 matrix cycles of a compute unit,
// half of what its LDS can deliver (eight waves of 64 x 128 read 192 KB and,
// with the copies' 64 KB of writes, saturate it).
//
// Two stages of 64 KB fill the LDS, so what hides the copies' latency is how
// early a piece of a stage is given back: a stage is four regions (the waves'
// first and second 64 weight rows, first and second 64 x rows), each read to
// registers a little before it is multiplied and copied anew in the phase after
// that.  A phase is half a step; the reads and copies are placed among its
// matrix instructions (one wave runs on a SIMD: nothing else would fill the
// gaps), and the wait and the barrier between phases are what is left over:
//   phase   multiplies       reads (step)              copies (step)
//     A     W0 X0, W1 X0     W1 (s), X1 (s)            X0, W0 (s + 2)
//     B     W0 X1, W1 X1     X0 (s + 1), W0 (s + 1)    W1, X1 (s + 2)
// (Four phases with a barrier each measured 100 cycles more per barrier.)
// Copies behind the last step go on from an empty buffer (they write zeros), so
// that the number in flight, which the waits count, stays the same.  Channels
// that do not fill a step are one more step after the loop.
//
// 8 experts, 32768 rows: 7168 to 4096 with swiglu and checkpoint 1.54 ms (1.25
// PFLOP/s; the matrix instructions run 70 to 74% of the cycles, at the 1.6 to 1.8
// GHz that the power allows), transposed 4096 to 7168 1.48 ms (1.30), 2048 to 7168
// with bias and residual 0.86 ms (1.12: a tile takes 60 us, 45 of them its 32 steps,
// the epilogue and the first copies the rest), fp8 7168 to 4096 0.82 ms (2.3).  A
// library product of 32768 x 4096 x 7168 without an
// epilogue reaches 1.56 (bf16) and 3.2 (fp8) on the same card.
template <int IN, bool WT, bool GATED>
__global__ __launch_bounds__(256, 1) void expert_linear_wide_kernel(LinearK a) {
    constexpr bool FP8 = IN != kBf16, EXACT = IN == kFp8Exact;
    constexpr int BM = 256, kWaves = 4;
    constexpr int kRegion = 128 * 128, kStage = 4 * kRegion;     // W0, W1, X0, X1
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int BK = 128 / ES;
    __shared__ __align__(1024) uint8_t lds[2 * kStage];
    __shared__ int red[16];

    TileAt at;
    if (!find_tile<64 * kWaves>(a.seg, BM, a.col_tiles, blockIdx.x, red, &at)) return;

    const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wn = wave & 1, wm = wave >> 1;
    const int K = a.k, N = a.n;
    const int half = N >> 1;
    const int row0 = at.mt * BM;                       // in the segment
    const int rows = min(BM, at.rows - row0);
    // first column of the 64 weight rows of region t of the waves with this wn
    auto column = [&](int n, int t) {
        if (!GATED) return at.nt * kBN + n * 128 + t * 64;
        return at.nt * (kBN / 2) + n * 64 + (t ? half : 0);
    };

    const uint32_t ld_bytes = (uint32_t)K * ES;
    const uint32_t w_bytes = (uint32_t)N * ld_bytes;
    const uint32_t x_bytes = (uint32_t)rows * ld_bytes;
    ep_i32x4 xb = biased_buffer(a.x + ((int64_t)at.row0 + row0) * ld_bytes, x_bytes);
    ep_i32x4 wb = biased_buffer(a.w + (int64_t)at.e * w_bytes, w_bytes);
    // copies: a wave moves 32 rows of 128 bytes of each region, 8 at a time
    // (transposed weights: 16 k rows of 128 columns, 4 at a time)
    uint32_t woff[2][4], xoff[2][4];
    const int cs = (lane & 7) ^ (lane >> 4);           // this lane's chunk of its rows, for even j
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = wave * 32 + j * 8 + (lane >> 3);         // row of the region, 0..127
        const int ch = cs ^ ((j & 1) * 4);                     // chunk (lane & 7) ^ (r / 2 & 7)
        const uint32_t bias = kDmaBias - j * 1024;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            xoff[t][j] = (uint32_t)((r >> 6) * 128 + t * 64 + (r & 63)) * ld_bytes + ch * 16 + bias;
            if (!WT) {
                const int c = column(r >> 6, t) + (r & 63);
                woff[t][j] = c < N ? (uint32_t)c * ld_bytes + ch * 16 + bias : kOutOfRange;
            } else {
                const int kr = wave * 16 + j * 4 + (lane >> 4);
                const int g = (lane >> 1 & 7) ^ granule_of(kr);        // 16 columns each
                const int c = column(g >> 2, t) + (g & 3) * 16 + (lane & 1) * 8;
                woff[t][j] = c < N ? ((uint32_t)kr * (uint32_t)N + (uint32_t)c) * 2 + bias : kOutOfRange;
            }
        }
    }
    const uint32_t lds0 = lds_offset(lds) + wave * 4096;
    const int steps = K / BK;                          // whole steps
    const uint32_t w_step = WT ? (uint32_t)BK * (uint32_t)N * 2 : 128;
    uint32_t xs_off = 0, ws_off = 0;                   // where the region being copied begins
    auto copy_w = [&](int s, int stage, int t, auto j) {
        constexpr int J = decltype(j)::value;
        if (J == 0) range_of(s, steps, w_bytes + kDmaBias, s * w_step, wb, &ws_off);
        dma16_of4<J>(wb, lds0 + stage * kStage + t * kRegion, woff[t][J], ws_off);
    };
    auto copy_x = [&](int s, int stage, int t, auto j) {
        constexpr int J = decltype(j)::value;
        if (J == 0) range_of(s, steps, x_bytes + kDmaBias, s * 128, xb, &xs_off);
        dma16_of4<J>(xb, lds0 + stage * kStage + (2 + t) * kRegion, xoff[t][J], xs_off);
    };

    // LDS addresses of this lane's operands, by stage and half
    const int slot = l16 * 128 + (q ^ (l16 >> 1)) * 16;
    const uint8_t *xat[2][2], *wat[2][2];
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            xat[st][h] = lds + st * kStage + 2 * kRegion + wm * 8192 + (slot ^ (h * 64));
            wat[st][h] = lds + st * kStage + wn * 8192 + (slot ^ (h * 64));
        }
    ep_u32x4 wf[2][4][2], xf[2][4][2];                 // [region][tile][half]
    auto read_w = [&](int stage, int t, int i) {       // one tile
#pragma unroll
        for (int h = 0; h < 2; ++h)
            wf[t][i][h] = WT ? transposed_operand<256>(lds + stage * kStage + t * kRegion, wn * 4 + i, h)
                             : *(const ep_u32x4 *)(wat[stage][h] + t * kRegion + i * 2048);
    };
    auto read_x = [&](int stage, int t, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            xf[t][i][h] = *(const ep_u32x4 *)(xat[stage][h] + t * kRegion + i * 2048);
    };

    ep_f32x4 acc[8][8];                                // [4 region + tile] of weights, of x
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t][i] = ep_f32x4{0, 0, 0, 0};
    // fp8: scale bytes of four steps.  (Copied to LDS byte by byte with the
    // operands, without a wait of their own, they took 912 us where these take
    // 825: 64 lines a copy keep the address unit busy.)
    int xs[8], ws[8];
    auto scales = [&](int s) {
        const int groups = K / kFp8Group;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = min(wm * 128 + i * 16 + l16, rows - 1);
            xs[i] = scales4(a.x_scales + ((int64_t)at.row0 + row0 + r) * groups, s, groups);
            const int c = min(column(wn, i >> 2) + (i & 3) * 16 + l16, N - 1);
            ws[i] = scales4(a.w_scales + ((int64_t)at.e * N + c) * groups, s, groups);
        }
    };
    // Half a phase: `read(i)` and `copy(i)`, i = 0..3, among the matrix instructions.
    auto part = [&](int tw, int tx, auto sb, auto read, auto copy) {
        constexpr int n = EXACT ? 64 : FP8 ? 16 : 32, SB = decltype(sb)::value;
        // exact: a piece of the four x tiles and of one weight tile, and the next
        // ones, converted while the matrix instructions run
        ep_u32x4 xp[2][4], wp[2];
        float sx[4], sw[4];
        if constexpr (EXACT) {
            each<4>([&](auto i) __attribute__((always_inline)) {
                sx[i] = scale_byte<SB>(xs[tx * 4 + i]);
                sw[i] = scale_byte<SB>(ws[tw * 4 + i]);
                // every part converts anew: kept for the other parts, the pieces
                // would push the copies' offsets out of the registers
                asm volatile("" : "+v"(sx[i]), "+v"(sw[i]));
                xp[0][i] = piece_of<0>(xf[tx][i], sx[i]);
            });
            wp[0] = piece_of<0>(wf[tw][0], sw[0]);
        }
        each<n>([&](auto mm) __attribute__((always_inline)) {
            constexpr int m = decltype(mm)::value;
            constexpr int h = m / 16, b = m / 4 % 4, c = m % 4;
            ep_f32x4 &d = acc[tw * 4 + b][tx * 4 + c];
            if constexpr (EXACT) {
                constexpr int next = m / 4 + 1;            // weight tile next % 4, piece next / 4
                d = mfma_bf16(wp[b & 1], xp[h & 1][c], d);
                if constexpr (c == 0 && next < 16) wp[next & 1] = piece_of<next / 4>(wf[tw][next % 4], sw[next % 4]);
                if constexpr (b == 1 && h < 3) xp[~h & 1][c] = piece_of<h + 1>(xf[tx][c], sx[c]);
            } else if constexpr (FP8) {
                d = mfma_fp8<SB>(wf[tw][b], xf[tx][c], d, ws[tw * 4 + b], xs[tx * 4 + c]);
            } else {
                d = mfma_bf16(wf[tw][b][h], xf[tx][c][h], d);
            }
            if constexpr (m % (n / 4) == 0) read(m / (n / 4));
            if constexpr (m % (n / 4) == n / 8) copy(std::integral_constant<int, m / (n / 4)>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // end of a phase: the regions the next one reads have landed (the copies of
    // the phase before and of this one, 8 each, may be in flight), and every wave
    // has read those this phase read
    auto turn = [&]() {
        dma_wait<16>();
        barrier_only();
        __builtin_amdgcn_sched_barrier(0);
    };

    Output<8, 4, 16, GATED> o;
    if (!EXACT) o.load(a, at, row0 + wm * 128, rows - wm * 128, column(wn, 0), 0);
    for (int s = 0; s < 2; ++s) {
        each<4>([&](auto j) { copy_x(s, s, 0, j); });
        each<4>([&](auto j) { copy_w(s, s, 0, j); });
        each<4>([&](auto j) { copy_w(s, s, 1, j); });
        each<4>([&](auto j) { copy_x(s, s, 1, j); });
    }
    dma_wait<24>();
    barrier_only();
    each<4>([&](auto i) { read_x(0, 0, i); });
    each<4>([&](auto i) { read_w(0, 0, i); });
    turn();

    auto step = [&](int s, auto stage, auto sb) {
        constexpr int st = decltype(stage)::value;
        part(0, 0, sb, [&](int i) { read_w(st, 1, i); }, [&](auto j) { copy_x(s + 2, st, 0, j); });
        part(1, 0, sb, [&](int i) { read_x(st, 1, i); }, [&](auto j) { copy_w(s + 2, st, 0, j); });
        turn();
        part(0, 1, sb, [&](int i) { read_x(st ^ 1, 0, i); }, [&](auto j) { copy_w(s + 2, st, 1, j); });
        part(1, 1, sb, [&](int i) { read_w(st ^ 1, 0, i); }, [&](auto j) { copy_x(s + 2, st, 1, j); });
        turn();
    };
    constexpr std::integral_constant<int, 0> c0{};
    constexpr std::integral_constant<int, 1> c1{};
    if (FP8) {
        for (int s = 0; s < steps; s += 4) {
            scales(s);
            step(s, c0, c0);
            if (s + 1 < steps) step(s + 1, c1, c1);
            if (s + 2 < steps) step(s + 2, c0, std::integral_constant<int, 2>{});
            if (s + 3 < steps) step(s + 3, c1, std::integral_constant<int, 3>{});
        }
    } else {
        for (int s = 0; s < steps; s += 2) {
            step(s, c0, c0);
            if (s + 1 < steps) step(s + 1, c1, c0);
        }
    }
    // no copy may still be on its way to this workgroup's LDS when it ends, or
    // when the rest of the channels takes stage 0
    dma_wait<0>();
    if (!FP8 && K > steps * BK) {
        barrier_only();
        const int left = K - steps * BK;
        each<2>([&](auto tt) {
            constexpr int t = decltype(tt)::value;
            each<4>([&](auto jj) {
                constexpr int J = decltype(jj)::value;
                const uint32_t past = (cs ^ ((J & 1) * 4)) * 8 >= left ? kOutOfRange : 0;
                if (J == 0) range_of(0, 1, x_bytes + kDmaBias, steps * 128, xb, &xs_off);
                dma16_of4<J>(xb, lds0 + (2 + t) * kRegion, xoff[t][J] | past, xs_off);
            });
            each<4>([&](auto jj) {
                constexpr int J = decltype(jj)::value;
                const uint32_t past = !WT && (cs ^ ((J & 1) * 4)) * 8 >= left ? kOutOfRange : 0;
                if (J == 0) range_of(0, 1, w_bytes + kDmaBias, steps * w_step, wb, &ws_off);
                dma16_of4<J>(wb, lds0 + t * kRegion, woff[t][J] | past, ws_off);
            });
        });
        dma_wait<0>();
        barrier_only();
        each<2>([&](auto t) { each<4>([&](auto i) { read_x(0, t, i); read_w(0, t, i); }); });
        each<2>([&](auto tw) { each<2>([&](auto tx) { each<32>([&](auto mm) {
            constexpr int m = decltype(mm)::value, h = m / 16, b = m / 4 % 4, c = m % 4;
            ep_f32x4 &d = acc[decltype(tw)::value * 4 + b][decltype(tx)::value * 4 + c];
            d = mfma_bf16(wf[decltype(tw)::value][b][h], xf[decltype(tx)::value][c][h], d);
        }); }); });
        dma_wait<0>();
    }
    barrier_only();                                    // the stages are the epilogue's now
    // exact: the registers for it hold the converted pieces until here
    if (EXACT) o.load(a, at, row0 + wm * 128, rows - wm * 128, column(wn, 0), 0);
    static_assert(kWaves * 32768 <= 2 * kStage, "a batch must fit the stages");
    epilogue<8, 8, 4, 16, GATED>(a, at, lds + wave * 32768, row0 + wm * 128, rows - wm * 128,
                             column(wn, 0), acc, o);
}

// Workgroups for row tiles of BM rows: each segment's last one may be partial.
int64_t grid_of(const LinearArgs &a, const LinearK &k, int BM) {
    const int64_t most = a.seg.pairs < a.seg.num_rows ? a.seg.pairs : a.seg.num_rows;
    const int64_t some = most < a.seg.E ? most : a.seg.E;
    return ((most / BM + some) * k.col_tiles + 7) / 8 * 8;
}

hipError_t launch_wide(const LinearArgs &a, const LinearK &k, bool gated, hipStream_t stream) {
    const int64_t grid = grid_of(a, k, 256);
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(256);
    if (a.fp8 && a.ckpt) {
        if (gated) expert_linear_wide_kernel<kFp8Exact, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_wide_kernel<kFp8Exact, false, false><<<g, t, 0, stream>>>(k);
    } else if (a.fp8) {
        if (gated) expert_linear_wide_kernel<kFp8, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_wide_kernel<kFp8, false, false><<<g, t, 0, stream>>>(k);
    } else if (a.transposed) {
        if (gated) expert_linear_wide_kernel<kBf16, true, true><<<g, t, 0, stream>>>(k);
        else expert_linear_wide_kernel<kBf16, true, false><<<g, t, 0, stream>>>(k);
    } else {
        if (gated) expert_linear_wide_kernel<kBf16, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_wide_kernel<kBf16, false, false><<<g, t, 0, stream>>>(k);
    }
    return hipGetLastError();
}

template <int BM, int WM, int WN, int NS>
hipError_t launch_bm(const LinearArgs &a, const LinearK &k, bool gated, hipStream_t stream) {
    const int64_t grid = grid_of(a, k, BM);
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(64 * WN * WM);
    if (a.fp8 && a.ckpt) {
        if (gated) expert_linear_kernel<BM, WM, WN, NS, kFp8Exact, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_kernel<BM, WM, WN, NS, kFp8Exact, false, false><<<g, t, 0, stream>>>(k);
    } else if (a.fp8) {
        if (gated) expert_linear_kernel<BM, WM, WN, NS, kFp8, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_kernel<BM, WM, WN, NS, kFp8, false, false><<<g, t, 0, stream>>>(k);
    } else if (a.transposed) {
        if constexpr (WN == 4) {
            if (gated) expert_linear_kernel<BM, WM, WN, NS, kBf16, true, true><<<g, t, 0, stream>>>(k);
            else expert_linear_kernel<BM, WM, WN, NS, kBf16, true, false><<<g, t, 0, stream>>>(k);
        }
    } else {
        if (gated) expert_linear_kernel<BM, WM, WN, NS, kBf16, false, true><<<g, t, 0, stream>>>(k);
        else expert_linear_kernel<BM, WM, WN, NS, kBf16, false, false><<<g, t, 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_linear(const LinearArgs &a, hipStream_t stream) {
    LinearK k = {};
    k.seg = a.seg;
    k.x = (const uint8_t *)a.x;
    k.x_scales = a.x_scales;
    k.w = (const uint8_t *)a.w;
    k.w_scales = a.w_scales;
    k.bias = (const uint16_t *)a.bias;
    k.residual = (const uint16_t *)a.residual;
    k.out = (uint16_t *)a.out;
    k.ckpt = a.ckpt;
    k.ckpt_scales = a.ckpt_scales;
    k.n = a.n;
    k.k = a.k;
    const bool gated = act_gated(a.act);
    k.m = gated ? a.n / 2 : a.n;
    k.kind = act_kind(a.act);
    const int per_tile = gated ? kBN / 2 : kBN;
    k.col_tiles = (k.m + per_tile - 1) / per_tile;
    // Row tiles by the rows an expert can expect (up to 256 experts of 7168 x 4096,
    // uniform routing).  Up to about 112 the weights' reads decide, and the deep
    // ring of the 128-row tile reads them in 2.4 ms (16 rows, 6.3 TB/s) to 2.8 ms
    // (110 rows, 5.5); around 128 half of the experts need a second 128-row tile,
    // where one of 192 rows and two stages does (3.14 against 3.26 ms; 2.95 against 2.50 ms at 64 rows); from 160
    // rows on the matrix instructions decide and the 256-row tile is the faster.  (The
    // rule does not count tiles: with fewer of them than compute units, as of 4
    // experts of 7168 x 4096 with 256 rows each, some stay idle: 126 us, of which
    // reading the weights is 40.)
    const int64_t avg = a.seg.pairs / a.seg.E;
    // A step of a small tile takes a workgroup hardly less time than one of a large
    // tile (0.3 against 0.4 to 1 us: LDS reads and a barrier's round trip), so while
    // the 64 x 64 tiles all run at once, two on a compute unit, they are the faster:
    // 16 experts of 7168 x 256, bf16, 1024 rows 80 and 41 us, 4096 rows 118 and 46
    // us; with twice as many tiles they lose (4 experts of 7168 x 4096, 1024 rows,
    // 127 and 151 us).
    if (!a.transposed) {
        const int per_small = gated ? 32 : 64;
        const int64_t cols = (k.m + per_small - 1) / per_small;
        const int64_t live = std::max<int64_t>(1, std::min<int64_t>(a.seg.pairs, a.seg.E));
        if (live * ((a.seg.pairs / live + 63) / 64) * cols <= 512) {
            k.col_tiles = (int)cols;
            return launch_bm<64, 4, 1, 4>(a, k, gated, stream);
        }
    }
    if (avg > 160) return launch_wide(a, k, gated, stream);
    if (avg > 112) return launch_bm<192, 2, 4, 2>(a, k, gated, stream);
    return launch_bm<128, 2, 4, 3>(a, k, gated, stream);
}

}  // namespace ep
