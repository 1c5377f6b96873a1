// Product of e4m3 rows, one fp32 scale per 128 channels, with e4m3 weights, one per
// 128 x 128 block, and its epilogue:
//   z[r, c] = sum_b sx[r, b] sw[c / 128, b] sum_(k in b) x[r, k] w[c, k]
//   out[r] = act(z[r] + bias[e]) + residual[r]        (rows r of segment e, or dense)
//
// The fp8 matrix instruction takes powers of two as scales, these are any fp32
// numbers.  One instruction of 16 x 16 x 128 sums one block of the contraction, so
// its result, begun at zero, is multiplied by the two scales and added to the fp32
// sums by ordinary instructions: four for the four values of a lane.  (Held in
// units of the latest scales instead, the sums would take as many.)  They run
// beside the matrix instructions of the other wave of the SIMD, and the sums have to
// lie in ordinary registers, so eight waves of 64 columns x 128 rows share a tile of
// 256 x 256, not four of 128 x 128.
//
// 8 experts of 4000 or 4096 rows each, 7168 to 4096 with swiglu, 0.88 ms (2.1 to 2.2
// PFLOP/s; one matrix for 32768 dense rows 0.82, 2.35), 2048 to 7168 0.53 to 0.54 (1.8;
// dense 0.48, 2.0).  A round of 256 tiles takes 106 to 111 and 36 to 38 us, and a partial
// one as long as a full one: with one row more than 4096 an expert 0.96 and 0.56 ms.  The
// matrix instructions run in 52% and 42% of the cycles; without the scales' instructions
// the dense product took 0.68 to 0.77 ms.
//
// The weights are the instruction's first operand: a lane's values are consecutive
// columns of one row, with one row scale, and a wave's 64 columns lie in one block
// of the weights (gated: 32 gate and 32 up columns in one each).
//
// Scales of four steps are copied to LDS with the operands of the first of them, in
// two buffers: ordinary loads would make the compiler wait for the copies in flight.
#include "ep_linear_device.h"

namespace ep {

namespace {

struct BlockK {
    LinearK l;
    const float *xs;       // [num_rows, k/128]
    const float *ws;       // [E, ceil(n/128), k/128]
};

template <int BM, int WM, int WN, int NS, bool GATED, int MODE = kPlain>
__global__ __launch_bounds__(64 * WN * WM, 2) void block_linear_kernel(BlockK p) {
    constexpr int kWaves = WN * WM;
    constexpr int BN = 64 * WN;
    constexpr int MT = BM / WM / 16;                   // 16-row tiles of a wave
    constexpr int kWStage = BN * 128, kXStage = BM * 128;
    constexpr int kStage = kWStage + kXStage;
    constexpr int WL = kWStage / 1024 / kWaves;        // copies of a wave per step
    constexpr int XL = kXStage / 1024 / kWaves;
    constexpr int SL = (BM / 16 + kWaves - 1) / kWaves;    // and of row scales, per four steps
    constexpr int kXScales = SL * kWaves * 256, kScales = kXScales + kWaves * 256;
    __shared__ __align__(1024) uint8_t lds[NS * kStage + 2 * kScales];
    __shared__ int red[16];
    const LinearK &a = p.l;
    uint8_t *const slds = lds + NS * kStage;

    TileAt at;
    if (!find_tile<64 * kWaves>(a.seg, BM, a.col_tiles, blockIdx.x, red, &at)) return;

    const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    const int K = a.k, N = a.n;
    const int half = N >> 1;
    const int row0 = at.mt * BM;                       // in the segment
    const int rows = min(BM, at.rows - row0);
    const int groups = K / kFp8Group;

    const uint32_t x_bytes = (uint32_t)rows * K;
    ep_i32x4 xb = buffer_of(a.x + ((int64_t)at.row0 + row0) * K, x_bytes);
    const uint32_t w_bytes = (uint32_t)N * K;
    ep_i32x4 wb = buffer_of(a.w + (int64_t)at.e * w_bytes, w_bytes);
    const int wblocks = (N + kFp8Group - 1) / kFp8Group;
    const ep_i32x4 xsb = buffer_of(p.xs + ((int64_t)at.row0 + row0) * groups, (uint32_t)(rows * groups) * 4);
    const ep_i32x4 wsb = buffer_of(p.ws + (int64_t)at.e * wblocks * groups, (uint32_t)(wblocks * groups) * 4);
    // column of z at place r of the tile: gated tiles hold, per wave, 32 gate
    // columns and the 32 up columns that go with them
    auto column = [&](int r) {
        if (!GATED) return at.nt * BN + r;
        const int c = at.nt * (BN / 2) + (r >> 6) * 32 + (r & 31);
        return (r & 32) ? half + c : c;
    };
    const int chunk = (lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7);
    uint32_t xoff[XL], woff[WL];
    for (int j = 0; j < XL; ++j) xoff[j] = (uint32_t)((j * kWaves + wave) * 8 + (lane >> 3)) * K + chunk * 16;
    for (int j = 0; j < WL; ++j) {
        const int c = column((j * kWaves + wave) * 8 + (lane >> 3));
        woff[j] = c < N ? (uint32_t)c * K + chunk * 16 : kOutOfRange;
    }
    // scales: lane l copies step l % 4 of row l / 4 (of this wave's weight blocks,
    // the gates' or only one and the ups')
    const int sk = lane & 3;
    uint32_t soff[SL], wsoff = kOutOfRange;
    for (int j = 0; j < SL; ++j) soff[j] = (uint32_t)(((j * kWaves + wave) * 16 + (lane >> 2)) * groups + sk) * 4;
    if (lane < 8) {
        const int c = column(wn * 64 + (lane >> 2) * 32);
        if (c < N) wsoff = (uint32_t)(c / kFp8Group * groups + sk) * 4;
    }
    const uint32_t lds0 = lds_offset(lds), slds0 = lds0 + NS * kStage;
    const int begin = MODE == kSums ? blockIdx.y * a.split : 0;
    const int steps = MODE == kSums ? min(groups, begin + a.split) : groups;
    // The scales of the group of four steps that begins with step s (kSums: the rest of
    // the group that the part begins in).
    auto copy_scales = [&](int s) __attribute__((always_inline)) {
        if ((s & 3) == 0 || (MODE == kSums && s == begin)) {
            const uint32_t base = slds0 + (s >> 2 & 1) * kScales + wave * 256;
            const int s4 = s & ~3;
            // (all in the lane's offset, see dma4: a group behind the last one may
            // begin past the whole buffer)
            const uint32_t past = s4 + sk >= groups ? kOutOfRange : 0;
            for (int i = 0; i < SL; ++i) dma4(xsb, base + i * kWaves * 256, (soff[i] + s4 * 4) | past);
            dma4(wsb, base + kXScales, (wsoff + s4 * 4) | past);
        }
    };
    // Copies behind the last step go on from empty buffers (they write zeros), so that
    // the number in flight, which the waits count, stays the same.
    uint32_t ws_off = 0, xs_off = 0;
    auto copy_w = [&](int s, int stage, int j) __attribute__((always_inline)) {
        if (j == 0) range_of(s, steps, w_bytes, s * 128, wb, &ws_off);
        dma16(wb, lds0 + stage * kStage + (j * kWaves + wave) * 1024, woff[j], ws_off);
    };
    auto copy_x = [&](int s, int stage, int j) __attribute__((always_inline)) {
        if (j == 0) range_of(s, steps, x_bytes, s * 128, xb, &xs_off);
        dma16(xb, lds0 + stage * kStage + kWStage + (j * kWaves + wave) * 1024, xoff[j], xs_off);
    };

    ep_f32x4 acc[4][MT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = ep_f32x4{0, 0, 0, 0};

    // A step multiplies its row tiles in turn, each by the four weight tiles, the last
    // two together.  When their operands are in registers, nothing more is read of the
    // stage: the wait for the next one and the barrier stand there, and the rows' copies
    // for step s + NS and the first reads of the next step go among the last products,
    // the weights' copies among the first ones of the next step, so that the matrix
    // instructions run on across the steps.  (A compute unit takes 16 cycles for the
    // addresses of each copy: all 64 of a step behind the barrier held the waves up, 3400
    // cycles a step where these take 2930, 2048 of them matrix instructions.)
    constexpr int kLast = MT >= 2 ? 2 : 1;             // row tiles behind the barrier
    constexpr int kFirst = 4 * (MT - kLast);           // products before it
    constexpr int kSlots = MT == 4 ? 4 : 3;            // x tiles in registers
    // (The last two lie in slots 0 and 1, or 2 and 3 of four; tile 0 not in the second's.)
    auto slot_of = [](int i) constexpr { return MT == 4 ? i : (i + 24 - (MT - kLast)) % 3; };
    auto row_of = [](int n) constexpr {
        return n < kFirst ? n / 4 : kLast == 1 ? 0 : MT - 2 + (0xCA >> (n - kFirst) & 1);
    };
    auto col_of = [](int n) constexpr {
        return n < kFirst || kLast == 1 ? n % 4 : (int)(0x32321100u >> (4 * (n - kFirst)) & 3);
    };
    const int place = l16 * 128 + (q ^ (l16 >> 1)) * 16;
    ep_u32x4 wf[4][2], xf[kSlots][2];
    float sx[kSlots], sw[2];
    auto read_w = [&](int stage, int t) __attribute__((always_inline)) {
        const uint8_t *p = lds + stage * kStage + (wn * 4 + t) * 2048;
#pragma unroll
        for (int h = 0; h < 2; ++h) wf[t][h] = *(const ep_u32x4 *)(p + (place ^ (h * 64)));
    };
    auto read_x = [&](int stage, int i) __attribute__((always_inline)) {
        const uint8_t *p = lds + stage * kStage + kWStage + (i * WM + wm) * 2048;
#pragma unroll
        for (int h = 0; h < 2; ++h) xf[slot_of(i)][h] = *(const ep_u32x4 *)(p + (place ^ (h * 64)));
    };
    auto scale_at = [&](int s, int offset) __attribute__((always_inline)) {
        return *(const float *)(slds + (s >> 2 & 1) * kScales + (s & 3) * 4 + offset);
    };
    auto x_scale = [&](int s, int i) { return scale_at(s, ((i * WM + wm) * 16 + l16) * 16); };
    auto w_scale = [&](int s, int g) { return scale_at(s, kXScales + wave * 256 + (GATED ? g * 16 : 0)); };
    // all but the newest copies have landed: those of the `ahead` steps behind step s
    auto landed = [&](int s, auto nn) {
        constexpr int ahead = decltype(nn)::value;
        bool scales = false;                           // those of a group of four among them
        for (int j = 1; j <= ahead; ++j) scales |= ((s + j) & 3) == 0;
        if (scales) dma_wait<ahead * (WL + XL) + SL + 1>();
        else dma_wait<ahead * (WL + XL)>();
        barrier_only();
    };

    // (the weights of the last stage are copied in the first step)
    for (int s = 0; s < NS; ++s) {
        if (kFirst == 0 || s < NS - 1)
            for (int j = 0; j < WL; ++j) copy_w(begin + s, s, j);
        copy_scales(begin + s);
        for (int j = 0; j < XL; ++j) copy_x(begin + s, s, j);
    }
    dma_wait<0>();
    barrier_only();
    read_x(0, 0);
    if (MT == 2) read_x(0, 1);
#pragma unroll
    for (int t = 0; t < 4; ++t) read_w(0, t);
    sx[slot_of(0)] = x_scale(begin, 0);
    sw[0] = w_scale(begin, 0);
    sw[1] = w_scale(begin, 1);
    int stage = 0;
    for (int s = begin; s < steps; ++s) {
        const int next = stage + 1 == NS ? 0 : stage + 1, before = stage == 0 ? NS - 1 : stage - 1;
        float sx_next = 0.0f, sw_next[2] = {0.0f, 0.0f};
        if (MT == 2) sx[slot_of(1)] = x_scale(s, 1);
        // a product is added to the sums two products later
        ep_f32x4 part[3];
        auto add = [&](auto nn) __attribute__((always_inline)) {
            constexpr int n = decltype(nn)::value, i = row_of(n), t = col_of(n);
            const float f = sx[slot_of(i)] * sw[t >> 1];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][i][j] = __builtin_fmaf(part[n % 3][j], f, acc[t][i][j]);
            pin(acc[t][i]);    // (the compiler would put all of them behind the products)
        };
        each<4 * MT>([&](auto nn) __attribute__((always_inline)) {
            constexpr int n = decltype(nn)::value, i = row_of(n), t = col_of(n);
            if constexpr (n == kFirst) {
                landed(s + 1, std::integral_constant<int, NS - 2>{});
                copy_scales(s + NS);
                __builtin_amdgcn_sched_barrier(0);
            }
            part[n % 3] = mfma_fp8_plain(wf[t], xf[slot_of(i)], ep_f32x4{0, 0, 0, 0});
            if constexpr (n < kFirst) {
                constexpr int kEvery = kFirst >= 16 ? 3 : 1;
                if constexpr (n % kEvery == 0 && n / kEvery < WL) copy_w(s + NS - 1, before, n / kEvery);
                // the next tile's operands (and, before the barrier, the one's after it)
                if constexpr (t == 0) {
                    read_x(stage, i + 1);
                    sx[slot_of(i + 1)] = x_scale(s, i + 1);
                }
                if constexpr (t == 2 && i == MT - 3) {
                    read_x(stage, MT - 1);
                    sx[slot_of(MT - 1)] = x_scale(s, MT - 1);
                }
            } else {
                constexpr int m = n - kFirst, kEvery = 4 * kLast / XL;
                if constexpr (kFirst == 0 && m == 0)
                    for (int j = 0; j < WL; ++j) copy_w(s + NS, stage, j);
                if constexpr (m % kEvery == 0 && m / kEvery < XL) copy_x(s + NS, stage, m / kEvery);
                if constexpr (i == MT - 1) read_w(next, t);         // the tile's last product
                if constexpr (m == (kLast == 2 ? 5 : 3)) {
                    read_x(next, 0);
                    sx_next = x_scale(s + 1, 0);
                    sw_next[0] = w_scale(s + 1, 0);
                    sw_next[1] = w_scale(s + 1, 1);
                }
            }
            if constexpr (n >= 2) add(std::integral_constant<int, n - 2>{});
            __builtin_amdgcn_sched_barrier(0);
        });
        if (MT == 2) read_x(next, 1);
        add(std::integral_constant<int, 4 * MT - 2>{});
        add(std::integral_constant<int, 4 * MT - 1>{});
        sx[slot_of(0)] = sx_next;
        sw[0] = sw_next[0];
        sw[1] = sw_next[1];
        stage = next;
    }
    dma_wait<0>();
    if constexpr (MODE == kSums) {
        store_sums<GATED, 4, MT>(a, blockIdx.y, row0 + wm * 16, WM * 16, rows - wm * 16, acc,
                                 [&](int t) { return column(wn * 64 + t * 16); });
        return;
    }
    barrier_only();                                    // the stages are the epilogue's now
    constexpr int BT = MT > 4 ? MT / 2 : MT;           // row tiles of an epilogue batch
    static_assert(kWaves * BT * 4096 <= NS * kStage && MT % BT == 0, "a batch must fit the stages");
    static_assert(NS <= 4, "a group's scales are read before the copies of the group after the next");
    Output<4, BT, WM * 16, GATED> o;
    o.load(a, at, row0 + wm * 16, rows - wm * 16, column(wn * 64), 0);
    epilogue<4, MT, BT, WM * 16, GATED, kPlain>(a, at, lds + wave * BT * 4096, row0 + wm * 16,
                                                rows - wm * 16, column(wn * 64), acc, o);
}

template <int BM, int WM, int WN, int NS, int MODE = kPlain>
hipError_t launch_tiles(BlockK &k, bool gated, int parts, hipStream_t stream) {
    const int per = gated ? WN * 32 : WN * 64;
    k.l.col_tiles = (k.l.m + per - 1) / per;
    const int64_t grid = grid_of(k.l.seg, k.l.col_tiles, BM);
    if (!launchable(grid, 64 * WN * WM)) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid, parts), t(64 * WN * WM);
    if (gated) block_linear_kernel<BM, WM, WN, NS, true, MODE><<<g, t, 0, stream>>>(k);
    else block_linear_kernel<BM, WM, WN, NS, false, MODE><<<g, t, 0, stream>>>(k);
    return hipGetLastError();
}

DensePlan plan_of(int64_t rows, int n, int k) { return dense_plan(rows, n, k / kFp8Group, false); }

hipError_t launch_dense(BlockK &k, bool gated, hipStream_t stream) {
    const DensePlan p = plan_of(k.l.seg.num_rows, k.l.n, k.l.k);
    if (p.rows == 256) return launch_tiles<256, 2, 4, 2>(k, gated, 1, stream);
    if (p.parts == 1 && p.cols == 64) return launch_tiles<64, 4, 1, 4>(k, gated, 1, stream);
    if (p.parts == 1)
        return p.rows == 128 ? launch_tiles<128, 2, 2, 2>(k, gated, 1, stream)
                             : launch_tiles<64, 2, 2, 3>(k, gated, 1, stream);
    k.l.split = p.split;
    const hipError_t rc = p.cols == 64 ? launch_tiles<64, 4, 1, 4, kSums>(k, gated, p.parts, stream)
                          : p.rows == 128 ? launch_tiles<128, 2, 2, 2, kSums>(k, gated, p.parts, stream)
                                          : launch_tiles<64, 2, 2, 3, kSums>(k, gated, p.parts, stream);
    if (rc != hipSuccess) return rc;
    return gated ? launch_finish<kPlain, true>(k.l, p.parts, stream)
                 : launch_finish<kPlain, false>(k.l, p.parts, stream);
}

}  // namespace

size_t block_linear_sums_bytes(int64_t rows, int n, int k) {
    return few_rows(rows, k) ? 0 : sums_bytes(plan_of(rows, n, k), rows, n);
}

size_t block_linear_sums_most(int64_t rows, int n, int k) {
    return few_rows(rows, k) ? 0 : sums_most(rows, n, k / kFp8Group);
}

hipError_t launch_block_linear(const BlockLinearArgs &a, hipStream_t stream) {
    if (!a.seg.offsets && few_rows(a.seg.num_rows, a.k)) {
        FewRowsArgs f = {};
        f.x = a.x;
        f.x_scales = a.x_scales;
        f.w = a.w;
        f.w_scales = a.w_scales;
        f.bias = a.bias;
        f.residual = a.residual;
        f.out = a.out;
        f.rows = (int)a.seg.num_rows;
        f.n = a.n;
        f.k = a.k;
        f.act = a.act;
        return launch_few_rows(f, stream);
    }
    BlockK k = {};
    k.l.seg = a.seg;
    k.l.x = (const uint8_t *)a.x;
    k.l.w = (const uint8_t *)a.w;
    k.l.bias = (const uint16_t *)a.bias;
    k.l.residual = (const uint16_t *)a.residual;
    k.l.out = (uint16_t *)a.out;
    k.l.n = a.n;
    k.l.k = a.k;
    k.xs = a.x_scales;
    k.ws = a.w_scales;
    const bool gated = act_gated(a.act);
    k.l.m = gated ? a.n / 2 : a.n;
    k.l.kind = act_kind(a.act);
    k.l.sums = a.sums;
    if (!a.seg.offsets) return launch_dense(k, gated, stream);
    // Small products as the experts' other ones.  Then by the rows an expert can expect:
    // 64 experts of 7168 x 4096, 128 rows each, uniform routing, 430 us in tiles of 128,
    // 441 of 192, 467 of 256 rows; 144 rows 512, 450, 473; 176 rows 487 of 256 rows.
    const RowTile tile = row_tile(a.seg, k.l.m, gated, false);
    if (tile.rows == 64) return launch_tiles<64, 4, 1, 4>(k, gated, 1, stream);
    const int64_t avg = a.seg.pairs / a.seg.E;
    if (avg <= 136) return launch_tiles<128, 2, 4, 3>(k, gated, 1, stream);
    if (avg <= 168) return launch_tiles<192, 2, 4, 2>(k, gated, 1, stream);
    return launch_tiles<256, 2, 4, 2>(k, gated, 1, stream);
}

}  // namespace ep
