// Weight gradient over the receive segments: dW[e] = dy^T x over the rows of
// segment e, and the bias gradient, the column sums of dy.
//
// Both operands lie with the summed index (the row) outermost, so both are
// staged as they lie, 64 rows a step, and read by the transposing LDS read (see
// granule_of).  The last step's missing rows are zeros (reads past the buffer's
// end).  x is the matrix instruction's first operand: a lane's four accumulators
// are four consecutive channels of one dW row.
//
// fp8 rows of x (kept in 8 bits by the forward pass) become bf16 on the way:
// exact, the scales are powers of two.
#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kRows = 64;        // rows per step

struct WgradK {
    SegmentRows seg;
    const uint8_t *dy;
    const uint8_t *x;
    const uint8_t *x_scales;
    const void *dw_in;
    const float *db_in;
    void *dw;
    float *db;
    int n, k;
    int tiles_n, tiles_k;
    int bf16_out;
};

// The tile (of edge T, the tile grid tiles_n x tiles_k per expert) of a
// workgroup.  Runs of 32 tiles (8 x 4 of them where the grid has them) go to one
// XCD, the runs to the XCDs in turn: the operands of a run meet in one L2, and
// an expert with more rows than others spreads over all XCDs.
__device__ __forceinline__ bool tile_of(const WgradK &a, int T, int *e, int *n0, int *k0) {
    const int j = blockIdx.x >> 3;
    const uint32_t t = ((uint32_t)(j >> 5) * 8 + (blockIdx.x & 7)) * 32 + (j & 31);
    const uint32_t per_e = (uint32_t)a.tiles_n * (uint32_t)a.tiles_k;
    *e = (int)(t / per_e);
    if (*e >= a.seg.E) return false;
    const int lt = (int)(t - (uint32_t)*e * per_e);
    const int g = lt / (8 * a.tiles_k);
    const int gm = min(8, a.tiles_n - g * 8);
    const int rem = lt - g * 8 * a.tiles_k;
    *n0 = (g * 8 + rem % gm) * T;
    *k0 = (rem / gm) * T;
    return true;
}

typedef __amdgpu_buffer_rsrc_t Buffer;

// A wave's NT x KT accumulator tiles: tile (t, i) holds dW rows n0 + 16 i +
// lane % 16, channels k0 + 16 t + 4 q .. + 3.  Row tile by row tile, what is
// added to the next one loaded while this one is stored; buffer accesses, so
// rows and channels that are not there need no branch.
template <bool BF16, int KT, int NT>
__device__ __forceinline__ void write_tiles_as(const WgradK &a, int e, int n0, int k0,
                                               ep_f32x4 (*acc)[NT]) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    constexpr int ES = BF16 ? 2 : 4;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int rows = max(0, min(NT * 16, a.n - n0));
    const int64_t from = ((int64_t)e * a.n + n0) * a.k * ES;
    const int bytes = wave_uniform(rows * a.k * ES);
    const Buffer out = __builtin_amdgcn_make_buffer_rsrc((uint8_t *)a.dw + from, 0, bytes, 0x00020000);
    const Buffer in = __builtin_amdgcn_make_buffer_rsrc((uint8_t *)a.dw_in + from, 0, a.dw_in ? bytes : 0, 0x00020000);
    const uint32_t at = ((uint32_t)l16 * a.k + k0 + 4 * q) * ES;
    const uint32_t step = 16 * (uint32_t)a.k * ES;
    // (everything in the lane's offset: the range check subtracts a scalar one
    // from the size, which rows that are not there would make negative)
    auto off = [&](int i, int t) { return k0 + t * 16 + 4 * q < a.k ? at + i * step + t * 16 * ES : kOutOfRange; };
    ep_f32x4 add[2][KT];
    auto load = [&](int i) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            ep_f32x4 &v = add[i & 1][t];
            if (BF16) {
                const ep_u32x2 o = __builtin_bit_cast(ep_u32x2, __builtin_amdgcn_raw_buffer_load_b64(in, off(i, t), 0, 0));
                v = ep_f32x4{bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y)};
            } else {
                v = __builtin_bit_cast(ep_f32x4, __builtin_amdgcn_raw_buffer_load_b128(in, off(i, t), 0, 0));
            }
        }
    };
    if (a.dw_in) load(0);
    each<NT>([&](auto ii) __attribute__((always_inline)) {
        constexpr int i = decltype(ii)::value;
        if (a.dw_in && i + 1 < NT) load(i + 1);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            ep_f32x4 v = acc[t][i];
            pin(v);
            if (a.dw_in) v += add[i & 1][t];
            if (BF16) {
                const ep_u32x2 o = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2, o), out, off(i, t), 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(ep_i32x4, v), out, off(i, t), 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    });
}

template <int KT, int NT>
__device__ __forceinline__ void write_tiles(const WgradK &a, int e, int n0, int k0,
                                            ep_f32x4 (*acc)[NT]) {
    if (a.bf16_out) write_tiles_as<true, KT, NT>(a, e, n0, k0, acc);
    else write_tiles_as<false, KT, NT>(a, e, n0, k0, acc);
}

// Column sums of dy (all rows of the accumulator alike) for dW rows n0 + lane % 16.
__device__ __forceinline__ void write_sum(const WgradK &a, int e, int n0, ep_f32x4 v) {
    const int lane = threadIdx.x & 63;
    if (lane < 16 && n0 + lane < a.n) {
        const int64_t b = (int64_t)e * a.n + n0 + lane;
        a.db[b] = v[0] + (a.db_in ? a.db_in[b] : 0.0f);
    }
}

// Tiles of 128 x 128, for few rows an expert or few tiles.  With few rows bound by
// writing dW, so what counts is many workgroups in flight (two on a compute unit);
// with many rows and few tiles by the steps of 64 rows, which one workgroup takes
// one after another, 0.6 us each (0.9 on fp8 rows): 4096 rows an expert take 41 to
// 44 us (60 to 64) from 4 experts of 128 x 128 to 4 of 1024 x 1024.  Four waves of 64
// x 64, two stages.  fp8 rows pass through registers while the step before is
// computed.  16 experts of 1408 x 1024, 129 rows each, added to fp32 gradients:
// 37 us, 0.195 GB at 5.3 TB/s (51 us with cold caches).
constexpr int kT = 128;
constexpr int kOperand = kRows * kT * 2;
constexpr int kStage = 2 * kOperand;

template <bool FP8, bool BIAS>
__global__ __launch_bounds__(256, 2) void expert_wgrad_kernel(WgradK a) {
    __shared__ __align__(1024) uint8_t lds[2 * kStage];
    int e, n0, k0;
    if (!tile_of(a, kT, &e, &n0, &k0)) return;
    int row0 = 0;
    const int rows = wave_uniform(segment_rows(a.seg, e, &row0));
    row0 = wave_uniform(row0);
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wk = wave & 1, wn = wave >> 1;
    const int N = a.n, K = a.k;

    constexpr int kCopies = kOperand / 1024 / 4;
    uint32_t yoff[kCopies], xoff[FP8 ? 1 : kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = (i * 4 + wave) * 4 + (lane >> 4);
        const int c16 = lane & 15;
        const int c = ((c16 >> 1) ^ granule_of(r)) * 16 + (c16 & 1) * 8;
        yoff[i] = (uint32_t)r * N * 2 + (uint32_t)(n0 + c) * 2;
        if (n0 + c >= N) yoff[i] = kOutOfRange;
        if (!FP8) {
            xoff[FP8 ? 0 : i] = (uint32_t)r * K * 2 + (uint32_t)(k0 + c) * 2;
            if (k0 + c >= K) xoff[FP8 ? 0 : i] = kOutOfRange;
        }
    }
    const uint32_t lds0 = lds_offset(lds);
    const int steps = (rows + kRows - 1) / kRows;
    auto copy = [&](int s, int stage) {
        // buffers of this step's rows alone: offsets stay in 32 bits, and
        // rows behind the last read as zeros
        const int left = min(kRows, rows - s * kRows);
        const int64_t r0 = (int64_t)row0 + s * kRows;
        const ep_i32x4 ybuf = buffer_of(a.dy + r0 * N * 2, (uint32_t)left * N * 2);
        const uint32_t base = lds0 + stage * kStage + wave * 1024;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) dma16(ybuf, base + kOperand + i * 4096, yoff[i], 0);
        if (!FP8) {
            const ep_i32x4 xbuf = buffer_of(a.x + r0 * K * 2, (uint32_t)left * K * 2);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) dma16(xbuf, base + i * 4096, xoff[FP8 ? 0 : i], 0);
        }
    };
    // fp8: this thread's 32 codes of row tid/4, channels (tid%4)*32 of the tile
    const int fr = tid >> 2, fc = (tid & 3) * 32;
    ep_u32x4 code[2];
    float scale = 0.0f;
    auto fetch = [&](int s) {
        code[0] = code[1] = ep_u32x4{0, 0, 0, 0};
        const int r = s * kRows + fr;
        if (r < rows && k0 + fc < K) {
            const int64_t row = (int64_t)row0 + r;
            const ep_u32x4 *p = (const ep_u32x4 *)(a.x + row * K + k0 + fc);
            code[0] = p[0];
            code[1] = p[1];
            scale = ue8m0_value(a.x_scales[row * (K / kFp8Group) + (k0 + fc) / kFp8Group]);
        }
    };
    auto place = [&](int stage) {
        uint8_t *row = lds + stage * kStage + fr * 256;
#pragma unroll
        for (int i = 0; i < 4; ++i) {           // 8 channels each
            ep_u32x4 v;
            const uint32_t lo = code[i >> 1][(i & 1) * 2], hi = code[i >> 1][(i & 1) * 2 + 1];
            v.x = fp8_pair_bf16<false>(lo, scale);
            v.y = fp8_pair_bf16<true>(lo, scale);
            v.z = fp8_pair_bf16<false>(hi, scale);
            v.w = fp8_pair_bf16<true>(hi, scale);
            const int c = fc + i * 8;
            *(ep_u32x4 *)(row + ((c >> 4) ^ granule_of(fr)) * 32 + (c & 8) * 2) = v;
        }
    };

    ep_f32x4 acc[4][4], sum[BIAS ? 4 : 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BIAS) sum[BIAS ? i : 0] = ep_f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) acc[t4][i] = ep_f32x4{0, 0, 0, 0};
    }
    const bool sums = BIAS && k0 == 0 && wk == 0;   // this wave also sums dy's columns
    const ep_u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

    auto compute = [&](int stage) {
        const uint8_t *xl = lds + stage * kStage;
        const uint8_t *yl = xl + kOperand;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ep_u32x4 xf[4], yf[4];
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) xf[t4] = transposed_operand<256>(xl, wk * 4 + t4, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) yf[i] = transposed_operand<256>(yl, wn * 4 + i, h);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t4 = 0; t4 < 4; ++t4) acc[t4][i] = mfma_bf16(xf[t4], yf[i], acc[t4][i]);
            if (sums) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[BIAS ? i : 0] = mfma_bf16(ones, yf[i], sum[BIAS ? i : 0]);
            }
        }
    };

    if (steps > 0) {
        if (FP8) fetch(0);
        copy(0, 0);
        if (FP8) place(0);
    }
    for (int s = 0; s < steps; ++s) {
        dma_wait<0>();
        barrier_only();
        if (s + 1 < steps) {
            if (FP8) fetch(s + 1);
            copy(s + 1, (s + 1) & 1);
        }
        compute(s & 1);
        if (FP8 && s + 1 < steps) place((s + 1) & 1);
    }

    write_tiles<4, 4>(a, e, n0 + wn * 64, k0 + wk * 64, acc);
    if (sums) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pin(sum[BIAS ? i : 0]);
            write_sum(a, e, n0 + wn * 64 + i * 16, sum[BIAS ? i : 0]);
        }
    }
}

// Tiles of 256 x 256, for many rows an expert: bound by the matrix instructions.
// Four waves of 128 x 128 in phases as in the linear kernel's wide tiles: regions
// X0, X1 (the waves' first and second 64 channels of x) and Y0, Y1 (of dy's
// columns), each [64 rows][128 columns]:
//   phase   multiplies       reads (step)              copies (step)
//     A     X0 Y0, X1 Y0     X1 (s), Y1 (s)            Y0, X0 (s + 2)
//     B     X0 Y1, X1 Y1     Y0 (s + 1), X0 (s + 1)    X1, Y1 (s + 2)
//
// fp8 rows are copied as they are, 16 KB a step and three steps ahead, with their
// scale bytes, and turned to bf16 from there by all threads, region X0 of the
// next step in phase A and X1 in phase B; these regions then need no second
// stage, which makes room for three raw steps.
//
// 8 experts of 4096 x 7168, 32768 rows: bf16 1.53 to 1.57 ms (1.22 PFLOP/s), fp8 rows
// 1.73 to 1.80 (1.1).  A library product with both operands transposed reaches 1.17.
constexpr int kWT = 256;
constexpr int kRegion = kRows * 128 * 2;

template <bool FP8, bool BIAS>
__global__ __launch_bounds__(256, 1) void expert_wgrad_wide_kernel(WgradK a) {
    constexpr int kX = FP8 ? 2 * kRegion : 4 * kRegion;          // x regions of all stages
    constexpr int kRaw = kRows * kWT, kRawStages = 3;
    constexpr int kScales = 4 * 256;                              // a wave's 64 bytes as dwords
    __shared__ __align__(1024) uint8_t lds[4 * kRegion + kX + (FP8 ? kRawStages * (kRaw + kScales) : 0)];
    uint8_t *const xlds = lds + 4 * kRegion;
    uint8_t *const raw = xlds + kX;
    int e, n0, k0;
    if (!tile_of(a, kWT, &e, &n0, &k0)) return;
    int row0 = 0;
    const int rows = wave_uniform(segment_rows(a.seg, e, &row0));
    row0 = wave_uniform(row0);
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wk = wave & 1, wn = wave >> 1;
    const int N = a.n, K = a.k;
    const int steps = (rows + kRows - 1) / kRows;

    // copies: a wave moves 16 rows of 256 bytes of each region, 4 at a time;
    // region 1 is 64 columns on.  Columns past the matrix read the next row's
    // (zeros behind the last): they reach only results that are not stored.
    uint32_t yoff[4], xoff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = wave * 16 + j * 4 + (lane >> 4);
        const int g = (lane >> 1 & 7) ^ granule_of(r);            // 16 columns each
        const uint32_t bias = kDmaBias - j * 1024;
        const int c = (g >> 2) * 128 + (g & 3) * 16 + (lane & 1) * 8;
        yoff[j] = ((uint32_t)r * (uint32_t)N + (uint32_t)(n0 + c)) * 2 + bias;
        // fp8: a raw row as it lies
        xoff[j] = FP8 ? (uint32_t)r * (uint32_t)K + (uint32_t)(k0 + l16 * 16) + bias
                      : ((uint32_t)r * (uint32_t)K + (uint32_t)(k0 + c)) * 2 + bias;
    }
    const int groups = K / kFp8Group;
    // this lane's row, the group of the wave's parity
    const uint32_t soff = k0 + (wave & 1) * 128 < K ? (uint32_t)lane * groups + k0 / kFp8Group + (wave & 1) : kOutOfRange;
    // the buffer of a step's rows: offsets stay in 32 bits, and rows behind the
    // last (all of them behind the last step) read as zeros
    uint32_t region1 = 0;             // byte offset of region 1, 0 in an empty buffer
    uint32_t from = 0;                // of the region being copied
    auto rows_of = [&](const uint8_t *p, int s, uint32_t row_bytes, uint32_t early) {
        const int left = max(0, min(kRows, rows - s * kRows));
        ep_i32x4 b = buffer_of(p + ((int64_t)row0 + s * kRows) * row_bytes - early, left * row_bytes + early);
        if (left == 0) b.z = 0;
        region1 = left == 0 ? 0 : 128;
        return b;
    };
    const uint32_t lds0 = lds_offset(lds) + wave * 4096, xlds0 = lds_offset(xlds) + wave * 4096;
    const uint32_t raw0 = lds_offset(raw);
    ep_i32x4 yb, xb;
    auto copy_y = [&](int s, int stage, int t, auto j) {
        constexpr int J = decltype(j)::value;
        if (J == 0) {
            yb = rows_of(a.dy, s, (uint32_t)N * 2, kDmaBias);
            from = t ? region1 : 0;
        }
        dma16_of4<J>(yb, lds0 + (stage * 2 + t) * kRegion, yoff[J], from);
    };
    auto copy_x = [&](int s, int stage, int t, auto j) {
        constexpr int J = decltype(j)::value;
        if (FP8) return;
        if (J == 0) {
            xb = rows_of(a.x, s, (uint32_t)K * 2, kDmaBias);
            from = t ? region1 : 0;
        }
        dma16_of4<J>(xb, xlds0 + (stage * 2 + t) * kRegion, xoff[J], from);
    };
    // a raw step: 16 KB of codes, and per wave 64 scale bytes (a dword each)
    auto copy_raw = [&](int s, auto j) {
        constexpr int J = decltype(j)::value;
        if (!FP8) return;
        const uint32_t at = raw0 + (s % kRawStages) * (kRaw + kScales);
        if (J == 0) {
            const ep_i32x4 sb = rows_of(a.x_scales, s, (uint32_t)groups, 0);
            dma1(sb, at + kRaw + wave * 256, soff, 0);
            xb = rows_of(a.x, s, (uint32_t)K, kDmaBias);
            from = 0;
        }
        dma16_of4<J>(xb, at + wave * 4096, xoff[J], from);
    };
    // raw codes of step s to region t: a thread's 32 channels of one row, in
    // four pieces of 8
    const int fr = tid >> 2, fc = (tid & 3) * 32;                 // row, column in the region
    auto convert = [&](int s, int t, int i) {
        if (!FP8) return;
        const uint8_t *from = raw + (s % kRawStages) * (kRaw + kScales);
        const int half = fc >> 6;                                 // the 128-channel group
        const ep_u32x2 codes = *(const ep_u32x2 *)(from + fr * 256 + half * 128 + t * 64 + (fc & 63) + i * 8);
        const float scale = ue8m0_value(*(const uint32_t *)(from + kRaw + half * 256 + fr * 4) & 0xFF);
        ep_u32x4 v;
        v.x = fp8_pair_bf16<false>(codes.x, scale);
        v.y = fp8_pair_bf16<true>(codes.x, scale);
        v.z = fp8_pair_bf16<false>(codes.y, scale);
        v.w = fp8_pair_bf16<true>(codes.y, scale);
        const int c = fc + i * 8;
        *(ep_u32x4 *)(xlds + t * kRegion + fr * 256 + ((c >> 4) ^ granule_of(fr)) * 32 + (c & 8) * 2) = v;
    };

    ep_u32x4 xf[2][4][2], yf[2][4][2];                            // [region][tile][half]
    auto read_x = [&](int stage, int t, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            xf[t][i][h] = transposed_operand<256>(xlds + ((FP8 ? 0 : stage * 2) + t) * kRegion, wk * 4 + i, h);
    };
    auto read_y = [&](int stage, int t, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            yf[t][i][h] = transposed_operand<256>(lds + (stage * 2 + t) * kRegion, wn * 4 + i, h);
    };

    ep_f32x4 acc[8][8], sum[BIAS ? 8 : 1];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (BIAS) sum[BIAS ? t : 0] = ep_f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t][i] = ep_f32x4{0, 0, 0, 0};
    }
    const bool sums = BIAS && k0 == 0 && wk == 0;   // this wave also sums dy's columns
    const ep_u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    auto part = [&](int tx, int ty, auto read, auto copy, auto work) {
        each<32>([&](auto mm) __attribute__((always_inline)) {
            constexpr int m = decltype(mm)::value, h = m / 16, b = m / 4 % 4, c = m % 4;
            ep_f32x4 &d = acc[tx * 4 + b][ty * 4 + c];
            d = mfma_bf16(xf[tx][b][h], yf[ty][c][h], d);
            if constexpr (m % 8 == 0) read(m / 8);
            if constexpr (m % 8 == 4) copy(std::integral_constant<int, m / 8>{});
            if constexpr (m % 8 == 2) work(m / 8);
            __builtin_amdgcn_sched_barrier(0);
        });
        if (BIAS && tx == 0 && sums) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ep_f32x4 &d = sum[BIAS ? ty * 4 + i % 4 : 0];
                d = mfma_bf16(ones, yf[ty][i % 4][i / 4], d);
            }
        }
    };
    // end of a phase: the regions the next one reads have landed, and every
    // wave has read those this phase read
    auto turn = [&](auto allowed) {
        dma_wait<decltype(allowed)::value>();
        barrier_only();
        __builtin_amdgcn_sched_barrier(0);
    };
    // What may still be in flight then: the copies issued behind the ones needed
    // next.  bf16: 8 a phase, and those of the phase before last are needed.  fp8:
    // a phase A issues 4 (Y0) and 5 (raw), a phase B 4 (Y1).  After A, Y0 of the A
    // before is needed: behind it 5 + 4 + 9.  After B, Y1 of the B before is: 9 +
    // 4; and the raw step that the next step turns to bf16, from the A three
    // phases back: 4 + 9 + 4, more than 13.
    constexpr std::integral_constant<int, FP8 ? 18 : 16> after_a{};
    constexpr std::integral_constant<int, FP8 ? 13 : 16> after_b{};
    constexpr std::integral_constant<int, 0> none{};

    if (steps > 0) {
        for (int s = 0; s < 3; ++s) each<4>([&](auto j) { copy_raw(s, j); });
        for (int s = 0; s < 2; ++s) {
            each<4>([&](auto j) { copy_y(s, s, 0, j); });
            each<4>([&](auto j) { copy_x(s, s, 0, j); });
            each<4>([&](auto j) { copy_x(s, s, 1, j); });
            each<4>([&](auto j) { copy_y(s, s, 1, j); });
        }
        turn(none);
        if (FP8) {
            each<4>([&](auto i) { convert(0, 0, i); convert(0, 1, i); });
            turn(none);
        }
        each<4>([&](auto i) { read_y(0, 0, i); });
        each<4>([&](auto i) { read_x(0, 0, i); });
        turn(none);
    }
    auto step = [&](int s, int st) {
        part(0, 0, [&](int i) { read_x(st, 1, i); }, [&](auto j) { copy_y(s + 2, st, 0, j); },
             [&](int i) { convert(s + 1, 0, i); });
        part(1, 0, [&](int i) { read_y(st, 1, i); },
             [&](auto j) { if (FP8) copy_raw(s + 3, j); else copy_x(s + 2, st, 0, j); }, [](int) {});
        turn(after_a);
        part(0, 1, [&](int i) { read_y(st ^ 1, 0, i); }, [&](auto j) { copy_x(s + 2, st, 1, j); },
             [&](int i) { convert(s + 1, 1, i); });
        part(1, 1, [&](int i) { read_x(st ^ 1, 0, i); }, [&](auto j) { copy_y(s + 2, st, 1, j); }, [](int) {});
        turn(after_b);
    };
    for (int s = 0; s < steps; ++s) step(s, s & 1);
    // no copy may still be on its way to this workgroup's LDS when it ends
    dma_wait<0>();
    write_tiles<8, 8>(a, e, n0 + wn * 128, k0 + wk * 128, acc);
    if (sums) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            pin(sum[BIAS ? i : 0]);
            write_sum(a, e, n0 + wn * 128 + i * 16, sum[BIAS ? i : 0]);
        }
    }
}

}  // namespace

hipError_t launch_expert_wgrad(const WgradArgs &a, hipStream_t stream) {
    WgradK k = {};
    k.seg = a.seg;
    k.dy = (const uint8_t *)a.dy;
    k.x = (const uint8_t *)a.x;
    k.x_scales = a.x_scales;
    k.dw_in = a.dw_in;
    k.db_in = a.db_in;
    k.dw = a.dw;
    k.db = a.db;
    k.n = a.n;
    k.k = a.k;
    k.bf16_out = a.bf16_out ? 1 : 0;
    // 256 x 256 tiles where they keep every compute unit busy and an expert's rows
    // pay for filling and draining them: 16 experts of 2048 x 2048, bf16, 1024 rows
    // each 165 us against 210 of the 128 x 128 tiles, 512 rows 113 against 125, 256
    // rows 88 against 86; 4 experts of 1024 x 1024 (64 wide tiles), 4096 rows each
    // 106 against 49.
    const int64_t wide_tiles = (int64_t)a.seg.E * ((a.n + kWT - 1) / kWT) * ((a.k + kWT - 1) / kWT);
    const bool wide = wide_tiles >= 256 && a.seg.pairs / a.seg.E > 384;
    const int T = wide ? kWT : kT;
    k.tiles_n = (a.n + T - 1) / T;
    k.tiles_k = (a.k + T - 1) / T;
    const int64_t tiles = (int64_t)a.seg.E * k.tiles_n * k.tiles_k;
    const int64_t grid = (tiles + 255) / 256 * 256;   // whole rounds of 8 runs of 32
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(256);
    if (wide) {
        if (a.fp8) {
            if (a.db) expert_wgrad_wide_kernel<true, true><<<g, t, 0, stream>>>(k);
            else expert_wgrad_wide_kernel<true, false><<<g, t, 0, stream>>>(k);
        } else {
            if (a.db) expert_wgrad_wide_kernel<false, true><<<g, t, 0, stream>>>(k);
            else expert_wgrad_wide_kernel<false, false><<<g, t, 0, stream>>>(k);
        }
    } else if (a.fp8) {
        if (a.db) expert_wgrad_kernel<true, true><<<g, t, 0, stream>>>(k);
        else expert_wgrad_kernel<true, false><<<g, t, 0, stream>>>(k);
    } else {
        if (a.db) expert_wgrad_kernel<false, true><<<g, t, 0, stream>>>(k);
        else expert_wgrad_kernel<false, false><<<g, t, 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace ep
