// Weight gradient over the receive segments: dW[e] = dy^T x over the rows of
// segment e, and the bias gradient, the column sums of dy.
//
// A workgroup computes a tile of 256 (dy columns) x 256 (x columns) of one
// expert, over K steps of 64 rows in LDS, two stages.  Both operands lie with
// the summed index (the row) outermost, so both are staged as they lie, 64
// rows of 512 bytes, and read by the transposing LDS read; 32-byte granule g
// of row r is in place g ^ (r & 3 | (r >> 3 & 1) << 2), so that the 16 rows a
// read takes lie in different banks.  The last step's missing rows are zeros
// (reads past the buffer's end).  x is the matrix instruction's first operand:
// a lane's four accumulators are four consecutive channels of one dW row.
//
// fp8 rows of x (kept in 8 bits by the forward pass) are loaded to registers,
// turned to bf16 (exact: the scales are powers of two) and written to the
// same place in LDS while the step before is computed.
#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kT = 256;          // tile edge
constexpr int kRows = 64;        // rows per step
constexpr int kOperand = kRows * kT * 2;
constexpr int kStage = 2 * kOperand;

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

template <bool FP8, bool BIAS>
__global__ __launch_bounds__(512, 2) void expert_wgrad_kernel(WgradK a) {
    __shared__ __align__(1024) uint8_t lds[2 * kStage];
    // Runs of 32 tiles (8 x 4 of them where the tile grid has them) go to one
    // XCD, the runs to the XCDs in turn: the operands of a run meet in one L2,
    // and an expert with more rows than others spreads over all of them.
    const int j = blockIdx.x >> 3;
    const int64_t t = ((int64_t)(j >> 5) * 8 + (blockIdx.x & 7)) * 32 + (j & 31);
    const int per_e = a.tiles_n * a.tiles_k;
    const int e = (int)(t / per_e);
    if (e >= a.seg.E) return;
    const int lt = (int)(t - (int64_t)e * per_e);
    const int g = lt / (8 * a.tiles_k);
    const int gm = min(8, a.tiles_n - g * 8);
    const int rem = lt - g * 8 * a.tiles_k;
    const int n0 = (g * 8 + rem % gm) * kT, k0 = (rem / gm) * kT;

    int row0 = 0;
    const int rows = wave_uniform(segment_rows(a.seg, e, &row0));
    row0 = wave_uniform(row0);
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int wk = wave & 3, wn = wave >> 2;
    const int N = a.n, K = a.k;

    constexpr int kCopies = kOperand / 1024 / 8;
    uint32_t yoff[kCopies], xoff[FP8 ? 1 : kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = (i * 8 + wave) * 2 + (lane >> 5);
        const int c16 = lane & 31;
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
        for (int i = 0; i < kCopies; ++i) dma16(ybuf, base + kOperand + i * 8192, yoff[i], 0);
        if (!FP8) {
            const ep_i32x4 xbuf = buffer_of(a.x + r0 * K * 2, (uint32_t)left * K * 2);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) dma16(xbuf, base + i * 8192, xoff[FP8 ? 0 : i], 0);
        }
    };
    // fp8: this thread's 32 codes of row tid/8, channels (tid%8)*32 of the tile
    const int fr = tid >> 3, fc = (tid & 7) * 32;
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
        uint8_t *row = lds + stage * kStage + fr * 512;
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

    ep_f32x4 acc[4][8], sum[BIAS ? 8 : 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (BIAS) sum[BIAS ? i : 0] = ep_f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) acc[t4][i] = ep_f32x4{0, 0, 0, 0};
    }
    const bool sums = BIAS && k0 == 0 && wk == 0;   // this wave also sums dy's columns
    ep_bf16x8 ones;
    for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

    auto tr8 = [&](const uint8_t *p) {
        const ep_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) ep_i16x4 *)p);
        const ep_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) ep_i16x4 *)(p + 4 * 512));
        ep_u32x4 v;
        v.xy = __builtin_bit_cast(ep_u32x2, lo);
        v.zw = __builtin_bit_cast(ep_u32x2, hi);
        return __builtin_bit_cast(ep_bf16x8, v);
    };
    auto compute = [&](int stage) {
        const uint8_t *xl = lds + stage * kStage;
        const uint8_t *yl = xl + kOperand;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int r = kk * 32 + q * 8 + (l16 >> 2);
            const int f = granule_of(r);
            const int at = r * 512 + (l16 & 3) * 8;
            ep_bf16x8 xf[4], yf[8];
#pragma unroll
            for (int t4 = 0; t4 < 4; ++t4) xf[t4] = tr8(xl + at + ((wk * 4 + t4) ^ f) * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) yf[i] = tr8(yl + at + ((wn * 8 + i) ^ f) * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int t4 = 0; t4 < 4; ++t4)
                    acc[t4][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[t4], yf[i], acc[t4][i], 0, 0, 0);
            if (sums) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum[BIAS ? i : 0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        ones, yf[i], sum[BIAS ? i : 0], 0, 0, 0);
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

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        for (int t4 = 0; t4 < 4; ++t4) pin(acc[t4][i]);
        if (BIAS) pin(sum[BIAS ? i : 0]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = n0 + wn * 128 + i * 16 + l16;
        if (n >= N) continue;
        const int64_t row = ((int64_t)e * N + n) * K;
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) {
            const int k = k0 + wk * 64 + t4 * 16 + 4 * q;
            if (k >= K) continue;
            ep_f32x4 v = acc[t4][i];
            if (a.bf16_out) {
                if (a.dw_in) {
                    const ep_u32x2 o = *(const ep_u32x2 *)((const uint16_t *)a.dw_in + row + k);
                    v[0] += bf16_lo(o.x); v[1] += bf16_hi(o.x);
                    v[2] += bf16_lo(o.y); v[3] += bf16_hi(o.y);
                }
                ep_u32x2 o;
                o.x = pack_bf16(v[0], v[1]);
                o.y = pack_bf16(v[2], v[3]);
                *(ep_u32x2 *)((uint16_t *)a.dw + row + k) = o;
            } else {
                if (a.dw_in) {
                    const ep_f32x4 o = *(const ep_f32x4 *)((const float *)a.dw_in + row + k);
                    for (int c = 0; c < 4; ++c) v[c] += o[c];
                }
                *(ep_f32x4 *)((float *)a.dw + row + k) = v;
            }
        }
        if (sums && q == 0) {
            const int64_t b = (int64_t)e * N + n;
            a.db[b] = sum[BIAS ? i : 0][0] + (a.db_in ? a.db_in[b] : 0.0f);
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
    k.tiles_n = (a.n + kT - 1) / kT;
    k.tiles_k = (a.k + kT - 1) / kT;
    k.bf16_out = a.bf16_out ? 1 : 0;
    const int64_t tiles = (int64_t)a.seg.E * k.tiles_n * k.tiles_k;
    const int64_t grid = (tiles + 255) / 256 * 256;   // whole rounds of 8 runs of 32
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(512);
    if (a.fp8) {
        if (a.db) expert_wgrad_kernel<true, true><<<g, t, 0, stream>>>(k);
        else expert_wgrad_kernel<true, false><<<g, t, 0, stream>>>(k);
    } else {
        if (a.db) expert_wgrad_kernel<false, true><<<g, t, 0, stream>>>(k);
        else expert_wgrad_kernel<false, false><<<g, t, 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace ep
