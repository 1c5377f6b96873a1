// Matrix product of few dense rows with its epilogue: out[t] = act(x[t] W^T + b)
// + residual[t] for up to 64 rows, bf16, or e4m3 codes with one fp32 scale per
// 128 channels of x and per 128 x 128 block of W.
//
// The weights are read once; the rows of x, from the caches, once per workgroup.  A
// workgroup takes 16 rows of W (gated: 8 gate rows and the 8 up rows that go with
// them), its four waves split the contraction, and each has its next units of 16
// rows x 128 bytes on their way to registers, in the matrix instruction's layout.
// The rows of x are its other operand, 16 columns a group.  The partial sums meet in
// LDS and are added in wave order.
//
// Many small workgroups hide the latency better than deep rings: four waves with two
// units each, where eight waves with eight units took (back to back) 13.6 us for one
// row of 7168 to 4096, gated, in bf16, these take 11.0 (5.3 TB/s); 13.9 and 7.2 for
// 2048 to 7168; e4m3 9.7 and 8.1, 12.5 and 5.2.  (Eight waves with one unit each 10.7 and
// 7.7, e4m3 7.4 and 5.5: better for the long contraction alone.)  Up to about 8 rows bound
// by reading the weights, in e4m3 of 7168 channels at 3.6 TB/s by a wave's seven round
// trips to memory; then by reading x: 16 rows 15.0, 64 rows 34 us.
#include "ep_expert_device.h"

namespace ep {

namespace {

typedef __amdgpu_buffer_rsrc_t Buffer;

constexpr int kUnit = 128;          // bytes of a row that a wave takes at once

struct FewK {
    FewRowsArgs a;
    int m, kind;
};

// One unit: a lane's pieces q and q + 4 of its weight row and of its rows of x.
template <int MT>
struct Unit {
    ep_u32x4 w[2], x[MT][2];
    float sw, sx[MT];
};

constexpr int kWaves = 4;

template <bool FP8, bool GATED, int MT>
__global__ __launch_bounds__(64 * kWaves) void few_rows_kernel(FewK p) {
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int D = MT == 1 ? 2 : 1;                     // units on their way
    constexpr int COLS = GATED ? 8 : 16;
    const FewRowsArgs &a = p.a;
    __shared__ float red[kWaves][MT][16][16];              // [wave][group][row of W][row of x]
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int c0 = blockIdx.x * COLS;
    const uint32_t ld = (uint32_t)a.k * ES;
    const int groups = a.k / kFp8Group;
    // row of W at place r: its column of z, or -1
    auto column = [&](int r) {
        const int c = c0 + (GATED ? r & 7 : r);
        if (c >= p.m) return -1;
        return GATED && r >= 8 ? p.m + c : c;
    };
    const Buffer wb = __builtin_amdgcn_make_buffer_rsrc((void *)a.w, 0, (int)((uint32_t)a.n * ld), 0x00020000);
    const Buffer xb = __builtin_amdgcn_make_buffer_rsrc((void *)a.x, 0, (int)((uint32_t)a.rows * ld), 0x00020000);
    const Buffer sxb = __builtin_amdgcn_make_buffer_rsrc((void *)a.x_scales, 0, a.rows * groups * 4, 0x00020000);
    const Buffer swb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)a.w_scales, 0, (a.n + kFp8Group - 1) / kFp8Group * groups * 4, 0x00020000);
    const int wr = column(l16);
    const uint32_t wat = wr < 0 ? kOutOfRange : (uint32_t)wr * ld + q * 16;
    // the accumulators of this lane are rows 4 q .. 4 q + 3 of W: all in one block
    const int sr = column(4 * q);
    const uint32_t swat = sr < 0 ? kOutOfRange : (uint32_t)(sr / kFp8Group) * groups * 4;
    uint32_t xat[MT], sxat[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int t = i * 16 + l16;
        xat[i] = t < a.rows ? (uint32_t)t * ld + q * 16 : kOutOfRange;
        sxat[i] = t < a.rows ? (uint32_t)(t * groups) * 4 : kOutOfRange;
    }
    const int units = (int)((ld + kUnit - 1) / kUnit);
    const int per = (units + kWaves - 1) / kWaves;
    const int u0 = min(units, wave * per), u1 = min(units, u0 + per);

    Unit<MT> ring[D];
    auto load = [&](Unit<MT> &v, int u) __attribute__((always_inline)) {
        // past the row (or this wave's part): zeros
        uint32_t out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            out[h] = u >= u1 || (uint32_t)u * kUnit + h * 64 + q * 16 >= ld ? kOutOfRange : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v.w[h] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                wb, (wat + (uint32_t)u * kUnit + h * 64) | out[h], 0, 0));
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v.x[i][h] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    xb, (xat[i] + (uint32_t)u * kUnit + h * 64) | out[h], 0, 0));
        if (FP8) {
            const uint32_t out = u >= u1 ? kOutOfRange : 0;
            v.sw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(swb, (swat + u * 4) | out, 0, 0));
#pragma unroll
            for (int i = 0; i < MT; ++i)
                v.sx[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    sxb, (sxat[i] + u * 4) | out, 0, 0));
        }
    };
    ep_f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = ep_f32x4{0, 0, 0, 0};
    auto multiply = [&](const Unit<MT> &v) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (FP8) {
                const ep_f32x4 s = mfma_fp8_plain(v.w, v.x[i], ep_f32x4{0, 0, 0, 0});
                const float f = v.sw * v.sx[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(s[j], f, acc[i][j]);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[i] = mfma_bf16(v.w[h], v.x[i][h], acc[i]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(ring[d], u0 + d);
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply(ring[d]);
            load(ring[d], u + D + d);
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[wave][i][4 * q + j][l16] = acc[i][j];
    __syncthreads();
    for (int at = tid; at < MT * 16 * COLS; at += 64 * kWaves) {
        const int j = at % COLS, t = at / COLS;
        const int c = c0 + j;
        if (t >= a.rows || c >= p.m) continue;
        float z[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 1); ++k) {
            for (int w = 0; w < kWaves; ++w) z[k] += red[w][t >> 4][k * 8 + j][t & 15];
            if (a.bias) z[k] += bf16_lo(((const uint16_t *)a.bias)[k * p.m + c]);
        }
        float y = p.kind == 0 ? z[0] : p.kind == 1 ? act_value<1>(z[0]) : act_value<2>(z[0]);
        if (GATED) y *= z[1];
        if (a.residual) y += bf16_lo(((const uint16_t *)a.residual)[(int64_t)t * p.m + c]);
        ((uint16_t *)a.out)[(int64_t)t * p.m + c] = (uint16_t)pack_bf16(y, 0.0f);
    }
}

template <bool FP8, bool GATED>
hipError_t launch(const FewK &k, hipStream_t stream) {
    const int cols = GATED ? 8 : 16;
    const dim3 g((unsigned)((k.m + cols - 1) / cols)), t(64 * kWaves);
    if (k.a.rows <= 16) few_rows_kernel<FP8, GATED, 1><<<g, t, 0, stream>>>(k);
    else if (k.a.rows <= 32) few_rows_kernel<FP8, GATED, 2><<<g, t, 0, stream>>>(k);
    else few_rows_kernel<FP8, GATED, 4><<<g, t, 0, stream>>>(k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_rows(const FewRowsArgs &a, hipStream_t stream) {
    if (a.rows > kFewRows) return hipErrorInvalidValue;
    FewK k = {};
    k.a = a;
    const bool gated = act_gated(a.act);
    k.m = gated ? a.n / 2 : a.n;
    k.kind = act_kind(a.act);
    if (a.x_scales) return gated ? launch<true, true>(k, stream) : launch<true, false>(k, stream);
    return gated ? launch<false, true>(k, stream) : launch<false, false>(k, stream);
}

}  // namespace ep
