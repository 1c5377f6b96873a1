// Backward pass of the experts' activation, from pre-activations kept in 8
// bits (e4m3, UE8M0 scales per 32 channels) or in bf16.
//
// For row r with weight w (1 without weights) and incoming dh, the gradient of
// the row w * h that a weighted combine saw:
//   h = f(g) u,  dweight = sum dh h,  dg = w dh u f'(g),  du = w dh f(g)
// (not gated: h = f(z), dz = w dh f'(z)), and w h, the other operand of the
// down product's weight gradient.  One pass: 10 1/16 bytes move per gated
// channel (dh 2, codes and scales 2 1/16, dz 4, w h 2) and nothing is read
// twice; it is bound by HBM: 32113 rows of 4096 pre-activations, swiglu, 0.66 GB in
// 122 us, 5.4 TB/s.
// One wave takes one row, a lane 8 channels at a time, so the row's sum ends
// in one wave reduction in a fixed order.
#include "ep_expert_device.h"

namespace ep {

namespace {

struct ActK {
    ActBackwardArgs a;
};

// 8 pre-activations of a row from channel c on.
template <bool FP8>
__device__ __forceinline__ void load8(const ActBackwardArgs &a, int64_t row, int c, float *z) {
    if (FP8) {
        const ep_u32x2 v = *(const ep_u32x2 *)((const uint8_t *)a.pre + row * a.n + c);
        const float s = ue8m0_value(a.pre_scales[row * (a.n >> 5) + (c >> 5)]);
        auto p0 = __builtin_amdgcn_cvt_pk_f32_fp8(v.x, false);
        auto p1 = __builtin_amdgcn_cvt_pk_f32_fp8(v.x, true);
        auto p2 = __builtin_amdgcn_cvt_pk_f32_fp8(v.y, false);
        auto p3 = __builtin_amdgcn_cvt_pk_f32_fp8(v.y, true);
        z[0] = p0[0] * s; z[1] = p0[1] * s; z[2] = p1[0] * s; z[3] = p1[1] * s;
        z[4] = p2[0] * s; z[5] = p2[1] * s; z[6] = p3[0] * s; z[7] = p3[1] * s;
    } else {
        const ep_u32x4 v = *(const ep_u32x4 *)((const uint16_t *)a.pre + row * a.n + c);
        for (int i = 0; i < 4; ++i) {
            z[2 * i] = bf16_lo(v[i]);
            z[2 * i + 1] = bf16_hi(v[i]);
        }
    }
}

__device__ __forceinline__ ep_u32x4 pack8(const float *y) {
    ep_u32x4 v;
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
    return v;
}

template <bool FP8, bool GATED>
__global__ __launch_bounds__(256) void act_backward_kernel(ActK k) {
    const ActBackwardArgs &a = k.a;
    const int lane = threadIdx.x & 63;
    const int64_t used = *a.total_rows;
    if (used > a.num_rows) {
        // rows that the buffers lack: only those that hold a pair are missed
        const int64_t end = used < a.entries ? used : a.entries;
        bool missed = used > a.entries;                // as the layout itself reports it
        for (int64_t r = a.num_rows + (int64_t)blockIdx.x * 256 + threadIdx.x; r < end;
             r += (int64_t)gridDim.x * 256)
            missed |= a.src_of_slot[r] >= 0;
        if (missed) atomicOr(a.status, kDevRecvOverflow);
    }
    const int64_t rows = used < a.num_rows ? used : a.num_rows;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= rows || a.src_of_slot[row] < 0) return;
    const float w = a.row_weights ? a.row_weights[row] : 1.0f;
    const uint16_t *dh = (const uint16_t *)a.dh + row * a.m;
    uint16_t *dpre = (uint16_t *)a.dpre + row * a.n;
    float dot = 0.0f;
    for (int c = lane * 8; c < a.m; c += 512) {
        float z[8], u[8], d[8], h[8], dz[8], du[8];
        load8<FP8>(a, row, c, z);
        if (GATED) load8<FP8>(a, row, a.m + c, u);
        const ep_u32x4 v = *(const ep_u32x4 *)(dh + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
            float f, df;
            act_both(z[i], a.kind, &f, &df);
            const float y = GATED ? f * u[i] : f;
            dot = __builtin_fmaf(d[i], y, dot);
            const float wd = w * d[i];
            h[i] = w * y;
            dz[i] = GATED ? wd * u[i] * df : wd * df;
            if (GATED) du[i] = wd * f;
        }
        *(ep_u32x4 *)(dpre + c) = pack8(dz);
        if (GATED) *(ep_u32x4 *)(dpre + a.m + c) = pack8(du);
        if (a.h) *(ep_u32x4 *)((uint16_t *)a.h + row * a.m + c) = pack8(h);
    }
    if (a.dweights) {
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
        if (lane == 0) a.dweights[row] = dot;
    }
}

}  // namespace

hipError_t launch_act_backward(const ActBackwardArgs &a, hipStream_t stream) {
    const int64_t grid = (a.num_rows + 3) / 4;
    const ActK k{a};
    const dim3 g((unsigned)grid), t(256);
    if (a.pre_scales) {
        if (a.gated) act_backward_kernel<true, true><<<g, t, 0, stream>>>(k);
        else act_backward_kernel<true, false><<<g, t, 0, stream>>>(k);
    } else {
        if (a.gated) act_backward_kernel<false, true><<<g, t, 0, stream>>>(k);
        else act_backward_kernel<false, false><<<g, t, 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace ep
