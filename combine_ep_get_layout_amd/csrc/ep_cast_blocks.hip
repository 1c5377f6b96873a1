// Weights to e4m3 codes with one fp32 scale per 128 x 128 block, and on request
// the same of the transposed matrix (the block's scale is the same), from one read.
//
// A workgroup takes one block, a thread 8 rows x 8 columns of it in registers.
// Bound by HBM.  The transposed codes are turned 8 x 8 in registers and leave
// through LDS, so that both matrices are written in lines of 128 bytes.
#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kB = kFp8Group;

// 4 x 4 bytes: byte j of r[i] and byte i of r[j] change places.
__device__ __forceinline__ void turn4(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    const uint32_t ab_lo = __builtin_amdgcn_perm(b, a, 0x05010400u);   // a0 b0 a1 b1
    const uint32_t ab_hi = __builtin_amdgcn_perm(b, a, 0x07030602u);   // a2 b2 a3 b3
    const uint32_t cd_lo = __builtin_amdgcn_perm(d, c, 0x05010400u);
    const uint32_t cd_hi = __builtin_amdgcn_perm(d, c, 0x07030602u);
    a = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u);
    b = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u);
    c = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u);
    d = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u);
}

template <bool TURNED>
__global__ __launch_bounds__(256) void cast_blocks_kernel(CastBlocksArgs a) {
    __shared__ float red[4];
    __shared__ __align__(16) uint8_t lds[TURNED ? kB * kB : 16];
    const int tid = threadIdx.x, r8 = tid >> 4, c8 = tid & 15;
    const int nb = (a.n + kB - 1) / kB, kb = (a.k + kB - 1) / kB;
    const int64_t per = (int64_t)nb * kb;
    const int64_t e = (int64_t)blockIdx.x / per;
    const int at = (int)(blockIdx.x - e * per), bi = at / kb, bj = at - bi * kb;
    const int row = bi * kB + r8 * 8, col = bj * kB + c8 * 8;
    const int64_t base = e * a.n * a.k;
    const uint16_t *w = (const uint16_t *)a.w + base;
    ep_u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = ep_u32x4{0, 0, 0, 0};
        if (row + i < a.n && col < a.k) v[i] = load_nt((const ep_u32x4 *)(w + (int64_t)(row + i) * a.k + col));
    }
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = fmaxf(big, amax8(v[i]));
    big = group_max(big, 64);
    if ((tid & 63) == 0) red[tid >> 6] = big;
    __syncthreads();
    const float s = scale_of(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float y = 1.0f / s;
    ep_u32x2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = encode8_y<false>(v[i], s, y);
    if (a.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row + i < a.n && col < a.k)
                *(ep_u32x2 *)(a.codes + base + (int64_t)(row + i) * a.k + col) = c[i];
        if (tid == 0) a.scales[e * per + at] = s;
    }
    if (!TURNED) return;
    uint32_t d[2][2][4];                           // [columns 4..7][rows 4..7][column]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        d[0][i >> 2][i & 3] = c[i].x;
        d[1][i >> 2][i & 3] = c[i].y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t *t = d[i >> 1][i & 1];
        turn4(t[0], t[1], t[2], t[3]);
    }
    // 8 bytes (rows r8 * 8 ..) of column j at place r8 ^ c8 of its line
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const ep_u32x2 o = {d[j >> 2][0][j & 3], d[j >> 2][1][j & 3]};
        *(ep_u32x2 *)(lds + (c8 * 8 + j) * kB + ((r8 ^ c8) * 8)) = o;
    }
    __syncthreads();
    const int row_t = bi * kB + c8 * 8;            // now lanes run along the rows of w
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = r8 * 8 + j;                  // column of the block; its c8 was r8
        const ep_u32x2 o = *(const ep_u32x2 *)(lds + k * kB + ((c8 ^ r8) * 8));
        if (bj * kB + k < a.k && row_t < a.n)
            *(ep_u32x2 *)(a.codes_t + base + (int64_t)(bj * kB + k) * a.n + row_t) = o;
    }
    if (tid == 0) a.scales_t[e * per + (int64_t)bj * nb + bi] = s;
}

}  // namespace

hipError_t launch_cast_blocks(const CastBlocksArgs &a, hipStream_t stream) {
    const int64_t grid = (int64_t)a.num * ((a.n + kB - 1) / kB) * ((a.k + kB - 1) / kB);
    if (!launchable(grid, 256)) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(256);
    if (a.codes_t) cast_blocks_kernel<true><<<g, t, 0, stream>>>(a);
    else cast_blocks_kernel<false><<<g, t, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ep
