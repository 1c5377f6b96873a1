// The experts' products over the receive segments: which kernel of
// ep_linear_device.h takes a call.
#include "ep_linear_device.h"

namespace ep {

namespace {

hipError_t launch_wide(const LinearArgs &a, const LinearK &k, bool gated, hipStream_t stream) {
    const int64_t grid = grid_of(a.seg, k.col_tiles, 256);
    if (!launchable(grid, 256)) return hipErrorInvalidConfiguration;
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
    const int64_t grid = grid_of(a.seg, k.col_tiles, BM);
    if (!launchable(grid, 64 * WN * WM)) return hipErrorInvalidConfiguration;
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
    const RowTile tile = row_tile(a.seg, k.m, gated, a.transposed);
    k.col_tiles = (k.m + tile.cols - 1) / tile.cols;
    if (tile.rows == 64) return launch_bm<64, 4, 1, 4>(a, k, gated, stream);
    if (tile.rows == 256) return launch_wide(a, k, gated, stream);
    if (tile.rows == 192) return launch_bm<192, 2, 4, 2>(a, k, gated, stream);
    return launch_bm<128, 2, 4, 3>(a, k, gated, stream);
}

}  // namespace ep
