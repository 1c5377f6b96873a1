// The experts' weight gradients over the receive segments: which kernel of
// ep_wgrad_device.h takes a call.
#include "ep_wgrad_device.h"

namespace ep {

namespace {

template <bool FP8, bool BIAS>
__global__ __launch_bounds__(256, 2) void expert_wgrad_kernel(WgradK a) {
    __shared__ __align__(1024) uint8_t lds[kWgradLds];
    wgrad_tile<FP8, BIAS>(a, tile_in_runs(blockIdx.x), lds);
}

template <bool FP8, bool BIAS>
__global__ __launch_bounds__(256, 1) void expert_wgrad_wide_kernel(WgradK a) {
    __shared__ __align__(1024) uint8_t lds[kWgradWideLds<FP8>];
    wgrad_wide_tile<FP8, BIAS>(a, tile_in_runs(blockIdx.x), lds);
}

}  // namespace

hipError_t launch_expert_wgrad(const WgradArgs &a, hipStream_t stream) {
    // 256 x 256 tiles where they keep every compute unit busy and an expert's rows
    // pay for filling and draining them: 16 experts of 2048 x 2048, bf16, 1024 rows
    // each 165 us against 210 of the 128 x 128 tiles, 512 rows 113 against 125, 256
    // rows 88 against 86; 4 experts of 1024 x 1024 (64 wide tiles), 4096 rows each
    // 106 against 49.
    const int64_t wide_tiles = (int64_t)a.seg.E * ((a.n + kWT - 1) / kWT) * ((a.k + kWT - 1) / kWT);
    const bool wide = wide_tiles >= 256 && a.seg.pairs / a.seg.E > 384;
    const int T = wide ? kWT : kT;
    const WgradK k = kernel_args(a, T);
    const int64_t grid = grid_of(k);
    if (!launchable(grid, 256)) return hipErrorInvalidConfiguration;
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
