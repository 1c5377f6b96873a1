// The gated feed-forward block that every token passes (a shared expert), and
// its gradients: dense rows through the matrix kernels of the experts.
//
// Forward: h = f(x Wg^T) * (x Wu^T) by one product whose tiles hold gate and up
// columns together, then out = h W2^T + residual.  Up to 64 rows go through the
// kernel for few rows, bound by reading the weights.
// Backward: the product dout W2 makes dh in its accumulators; its epilogue reads z
// and writes dz = [dgate | dup] and h, so that dh is never stored or rounded.  Then
// dW2 = dout^T h, dW1 = dz^T x and dx = dz W1.  dz and h are rounded to bf16, the
// type that the matrix instructions of these products take.
#include "ep_linear_device.h"

namespace ep {

namespace {

constexpr int kStep = 64;        // channels of a step of the matrix kernels

DensePlan plan_of(int64_t rows, int n, int k, bool transposed) {
    return dense_plan(rows, n, (k + kStep - 1) / kStep, transposed);
}

template <int BM, int WM, int WN, int NS, bool WT, bool GATED, int MODE>
hipError_t launch_tiles(LinearK &k, int parts, hipStream_t stream) {
    const int per = GATED ? WN * 32 : WN * 64;
    k.col_tiles = (k.m + per - 1) / per;
    const int64_t grid = grid_of(k.seg, k.col_tiles, BM);
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    expert_linear_kernel<BM, WM, WN, NS, kBf16, WT, GATED, MODE>
        <<<dim3((unsigned)grid, parts), 64 * WM * WN, 0, stream>>>(k);
    return hipGetLastError();
}

// A product of dense rows with the epilogue MODE; `sums` holds what its plan asks for.
template <bool WT, bool GATED, int MODE>
hipError_t product(LinearK k, int64_t rows, float *sums, hipStream_t stream) {
    k.seg = {};
    k.seg.E = 1;
    k.seg.num_rows = k.seg.pairs = k.seg.each = rows;
    const DensePlan p = plan_of(rows, k.n, k.k, WT);
    if (p.rows == 256) {
        const int per = GATED ? kBN / 2 : kBN;
        k.col_tiles = (k.m + per - 1) / per;
        const int64_t grid = grid_of(k.seg, k.col_tiles, 256);
        if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
        expert_linear_wide_kernel<kBf16, WT, GATED, MODE><<<dim3((unsigned)grid), 256, 0, stream>>>(k);
        return hipGetLastError();
    }
    k.sums = sums;
    k.split = p.split;
    if constexpr (!WT) {
        if (p.cols == 64) {
            if (p.parts == 1) return launch_tiles<64, 4, 1, 4, WT, GATED, MODE>(k, 1, stream);
            const hipError_t rc = launch_tiles<64, 4, 1, 4, WT, GATED, kSums>(k, p.parts, stream);
            return rc != hipSuccess ? rc : launch_finish<MODE, GATED>(k, p.parts, stream);
        }
    }
    if (p.parts == 1)
        return p.rows == 128 ? launch_tiles<128, 2, 2, 2, WT, GATED, MODE>(k, 1, stream)
                             : launch_tiles<64, 2, 2, 3, WT, GATED, MODE>(k, 1, stream);
    const hipError_t rc = p.rows == 128 ? launch_tiles<128, 2, 2, 2, WT, GATED, kSums>(k, p.parts, stream)
                                        : launch_tiles<64, 2, 2, 3, WT, GATED, kSums>(k, p.parts, stream);
    return rc != hipSuccess ? rc : launch_finish<MODE, GATED>(k, p.parts, stream);
}

// The same on weights as they lie, through the kernel for few rows where it is the faster.
template <bool GATED>
hipError_t forward_product(const LinearK &k, int act, int64_t rows, float *sums, hipStream_t stream) {
    if (!few_rows(rows, (int64_t)k.k * 2)) return product<false, GATED, kPlain>(k, rows, sums, stream);
    FewRowsArgs f = {};
    f.x = k.x;
    f.w = k.w;
    f.residual = k.residual;
    f.out = k.out;
    f.rows = (int)rows;
    f.n = k.n;
    f.k = k.k;
    f.act = act;
    return launch_few_rows(f, stream);
}

}  // namespace

size_t gated_ffn_sums_bytes(int64_t rows, int hidden, int inter, bool backward) {
    const auto of = [&](int n, int k) { return sums_bytes(plan_of(rows, n, k, backward), rows, n); };
    return backward ? std::max({of(inter, hidden), of(hidden, 2 * inter),
                                wgrad_pair_sums_bytes(rows, 2 * inter, hidden, hidden, inter)})
                    : std::max(of(2 * inter, hidden), of(hidden, inter));
}

hipError_t launch_gated_ffn(const FfnArgs &a, hipStream_t stream) {
    LinearK k = {};
    k.x = (const uint8_t *)a.x;
    k.w = (const uint8_t *)a.w1;
    k.out = (uint16_t *)a.h;
    k.kept = (uint16_t *)a.z;
    k.n = 2 * a.inter;
    k.k = a.hidden;
    k.m = a.inter;
    k.kind = act_kind(a.act);
    const hipError_t rc = a.z ? product<false, true, kKeep>(k, a.rows, a.sums, stream)
                              : forward_product<true>(k, a.act, a.rows, a.sums, stream);
    if (rc != hipSuccess) return rc;
    LinearK d = {};
    d.x = (const uint8_t *)a.h;
    d.w = (const uint8_t *)a.w2;
    d.residual = (const uint16_t *)a.residual;
    d.out = (uint16_t *)a.out;
    d.n = d.m = a.hidden;
    d.k = a.inter;
    return forward_product<false>(d, EP_ACT_NONE, a.rows, a.sums, stream);
}

hipError_t launch_gated_ffn_backward(const FfnBackwardArgs &a, hipStream_t stream) {
    if (a.rows > 0) {
        LinearK k = {};
        k.x = (const uint8_t *)a.dout;
        k.w = (const uint8_t *)a.w2;
        k.out = (uint16_t *)a.dz;
        k.pre = (const uint16_t *)a.z;
        k.h = (uint16_t *)a.h;
        k.n = k.m = a.inter;
        k.k = a.hidden;
        k.kind = act_kind(a.act);
        const hipError_t rc = product<true, false, kBackward>(k, a.rows, a.sums, stream);
        if (rc != hipSuccess) return rc;
    }
    auto wgrad = [&](const void *dy, int n, const void *x, int k, const void *dw_in, void *dw) {
        WgradArgs g = {};
        g.seg.E = 1;
        g.seg.num_rows = g.seg.pairs = g.seg.each = a.rows;
        g.dy = dy;
        g.x = x;
        g.dw_in = dw_in;
        g.dw = dw;
        g.n = n;
        g.k = k;
        g.bf16_out = a.bf16_out;
        return g;
    };
    const hipError_t rc = launch_wgrad_pair(wgrad(a.dz, 2 * a.inter, a.x, a.hidden, a.dw1_in, a.dw1),
                                            wgrad(a.dout, a.hidden, a.h, a.inter, a.dw2_in, a.dw2), a.sums, stream);
    if (rc != hipSuccess || !a.dx || a.rows == 0) return rc;
    LinearK d = {};
    d.x = (const uint8_t *)a.dz;
    d.w = (const uint8_t *)a.w1;
    d.out = (uint16_t *)a.dx;
    d.n = d.m = a.hidden;
    d.k = 2 * a.inter;
    return product<true, false, kPlain>(d, a.rows, a.sums, stream);
}

}  // namespace ep
