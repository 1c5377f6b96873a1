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

SegmentRows dense(int64_t rows) {
    SegmentRows s = {};
    s.E = 1;
    s.num_rows = s.pairs = s.each = rows;
    return s;
}

// A product with an epilogue of its own: z kept (gated columns), or dz and h
// from transposed weights.
template <bool WT, bool GATED, int MODE>
hipError_t launch_mode(LinearK &k, hipStream_t stream) {
    const RowTile tile = row_tile(k.seg, k.m, GATED, WT);
    k.col_tiles = (k.m + tile.cols - 1) / tile.cols;
    const int64_t grid = grid_of(k.seg, k.col_tiles, tile.rows);
    if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid);
    if (tile.rows == 256) expert_linear_wide_kernel<kBf16, WT, GATED, MODE><<<g, 256, 0, stream>>>(k);
    else if (tile.rows == 192) expert_linear_kernel<192, 2, 4, 2, kBf16, WT, GATED, MODE><<<g, 512, 0, stream>>>(k);
    else if (tile.rows == 128) expert_linear_kernel<128, 2, 4, 3, kBf16, WT, GATED, MODE><<<g, 512, 0, stream>>>(k);
    else if constexpr (!WT) expert_linear_kernel<64, 4, 1, 4, kBf16, WT, GATED, MODE><<<g, 256, 0, stream>>>(k);
    return hipGetLastError();
}

hipError_t product(const void *x, const void *w, int n, int k, int act, const void *residual,
                   bool transposed, int64_t rows, void *out, hipStream_t stream) {
    if (!transposed && rows <= kFewRows) {
        FewRowsArgs f = {};
        f.x = x;
        f.w = w;
        f.residual = residual;
        f.out = out;
        f.rows = (int)rows;
        f.n = n;
        f.k = k;
        f.act = act;
        return launch_few_rows(f, stream);
    }
    LinearArgs a = {};
    a.seg = dense(rows);
    a.x = x;
    a.w = w;
    a.residual = residual;
    a.out = out;
    a.n = n;
    a.k = k;
    a.act = act;
    a.transposed = transposed;
    return launch_expert_linear(a, stream);
}

}  // namespace

hipError_t launch_gated_ffn(const FfnArgs &a, hipStream_t stream) {
    hipError_t rc;
    if (a.z) {
        LinearK k = {};
        k.seg = dense(a.rows);
        k.x = (const uint8_t *)a.x;
        k.w = (const uint8_t *)a.w1;
        k.out = (uint16_t *)a.h;
        k.kept = (uint16_t *)a.z;
        k.n = 2 * a.inter;
        k.k = a.hidden;
        k.m = a.inter;
        k.kind = act_kind(a.act);
        rc = launch_mode<false, true, kKeep>(k, stream);
    } else {
        rc = product(a.x, a.w1, 2 * a.inter, a.hidden, a.act, nullptr, false, a.rows, a.h, stream);
    }
    if (rc != hipSuccess) return rc;
    return product(a.h, a.w2, a.hidden, a.inter, EP_ACT_NONE, a.residual, false, a.rows, a.out, stream);
}

hipError_t launch_gated_ffn_backward(const FfnBackwardArgs &a, hipStream_t stream) {
    if (a.rows > 0) {
        LinearK k = {};
        k.seg = dense(a.rows);
        k.x = (const uint8_t *)a.dout;
        k.w = (const uint8_t *)a.w2;
        k.out = (uint16_t *)a.dz;
        k.pre = (const uint16_t *)a.z;
        k.h = (uint16_t *)a.h;
        k.n = k.m = a.inter;
        k.k = a.hidden;
        k.kind = act_kind(a.act);
        const hipError_t rc = launch_mode<true, false, kBackward>(k, stream);
        if (rc != hipSuccess) return rc;
    }
    auto wgrad = [&](const void *dy, int n, const void *x, int k, const void *dw_in, void *dw) {
        WgradArgs g = {};
        g.seg = dense(a.rows);
        g.dy = dy;
        g.x = x;
        g.dw_in = dw_in;
        g.dw = dw;
        g.n = n;
        g.k = k;
        g.bf16_out = a.bf16_out;
        return launch_expert_wgrad(g, stream);
    };
    hipError_t rc = wgrad(a.dout, a.hidden, a.h, a.inter, a.dw2_in, a.dw2);
    if (rc != hipSuccess) return rc;
    rc = wgrad(a.dz, 2 * a.inter, a.x, a.hidden, a.dw1_in, a.dw1);
    if (rc != hipSuccess || !a.dx || a.rows == 0) return rc;
    return product(a.dz, a.w1, a.hidden, 2 * a.inter, EP_ACT_NONE, nullptr, true, a.rows, a.dx, stream);
}

}  // namespace ep
