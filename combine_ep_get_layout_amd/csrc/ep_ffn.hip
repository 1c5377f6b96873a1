// The gated feed-forward block that every token passes (a shared expert), and
// its gradients: dense rows through the matrix kernels of the experts.
//
// Forward: h = f(x Wg^T) * (x Wu^T) by one product whose tiles hold gate and up
// columns together, then out = h W2^T + residual.  Few rows go through a kernel of
// their own, bound by reading the weights.
// Backward: the product dout W2 makes dh in its accumulators; its epilogue reads z
// and writes dz = [dgate | dup] and h, so that dh is never stored or rounded.  Then
// dW2 = dout^T h, dW1 = dz^T x and dx = dz W1.  dz and h are rounded to bf16, the
// type that the matrix instructions of these products take.
//
// 16384 tokens 7168/2048, back to back on one card: forward 1.02 to 1.06 ms (1.36 to
// 1.41 PFLOP/s; a library product reaches 1.54), backward 2.23 to 2.34 (1.23 to 1.29), bound by
// the matrix instructions under the power limit.
#include "ep_linear_device.h"
#include "ep_wgrad_device.h"

namespace ep {

namespace {

SegmentRows dense(int64_t rows) {
    SegmentRows s = {};
    s.E = 1;
    s.num_rows = s.pairs = s.each = rows;
    return s;
}

constexpr int kStep = 64;        // channels of a step of the matrix kernels

DensePlan plan_of(int64_t rows, int n, int k, bool transposed) {
    return dense_plan(rows, n, (k + kStep - 1) / kStep, transposed);
}

template <int BM, int WM, int WN, int NS, bool WT, bool GATED, int MODE>
hipError_t launch_tiles(LinearK &k, int parts, hipStream_t stream) {
    const int per = GATED ? WN * 32 : WN * 64;
    k.col_tiles = (k.m + per - 1) / per;
    const int64_t grid = grid_of(k.seg, k.col_tiles, BM);
    if (!launchable(grid, 64 * WM * WN)) return hipErrorInvalidConfiguration;
    expert_linear_kernel<BM, WM, WN, NS, kBf16, WT, GATED, MODE>
        <<<dim3((unsigned)grid, parts), 64 * WM * WN, 0, stream>>>(k);
    return hipGetLastError();
}

// A product of dense rows with the epilogue MODE; `sums` holds what its plan asks for.
template <bool WT, bool GATED, int MODE>
hipError_t product(LinearK k, int64_t rows, float *sums, hipStream_t stream) {
    k.seg = dense(rows);
    const DensePlan p = plan_of(rows, k.n, k.k, WT);
    if (p.rows == 256) {
        const int per = GATED ? kBN / 2 : kBN;
        k.col_tiles = (k.m + per - 1) / per;
        const int64_t grid = grid_of(k.seg, k.col_tiles, 256);
        if (!launchable(grid, 256)) return hipErrorInvalidConfiguration;
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

// The gradients from the parts that runs of rows left in fp32, added in order: 8
// elements a thread, of the first product, then of the second.
struct WgradSums {
    const float *sums[2];        // [parts, count]
    const void *dw_in[2];
    void *dw[2];
    int64_t count[2];            // elements of a gradient, a multiple of 8
    int parts, bf16_out;
};

__global__ __launch_bounds__(256) void wgrad_finish_kernel(WgradSums a) {
    int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const bool second = at >= a.count[0];
    if (second) at -= a.count[0];
    const int64_t count = second ? a.count[1] : a.count[0];
    if (at >= count) return;
    const float *p = (second ? a.sums[1] : a.sums[0]) + at;
    const void *in = second ? a.dw_in[1] : a.dw_in[0];
    void *out = second ? a.dw[1] : a.dw[0];
    ep_f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < a.parts; ++s) {
        lo += *(const ep_f32x4 *)(p + s * count);
        hi += *(const ep_f32x4 *)(p + s * count + 4);
    }
    if (a.bf16_out) {
        if (in) {
            const ep_u32x4 v = *(const ep_u32x4 *)((const uint16_t *)in + at);
            lo += ep_f32x4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
            hi += ep_f32x4{bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
        }
        *(ep_u32x4 *)((uint16_t *)out + at) =
            ep_u32x4{pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
    } else {
        if (in) {
            lo += *(const ep_f32x4 *)((const float *)in + at);
            hi += *(const ep_f32x4 *)((const float *)in + at + 4);
        }
        *(ep_f32x4 *)((float *)out + at) = lo;
        *(ep_f32x4 *)((float *)out + at + 4) = hi;
    }
}

// How the two gradients of dense rows are divided: tiles of 256 or of 128 rows and
// columns, and, where tiles are few, runs of rows whose sums pass through memory.  By
// what they are expected to take, from measured times: a round of 256 tiles of 256 x
// 256 takes 1.55 us a step of 64 rows and 13 us for its ends, a round of 512 of 128 x
// 128 (two on a compute unit) 1.6 us and 4.5 us, 256 or fewer of them 1.0 us; the sums
// 5 us for their launch and 4 bytes an element and run, written and read, at 4 TB/s.
struct PairPlan { int edge, parts; int64_t each; };

constexpr int kRuns[] = {1, 2, 3, 4, 6, 8};

// Runs of `each` rows, if `rows` rows are cut into `parts` of them (0: they are not):
// of 256 rows at least, and with sums of 256 MB at most (bounds of the choice and of
// the workspace, whose other sides are not measured).
int64_t run_of(int64_t rows, int parts, double elements) {
    if (parts == 1) return rows;
    const int64_t each = ((rows + parts - 1) / parts + kRows - 1) / kRows * kRows;
    return each < 256 || parts * elements > 64e6 ? 0 : each;
}

PairPlan pair_plan(int64_t rows, int n0, int k0, int n1, int k1) {
    const double elements = (double)n0 * k0 + (double)n1 * k1;
    PairPlan best = {kT, 1, rows};
    double least = 1e300;
    for (const int T : {kT, kWT}) {
        auto tiles = [&](int n, int k) { return (int64_t)((n + T - 1) / T) * ((k + T - 1) / T); };
        const int64_t all = tiles(n0, k0) + tiles(n1, k1);
        for (const int parts : kRuns) {
            const int64_t each = run_of(rows, parts, elements);
            if (parts > 1 && (each == 0 || (rows + each - 1) / each != parts)) continue;
            const int64_t total = all * parts, round = T == kWT ? 256 : 512;
            const double steps = (double)((each + kRows - 1) / kRows);
            const double step = T == kWT ? 1.55 : total <= 256 ? 1.0 : 1.6;
            double us = (double)((total + round - 1) / round) * (steps * step + (T == kWT ? 13.0 : 4.5));
            if (parts > 1) us += 5.0 + parts * elements * 8.0 / 4e6;
            if (us < least) {
                least = us;
                best = {T, parts, each};
            }
        }
    }
    return best;
}

// What the backward pass computes from dz and h: both weight gradients and dx, in one
// launch.  None of the three needs another's result, and they fill each other's rounds
// and waits: 333 tokens 1024/1408 16 us, one after another 25; 16384 tokens 7168/2048 1.93
// ms and 1.96.  What takes a workgroup longest goes first: the weight gradients' 256 x 256
// tiles of many rows, or dx, whose contraction takes few tokens as long as many.
struct Gradients {
    WgradPair w;
    LinearK x;
    int w_blocks, x_blocks;      // workgroups of the weight gradients; of a part of dx
    int parts;                   // of dx
};

__global__ __launch_bounds__(256, 1) void gradients_wide_kernel(Gradients p) {
    __shared__ __align__(1024) uint8_t lds[std::max(kLinearWideLds, kWgradWideLds<false>)];
    __shared__ int red[16];
    if ((int)blockIdx.x >= p.w_blocks) {
        linear_wide_tile<kBf16, true, false, kPlain>(p.x, blockIdx.x - p.w_blocks, lds, red);
        return;
    }
    WgradK a;
    uint32_t tile;
    if (pick(p.w, blockIdx.x, &a, &tile)) wgrad_wide_tile<false, false>(a, tile, lds);
}

// dx in tiles of 64 x 128 or 128 x 128, whole or in parts.
template <int BM, int NS, int MODE>
__global__ __launch_bounds__(256, 2) void gradients_kernel(Gradients p) {
    __shared__ __align__(1024) uint8_t lds[std::max(kLinearLds<BM, 2, 2, NS>, kWgradLds)];
    __shared__ int red[16];
    const int block = blockIdx.x - p.x_blocks * p.parts;
    if (block < 0) {
        const int part = MODE == kSums ? (int)blockIdx.x / p.x_blocks : 0;
        linear_tile<BM, 2, 2, NS, kBf16, true, false, MODE>(p.x, blockIdx.x - part * p.x_blocks, part, lds, red);
        return;
    }
    WgradK a;
    uint32_t tile;
    if (pick(p.w, block, &a, &tile)) wgrad_tile<false, false>(a, tile, lds);
}

// The weight gradients alone: without dx, or where its tiles have no kernel with theirs.
__global__ __launch_bounds__(256, 1) void wgrad_wide_pair_kernel(WgradPair p) {
    __shared__ __align__(1024) uint8_t lds[kWgradWideLds<false>];
    WgradK a;
    uint32_t tile;
    if (pick(p, blockIdx.x, &a, &tile)) wgrad_wide_tile<false, false>(a, tile, lds);
}

__global__ __launch_bounds__(256, 2) void wgrad_pair_kernel(WgradPair p) {
    __shared__ __align__(1024) uint8_t lds[kWgradLds];
    WgradK a;
    uint32_t tile;
    if (pick(p, blockIdx.x, &a, &tile)) wgrad_tile<false, false>(a, tile, lds);
}

}  // namespace

size_t gated_ffn_sums_bytes(int64_t rows, int hidden, int inter, bool backward) {
    const auto of = [&](int n, int k) { return sums_bytes(plan_of(rows, n, k, backward), rows, n); };
    if (!backward) return std::max(of(2 * inter, hidden), of(hidden, inter));
    // dh's are read before the others' are written
    const PairPlan p = pair_plan(rows, 2 * inter, hidden, hidden, inter);
    const size_t weights = p.parts > 1 ? (size_t)p.parts * 3 * hidden * inter * 4 : 0;
    return std::max(of(inter, hidden), of(hidden, 2 * inter) + weights);
}

size_t gated_ffn_sums_most(int64_t rows, int hidden, int inter, bool backward) {
    const auto of = [&](int n, int k) { return sums_most(rows, n, (k + kStep - 1) / kStep); };
    if (!backward) return std::max(of(2 * inter, hidden), of(hidden, inter));
    // (a run grows with the rows, so what cuts fewer rows cuts these)
    const double elements = 3.0 * hidden * inter;
    int parts = 0;
    for (const int p : kRuns)
        if (p > 1 && run_of(rows, p, elements) > 0) parts = p;
    return std::max(of(inter, hidden), of(hidden, 2 * inter) + (size_t)parts * 3 * hidden * inter * 4);
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
        g.seg = dense(a.rows);
        g.dy = dy;
        g.x = x;
        g.dw_in = dw_in;
        g.dw = dw;
        g.n = n;
        g.k = k;
        g.bf16_out = a.bf16_out;
        return g;
    };
    const PairPlan plan = pair_plan(a.rows, 2 * a.inter, a.hidden, a.hidden, a.inter);
    Gradients p = {};
    p.w.a = kernel_args(wgrad(a.dz, 2 * a.inter, a.x, a.hidden, a.dw1_in, a.dw1), plan.edge);
    p.w.b = kernel_args(wgrad(a.dout, a.hidden, a.h, a.inter, a.dw2_in, a.dw2), plan.edge);
    WgradSums f = {};
    // the sums of the weight gradients lie behind those of dx
    const DensePlan dx = plan_of(a.rows, a.hidden, 2 * a.inter, true);
    if (plan.parts > 1) {
        f.count[0] = (int64_t)2 * a.inter * a.hidden;
        f.count[1] = (int64_t)a.hidden * a.inter;
        f.parts = plan.parts;
        f.bf16_out = a.bf16_out ? 1 : 0;
        float *sums = a.sums + sums_bytes(dx, a.rows, a.hidden) / 4;
        WgradK *k[2] = {&p.w.a, &p.w.b};
        for (int i = 0; i < 2; ++i) {
            f.dw_in[i] = k[i]->dw_in;
            f.dw[i] = k[i]->dw;
            f.sums[i] = sums;
            k[i]->seg.E = plan.parts;
            k[i]->seg.each = plan.each;
            k[i]->dw_in = nullptr;
            k[i]->dw = sums;
            k[i]->bf16_out = 0;
            sums += plan.parts * f.count[i];
        }
    }
    const auto tiles = [](const WgradK &k) { return (int64_t)k.seg.E * k.tiles_n * k.tiles_k; };
    const int64_t all = tiles(p.w.a) + tiles(p.w.b), w_blocks = (all + 255) / 256 * 256;
    p.w.first = (uint32_t)tiles(p.w.a);
    p.w.tiles = (uint32_t)all;
    p.w_blocks = (int)w_blocks;
    p.parts = dx.parts;
    p.x.seg = dense(a.rows);
    p.x.x = (const uint8_t *)a.dz;
    p.x.w = (const uint8_t *)a.w1;
    p.x.out = (uint16_t *)a.dx;
    p.x.n = p.x.m = a.hidden;
    p.x.k = 2 * a.inter;
    p.x.sums = a.sums;
    p.x.split = dx.split;
    p.x.col_tiles = (a.hidden + dx.cols - 1) / dx.cols;
    p.x_blocks = (int)grid_of(p.x.seg, p.x.col_tiles, dx.rows);
    const bool with_dx = a.dx && a.rows > 0, wide = plan.edge == kWT;
    const bool together = with_dx && wide == (dx.rows == 256);
    const int64_t grid = together ? w_blocks + (int64_t)p.x_blocks * dx.parts : w_blocks;
    // (x_blocks, in 32 bits, too)
    if (!launchable(grid, 256) || !launchable((int64_t)p.x.col_tiles * (a.rows / dx.rows + 1), 256))
        return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), t(256);
    if (!together) {
        if (wide) wgrad_wide_pair_kernel<<<g, t, 0, stream>>>(p.w);
        else wgrad_pair_kernel<<<g, t, 0, stream>>>(p.w);
    } else if (wide) {
        gradients_wide_kernel<<<g, t, 0, stream>>>(p);
    } else if (dx.parts > 1) {
        if (dx.rows == 128) gradients_kernel<128, 2, kSums><<<g, t, 0, stream>>>(p);
        else gradients_kernel<64, 3, kSums><<<g, t, 0, stream>>>(p);
    } else {
        if (dx.rows == 128) gradients_kernel<128, 2, kPlain><<<g, t, 0, stream>>>(p);
        else gradients_kernel<64, 3, kPlain><<<g, t, 0, stream>>>(p);
    }
    hipError_t rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
    if (together && dx.parts > 1) rc = launch_finish<kPlain, false>(p.x, dx.parts, stream);
    if (rc != hipSuccess) return rc;
    if (plan.parts > 1) {
        const int64_t threads = (f.count[0] + f.count[1]) / 8;
        wgrad_finish_kernel<<<dim3((unsigned)((threads + 255) / 256)), t, 0, stream>>>(f);
        rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    return with_dx && !together ? product<true, false, kPlain>(p.x, a.rows, a.sums, stream) : hipSuccess;
}

}  // namespace ep
