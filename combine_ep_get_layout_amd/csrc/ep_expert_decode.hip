// A whole mixture-of-experts layer for a few tokens, in two kernels:
//   h[t,k] = act(W1[e] x[t] + b1[e])                       (rounded to bf16)
//   out[t] = res0 + res1 + sum_k w[t,k] (W2[e] h[t,k] + b2[e]),  e = topk_idx[t,k]
// There is no layout and no permutation: the pairs of an expert are found in
// topk_idx by every workgroup that needs them.
//
// The layer reads every chosen expert's weights once (more than 16 pairs of
// one expert: once per 16, from the caches after the first) and little else,
// so it is bound by HBM.  The weights are the matrix instruction's first
// operand and go from memory to registers in its layout, 16 rows x 64 bytes a
// load; the pairs are the other, 16 columns of which most are empty.
//
// First kernel: a workgroup takes one expert and 16 columns of h (16 gate and
// 16 up rows of W1); its four waves split the sum over the hidden channels and
// add up in LDS in wave order.
// Second kernel: a workgroup takes 16 channels of the output and all pairs:
// its waves take the chosen experts in turn, every pair's 16 sums go to LDS in
// fp32, and the tokens' weighted sums are formed from there in ascending k, as
// ep_combine forms them: no atomics, no rounding between the two, and a
// token's result does not depend on the other tokens of the batch.
#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kMaxPairs = EP_MAX_DECODE_PAIRS;

struct DecodeK {
    MoeDecodeArgs a;
    int pairs;
    int by_pair;      // first kernel: a workgroup's expert is that of pair blockIdx.y
};

// One matrix-instruction operand of 32 channels: 8 consecutive bf16 per lane.
// Row pointers are per lane; channels at or past n are zeros.
template <bool FP8>
struct Weights;

template <>
struct Weights<false> {
    const uint16_t *row;
    __device__ __forceinline__ Weights(const void *w, const uint8_t *, int64_t r, int n)
        : row((const uint16_t *)w + r * n) {}
    // channels c + 32 j + 8 q .. + 7 for j = 0..3, c a multiple of 128
    __device__ __forceinline__ void load(int c, int q, int n, ep_u32x4 *v, float *) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = c + j * 32 + q * 8;
            v[j] = at < n ? load_nt((const ep_u32x4 *)(row + at)) : ep_u32x4{0, 0, 0, 0};
        }
    }
    static __device__ __forceinline__ ep_bf16x8 operand(const ep_u32x4 *v, float, int j) {
        return __builtin_bit_cast(ep_bf16x8, v[j]);
    }
    // first channel of operand j's 8
    static __device__ __forceinline__ int channel(int c, int j, int q) { return c + j * 32 + q * 8; }
    static constexpr int kLoads = 4;
};

template <>
struct Weights<true> {
    const uint8_t *row, *scale;
    __device__ __forceinline__ Weights(const void *w, const uint8_t *s, int64_t r, int n)
        : row((const uint8_t *)w + r * n), scale(s + r * (n / kFp8Group)) {}
    // channels c + 64 i + 16 q .. + 15 for i = 0, 1
    __device__ __forceinline__ void load(int c, int q, int n, ep_u32x4 *v, float *s) const {
        v[0] = load_nt((const ep_u32x4 *)(row + c + q * 16));
        v[1] = load_nt((const ep_u32x4 *)(row + c + 64 + q * 16));
        *s = ue8m0_value(scale[c / kFp8Group]);
    }
    static __device__ __forceinline__ ep_bf16x8 operand(const ep_u32x4 *v, float s, int j) {
        const uint32_t lo = v[j >> 1][(j & 1) * 2], hi = v[j >> 1][(j & 1) * 2 + 1];
        ep_u32x4 r;
        r.x = fp8_pair_bf16<false>(lo, s);
        r.y = fp8_pair_bf16<true>(lo, s);
        r.z = fp8_pair_bf16<false>(hi, s);
        r.w = fp8_pair_bf16<true>(hi, s);
        return __builtin_bit_cast(ep_bf16x8, r);
    }
    static __device__ __forceinline__ int channel(int c, int j, int q) {
        return c + (j >> 1) * 64 + q * 16 + (j & 1) * 8;
    }
    static constexpr int kLoads = 2;
};

// The pairs of expert e, ascending, to list[]; returns how many.  `red` is LDS
// of 8 ints; the whole workgroup calls this.
template <int THREADS>
__device__ int pairs_of(const int64_t *topk_idx, int pairs, int64_t e, int16_t *list, int *red) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int count = 0;
    for (int p0 = 0; p0 < pairs; p0 += THREADS) {
        const int p = p0 + tid;
        const bool mine = p < pairs && topk_idx[p] == e;
        const uint64_t m = __ballot(mine);
        if (lane == 0) red[wave] = __popcll(m);
        __syncthreads();
        int base = count;
        for (int w = 0; w < THREADS / 64; ++w) {
            const int v = red[w];
            if (w < wave) base += v;
            count += v;
        }
        if (mine) list[base + __popcll(m & lanes_below())] = (int16_t)p;
        __syncthreads();
    }
    return count;
}

template <bool FP8, bool GATED>
__global__ __launch_bounds__(256) void moe_decode_up_kernel(DecodeK k) {
    const MoeDecodeArgs &a = k.a;
    __shared__ int16_t list[kMaxPairs];
    __shared__ int red[8];
    __shared__ float part[4][GATED ? 2 : 1][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, q = lane >> 4;
    const int64_t e = k.by_pair ? a.topk_idx[blockIdx.y] : (int64_t)blockIdx.y;
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0) {
        bool bad = false;
        for (int p = tid; p < k.pairs; p += 256) bad |= a.topk_idx[p] < -1 || a.topk_idx[p] >= a.E;
        if (bad) atomicOr(a.status, kDevBadExpert);
    }
    if (e < 0 || e >= a.E) return;
    const int count = pairs_of<256>(a.topk_idx, k.pairs, e, list, red);
    // by pair: only the expert's first pair computes
    if (count == 0 || (k.by_pair && list[0] != (int)blockIdx.y)) return;

    const int I = a.I, H = a.H, n1 = GATED ? 2 * I : I;
    const int col0 = blockIdx.x * 16;
    const int wcol = min(col0 + l16, I - 1);
    const Weights<FP8> wg(a.w1, a.w1_scales, e * n1 + wcol, H);
    const Weights<FP8> wu(a.w1, a.w1_scales, e * n1 + (GATED ? I : 0) + wcol, H);
    // the waves take the 128-channel steps in turn
    for (int g0 = 0; g0 < count; g0 += 16) {
        const int live = min(16, count - g0);
        const int pair = l16 < live ? list[g0 + l16] : 0;
        const uint16_t *x = (const uint16_t *)a.x + (int64_t)(pair / a.K) * H;
        ep_f32x4 acc_g = {0, 0, 0, 0}, acc_u = {0, 0, 0, 0};
#pragma unroll 2
        for (int c = wave * 128; c < H; c += 512) {
            ep_u32x4 vg[4], vu[4];
            float sg = 0.0f, su = 0.0f;
            wg.load(c, q, H, vg, &sg);
            if (GATED) wu.load(c, q, H, vu, &su);
            ep_u32x4 xv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = Weights<FP8>::channel(c, j, q);
                xv[j] = l16 < live && at < H ? *(const ep_u32x4 *)(x + at) : ep_u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const ep_bf16x8 b = __builtin_bit_cast(ep_bf16x8, xv[j]);
                acc_g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Weights<FP8>::operand(vg, sg, j), b, acc_g, 0, 0, 0);
                if (GATED)
                    acc_u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Weights<FP8>::operand(vu, su, j), b, acc_u, 0, 0, 0);
            }
        }
        pin(acc_g);
        pin(acc_u);
        for (int i = 0; i < 4; ++i) {
            part[wave][0][4 * q + i][l16] = acc_g[i];
            if (GATED) part[wave][GATED ? 1 : 0][4 * q + i][l16] = acc_u[i];
        }
        __syncthreads();
        {
            // one column of one pair per thread
            const int c = tid & 15, r = tid >> 4;
            if (r < live && col0 + c < I) {
                float z[2] = {0.0f, 0.0f};
                for (int s = 0; s < (GATED ? 2 : 1); ++s) {
                    for (int w = 0; w < 4; ++w) z[s] += part[w][s][c][r];
                    if (a.bias1)
                        z[s] += __uint_as_float((uint32_t)((const uint16_t *)a.bias1)[e * n1 + s * I + col0 + c] << 16);
                }
                float y = a.kind == 1 ? act_value<1>(z[0]) : a.kind == 2 ? act_value<2>(z[0]) : z[0];
                if (GATED) y *= z[1];
                // bf16: the type a dispatch would carry and the matrix
                // instruction takes; the one rounding between x and out
                ((__bf16 *)a.h)[(int64_t)list[g0 + r] * I + col0 + c] = (__bf16)y;
            }
        }
        __syncthreads();
    }
}

// Waves of the second kernel.
constexpr int kDownWaves = 8;

template <bool FP8>
__global__ __launch_bounds__(64 * kDownWaves) void moe_decode_down_kernel(DecodeK k) {
    const MoeDecodeArgs &a = k.a;
    extern __shared__ __align__(16) float y[];             // [pairs][16]
    int *first = (int *)(y + k.pairs * 16);                // [E] first pair of an expert
    int16_t *id = (int16_t *)(first + a.E);                // [pairs] expert of a pair
    int16_t *leader = id + ((k.pairs + 7) & ~7);           // [pairs] the experts' first pairs
    int16_t *mine = leader + ((k.pairs + 7) & ~7) + (threadIdx.x >> 6) * 16;   // a wave's 16 pairs
    __shared__ int red[kDownWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, q = lane >> 4;
    constexpr int kThreads = 64 * kDownWaves;
    const int H = a.H, I = a.I;
    const int h0 = blockIdx.x * 16;

    for (int e = tid; e < a.E; e += kThreads) first[e] = k.pairs;
    __syncthreads();
    for (int p = tid; p < k.pairs; p += kThreads) {
        const int64_t e = a.topk_idx[p];
        const bool ok = e >= 0 && e < a.E;
        id[p] = ok ? (int16_t)e : (int16_t)-1;
        if (ok) atomicMin(&first[e], p);
    }
    __syncthreads();
    int experts = 0;
    for (int p0 = 0; p0 < k.pairs; p0 += kThreads) {
        const int p = p0 + tid;
        const bool lead = p < k.pairs && id[p] >= 0 && first[id[p]] == p;
        const uint64_t m = __ballot(lead);
        if (lane == 0) red[wave] = __popcll(m);
        __syncthreads();
        int base = experts;
        for (int w = 0; w < kDownWaves; ++w) {
            const int v = red[w];
            if (w < wave) base += v;
            experts += v;
        }
        if (lead) leader[base + __popcll(m & lanes_below())] = (int16_t)p;
        __syncthreads();
    }

    const int wrow = min(h0 + l16, H - 1);
    for (int s = wave; s < experts; s += kDownWaves) {
        const int p0 = leader[s];
        const int e = id[p0];
        const Weights<FP8> w(a.w2, a.w2_scales, (int64_t)e * H + wrow, I);
        // the expert's pairs, 16 at a time in ascending order
        int from = p0;
        while (from < k.pairs) {
            int live = 0;
            int p = from;
            for (; p < k.pairs && live < 16; p += 64) {
                const bool hit = p + lane < k.pairs && id[p + lane] == e;
                const uint64_t m = __ballot(hit);
                const int at = live + __popcll(m & lanes_below());
                if (hit && at < 16) mine[at] = (int16_t)(p + lane);
                live += __popcll(m);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            const int n = min(live, 16);
            if (n == 0) break;
            const int pair = mine[l16 < n ? l16 : 0];
            const int last = wave_uniform((int)mine[n - 1]);
            const uint16_t *h = (const uint16_t *)a.h + (int64_t)pair * I;
            ep_f32x4 acc = {0, 0, 0, 0};
#pragma unroll 4
            for (int c = 0; c < I; c += 128) {
                ep_u32x4 v[4], hv[4];
                float sc = 0.0f;
                w.load(c, q, I, v, &sc);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = Weights<FP8>::channel(c, j, q);
                    hv[j] = l16 < n && at < I ? *(const ep_u32x4 *)(h + at) : ep_u32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        Weights<FP8>::operand(v, sc, j), __builtin_bit_cast(ep_bf16x8, hv[j]), acc, 0, 0, 0);
            }
            pin(acc);
            if (a.bias2) {
                for (int i = 0; i < 4; ++i)
                    if (h0 + 4 * q + i < H)
                        acc[i] += __uint_as_float((uint32_t)((const uint16_t *)a.bias2)[(int64_t)e * H + h0 + 4 * q + i] << 16);
            }
            if (l16 < n) *(ep_f32x4 *)(y + pair * 16 + 4 * q) = acc;
            if (live < 16) break;        // all pairs were seen
            from = last + 1;
        }
    }
    __syncthreads();

    // out[t, h0 .. h0 + 15] in pieces of 8 channels
    for (int i = tid; i < a.T * 2; i += kThreads) {
        const int t = i >> 1, c = (i & 1) * 8;
        if (h0 + c >= H) continue;
        const int64_t o = (int64_t)t * H + h0 + c;
        float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int b = 0; b < 2; ++b) {
            const void *r = b ? a.res1 : a.res0;
            if (!r) continue;
            const ep_u32x4 v = *(const ep_u32x4 *)((const uint16_t *)r + o);
            for (int j = 0; j < 8; ++j) s[j] += (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
        }
        for (int kk = 0; kk < a.K; ++kk) {
            const int p = t * a.K + kk;
            if (id[p] < 0) continue;
            const float w = a.topk_weights ? a.topk_weights[p] : 1.0f;
            for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(w, y[p * 16 + c + j], s[j]);
        }
        ep_u32x4 v;
        for (int j = 0; j < 4; ++j) v[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
        *(ep_u32x4 *)((uint16_t *)a.out + o) = v;
    }
}

size_t down_lds(int pairs, int E) {
    return (size_t)pairs * 64 + (size_t)E * 4 + (size_t)((pairs + 7) & ~7) * 4 + kDownWaves * 32;
}

}  // namespace

hipError_t launch_moe_decode(const MoeDecodeArgs &a, hipStream_t stream) {
    DecodeK k = {};
    k.a = a;
    k.pairs = a.T * a.K;
    k.by_pair = k.pairs <= a.E ? 1 : 0;
    const dim3 up((unsigned)((a.I + 15) / 16), (unsigned)(k.by_pair ? k.pairs : a.E));
    const dim3 down((unsigned)((a.H + 15) / 16));
    const size_t lds = down_lds(k.pairs, a.E);
    if (a.fp8) {
        if (a.gated) moe_decode_up_kernel<true, true><<<up, dim3(256), 0, stream>>>(k);
        else moe_decode_up_kernel<true, false><<<up, dim3(256), 0, stream>>>(k);
        moe_decode_down_kernel<true><<<down, dim3(64 * kDownWaves), lds, stream>>>(k);
    } else {
        if (a.gated) moe_decode_up_kernel<false, true><<<up, dim3(256), 0, stream>>>(k);
        else moe_decode_up_kernel<false, false><<<up, dim3(256), 0, stream>>>(k);
        moe_decode_down_kernel<false><<<down, dim3(64 * kDownWaves), lds, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace ep
