// A whole mixture-of-experts layer for a few tokens, in two kernels:
//   h[t,k] = act(W1[e] x[t] + b1[e])                       (16 significant bits)
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
// Second kernel: a workgroup takes 32 channels of the output and all pairs, or,
// where the output has few channels, those of a run of tokens (h is read once per
// workgroup; 16 channels read it twice as often: 128 tokens of fp8
// weights took 1026 us against 773): its waves take the chosen experts in turn,
// every pair's 32 sums go to LDS in fp32, and the tokens' weighted sums are
// formed from there in ascending k, as ep_combine forms them: no atomics, no
// rounding between the two, and a token's result does not depend on the other
// tokens of the batch.
//
// hidden 7168, intermediate 2048, 256 experts, 8 per token, gated, both kernels:
//   bf16  1 token  126 us (5.6 TB/s of weights)   128 tokens 3700 us (6.0 TB/s)
//   fp8   1 token   74 us (4.8 TB/s)              128 tokens 2090 to 2220 us (5.3 to 5.0)
// where a kernel that only reads reaches 6.4 TB/s.  One token: 0.35 GB of fp8
// weights are 56 us, two launches and their first loads the rest.
#include <algorithm>

#include "ep_expert_device.h"

namespace ep {

namespace {

constexpr int kMaxPairs = EP_MAX_DECODE_PAIRS;

struct DecodeK {
    MoeDecodeArgs a;
    int pairs;
    int by_pair;      // first kernel: a workgroup's expert is that of pair blockIdx.y
    int tokens;       // second kernel: tokens of a workgroup
};

typedef __amdgpu_buffer_rsrc_t Buffer;

// Reads past `bytes` return zeros; no buffer here has kOutOfRange bytes.
__device__ __forceinline__ Buffer buffer(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)bytes, 0x00020000);
}

// An expert's weights and their scales.
struct Weights {
    const uint8_t *w, *scales;
    int bytes, scale_bytes;
    __device__ __forceinline__ Weights(const void *base, const void *scale_base, int e, int64_t rows,
                                       int64_t row_bytes, int64_t groups)
        : w((const uint8_t *)base + e * rows * row_bytes), scales((const uint8_t *)scale_base + e * rows * groups),
          bytes((int)(rows * row_bytes)), scale_bytes((int)(rows * groups)) {}
};

// 256 bytes of the rows of CT weight tiles (16 rows each), and the same channels
// of up to 16 token rows, as they come from memory: a lane has 4 pieces of 16
// bytes of a weight row, 8 consecutive bf16 or 16 fp8 channels (with two scale
// bytes); the token rows' pieces follow the weights' order.  The weights pass
// the caches in the ordinary way: the 16 rows x 64 bytes of one load are half
// lines, and with the non-temporal hint the halves were fetched apart (5.1
// against 5.9 TB/s).
template <bool FP8, int CT>
struct Chunk {
    static constexpr int kChannels = FP8 ? 256 : 128;
    static constexpr int kX = FP8 ? 8 : 4;
    ep_u32x4 w[CT][4];
    uint32_t scale;               // of tile q % CT, 128 channels q / CT

    // wv, xv: this lane's byte offsets of its rows, sv of its scales (kOutOfRange:
    // zeros).  Without `some` nothing is read.
    __device__ __forceinline__ void load_w(const Weights &src, const uint32_t *wv, uint32_t sv,
                                           int chunk, int channels, bool some = true) {
        const Buffer wb = buffer(src.w, src.bytes), sb = buffer(src.scales, src.scale_bytes);
        const int q = (threadIdx.x & 63) >> 4;
        const int c = some ? chunk * kChannels : channels;
        chunk = some ? chunk : 0;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t o = wv[t] + q * 16 + j * 64;
                if (FP8 ? c + j * 64 >= channels : c + j * 32 + q * 8 >= channels) o = kOutOfRange;
                w[t][j] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(wb, o, chunk * 256, 0));
            }
        // one byte a lane for the four (or two) scales of a row pair
        if (FP8) scale = __builtin_amdgcn_raw_buffer_load_b8(sb, c + q / CT * 128 < channels ? sv : kOutOfRange,
                                                             chunk * 2, 0);
    }
    static __device__ __forceinline__ uint32_t scale_offset(const int *row, int rows, int groups) {
        const int q = (threadIdx.x & 63) >> 4;
        const int r = row[q % CT];
        return q < 2 * CT && r < rows ? (uint32_t)(r * groups + q / CT) : kOutOfRange;
    }
    static __device__ __forceinline__ void load_x(Buffer xb, uint32_t xv, int chunk, int channels, ep_u32x4 *x) {
        const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            // first of the 8 channels
            const int c = chunk * kChannels + (FP8 ? (j >> 1) * 64 + q * 16 + (j & 1) * 8 : j * 32 + q * 8);
            const uint32_t o = xv == kOutOfRange || c >= channels ? kOutOfRange : xv + c * 2;
            x[j] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, o, 0, 0));
        }
    }
    // acc[g][t] += weight tile t x token rows g
    template <int GROUPS>
    __device__ __forceinline__ void multiply(const ep_u32x4 (*x)[kX], ep_f32x4 (*acc)[CT]) const {
        float s[CT][2];
        if (FP8) {
#pragma unroll
            for (int i = 0; i < 2 * CT; ++i)
                s[i % CT][i / CT] = ue8m0_value(__shfl((int)scale, i * 16 + (threadIdx.x & 15)));
        }
#pragma unroll
        for (int j = 0; j < kX; ++j)
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                ep_u32x4 v;
                if (FP8) {
                    const float f = s[t][FP8 ? j >> 2 : 0];
                    const uint32_t lo = w[t][j >> 1][(j & 1) * 2], hi = w[t][j >> 1][(j & 1) * 2 + 1];
                    v.x = fp8_pair_bf16<false>(lo, f);
                    v.y = fp8_pair_bf16<true>(lo, f);
                    v.z = fp8_pair_bf16<false>(hi, f);
                    v.w = fp8_pair_bf16<true>(hi, f);
                } else {
                    v = w[t][FP8 ? 0 : j];
                }
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) acc[g][t] = mfma_bf16(v, x[g][j], acc[g][t]);
            }
    }
};

// acc[g][t] += weights x rows g over chunks [from, to): a chunk's token rows
// (from the caches) are asked for just before the next chunk's weights (from
// memory), so that waiting for them leaves the weights in flight.  That needs a
// loop without conditional loads: where one may be left out, the wait counts
// every load behind it as possibly the one waited for.  `a` holds the weights
// of chunk `from`; it is left with those of chunk next_from of `next`, if there
// are `more`.
template <int GROUPS, bool FP8, int CT>
__device__ __forceinline__ void sweep(Chunk<FP8, CT> &a, const Weights &src, const uint32_t *wv, uint32_t sv,
                                      Buffer xb, const uint32_t *xv, int from, int to, int channels,
                                      ep_f32x4 (*acc)[CT], const Weights &next, int next_from, bool more) {
    typedef Chunk<FP8, CT> C;
    C b;
    ep_u32x4 x[GROUPS][C::kX];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[g][t] = ep_f32x4{0, 0, 0, 0};
    auto load_x = [&](int c) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) C::load_x(xb, xv[g], c, channels, x[g]);
    };
    // the order of loads and products is as written
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
    int c = from;
    for (; c + 1 < to; c += 2) {
        load_x(c);
        fence();
        b.load_w(src, wv, sv, c + 1, channels);
        fence();
        a.template multiply<GROUPS>(x, acc);
        fence();
        load_x(c + 1);
        fence();
        const bool here = c + 2 < to;
        Weights then = src;
        then.w = here ? src.w : next.w;
        then.scales = here ? src.scales : next.scales;
        a.load_w(then, wv, sv, here ? c + 2 : next_from, channels, here || more);
        fence();
        b.template multiply<GROUPS>(x, acc);
        fence();
    }
    if (c < to) {
        load_x(c);
        a.template multiply<GROUPS>(x, acc);
        a.load_w(next, wv, sv, next_from, channels, more);
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int t = 0; t < CT; ++t) pin(acc[g][t]);
}

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

constexpr int kUpCols = 16;       // columns of h of a workgroup of the first kernel

template <bool FP8, bool GATED>
__global__ __launch_bounds__(256) void moe_decode_up_kernel(DecodeK k) {
    const MoeDecodeArgs &a = k.a;
    constexpr int CT = GATED ? 2 : 1;
    __shared__ int16_t list[kMaxPairs];
    __shared__ int red[8];
    __shared__ float part[4][CT][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int e = k.by_pair ? (int)a.topk_idx[blockIdx.y] : (int)blockIdx.y;
    const bool known = !k.by_pair || (a.topk_idx[blockIdx.y] >= 0 && a.topk_idx[blockIdx.y] < a.E);
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0) {
        bool bad = false;
        for (int p = tid; p < k.pairs; p += 256) bad |= a.topk_idx[p] < -1 || a.topk_idx[p] >= a.E;
        if (bad) atomicOr(a.status, kDevBadExpert);
    }
    if (!known) return;

    const int I = a.I, H = a.H, n1 = GATED ? 2 * I : I;
    const int col0 = blockIdx.x * kUpCols;
    const int groups = FP8 ? H / kFp8Group : 0;
    const Weights weights(a.w1, a.w1_scales, e, n1, (int64_t)H * (FP8 ? 1 : 2), groups);
    const Buffer xb = buffer(a.x, (int64_t)a.T * H * 2);
    uint32_t wv[CT];
    int row[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        // gated: a tile of gates, then of their ups
        row[t] = col0 + l16 < I ? col0 + l16 + t * I : n1;
        wv[t] = row[t] < n1 ? (uint32_t)row[t] * H * (FP8 ? 1 : 2) : kOutOfRange - 1024;
    }
    const uint32_t sv = Chunk<FP8, CT>::scale_offset(row, n1, groups);
    // the waves take equal runs of the row's chunks
    const int chunks = (H + Chunk<FP8, CT>::kChannels - 1) / Chunk<FP8, CT>::kChannels;
    const int from = chunks * wave / 4, to = chunks * (wave + 1) / 4;
    // by pair, the first weights are on their way while the pairs are found
    Chunk<FP8, CT> chunk;
    if (k.by_pair) chunk.load_w(weights, wv, sv, from, H);
    const int count = wave_uniform(pairs_of<256>(a.topk_idx, k.pairs, e, list, red));
    // by pair: only the expert's first pair computes
    if (count == 0 || (k.by_pair && list[0] != (int)blockIdx.y)) return;
    if (!k.by_pair) chunk.load_w(weights, wv, sv, from, H);
    for (int g0 = 0; g0 < count; g0 += 16) {
        const int live = min(16, count - g0);
        const uint32_t xv = l16 < live ? (uint32_t)(list[g0 + l16] / a.K) * H * 2 : kOutOfRange;
        ep_f32x4 acc[1][CT];
        sweep<1>(chunk, weights, wv, sv, xb, &xv, from, to, H, acc, weights, from, g0 + 16 < count);
#pragma unroll
        for (int t = 0; t < CT; ++t)
            for (int i = 0; i < 4; ++i) part[wave][t][4 * q + i][l16] = acc[0][t][i];
        __syncthreads();
        for (int i = tid; i < kUpCols * 16; i += 256) {
            // one column of one pair per thread
            const int c = i % kUpCols, r = i / kUpCols, col = col0 + c;
            if (r < live && col < I) {
                float z[2] = {0.0f, 0.0f};
                for (int s = 0; s < (GATED ? 2 : 1); ++s) {
                    for (int w = 0; w < 4; ++w) z[s] += part[w][s][c][r];
                    if (a.bias1)
                        z[s] += __uint_as_float((uint32_t)((const uint16_t *)a.bias1)[(int64_t)e * n1 + s * I + col] << 16);
                }
                float y = a.kind == 1 ? act_value<1>(z[0]) : a.kind == 2 ? act_value<2>(z[0]) : z[0];
                if (GATED) y *= z[1];
                // the matrix instruction takes bf16: y as the sum of two of
                // them keeps 16 significant bits, so that out is rounded once
                __bf16 *h = (__bf16 *)a.h + (int64_t)list[g0 + r] * 2 * I + col;
                const __bf16 hi = (__bf16)y;
                h[0] = hi;
                h[I] = __builtin_isfinite((float)hi) ? (__bf16)(y - (float)hi) : (__bf16)0.0f;
            }
        }
        __syncthreads();
    }
}

// Waves of the second kernel.
constexpr int kDownWaves = 8;
constexpr int kDownCols = 32;     // channels of out of its workgroup

template <bool FP8>
__global__ __launch_bounds__(64 * kDownWaves) void moe_decode_down_kernel(DecodeK k) {
    const MoeDecodeArgs &a = k.a;
    extern __shared__ __align__(16) float y[];             // [pairs][kDownCols]
    // its tokens and their pairs, numbered from 0 here
    const int t0 = blockIdx.y * k.tokens, tokens = min(k.tokens, a.T - t0);
    const int pairs = tokens * a.K;
    const int64_t *topk_idx = a.topk_idx + (int64_t)t0 * a.K;
    int *first = (int *)(y + pairs * kDownCols);           // [E] first pair of an expert
    int16_t *id = (int16_t *)(first + a.E);                // [pairs] expert of a pair
    int16_t *leader = id + ((pairs + 7) & ~7);             // [pairs] the experts' first pairs
    int16_t *mine = leader + ((pairs + 7) & ~7) + (threadIdx.x >> 6) * 16;     // a wave's 16 pairs
    __shared__ int red[kDownWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    constexpr int kThreads = 64 * kDownWaves;
    const int H = a.H, I = a.I;
    const int h0 = blockIdx.x * kDownCols;

    for (int e = tid; e < a.E; e += kThreads) first[e] = pairs;
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int64_t e = topk_idx[p];
        const bool ok = e >= 0 && e < a.E;
        id[p] = ok ? (int16_t)e : (int16_t)-1;
        if (ok) atomicMin(&first[e], p);
    }
    __syncthreads();
    int experts = 0;
    for (int p0 = 0; p0 < pairs; p0 += kThreads) {
        const int p = p0 + tid;
        const bool lead = p < pairs && id[p] >= 0 && first[id[p]] == p;
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

    const int groups = FP8 ? I / kFp8Group : 0;
    constexpr int CT = kDownCols / 16;
    const Buffer hb = buffer((const uint16_t *)a.h + (int64_t)t0 * a.K * 2 * I, (int64_t)pairs * I * 4);
    uint32_t wv[CT];
    int row[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        row[t] = h0 + t * 16 + l16;
        wv[t] = row[t] < H ? (uint32_t)row[t] * I * (FP8 ? 1 : 2) : kOutOfRange - 1024;
    }
    const uint32_t sv = Chunk<FP8, CT>::scale_offset(row, H, groups);
    const int chunks = (I + Chunk<FP8, CT>::kChannels - 1) / Chunk<FP8, CT>::kChannels;
    auto weights = [&](int e) { return Weights(a.w2, a.w2_scales, e, H, (int64_t)I * (FP8 ? 1 : 2), groups); };
    auto expert = [&](int s) { return wave_uniform((int)id[wave_uniform((int)leader[s])]); };
    Chunk<FP8, CT> chunk;
    if (wave < experts) chunk.load_w(weights(expert(wave)), wv, sv, 0, I);
    for (int s = wave; s < experts; s += kDownWaves) {
        const int e = expert(s);
        // the expert that this wave takes after this one
        const bool another = s + kDownWaves < experts;
        const int e1 = expert(another ? s + kDownWaves : s);
        // the expert's pairs, 16 at a time in ascending order
        int from = wave_uniform((int)leader[s]);
        bool more = true;
        while (more) {
            int live = 0;
            for (int p = from; p < pairs && live <= 16; p += 64) {
                const bool hit = p + lane < pairs && id[p + lane] == e;
                const uint64_t m = __ballot(hit);
                const int at = live + __popcll(m & lanes_below());
                if (hit && at < 16) mine[at] = (int16_t)(p + lane);
                live += __popcll(m);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            const int n = min(live, 16);
            more = live > 16;
            from = wave_uniform((int)mine[n - 1]) + 1;
            // columns 0..7 of the product are eight pairs' high parts of h,
            // columns 8..15 the low parts of the same pairs
            uint32_t hv[2];
            int pair[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int i = g * 8 + (l16 & 7);
                pair[g] = mine[i < n ? i : 0];
                hv[g] = i < n ? (uint32_t)pair[g] * I * 4 + (l16 >> 3) * I * 2 : kOutOfRange;
            }
            auto products = [&](auto groups_tag) {
                constexpr int G = decltype(groups_tag)::value;
                ep_f32x4 acc[G][CT];
                sweep<G>(chunk, weights(e), wv, sv, hb, hv, 0, chunks, I, acc, weights(more ? e : e1), 0,
                         more || another);
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int t = 0; t < CT; ++t) {
                        ep_f32x4 v = acc[g][t];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] += __shfl_xor(v[i], 8);
                            const int c = h0 + t * 16 + 4 * q + i;
                            if (a.bias2 && c < H)
                                v[i] += __uint_as_float((uint32_t)((const uint16_t *)a.bias2)[(int64_t)e * H + c] << 16);
                        }
                        if (l16 < 8 && g * 8 + l16 < n) *(ep_f32x4 *)(y + pair[g] * kDownCols + t * 16 + 4 * q) = v;
                    }
            };
            // one or two groups of eight: a pair's sums are the same in both
            if (n <= 8) products(std::integral_constant<int, 1>());
            else products(std::integral_constant<int, 2>());
        }
    }
    __syncthreads();

    // out[t, h0 .. h0 + 31] in pieces of 8 channels
    constexpr int kParts = kDownCols / 8;
    for (int i = tid; i < tokens * kParts; i += kThreads) {
        const int t = i / kParts, c = i % kParts * 8;
        if (h0 + c >= H) continue;
        const int64_t o = (int64_t)(t0 + t) * H + h0 + c;
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
            const float w = a.topk_weights ? a.topk_weights[(int64_t)t0 * a.K + p] : 1.0f;
            for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(w, y[p * kDownCols + c + j], s[j]);
        }
        ep_u32x4 v;
        for (int j = 0; j < 4; ++j) v[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
        *(ep_u32x4 *)((uint16_t *)a.out + o) = v;
    }
}

size_t down_lds(int pairs, int E) {
    return (size_t)pairs * kDownCols * 4 + (size_t)E * 4 + (size_t)((pairs + 7) & ~7) * 4 + kDownWaves * 32;
}

}  // namespace

hipError_t launch_moe_decode(const MoeDecodeArgs &a, hipStream_t stream) {
    DecodeK k = {};
    k.a = a;
    k.pairs = a.T * a.K;
    k.by_pair = k.pairs <= a.E ? 1 : 0;
    const dim3 up((unsigned)((a.I + kUpCols - 1) / kUpCols), (unsigned)(k.by_pair ? k.pairs : a.E));
    // A compute unit holds one workgroup of the second kernel, so with few output
    // channels the tokens are divided among more of them, as far as they all run
    // at once (experts that two of them share are read twice).  Both kernels, with
    // one group against several: hidden 2048, intermediate 1408, 60 experts, 4 per
    // token, 8 tokens bf16 129 and 92 us, 128 tokens fp8 255 and 195 us; hidden
    // 256, intermediate 1280, 32 tokens 300 and 65 us.
    const int cols = (a.H + kDownCols - 1) / kDownCols;
    const int groups = std::max(1, std::min(a.T, 256 / cols));
    k.tokens = (a.T + groups - 1) / groups;
    const dim3 down((unsigned)cols, (unsigned)((a.T + k.tokens - 1) / k.tokens));
    const size_t lds = down_lds(k.tokens * a.K, a.E);
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
