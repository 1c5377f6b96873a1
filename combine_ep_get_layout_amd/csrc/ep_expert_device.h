// Device helpers of the expert operators (internal header): the segment
// search, the LDS copies of the matrix products, activations and roundings.
#pragma once

#include "ep_device.h"
#include "ep_expert.h"

typedef __bf16 ep_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 ep_bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 ep_bf16x2 __attribute__((ext_vector_type(2)));
typedef float ep_f32x4 __attribute__((ext_vector_type(4)));
typedef short ep_i16x4 __attribute__((ext_vector_type(4)));
typedef int ep_i32x4 __attribute__((ext_vector_type(4)));
typedef int ep_i32x8 __attribute__((ext_vector_type(8)));

namespace ep {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// One workgroup's tile of a segmented product.
struct TileAt {
    int e;       // segment
    int mt, nt;  // tile of rows inside the segment, tile of columns
    int row0;    // first row of the segment
    int rows;    // rows of the segment
};

// Rows of segment e that hold a pair and exist.
__device__ __forceinline__ int segment_rows(const SegmentRows &s, int e, int *row0) {
    const int o = s.offsets[e];
    const int have = s.offsets[e + 1] - o;
    const int c = min(s.counts[e], have);
    *row0 = o;
    const int64_t room = s.num_rows - o;
    if (c > room) {
        atomicOr(s.status, kDevRecvOverflow);
        return room > 0 ? (int)room : 0;
    }
    return c;
}

// The tile of workgroup `block`: all segments' (row tile, column tile) pairs
// in one sequence, segment after segment, found by a scan of the segments'
// counts (a load and a wave scan, about 2 us, once per workgroup).  The
// sequence is cut into 8 equal runs, one per XCD (workgroups go to the XCDs
// in turn), and walks, inside a segment, 8 row tiles before the next column
// tile, so that the tiles running together on one XCD share their operands in
// its L2.  `red` is LDS of at least 16 ints; the whole workgroup calls this.
// Returns false for a workgroup without a tile.
template <int THREADS>
__device__ bool find_tile(const SegmentRows &s, int tile_rows, int col_tiles, int block,
                          int *red, TileAt *at) {
    constexpr int kWaves = THREADS / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (s.E + THREADS - 1) / THREADS;
    const int beg = min(s.E, tid * per), end = min(s.E, beg + per);
    int local = 0, row0 = 0;
    for (int e = beg; e < end; ++e)
        local += (segment_rows(s, e, &row0) + tile_rows - 1) / tile_rows;
    int incl = local;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 63) red[wave] = incl;
    __syncthreads();
    int base = 0, total = 0;
    for (int w = 0; w < kWaves; ++w) {
        const int v = red[w];
        base += w < wave ? v : 0;
        total += v;
    }
    const int64_t tiles = (int64_t)total * col_tiles;
    const int64_t run = (tiles + 7) >> 3;
    const int64_t t = (int64_t)(block & 7) * run + (block >> 3);
    if ((block >> 3) >= run || t >= tiles) return false;
    const int u = (int)(t / col_tiles);
    int first = base + incl - local;
    if (u >= first && u < first + local) {
        for (int e = beg; e < end; ++e) {
            const int rows = segment_rows(s, e, &row0);
            const int n = (rows + tile_rows - 1) / tile_rows;
            if (u < first + n) {
                const int lt = (int)(t - (int64_t)first * col_tiles);
                const int g = lt / (8 * col_tiles);
                const int gm = min(8, n - g * 8);
                const int rem = lt - g * 8 * col_tiles;
                red[8] = e;
                red[9] = g * 8 + rem % gm;
                red[10] = rem / gm;
                red[11] = row0;
                red[12] = rows;
                break;
            }
            first += n;
        }
    }
    __syncthreads();
    at->e = wave_uniform(red[8]);
    at->mt = wave_uniform(red[9]);
    at->nt = wave_uniform(red[10]);
    at->row0 = wave_uniform(red[11]);
    at->rows = wave_uniform(red[12]);
    return true;
}

// A buffer descriptor over `bytes` bytes at p: reads past them return zeros.
__device__ __forceinline__ ep_i32x4 buffer_of(const void *p, uint32_t bytes) {
    const uint64_t a = (uint64_t)p;
    ep_i32x4 r;
    r.x = wave_uniform((int)(uint32_t)a);
    r.y = wave_uniform((int)(uint32_t)(a >> 32) & 0xFFFF);
    r.z = wave_uniform((int)bytes);
    r.w = 0x00020000;
    return r;
}
constexpr uint32_t kOutOfRange = 0x80000000u;   // no buffer here is longer

// 64 lanes x 16 bytes from buffer offsets voff + soff to LDS bytes
// [lds, lds + 1024), in lane order, without passing through registers; lanes
// out of the buffer's range write zeros.  Asynchronous: the data is in LDS
// after a wait on the vector memory count (dma_wait).  There is no output
// register, so nothing the compiler could reuse too early; it does not know of
// the copy, and the waits below carry the order.
__device__ __forceinline__ void dma16(const ep_i32x4 &rsrc, uint32_t lds, uint32_t voff,
                                      uint32_t soff) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
        : "m0");
}

// All but the newest N copies of this wave have landed, and its own LDS reads
// have returned (so that a barrier after it releases the buffers they read).
template <int N>
__device__ __forceinline__ void dma_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ void barrier_only() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// Holds a matrix instruction's result at this point: the compiler may
// otherwise move the instruction into a branch that only some lanes take, and
// it needs all lanes' operands.
__device__ __forceinline__ void pin(ep_f32x4 &v) { asm volatile("" : "+v"(v)); }

// fp32 pairs to packed bf16, nearest even (the hardware conversion).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    ep_bf16x2 v;
    v.x = (__bf16)a;
    v.y = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

// exp(x) through the hardware's base-2 exponential: x log2(e) is formed as a
// product and its exact remainder, so that large |x| keep their relative
// accuracy.  Outside [-104, 89] it is 0 or inf.
__device__ __forceinline__ float fast_exp(float x) {
    x = fminf(fmaxf(x, -104.0f), 89.0f);
    const float kLog2e = 1.44269504f, kLog2eLo = 1.92596299e-8f;
    const float p = x * kLog2e;
    const float r = __builtin_fmaf(x, kLog2e, -p) + x * kLog2eLo;
    return __builtin_amdgcn_exp2f(p) * __builtin_fmaf(r, 0.693147181f, 1.0f);
}

// 1 / (1 + exp(-z)); exp(-z) = inf gives 0.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + fast_exp(-z));
}

// gelu's tanh form as a sigmoid: (1 + tanh(y)) / 2 = sigmoid(2 y),
// y = sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ float gelu_gate(float z) {
    const float c = 1.59576912f;   // 2 sqrt(2/pi)
    return sigmoid(c * z * __builtin_fmaf(0.044715f * z, z, 1.0f));
}

// Activation functions of one value: kind 0 none, 1 silu, 2 gelu.  z times a
// gate that underflowed to 0 is 0 for every finite z; -inf gives -inf * 0 =
// NaN, as the formula does.
__device__ __forceinline__ float act_value(float z, int kind) {
    if (kind == 1) return z * sigmoid(z);
    if (kind == 2) return z * gelu_gate(z);
    return z;
}

// Value and derivative of an activation function.
__device__ __forceinline__ void act_both(float z, int kind, float *f, float *df) {
    if (kind == 1) {
        const float p = sigmoid(z);
        *f = z * p;
        *df = __builtin_fmaf(*f, 1.0f - p, p);
    } else if (kind == 2) {
        // p = sigmoid(2 y): d/dz (z p) = p + z p (1 - p) 2 y'
        const float p = gelu_gate(z);
        *f = z * p;
        *df = __builtin_fmaf(*f * (1.0f - p), 1.59576912f * __builtin_fmaf(0.134145f * z, z, 1.0f), p);
    } else {
        *f = z;
        *df = 1.0f;
    }
}

// UE8M0 byte b as the float 2^(b - 127).
__device__ __forceinline__ float ue8m0_value(uint32_t b) {
    return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Two e4m3 codes (a half of the dword) times a power of two, as packed bf16:
// exact, a code's four significant bits fit bf16's eight.
template <bool HI>
__device__ __forceinline__ uint32_t fp8_pair_bf16(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HI));
}

}  // namespace ep
