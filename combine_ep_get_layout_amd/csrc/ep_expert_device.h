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
    if (c > 0 && c > room) {    // an empty segment may begin behind the buffers
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
__device__ __forceinline__ bool find_tile(const SegmentRows &s, int tile_rows, int col_tiles, int block,
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
    const uint32_t tiles = (uint32_t)total * (uint32_t)col_tiles;   // at most the grid
    const uint32_t run = (tiles + 7) >> 3;
    const uint32_t t = (uint32_t)(block & 7) * run + (uint32_t)(block >> 3);
    if ((uint32_t)(block >> 3) >= run || t >= tiles) return false;
    const int u = (int)(t / (uint32_t)col_tiles);
    int first = base + incl - local;
    if (u >= first && u < first + local) {
        for (int e = beg; e < end; ++e) {
            const int rows = segment_rows(s, e, &row0);
            const int n = (rows + tile_rows - 1) / tile_rows;
            if (u < first + n) {
                const int lt = (int)(t - (uint32_t)first * (uint32_t)col_tiles);
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
// the copy, and the waits below carry the order.  m0, the LDS address, is an
// operand: whatever is compiled between two copies, each finds its own there (the
// compiler leaves out the writes that change nothing).  The wait states are the
// copy's own, since the compiler does not look into the statement: one after a
// write of m0, and five where a vector instruction (a broadcast, a reload of a
// spilled scalar) has just written the descriptor or the offset.
__device__ __forceinline__ void dma16(const ep_i32x4 &rsrc, uint32_t lds, uint32_t voff,
                                      uint32_t soff) {
    ep_i32x4 r;
    for (int i = 0; i < 4; ++i) r[i] = wave_uniform(rsrc[i]);
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds"
        :
        : "v"(voff), "s"(r), "s"(wave_uniform((int)soff)), "{m0}"(wave_uniform((int)lds)));
}

// The same for four copies to consecutive kilobytes of LDS, one call each with
// J = 0, 1, 2, 3 in this order and the first one's LDS address: the instruction
// offset J * 1024 moves both addresses, so the caller's voff is kDmaBias - J *
// 1024 more than the source's and its buffer starts kDmaBias early (biased_buffer).
// The first waits for the descriptor and the offset, the others take them from it:
// there a wait of five states cost 3% of a large product.
constexpr uint32_t kDmaBias = 3 * 1024;
__device__ __forceinline__ ep_i32x4 biased_buffer(const void *p, uint32_t bytes) {
    return buffer_of((const uint8_t *)p - kDmaBias, bytes + kDmaBias);
}

// `bytes` and `soff` when the copies of step s exist (s < steps), else an empty
// buffer: scalar code, so that they stay scalar registers.  (The offset is
// cleared too: a buffer's range check subtracts it from the size.)
__device__ __forceinline__ void range_of(int s, int steps, uint32_t bytes, uint32_t soff,
                                         ep_i32x4 &buffer, uint32_t *out) {
    uint32_t z, o;
    asm volatile("s_cmp_lt_i32 %2, %3\n\ts_cselect_b32 %0, %4, 0\n\ts_cselect_b32 %1, %5, 0"
                 : "=&s"(z), "=&s"(o)
                 : "s"(wave_uniform(s)), "s"(wave_uniform(steps)), "s"(wave_uniform((int)bytes)),
                   "s"(wave_uniform((int)soff))
                 : "scc");
    buffer.z = (int)z;
    *out = o;
}

template <int J>
__device__ __forceinline__ void dma16_of4(ep_i32x4 &rsrc, uint32_t lds, uint32_t voff,
                                          uint32_t &soff) {
    if (J == 0) {
        ep_i32x4 r;
        for (int i = 0; i < 4; ++i) r[i] = wave_uniform(rsrc[i]);
        uint32_t o = wave_uniform((int)soff);
        asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %2, %0, %1 offen lds"
                     : "+s"(r), "+s"(o)
                     : "v"(voff), "{m0}"(wave_uniform((int)lds)));
        rsrc = r;
        soff = o;
    } else {
        asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %2, %0, %1 offen offset:%3 lds"
                     : "+s"(rsrc), "+s"(soff)
                     : "v"(voff), "n"(J * 1024), "{m0}"(wave_uniform((int)lds)));
    }
}

// 64 lanes x 1 byte, one dword of LDS each (the byte, zero extended).
__device__ __forceinline__ void dma1(const ep_i32x4 &rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    ep_i32x4 r;
    for (int i = 0; i < 4; ++i) r[i] = wave_uniform(rsrc[i]);
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_ubyte %0, %1, %2 offen lds"
        :
        : "v"(voff), "s"(r), "s"(wave_uniform((int)soff)), "{m0}"(wave_uniform((int)lds)));
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

// Tiles staged with the summed index outermost ([64 rows][128 or 256 columns]
// of bf16, ROW bytes a row): the 32-byte granule g of row r is in place
// g ^ granule_of(r), so that the 16 rows one transposing read takes lie in
// different banks.
__device__ __forceinline__ int granule_of(int r) { return (r & 3) | ((r >> 3 & 1) << 2); }

// The matrix operand of 16 columns (granule g) and rows [32 h, 32 h + 32) of
// such a tile, by the transposing LDS read: lane l of a 16-lane group names row
// l/4 and column 4 (l % 4) of a 4 x 16 block and receives its column l.
template <int ROW>
__device__ __forceinline__ ep_u32x4 transposed_operand(const uint8_t *tile, int g, int h) {
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int r = h * 32 + (lane >> 4) * 8 + (l16 >> 2);
    const uint8_t *p = tile + r * ROW + (g ^ granule_of(r)) * 32 + (l16 & 3) * 8;
    const ep_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) ep_i16x4 *)p);
    const ep_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) ep_i16x4 *)(p + 4 * ROW));
    ep_u32x4 v;
    v.xy = __builtin_bit_cast(ep_u32x2, lo);
    v.zw = __builtin_bit_cast(ep_u32x2, hi);
    return v;
}

__device__ __forceinline__ ep_f32x4 mfma_bf16(ep_u32x4 a, ep_u32x4 b, ep_f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(ep_bf16x8, a),
                                                   __builtin_bit_cast(ep_bf16x8, b), c, 0, 0, 0);
}

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

// f(0), ..., f(N - 1) with constant arguments: accumulators indexed by them
// stay in registers whatever the body's size.
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
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

// Activation functions of one value that is rounded to bf16 next: kind 0 none,
// 1 silu, 2 gelu.  The gate's exponential takes its argument rounded to fp32
// (relative error |z| 2^-24, under bf16's 2^-8 by far) without fast_exp's
// remainder: half the instructions.  A gate that underflowed to 0 gives 0 for
// every finite z; -inf gives -inf * 0 = NaN, as the formula does.
template <int KIND>
__device__ __forceinline__ float act_value(float z) {
    if (KIND == 0) return z;
    const float y = KIND == 1 ? z * -1.44269504f
                              : z * __builtin_fmaf(z * z, -0.102943240f, -2.30220819f);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y));
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
        // (p is 0 or 1 long before |z| = 64: the cut keeps y' finite, and its term 0)
        const float c = fminf(fmaxf(z, -64.0f), 64.0f);
        *df = __builtin_fmaf(*f * (1.0f - p), 1.59576912f * __builtin_fmaf(0.134145f * c, c, 1.0f), p);
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
