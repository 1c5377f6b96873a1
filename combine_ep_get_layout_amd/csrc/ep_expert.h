// Host-side launchers of the expert operators, shared between their kernel
// files and the C ABI (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ep.h"

namespace ep {

// Channels per UE8M0 scale: of fp8 rows and weights in the products, and of
// the pre-activations' 8-bit checkpoint.
constexpr int kFp8Group = 128;
constexpr int kCheckpointGroup = 32;

// Rows of a receive layout by segment: segment e holds rows
// [offsets[e], offsets[e] + min(counts[e], offsets[e+1] - offsets[e])), of
// which only those under num_rows exist.  Without a layout (offsets NULL) rows
// [e * each, min((e + 1) * each, num_rows)).
struct SegmentRows {
    const int32_t *counts;
    const int32_t *offsets;
    int32_t *status;      // EP_DEV_RECV_OVERFLOW where rows at or past num_rows would be used
    int E;
    int64_t num_rows;
    int64_t pairs;        // upper bound of the rows that hold a pair
    int64_t each;         // rows of a segment without a layout
};

struct LinearArgs {
    SegmentRows seg;
    const void *x;               // [num_rows, k]
    const uint8_t *x_scales;     // fp8: [num_rows, k/128]
    const void *w;               // [E, n, k], transposed: [E, k, n]
    const uint8_t *w_scales;     // fp8: [E, n, k/128]
    const void *bias;            // bf16 [E, n] or NULL
    const void *residual;        // bf16 [num_rows, m] or NULL, m the columns of out
    void *out;                   // bf16 [num_rows, m]
    uint8_t *ckpt;               // e4m3 [num_rows, n] or NULL
    uint8_t *ckpt_scales;        // [num_rows, n/32]
    int n, k;
    int act;                     // EP_ACT_*
    bool fp8, transposed;
};

hipError_t launch_expert_linear(const LinearArgs &a, hipStream_t stream);

struct WgradArgs {
    SegmentRows seg;
    const void *dy;              // bf16 [num_rows, n]
    const void *x;               // [num_rows, k]
    const uint8_t *x_scales;     // fp8: [num_rows, k/128]
    const void *dw_in;           // dw's type [E, n, k] or NULL: added to the gradient
    const float *db_in;          // [E, n] or NULL
    void *dw;                    // fp32 or bf16 [E, n, k]
    float *db;                   // [E, n] or NULL
    int n, k;
    bool fp8, bf16_out;
};

hipError_t launch_expert_wgrad(const WgradArgs &a, hipStream_t stream);

struct ActBackwardArgs {
    const int32_t *src_of_slot;  // [entries] >= 0 where a row holds a pair
    const int32_t *total_rows;   // rows in use
    int32_t *status;
    int64_t num_rows;            // rows of the buffers, at most `entries`
    int64_t entries;
    const void *dh;              // bf16 [num_rows, m]
    const void *pre;             // bf16 or e4m3 [num_rows, n]
    const uint8_t *pre_scales;   // [num_rows, n/32] when pre is e4m3, else NULL
    const float *row_weights;    // [num_rows] or NULL
    void *dpre;                  // bf16 [num_rows, n]
    void *h;                     // bf16 [num_rows, m] or NULL
    float *dweights;             // [num_rows] or NULL
    int n, m, kind;
    bool gated;
};

hipError_t launch_act_backward(const ActBackwardArgs &a, hipStream_t stream);

// Whether HIP launches so many workgroups: fewer than 2^32 threads.
inline bool launchable(int64_t grid, int threads) { return grid <= 0xffffffff / threads; }

// The activation function of an EP_ACT_* (0 none, 1 silu, 2 gelu).
inline int act_kind(int act) {
    return act == EP_ACT_SILU || act == EP_ACT_SWIGLU ? 1
           : act == EP_ACT_GELU || act == EP_ACT_GEGLU ? 2 : 0;
}
inline bool act_gated(int act) { return act == EP_ACT_SWIGLU || act == EP_ACT_GEGLU; }

// Dense rows, at most kFewRows of them.  Taken up to 16 rows, and for more while
// they have few bytes, since every workgroup reads them.  Both sides, us here and in
// tiles, whole or in parts:
//   bf16  7168 to 4096, gated, 24 rows 18.9 and 18.2, 64 rows 34 and 21; 2048 to 7168
//         32 rows 13.7 and 12.4; but 1024 to 4096, gated, 64 rows 7.5 and 9.2
//   e4m3  7168 to 4096, gated, 16 rows 10.7 and 15.6, 32 rows 15.2 and 16.2, 48 rows
//         21 and 17; 4096 to 4096 32 rows 10.1 and 13.0; 1024 to 4096, gated, 64 rows
//         6.5 and 7.5
// (The limit in bytes was chosen for bf16.  In e4m3 it is too high for many columns of
// short rows, 2048 to 7168 32 rows 10.3 and 9.8, 64 rows 16.2 and 10.0, and a little
// low for 24 and 32 rows of 7168.)
constexpr int kFewRows = 64;
inline bool few_rows(int64_t rows, int64_t row_bytes) {
    return rows <= 16 || (rows <= kFewRows && rows * row_bytes <= 128 * 1024);
}
struct FewRowsArgs {
    const void *x;               // [rows, k]
    const float *x_scales;       // e4m3: [rows, k/128], bf16: NULL
    const void *w;               // [n, k]
    const float *w_scales;       // e4m3: [ceil(n/128), k/128]
    const void *bias;            // bf16 [n] or NULL
    const void *residual;        // bf16 [rows, m] or NULL
    void *out;                   // bf16 [rows, m]
    int rows, n, k;
    int act;                     // EP_ACT_*
};

hipError_t launch_few_rows(const FewRowsArgs &a, hipStream_t stream);

// The product of e4m3 rows with fp32 scales per 128 channels and e4m3 weights
// with fp32 scales per 128 x 128 block.
struct BlockLinearArgs {
    SegmentRows seg;
    const void *x;               // [num_rows, k]
    const float *x_scales;       // [num_rows, k/128]
    const void *w;               // [E, n, k]
    const float *w_scales;       // [E, ceil(n/128), k/128]
    const void *bias;            // bf16 [E, n] or NULL
    const void *residual;        // bf16 [num_rows, m] or NULL
    float *sums;                 // workspace: block_linear_sums_bytes
    void *out;                   // bf16 [num_rows, m]
    int n, k;
    int act;                     // EP_ACT_*
};

// Bytes that a product of dense rows needs for the sums of its parts, and the most
// that any number of rows up to `rows` needs.
size_t block_linear_sums_bytes(int64_t rows, int n, int k);
size_t block_linear_sums_most(int64_t rows, int n, int k);

hipError_t launch_block_linear(const BlockLinearArgs &a, hipStream_t stream);

struct CastBlocksArgs {
    const void *w;               // bf16 [num, n, k]
    uint8_t *codes;              // [num, n, k] or NULL
    float *scales;               // [num, ceil(n/128), ceil(k/128)]
    uint8_t *codes_t;            // [num, k, n] or NULL
    float *scales_t;             // [num, ceil(k/128), ceil(n/128)]
    int num, n, k;
};

hipError_t launch_cast_blocks(const CastBlocksArgs &a, hipStream_t stream);

// The gated feed-forward block over dense rows.
struct FfnArgs {
    const void *x;               // bf16 [rows, hidden]
    const void *w1, *w2;         // bf16 [2 inter, hidden], [hidden, inter]
    const void *residual;        // bf16 [rows, hidden] or NULL
    void *z;                     // bf16 [rows, 2 inter] or NULL
    void *h;                     // workspace: bf16 [rows, inter]
    float *sums;                 // workspace: gated_ffn_sums_bytes
    void *out;                   // bf16 [rows, hidden]
    int64_t rows;
    int hidden, inter, act;
};

// Bytes that the products of a pass need for the sums of their parts, and the most
// that any number of rows up to `rows` needs.
size_t gated_ffn_sums_bytes(int64_t rows, int hidden, int inter, bool backward);
size_t gated_ffn_sums_most(int64_t rows, int hidden, int inter, bool backward);

hipError_t launch_gated_ffn(const FfnArgs &a, hipStream_t stream);

struct FfnBackwardArgs {
    const void *dout, *x, *z;    // bf16 [rows, hidden], [rows, hidden], [rows, 2 inter]
    const void *w1, *w2;
    const void *dw1_in, *dw2_in; // dw's type, or NULL
    void *dz, *h;                // workspace: bf16 [rows, 2 inter], [rows, inter]
    float *sums;                 // workspace: gated_ffn_sums_bytes
    void *dx;                    // bf16 [rows, hidden] or NULL
    void *dw1, *dw2;             // fp32 or bf16
    int64_t rows;
    int hidden, inter, act;
    bool bf16_out;
};

hipError_t launch_gated_ffn_backward(const FfnBackwardArgs &a, hipStream_t stream);

struct MoeDecodeArgs {
    const void *x;               // bf16 [T, H]
    const int64_t *topk_idx;     // [T, K]
    const float *topk_weights;   // [T, K] or NULL
    const void *w1, *w2;         // [E, n1, H], [E, H, I]; bf16 or e4m3
    const uint8_t *w1_scales, *w2_scales;
    const void *bias1, *bias2;   // bf16 [E, n1], [E, H] or NULL
    const void *res0, *res1;     // bf16 [T, H] or NULL
    void *h;                     // workspace: bf16 [T*K, 2, I], high and low parts
    void *out;                   // bf16 [T, H]
    int32_t *status;             // or NULL
    int T, K, E, H, I, kind;
    bool gated, fp8;
};

hipError_t launch_moe_decode(const MoeDecodeArgs &a, hipStream_t stream);

}  // namespace ep
