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
// which only those under num_rows exist.
struct SegmentRows {
    const int32_t *counts;
    const int32_t *offsets;
    int32_t *status;      // EP_DEV_RECV_OVERFLOW where rows at or past num_rows would be used
    int E;
    int64_t num_rows;
    int64_t pairs;        // upper bound of the rows that hold a pair
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

// The activation function of an EP_ACT_* (0 none, 1 silu, 2 gelu).
inline int act_kind(int act) {
    return act == EP_ACT_SILU || act == EP_ACT_SWIGLU ? 1
           : act == EP_ACT_GELU || act == EP_ACT_GEGLU ? 2 : 0;
}
inline bool act_gated(int act) { return act == EP_ACT_SWIGLU || act == EP_ACT_GEGLU; }

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
