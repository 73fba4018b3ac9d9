// Internal declarations of the attention-side operators: the per-head norm with
// rotation and the attention to encoder states and shared contexts.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "h3fp4_internal.h"

namespace h3fp4 {

constexpr int kNormMaxD = 256;
constexpr int kAttnMaxD = 128;
constexpr float kLog2E = 1.4426950408889634f;

// One of the tensors the norm runs over.
struct NormTensor {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    int64_t x_row, x_head, y_row, y_head;  // strides in elements
    const float* weight;                   // [nseg][D] or null
    int heads;                             // 0: absent
};

struct NormRopeJob {
    NormTensor t[2];  // queries, keys
    int64_t M;
    int D;
    const float* cos;  // [M][rot/2] or null
    const float* sin;
    int rot;
    bool pairs;
    float eps;
    Segments seg;
};

cudaError_t launch_norm_rope(const NormRopeJob& job, cudaStream_t s);

struct HeadsIn {
    const __nv_bfloat16* p;
    int64_t row, head;
};

struct AttnJob {
    HeadsIn q, k, v, kc, vc;
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float* lse;                // [M][Hq] or null
    int64_t M, T, C;
    int Hq, Hkv, D, nseg;
    const int64_t* q_off;      // host, nseg + 1, validated
    const int64_t* kv_off;
    const uint8_t* key_mask;   // device, T bytes or null
    const uint8_t* ctx_mask;   // device, C bytes or null
    float scale;
    uint8_t* ws;
    int stall;                 // self-test: no loads, so every wait runs out
    uint64_t wait_limit_ns;
};

// Launches the call as `plan` (attn_plan.h, made from `job`) cuts it.
struct AttnPlan;
cudaError_t launch_attn(const AttnJob& job, const AttnPlan& plan, cudaStream_t s);

// The limit set with h3fp4_set_wait_limit_ns.
uint64_t wait_limit_ns();

}  // namespace h3fp4
