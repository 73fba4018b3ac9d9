// Internal declarations of a token's way through a block: the norms around a
// block, the linear of a few rows, the paged 4-bit cache and its attention.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "h3fp4_heads.h"
#include "h3fp4_internal.h"

namespace h3fp4 {

constexpr int kBlockNormMaxK = 32768;

struct BlockNormJob {
    const __nv_bfloat16* x;   // [M][K]
    const __nv_bfloat16* y;   // [M][K] or null
    __nv_bfloat16* x_out;     // [M][K] or null
    __nv_bfloat16* out;       // [M][K] or null
    const float* y_weight;    // [nseg][K] or null, as all vectors
    const float* gate;
    const float* weight;
    const float* shift;
    const float* scale;
    float x_scale, eps;
    bool post, layer;
    float* amax;              // device fp32 or null
    int64_t M;
    int K;
    Segments seg;
};

cudaError_t launch_block_norm(const BlockNormJob& job, cudaStream_t s);

constexpr int kCacheMaxD = 256;
constexpr int kCacheGroup = 16;        // tokens that are stored together
constexpr int kCacheMaxPage = 1024;
constexpr int kCacheMaxSeqs = 1024;

// Elements that a head of D takes in the cache: 64, 128 or 256 (zeros behind D).
constexpr int cache_width(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// A cache, its sequences, and which packed rows of a call belong to them.
struct CacheView {
    uint8_t* pool;            // [n_pages][Hkv][page / 16][18 * cache_width(D)] bytes
    int64_t n_pages;
    const int32_t* table;     // device [nseq][max_pages], page numbers
    const int32_t* length;    // device [nseq]
    const int32_t* row_off;   // device [nseq + 1], or null: row i is sequence i's
    const float* k_gscale;    // device [Hkv], or null: ones
    const float* v_gscale;
    int64_t max_pages;
    int page, Hkv, D, nseq;
};

// Writes the rows k, v [M][Hkv][D] to their places, or (read) reads them back.
struct CacheRowsJob {
    CacheView c;
    HeadsIn k, v;             // append: the rows
    __nv_bfloat16 *k_out, *v_out;  // read: where they go, with the strides of k and v
    int64_t M;
};

cudaError_t launch_cache_append(const CacheRowsJob& job, cudaStream_t s);
cudaError_t launch_cache_read(const CacheRowsJob& job, cudaStream_t s);

struct CacheAttnJob {
    CacheView c;
    HeadsIn q;
    __nv_bfloat16* out;
    int64_t out_row, out_head;
    float* lse;               // [M][Hq] or null
    int64_t M;
    int Hq;
    bool causal;
    float scale;
    uint8_t* ws;
    uint64_t wait_limit_ns;
    int stall;                // self-test: no copies, so every wait runs out
};

size_t cache_attn_workspace_bytes(int D);
cudaError_t launch_cache_attn(const CacheAttnJob& job, cudaStream_t s);

constexpr int kRowsMax = 64;           // rows of the linear of a few rows

struct LinearRowsJob {
    const __nv_bfloat16* x;   // [M][K]
    const uint8_t* w_codes;   // [N][K/2]
    const uint8_t* w_sf;
    const float* w_gscale;
    const float* gate;        // or null: row m at gate + m * gate_stride
    int64_t gate_stride;
    const __nv_bfloat16* bias;   // [N] or null
    const __nv_bfloat16* resid;  // [M][N], with gate
    __nv_bfloat16* out;       // [M][N], or [M][N/2] with swiglu
    bool swiglu;
    int64_t M, N, K;
    uint8_t* ws;
    uint64_t wait_limit_ns;
    int stall;                // self-test: no copies, so every wait runs out
};

size_t linear_rows_workspace_bytes(int64_t M, int64_t N, int64_t K);
cudaError_t launch_linear_rows(const LinearRowsJob& job, cudaStream_t s);

}  // namespace h3fp4
