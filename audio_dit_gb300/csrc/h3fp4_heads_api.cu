// C ABI of the attention-side operators (h3fp4_qk_norm_rope, h3fp4_cross_attn,
// h3fp4_shared_attn): argument validation and job set-up.  Nothing here
// allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "attn_plan.h"
#include "h3fp4_heads.h"

namespace h3fp4 {

namespace {
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements: row pitches below the 2^40 bytes a TMA map holds
}  // namespace

// Strides are positive multiples of 8 elements (16 bytes).
static bool good_strides(const h3fp4_heads& t)
{
    return t.row_stride > 0 && t.head_stride > 0 && t.row_stride % 8 == 0 && t.head_stride % 8 == 0 &&
           t.row_stride <= kMaxStride && t.head_stride <= kMaxStride;
}

// An input of `rows` rows: H3FP4_OK, or what is wrong with it.
h3fp4_status check_in(const h3fp4_heads* t, int64_t rows)
{
    if (rows == 0) return H3FP4_OK;
    if (!t || !t->ptr) return H3FP4_ERR_INVALID;
    if (!aligned16(t->ptr) || !good_strides(*t)) return H3FP4_ERR_ALIGN;
    return H3FP4_OK;
}

// An output: as an input, and no two of its elements in one place.
h3fp4_status check_out(const h3fp4_heads* t, int64_t rows, int heads, int D)
{
    const h3fp4_status st = check_in(t, rows);
    if (st != H3FP4_OK || rows == 0) return st;
    const bool rows_outer = t->row_stride >= t->head_stride;
    const int64_t inner = rows_outer ? t->head_stride : t->row_stride;
    const int64_t outer = rows_outer ? t->row_stride : t->head_stride;
    const int64_t n_inner = rows_outer ? heads : rows, n_outer = rows_outer ? rows : heads;
    if (n_inner > 1 && inner < D) return H3FP4_ERR_INVALID;
    if (n_outer > 1 && (n_inner - 1) * inner + D > outer) return H3FP4_ERR_INVALID;
    return H3FP4_OK;
}

HeadsIn in(const h3fp4_heads* t)
{
    if (!t) return HeadsIn{nullptr, 0, 0};
    return HeadsIn{static_cast<const __nv_bfloat16*>(t->ptr), t->row_stride, t->head_stride};
}

namespace {

constexpr int64_t kMaxRows = INT32_MAX - 255;  // rows are counted in 32 bits, up to two tiles past the last
constexpr int kMaxHeads = INT32_MAX - 255;     // the norm's heads too, up to a warp's places past the last

bool same_view(const h3fp4_heads& a, const h3fp4_heads& b)
{
    return a.ptr == b.ptr && a.row_stride == b.row_stride && a.head_stride == b.head_stride;
}

bool good_table(const int64_t* off, int nseg, int64_t rows)
{
    if (off[0] != 0 || off[nseg] != rows) return false;
    for (int i = 0; i < nseg; ++i)
        if (off[i + 1] < off[i]) return false;
    return true;
}

// Sizes and segment tables of the attention calls, into `job`.  `one_q` and
// `one_kv` (two elements each) hold the tables of a call without any.
h3fp4_status attn_sizes(int64_t M, int64_t T, int64_t C, int Hq, int Hkv, int D, const int64_t* q_off,
                        const int64_t* kv_off, int nseg, int64_t* one_q, int64_t* one_kv, AttnJob* job)
{
    if (M < 0 || T < 0 || C < 0 || M > kMaxRows || T > kMaxRows || C > kMaxRows) return H3FP4_ERR_SHAPE;
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 8 || D > kAttnMaxD || D % 8 != 0) return H3FP4_ERR_SHAPE;
    if (M * (int64_t)Hq > INT32_MAX) return H3FP4_ERR_SHAPE;
    if ((q_off == nullptr) != (kv_off == nullptr)) return H3FP4_ERR_INVALID;
    if (q_off == nullptr) {
        if (nseg > 1) return H3FP4_ERR_INVALID;
        one_q[0] = one_kv[0] = 0;
        one_q[1] = M;
        one_kv[1] = T;
        q_off = one_q;
        kv_off = one_kv;
        nseg = 1;
    }
    if (nseg < 1 || nseg > H3FP4_ATTN_MAX_SEGMENTS) return H3FP4_ERR_SHAPE;
    if (!good_table(q_off, nseg, M) || !good_table(kv_off, nseg, T)) return H3FP4_ERR_INVALID;
    job->M = M;
    job->T = T;
    job->C = C;
    job->Hq = Hq;
    job->Hkv = Hkv;
    job->D = D;
    job->nseg = nseg;
    job->q_off = q_off;
    job->kv_off = kv_off;
    return H3FP4_OK;
}

h3fp4_status attn(const h3fp4_heads* q, const h3fp4_heads* k, const h3fp4_heads* v, const h3fp4_heads* kc,
                  const h3fp4_heads* vc, int64_t M, int64_t T, int64_t C, int Hq, int Hkv, int D,
                  const int64_t* q_off, const int64_t* kv_off, int nseg, const uint8_t* key_mask,
                  const uint8_t* ctx_mask, float scale, const h3fp4_heads* out, float* lse, void* ws,
                  size_t ws_bytes, cudaStream_t stream)
{
    AttnJob job{};
    int64_t one_q[2], one_kv[2];
    h3fp4_status st = attn_sizes(M, T, C, Hq, Hkv, D, q_off, kv_off, nseg, one_q, one_kv, &job);
    if (st != H3FP4_OK) return st;
    // (the kernel's exponents are in base 2)
    if (!(scale > 0.0f) || std::isinf(scale * kLog2E)) return H3FP4_ERR_INVALID;
    if ((st = check_in(q, M)) != H3FP4_OK || (st = check_in(k, T)) != H3FP4_OK || (st = check_in(v, T)) != H3FP4_OK ||
        (st = check_in(kc, C)) != H3FP4_OK || (st = check_in(vc, C)) != H3FP4_OK ||
        (st = check_out(out, M, Hq, D)) != H3FP4_OK)
        return st;
    const AttnPlan plan = make_plan(job);
    if (plan.bytes == 0) return H3FP4_ERR_SHAPE;
    if (!ws || ws_bytes < plan.bytes) return H3FP4_ERR_INVALID;
    if (!aligned16(ws) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return H3FP4_ERR_ALIGN;
    if (M > 0 && (out->ptr == q->ptr || (T > 0 && (out->ptr == k->ptr || out->ptr == v->ptr)) ||
                  (C > 0 && (out->ptr == kc->ptr || out->ptr == vc->ptr))))
        return H3FP4_ERR_INVALID;
    if ((st = check_device()) != H3FP4_OK) return st;
    if (M == 0) return H3FP4_OK;
    job.q = in(q);
    job.k = in(k);
    job.v = in(v);
    job.kc = in(kc);
    job.vc = in(vc);
    job.out = static_cast<__nv_bfloat16*>(out->ptr);
    job.out_row = out->row_stride;
    job.out_head = out->head_stride;
    job.lse = lse;
    job.key_mask = key_mask;
    job.ctx_mask = ctx_mask;
    job.scale = scale;
    job.ws = static_cast<uint8_t*>(ws);
    job.wait_limit_ns = wait_limit_ns();
    return launch_attn(job, plan, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

}  // namespace
}  // namespace h3fp4

using namespace h3fp4;

extern "C" {

h3fp4_status h3fp4_qk_norm_rope(const h3fp4_heads* q, const h3fp4_heads* k, int64_t M, int Hq, int Hk, int D,
                                const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                                int rot, const int64_t* seg_off, int nseg, float eps, const h3fp4_heads* q_out,
                                const h3fp4_heads* k_out, int flags, cudaStream_t stream)
{
    if (M < 0 || M > INT32_MAX || D < 8 || D > kNormMaxD || D % 8 != 0) return H3FP4_ERR_SHAPE;
    if (rot < 0 || rot > D || rot % 16 != 0) return H3FP4_ERR_SHAPE;
    const bool with_k = k != nullptr;
    if (Hq < 1 || Hq > kMaxHeads || (with_k && (Hk < 1 || Hk > kMaxHeads))) return H3FP4_ERR_SHAPE;
    if (flags & ~H3FP4_ROPE_PAIRS) return H3FP4_ERR_INVALID;
    if (with_k != (k_out != nullptr) || !q || !q_out) return H3FP4_ERR_INVALID;
    if (!(eps >= 0.0f) || std::isinf(eps)) return H3FP4_ERR_INVALID;
    if (M > 0 && rot > 0 && (!cos || !sin)) return H3FP4_ERR_INVALID;
    h3fp4_status st;
    if ((st = check_in(q, M)) != H3FP4_OK || (st = check_out(q_out, M, Hq, D)) != H3FP4_OK) return st;
    if (with_k && ((st = check_in(k, M)) != H3FP4_OK || (st = check_out(k_out, M, Hk, D)) != H3FP4_OK)) return st;
    if (!aligned16(q_weight) || !aligned16(k_weight) || (rot > 0 && (!aligned16(cos) || !aligned16(sin))))
        return H3FP4_ERR_ALIGN;
    // in place means the very same view; another view of the same start overlaps
    if (M > 0 && q_out->ptr == q->ptr && !same_view(*q_out, *q)) return H3FP4_ERR_INVALID;
    if (M > 0 && with_k &&
        ((k_out->ptr == k->ptr && !same_view(*k_out, *k)) || q_out->ptr == k->ptr || k_out->ptr == q->ptr ||
         q_out->ptr == k_out->ptr))
        return H3FP4_ERR_INVALID;
    NormRopeJob job{};
    if ((st = make_segments(seg_off, seg_off == nullptr && nseg <= 0 ? 1 : nseg, M, &job.seg)) != H3FP4_OK) return st;
    if ((st = check_device()) != H3FP4_OK) return st;
    if (M == 0) return H3FP4_OK;
    auto tensor = [](const h3fp4_heads& x, const h3fp4_heads& y, const float* w, int heads) {
        return NormTensor{static_cast<const __nv_bfloat16*>(x.ptr), static_cast<__nv_bfloat16*>(y.ptr),
                          x.row_stride, x.head_stride, y.row_stride, y.head_stride, w, heads};
    };
    job.t[0] = tensor(*q, *q_out, q_weight, Hq);
    if (with_k) job.t[1] = tensor(*k, *k_out, k_weight, Hk);
    job.M = M;
    job.D = D;
    job.cos = cos;
    job.sin = sin;
    job.rot = rot;
    job.pairs = (flags & H3FP4_ROPE_PAIRS) != 0;
    job.eps = eps;
    return launch_norm_rope(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

h3fp4_status h3fp4_cross_attn(const h3fp4_heads* q, const h3fp4_heads* k, const h3fp4_heads* v, int64_t M, int64_t T,
                              int Hq, int Hkv, int D, const int64_t* q_off, const int64_t* kv_off, int nseg,
                              const uint8_t* key_mask, float scale, const h3fp4_heads* out, float* lse, void* ws,
                              size_t ws_bytes, cudaStream_t stream)
{
    return attn(q, k, v, nullptr, nullptr, M, T, 0, Hq, Hkv, D, q_off, kv_off, nseg, key_mask, nullptr, scale, out,
                lse, ws, ws_bytes, stream);
}

h3fp4_status h3fp4_shared_attn(const h3fp4_heads* q, const h3fp4_heads* k, const h3fp4_heads* v,
                               const h3fp4_heads* k_ctx, const h3fp4_heads* v_ctx, int64_t M, int64_t T, int64_t C,
                               int Hq, int Hkv, int D, const int64_t* q_off, const int64_t* kv_off, int nseg,
                               const uint8_t* key_mask, const uint8_t* ctx_mask, float scale,
                               const h3fp4_heads* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    return attn(q, k, v, k_ctx, v_ctx, M, T, C, Hq, Hkv, D, q_off, kv_off, nseg, key_mask, ctx_mask, scale, out, lse,
                ws, ws_bytes, stream);
}

h3fp4_status h3fp4_selftest_attn_timeout(void* ws, uint64_t limit_ns, cudaStream_t stream)
{
    if (!ws) return H3FP4_ERR_INVALID;
    if (!aligned16(ws)) return H3FP4_ERR_ALIGN;
    const h3fp4_status st = check_device();
    if (st != H3FP4_OK) return st;
    // One query and one key of one head of 64, in the workspace behind the status word.
    int64_t one_q[2], one_kv[2];
    AttnJob job{};
    if (attn_sizes(1, 1, 0, 1, 1, 64, nullptr, nullptr, 1, one_q, one_kv, &job) != H3FP4_OK) return H3FP4_ERR_INVALID;
    __nv_bfloat16* data = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(ws) + 256);
    job.q = HeadsIn{data, 64, 64};
    job.k = HeadsIn{data + 128, 64, 64};
    job.v = HeadsIn{data + 256, 64, 64};
    job.out = data + 384;
    job.out_row = job.out_head = 64;
    job.scale = 1.0f;
    job.ws = static_cast<uint8_t*>(ws);
    job.stall = 1;
    job.wait_limit_ns = limit_ns ? limit_ns : 1;
    return launch_attn(job, make_plan(job), stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

size_t h3fp4_attn_workspace_bytes(int64_t M, int64_t T, int64_t C, int Hq, int Hkv, int D, const int64_t* q_off,
                                  const int64_t* kv_off, int nseg)
{
    AttnJob job{};
    int64_t one_q[2], one_kv[2];
    if (attn_sizes(M, T, C, Hq, Hkv, D, q_off, kv_off, nseg, one_q, one_kv, &job) != H3FP4_OK) return 0;
    return make_plan(job).bytes;
}

}  // extern "C"
