// C ABI of a token's way through a block (h3fp4_block_norm, h3fp4_linear_rows,
// h3fp4_cache_append, h3fp4_cache_read, h3fp4_cache_attn): argument validation and job
// set-up.  Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "h3fp4_token.h"
#include "spans.h"

namespace h3fp4 {
namespace {

bool overlap(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + b_bytes && y < x + a_bytes;
}

bool overlap(const void* a, const void* b, int64_t bytes)
{
    return overlap(a, (uint64_t)bytes, b, (uint64_t)bytes);
}

Span run(const void* p, uint64_t bytes) { return Span{p, 1, 0, 1, 0, p ? bytes : 0}; }

Span view(const h3fp4_heads& t, int64_t rows, int64_t heads, int D)
{
    return Span{t.ptr, rows, 2 * t.row_stride, heads, 2 * t.head_stride, 2 * (uint64_t)D};
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A cache and its sequences, of a call of M rows.
h3fp4_status cache_view(const h3fp4_cache* c, int64_t M, CacheView* out)
{
    if (!c) return H3FP4_ERR_INVALID;
    if (M < 0 || M > INT32_MAX - 255) return H3FP4_ERR_SHAPE;
    if (c->dim < 16 || c->dim > kCacheMaxD || c->dim % 16 != 0 || c->heads < 1 || c->heads > 4096 ||
        c->page < kCacheGroup || c->page > kCacheMaxPage || c->page % kCacheGroup != 0 || c->nseq < 1 ||
        c->nseq > kCacheMaxSeqs || c->n_pages < 1 || c->n_pages > INT32_MAX || c->max_pages < 1 ||
        c->max_pages > INT32_MAX)
        return H3FP4_ERR_SHAPE;
    if (!c->pool || !c->table || !c->length) return H3FP4_ERR_INVALID;
    if (!c->row_off && M != c->nseq) return H3FP4_ERR_INVALID;
    if (!aligned16(c->pool) || !aligned4(c->table) || !aligned4(c->length) || !aligned4(c->row_off) ||
        !aligned4(c->k_gscale) || !aligned4(c->v_gscale))
        return H3FP4_ERR_ALIGN;
    out->pool = static_cast<uint8_t*>(c->pool);
    out->n_pages = c->n_pages;
    out->table = c->table;
    out->length = c->length;
    out->row_off = c->row_off;
    out->k_gscale = c->k_gscale;
    out->v_gscale = c->v_gscale;
    out->max_pages = c->max_pages;
    out->page = (int)c->page;
    out->Hkv = (int)c->heads;
    out->D = (int)c->dim;
    out->nseq = (int)c->nseq;
    return H3FP4_OK;
}

// Whether `s`, which a call writes, shares memory with the cache's pool or what describes its sequences.
bool overlaps_cache(const Span& s, const CacheView& c)
{
    const uint64_t page = h3fp4_cache_page_bytes(c.Hkv, c.D, c.page), heads = 4 * (uint64_t)c.Hkv;
    for (const Span& o : {run(c.pool, (uint64_t)c.n_pages * page), run(c.table, 4 * (uint64_t)c.nseq * (uint64_t)c.max_pages),
                          run(c.length, 4 * (uint64_t)c.nseq), run(c.row_off, 4 * ((uint64_t)c.nseq + 1)),
                          run(c.k_gscale, heads), run(c.v_gscale, heads)})
        if (overlap(s, o)) return true;
    return false;
}

h3fp4_status cache_rows(const h3fp4_heads* k, const h3fp4_heads* v, int64_t M, const h3fp4_cache* cache, bool read,
                        cudaStream_t stream)
{
    CacheRowsJob job{};
    h3fp4_status st = cache_view(cache, M, &job.c);
    if (st != H3FP4_OK) return st;
    for (const h3fp4_heads* t : {k, v})
        if ((st = read ? check_out(t, M, job.c.Hkv, job.c.D) : check_in(t, M)) != H3FP4_OK) return st;
    if (M > 0) {
        const Span rows[] = {view(*k, M, job.c.Hkv, job.c.D), view(*v, M, job.c.Hkv, job.c.D)};
        const Span pool = run(job.c.pool, (uint64_t)job.c.n_pages * h3fp4_cache_page_bytes(job.c.Hkv, job.c.D, job.c.page));
        if (read && overlap(rows[0], rows[1])) return H3FP4_ERR_INVALID;
        for (const Span& s : rows)
            if (read ? overlaps_cache(s, job.c) : overlap(s, pool)) return H3FP4_ERR_INVALID;
    }
    if ((st = check_device()) != H3FP4_OK) return st;
    if (M == 0) return H3FP4_OK;
    job.k = in(k);
    job.v = in(v);
    job.k_out = static_cast<__nv_bfloat16*>(k->ptr);
    job.v_out = static_cast<__nv_bfloat16*>(v->ptr);
    job.M = M;
    const cudaError_t e = read ? launch_cache_read(job, stream) : launch_cache_append(job, stream);
    return e == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

h3fp4_status rows_shape(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || M > kRowsMax || N < 8 || N % 8 != 0 || N > (1 << 24)) return H3FP4_ERR_SHAPE;
    if (K < 64 || K % 64 != 0 || K > (1 << 16)) return H3FP4_ERR_SHAPE;
    return H3FP4_OK;
}

}  // namespace
}  // namespace h3fp4

using namespace h3fp4;

extern "C" {

h3fp4_status h3fp4_block_norm(const void* x, const void* y, int64_t M, int64_t K, const float* y_weight,
                              const float* gate, float x_scale, const float* weight, const float* shift,
                              const float* scale, const int64_t* seg_off, int nseg, float eps, void* x_out, void* out,
                              float* out_amax, int flags, cudaStream_t stream)
{
    if (M < 0 || M > INT32_MAX || K < 8 || K > kBlockNormMaxK || K % 8 != 0) return H3FP4_ERR_SHAPE;
    if (flags & ~(H3FP4_NORM_POST | H3FP4_NORM_LAYER)) return H3FP4_ERR_INVALID;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(x_scale)) return H3FP4_ERR_INVALID;
    if (M > 0) {
        if (!x || (!out && !x_out)) return H3FP4_ERR_INVALID;
        if (!out && (weight || shift || scale || out_amax || (flags & H3FP4_NORM_LAYER))) return H3FP4_ERR_INVALID;
        if (!y && (x_out || y_weight || gate || (flags & H3FP4_NORM_POST))) return H3FP4_ERR_INVALID;
        if (y_weight && !(flags & H3FP4_NORM_POST)) return H3FP4_ERR_INVALID;
    }
    for (const void* p : {x, y, static_cast<const void*>(y_weight), static_cast<const void*>(gate),
                          static_cast<const void*>(weight), static_cast<const void*>(shift),
                          static_cast<const void*>(scale), static_cast<const void*>(x_out),
                          static_cast<const void*>(out)})
        if (!aligned16(p)) return H3FP4_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(out_amax) & 3u) return H3FP4_ERR_ALIGN;
    // an output is an input itself or apart from it, and apart from the other output
    const int64_t bytes = M * K * 2;
    if (overlap(x_out, out, bytes)) return H3FP4_ERR_INVALID;
    for (const void* o : {static_cast<const void*>(x_out), static_cast<const void*>(out)})
        for (const void* i : {x, y})
            if (o != i && overlap(o, i, bytes)) return H3FP4_ERR_INVALID;
    BlockNormJob job{};
    h3fp4_status st = make_segments(seg_off, seg_off == nullptr && nseg <= 0 ? 1 : nseg, M, &job.seg);
    if (st != H3FP4_OK) return st;
    for (const float* v : {y_weight, gate, weight, shift, scale}) {
        const uint64_t vec = 4 * (uint64_t)job.seg.nseg * (uint64_t)K;
        if (overlap(x_out, (uint64_t)bytes, v, vec) || overlap(out, (uint64_t)bytes, v, vec) || overlap(out_amax, 4, v, vec))
            return H3FP4_ERR_INVALID;
    }
    for (const void* o : {x, y, static_cast<const void*>(x_out), static_cast<const void*>(out)})
        if (overlap(out_amax, 4, o, (uint64_t)bytes)) return H3FP4_ERR_INVALID;
    if ((st = check_device()) != H3FP4_OK) return st;
    job.x = static_cast<const __nv_bfloat16*>(x);
    job.y = static_cast<const __nv_bfloat16*>(y);
    job.x_out = static_cast<__nv_bfloat16*>(x_out);
    job.out = static_cast<__nv_bfloat16*>(out);
    job.y_weight = y_weight;
    job.gate = gate;
    job.weight = weight;
    job.shift = shift;
    job.scale = scale;
    job.x_scale = x_scale;
    job.eps = eps;
    job.post = (flags & H3FP4_NORM_POST) != 0;
    job.layer = (flags & H3FP4_NORM_LAYER) != 0;
    job.amax = out_amax;
    job.M = M;
    job.K = (int)K;
    return launch_block_norm(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

size_t h3fp4_linear_rows_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    return rows_shape(M, N, K) == H3FP4_OK ? linear_rows_workspace_bytes(M, N, K) : 0;
}

h3fp4_status h3fp4_linear_rows(const void* x, int64_t M, int64_t N, int64_t K, const void* w_codes, const void* w_sf,
                               const float* w_gscale, const float* gate, int64_t gate_stride, const void* bias,
                               const void* resid, void* out, int flags, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    h3fp4_status st = rows_shape(M, N, K);
    if (st != H3FP4_OK) return st;
    if (flags & ~(H3FP4_EPI_BIAS | H3FP4_EPI_GATE_RESID | H3FP4_EPI_SWIGLU)) return H3FP4_ERR_INVALID;
    const bool swiglu = (flags & H3FP4_EPI_SWIGLU) != 0, gated = (flags & H3FP4_EPI_GATE_RESID) != 0;
    if (swiglu && gated) return H3FP4_ERR_INVALID;
    if (swiglu && N % 256 != 0) return H3FP4_ERR_SHAPE;
    if (!x || !w_codes || !w_sf || !w_gscale || !out || !ws) return H3FP4_ERR_INVALID;
    if (((flags & H3FP4_EPI_BIAS) != 0) != (bias != nullptr) || gated != (gate != nullptr) ||
        gated != (resid != nullptr))
        return H3FP4_ERR_INVALID;
    if (gated && gate_stride != 0 && gate_stride < N) return H3FP4_ERR_INVALID;
    for (const void* p : {x, w_codes, w_sf, bias, resid, static_cast<const void*>(out), static_cast<const void*>(ws)})
        if (!aligned16(p)) return H3FP4_ERR_ALIGN;
    if (!aligned4(w_gscale) || !aligned4(gate)) return H3FP4_ERR_ALIGN;
    const size_t need = linear_rows_workspace_bytes(M, N, K);
    if (ws_bytes < need) return H3FP4_ERR_INVALID;
    // resid may be out itself; nothing else may overlap it, or the workspace
    const uint64_t outs = (uint64_t)(M * (swiglu ? N / 2 : N)) * 2;
    if (out != resid && overlap(out, outs, resid, outs)) return H3FP4_ERR_INVALID;
    const struct {
        const void* p;
        int64_t bytes;
    } read[] = {{w_gscale, 4}, {x, M * K * 2}, {w_codes, N * K / 2}, {w_sf, (N + 127) / 128 * 128 * K / 16}, {bias, N * 2},
                {gate, ((M - 1) * gate_stride + N) * 4}};
    for (const auto& r : read)
        if (overlap(out, outs, r.p, (uint64_t)r.bytes) || overlap(ws, need, r.p, (uint64_t)r.bytes))
            return H3FP4_ERR_INVALID;
    if (overlap(out, outs, ws, need) || overlap(resid, outs, ws, need)) return H3FP4_ERR_INVALID;
    if ((st = check_device()) != H3FP4_OK) return st;
    LinearRowsJob job{};
    job.x = static_cast<const __nv_bfloat16*>(x);
    job.w_codes = static_cast<const uint8_t*>(w_codes);
    job.w_sf = static_cast<const uint8_t*>(w_sf);
    job.w_gscale = w_gscale;
    job.gate = gate;
    job.gate_stride = gate_stride;
    job.bias = static_cast<const __nv_bfloat16*>(bias);
    job.resid = static_cast<const __nv_bfloat16*>(resid);
    job.out = static_cast<__nv_bfloat16*>(out);
    job.swiglu = swiglu;
    job.M = M;
    job.N = N;
    job.K = K;
    job.ws = static_cast<uint8_t*>(ws);
    job.wait_limit_ns = wait_limit_ns();
    return launch_linear_rows(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

h3fp4_status h3fp4_selftest_linear_rows_timeout(void* ws, uint64_t limit_ns, cudaStream_t stream)
{
    if (!ws) return H3FP4_ERR_INVALID;
    if (!aligned16(ws)) return H3FP4_ERR_ALIGN;
    const h3fp4_status st = check_device();
    if (st != H3FP4_OK) return st;
    // One and nine rows (the one-kernel and the other form) of 256 columns and 128 outputs, all data (whatever
    // it is) in the workspace of another size.
    uint8_t* data = static_cast<uint8_t*>(ws) + linear_rows_workspace_bytes(9, 128, 256);
    LinearRowsJob job{};
    job.x = reinterpret_cast<const __nv_bfloat16*>(data);
    job.w_codes = data;
    job.w_sf = data;
    job.w_gscale = reinterpret_cast<const float*>(data);
    job.out = reinterpret_cast<__nv_bfloat16*>(data + 128 * 128);
    job.N = 128;
    job.K = 256;
    job.ws = static_cast<uint8_t*>(ws);
    job.wait_limit_ns = limit_ns ? limit_ns : 1;
    job.stall = 1;
    for (int rows : {1, 9}) {
        job.M = rows;
        if (launch_linear_rows(job, stream) != cudaSuccess) return H3FP4_ERR_CUDA;
    }
    return H3FP4_OK;
}

size_t h3fp4_cache_page_bytes(int heads, int dim, int page)
{
    if (heads < 1 || heads > 4096 || dim < 16 || dim > kCacheMaxD || dim % 16 != 0 || page < kCacheGroup ||
        page > kCacheMaxPage || page % kCacheGroup != 0)
        return 0;
    return (size_t)heads * (size_t)page * (size_t)(cache_width(dim) * 9 / 8);
}

h3fp4_status h3fp4_cache_append(const h3fp4_heads* k, const h3fp4_heads* v, int64_t M, const h3fp4_cache* cache,
                                cudaStream_t stream)
{
    return cache_rows(k, v, M, cache, false, stream);
}

h3fp4_status h3fp4_cache_read(const h3fp4_heads* k, const h3fp4_heads* v, int64_t M, const h3fp4_cache* cache,
                              cudaStream_t stream)
{
    return cache_rows(k, v, M, cache, true, stream);
}

size_t h3fp4_cache_attn_workspace_bytes(int dim)
{
    return dim < 16 || dim > kCacheMaxD || dim % 16 != 0 ? 0 : cache_attn_workspace_bytes(dim);
}

h3fp4_status h3fp4_cache_attn(const h3fp4_heads* q, int64_t M, int Hq, const h3fp4_cache* cache, float scale,
                              const h3fp4_heads* out, float* lse, int flags, void* ws, size_t ws_bytes,
                              cudaStream_t stream)
{
    CacheAttnJob job{};
    h3fp4_status st = cache_view(cache, M, &job.c);
    if (st != H3FP4_OK) return st;
    if (Hq < 1 || Hq % job.c.Hkv != 0 || M * (int64_t)Hq > INT32_MAX) return H3FP4_ERR_SHAPE;
    if (flags & ~H3FP4_CAUSAL) return H3FP4_ERR_INVALID;
    if (!(scale > 0.0f) || std::isinf(scale * kLog2E)) return H3FP4_ERR_INVALID;
    if ((st = check_in(q, M)) != H3FP4_OK || (st = check_out(out, M, Hq, job.c.D)) != H3FP4_OK) return st;
    if (!ws || ws_bytes < cache_attn_workspace_bytes(job.c.D)) return H3FP4_ERR_INVALID;
    if (!aligned16(ws) || !aligned4(lse)) return H3FP4_ERR_ALIGN;
    if (M > 0) {
        const Span qs = view(*q, M, Hq, job.c.D), outs = view(*out, M, Hq, job.c.D);
        const Span sums = run(lse, 4 * (uint64_t)M * (uint64_t)Hq), work = run(ws, cache_attn_workspace_bytes(job.c.D));
        if (overlap(outs, qs) || overlap(sums, qs) || overlap(work, qs) || overlap(outs, sums) || overlap(outs, work) ||
            overlap(sums, work))
            return H3FP4_ERR_INVALID;
        for (const Span& s : {outs, sums, work})
            if (overlaps_cache(s, job.c)) return H3FP4_ERR_INVALID;
    }
    if ((st = check_device()) != H3FP4_OK) return st;
    if (M == 0) return H3FP4_OK;
    job.q = in(q);
    job.out = static_cast<__nv_bfloat16*>(out->ptr);
    job.out_row = out->row_stride;
    job.out_head = out->head_stride;
    job.lse = lse;
    job.M = M;
    job.Hq = Hq;
    job.causal = (flags & H3FP4_CAUSAL) != 0;
    job.scale = scale;
    job.ws = static_cast<uint8_t*>(ws);
    job.wait_limit_ns = wait_limit_ns();
    return launch_cache_attn(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

h3fp4_status h3fp4_selftest_cache_attn_timeout(void* ws, uint64_t limit_ns, cudaStream_t stream)
{
    if (!ws) return H3FP4_ERR_INVALID;
    if (!aligned16(ws)) return H3FP4_ERR_ALIGN;
    const h3fp4_status st = check_device();
    if (st != H3FP4_OK) return st;
    // One row of one head of 64 over a page of 16 tokens, in the workspace's last bytes: a length and a
    // page number of 0x01010101, so that the page is full and not one of the pool's.
    uint8_t* data = static_cast<uint8_t*>(ws) + (cache_attn_workspace_bytes(64) - 1024) / 16 * 16;
    if (cudaMemsetAsync(data, 1, 512, stream) != cudaSuccess) return H3FP4_ERR_CUDA;
    CacheAttnJob job{};
    job.c.pool = data;
    job.c.n_pages = job.c.max_pages = job.c.Hkv = job.c.nseq = 1;
    job.c.table = job.c.length = reinterpret_cast<const int32_t*>(data);
    job.c.page = kCacheGroup;
    job.c.D = 64;
    job.q = HeadsIn{reinterpret_cast<const __nv_bfloat16*>(data), 64, 64};
    job.out = reinterpret_cast<__nv_bfloat16*>(data + 512);
    job.out_row = job.out_head = 64;
    job.M = job.Hq = 1;
    job.scale = 1.0f;
    job.ws = static_cast<uint8_t*>(ws);
    job.wait_limit_ns = limit_ns ? limit_ns : 1;
    job.stall = 1;
    return launch_cache_attn(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

}  // extern "C"
