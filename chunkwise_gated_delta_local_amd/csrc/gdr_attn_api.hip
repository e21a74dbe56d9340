// Host side of the window attention declared in include/gdr_attn.h: argument checks
// and launch arguments.
#include <cmath>

#include "gdr_attn.hpp"
#include "gdr_checks.hpp"

namespace {

using namespace gdr;

constexpr int kMostHeadDim = 128;

gdr_status_t check_attn(const gdr_attn_problem_t* p, int64_t most_stride) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    if (p->num_kv_heads < 1 || p->num_q_heads < 1 || p->num_q_heads % p->num_kv_heads != 0)
        return fail(GDR_ERR_SHAPE, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)", p->num_q_heads,
                    p->num_kv_heads);
    GDR_TRY(check_tokens(p->batch, p->seq_len, p->num_seqs, p->num_q_heads));
    if (p->head_dim_qk < 1 || p->head_dim_v < 1) return fail(GDR_ERR_SHAPE, "head dimensions must be positive");
    if (p->head_dim_qk > kMostHeadDim || p->head_dim_v > kMostHeadDim)
        return fail(GDR_ERR_UNSUPPORTED, "head dimensions %d, %d not supported (1 to %d)", p->head_dim_qk,
                    p->head_dim_v, kMostHeadDim);
    if (p->window < 1 || p->sinks < 0) return fail(GDR_ERR_SHAPE, "window must be positive and sinks >= 0");
    if ((int64_t)p->window + p->sinks >= (int64_t)1 << 31)
        return fail(GDR_ERR_SHAPE, "sinks + window must be below 2^31");
    if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return fail(GDR_ERR_SHAPE, "scale must be positive and finite");
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    if (!io_or_f32(p->out_dtype, p->io_dtype) || !io_or_f32(p->do_dtype, p->io_dtype) ||
        !io_or_f32(p->grad_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "out_dtype, do_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    const int64_t qw = (int64_t)p->num_q_heads * p->head_dim_qk, kw = (int64_t)p->num_kv_heads * p->head_dim_qk,
                  vw = (int64_t)p->num_kv_heads * p->head_dim_v, ow = (int64_t)p->num_q_heads * p->head_dim_v;
    if (qw > kMostTileStride || vw > kMostTileStride || ow > kMostTileStride)
        return fail(GDR_ERR_SHAPE, "the heads of a token must be at most %lld elements", (long long)kMostTileStride);
    GDR_TRY(check_stride("q_stride", p->q_stride, qw, most_stride));
    GDR_TRY(check_stride("k_stride", p->k_stride, kw, most_stride));
    return check_stride("v_stride", p->v_stride, vw, most_stride);
}

AttnArgs attn_args(const gdr_attn_problem_t* p, const void* q, const void* k, const void* v, void* kc, void* vc,
                   const int32_t* lens, const int32_t* cu, void* ws, void* stream) {
    AttnArgs a{};
    a.p = *p;
    a.Ttot = p->batch * p->seq_len;
    a.q = q; a.k = k; a.v = v; a.kc = kc; a.vc = vc; a.lens = lens; a.cu = cu;
    a.ws = static_cast<float*>(ws);
    a.stream = static_cast<hipStream_t>(stream);
    // rows in 16-byte pieces: every head of every token begins at a 16-byte address
    const int64_t unit = 16 / size_of(p->io_dtype);
    a.vec = p->head_dim_qk % unit == 0 && p->head_dim_v % unit == 0 && p->q_stride % unit == 0 &&
            p->k_stride % unit == 0 && p->v_stride % unit == 0;
    for (const void* x : {q, k, v, (const void*)kc, (const void*)vc}) a.vec = a.vec && aligned(x, 16);
    return a;
}

gdr_status_t check_caches(const gdr_attn_problem_t* p, const void* kc, const void* vc, const int32_t* lens) {
    if ((kc == nullptr) != (vc == nullptr)) return fail(GDR_ERR_NULL, "k_cache and v_cache must both be given or both be NULL");
    if (lens && !kc) return fail(GDR_ERR_NULL, "lens without caches");
    return GDR_OK;
}

}  // namespace

extern "C" {

gdr_status_t gdr_window_attn_fwd_workspace_size(const gdr_attn_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_attn(p, kMostTileStride));
    *bytes = attn_fwd_workspace(*p);
    return GDR_OK;
}

gdr_status_t gdr_window_attn_fwd(const gdr_attn_problem_t* p, const void* q, const void* k, const void* v,
                                 void* k_cache, void* v_cache, const int32_t* lens, const int32_t* cu_dev,
                                 const int32_t* cu_host, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    GDR_TRY(check_attn(p, kMostTileStride));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const int32_t io = p->io_dtype;
    const Ptr ptrs[] = {{q, io, true, "q"}, {k, io, true, "k"}, {v, io, true, "v"}, {k_cache, io, false, "k_cache"},
                        {v_cache, io, false, "v_cache"}, {lens, GDR_F32, false, "lens"}, {o, p->out_dtype, true, "o"},
                        {lse, GDR_F32, false, "lse"}};
    GDR_TRY(check_ptrs(ptrs, p->batch * p->seq_len > 0));
    GDR_TRY(check_caches(p, k_cache, v_cache, lens));
    GDR_TRY(check_workspace(workspace, workspace_bytes, attn_fwd_workspace(*p)));
    AttnArgs a = attn_args(p, q, k, v, k_cache, v_cache, lens, cu_dev, workspace, stream);
    a.k_ld = (int32_t)p->k_stride;
    a.v_ld = (int32_t)p->v_stride;
    a.o = o;
    a.lse = lse;
    return done(launch_attn_fwd(a));
}

gdr_status_t gdr_window_attn_step_workspace_size(const gdr_attn_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_attn(p, kMostStride));
    *bytes = attn_step_workspace(*p);
    return GDR_OK;
}

gdr_status_t gdr_window_attn_step(const gdr_attn_problem_t* p, const void* q, const void* k, const void* v,
                                  void* k_cache, void* v_cache, const int32_t* lens, void* o, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    GDR_TRY(check_attn(p, kMostStride));
    if (p->batch != p->num_seqs || p->seq_len != 1)
        return fail(GDR_ERR_SHAPE, "one token a sequence: batch must equal num_seqs and seq_len 1");
    const int32_t io = p->io_dtype;
    const Ptr ptrs[] = {{q, io, true, "q"}, {k, io, true, "k"}, {v, io, true, "v"}, {k_cache, io, true, "k_cache"},
                        {v_cache, io, true, "v_cache"}, {lens, GDR_F32, true, "lens"}, {o, p->out_dtype, true, "o"}};
    GDR_TRY(check_ptrs(ptrs, p->batch > 0));
    GDR_TRY(check_workspace(workspace, workspace_bytes, attn_step_workspace(*p)));
    AttnArgs a = attn_args(p, q, k, v, k_cache, v_cache, lens, nullptr, workspace, stream);
    a.o = o;
    return done(launch_attn_step(a));
}

gdr_status_t gdr_window_attn_bwd_workspace_size(const gdr_attn_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_attn(p, kMostTileStride));
    *bytes = attn_bwd_workspace(*p);
    return GDR_OK;
}

gdr_status_t gdr_window_attn_bwd(const gdr_attn_problem_t* p, const void* q, const void* k, const void* v,
                                 const void* o, const float* lse, const void* d_o, const int32_t* cu_dev,
                                 const int32_t* cu_host, void* dq, void* dk, void* dv, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    GDR_TRY(check_attn(p, kMostTileStride));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const int32_t io = p->io_dtype, gr = p->grad_dtype;
    const Ptr ptrs[] = {{q, io, true, "q"}, {k, io, true, "k"}, {v, io, true, "v"}, {o, p->out_dtype, true, "o"},
                        {lse, GDR_F32, true, "lse"}, {d_o, p->do_dtype, true, "d_o"}, {dq, gr, true, "dq"},
                        {dk, gr, true, "dk"}, {dv, gr, true, "dv"}};
    GDR_TRY(check_ptrs(ptrs, p->batch * p->seq_len > 0));
    GDR_TRY(check_workspace(workspace, workspace_bytes, attn_bwd_workspace(*p)));
    AttnArgs a = attn_args(p, q, k, v, nullptr, nullptr, nullptr, cu_dev, workspace, stream);
    a.q_ld = (int32_t)p->q_stride;
    a.k_ld = (int32_t)p->k_stride;
    a.v_ld = (int32_t)p->v_stride;
    a.oin = o; a.lse_in = lse; a.d_o = d_o;
    a.dq = dq; a.dk = dk; a.dv = dv;
    // d_o's rows are read in the same pieces (a rounded copy of it lies in the workspace)
    a.vec = a.vec && (p->do_dtype != io || aligned(d_o, 16));
    return done(launch_attn_bwd(a));
}

}  // extern "C"
