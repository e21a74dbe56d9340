// Host side of the layer operators declared in include/gdr_mixer.h: argument
// checks and launch arguments.
#include "gdr_mixer.hpp"

namespace {

using gdr::fail;
using gdr::kMostTileStride;

bool is_dtype(int32_t t) { return t == GDR_F32 || t == GDR_BF16; }
// a type that may be the io type or fp32
bool io_or_f32(int32_t t, int32_t io) { return t == io || t == GDR_F32; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

struct Ptr {
    const void* p;
    int32_t dtype;
    bool required;
    const char* name;
};
template <int N>
gdr_status_t check_ptrs(const Ptr (&ptrs)[N], bool any) {
    for (const Ptr& t : ptrs) {
        if (t.required && any && !t.p) return fail(GDR_ERR_NULL, "%s is required", t.name);
        if (!aligned(t.p, (size_t)gdr::size_of(t.dtype)))
            return fail(GDR_ERR_SHAPE, "%s is not aligned to its element type", t.name);
    }
    return GDR_OK;
}

gdr_status_t check_tokens(int64_t batch, int64_t seq_len, int32_t num_seqs, int32_t channels) {
    if (batch < 0 || seq_len < 0 || num_seqs < 0)
        return fail(GDR_ERR_SHAPE, "batch, seq_len and num_seqs must be >= 0");
    if (channels < 1) return fail(GDR_ERR_SHAPE, "channels must be positive (got %d)", channels);
    const int64_t most = ((int64_t)1 << 31) - 1 - 64;
    if (batch > most || seq_len > most || (batch > 0 && seq_len > most / batch))
        return fail(GDR_ERR_SHAPE, "total tokens exceed the int32 token index");
    return GDR_OK;
}

// Sequences of a call; *max_len: the longest (host).
gdr_status_t check_seqs(int64_t batch, int64_t seq_len, int32_t num_seqs, const int32_t* cu_dev,
                        const int32_t* cu_host, int64_t* max_len) {
    if ((cu_dev == nullptr) != (cu_host == nullptr))
        return fail(GDR_ERR_NULL, "cu_seqlens_dev and cu_seqlens_host must both be given or both be NULL");
    if (!cu_host) {
        if (num_seqs != batch)
            return fail(GDR_ERR_SHAPE, "num_seqs (%d) must equal batch (%lld) without cu_seqlens", num_seqs,
                        (long long)batch);
        *max_len = seq_len;
        return GDR_OK;
    }
    if (batch != 1) return fail(GDR_ERR_SEQLENS, "cu_seqlens requires batch == 1");
    if (num_seqs < 1) return fail(GDR_ERR_SEQLENS, "cu_seqlens needs num_seqs >= 1");
    if (!aligned(cu_dev, 4)) return fail(GDR_ERR_SHAPE, "cu_seqlens_dev is not aligned to its element type");
    if (cu_host[0] != 0) return fail(GDR_ERR_SEQLENS, "cu_seqlens[0] = %d, expected 0", cu_host[0]);
    *max_len = 0;
    for (int32_t n = 0; n < num_seqs; ++n) {
        if (cu_host[n + 1] < cu_host[n]) return fail(GDR_ERR_SEQLENS, "cu_seqlens decreases at %d", n);
        const int64_t len = (int64_t)cu_host[n + 1] - cu_host[n];
        *max_len = len > *max_len ? len : *max_len;
    }
    if ((int64_t)cu_host[num_seqs] != seq_len)
        return fail(GDR_ERR_SEQLENS, "cu_seqlens[N] = %d but seq_len = %lld", cu_host[num_seqs], (long long)seq_len);
    return GDR_OK;
}

constexpr int64_t kMostStride = (int64_t)1 << 40;
gdr_status_t check_stride(const char* name, int64_t stride, int64_t row, int64_t most = kMostStride) {
    if (stride < row || stride > most)
        return fail(GDR_ERR_SHAPE, "%s (%lld) must be at least the row's %lld elements and at most %lld", name,
                    (long long)stride, (long long)row, (long long)most);
    return GDR_OK;
}

gdr_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDR_OK;
    if (!ws) return fail(GDR_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(GDR_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (have < need) return fail(GDR_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return GDR_OK;
}

gdr_status_t done(hipError_t e) {
    if (e == hipErrorInvalidConfiguration) return fail(GDR_ERR_SHAPE, "problem too large for one launch");
    if (e != hipSuccess) return fail(GDR_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    gdr::clear_error();
    return GDR_OK;
}

#define GDR_TRY(expr)                            \
    do {                                         \
        const gdr_status_t st_ = (expr);         \
        if (st_ != GDR_OK) return st_;           \
    } while (0)

// ---------------------------------------------------------------- convolution
gdr_status_t check_conv(const gdr_conv_problem_t* p) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    GDR_TRY(check_tokens(p->batch, p->seq_len, p->num_seqs, p->channels));
    // the kernels count channels in an int, past the last one by a workgroup's
    if (p->channels > (1 << 30)) return fail(GDR_ERR_SHAPE, "channels must be at most 2^30 (got %d)", p->channels);
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    if (!io_or_f32(p->param_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "param_dtype must equal io_dtype or be GDR_F32");
    if (!io_or_f32(p->dy_dtype, p->io_dtype) || !io_or_f32(p->grad_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "dy_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    if (p->activation != GDR_ACT_NONE && p->activation != GDR_ACT_SILU)
        return fail(GDR_ERR_UNSUPPORTED, "unknown activation %d", p->activation);
    if (p->width < 2 || p->width > 4) return fail(GDR_ERR_UNSUPPORTED, "width %d not supported (2, 3 or 4)", p->width);
    return check_stride("x_stride", p->x_stride, p->channels);
}

gdr::ConvArgs conv_args(const gdr_conv_problem_t* p, const void* x, const void* weight, const void* bias,
                        const void* S0, const int32_t* cu, void* stream) {
    gdr::ConvArgs a{};
    a.p = *p;
    a.Ttot = p->batch * p->seq_len;
    a.x = x; a.weight = weight; a.bias = bias; a.S0 = S0; a.cu = cu;
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

size_t conv_bwd_bytes(const gdr_conv_problem_t* p) {
    return (size_t)gdr::conv_bwd_tiles(p->batch * p->seq_len, p->channels) * (p->width + 1) * p->channels * 4;
}

// ---------------------------------------------------------------- scan
gdr_status_t check_scan(const gdr_scan_problem_t* p, bool has_z, int64_t most = kMostTileStride) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    GDR_TRY(check_tokens(p->batch, p->seq_len, p->num_seqs, p->channels));
    if (p->groups < 1 || p->channels % p->groups != 0)
        return fail(GDR_ERR_SHAPE, "channels (%d) must be a positive multiple of groups (%d)", p->channels, p->groups);
    if (p->state_dim < 1) return fail(GDR_ERR_SHAPE, "state_dim must be positive (got %d)", p->state_dim);
    if (p->state_dim > 64) return fail(GDR_ERR_UNSUPPORTED, "state_dim %d not supported (1 to 64)", p->state_dim);
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    if (!io_or_f32(p->out_dtype, p->io_dtype) || !io_or_f32(p->dy_dtype, p->io_dtype) ||
        !io_or_f32(p->grad_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "out_dtype, dy_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    if (p->dt_softplus != 0 && p->dt_softplus != 1)
        return fail(GDR_ERR_UNSUPPORTED, "dt_softplus must be 0 or 1 (got %d)", p->dt_softplus);
    const int64_t rows = (int64_t)p->groups * p->state_dim;
    if (p->channels > kMostTileStride)
        return fail(GDR_ERR_SHAPE, "channels must be at most %lld", (long long)kMostTileStride);
    GDR_TRY(check_stride("x_stride", p->x_stride, p->channels, most));
    GDR_TRY(check_stride("dt_stride", p->dt_stride, p->channels, most));
    if (has_z) GDR_TRY(check_stride("z_stride", p->z_stride, p->channels, most));
    GDR_TRY(check_stride("b_stride", p->b_stride, rows, most));
    return check_stride("c_stride", p->c_stride, rows, most);
}

gdr::ScanArgs scan_args(const gdr_scan_problem_t* p, const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* D, const void* z, const float* dt_bias, const float* S0,
                        const int32_t* cu, int64_t max_len, void* ws, void* stream) {
    gdr::ScanArgs a{};
    a.p = *p;
    a.Ttot = p->batch * p->seq_len;
    a.max_len = max_len;
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.z = z; a.dt_bias = dt_bias; a.S0 = S0; a.cu = cu;
    a.ws = static_cast<char*>(ws);
    a.stream = static_cast<hipStream_t>(stream);
    return a;
}

// ---------------------------------------------------------------- layer norm
gdr_status_t check_norm(const gdr_norm_problem_t* p) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    if (p->rows < 0 || p->cols < 1) return fail(GDR_ERR_SHAPE, "rows must be >= 0 and cols positive");
    if (p->cols > 16384) return fail(GDR_ERR_UNSUPPORTED, "cols %d not supported (1 to 16384)", p->cols);
    if (p->rows > ((int64_t)1 << 40)) return fail(GDR_ERR_SHAPE, "too many rows");
    if (!(p->eps >= 0.f)) return fail(GDR_ERR_SHAPE, "eps must be >= 0");
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    if (!io_or_f32(p->param_dtype, p->io_dtype) || !io_or_f32(p->out_dtype, p->io_dtype) ||
        !io_or_f32(p->dy_dtype, p->io_dtype) || !io_or_f32(p->grad_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "param_dtype, out_dtype, dy_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    return check_stride("x_stride", p->x_stride, p->cols);
}
size_t norm_bwd_bytes(const gdr_norm_problem_t* p) { return (size_t)gdr::norm_bwd_blocks(*p) * 2 * p->cols * 4; }

}  // namespace

extern "C" {

gdr_status_t gdr_conv_fwd(const gdr_conv_problem_t* p, const void* x, const void* weight, const void* bias,
                          const void* initial_state, const int32_t* cu_dev, const int32_t* cu_host, void* y,
                          void* final_state, void* stream) {
    GDR_TRY(check_conv(p));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const bool any = p->batch * p->seq_len > 0;
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {weight, p->param_dtype, true, "weight"},
                        {bias, p->param_dtype, false, "bias"}, {initial_state, p->io_dtype, false, "initial_state"},
                        {y, p->io_dtype, true, "y"}, {final_state, p->io_dtype, false, "final_state"}};
    GDR_TRY(check_ptrs(ptrs, any));
    gdr::ConvArgs a = conv_args(p, x, weight, bias, initial_state, cu_dev, stream);
    a.y = y;
    a.ST = final_state;
    return done(gdr::launch_conv_fwd(a));
}

gdr_status_t gdr_conv_step(const gdr_conv_problem_t* p, const void* x, const void* weight, const void* bias,
                           void* state, void* y, void* stream) {
    GDR_TRY(check_conv(p));
    if (p->batch != p->num_seqs || p->seq_len != 1)
        return fail(GDR_ERR_SHAPE, "one token a sequence: batch must equal num_seqs and seq_len 1");
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {weight, p->param_dtype, true, "weight"},
                        {bias, p->param_dtype, false, "bias"}, {state, p->io_dtype, true, "state"},
                        {y, p->io_dtype, true, "y"}};
    GDR_TRY(check_ptrs(ptrs, p->batch > 0));
    gdr::ConvArgs a = conv_args(p, x, weight, bias, nullptr, nullptr, stream);
    a.y = y;
    a.ST = state;
    return done(gdr::launch_conv_step(a));
}

gdr_status_t gdr_conv_bwd_workspace_size(const gdr_conv_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_conv(p));
    *bytes = conv_bwd_bytes(p);
    return GDR_OK;
}

gdr_status_t gdr_conv_bwd(const gdr_conv_problem_t* p, const void* x, const void* weight, const void* bias,
                          const void* initial_state, const int32_t* cu_dev, const int32_t* cu_host, const void* d_y,
                          const void* d_final_state, void* dx, float* dweight, float* dbias, void* d_initial_state,
                          void* workspace, size_t workspace_bytes, void* stream) {
    GDR_TRY(check_conv(p));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const bool any = p->batch * p->seq_len > 0;
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {weight, p->param_dtype, true, "weight"},
                        {bias, p->param_dtype, false, "bias"}, {initial_state, p->io_dtype, false, "initial_state"},
                        {d_y, p->dy_dtype, true, "d_y"}, {d_final_state, p->dy_dtype, false, "d_final_state"},
                        {dx, p->grad_dtype, true, "dx"}, {d_initial_state, p->grad_dtype, false, "d_initial_state"}};
    GDR_TRY(check_ptrs(ptrs, any));
    const Ptr sums[] = {{dweight, GDR_F32, true, "dweight"}, {dbias, GDR_F32, false, "dbias"}};
    GDR_TRY(check_ptrs(sums, true));
    GDR_TRY(check_workspace(workspace, workspace_bytes, conv_bwd_bytes(p)));
    gdr::ConvArgs a = conv_args(p, x, weight, bias, initial_state, cu_dev, stream);
    a.d_y = d_y; a.dST = d_final_state; a.dx = dx; a.dS0 = d_initial_state;
    a.dweight = dweight; a.dbias = dbias;
    a.partial = static_cast<float*>(workspace);
    return done(gdr::launch_conv_bwd(a));
}

gdr_status_t gdr_scan_fwd_workspace_size(const gdr_scan_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_scan(p, false));
    *bytes = gdr::scan_fwd_workspace(*p);
    return GDR_OK;
}

gdr_status_t gdr_scan_fwd(const gdr_scan_problem_t* p, const void* x, const void* dt, const float* A, const void* B,
                          const void* C, const float* D, const void* z, const float* dt_bias,
                          const float* initial_state, const int32_t* cu_dev, const int32_t* cu_host, void* y,
                          float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    GDR_TRY(check_scan(p, z != nullptr));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const int32_t io = p->io_dtype;
    const Ptr ptrs[] = {{x, io, true, "x"}, {dt, io, true, "dt"}, {A, GDR_F32, true, "A"}, {B, io, true, "B"},
                        {C, io, true, "C"}, {D, GDR_F32, false, "D"}, {z, io, false, "z"},
                        {dt_bias, GDR_F32, false, "dt_bias"}, {initial_state, GDR_F32, false, "initial_state"},
                        {y, p->out_dtype, true, "y"}, {final_state, GDR_F32, false, "final_state"}};
    GDR_TRY(check_ptrs(ptrs, p->batch * p->seq_len > 0));
    if (p->num_seqs > 0 && !A) return fail(GDR_ERR_NULL, "A is required");
    GDR_TRY(check_workspace(workspace, workspace_bytes, gdr::scan_fwd_workspace(*p)));
    gdr::ScanArgs a = scan_args(p, x, dt, A, B, C, D, z, dt_bias, initial_state, cu_dev, max_len, workspace, stream);
    a.y = y;
    a.ST = final_state;
    return done(gdr::launch_scan_fwd(a));
}

gdr_status_t gdr_scan_step(const gdr_scan_problem_t* p, const void* x, const void* dt, const float* A, const void* B,
                           const void* C, const float* D, const void* z, const float* dt_bias, float* state, void* y,
                           void* stream) {
    GDR_TRY(check_scan(p, z != nullptr, kMostStride));          // indexed in 64 bits
    if (p->batch != p->num_seqs || p->seq_len != 1)
        return fail(GDR_ERR_SHAPE, "one token a sequence: batch must equal num_seqs and seq_len 1");
    const int32_t io = p->io_dtype;
    const Ptr ptrs[] = {{x, io, true, "x"}, {dt, io, true, "dt"}, {A, GDR_F32, true, "A"}, {B, io, true, "B"},
                        {C, io, true, "C"}, {D, GDR_F32, false, "D"}, {z, io, false, "z"},
                        {dt_bias, GDR_F32, false, "dt_bias"}, {state, GDR_F32, true, "state"},
                        {y, p->out_dtype, true, "y"}};
    GDR_TRY(check_ptrs(ptrs, p->batch > 0));
    gdr::ScanArgs a = scan_args(p, x, dt, A, B, C, D, z, dt_bias, nullptr, nullptr, 1, nullptr, stream);
    a.state = state;
    a.y = y;
    return done(gdr::launch_scan_step(a));
}

gdr_status_t gdr_scan_bwd_workspace_size(const gdr_scan_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_scan(p, false));
    *bytes = gdr::scan_bwd_workspace(*p);
    return GDR_OK;
}

gdr_status_t gdr_scan_bwd(const gdr_scan_problem_t* p, const void* x, const void* dt, const float* A, const void* B,
                          const void* C, const float* D, const void* z, const float* dt_bias,
                          const float* initial_state, const int32_t* cu_dev, const int32_t* cu_host, const void* d_y,
                          const float* d_final_state, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD,
                          void* dz, float* ddt_bias, float* d_initial_state, void* workspace, size_t workspace_bytes,
                          void* stream) {
    GDR_TRY(check_scan(p, z != nullptr));
    int64_t max_len = 0;
    GDR_TRY(check_seqs(p->batch, p->seq_len, p->num_seqs, cu_dev, cu_host, &max_len));
    const int32_t io = p->io_dtype, gr = p->grad_dtype;
    const Ptr ptrs[] = {{x, io, true, "x"}, {dt, io, true, "dt"}, {B, io, true, "B"}, {C, io, true, "C"},
                        {D, GDR_F32, false, "D"}, {z, io, false, "z"}, {dt_bias, GDR_F32, false, "dt_bias"},
                        {initial_state, GDR_F32, false, "initial_state"}, {d_y, p->dy_dtype, true, "d_y"},
                        {d_final_state, GDR_F32, false, "d_final_state"}, {dx, gr, true, "dx"}, {ddt, gr, true, "ddt"},
                        {dB, gr, true, "dB"}, {dC, gr, true, "dC"}, {dz, gr, z != nullptr, "dz"},
                        {d_initial_state, GDR_F32, false, "d_initial_state"}};
    GDR_TRY(check_ptrs(ptrs, p->batch * p->seq_len > 0));
    const Ptr sums[] = {{A, GDR_F32, true, "A"}, {dA, GDR_F32, true, "dA"}, {dD, GDR_F32, false, "dD"},
                        {ddt_bias, GDR_F32, false, "ddt_bias"}};
    GDR_TRY(check_ptrs(sums, true));
    GDR_TRY(check_workspace(workspace, workspace_bytes, gdr::scan_bwd_workspace(*p)));
    gdr::ScanArgs a = scan_args(p, x, dt, A, B, C, D, z, dt_bias, initial_state, cu_dev, max_len, workspace, stream);
    a.d_y = d_y; a.dST = d_final_state;
    a.dx = dx; a.ddt = ddt; a.dB = dB; a.dC = dC; a.dz = dz;
    a.dA = dA; a.dD = dD; a.ddt_bias = ddt_bias; a.dS0 = d_initial_state;
    return done(gdr::launch_scan_bwd(a));
}

gdr_status_t gdr_layer_norm_fwd(const gdr_norm_problem_t* p, const void* x, const void* weight, const void* bias,
                                void* y, float* mean, float* rstd, void* stream) {
    GDR_TRY(check_norm(p));
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {weight, p->param_dtype, false, "weight"},
                        {bias, p->param_dtype, false, "bias"}, {y, p->out_dtype, true, "y"},
                        {mean, GDR_F32, false, "mean"}, {rstd, GDR_F32, false, "rstd"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    gdr::NormArgs a{};
    a.p = *p;
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_norm_fwd(a));
}

gdr_status_t gdr_layer_norm_bwd_workspace_size(const gdr_norm_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_norm(p));
    *bytes = norm_bwd_bytes(p);
    return GDR_OK;
}

gdr_status_t gdr_layer_norm_bwd(const gdr_norm_problem_t* p, const void* x, const void* d_y, const void* weight,
                                const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                                void* workspace, size_t workspace_bytes, void* stream) {
    GDR_TRY(check_norm(p));
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {d_y, p->dy_dtype, true, "d_y"},
                        {weight, p->param_dtype, false, "weight"}, {mean, GDR_F32, true, "mean"},
                        {rstd, GDR_F32, true, "rstd"}, {dx, p->grad_dtype, true, "dx"},
                        {dweight, GDR_F32, false, "dweight"}, {dbias, GDR_F32, false, "dbias"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    GDR_TRY(check_workspace(workspace, workspace_bytes, norm_bwd_bytes(p)));
    gdr::NormArgs a{};
    a.p = *p;
    a.x = x; a.d_y = d_y; a.weight = weight; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.partial = static_cast<float*>(workspace);
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_norm_bwd(a));
}

}  // extern "C"
