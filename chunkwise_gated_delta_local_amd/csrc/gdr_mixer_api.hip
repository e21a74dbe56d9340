// Host side of the layer operators declared in include/gdr_mixer.h: argument
// checks and launch arguments.
#include <cmath>

#include "gdr_checks.hpp"

namespace {

using namespace gdr;

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

// ---------------------------------------------------------------- norms
// what the three kinds of norms share
gdr_status_t check_rows(int64_t rows, int32_t cols, float eps) {
    if (rows < 0 || cols < 1) return fail(GDR_ERR_SHAPE, "rows must be >= 0 and cols positive");
    if (cols > 16384) return fail(GDR_ERR_UNSUPPORTED, "cols %d not supported (1 to 16384)", cols);
    if (rows > ((int64_t)1 << 40)) return fail(GDR_ERR_SHAPE, "too many rows");
    if (!(eps >= 0.f)) return fail(GDR_ERR_SHAPE, "eps must be >= 0");
    return GDR_OK;
}
gdr_status_t check_norm(const gdr_norm_problem_t* p) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    GDR_TRY(check_rows(p->rows, p->cols, p->eps));
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    if (!io_or_f32(p->param_dtype, p->io_dtype) || !io_or_f32(p->out_dtype, p->io_dtype) ||
        !io_or_f32(p->dy_dtype, p->io_dtype) || !io_or_f32(p->grad_dtype, p->io_dtype))
        return fail(GDR_ERR_DTYPE, "param_dtype, out_dtype, dy_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    return check_stride("x_stride", p->x_stride, p->cols);
}
gdr_status_t check_gated(const gdr_gated_norm_problem_t* p) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    GDR_TRY(check_rows(p->rows, p->cols, p->eps));
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    for (int32_t t : {p->param_dtype, p->out_dtype, p->dy_dtype, p->grad_dtype})
        if (!io_or_f32(t, p->io_dtype))
            return fail(GDR_ERR_DTYPE, "param_dtype, out_dtype, dy_dtype and grad_dtype must equal io_dtype or be GDR_F32");
    if (p->activation != GDR_ACT_SILU && p->activation != GDR_ACT_SIGMOID)
        return fail(GDR_ERR_UNSUPPORTED, "activation %d not supported (GDR_ACT_SILU or GDR_ACT_SIGMOID)", p->activation);
    GDR_TRY(check_stride("x_stride", p->x_stride, p->cols));
    return check_stride("z_stride", p->z_stride, p->cols);
}
gdr_status_t check_residual(const gdr_residual_norm_problem_t* p) {
    if (!p) return fail(GDR_ERR_NULL, "problem is NULL");
    GDR_TRY(check_rows(p->rows, p->cols, p->eps));
    if (!std::isfinite(p->scale)) return fail(GDR_ERR_SHAPE, "scale must be finite");
    if (!is_dtype(p->io_dtype)) return fail(GDR_ERR_DTYPE, "unknown io_dtype %d", p->io_dtype);
    for (int32_t t : {p->param_dtype, p->stream_dtype, p->out_dtype, p->dy_dtype, p->dh_dtype, p->grad_dtype, p->dres_dtype})
        if (!io_or_f32(t, p->io_dtype))
            return fail(GDR_ERR_DTYPE, "param, stream, out, dy, dh, grad and dres dtype must equal io_dtype or be GDR_F32");
    if (p->gate < GDR_GATE_NONE || p->gate > GDR_GATE_TOKEN) return fail(GDR_ERR_UNSUPPORTED, "unknown gate %d", p->gate);
    GDR_TRY(check_stride("x_stride", p->x_stride, p->cols));
    if (p->gate == GDR_GATE_TOKEN) GDR_TRY(check_stride("gate_stride", p->gate_stride, p->cols));
    return check_stride("residual_stride", p->residual_stride, p->cols);
}
gdr_status_t check_gate(const gdr_residual_norm_problem_t* p, const void* gate) {
    if ((gate == nullptr) != (p->gate == GDR_GATE_NONE) && (gate || p->rows > 0))
        return fail(GDR_ERR_NULL, "the gate must be NULL for GDR_GATE_NONE and given otherwise");
    return GDR_OK;
}
size_t gated_bwd_bytes(const gdr_gated_norm_problem_t* p) { return (size_t)gdr::gated_norm_bwd_blocks(*p) * p->cols * 4; }
size_t residual_bwd_bytes(const gdr_residual_norm_problem_t* p) {
    return (size_t)gdr::residual_norm_bwd_blocks(*p) * 3 * p->cols * 4;
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

gdr_status_t gdr_gated_norm_fwd(const gdr_gated_norm_problem_t* p, const void* x, const void* z, const void* weight,
                                void* y, float* rstd, void* stream) {
    GDR_TRY(check_gated(p));
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {z, p->io_dtype, true, "z"}, {weight, p->param_dtype, false, "weight"},
                        {y, p->out_dtype, true, "y"}, {rstd, GDR_F32, false, "rstd"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    gdr::GatedNormArgs a{};
    a.p = *p;
    a.x = x; a.z = z; a.weight = weight; a.y = y; a.rstd = rstd;
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_gated_norm_fwd(a));
}

gdr_status_t gdr_gated_norm_bwd_workspace_size(const gdr_gated_norm_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_gated(p));
    *bytes = gated_bwd_bytes(p);
    return GDR_OK;
}

gdr_status_t gdr_gated_norm_bwd(const gdr_gated_norm_problem_t* p, const void* x, const void* z, const void* d_y,
                                const void* weight, const float* rstd, void* dx, void* dz, float* dweight,
                                void* workspace, size_t workspace_bytes, void* stream) {
    GDR_TRY(check_gated(p));
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {z, p->io_dtype, true, "z"}, {d_y, p->dy_dtype, true, "d_y"},
                        {weight, p->param_dtype, false, "weight"}, {rstd, GDR_F32, true, "rstd"},
                        {dx, p->grad_dtype, true, "dx"}, {dz, p->grad_dtype, true, "dz"},
                        {dweight, GDR_F32, false, "dweight"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    GDR_TRY(check_workspace(workspace, workspace_bytes, gated_bwd_bytes(p)));
    gdr::GatedNormArgs a{};
    a.p = *p;
    a.x = x; a.z = z; a.d_y = d_y; a.weight = weight; a.rstd = const_cast<float*>(rstd);
    a.dx = dx; a.dz = dz; a.dweight = dweight;
    a.partial = static_cast<float*>(workspace);
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_gated_norm_bwd(a));
}

gdr_status_t gdr_residual_norm_fwd(const gdr_residual_norm_problem_t* p, const void* x, const void* residual,
                                   const void* weight, const void* x_weight, const void* gate, void* y, void* h,
                                   float* rstd, float* x_rstd, void* stream) {
    GDR_TRY(check_residual(p));
    const int32_t gate_dtype = p->gate == GDR_GATE_TOKEN ? p->io_dtype : p->param_dtype;
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {residual, p->stream_dtype, true, "residual"},
                        {weight, p->param_dtype, false, "weight"}, {x_weight, p->param_dtype, false, "x_weight"},
                        {gate, gate_dtype, false, "gate"}, {y, p->out_dtype, true, "y"}, {h, p->stream_dtype, true, "h"},
                        {rstd, GDR_F32, false, "rstd"}, {x_rstd, GDR_F32, false, "x_rstd"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    GDR_TRY(check_gate(p, gate));
    gdr::ResidualNormArgs a{};
    a.p = *p;
    a.x = x; a.residual = residual; a.weight = weight; a.x_weight = x_weight; a.gate = gate;
    a.y = y; a.h = h; a.rstd = rstd; a.x_rstd = x_rstd;
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_residual_norm_fwd(a));
}

gdr_status_t gdr_residual_norm_bwd_workspace_size(const gdr_residual_norm_problem_t* p, size_t* bytes) {
    if (!bytes) return fail(GDR_ERR_NULL, "bytes is NULL");
    GDR_TRY(check_residual(p));
    *bytes = residual_bwd_bytes(p);
    return GDR_OK;
}

gdr_status_t gdr_residual_norm_bwd(const gdr_residual_norm_problem_t* p, const void* x, const void* h, const void* d_y,
                                   const void* d_h, const void* weight, const void* x_weight, const void* gate,
                                   const float* rstd, const float* x_rstd, void* dx, void* dresidual, float* dweight,
                                   float* dx_weight, void* dgate, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    GDR_TRY(check_residual(p));
    const bool token = p->gate == GDR_GATE_TOKEN;
    const int32_t gate_dtype = token ? p->io_dtype : p->param_dtype;
    const Ptr ptrs[] = {{x, p->io_dtype, true, "x"}, {h, p->stream_dtype, true, "h"}, {d_y, p->dy_dtype, true, "d_y"},
                        {d_h, p->dh_dtype, false, "d_h"}, {weight, p->param_dtype, false, "weight"},
                        {x_weight, p->param_dtype, false, "x_weight"}, {gate, gate_dtype, false, "gate"},
                        {rstd, GDR_F32, true, "rstd"}, {x_rstd, GDR_F32, x_weight != nullptr, "x_rstd"},
                        {dx, p->grad_dtype, true, "dx"}, {dresidual, p->dres_dtype, true, "dresidual"},
                        {dweight, GDR_F32, false, "dweight"}, {dx_weight, GDR_F32, false, "dx_weight"},
                        {dgate, token ? p->grad_dtype : GDR_F32, false, "dgate"}};
    GDR_TRY(check_ptrs(ptrs, p->rows > 0));
    GDR_TRY(check_gate(p, gate));
    GDR_TRY(check_workspace(workspace, workspace_bytes, residual_bwd_bytes(p)));
    gdr::ResidualNormArgs a{};
    a.p = *p;
    a.x = x; a.h_in = h; a.d_y = d_y; a.d_h = d_h; a.weight = weight; a.x_weight = x_weight; a.gate = gate;
    a.rstd = const_cast<float*>(rstd); a.x_rstd = const_cast<float*>(x_rstd);
    a.dx = dx; a.dresidual = dresidual; a.dweight = dweight; a.dx_weight = dx_weight; a.dgate = dgate;
    a.partial = static_cast<float*>(workspace);
    a.stream = static_cast<hipStream_t>(stream);
    return done(gdr::launch_residual_norm_bwd(a));
}

}  // extern "C"
