// Internal interface of the layer operators (include/gdr_mixer.h): launch
// arguments, and device helpers that their kernels share.
#pragma once

#include "gdr_device.hpp"
#include "gdr_mixer.h"

namespace gdr {

// Sets the calling thread's error message (gdr_last_error_message) and returns st.
gdr_status_t fail(gdr_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();

struct ConvArgs {
    gdr_conv_problem_t p;
    int64_t Ttot;
    const void *x, *weight, *bias, *S0;
    const int32_t* cu;
    void *y, *ST;
    // backward
    const void *d_y, *dST;
    void *dx, *dS0;
    float *dweight, *dbias;
    float* partial;            // [tiles][W + 1][D]
    hipStream_t stream;
};
int64_t conv_bwd_tiles(int64_t Ttot, int32_t channels);
hipError_t launch_conv_fwd(const ConvArgs& a);
hipError_t launch_conv_step(const ConvArgs& a);
hipError_t launch_conv_bwd(const ConvArgs& a);

struct NormArgs {
    gdr_norm_problem_t p;
    const void *x, *weight, *bias, *d_y;
    void *y, *dx;
    float *mean, *rstd;
    float *dweight, *dbias;
    float* partial;            // [blocks][2][cols]
    hipStream_t stream;
};
int norm_bwd_blocks(const gdr_norm_problem_t& p);
hipError_t launch_norm_fwd(const NormArgs& a);
hipError_t launch_norm_bwd(const NormArgs& a);

struct GatedNormArgs {
    gdr_gated_norm_problem_t p;
    const void *x, *z, *weight, *d_y;
    void *y, *dx, *dz;
    float *rstd, *dweight;
    float* partial;            // [blocks][cols]
    hipStream_t stream;
};
int gated_norm_bwd_blocks(const gdr_gated_norm_problem_t& p);
hipError_t launch_gated_norm_fwd(const GatedNormArgs& a);
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a);

struct ResidualNormArgs {
    gdr_residual_norm_problem_t p;
    const void *x, *residual, *weight, *x_weight, *gate, *h_in, *d_y, *d_h;
    void *y, *h, *dx, *dresidual, *dgate;
    float *rstd, *x_rstd, *dweight, *dx_weight;
    float* partial;            // [blocks][3][cols]: dweight, dx_weight, dgate of a gate per channel
    hipStream_t stream;
};
int residual_norm_bwd_blocks(const gdr_residual_norm_problem_t& p);
hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a);
hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a);

struct ScanArgs {
    gdr_scan_problem_t p;
    int64_t Ttot, max_len;     // total tokens, longest sequence (host)
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias, *S0;
    const int32_t* cu;
    void* y;
    float* ST;
    float* state;              // single token: in and out
    // backward
    const void* d_y;
    const float* dST;
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *ddt_bias, *dS0;
    char* ws;
    hipStream_t stream;
};
// Elements between tokens that the scan's tile kernels take, and channels: a tile of
// 128 tokens lies within the 2^31 bytes of a buffer's offsets.
constexpr int64_t kMostTileStride = ((int64_t)1 << 22) - 1;
size_t scan_fwd_workspace(const gdr_scan_problem_t& p);
size_t scan_bwd_workspace(const gdr_scan_problem_t& p);
hipError_t launch_scan_fwd(const ScanArgs& a);
hipError_t launch_scan_step(const ScanArgs& a);
hipError_t launch_scan_bwd(const ScanArgs& a);

// ---------------------------------------------------------------- device helpers
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// 1 / (1 + exp(-x)); v_exp_f32 and v_rcp_f32 are good to one unit in the last place
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-x)); }
// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|) <= 1. With u = fl(1 + e),
// log1p(e) = log(u) + (e - (u - 1)) up to (e - (u - 1))(1 - 1/u): the rounding of
// u is put back, so that a small e keeps its relative precision.
__device__ __forceinline__ float softplus(float x) {
    const float e = exp_fast(-fabsf(x));
    const float u = 1.f + e;
    const float c = e - (u - 1.f);
    return fmaxf(x, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(u), kLn2, c);
}
// softplus and its derivative 1 / (1 + exp(-x)) = (1 or e) / u
__device__ __forceinline__ float softplus(float x, float* slope) {
    const float e = exp_fast(-fabsf(x));
    const float u = 1.f + e;
    const float c = e - (u - 1.f);
    *slope = (x < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(u);
    return fmaxf(x, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(u), kLn2, c);
}
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// d/dx [x sigmoid(x)], from s = sigmoid(x)
__device__ __forceinline__ float silu_slope(float x, float s) { return s * __builtin_fmaf(x, 1.f - s, 1.f); }
__device__ __forceinline__ float silu_grad(float x) { return silu_slope(x, sigmoid(x)); }

// element idx of a tensor that is fp32 (f32) or of type T
template <typename T>
__device__ __forceinline__ float load_as(const void* p, int64_t idx, int f32) {
    return f32 ? reinterpret_cast<const float*>(p)[idx] : to_f(reinterpret_cast<const T*>(p)[idx]);
}
template <typename T>
__device__ __forceinline__ void store_as(void* p, int64_t idx, float v, int f32) {
    if (f32) reinterpret_cast<float*>(p)[idx] = v;
    else reinterpret_cast<T*>(p)[idx] = to_t<T>(v);
}

// V consecutive elements, moved in one access; global memory takes 4, 8 and 16
// bytes at the alignment of an element
template <typename T, int V> struct Raw {
    typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
template <typename T> struct Raw<T, 1> {
    typedef T type;
};
// ONCE: past the caches, for data that they could not hold until its next use
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ typename Raw<T, V>::type load_raw(const T* p) {
    auto* q = reinterpret_cast<const typename Raw<T, V>::type*>(p);
    if constexpr (ONCE) return __builtin_nontemporal_load(q);
    else return *q;
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_raw(T* p, typename Raw<T, V>::type r) {
    auto* q = reinterpret_cast<typename Raw<T, V>::type*>(p);
    if constexpr (ONCE) __builtin_nontemporal_store(r, q);
    else *q = r;
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Raw<T, V>::type& r, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = to_f(r);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f(r[i]);
    }
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    typename Raw<T, V>::type r;
    if constexpr (V == 1) {
        r = to_t<T>(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = to_t<T>(f[i]);
    }
    store_raw<T, V, ONCE>(p, r);
}
// V consecutive elements of a tensor that is fp32 or T; fp32 elements move 4 at a time
template <typename T, int V>
__device__ __forceinline__ void load_vec_as(const void* p, int64_t idx, int f32, float (&f)[V]) {
    if (f32) {
        const float* q = reinterpret_cast<const float*>(p) + idx;
        if constexpr (V == 1) {
            f[0] = q[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const auto v = load_raw<float, 4>(q + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i + j] = v[j];
            }
        }
    } else {
        unpack<T, V>(load_raw<T, V>(reinterpret_cast<const T*>(p) + idx), f);
    }
}

// Token range of sequence n, clamped to the token axis whatever cu holds.
__device__ __forceinline__ void seq_range(const int32_t* cu, int n, int64_t T_row, int64_t Ttot, int64_t* s,
                                          int64_t* e) {
    int64_t b = cu ? (int64_t)cu[n] : (int64_t)n * T_row;
    int64_t f = cu ? (int64_t)cu[n + 1] : (int64_t)(n + 1) * T_row;
    b = b < 0 ? 0 : (b > Ttot ? Ttot : b);
    f = f < b ? b : (f > Ttot ? Ttot : f);
    *s = b;
    *e = f;
}
// Sequence that holds token t: the last n in [0, N) with start <= t (packed
// sequences; empty ones before it end at its start and are passed over). All 64
// lanes of the wavefront call it with the same t: each looks at a 64th of what is
// left, so that thousands of sequences take two loads in a row.
__device__ __forceinline__ int seq_of_token(const int32_t* cu, int N, int64_t T_row, int64_t t) {
    if (!cu) {
        const int64_t n = (uint32_t)t / (uint32_t)T_row;     // token indices fit 31 bits
        return (int)(n < N ? n : N - 1);
    }
    int lo = 0, len = N;                       // the answer is in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 63) / 64, i = lo + (int)(threadIdx.x & 63) * step;
        const bool before = i < lo + len && (int64_t)cu[i] <= t;
        const int k = __popcll(__ballot(before));            // starts are sorted: the first k lanes
        const int at = k > 0 ? (k - 1) * step : 0;
        len = len - at < step ? len - at : step;
        lo += at;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Whether a call moves more bytes than the last cache holds (256 MB): its rows then
// go past the caches. Below, the next operator finds them there; above, hardly any
// (us from the caches and past them, 4,096 bf16 columns):
//   a convolution and the norm of its output    192 MB each 76, 82; 272: 125, 123; 320: 147, 135; 512: 215, 208
//   backward, the norm and then the convolution 192 MB each 92, 97; 288: 128, 138; 408: 195, 189; 768: 308, 288
// Rows that nothing left in the caches are 3 to 6 % faster past them from 150 MB on.
inline bool beyond_caches(int64_t bytes) { return bytes > ((int64_t)256 << 20); }
inline int64_t size_of(int32_t dtype) { return dtype == GDR_BF16 ? 2 : 4; }

// Workgroups of a one-dimensional launch: HIP counts its threads in 32 bits.
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads < ((int64_t)1 << 32); }

// out(i) = sum over p < P of part[p * stride + i], i < n, in a fixed order: the
// NW wavefronts of a workgroup take every NW-th p for the same 64 i.
template <int NW, typename Out>
__global__ __launch_bounds__(64 * NW) void k_sum_partials(const float* __restrict__ part, int64_t P, int64_t stride,
                                                          int64_t n, Out out) {
    __shared__ float red[NW][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int64_t i0 = (int64_t)blockIdx.x * 64; i0 < n; i0 += (int64_t)gridDim.x * 64) {
        const int64_t i = i0 + lane;
        float s = 0.f;
        if (i < n) {
#pragma unroll 8
            for (int64_t p = w; p < P; p += NW) s += part[p * stride + i];
        }
        red[w][lane] = s;
        __syncthreads();
        if (w == 0 && i < n) {
            float v = red[0][lane];
#pragma unroll
            for (int k = 1; k < NW; ++k) v += red[k][lane];
            out(i, v);
        }
        __syncthreads();
    }
}

// 16 wavefronts share the partials where there are many of them for few sums
// (512 for 5,122, in a layer norm's backward pass of 4,001 rows: 33.2 us in all; with 4: 36.6), else 4.
template <typename Out>
hipError_t sum_partials(const float* part, int64_t P, int64_t n, Out out, hipStream_t stream) {
    if (n == 0) return hipSuccess;
    const int64_t blocks = (n + 63) / 64, most = 1 << 20;
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    if (P >= 64 && blocks < 1024) k_sum_partials<16><<<grid, 1024, 0, stream>>>(part, P, n, n, out);
    else k_sum_partials<4><<<grid, 256, 0, stream>>>(part, P, n, n, out);
    return hipGetLastError();
}

}  // namespace gdr
