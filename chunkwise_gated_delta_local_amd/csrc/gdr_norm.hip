// Layer norm over rows, forward and backward (include/gdr_mixer.h). A few
// operations an element: HBM bounds both, so a row is read once and stays in
// registers between the statistics and the output. TPR threads share a row,
// each holding NV groups of V consecutive elements; rows go round a grid that
// fills the card once, and the weights stay in registers meanwhile.
#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

namespace {

constexpr int kThreads = 256;

// Sum over the TPR threads of a row: butterfly inside a wavefront, LDS across.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[w] = v;
        __syncthreads();
        v = (red[0] + red[1]) + (red[2] + red[3]);
        __syncthreads();
    }
    return v;
}

template <typename T, int V, int NV, int TPR>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(NormArgs a) {
    __shared__ float red[4];
    const int C = a.p.cols, rpb = kThreads / TPR, l = threadIdx.x % TPR;
    const int w32 = a.p.param_dtype == GDR_F32, o32 = a.p.out_dtype == GDR_F32;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + l) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w[i][v] = a.weight && c < C ? load_as<T>(a.weight, c + v, w32) : 1.f;
            b[i][v] = a.bias && c < C ? load_as<T>(a.bias, c + v, w32) : 0.f;
        }
    }
    const float inv = 1.f / (float)C;
    // every thread of a workgroup makes the same trips (row_sum meets in barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.p.rows; r0 += (int64_t)gridDim.x * rpb) {
        const int64_t r = r0 + threadIdx.x / TPR;
        const bool live = r < a.p.rows;
        float x[NV][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (live && c < C) unpack<T, V>(load_raw<T, V>((const T*)a.x + r * a.p.x_stride + c), x[i]);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) x[i][v] = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += x[i][v];
        }
        const float mean = row_sum<TPR>(sum, red) * inv;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = (i * TPR + l) * V < C;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[i][v] = in ? x[i][v] - mean : 0.f;
                sq = __builtin_fmaf(x[i][v], x[i][v], sq);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(sq, red) * inv + a.p.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = __builtin_fmaf(x[i][v] * rstd, w[i][v], b[i][v]);
            store_vec_as<T, V>(a.y, r * C + c, y, o32);
        }
        if (l == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// Backward: with xhat = (x - mean) rstd and c = d_y weight,
//   dx = rstd (c - mean(c) - xhat mean(c xhat)).
// Each thread also sums d_y xhat and d_y of its columns over its rows; the rows
// of a workgroup are joined in LDS, the workgroups by k_sum_partials.
template <typename T, int V, int NV, int TPR>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(NormArgs a) {
    constexpr int RPB = kThreads / TPR;
    __shared__ float red[4];
    __shared__ float cols[RPB > 1 ? RPB : 1][RPB > 1 ? NV * TPR * V : 1];
    const int C = a.p.cols, l = threadIdx.x % TPR, rr = threadIdx.x / TPR;
    const int w32 = a.p.param_dtype == GDR_F32, dy32 = a.p.dy_dtype == GDR_F32, g32 = a.p.grad_dtype == GDR_F32;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + l) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w[i][v] = a.weight && c < C ? load_as<T>(a.weight, c + v, w32) : 1.f;
            dw[i][v] = db[i][v] = 0.f;
        }
    }
    const float inv = 1.f / (float)C;
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + rr;
        const bool live = r < a.p.rows;
        const float mean = live ? a.mean[r] : 0.f, rstd = live ? a.rstd[r] : 0.f;
        float h[NV][V], g[NV][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (live && c < C) {
                unpack<T, V>(load_raw<T, V>((const T*)a.x + r * a.p.x_stride + c), h[i]);
                load_vec_as<T, V>(a.d_y, r * C + c, dy32, g[i]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[i][v] = mean;
                    g[i][v] = 0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[i][v] = (h[i][v] - mean) * rstd;
                dw[i][v] = __builtin_fmaf(g[i][v], h[i][v], dw[i][v]);
                db[i][v] += g[i][v];
                g[i][v] *= w[i][v];
                s1 += g[i][v];
                s2 = __builtin_fmaf(g[i][v], h[i][v], s2);
            }
        s1 = row_sum<TPR>(s1, red) * inv;
        s2 = row_sum<TPR>(s2, red) * inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float d[V];
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = rstd * (g[i][v] - s1 - h[i][v] * s2);
            store_vec_as<T, V>(a.dx, r * C + c, d, g32);
        }
    }
    float* part = a.partial + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (RPB > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) cols[rr][(i * TPR + l) * V + v] = k ? db[i][v] : dw[i][v];
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += kThreads) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < RPB; ++j) s += cols[j][c];
                part[(int64_t)k * C + c] = s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + l) * V;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (c + v < C) part[(int64_t)k * C + c + v] = k ? db[i][v] : dw[i][v];
            }
        }
    }
}

struct NormGradOut {
    float *dweight, *dbias;
    int C;
    __device__ void operator()(int64_t i, float v) const {
        if (i < C) {
            if (dweight) dweight[i] = v;
        } else if (dbias) {
            dbias[i - C] = v;
        }
    }
};

// The variant for a row of C elements: the fewest threads a row (16, 64 or 256)
// whose registers hold it.
struct Shape {
    int V, NV, TPR;
};
Shape shape_of(bool bf, bool wide, int C) {
    const int V = wide ? (bf ? 8 : 4) : 1;
    const int units = (C + V - 1) / V;
    if (wide && units <= 16) return {V, 1, 16};
    if (wide && !bf && units <= 32) return {V, 2, 16};
    const int most64 = wide ? (bf ? 2 : 4) : 8;            // groups a thread holds with a wavefront a row
    for (int nv = 1; nv <= most64; nv *= 2)
        if (units <= 64 * nv) return {V, nv, 64};
    for (int nv = 1; nv <= 64; nv *= 2)
        if (units <= 256 * nv) return {V, nv, 256};
    return {V, 0, 0};
}

template <typename F>
hipError_t by_shape(const NormArgs& a, F f) {
    const Shape s = shape_of(a.p.io_dtype == GDR_BF16, a.wide, a.p.cols);
#define GDR_NORM(T, V_, NV_, TPR_)                                                                                    \
    if (s.V == V_ && s.NV == NV_ && s.TPR == TPR_) {                                                                  \
        f(T{}, std::integral_constant<int, V_>{}, std::integral_constant<int, NV_>{}, std::integral_constant<int, TPR_>{}); \
        return hipGetLastError();                                                                                     \
    }
#define GDR_NORM_SCALAR(T)                                                                                            \
    GDR_NORM(T, 1, 1, 64) GDR_NORM(T, 1, 2, 64) GDR_NORM(T, 1, 4, 64) GDR_NORM(T, 1, 8, 64)                           \
    GDR_NORM(T, 1, 4, 256) GDR_NORM(T, 1, 8, 256) GDR_NORM(T, 1, 16, 256) GDR_NORM(T, 1, 32, 256) GDR_NORM(T, 1, 64, 256)
    if (a.p.io_dtype == GDR_BF16) {
        GDR_NORM(bf16, 8, 1, 16) GDR_NORM(bf16, 8, 1, 64) GDR_NORM(bf16, 8, 2, 64)
        GDR_NORM(bf16, 8, 1, 256) GDR_NORM(bf16, 8, 2, 256) GDR_NORM(bf16, 8, 4, 256) GDR_NORM(bf16, 8, 8, 256)
        GDR_NORM_SCALAR(bf16)
    } else {
        GDR_NORM(float, 4, 1, 16) GDR_NORM(float, 4, 2, 16) GDR_NORM(float, 4, 1, 64) GDR_NORM(float, 4, 2, 64)
        GDR_NORM(float, 4, 4, 64) GDR_NORM(float, 4, 2, 256) GDR_NORM(float, 4, 4, 256) GDR_NORM(float, 4, 8, 256)
        GDR_NORM(float, 4, 16, 256) GDR_NORM_SCALAR(float)
    }
#undef GDR_NORM
#undef GDR_NORM_SCALAR
    return hipErrorInvalidValue;
}

int64_t row_blocks(const NormArgs& a, int TPR) { return (a.p.rows + kThreads / TPR - 1) / (kThreads / TPR); }

}  // namespace

// Workgroups of the backward pass: two for each of the 256 compute units (their
// partial sums are written and read once more), fewer when there are fewer rows.
int norm_bwd_blocks(const gdr_norm_problem_t& p) {
    const int64_t n = (p.rows + 15) / 16;                  // every shape holds at most 16 rows a workgroup
    return (int)(n < 512 ? n : 512);
}

hipError_t launch_norm_fwd(const NormArgs& a) {
    if (a.p.rows == 0) return hipSuccess;
    return by_shape(a, [&](auto type, auto vec, auto nv, auto tpr) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value;
        const int64_t n = row_blocks(a, TPR), most = 2048;
        k_norm_fwd<T, V, NV, TPR><<<dim3((unsigned)(n < most ? n : most)), kThreads, 0, a.stream>>>(a);
    });
}

hipError_t launch_norm_bwd(const NormArgs& a) {
    const int blocks = norm_bwd_blocks(a.p);
    if (blocks > 0) {
        hipError_t e = by_shape(a, [&](auto type, auto vec, auto nv, auto tpr) {
            typedef decltype(type) T;
            constexpr int V = decltype(vec)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value;
            k_norm_bwd<T, V, NV, TPR><<<dim3((unsigned)blocks), kThreads, 0, a.stream>>>(a);
        });
        if (e != hipSuccess) return e;
    }
    if (!a.dweight && !a.dbias) return hipSuccess;
    return sum_partials(a.partial, blocks, 2 * (int64_t)a.p.cols, NormGradOut{a.dweight, a.dbias, a.p.cols}, a.stream);
}

}  // namespace gdr
