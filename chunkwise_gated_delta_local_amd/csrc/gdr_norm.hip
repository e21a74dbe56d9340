// Layer norm over rows, forward and backward (include/gdr_mixer.h). A few
// operations an element: HBM bounds both, so a row is read once and stays in
// registers between the statistics and the output (but for the backward pass of
// more than 12,288 columns, whose sums overflow into scratch: 208 to 584 bytes a
// lane in bf16, 928 in fp32; 4,096 rows of 16,384 take 176 and 414 us, of 12,288
// 104 and 127). TPR threads share a row,
// each holding NV pieces of V = 16 bytes; rows go round the grid, the weights
// stay in registers meanwhile, and the next row is on its way while one is
// worked on.
//
// Rows of any length and alignment move in 16-byte accesses (global memory
// takes them at the alignment of an element); only the piece that the row's end
// cuts is moved by elements.
#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

namespace {

constexpr int kThreads = 256;

// elements c .. c + V - 1 of a row of C, zero past its end
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ typename Raw<T, V>::type load_piece(const T* row, int c, int C) {
    typename Raw<T, V>::type r;
    if (c + V <= C) return load_raw<T, V, ONCE>(row + c);
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = c + v < C ? row[c + v] : to_t<T>(0.f);
    return r;
}
// a parameter's elements, which are T or fp32; `none` where there is no parameter
template <typename T, int V>
__device__ __forceinline__ void load_param(const void* p, int c, int C, int f32, float none, float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = none;
    if (!p || c >= C) return;
    if (f32) unpack<float, V>(load_piece<float, V>((const float*)p, c, C), f);
    else unpack<T, V>(load_piece<T, V>((const T*)p, c, C), f);
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_piece(T* row, int c, int C, const float (&f)[V]) {
    typename Raw<T, V>::type r;
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = to_t<T>(f[v]);
    if (c + V <= C) {
        store_raw<T, V, ONCE>(row + c, r);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < C) row[c + v] = r[v];
    }
}

// Sum over the TPR threads of a row: butterfly inside a wavefront, LDS across;
// the caller alternates between two LDS slots, so that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[4], int& slot) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        v = (red[slot][0] + red[slot][1]) + (red[slot][2] + red[slot][3]);
        slot ^= 1;
    }
    return v;
}

// ONCE: x and y go past the caches
template <typename T, typename OT, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(NormArgs a) {
    __shared__ float red[2][4];
    int slot = 0;
    const int C = a.p.cols, rpb = kThreads / TPR, l = threadIdx.x % TPR;
    const int w32 = a.p.param_dtype == GDR_F32;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + l) * V;
        load_param<T, V>(a.weight, c, C, w32, 1.f, w[i]);
        load_param<T, V>(a.bias, c, C, w32, 0.f, b[i]);
    }
    const float inv = 1.f / (float)C;
    typename Raw<T, V>::type raw[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (r < a.p.rows && (i * TPR + l) * V < C)
                raw[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, (i * TPR + l) * V, C);
    };
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t r = (int64_t)blockIdx.x * rpb + threadIdx.x / TPR;
    fetch(r);
    // every thread of a workgroup makes the same trips (row_sum meets in barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        float x[NV][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = live && (i * TPR + l) * V < C;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[i][v] = in ? to_f(raw[i][v]) : 0.f;
                sum += x[i][v];
            }
        }
        fetch(r + step);
        const float mean = row_sum<TPR>(sum, red, slot) * inv;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[i][v] = (i * TPR + l) * V + v < C ? x[i][v] - mean : 0.f;
                sq = __builtin_fmaf(x[i][v], x[i][v], sq);
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(sq, red, slot) * inv + a.p.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = __builtin_fmaf(x[i][v] * rstd, w[i][v], b[i][v]);
            store_piece<OT, V, ONCE>((OT*)a.y + r * C, c, C, y);
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
// of a workgroup are joined in LDS, the workgroups by k_sum_partials. ONCE: x,
// d_y and dx go past the caches.
template <typename T, typename DT, typename GT, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(NormArgs a) {
    constexpr int RPB = kThreads / TPR;
    __shared__ float red[2][2][4];
    __shared__ float cols[RPB > 1 ? RPB : 1][RPB > 1 ? NV * TPR * V : 1];
    int slot = 0;
    const int C = a.p.cols, l = threadIdx.x % TPR, rr = threadIdx.x / TPR;
    const int w32 = a.p.param_dtype == GDR_F32;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + l) * V;
        load_param<T, V>(a.weight, c, C, w32, 1.f, w[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = db[i][v] = 0.f;
    }
    const float inv = 1.f / (float)C;
    typename Raw<T, V>::type rx[NV];
    typename Raw<DT, V>::type rdy[NV];
    float rmean = 0.f, rrstd = 0.f;
    auto fetch = [&](int64_t r) {
        if (r >= a.p.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + l) * V < C) {
                rx[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, (i * TPR + l) * V, C);
                rdy[i] = load_piece<DT, V, ONCE>((const DT*)a.d_y + r * C, (i * TPR + l) * V, C);
            }
        rmean = a.mean[r];
        rrstd = a.rstd[r];
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t r = (int64_t)blockIdx.x * RPB + rr;
    fetch(r);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        const float mean = rmean, rstd = rrstd;
        float h[NV][V], g[NV][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = live && (i * TPR + l) * V + v < C;
                h[i][v] = in ? (to_f(rx[i][v]) - mean) * rstd : 0.f;
                g[i][v] = in ? to_f(rdy[i][v]) : 0.f;
            }
        fetch(r + step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dw[i][v] = __builtin_fmaf(g[i][v], h[i][v], dw[i][v]);
                db[i][v] += g[i][v];
                g[i][v] *= w[i][v];
                s1 += g[i][v];
                s2 = __builtin_fmaf(g[i][v], h[i][v], s2);
            }
#pragma unroll
        for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) {
            s1 += __shfl_xor(s1, m, 64);
            s2 += __shfl_xor(s2, m, 64);
        }
        if constexpr (TPR > 64) {                       // both sums in one exchange, two slots in turn
            if ((threadIdx.x & 63) == 0) {
                red[slot][0][threadIdx.x >> 6] = s1;
                red[slot][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            s1 = (red[slot][0][0] + red[slot][0][1]) + (red[slot][0][2] + red[slot][0][3]);
            s2 = (red[slot][1][0] + red[slot][1][1]) + (red[slot][1][2] + red[slot][1][3]);
            slot ^= 1;
        }
        s1 *= inv;
        s2 *= inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float d[V];
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = rstd * (g[i][v] - s1 - h[i][v] * s2);
            store_piece<GT, V, ONCE>((GT*)a.dx + r * C, c, C, d);
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
                if (c < C) store_piece<float, V>(part + (int64_t)k * C, c, C, k ? db[i] : dw[i]);
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
    int NV, TPR;
};
Shape shape_of(bool bf, int C) {
    const int V = bf ? 8 : 4, units = (C + V - 1) / V;
    if (units <= 16) return {1, 16};
    if (!bf && units <= 32) return {2, 16};
    const int most64 = bf ? 2 : 4;                         // pieces a thread holds with a wavefront a row
    for (int nv = 1; nv <= most64; nv *= 2)
        if (units <= 64 * nv) return {nv, 64};
    const int steps[] = {1, 2, 3, 4, 6, 8, 12, 16};
    for (int nv : steps)
        if (units <= 256 * nv) return {nv, 256};
    return {0, 0};
}

// f(io type, V, NV, TPR)
template <typename F>
hipError_t by_shape(const NormArgs& a, F f) {
    const Shape s = shape_of(a.p.io_dtype == GDR_BF16, a.p.cols);
#define GDR_NORM(T, V_, NV_, TPR_)                                                                                    \
    if (s.NV == NV_ && s.TPR == TPR_) {                                                                               \
        f(T{}, std::integral_constant<int, V_>{}, std::integral_constant<int, NV_>{}, std::integral_constant<int, TPR_>{}); \
        return hipGetLastError();                                                                                     \
    }
    if (a.p.io_dtype == GDR_BF16) {
        GDR_NORM(bf16, 8, 1, 16) GDR_NORM(bf16, 8, 1, 64) GDR_NORM(bf16, 8, 2, 64)
        GDR_NORM(bf16, 8, 1, 256) GDR_NORM(bf16, 8, 2, 256) GDR_NORM(bf16, 8, 3, 256) GDR_NORM(bf16, 8, 4, 256)
        GDR_NORM(bf16, 8, 6, 256) GDR_NORM(bf16, 8, 8, 256)
    } else {
        GDR_NORM(float, 4, 1, 16) GDR_NORM(float, 4, 2, 16) GDR_NORM(float, 4, 1, 64) GDR_NORM(float, 4, 2, 64)
        GDR_NORM(float, 4, 4, 64) GDR_NORM(float, 4, 2, 256) GDR_NORM(float, 4, 3, 256) GDR_NORM(float, 4, 4, 256)
        GDR_NORM(float, 4, 6, 256) GDR_NORM(float, 4, 8, 256) GDR_NORM(float, 4, 12, 256) GDR_NORM(float, 4, 16, 256)
    }
#undef GDR_NORM
    return hipErrorInvalidValue;
}

int64_t row_blocks(int64_t rows, int TPR) { return (rows + kThreads / TPR - 1) / (kThreads / TPR); }

// Workgroups of the forward pass, for n that one trip each would take: four trips a
// workgroup (2,097,152 rows of 128: 192 us, with 8 trips 198, 16 205, one 249; 65,536
// of 4,096: 180, 187, 187 and 234), and more where a launch's threads would pass 32 bits.
int64_t norm_fwd_blocks(int64_t n) {
    constexpr int64_t least = 8192, most = (int64_t)1 << 22;
    static_assert(most * kThreads < ((int64_t)1 << 32), "threads of a launch");
    const int64_t quarter = n / 4 > least ? n / 4 : least;
    return n < quarter ? n : quarter < most ? quarter : most;
}

}  // namespace

// Workgroups of the backward pass, whose partial sums are written and read once
// more: 512, two a compute unit (16,384 x 4,096 bf16: 85 us; 256: 104, 1024: 98;
// 4,001 x 2,561 fp32: 34, 41 and 38).
int norm_bwd_blocks(const gdr_norm_problem_t& p) {
    const int64_t n = row_blocks(p.rows, shape_of(p.io_dtype == GDR_BF16, p.cols).TPR), most = 512;
    return (int)(n < most ? n : most);
}

hipError_t launch_norm_fwd(const NormArgs& a) {
    if (a.p.rows == 0) return hipSuccess;
    return by_shape(a, [&](auto type, auto vec, auto nv, auto tpr) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value;
        const dim3 grid((unsigned)norm_fwd_blocks(row_blocks(a.p.rows, TPR)));
        // (65,536 x 4,096: 180 us against 189, 2,097,152 x 128: 188 against 206; y alone 184 and 194, x alone 186 and 201)
        const bool once = beyond_caches(a.p.rows * a.p.cols * (size_of(a.p.io_dtype) + size_of(a.p.out_dtype)));
        auto go = [&](auto otype, auto past) {
            k_norm_fwd<T, decltype(otype), V, NV, TPR, decltype(past)::value><<<grid, kThreads, 0, a.stream>>>(a);
        };
        auto by_out = [&](auto past) { a.p.out_dtype == GDR_F32 ? go(float{}, past) : go(T{}, past); };
        once ? by_out(std::true_type{}) : by_out(std::false_type{});
    });
}

hipError_t launch_norm_bwd(const NormArgs& a) {
    const int blocks = norm_bwd_blocks(a.p);
    if (blocks > 0) {
        hipError_t e = by_shape(a, [&](auto type, auto vec, auto nv, auto tpr) {
            typedef decltype(type) T;
            constexpr int V = decltype(vec)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value;
            // (65,536 x 4,096 bf16: 281 us against 290, 16,384 x 4,096: 85 against 87; the reads alone 295 and 84)
            const bool once = beyond_caches(
                a.p.rows * a.p.cols * (size_of(a.p.io_dtype) + size_of(a.p.dy_dtype) + size_of(a.p.grad_dtype)));
            auto go = [&](auto dtype, auto gtype, auto past) {
                k_norm_bwd<T, decltype(dtype), decltype(gtype), V, NV, TPR, decltype(past)::value>
                    <<<dim3((unsigned)blocks), kThreads, 0, a.stream>>>(a);
            };
            auto by_dy = [&](auto gtype, auto past) { a.p.dy_dtype == GDR_F32 ? go(float{}, gtype, past) : go(T{}, gtype, past); };
            auto by_grad = [&](auto past) { a.p.grad_dtype == GDR_F32 ? by_dy(float{}, past) : by_dy(T{}, past); };
            once ? by_grad(std::true_type{}) : by_grad(std::false_type{});
        });
        if (e != hipSuccess) return e;
    }
    if (!a.dweight && !a.dbias) return hipSuccess;
    return sum_partials(a.partial, blocks, 2 * (int64_t)a.p.cols, NormGradOut{a.dweight, a.dbias, a.p.cols}, a.stream);
}

}  // namespace gdr
