// The RMS norm with a gate and the residual sum with its norms, forward and backward
// (include/gdr_mixer.h). A few operations an element: HBM bounds them, so a row is
// read once and stays in registers between its sums and its outputs. TPR threads share
// a row, each holding NV pieces of V elements: 16 bytes of the io type, or four elements
// in bf16 beside a stream in fp32 (in_fours). Rows go round the grid, and up to 512 threads
// a row (forward wherever a thread holds eight elements at most) the next row is on its way
// while one is worked on, with the parameters in registers. A thread holds eight elements
// where it can, one piece in bf16, two of four otherwise: 4,096 rows of 8,192 took the backward
// pass 276 us with four pieces and 256 threads, 152 with one, 132 with the parameters' sums in
// LDS. Rows beyond 8,192 overflow into scratch all the same, 212 to 832 bytes a thread (4,096 rows
// of 16,384 in bf16, forward and backward: gated 91 and 257 us, where a copy would take 68 and 113;
// residual sums 198 and 573, 91 and 181), but for the gated forward pass; residual sums' backward
// pass from 4,097 columns on, 84 to 88 bytes.
//
// Measured, at the rate of a copy (5.92 TB/s) in brackets. bf16: gated rows of 128, 2,097,152 of
// them, 279 us (274), 524,288 backward 114 us (114); residual sums of rows of 4,096, 16,384 of them, with
// both norms and a gate per channel 101 us (91), backward with a gate per token 185 us (181); 256
// rows 5.0 us replayed from a graph. fp32: gated rows of 128, 1,048,576 of them, 263 us (273), 262,144
// backward 121 us (114); residual sums of 16,384 rows of 4,096 as above 185 us (181), 8,192 backward
// 183 us (181). Backward, rows of 1,025 to 2,048 have one workgroup of 256 threads to a compute unit:
// 32,768 of 2,048 in bf16 gated 160 us (113), residual 252 us (136).
#include <type_traits>

#include "gdr_norm.hpp"

namespace gdr {

namespace {

template <int TPR> constexpr int kBlock = TPR < 256 ? 256 : TPR;

// Sum over the TPR threads of a row, as in gdr_norm.hip, for any number of wavefronts
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[kBlock<TPR> / 64], int& slot) {
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        const int first = (int)threadIdx.x / TPR * (TPR / 64);
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[slot][first + i];
        slot ^= 1;
    }
    return v;
}

// A parameter's pieces: kept in registers or read again for every row
template <typename T, int V, int NV, int TPR, bool KEEP>
struct Param {
    const void* p;
    int C, f32;
    float none, kept[KEEP ? NV : 1][V];
    __device__ __forceinline__ Param(const void* p_, int C_, int f32_, float none_) : p(p_), C(C_), f32(f32_), none(none_) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                load_param<T, V>(p, (i * TPR + (int)threadIdx.x % TPR) * V, C, f32, none, kept[i]);
        }
    }
    __device__ __forceinline__ void get(int i, float (&f)[V]) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = kept[i][v];
        } else {
            load_param<T, V>(p, (i * TPR + (int)threadIdx.x % TPR) * V, C, f32, none, f);
        }
    }
};

// act(z); silu is z sigmoid(z)
__device__ __forceinline__ float gate_of(float z, bool silu_) {
    const float s = sigmoid(z);
    return silu_ ? z * s : s;
}

// ---------------------------------------------------------------- gated norm
template <typename T, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kBlock<TPR>) void k_gated_norm_fwd(GatedNormArgs a) {
    constexpr int RPB = kBlock<TPR> / TPR;
    constexpr bool AHEAD = NV * V <= 8;
    __shared__ float red[2][kBlock<TPR> / 64];
    int slot = 0;
    const int C = a.p.cols, l = threadIdx.x % TPR;
    const bool act = a.p.activation == GDR_ACT_SILU;
    const Param<T, V, NV, TPR, NV * V <= 8> w(a.weight, C, a.p.param_dtype == GDR_F32, 1.f);
    const float inv = 1.f / (float)C;
    typename Raw<T, V>::type rx[NV], rz[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (r < a.p.rows && c < C) {
                rx[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, c, C);
                rz[i] = load_piece<T, V, ONCE>((const T*)a.z + r * a.p.z_stride, c, C);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (AHEAD) fetch(r);
    // every thread of a workgroup makes the same trips (row_sum meets in barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        if (!AHEAD) fetch(r);
        float x[NV][V], g[NV][V], sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = live && (i * TPR + l) * V + v < C;
                x[i][v] = in ? to_f(rx[i][v]) : 0.f;
                g[i][v] = in ? to_f(rz[i][v]) : 0.f;
                sq = __builtin_fmaf(x[i][v], x[i][v], sq);
            }
        if (AHEAD) fetch(r + step);
        const float rstd = 1.f / sqrtf(row_sum<TPR>(sq, red, slot) * inv + a.p.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float y[V];
            w.get(i, y);
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] *= x[i][v] * rstd * gate_of(g[i][v], act);
            store_any<T, V, ONCE>(a.y, r * C, c, C, a.p.out_dtype == GDR_F32, y);
        }
        if (l == 0 && a.rstd) a.rstd[r] = rstd;
    }
}

// A thread's sums over its rows, a parameter's gradient: in registers, or in LDS where a
// row has 1,024 threads, whose 128 registers would overflow into scratch
template <int V, int NV, int TPR, bool SHARED>
struct Sums {
    float r[NV][V];
    __device__ __forceinline__ explicit Sums(float*) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) r[i][v] = 0.f;
    }
    __device__ __forceinline__ void add(int i, const float (&x)[V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) r[i][v] += x[v];
    }
    __device__ __forceinline__ void get(int i, float (&x)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = r[i][v];
    }
};
template <int V, int NV, int TPR>
struct Sums<V, NV, TPR, true> {
    f32x4* p;                      // [NV][V / 4][TPR], so that the lanes' 16 bytes follow each other
    __device__ __forceinline__ explicit Sums(float* lds) : p((f32x4*)lds + threadIdx.x) {
#pragma unroll
        for (int i = 0; i < NV * V / 4; ++i) p[i * TPR] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void add(int i, const float (&x)[V]) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            p[(i * (V / 4) + j) * TPR] += f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
    }
    __device__ __forceinline__ void get(int i, float (&x)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = p[(i * (V / 4) + v / 4) * TPR][v % 4];
    }
};

// A workgroup's sums of its rows to memory: in LDS over the rows that it takes at a
// time, then a thread a column.
template <int V, int NV, int TPR, bool SHARED>
__device__ __forceinline__ void put_sums(float* part, const Sums<V, NV, TPR, SHARED>& s, int C, float* cols) {
    constexpr int RPB = kBlock<TPR> / TPR;
    const int l = threadIdx.x % TPR, rr = threadIdx.x / TPR;
    if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) cols[rr * (NV * TPR * V) + (i * TPR + l) * V + v] = s.r[i][v];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kBlock<TPR>) {
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < RPB; ++j) x += cols[j * (NV * TPR * V) + c];
            part[c] = x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            float x[V];
            s.get(i, x);
            if (c < C) store_piece<float, V>(part, c, C, x);
        }
    }
}

// With xhat = x rstd, da = d_y act(z) and c = da weight:
//   dx = rstd (c - xhat mean(c xhat)),   dz = d_y xhat weight act'(z),   dweight = sum of da xhat
template <typename T, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kBlock<TPR>) void k_gated_norm_bwd(GatedNormArgs a) {
    constexpr int RPB = kBlock<TPR> / TPR;
    constexpr bool AHEAD = TPR <= 512;
    __shared__ float red[2][kBlock<TPR> / 64];
    constexpr bool SHARED = TPR == 1024;
    __shared__ __attribute__((aligned(16))) float cols[RPB > 1 || SHARED ? RPB * NV * TPR * V : 1];
    int slot = 0;
    const int C = a.p.cols, l = threadIdx.x % TPR;
    const int dy32 = a.p.dy_dtype == GDR_F32, g32 = a.p.grad_dtype == GDR_F32;
    const bool act = a.p.activation == GDR_ACT_SILU;
    const Param<T, V, NV, TPR, NV * V <= 8> w(a.weight, C, a.p.param_dtype == GDR_F32, 1.f);
    const float inv = 1.f / (float)C;
    Sums<V, NV, TPR, SHARED> dw(cols);
    typename Raw<T, V>::type rx[NV], rz[NV];
    AnyPiece<V> rd[NV];
    float rr = 0.f;
    auto fetch = [&](int64_t r) {
        if (r >= a.p.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            rx[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, c, C);
            rz[i] = load_piece<T, V, ONCE>((const T*)a.z + r * a.p.z_stride, c, C);
            load_any<T, V, ONCE>(rd[i], a.d_y, r * C, c, C, dy32);
        }
        rr = a.rstd[r];
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (AHEAD) fetch(r);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        if (!AHEAD) fetch(r);
        const float rstd = rr;
        float x[NV][V], z[NV][V], g[NV][V], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack_any<T, V>(rd[i], dy32, g[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = live && (i * TPR + l) * V + v < C;
                x[i][v] = in ? to_f(rx[i][v]) * rstd : 0.f;
                z[i][v] = in ? to_f(rz[i][v]) : 0.f;
                g[i][v] = in ? g[i][v] : 0.f;
            }
        }
        if (AHEAD) fetch(r + step);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V], e[V];
            w.get(i, f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float sg = sigmoid(z[i][v]), ac = act ? z[i][v] * sg : sg;
                const float slope = act ? silu_slope(z[i][v], sg) : sg * (1.f - sg);
                const float da = g[i][v] * ac;
                e[v] = da * x[i][v];
                z[i][v] = g[i][v] * x[i][v] * f[v] * slope;        // dz
                g[i][v] = da * f[v];                               // c
                s = __builtin_fmaf(g[i][v], x[i][v], s);
            }
            dw.add(i, e);
        }
        s = row_sum<TPR>(s, red, slot) * inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float d[V];
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = rstd * (g[i][v] - x[i][v] * s);
            store_any<T, V, ONCE>(a.dx, r * C, c, C, g32, d);
            store_any<T, V, ONCE>(a.dz, r * C, c, C, g32, z[i]);
        }
    }
    if (a.dweight) put_sums(a.partial + (int64_t)blockIdx.x * C, dw, C, cols);
}

// ---------------------------------------------------------------- residual sum with norms
template <typename T, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kBlock<TPR>) void k_residual_norm_fwd(ResidualNormArgs a) {
    constexpr int RPB = kBlock<TPR> / TPR;
    constexpr bool AHEAD = NV * V <= 8;
    __shared__ float red[2][kBlock<TPR> / 64];
    int slot = 0;
    const int C = a.p.cols, l = threadIdx.x % TPR, p32 = a.p.param_dtype == GDR_F32, s32 = a.p.stream_dtype == GDR_F32;
    const bool post = a.x_weight != nullptr, token = a.p.gate == GDR_GATE_TOKEN;
    const Param<T, V, NV, TPR, TPR <= 512> w(a.weight, C, p32, 1.f), xw(a.x_weight, C, p32, 1.f);
    const Param<T, V, NV, TPR, TPR <= 512> gc(a.p.gate == GDR_GATE_CHANNEL ? a.gate : nullptr, C, p32, 1.f);
    const float inv = 1.f / (float)C;
    typename Raw<T, V>::type rx[NV], rg[NV];
    AnyPiece<V> rs[NV];
    auto fetch = [&](int64_t r) {
        if (r >= a.p.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            rx[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, c, C);
            load_any<T, V, ONCE>(rs[i], a.residual, r * a.p.residual_stride, c, C, s32);
            if (token) rg[i] = load_piece<T, V, ONCE>((const T*)a.gate + r * a.p.gate_stride, c, C);
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (AHEAD) fetch(r);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        if (!AHEAD) fetch(r);
        float x[NV][V], h[NV][V], g[NV][V], sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack_any<T, V>(rs[i], s32, h[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = live && (i * TPR + l) * V + v < C;
                x[i][v] = in ? to_f(rx[i][v]) : 0.f;
                h[i][v] = in ? h[i][v] : 0.f;
                g[i][v] = token ? (in ? to_f(rg[i][v]) : 0.f) : 1.f;
                sq = __builtin_fmaf(x[i][v], x[i][v], sq);
            }
        }
        if (AHEAD) fetch(r + step);
        float xr = 1.f;
        if (post) xr = 1.f / sqrtf(row_sum<TPR>(sq, red, slot) * inv + a.p.eps);
        sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V], k[V];
            xw.get(i, f);
            gc.get(i, k);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float m = a.p.scale * (k[v] * g[i][v]);
                h[i][v] = __builtin_fmaf(m, x[i][v] * xr * f[v], h[i][v]);
                sq = __builtin_fmaf(h[i][v], h[i][v], sq);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(sq, red, slot) * inv + a.p.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float y[V];
            w.get(i, y);
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] *= h[i][v] * rstd;
            store_any<T, V, ONCE>(a.y, r * C, c, C, a.p.out_dtype == GDR_F32, y);
            store_any<T, V, ONCE>(a.h, r * C, c, C, s32, h[i]);
        }
        if (l == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if (a.x_rstd && post) a.x_rstd[r] = xr;
        }
    }
}

// With hhat = h rstd, xhat = x x_rstd and m = scale gate:
//   c = d_y weight,          dh = d_h + rstd (c - hhat mean(c hhat)),   dresidual = dh,   dweight = sum of d_y hhat
//   e = m dh x_weight,       dx = x_rstd (e - xhat mean(e xhat)) (or m dh),   dx_weight = sum of m dh xhat
//   dgate = scale dh xhat x_weight (or scale dh x), summed over the rows for a gate per channel
template <typename T, int V, int NV, int TPR, bool ONCE>
__global__ __launch_bounds__(kBlock<TPR>) void k_residual_norm_bwd(ResidualNormArgs a) {
    constexpr int RPB = kBlock<TPR> / TPR;
    constexpr bool AHEAD = TPR <= 512;
    __shared__ float red[2][kBlock<TPR> / 64];
    constexpr bool SHARED = TPR == 1024;
    __shared__ __attribute__((aligned(16))) float cols[RPB > 1 ? RPB * NV * TPR * V : SHARED ? 2 * NV * TPR * V : 1];
    int slot = 0;
    const int C = a.p.cols, l = threadIdx.x % TPR, p32 = a.p.param_dtype == GDR_F32, s32 = a.p.stream_dtype == GDR_F32;
    const int dy32 = a.p.dy_dtype == GDR_F32, dh32 = a.p.dh_dtype == GDR_F32;
    const bool post = a.x_weight != nullptr, token = a.p.gate == GDR_GATE_TOKEN, chan = a.p.gate == GDR_GATE_CHANNEL;
    const Param<T, V, NV, TPR, TPR <= 512> w(a.weight, C, p32, 1.f), xw(a.x_weight, C, p32, 1.f), gc(chan ? a.gate : nullptr, C, p32, 1.f);
    const float inv = 1.f / (float)C;
    Sums<V, NV, TPR, SHARED> dw(cols), dxw(cols + NV * TPR * V * SHARED);
    Sums<V, NV, TPR, false> dg(nullptr);
    typename Raw<T, V>::type rx[NV], rg[NV];
    AnyPiece<V> rh[NV], ry[NV], rd[NV];
    float r1 = 0.f, r2 = 1.f;
    auto fetch = [&](int64_t r) {
        if (r >= a.p.rows) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            rx[i] = load_piece<T, V, ONCE>((const T*)a.x + r * a.p.x_stride, c, C);
            load_any<T, V, ONCE>(rh[i], a.h_in, r * C, c, C, s32);
            load_any<T, V, ONCE>(ry[i], a.d_y, r * C, c, C, dy32);
            if (a.d_h) load_any<T, V, ONCE>(rd[i], a.d_h, r * C, c, C, dh32);
            if (token) rg[i] = load_piece<T, V, ONCE>((const T*)a.gate + r * a.p.gate_stride, c, C);
        }
        r1 = a.rstd[r];
        if (post) r2 = a.x_rstd[r];
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (AHEAD) fetch(r);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.p.rows; r0 += step, r += step) {
        const bool live = r < a.p.rows;
        if (!AHEAD) fetch(r);
        const float rstd = r1, xr = r2;
        float x[NV][V], h[NV][V], c1[NV][V], d[NV][V], g[NV][V], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack_any<T, V>(rh[i], s32, h[i]);
            unpack_any<T, V>(ry[i], dy32, c1[i]);
            unpack_any<T, V>(rd[i], dh32, d[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool in = live && (i * TPR + l) * V + v < C;
                x[i][v] = in ? to_f(rx[i][v]) * xr : 0.f;
                h[i][v] = in ? h[i][v] * rstd : 0.f;
                c1[i][v] = in ? c1[i][v] : 0.f;
                d[i][v] = in && a.d_h ? d[i][v] : 0.f;
                g[i][v] = token ? (in ? to_f(rg[i][v]) : 0.f) : 1.f;
            }
        }
        if (AHEAD) fetch(r + step);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V], e[V];
            w.get(i, f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e[v] = c1[i][v] * h[i][v];
                c1[i][v] *= f[v];
                s = __builtin_fmaf(c1[i][v], h[i][v], s);
            }
            dw.add(i, e);
        }
        s = row_sum<TPR>(s, red, slot) * inv;
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            float f[V], k[V], e[V];
            xw.get(i, f);
            gc.get(i, k);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[i][v] = __builtin_fmaf(rstd, c1[i][v] - h[i][v] * s, d[i][v]);       // dh
                const float m = a.p.scale * (k[v] * g[i][v]) * d[i][v];
                e[v] = m * x[i][v];
                g[i][v] = a.p.scale * d[i][v] * x[i][v] * f[v];                        // dgate
                h[i][v] = m * f[v];
                t = __builtin_fmaf(h[i][v], x[i][v], t);
            }
            dxw.add(i, e);
            dg.add(i, g[i]);
            if (!live || c >= C) continue;
            store_any<T, V, ONCE>(a.dresidual, r * C, c, C, a.p.dres_dtype == GDR_F32, d[i]);
            if (token && a.dgate) store_any<T, V, ONCE>(a.dgate, r * C, c, C, a.p.grad_dtype == GDR_F32, g[i]);
        }
        if (post) t = row_sum<TPR>(t, red, slot) * inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + l) * V;
            if (c >= C) continue;
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = post ? xr * (h[i][v] - x[i][v] * t) : h[i][v];
            store_any<T, V, ONCE>(a.dx, r * C, c, C, a.p.grad_dtype == GDR_F32, y);
        }
    }
    float* part = a.partial + (int64_t)blockIdx.x * 3 * C;
    put_sums(part, dw, C, cols);
    if (post) put_sums(part + C, dxw, C, cols);
    if (chan) put_sums(part + 2 * (int64_t)C, dg, C, cols);
}

struct OneSum {
    float* out;
    __device__ void operator()(int64_t i, float v) const { out[i] = v; }
};
struct ThreeSums {
    float *a, *b, *c;
    int C;
    __device__ void operator()(int64_t i, float v) const {
        float* p = i < C ? a : i < 2 * (int64_t)C ? b : c;
        if (p) p[i % C] = v;
    }
};

// The variant for a row of C elements: the fewest threads whose registers hold it
struct Shape {
    int NV, TPR;
};
Shape shape_of(bool bf, int C) {
    const Shape b[] = {{1, 8}, {1, 16}, {1, 32}, {1, 64}, {1, 128}, {1, 256}, {1, 512}, {1, 1024}, {2, 1024}};
    const Shape f[] = {{1, 16}, {2, 16}, {2, 32}, {2, 64}, {2, 128}, {2, 256}, {2, 512}, {2, 1024}, {4, 1024}};
    const int V = bf ? 8 : 4, n = 9;
    for (int i = 0; i < n; ++i) {
        const Shape s = bf ? b[i] : f[i];
        if (C <= V * s.NV * s.TPR) return s;
    }
    return {0, 0};
}

// Whether bf16 rows beside a stream in fp32 go in pieces of four elements, so that a
// wavefront's accesses to the stream lie side by side, or of eight. us for 256 MB of x, eight and four:
//   both norms, gate per channel    56: 386 321    104: 386 426   192: 367 298   264: 422 367   640: 367 302
//                                   1,024: 407 294   4,096: 404 302   8,192: 403 303   10,000: 567 521
//   one parameter                   56: 323 274    104: 327 372   120: 322 350   200: 332 360   264: 429 486
//                                   448: 325 323   640: 378 421   896: 346 327   1,024: 339 297   4,096: 348 308
//                                   8,192: 390 357   10,000: 1,071 1,264   16,384: 752 821
// and 4 MB of rows of 100, whose end cuts a piece of eight: 9.1 and 7.9; of others up to 960 eights are 0
// to 6 % faster there, of 8,200 15 %. Four for wide rows, for ones that fill the threads of their
// variant or nearly so, for ones that eights cut, and where several parameters are kept.
bool in_fours(int C, bool one) {
    if (C > 8192) return false;
    return C >= 1024 || C % 8 != 0 || C >= 7 * shape_of(true, C).TPR || (!one && C > 128);
}

// f(io type, V, NV, TPR). FOURS: bf16 rows in pieces of four, up to 8,192 columns
template <bool FOURS = false, typename F>
hipError_t by_shape(bool bf, int C, F f) {
    const Shape s = shape_of(bf && !FOURS, C);
#define GDR_SHAPE(T, V_, NV_, TPR_)                                                                                   \
    if (s.NV == NV_ && s.TPR == TPR_) {                                                                               \
        f(T{}, std::integral_constant<int, V_>{}, std::integral_constant<int, NV_>{}, std::integral_constant<int, TPR_>{}); \
        return hipGetLastError();                                                                                     \
    }
#define GDR_FOURS(T)                                                                                                   \
    GDR_SHAPE(T, 4, 1, 16) GDR_SHAPE(T, 4, 2, 16) GDR_SHAPE(T, 4, 2, 32) GDR_SHAPE(T, 4, 2, 64) GDR_SHAPE(T, 4, 2, 128) \
    GDR_SHAPE(T, 4, 2, 256) GDR_SHAPE(T, 4, 2, 512) GDR_SHAPE(T, 4, 2, 1024)
    if (!bf) {
        GDR_FOURS(float) GDR_SHAPE(float, 4, 4, 1024)
    } else if constexpr (FOURS) {
        GDR_FOURS(bf16)
    } else {
        GDR_SHAPE(bf16, 8, 1, 8) GDR_SHAPE(bf16, 8, 1, 16) GDR_SHAPE(bf16, 8, 1, 32) GDR_SHAPE(bf16, 8, 1, 64)
        GDR_SHAPE(bf16, 8, 1, 128) GDR_SHAPE(bf16, 8, 1, 256) GDR_SHAPE(bf16, 8, 1, 512) GDR_SHAPE(bf16, 8, 1, 1024)
        GDR_SHAPE(bf16, 8, 2, 1024)
    }
#undef GDR_FOURS
#undef GDR_SHAPE
    return hipErrorInvalidValue;
}

int64_t row_blocks(int64_t rows, int TPR) {
    const int rpb = TPR < 256 ? 256 / TPR : 1;
    return (rows + rpb - 1) / rpb;
}
// Workgroups that the rows go round, forward. With one parameter a workgroup for the rows
// that it takes at a time: 2,097,152 gated rows of 128 took 276 us so and 310 in 8,192
// workgroups; sums onto a stream in fp32, 256 MB of rows of 512, 312 and 386. With more of
// them a workgroup that reads them all for one row pays: with both norms and a gate per
// channel 256 MB of rows of 512 took 242 us so, 197 in 8,192 workgroups, 212 in 2,048; rows
// of 4,096 245, 206 and 196, and 64 MB of these 61, 60, 52 and in 1,024 49.
unsigned fwd_blocks(int64_t rows, int TPR, bool one) {
    const int64_t n = row_blocks(rows, TPR), most = one ? (int64_t)1 << 21 : TPR < 256 ? 8192 : 1024;
    return (unsigned)(n < most ? n : most);
}
// Backward, each workgroup leaves its sums for the parameters: rows of 1,024 took 274 us in
// 256 workgroups, 201 in 512 and 205 in 1,024, rows of 4,096 188, 192 and 201.
int bwd_blocks(int64_t rows, bool bf, int C) {
    const int TPR = shape_of(bf, C).TPR;
    const int64_t n = row_blocks(rows, TPR), most = TPR < 256 ? 512 : 256;
    return (int)(n < most ? n : most);
}

}  // namespace

int gated_norm_bwd_blocks(const gdr_gated_norm_problem_t& p) { return bwd_blocks(p.rows, p.io_dtype == GDR_BF16, p.cols); }
int residual_norm_bwd_blocks(const gdr_residual_norm_problem_t& p) {
    return bwd_blocks(p.rows, p.io_dtype == GDR_BF16, p.cols);
}

#define GDR_LAUNCH(kernel, grid, once, a)                                                                         \
    do {                                                                                                          \
        typedef decltype(type) T;                                                                                 \
        constexpr int V = decltype(vec)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value;             \
        if (once) kernel<T, V, NV, TPR, true><<<dim3(grid), kBlock<TPR>, 0, (a).stream>>>(a);                     \
        else kernel<T, V, NV, TPR, false><<<dim3(grid), kBlock<TPR>, 0, (a).stream>>>(a);                         \
    } while (0)

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a) {
    if (a.p.rows == 0) return hipSuccess;
    const bool once = beyond_caches(a.p.rows * a.p.cols * (2 * size_of(a.p.io_dtype) + size_of(a.p.out_dtype)));
    return by_shape(a.p.io_dtype == GDR_BF16, a.p.cols, [&](auto type, auto vec, auto nv, auto tpr) {
        GDR_LAUNCH(k_gated_norm_fwd, fwd_blocks(a.p.rows, TPR, true), once, a);
    });
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a) {
    const int blocks = gated_norm_bwd_blocks(a.p);
    if (blocks > 0) {
        const bool once = beyond_caches(a.p.rows * a.p.cols *
                                        (2 * size_of(a.p.io_dtype) + size_of(a.p.dy_dtype) + 2 * size_of(a.p.grad_dtype)));
        const hipError_t e = by_shape(a.p.io_dtype == GDR_BF16, a.p.cols, [&](auto type, auto vec, auto nv, auto tpr) {
            GDR_LAUNCH(k_gated_norm_bwd, (unsigned)blocks, once, a);
        });
        if (e != hipSuccess) return e;
    }
    return a.dweight ? sum_partials(a.partial, blocks, a.p.cols, OneSum{a.dweight}, a.stream) : hipSuccess;
}

hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a) {
    if (a.p.rows == 0) return hipSuccess;
    const int token = a.p.gate == GDR_GATE_TOKEN;
    const bool one = !a.x_weight && a.p.gate != GDR_GATE_CHANNEL;
    const bool once = beyond_caches(a.p.rows * a.p.cols * ((1 + token) * size_of(a.p.io_dtype) + size_of(a.p.out_dtype) +
                                                           2 * size_of(a.p.stream_dtype)));
    auto go = [&](auto type, auto vec, auto nv, auto tpr) {
        GDR_LAUNCH(k_residual_norm_fwd, fwd_blocks(a.p.rows, TPR, one), once, a);
    };
    if (a.p.io_dtype == GDR_BF16 && a.p.stream_dtype == GDR_F32 && in_fours(a.p.cols, one))
        return by_shape<true>(true, a.p.cols, go);
    return by_shape(a.p.io_dtype == GDR_BF16, a.p.cols, go);
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a) {
    const int blocks = residual_norm_bwd_blocks(a.p);
    const bool chan = a.p.gate == GDR_GATE_CHANNEL;
    if (blocks > 0) {
        const int token = a.p.gate == GDR_GATE_TOKEN;
        const bool once = beyond_caches(a.p.rows * a.p.cols *
                                        ((1 + token) * (size_of(a.p.io_dtype) + size_of(a.p.grad_dtype)) +
                                         size_of(a.p.stream_dtype) + size_of(a.p.dy_dtype) + size_of(a.p.dh_dtype) +
                                         size_of(a.p.dres_dtype)));
        const hipError_t e = by_shape(a.p.io_dtype == GDR_BF16, a.p.cols, [&](auto type, auto vec, auto nv, auto tpr) {
            GDR_LAUNCH(k_residual_norm_bwd, (unsigned)blocks, once, a);
        });
        if (e != hipSuccess) return e;
    }
    ThreeSums out{a.dweight, a.x_weight ? a.dx_weight : nullptr, chan ? (float*)a.dgate : nullptr, a.p.cols};
    if (!out.a && !out.b && !out.c) return hipSuccess;
    return sum_partials(a.partial, blocks, 3 * (int64_t)a.p.cols, out, a.stream);
}

}  // namespace gdr
