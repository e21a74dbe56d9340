// Short causal convolution, one filter of W = 2, 3 or 4 taps per channel, for
// packed sequences with initial and final rows: forward, one token per
// sequence, backward (include/gdr_mixer.h).
//
//   p_t = bias + sum_w weight[w] u_{t-(W-1)+w},  u = (initial rows | x),  y = p or p sigmoid(p)
//
// 2 W + 5 operations on 4 to 8 bytes: HBM bounds every form. So each element
// moves once, 16 bytes a lane (a wavefront reads 1 KB of a token's row), and a
// lane walks kRun tokens of its channels with the last W - 1 rows in registers;
// only the W - 1 rows before a run are read again.
#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

namespace {

constexpr int kRun = 32;       // tokens a wavefront walks
constexpr int kWaves = 4;      // wavefronts of a workgroup: consecutive runs of the same channels
constexpr int kGroup = 8;      // rows loaded together, ahead of their use

// One row of a sequence's u at token t (t may lie before its start s)
template <typename T, int V>
__device__ __forceinline__ void load_u(const ConvArgs& a, int64_t t, int64_t s, int q, int W, int ch, float (&f)[V]) {
    if (t >= s) {
        unpack<T, V>(load_raw<T, V>((const T*)a.x + t * a.p.x_stride + ch), f);
    } else if (const int64_t j = t - s + (W - 1); a.S0 && j >= 0) {
        unpack<T, V>(load_raw<T, V>((const T*)a.S0 + ((int64_t)q * (W - 1) + j) * a.p.channels + ch), f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
}

template <typename T, int V, int W>
struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvArgs& a, int ch) {
        const int f32 = a.p.param_dtype == GDR_F32;
#pragma unroll
        for (int i = 0; i < W; ++i) {                    // V W consecutive elements, V at a time
            float part[V];
            load_vec_as<T, V>(a.weight, (int64_t)ch * W + i * V, f32, part);
#pragma unroll
            for (int v = 0; v < V; ++v) w[(i * V + v) % W][(i * V + v) / W] = part[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = 0.f;
        if (a.bias) load_vec_as<T, V>(a.bias, ch, f32, b);
    }
    // p of the token whose row is `x`, after the rows hist[0..W-2] (oldest first)
    __device__ __forceinline__ float at(const float (&hist)[W - 1][V], const float (&x)[V], int v) const {
        float p = b[v];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) p = __builtin_fmaf(w[i][v], hist[i][v], p);
        return __builtin_fmaf(w[W - 1][v], x[v], p);
    }
};

template <int W, int V>
__device__ __forceinline__ void push(float (&hist)[W - 1][V], const float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i) hist[i][v] = hist[i + 1][v];
        hist[W - 2][v] = x[v];
    }
}

template <typename T, int V, int W>
__global__ __launch_bounds__(256) void k_conv_fwd(ConvArgs a, int ncb, int64_t ntiles) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cb = blockIdx.x % ncb;
    const int64_t tile = blockIdx.x / ncb;
    const int D = a.p.channels, ch = (cb * 64 + lane) * V;
    if (ch >= D) return;
    if (tile >= ntiles) {                                // the final rows of sequences, kWaves of them a workgroup
        const int64_t q = (tile - ntiles) * kWaves + wave;
        if (q >= a.p.num_seqs) return;
        int64_t s, e;
        seq_range(a.cu, (int)q, a.p.seq_len, a.Ttot, &s, &e);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float f[V];
            load_u<T, V>(a, e - (W - 1) + j, s, (int)q, W, ch, f);
            store_vec<T, V>((T*)a.ST + (q * (W - 1) + j) * D + ch, f);
        }
        return;
    }
    const int64_t t0 = (tile * kWaves + wave) * kRun;
    if (t0 >= a.Ttot) return;
    const int64_t t1 = t0 + kRun < a.Ttot ? t0 + kRun : a.Ttot;
    Taps<T, V, W> taps;
    taps.load(a, ch);
    const bool silu_on = a.p.activation == GDR_ACT_SILU;
    int q = seq_of_token(a.cu, a.p.num_seqs, a.p.seq_len, t0);
    int64_t s, e;
    seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
    float hist[W - 1][V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_u<T, V>(a, t0 - (W - 1) + i, s, q, W, ch, hist[i]);
    for (int64_t tb = t0; tb < t1; tb += kGroup) {
        typename Raw<T, V>::type raw[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (tb + j < t1) raw[j] = load_raw<T, V>((const T*)a.x + (tb + j) * a.p.x_stride + ch);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            const int64_t t = tb + j;
            if (t >= t1) break;
            if (t >= e && q + 1 < a.p.num_seqs) {        // the next sequence that is not empty starts here
                do {
                    ++q;
                    seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
                } while (t >= e && q + 1 < a.p.num_seqs);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) load_u<T, V>(a, s - (W - 1) + i, s, q, W, ch, hist[i]);
            }
            float x[V], y[V];
            unpack<T, V>(raw[j], x);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float p = taps.at(hist, x, v);
                y[v] = silu_on ? silu(p) : p;
            }
            store_vec<T, V>((T*)a.y + t * D + ch, y);
            push<W, V>(hist, x);
        }
    }
}

// One token of every sequence; a lane reads its W - 1 state rows before it
// overwrites them, so the state changes in place.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void k_conv_step(ConvArgs a, int ncb) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cb = blockIdx.x % ncb;
    const int64_t n = (int64_t)(blockIdx.x / ncb) * kWaves + wave;
    const int D = a.p.channels, ch = (cb * 64 + lane) * V;
    if (ch >= D || n >= a.p.num_seqs) return;
    T* st = (T*)a.ST + n * (W - 1) * D + ch;
    typename Raw<T, V>::type raw[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) raw[i] = load_raw<T, V>(st + (int64_t)i * D);
    raw[W - 1] = load_raw<T, V>((const T*)a.x + n * a.p.x_stride + ch);
    Taps<T, V, W> taps;
    taps.load(a, ch);
    float hist[W - 1][V], x[V], y[V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) unpack<T, V>(raw[i], hist[i]);
    unpack<T, V>(raw[W - 1], x);
    const bool silu_on = a.p.activation == GDR_ACT_SILU;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float p = taps.at(hist, x, v);
        y[v] = silu_on ? silu(p) : p;
    }
    store_vec<T, V>((T*)a.y + n * D + ch, y);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) *reinterpret_cast<typename Raw<T, V>::type*>(st + (int64_t)i * D) = raw[i + 1];
}

// Backward. With dp = d_y act'(p), position r of u (a token, or an initial row)
// receives du_r = sum_w weight[w] dp_{r+(W-1)-w} over the tokens of its sequence,
// plus the final state's gradient where r is among the last W - 1 positions. A
// run walks its tokens and up to W - 1 more of the same sequence; having formed
// dp_t it can finish position r = t - (W - 1). At the end of a sequence it feeds
// W - 1 zeros. A position is stored by the run that holds its token; an initial
// row by the run that holds the sequence's first token.
template <typename T, int V, int W>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvArgs a, int ncb, int64_t ntiles) {
    __shared__ float red[kWaves][W + 1][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cb = blockIdx.x % ncb;
    const int64_t tile = blockIdx.x / ncb;
    const int D = a.p.channels, ch = (cb * 64 + lane) * V;
    const bool active = ch < D;
    const int dy32 = a.p.dy_dtype == GDR_F32, g32 = a.p.grad_dtype == GDR_F32;
    if (tile >= ntiles) {                                // empty sequences: d_initial_state = d_final_state
        const int64_t q = (tile - ntiles) * kWaves + wave;
        if (!active || q >= a.p.num_seqs) return;
        int64_t s, e;
        seq_range(a.cu, (int)q, a.p.seq_len, a.Ttot, &s, &e);
        if (e > s) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t at = (q * (W - 1) + j) * D + ch;
            float f[V] = {};
            if (a.dST) load_vec_as<T, V>(a.dST, at, dy32, f);
            store_vec_as<T, V>(a.dS0, at, f, g32);
        }
        return;
    }
    const int64_t t0 = (tile * kWaves + wave) * kRun;
    float dw[W][V] = {}, db[V] = {};
    if (active && t0 < a.Ttot) {
        const int64_t t1 = t0 + kRun < a.Ttot ? t0 + kRun : a.Ttot;
        Taps<T, V, W> taps;
        taps.load(a, ch);
        const bool silu_on = a.p.activation == GDR_ACT_SILU;
        int q = seq_of_token(a.cu, a.p.num_seqs, a.p.seq_len, t0);
        int64_t s, e;
        seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
        float hist[W - 1][V], dph[W - 1][V];             // rows before the token; dp of the tokens before it
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            load_u<T, V>(a, t0 - (W - 1) + i, s, q, W, ch, hist[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) dph[i][v] = 0.f;
        }
        // finishes position r with the newest dp
        auto emit = [&](int64_t r, const float (&dp)[V]) {
            const bool mine = r >= s ? (r >= t0 && r < t1) : (s >= t0 && s < t1 && a.dS0 != nullptr);
            if (!mine) return;
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[v] = taps.w[0][v] * dp[v];
#pragma unroll
                for (int w = 1; w < W; ++w) f[v] = __builtin_fmaf(taps.w[w][v], dph[W - 1 - w][v], f[v]);
            }
            if (a.dST && r >= e - (W - 1)) {
                float g[V];
                load_vec_as<T, V>(a.dST, ((int64_t)q * (W - 1) + (r - (e - (W - 1)))) * D + ch, dy32, g);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] += g[v];
            }
            if (r >= s) store_vec_as<T, V>(a.dx, r * D + ch, f, g32);
            else store_vec_as<T, V>(a.dS0, ((int64_t)q * (W - 1) + (r - s + W - 1)) * D + ch, f, g32);
        };
        int64_t t = t0;
        while (true) {
            if (t >= e) {                                // the sequence has ended: its last W - 1 positions
                float zero[V] = {};
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    emit(e - (W - 1) + i, zero);
                    push<W, V>(dph, zero);
                }
                while (t >= e && q + 1 < a.p.num_seqs) {
                    ++q;
                    seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
                }
                if (t >= t1 || t >= e) break;
#pragma unroll
                for (int i = 0; i < W - 1; ++i) load_u<T, V>(a, s - (W - 1) + i, s, q, W, ch, hist[i]);
            }
            // up to W - 1 tokens behind the run while it has positions to finish
            const int64_t stop = e < t1 + (W - 1) ? e : t1 + (W - 1);
            if (t >= stop) break;
            const int m = (int)(stop - t < kGroup ? stop - t : kGroup);
            typename Raw<T, V>::type rx[kGroup];
            float dy[kGroup][V];
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (j < m) {
                    rx[j] = load_raw<T, V>((const T*)a.x + (t + j) * a.p.x_stride + ch);
                    load_vec_as<T, V>(a.d_y, (t + j) * D + ch, dy32, dy[j]);
                }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (j >= m) break;
                float x[V], dp[V];
                unpack<T, V>(rx[j], x);
                const bool own = t + j < t1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dp[v] = silu_on ? dy[j][v] * silu_grad(taps.at(hist, x, v)) : dy[j][v];
                    if (own) {
#pragma unroll
                        for (int w = 0; w < W - 1; ++w) dw[w][v] = __builtin_fmaf(dp[v], hist[w][v], dw[w][v]);
                        dw[W - 1][v] = __builtin_fmaf(dp[v], x[v], dw[W - 1][v]);
                        db[v] += dp[v];
                    }
                }
                emit(t + j - (W - 1), dp);
                push<W, V>(hist, x);
                push<W, V>(dph, dp);
            }
            t += m;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int w = 0; w < W; ++w) red[wave][w][lane * V + v] = dw[w][v];
        red[wave][W][lane * V + v] = db[v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 256) {
        const int w = i / (64 * V), c = i % (64 * V), d = cb * 64 * V + c;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += red[k][w][c];
        if (d < D) a.partial[(tile * (W + 1) + w) * D + d] = v;
    }
}

struct ConvGradOut {
    float *dweight, *dbias;
    int D, W;
    __device__ void operator()(int64_t i, float v) const {
        const int w = (int)(i / D), d = (int)(i % D);
        if (w < W) dweight[(int64_t)d * W + w] = v;
        else if (dbias) dbias[d] = v;
    }
};

template <typename F>
hipError_t by_type(const ConvArgs& a, F f) {
    auto by_width = [&](auto type, auto vec) {
        switch (a.p.width) {
            case 2: return f(type, vec, std::integral_constant<int, 2>{});
            case 3: return f(type, vec, std::integral_constant<int, 3>{});
            case 4: return f(type, vec, std::integral_constant<int, 4>{});
        }
        return hipErrorInvalidValue;
    };
    if (a.p.io_dtype == GDR_BF16)
        return a.wide ? by_width(bf16{}, std::integral_constant<int, 8>{}) : by_width(bf16{}, std::integral_constant<int, 1>{});
    return a.wide ? by_width(float{}, std::integral_constant<int, 4>{}) : by_width(float{}, std::integral_constant<int, 1>{});
}

int channel_blocks(const ConvArgs& a, int V) { return (a.p.channels + 64 * V - 1) / (64 * V); }
int64_t run_tiles(int64_t Ttot) { return (Ttot + kRun * kWaves - 1) / (kRun * kWaves); }
int64_t seq_tiles(const ConvArgs& a) { return ((int64_t)a.p.num_seqs + kWaves - 1) / kWaves; }

}  // namespace

int64_t conv_bwd_tiles(int64_t Ttot, int32_t) { return run_tiles(Ttot); }

hipError_t launch_conv_fwd(const ConvArgs& a) {
    return by_type(a, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int ncb = channel_blocks(a, V);
        const int64_t ntiles = run_tiles(a.Ttot), all = ntiles + (a.ST ? seq_tiles(a) : 0);
        if (!grid_fits(all * ncb, 256)) return hipErrorInvalidConfiguration;
        if (all > 0) k_conv_fwd<T, V, W><<<dim3((unsigned)(all * ncb)), 256, 0, a.stream>>>(a, ncb, ntiles);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(const ConvArgs& a) {
    return by_type(a, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int ncb = channel_blocks(a, V);
        if (!grid_fits(seq_tiles(a) * ncb, 256)) return hipErrorInvalidConfiguration;
        if (seq_tiles(a) > 0) k_conv_step<T, V, W><<<dim3((unsigned)(seq_tiles(a) * ncb)), 256, 0, a.stream>>>(a, ncb);
        return hipGetLastError();
    });
}

hipError_t launch_conv_bwd(const ConvArgs& a) {
    const int64_t ntiles = run_tiles(a.Ttot);
    hipError_t e = by_type(a, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int ncb = channel_blocks(a, V);
        const int64_t all = ntiles + (a.dS0 ? seq_tiles(a) : 0);
        if (!grid_fits(all * ncb, 256)) return hipErrorInvalidConfiguration;
        if (all > 0) k_conv_bwd<T, V, W><<<dim3((unsigned)(all * ncb)), 256, 0, a.stream>>>(a, ncb, ntiles);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const int D = a.p.channels, W = a.p.width;
    return sum_partials(a.partial, ntiles, (int64_t)(W + 1) * D, ConvGradOut{a.dweight, a.dbias, D, W}, a.stream);
}

}  // namespace gdr
