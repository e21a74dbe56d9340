// Short causal convolution, one filter of W = 2, 3 or 4 taps per channel, for
// packed sequences with initial and final rows: forward, one token per
// sequence, backward (include/gdr_mixer.h).
//
//   p_t = bias + sum_w weight[w] u_{t-(W-1)+w},  u = (initial rows | x),  y = p or p sigmoid(p)
//
// 2 W + 5 operations on 4 to 8 bytes: HBM bounds every form. So each element
// moves once, 8 or 16 bytes a lane, and a wavefront walks a run of tokens with
// the last W - 1 rows of its channels in registers; only the W - 1 rows before
// a run (and, backward, behind it) are read again. 65,536 tokens of 8,192 bf16
// channels: 385 to 400 us by the run, 5.4 to 5.6 TB/s (copies of 1 GiB: torch's
// 5.2, one past the caches 5.9).
#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

namespace {

constexpr int kWaves = 4;      // wavefronts of a workgroup
constexpr int kGroup = 4;      // rows loaded together (8: 405 us instead of 385; 2: 396)
// Elements of a bf16 row a lane moves at once. Forward 8 (4: 401 us instead of
// 385). Backward 4: with 8 the registers of taps, their sums and two histories
// leave one wavefront on a SIMD instead of three (150 us instead of 130 on 16,384
// tokens of 6,144 channels).
constexpr int kFwdV = 8, kBwdV = 4;

// Tokens a wavefront walks: the longest run, up to `most`, that still makes 2048
// wavefronts (two a SIMD); one group where there is too little work for that. Longest:
// forward 64 (32: 411 us, 128: 405, 64: 385), backward 128 (64: 133 us, 128: 130).
int run_length(int64_t Ttot, int wavefronts, int most) {
    int run = most;
    while (run > kGroup && (Ttot + run - 1) / run * wavefronts < 2048) run /= 2;
    return run;
}

// A lane's first channel. Where V does not divide the channels the last lanes of a
// row overlap and store the same values twice.
template <int V>
__device__ __forceinline__ int first_channel(int at, int D) { return at + V <= D ? at : D - V; }

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

// ONCE: x and y go past the caches
template <typename T, int V, int W, bool ONCE>
__global__ __launch_bounds__(256) void k_conv_fwd(ConvArgs a, int ncb, int64_t ntiles, int run) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cb = blockIdx.x % ncb;
    const int64_t tile = blockIdx.x / ncb;
    const int D = a.p.channels, at = (cb * 64 + lane) * V, ch = first_channel<V>(at, D);
    const int64_t t0 = (tile * kWaves + wave) * run;
    int q = 0;
    if (tile < ntiles) {
        if (t0 >= a.Ttot) return;
        q = seq_of_token(a.cu, a.p.num_seqs, a.p.seq_len, t0);
    }
    if (at >= D) return;
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
    const int64_t t1 = t0 + run < a.Ttot ? t0 + run : a.Ttot;
    Taps<T, V, W> taps;
    taps.load(a, ch);
    const bool silu_on = a.p.activation == GDR_ACT_SILU;
    int64_t s, e;
    seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
    float hist[W - 1][V];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_u<T, V>(a, t0 - (W - 1) + i, s, q, W, ch, hist[i]);
    for (int64_t tb = t0; tb < t1; tb += kGroup) {
        typename Raw<T, V>::type raw[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (tb + j < t1) raw[j] = load_raw<T, V, ONCE>((const T*)a.x + (tb + j) * a.p.x_stride + ch);
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
            store_vec<T, V, ONCE>((T*)a.y + t * D + ch, y);
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
// DT: the type of d_y and d_final_state; GT: that of dx and d_initial_state;
// ONCE: x, d_y and dx go past the caches.
template <typename T, typename DT, typename GT, int V, int W, bool SILU, bool ONCE>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvArgs a, int ncb, int64_t ntiles, int run) {
    const int64_t tile = blockIdx.x / ncb;
    const int D = a.p.channels, at = ((int)(blockIdx.x % ncb) * (int)blockDim.x + (int)threadIdx.x) * V;
    const int ch = first_channel<V>(at, D);
    const int64_t t0 = tile * run;
    int q = tile < ntiles ? seq_of_token(a.cu, a.p.num_seqs, a.p.seq_len, t0) : 0;
    if (at >= D) return;
    GT* dxp = (GT*)a.dx;
    GT* dS0 = (GT*)a.dS0;
    const DT* dyp = (const DT*)a.d_y;
    const DT* dST = (const DT*)a.dST;
    if (tile >= ntiles) {                                // empty sequences: d_initial_state = d_final_state
        const int64_t q = tile - ntiles;
        int64_t s, e;
        seq_range(a.cu, (int)q, a.p.seq_len, a.Ttot, &s, &e);
        if (e > s) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t i = (q * (W - 1) + j) * D + ch;
            float f[V] = {};
            if (dST) unpack<DT, V>(load_raw<DT, V>(dST + i), f);
            store_vec<GT, V>(dS0 + i, f);
        }
        return;
    }
    float dw[W][V] = {}, db[V] = {};
    {
        const int64_t t1 = t0 + run < a.Ttot ? t0 + run : a.Ttot;
        Taps<T, V, W> taps;
        taps.load(a, ch);
        int64_t s, e;
        seq_range(a.cu, q, a.p.seq_len, a.Ttot, &s, &e);
        float hist[W - 1][V], dph[W - 1][V];             // rows before the token; dp of the tokens before it
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            load_u<T, V>(a, t0 - (W - 1) + i, s, q, W, ch, hist[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) dph[i][v] = 0.f;
        }
        // du of the position W - 1 before the newest dp
        auto gather = [&](const float (&dp)[V], float (&f)[V]) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[v] = taps.w[0][v] * dp[v];
#pragma unroll
                for (int w = 1; w < W; ++w) f[v] = __builtin_fmaf(taps.w[w][v], dph[W - 1 - w][v], f[v]);
            }
        };
        auto finish = [&](int64_t r, const float (&dp)[V]) {
            const bool mine = r >= s ? (r >= t0 && r < t1) : (r >= s - (W - 1) && s >= t0 && s < t1 && dS0 != nullptr);
            if (!mine) return;
            float f[V];
            gather(dp, f);
            if (dST && r >= e - (W - 1)) {
                float g[V];
                unpack<DT, V>(load_raw<DT, V>(dST + ((int64_t)q * (W - 1) + (r - (e - (W - 1)))) * D + ch), g);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] += g[v];
            }
            if (r >= s) store_vec<GT, V>(dxp + r * D + ch, f);
            else store_vec<GT, V>(dS0 + ((int64_t)q * (W - 1) + (r - s + W - 1)) * D + ch, f);
        };
        auto token = [&](const typename Raw<T, V>::type& rx, const typename Raw<DT, V>::type& rdy, bool own,
                         auto done) {
            float x[V], dp[V];
            unpack<T, V>(rx, x);
            unpack<DT, V>(rdy, dp);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (SILU) dp[v] *= silu_grad(taps.at(hist, x, v));
                if (own) {
#pragma unroll
                    for (int w = 0; w < W - 1; ++w) dw[w][v] = __builtin_fmaf(dp[v], hist[w][v], dw[w][v]);
                    dw[W - 1][v] = __builtin_fmaf(dp[v], x[v], dw[W - 1][v]);
                    db[v] += dp[v];
                }
            }
            done(dp);
            push<W, V>(hist, x);
            push<W, V>(dph, dp);
        };
        const T* xp = (const T*)a.x + ch;
        int64_t t = t0;
        while (true) {
            if (t >= e) {                                // the sequence has ended: its last W - 1 positions
                float zero[V] = {};
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    finish(e - (W - 1) + i, zero);
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
            typename Raw<T, V>::type rx[kGroup];
            typename Raw<DT, V>::type rdy[kGroup];
            // away from the ends of the run and of its sequence no token needs a decision, and a group's rows are
            // loaded while the group before it is worked on
            auto inside = [&](int64_t t) {
                return t - (W - 1) >= (s > t0 ? s : t0) && t + kGroup <= (e < t1 ? e : t1);
            };
            if (inside(t)) {
                auto load = [&](int64_t t) {
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) {
                        rx[j] = load_raw<T, V, ONCE>(xp + (t + j) * a.p.x_stride);
                        rdy[j] = load_raw<DT, V, ONCE>(dyp + (t + j) * D + ch);
                    }
                };
                load(t);
                bool more;
                do {
                    typename Raw<T, V>::type cx[kGroup];
                    typename Raw<DT, V>::type cdy[kGroup];
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) {
                        cx[j] = rx[j];
                        cdy[j] = rdy[j];
                    }
                    more = inside(t + kGroup);
                    if (more) load(t + kGroup);
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
                        token(cx[j], cdy[j], true, [&](const float (&dp)[V]) {
                            float f[V];
                            gather(dp, f);
                            store_vec<GT, V, ONCE>(dxp + (t + j - (W - 1)) * D + ch, f);
                        });
                    t += kGroup;
                } while (more);
                continue;
            }
            const int m = (int)(stop - t < kGroup ? stop - t : kGroup);
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (j < m) {
                    rx[j] = load_raw<T, V>(xp + (t + j) * a.p.x_stride);
                    rdy[j] = load_raw<DT, V>(dyp + (t + j) * D + ch);
                }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (j >= m) break;
                token(rx[j], rdy[j], t + j < t1, [&](const float (&dp)[V]) { finish(t + j - (W - 1), dp); });
            }
            t += m;
        }
    }
    float* part = a.partial + tile * (W + 1) * D + ch;
#pragma unroll
    for (int w = 0; w < W; ++w) store_vec<float, V>(part + (int64_t)w * D, dw[w]);
    store_vec<float, V>(part + (int64_t)W * D, db);
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

// f(io type, elements a lane moves at once, taps); VB of them for bf16
template <int VB, typename F>
hipError_t by_type(const ConvArgs& a, bool wide, F f) {
    auto by_width = [&](auto type, auto vec) {
        switch (a.p.width) {
            case 2: return f(type, vec, std::integral_constant<int, 2>{});
            case 3: return f(type, vec, std::integral_constant<int, 3>{});
            case 4: return f(type, vec, std::integral_constant<int, 4>{});
        }
        return hipErrorInvalidValue;
    };
    if (a.p.io_dtype == GDR_BF16)
        return wide ? by_width(bf16{}, std::integral_constant<int, VB>{}) : by_width(bf16{}, std::integral_constant<int, 1>{});
    return wide ? by_width(float{}, std::integral_constant<int, 4>{}) : by_width(float{}, std::integral_constant<int, 1>{});
}

int channel_blocks(const ConvArgs& a, int V) { return (a.p.channels + 64 * V - 1) / (64 * V); }
int64_t seq_tiles(const ConvArgs& a) { return ((int64_t)a.p.num_seqs + kWaves - 1) / kWaves; }
int bwd_run(int64_t Ttot, int32_t channels) { return run_length(Ttot, (channels + 64 * kBwdV - 1) / (64 * kBwdV), 128); }

}  // namespace

int64_t conv_bwd_tiles(int64_t Ttot, int32_t channels) {
    const int run = bwd_run(Ttot, channels);
    return (Ttot + run - 1) / run;
}

hipError_t launch_conv_fwd(const ConvArgs& a) {
    return by_type<kFwdV>(a, a.p.channels >= kFwdV, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int ncb = channel_blocks(a, V), run = run_length(a.Ttot, ncb, 64);
        const int64_t ntiles = (a.Ttot + run * kWaves - 1) / (run * kWaves), all = ntiles + (a.ST ? seq_tiles(a) : 0);
        if (!grid_fits(all * ncb, 256)) return hipErrorInvalidConfiguration;
        if (all == 0) return hipSuccess;
        const dim3 grid((unsigned)(all * ncb));
        // (65,536 x 8,192 bf16: 387 us against 417; x alone 438, y alone 404)
        if (beyond_caches(2 * a.Ttot * a.p.channels * size_of(a.p.io_dtype)))
            k_conv_fwd<T, V, W, true><<<grid, 256, 0, a.stream>>>(a, ncb, ntiles, run);
        else k_conv_fwd<T, V, W, false><<<grid, 256, 0, a.stream>>>(a, ncb, ntiles, run);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(const ConvArgs& a) {
    // the state changes in place, so no two lanes may hold the same channel
    const bool wide = a.p.channels % (a.p.io_dtype == GDR_BF16 ? kFwdV : 4) == 0;
    return by_type<kFwdV>(a, wide, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int ncb = channel_blocks(a, V);
        if (!grid_fits(seq_tiles(a) * ncb, 256)) return hipErrorInvalidConfiguration;
        if (seq_tiles(a) > 0) k_conv_step<T, V, W><<<dim3((unsigned)(seq_tiles(a) * ncb)), 256, 0, a.stream>>>(a, ncb);
        return hipGetLastError();
    });
}

hipError_t launch_conv_bwd(const ConvArgs& a) {
    const int64_t ntiles = conv_bwd_tiles(a.Ttot, a.p.channels);
    const int run = bwd_run(a.Ttot, a.p.channels);
    hipError_t e = by_type<kBwdV>(a, a.p.channels >= kBwdV, [&](auto type, auto vec, auto width) {
        typedef decltype(type) T;
        constexpr int V = decltype(vec)::value, W = decltype(width)::value;
        const int cbs = channel_blocks(a, V), nw = cbs < kWaves ? cbs : kWaves, ncb = (cbs + nw - 1) / nw;
        const int64_t all = ntiles + (a.dS0 ? a.p.num_seqs : 0);
        if (!grid_fits(all * ncb, 256)) return hipErrorInvalidConfiguration;
        if (all == 0) return hipSuccess;
        const dim3 grid((unsigned)(all * ncb));
        auto go = [&](auto dtype, auto gtype, auto silu_on) {
            typedef decltype(dtype) DT;
            typedef decltype(gtype) GT;
            constexpr bool SILU = decltype(silu_on)::value;
            // (16,384 x 6,144 bf16: 126 us against 138, the reads alone 135, dx alone 134; what the caches hold is 5 %
            // faster from them)
            if (beyond_caches(a.Ttot * a.p.channels * (int64_t)(sizeof(T) + sizeof(DT) + sizeof(GT))))
                k_conv_bwd<T, DT, GT, V, W, SILU, true><<<grid, 64 * nw, 0, a.stream>>>(a, ncb, ntiles, run);
            else k_conv_bwd<T, DT, GT, V, W, SILU, false><<<grid, 64 * nw, 0, a.stream>>>(a, ncb, ntiles, run);
        };
        auto by_dy = [&](auto gtype, auto silu_on) {
            a.p.dy_dtype == GDR_F32 ? go(float{}, gtype, silu_on) : go(T{}, gtype, silu_on);
        };
        auto by_grad = [&](auto silu_on) { a.p.grad_dtype == GDR_F32 ? by_dy(float{}, silu_on) : by_dy(T{}, silu_on); };
        if (a.p.activation == GDR_ACT_SILU) by_grad(std::true_type{});
        else by_grad(std::false_type{});
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const int D = a.p.channels, W = a.p.width;
    return sum_partials(a.partial, ntiles, (int64_t)(W + 1) * D, ConvGradOut{a.dweight, a.dbias, D, W}, a.stream);
}

}  // namespace gdr
