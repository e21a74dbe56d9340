// Window attention, forward (include/gdr_attn.h; tile conventions in gdr_attn.hpp).
#include <type_traits>

#include "gdr_attn.hpp"

namespace gdr {

namespace {

// ---------------------------------------------------------------- softmax over tiles
// What a lane keeps of its query: the output's dims 32 t + 8 i + 4 h + j in o[t][4 i + j],
// the raw score m that the weights refer to and its product mc with c = scale log2(e) as
// it was rounded, and its half's sum of the weights. Weights and sums share the rounding
// of mc, so that it cancels in o.
template <int DV>
struct State {
    f32x16 o[DV / 32];
    float m, mc, l;
    __device__ void clear() {
#pragma unroll
        for (int t = 0; t < DV / 32; ++t) o[t] = zero16();
        m = mc = kNegInf;
        l = 0.f;
    }
};
// the factor from sums that refer to a to sums that refer to b >= a (either may be -inf)
__device__ __forceinline__ float refer(float a, float b) { return a == b ? 1.f : __builtin_amdgcn_exp2f(a - b); }

// Whether a tile of N elements holds Inf or NaN, by a wavefront
template <typename T, int N>
__device__ __forceinline__ bool any_special(const T* tile) {
    uint32_t top = 0;
#pragma unroll 4
    for (int i = (int)(threadIdx.x & 63) * kUnit<T>; i < N; i += 64 * kUnit<T>) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(tile + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // without their signs; two elements of 16 bits compare as the upper halves do
            const uint32_t a = x[e] & 0x7fffffffu, b = sizeof(T) == 2 ? x[e] << 16 & 0x7fffffffu : 0u;
            top = top > a ? top : a;
            top = top > b ? top : b;
        }
    }
    return __any(top >= 0x7f800000u);
}

// A weight of zero does not stop an infinite or NaN v. Copies a tile of ROWS rows with
// zeros for such elements (`to` may be `from`), by a wavefront, and returns the keys
// that had one: the lane's key 8 i + 4 h + j of subtile k in bit 16 k + 4 i + j.
template <typename T, int D, int ROWS>
__device__ __forceinline__ uint32_t copy_finite(const T* from, T* to) {
    constexpr int UN = D / kUnit<T>;                       // units (lanes) to a row
    static_assert(UN <= 64 && 64 % UN == 0, "whole rows a step");
    const int lane = threadIdx.x & 63, h = lane >> 5;
    uint32_t lost = 0;
#pragma unroll 1
    for (int r0 = 0; r0 < ROWS; r0 += 64 / UN) {
        typename Raw<T, kUnit<T>>::type x = load_raw<T, kUnit<T>>(from + (r0 * UN + lane) * kUnit<T>);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) {
            const bool ok = fabsf(to_f(x[e])) < __builtin_inff();
            bad |= !ok;
            x[e] = ok ? x[e] : to_t<T>(0.f);
        }
        store_raw<T, kUnit<T>>(to + (r0 * UN + lane) * kUnit<T>, x);
        const uint64_t who = __ballot(bad);
#pragma unroll
        for (int k = 0; k < 64 / UN; ++k) {
            const int key = r0 + k;
            if ((who >> (k * UN)) << (64 - UN) && (key >> 2 & 1) == h)
                lost |= 1u << (16 * (key >> 5) + 4 * (key >> 3 & 3) + (key & 3));
        }
    }
    return lost;
}

// One tile of 32 NT keys, whose raw scores are s (overwritten by the weights) and
// whose values lie in V. partial: some query may not see some key; the values are then
// copied to `clean` first.
//
// Weights are exp2(c s - mc). m follows the maximum only when that has grown by more
// than 8 in the exponent: weights then stay below 2^9 and the sums, in fp32, hardly
// notice, while most tiles are spared the product of o with the change. Beyond 2^24 the
// rounding of mc reaches the exponent's units, and the difference is formed first.
template <typename T, int DV, int NT>
__device__ __forceinline__ void absorb(State<DV>& st, f32x16 (&s)[NT], const T* V, T* clean, float c,
                                       bool partial, const Sight& sees) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int co = fresh(col_offset<T, DV>(lane));
    if (partial) {
        asm volatile("");                                  // a branch: most tiles are seen whole
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[k][i] = sees(32 * k + 8 * (i >> 2) + 4 * h + (i & 3)) ? s[k][i] : kNegInf;
    }
    float top = s[0][0];
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_elementwise_maximum(top, s[k][i]);
    top = pair_max(top);
    if (__any((top - st.m) * c > 8.f)) {
        const float m = fmaxf(st.m, top), mc = m * c, f = refer(st.mc, mc);
        st.l *= f;
#pragma unroll
        for (int t = 0; t < DV / 32; ++t) st.o[t] = st.o[t] * f;
        st.m = m;
        st.mc = mc;
    }
    const float mc = st.m == kNegInf ? 0.f : st.mc;
    if (__any(fabsf(mc) > 16777216.f)) {
        const float m = st.m == kNegInf ? 0.f : st.m;
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k][i] = __builtin_amdgcn_exp2f((s[k][i] - m) * c);
    } else {
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i], c, -mc));
    }
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) st.l += s[k][i];
    if (partial && any_special<T, 32 * NT * DV>(V)) {
        const uint32_t lost = copy_finite<T, DV, 32 * NT>(V, clean);
        if (lost) {                                        // who sees such a key loses its sum
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if ((lost >> (16 * k + i) & 1) && sees(32 * k + 8 * (i >> 2) + 4 * h + (i & 3)))
                        st.l = __builtin_nanf("");
        }
        V = clean;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const auto w = acc_frag<T>(s[k], q);
#pragma unroll
            for (int t = 0; t < DV / 32; ++t) st.o[t] = mma(col_frag<DV>(V, 32 * k + 16 * q, t, co), w, st.o[t]);
        }
}

template <typename T, int DK, bool VEC>
__device__ __forceinline__ void load_query(const AttnArgs& a, const Query& q, frag_t<T> (&x)[DK / (2 * kUnit<T>)]) {
    const T* row = (const T*)a.q + q.token * a.p.q_stride + (int64_t)q.head * a.p.head_dim_qk;
#pragma unroll
    for (int t = 0; t < DK / (2 * kUnit<T>); ++t)
        x[t] = load_frag_row<T, VEC>(row, 2 * t + ((threadIdx.x >> 5) & 1), a.p.head_dim_qk, q.live);
}

template <typename T, int DV>
__device__ __forceinline__ void store_rows(const AttnArgs& a, const Query& q, const State<DV>& st, float l) {
    if (!q.live) return;
    const int h = (threadIdx.x >> 5) & 1, dv = a.p.head_dim_v;
    const int64_t row = q.token * a.p.num_q_heads + q.head;
    const float inv = 1.f / l;
#pragma unroll
    for (int t = 0; t < DV / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = st.o[t][4 * i + j] * inv;
            const int d = 32 * t + 8 * i + 4 * h;
            if (a.p.out_dtype == GDR_F32) store4((float*)a.o + row * dv, d, dv, y);
            else store4((T*)a.o + row * dv, d, dv, y);
        }
    if (a.lse && h == 0)
        a.lse[row] = (st.mc + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---------------------------------------------------------------- many rows
// A workgroup of NW wavefronts takes 32 NW rows (tokens times heads of one key head)
// and walks the keys they see in tiles of KT, keys and values in LDS, two tiles in
// turn; the next tile's loads are under way during a tile's products.
template <typename T> constexpr int kTileKeys = sizeof(T) == 2 ? 64 : 32;

template <typename T, int DK, int DV, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, 2) void k_window_rows(AttnArgs a, RowBlock rb, int nblk, int nwork) {
    constexpr int KT = kTileKeys<T>, NT = KT / 32, KF = DK / (2 * kUnit<T>);
    __shared__ __attribute__((aligned(16))) T K0[KT * DK], K1[KT * DK], V0[KT * DV], V1[KT * DV];
    // the finite values of a tile at an edge: all wavefronts that need it write the same
    __shared__ __attribute__((aligned(16))) T Clean[KT * DV];
    // consecutive blocks of a key head on one XCD: their windows overlap
    const int per = (nwork + 7) / 8, id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= nwork) return;
    const int hh = id / nblk, G = a.p.num_q_heads / a.p.num_kv_heads, hk = hh / rb.HC, hc = hh % rb.HC;
    Block b;
    if (!find_block(a.cu, a.p.num_seqs, a.p.seq_len, a.Ttot, rb.TPB, id % nblk, &b)) return;
    const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
    const int len = past_len(a, b.n), W = a.p.window, S = a.p.sinks;
    const int dk = a.p.head_dim_qk, dv = a.p.head_dim_v;
    const Query q = query_of(b, rb, G, hk, hc, 32 * w + (lane & 31), len);
    // first and last position of this wavefront's queries
    const int pa = __builtin_amdgcn_readlane(q.p, 0), pb = __builtin_amdgcn_readlane(q.p, 31);
    frag_t<T> qf[KF];
    load_query<T, DK, VEC>(a, q, qf);
    State<DV> st;
    st.clear();
    const float c = a.p.scale * kLog2e;

    Keys keys(len + b.t0, len + b.t0 + b.tn - 1, len, W, S);
    Copy<T, DK, KT, 64 * NW, VEC> ck;
    Copy<T, DV, KT, 64 * NW, VEC> cv;
    int pos, cnt, row;
    bool cached;
    auto fetch = [&](T* K, T* V) {
        keys.next(KT, &pos, &cnt, &row, &cached);
        if (cnt == 0) return;
        const Source<T> s = source<T>(a, b, hk, row, cached);
        ck.start(K, s.k, s.kld, cnt, dk, tid);
        cv.start(V, s.v, s.vld, cnt, dv, tid);
    };
    auto land = [&](T* K, T* V) {
        if (cnt > 0) {
            ck.finish(K, tid);
            cv.finish(V, tid);
        }
        __syncthreads();
    };
    // a tile in (K, V), the next one on its way to (Kn, Vn)
    auto turn = [&](const T* K, const T* V, T* Kn, T* Vn) {
        const int pos0 = pos, n = cnt, ro = fresh(row_offset<T, DK>(lane));
        fetch(Kn, Vn);
        // some query of this wavefront sees a key of the tile
        if (pos0 <= pb && (pos0 < S || pos0 + n - 1 > pa - W)) {
            f32x16 s[NT];
#pragma unroll
            for (int k = 0; k < NT; ++k) s[k] = zero16();
#pragma unroll
            for (int t = 0; t < KF; ++t)
#pragma unroll
                for (int k = 0; k < NT; ++k) s[k] = mma(row_frag<T, DK>(K, 32 * k, t, ro), qf[t], s[k]);
            const bool partial = n < KT || pos0 + KT - 1 > pa || (pos0 <= pb - W && pos0 + KT > S);
            absorb<T, DV, NT>(st, s, V, Clean, c, partial, Sight{pos0, n, q.p, W, S});
        }
        land(Kn, Vn);
    };
    fetch(K0, V0);
    land(K0, V0);
    while (cnt > 0) {
        turn(K0, V0, K1, V1);
        if (cnt == 0) break;
        turn(K1, V1, K0, V0);
    }
    store_rows<T, DV>(a, q, st, pair_sum(st.l));
}

// ---------------------------------------------------------------- few rows
// 32 rows a workgroup (a token's heads of one key head, when decoding): its NW
// wavefronts, and `splits` workgroups, share the keys. A wavefront takes 32 keys at a
// time straight into the operand's registers, the values through LDS of its own; the
// next 32 are under way meanwhile. What they have summed is joined in LDS, the
// workgroups' by k_window_join.
template <typename T, int DK, int DV, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_window_split(AttnArgs a, RowBlock rb, int nblk, int splits) {
    constexpr int KF = DK / (2 * kUnit<T>);
    __shared__ __attribute__((aligned(16))) T Vs[NW][32 * DV];
    __shared__ float ml[NW][2][32];
    static_assert(32 * DV * sizeof(T) >= 32 * 32 * 4, "a wavefront's values make room for a tile of its outputs");
    const int sp = blockIdx.x % splits, id = blockIdx.x / splits;
    const int hh = id % (a.p.num_kv_heads * rb.HC), G = a.p.num_q_heads / a.p.num_kv_heads;
    const int hk = hh / rb.HC, hc = hh % rb.HC;
    Block b;
    if (!find_block(a.cu, a.p.num_seqs, a.p.seq_len, a.Ttot, rb.TPB, id / (a.p.num_kv_heads * rb.HC), &b)) return;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int W = a.p.window, S = a.p.sinks, dk = a.p.head_dim_qk, dv = a.p.head_dim_v;
    const int len = past_len(a, b.n);
    const Query q = query_of(b, rb, G, hk, hc, lane & 31, len);
    const bool idle = a.one && __builtin_amdgcn_readfirstlane(a.lens[b.n]) < 0;
    if (a.one && !idle && hc == 0 && sp == 0) {
        // the token's row in the caches held one that no query sees any more
        const int64_t at = (int64_t)b.n * ((int64_t)S + W) + (len < S ? len : S + (len - S) % W);
        const Source<T> s = source<T>(a, b, hk, 0, false);
        for (int d = tid; d < dk; d += 64 * NW) ((T*)a.kc)[(at * a.p.num_kv_heads + hk) * dk + d] = s.k[d];
        for (int d = tid; d < dv; d += 64 * NW) ((T*)a.vc)[(at * a.p.num_kv_heads + hk) * dv + d] = s.v[d];
    }
    const int pa = __builtin_amdgcn_readlane(q.p, 0), pb = __builtin_amdgcn_readlane(q.p, 31);
    State<DV> st;
    st.clear();
    const float c = a.p.scale * kLog2e;
    Keys keys(len + b.t0, len + b.t0 + b.tn - 1, len, W, S);
    // this wavefront's share of the keys, in tiles
    const int all = keys.total(), parts = splits * NW, part = sp * NW + w;
    const int share = ((all + parts - 1) / parts + 31) / 32 * 32;
    int64_t first = (int64_t)share * part;
    int left = idle || first >= all ? 0 : (int)(all - first < share ? all - first : share);
    if (left > 0) keys.skip((int)first);
    if (left > 0) {
        frag_t<T> qf[KF], kf[KF];
        load_query<T, DK, VEC>(a, q, qf);
        OwnCopy<T, DV, 32, VEC> sv;
        int pos = 0, cnt = 0, row = 0;
        bool cached = false;
        auto next = [&] {
            cnt = 0;
            if (left <= 0) return;
            keys.next(left < 32 ? left : 32, &pos, &cnt, &row, &cached);
            left -= cnt;
        };
        auto load_keys = [&] {
            const Source<T> s = source<T>(a, b, hk, row, cached);
            const uint32_t row_bytes = (uint32_t)s.kld * sizeof(T);
            const auto rs = buf_rsrc(s.k, cnt > 0 ? (cnt - 1) * row_bytes + dk * (uint32_t)sizeof(T) : 0);
#pragma unroll
            for (int t = 0; t < KF; ++t)
                kf[t] = __builtin_bit_cast(frag_t<T>, load_unit<T, VEC>(rs, (lane & 31) * (int)row_bytes,
                                                                        2 * t + (lane >> 5), dk));
        };
        auto load_values = [&] {
            const Source<T> s = source<T>(a, b, hk, row, cached);
            sv.load(s.v, s.vld, cnt, dv);
        };
        next();
        load_keys();
        load_values();
        while (cnt > 0) {
            const int pos0 = pos, n = cnt;
            sv.store(Vs[w]);
            next();
            load_values();
            f32x16 s[1] = {zero16()};
#pragma unroll
            for (int t = 0; t < KF; ++t) s[0] = mma(kf[t], qf[t], s[0]);
            load_keys();
            const bool partial = n < 32 || pos0 + 31 > pa || (pos0 <= pb - W && pos0 + 32 > S);
            absorb<T, DV, 1>(st, s, Vs[w], Vs[w], c, partial, Sight{pos0, n, q.p, W, S});
        }
    }
    // join the wavefronts: a common maximum, then one tile of 32 dims after another
    st.l = pair_sum(st.l);
    if (lane < 32) {
        ml[w][0][lane] = st.mc;
        ml[w][1][lane] = st.l;
    }
    __syncthreads();
    float m = kNegInf, l = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) m = fmaxf(m, ml[i][0][lane & 31]);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const float mi = ml[i][0][lane & 31], li = ml[i][1][lane & 31];
        l += li * refer(mi, m);
    }
    const float f = refer(st.mc, m);
    const int64_t row = q.token * a.p.num_q_heads + q.head, rows = a.Ttot * a.p.num_q_heads;
    const int h = lane >> 5;
    float* part_o = a.ws + (int64_t)sp * rows * (dv + 2);
    const float inv = idle ? 0.f : 1.f / l;
#pragma unroll
    for (int t = 0; t < DV / 32; ++t) {
        float* mine = reinterpret_cast<float*>(Vs[w]);
        if (t > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[i * 64 + lane] = st.o[t][i] * f;
        __syncthreads();
        // register i of all wavefronts: 16 registers, NW wavefronts
#pragma unroll
        for (int i0 = 0; i0 < 16; i0 += NW) {
            const int i = i0 + w;
            if (i >= 16) break;
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) y += reinterpret_cast<const float*>(Vs[k])[i * 64 + lane];
            const int d = 32 * t + 8 * (i >> 2) + 4 * h + (i & 3);
            if (!q.live || d >= dv) continue;
            if (splits > 1) part_o[row * (dv + 2) + d] = y;
            else store_as<T>(a.o, row * dv + d, idle ? 0.f : y * inv, a.p.out_dtype == GDR_F32);
        }
    }
    if (w == 0 && h == 0 && q.live) {
        if (splits > 1) {
            part_o[row * (dv + 2) + dv] = idle ? 0.f : m;
            part_o[row * (dv + 2) + dv + 1] = idle ? -1.f : l;
        } else if (a.lse) {
            a.lse[row] = (m + __builtin_amdgcn_logf(l)) * kLn2;
        }
    }
}

// o and lse of a row from the parts of `splits` workgroups, 64 lanes a row. A part's
// sum of -1 marks a sequence that was passed over.
template <typename T>
__global__ __launch_bounds__(256) void k_window_join(AttnArgs a, int splits) {
    const int64_t rows = a.Ttot * a.p.num_q_heads, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= rows) return;
    const int dv = a.p.head_dim_v, lane = threadIdx.x & 63;
    const float* part = a.ws + row * (dv + 2);
    const int64_t step = rows * (dv + 2);
    float m = kNegInf, l = 0.f, y[2] = {0.f, 0.f};
    const bool idle = part[dv + 1] < 0.f;
    for (int i = 0; i < splits; ++i) m = fmaxf(m, part[i * step + dv]);
    for (int i = 0; i < splits; ++i) {
        const float mi = part[i * step + dv], f = refer(mi, m);
        l = __builtin_fmaf(part[i * step + dv + 1], f, l);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (lane + 64 * j < dv) y[j] = __builtin_fmaf(part[i * step + lane + 64 * j], f, y[j]);
    }
    const float inv = idle ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 64 * j < dv)
            store_as<T>(a.o, row * dv + lane + 64 * j, idle ? 0.f : y[j] * inv, a.p.out_dtype == GDR_F32);
    if (a.lse && lane == 0) a.lse[row] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---------------------------------------------------------------- the new tokens into the caches
// After the attention has read them, a wavefront a token: the sinks, and the last
// `window` of a sequence's other tokens.
template <typename T, bool VEC>
__device__ __forceinline__ void copy_row(T* to, const T* from, int n) {
    const int lane = threadIdx.x & 63;
    if constexpr (VEC) {
        for (int i = lane * kUnit<T>; i < n; i += 64 * kUnit<T>)
            *reinterpret_cast<u32x4*>(to + i) = *reinterpret_cast<const u32x4*>(from + i);
    } else {
        for (int i = lane; i < n; i += 64) to[i] = from[i];
    }
}
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_window_keep(AttnArgs a) {
    const int W = a.p.window, S = a.p.sinks, Nk = a.p.num_kv_heads;
    const int kw = Nk * a.p.head_dim_qk, vw = Nk * a.p.head_dim_v;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.Ttot; t += (int64_t)gridDim.x * 4) {
        const int n = seq_of_token(a.cu, a.p.num_seqs, a.p.seq_len, t);
        int64_t s, e;
        seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
        if (t < s || t >= e) continue;
        const int len = past_len(a, n), p = len + (int)(t - s);
        if (p >= S && e - t > W) continue;
        const int64_t at = (int64_t)n * ((int64_t)S + W) + (p < S ? p : S + (p - S) % W);
        copy_row<T, VEC>((T*)a.kc + at * kw, (const T*)a.k + t * a.p.k_stride, kw);
        copy_row<T, VEC>((T*)a.vc + at * vw, (const T*)a.v + t * a.p.v_stride, vw);
    }
}

// ---------------------------------------------------------------- launches
// Whether 32 rows a workgroup, its wavefronts sharing the keys, or 32 rows a wavefront
struct Plan {
    bool split;
    int NW, splits;
    RowBlock rb;
    int64_t nblk, nwork;
};
Plan plan_of(const gdr_attn_problem_t& p) {
    Plan x{};
    const int G = group(p);
    const bool packed = p.batch == 1 && p.num_seqs != 1;
    const int64_t rows = p.batch * p.seq_len * p.num_q_heads;
    const int64_t keys = (int64_t)p.sinks + p.window;
    // 32-row blocks of all heads, if none were shared out further
    x.rb = row_block(32, G);
    const int64_t few = token_blocks(p.batch, p.seq_len, p.num_seqs, packed, x.rb.TPB) * p.num_kv_heads * x.rb.HC;
    x.split = rows <= 32 * 1024;
    if (p.seq_len == 1 && !packed) x.split = true;
    if (x.split) {
        x.NW = p.io_dtype == GDR_BF16 ? 8 : 4;
        x.nblk = few / (p.num_kv_heads * x.rb.HC);
        x.nwork = few;
        const int64_t want = few > 0 ? 512 / few : 1, most = (keys + 32 * x.NW - 1) / (32 * x.NW);
        const int64_t s = want < most ? want : most;
        x.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
        return x;
    }
    x.NW = 8;
    x.splits = 1;
    x.rb = row_block(32 * x.NW, G);
    x.nblk = token_blocks(p.batch, p.seq_len, p.num_seqs, packed, x.rb.TPB);
    x.nwork = x.nblk * p.num_kv_heads * x.rb.HC;
    return x;
}

}  // namespace

size_t attn_fwd_workspace(const gdr_attn_problem_t& p) {
    const Plan x = plan_of(p);
    if (x.splits <= 1) return 0;
    return (size_t)x.splits * p.batch * p.seq_len * p.num_q_heads * (p.head_dim_v + 2) * 4;
}

hipError_t launch_attn_fwd(const AttnArgs& a) {
    if (a.Ttot == 0) return hipSuccess;
    const Plan x = plan_of(a.p);
    if (x.nwork >= (int64_t)1 << 31 || !grid_fits(x.nwork * x.splits + 8, 64 * x.NW)) return hipErrorInvalidConfiguration;
    hipError_t e = hipSuccess;
    by_dims(a.p, [&](auto type, auto dk, auto dv) {
        typedef decltype(type) T;
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, NWS = sizeof(T) == 2 ? 8 : 4;
        if (x.split) {
            const dim3 grid((unsigned)(x.nwork * x.splits));
            if (a.vec) k_window_split<T, DK, DV, NWS, true><<<grid, 64 * NWS, 0, a.stream>>>(a, x.rb, (int)x.nblk, x.splits);
            else k_window_split<T, DK, DV, NWS, false><<<grid, 64 * NWS, 0, a.stream>>>(a, x.rb, (int)x.nblk, x.splits);
            if (x.splits > 1) {
                const int64_t rows = a.Ttot * a.p.num_q_heads;
                k_window_join<T><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, a.stream>>>(a, x.splits);
            }
        } else {
            const dim3 grid((unsigned)((x.nwork + 7) / 8 * 8));
            if (a.vec) k_window_rows<T, DK, DV, 8, true><<<grid, 512, 0, a.stream>>>(a, x.rb, (int)x.nblk, (int)x.nwork);
            else k_window_rows<T, DK, DV, 8, false><<<grid, 512, 0, a.stream>>>(a, x.rb, (int)x.nblk, (int)x.nwork);
        }
        e = hipGetLastError();
        if (e == hipSuccess && a.kc && !a.one) {
            const int64_t need = (a.Ttot + 3) / 4, most = 8192;
            const dim3 grid((unsigned)(need < most ? need : most));
            if (a.vec) k_window_keep<T, true><<<grid, 256, 0, a.stream>>>(a);
            else k_window_keep<T, false><<<grid, 256, 0, a.stream>>>(a);
            e = hipGetLastError();
        }
    });
    return e;
}

}  // namespace gdr
