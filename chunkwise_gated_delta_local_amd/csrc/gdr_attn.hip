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
__device__ __forceinline__ bool any_special(lds_c tile) {
    uint32_t top = 0;
#pragma unroll 4
    for (int i = (int)(threadIdx.x & 63) * 16; i < N * (int)sizeof(T); i += 1024) {
        const u32x4 x = *(lds_p<u32x4>)(tile + i);
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
__device__ __forceinline__ uint32_t copy_finite(lds_c from, lds_c to) {
    constexpr int UN = D / kUnit<T>;                       // units (lanes) to a row
    static_assert(UN <= 64 && 64 % UN == 0, "whole rows a step");
    const int lane = threadIdx.x & 63, h = lane >> 5;
    uint32_t lost = 0;
#pragma unroll 1
    for (int r0 = 0; r0 < ROWS; r0 += 64 / UN) {
        auto x = __builtin_bit_cast(typename Raw<T, kUnit<T>>::type, *(lds_p<u32x4>)(from + (r0 * UN + lane) * 16));
        bool bad = false;
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) {
            const bool ok = fabsf(to_f(x[e])) < __builtin_inff();
            bad |= !ok;
            x[e] = ok ? x[e] : to_t<T>(0.f);
        }
        *(lds_p<u32x4>)(to + (r0 * UN + lane) * 16) = __builtin_bit_cast(u32x4, x);
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

// The weights of one tile of 32 NT keys, whose raw scores are s, in their place.
// partial: some query may not see some key.
//
// Weights are exp2(c s - mc). m follows the maximum only when that has grown by more
// than 8 in the exponent: weights then stay below 2^9 and the sums, in fp32, hardly
// notice, while most tiles are spared the product of o with the change. Beyond 2^24 the
// rounding of mc reaches the exponent's units, and the difference is formed first. Both are
// a query's own choice: what the others of its wavefront score does not change its bits.
template <int DV, int NT>
__device__ __forceinline__ void weigh(State<DV>& st, f32x16 (&s)[NT], float c, bool partial, const Sight& sees) {
    const int h = (threadIdx.x >> 5) & 1;
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
    const bool grown = (top - st.m) * c > 8.f;
    if (__any(grown)) {
        const float m = grown ? top : st.m, mc = grown ? m * c : st.mc, f = grown ? refer(st.mc, mc) : 1.f;
        st.l *= f;
#pragma unroll
        for (int t = 0; t < DV / 32; ++t) st.o[t] = st.o[t] * f;
        st.m = m;
        st.mc = mc;
        arrived(st.o);
    }
    float mc = st.m == kNegInf ? 0.f : st.mc;
    const bool far = fabsf(mc) > 16777216.f;
    if (__any(far)) {
        asm volatile("");
        const float m = far ? st.m : 0.f;
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k][i] -= m;
        mc = far ? 0.f : mc;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i], c, -mc));
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) st.l += s[k][i];
}

// o += V^T P: a tile's values in V, its weights packed in w. Where some query may not see
// some key, values with Inf or NaN are copied to `clean` first.
template <typename T, int DV, int NT>
__device__ __forceinline__ void add_values(State<DV>& st, const typename Vec<T>::v8 (&w)[2 * NT], lds_c V, lds_c clean,
                                           bool partial, const Sight& sees) {
    const int lane = threadIdx.x & 63, h = lane >> 5, co = fresh(col_offset<T, DV>(lane));
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
    for (int q = 0; q < 2 * NT; ++q)
#pragma unroll
        for (int t = 0; t < DV / 32; ++t) st.o[t] = mma(col_frag<T, DV>(V, 16 * q, t, co), w[q], st.o[t]);
    arrived(st.o);
    feed<2 * NT * DV / 32, sizeof(T) == 2 ? 2 : 8, sizeof(T) == 2 ? 1 : 8>();
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
//
// The matrix cores and the vector operations bound it, a wavefront's one against the
// other's: 65,536 tokens of 32 heads over 8, 128 x 128, window 4,096, take 4.2 ms, 1,010
// TFLOP/s of what is seen, 80 % of a large library product's rate here, with the matrix cores
// busy 54 % of the cycles and 7.6 vector operations to a product of 32 cycles, of which
// the exponentials take four times as long. With dims of 64 a product does half for the
// same exponentials: 65,536 tokens of 16 heads, window 2,048, 708 us, 760 TFLOP/s.
template <typename T, int DK, int DV, int NW, int KT, bool VEC>
__global__ __launch_bounds__(64 * NW, 2) void k_window_rows(AttnArgs a, RowBlock rb, int nblk, int nwork) {
    constexpr int NT = KT / 32, KF = DK / (2 * kUnit<T>);
    __shared__ __attribute__((aligned(16))) T Ks[2][KT * DK], Vs[2][KT * DV];
    // the finite values of a tile at an edge: all wavefronts that need them write the same
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
    const lds_c K0 = lds_of(Ks[0]), K1 = lds_of(Ks[1]), V0 = lds_of(Vs[0]), V1 = lds_of(Vs[1]), clean = lds_of(Clean);

    Keys keys(len + b.t0, len + b.t0 + b.tn - 1, len, W, S);
    Copy<T, DK, KT, 64 * NW, VEC> ck;
    Copy<T, DV, KT, 64 * NW, VEC> cv;
    int pos, cnt, row;
    bool cached;
    auto fetch = [&](lds_c K, lds_c V) {
        keys.next(KT, &pos, &cnt, &row, &cached);
        if (cnt == 0) return;
        const Source<T> s = source<T>(a, b, hk, row, cached);
        ck.start(K, s.k, s.kld, cnt, dk, tid);
        cv.start(V, s.v, s.vld, cnt, dv, tid);
    };
    auto land = [&](lds_c K, lds_c V) {
        if (cnt > 0) {
            ck.finish(K, tid);
            cv.finish(V, tid);
        }
        landed();
    };
    // a tile in (K, V), the next one on its way to (Kn, Vn). Tiles that none of a
    // wavefront's queries sees are few and give weights of zero.
    auto turn = [&](lds_c K, lds_c V, lds_c Kn, lds_c Vn) {
        const int pos0 = pos, n = cnt, ro = fresh(row_offset<T, DK>(lane));
        fetch(Kn, Vn);
        f32x16 s[NT];
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < NT; ++k) s[k] = zero16();
#pragma unroll
        for (int t = 0; t < KF; ++t)
#pragma unroll
            for (int k = 0; k < NT; ++k) s[k] = mma(row_frag<T, DK>(K, 32 * k, t, ro), qf[t], s[k]);
        feed<KF * NT, 1, sizeof(T) == 2 ? 1 : 4>();
        __builtin_amdgcn_s_setprio(0);
        const bool partial = n < KT || pos0 + KT - 1 > pa || (pos0 <= pb - W && pos0 + KT > S);
        const Sight sees{pos0, n, q.p, W, S};
        weigh<DV, NT>(st, s, c, partial, sees);
        __builtin_amdgcn_s_setprio(1);
        typename Vec<T>::v8 wt[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) wt[i] = acc_frag<T>(s[i >> 1], i & 1);
        add_values<T, DV, NT>(st, wt, V, clean, partial, sees);
        __builtin_amdgcn_s_setprio(0);
        land(Kn, Vn);
    };
    fetch(K0, V0);
    arrived(qf);
    land(K0, V0);
    while (cnt > 0) {
        turn(K0, V0, K1, V1);
        if (cnt == 0) break;
        turn(K1, V1, K0, V0);
    }
    store_rows<T, DV>(a, q, st, pair_sum(st.l));
}

// ---------------------------------------------------------------- few rows
// 32 rows a workgroup: its NW wavefronts, and `splits` workgroups, share the keys. A wavefront takes 32 keys at a
// time straight into the operand's registers, the values through LDS of its own; the
// next 32 are under way meanwhile. What they have summed is joined in LDS, the
// workgroups' by k_window_join. The latency of a chain of tiles bounds it: 682 tokens of
// 6 heads, 128 x 128, window 512, take 16 us (fp32 43), where a wavefront of k_window_rows
// walks all keys in 23 (93).
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
    const int pa = __builtin_amdgcn_readlane(q.p, 0), pb = __builtin_amdgcn_readlane(q.p, 31);
    State<DV> st;
    st.clear();
    const float c = a.p.scale * kLog2e;
    Keys keys(len + b.t0, len + b.t0 + b.tn - 1, len, W, S);
    const lds_c mine_v = lds_of(&Vs[0][0]) + w * 32 * DV * (int)sizeof(T);
    // this wavefront's share of the keys, in tiles
    const int all = keys.total(), parts = splits * NW, part = sp * NW + w;
    const int64_t share = (((int64_t)all + parts - 1) / parts + 31) / 32 * 32, first = share * part;
    int left = first >= all ? 0 : (int)(all - first < share ? all - first : share);
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
            sv.store(mine_v);
            next();
            load_values();
            f32x16 s[1] = {zero16()};
#pragma unroll
            for (int t = 0; t < KF; ++t) s[0] = mma(kf[t], qf[t], s[0]);
            load_keys();
            const bool partial = n < 32 || pos0 + 31 > pa || (pos0 <= pb - W && pos0 + 32 > S);
            const Sight sees{pos0, n, q.p, W, S};
            weigh<DV, 1>(st, s, c, partial, sees);
            const typename Vec<T>::v8 wt[2] = {acc_frag<T>(s[0], 0), acc_frag<T>(s[0], 1)};
            add_values<T, DV, 1>(st, wt, mine_v, mine_v, partial, sees);
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
    const float inv = 1.f / l;
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
            else store_as<T>(a.o, row * dv + d, y * inv, a.p.out_dtype == GDR_F32);
        }
    }
    if (w == 0 && h == 0 && q.live) {
        if (splits > 1) {
            part_o[row * (dv + 2) + dv] = m;
            part_o[row * (dv + 2) + dv + 1] = l;
        } else if (a.lse) {
            a.lse[row] = (m + __builtin_amdgcn_logf(l)) * kLn2;
        }
    }
}

// ---------------------------------------------------------------- single tokens
// The token at position p sees the first min(p + 1, sinks + window) rows of its
// sequence's caches, in whatever order, its own row taken from the call. Up to 16 heads
// of a key head are the columns of 16x16 tiles (layouts as in gdr_device.hpp): scores
// transposed, 32 rows of the caches at a time, k straight into the operand's registers,
// v through LDS of the wavefront's own, the next 32 under way meanwhile. NW wavefronts
// and `splits` workgroups share the rows; rows behind the last one are read as the last
// one, with a weight of zero.
//
// The caches' bytes bound it: 128 sequences of 32 heads over 8, 128 x 128, window 4,096, read
// 2.06 GB in 378 us, 5.45 TB/s (a copy reaches 5.92). Tiles of 32x32 with half of their columns
// empty took 404. Few sequences wait for their chain of loads: one of 16 heads over 4, window
// 1,024, takes 14 us, of which a tile's loads are about 2 each.
template <typename T, int D> struct StepTile {
    static constexpr int UN = D / kUnit<T>;
    // v's rows in LDS, so that the operand's reads spread over the banks
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (sizeof(T) == 4) return (row >> 2 & 3) << 2;
        else if constexpr (UN == 8) return (row >> 1 & 3) << 1;
        else return (row & 7) << 1;
    }
    // dims 16 t + lane % 16 of rows 4 qd + j and 16 + 4 qd + j
    static __device__ __forceinline__ typename Vec<T>::v8 operand(lds_c tile, int t) {
        const int lane = threadIdx.x & 63, r = lane & 15, qd = lane >> 4;
        typename Vec<T>::v8 v;
        if constexpr (sizeof(T) == 2) {
            s16x4 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 16 * i + 4 * qd + (r >> 2), unit = 2 * t + (r >> 1 & 1);
                x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p<s16x4>)(tile + row * D * 2 + (unit ^ swz(row)) * 16 + 8 * (r & 1)));
            }
            v = __builtin_bit_cast(typename Vec<T>::v8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 16 * (e >> 2) + 4 * qd + (e & 3), unit = 4 * t + (r >> 2);
                v[e] = *(lds_p<float>)(tile + row * D * 4 + (unit ^ swz(row)) * 16 + 4 * (r & 3));
            }
        }
        return v;
    }
};
// 8 elements of a row at dim d0; VEC: in 16-byte pieces
template <typename T, bool VEC, bool ONCE>
__device__ __forceinline__ typename Vec<T>::v8 load8(const T* row, int d0, int d) {
    typename Vec<T>::v8 x;
    if constexpr (VEC) {
        constexpr int U = kUnit<T>;
#pragma unroll
        for (int i = 0; i < 8; i += U) {
            typename Raw<T, U>::type y;
            if (d0 + i < d) y = load_raw<T, U, ONCE>(row + d0 + i);
            else y = typename Raw<T, U>::type{};
#pragma unroll
            for (int e = 0; e < U; ++e) x[i + e] = y[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = d0 + e < d ? row[d0 + e] : to_t<T>(0.f);
    }
    return x;
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16, 64));
    return pair_max(x);
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    return pair_sum(x);
}

template <typename T, int DK, int DV, int NW, bool VEC, bool ONCE>
__global__ __launch_bounds__(64 * NW, 2) void k_window_step(AttnArgs a, int splits) {
    typedef StepTile<T, DV> Tile;
    constexpr int KS = DK / 32, VS = DV / 16, VU = 32 * Tile::UN / 64;
    __shared__ __attribute__((aligned(16))) T Vs[NW][32 * DV];
    __shared__ float ml[NW][2][16];
    const int Nk = a.p.num_kv_heads, G = a.p.num_q_heads / Nk, HC = (G + 15) / 16, HPB = G < 16 ? G : 16;
    const int sp = blockIdx.x % splits, id = blockIdx.x / splits, hh = id % (Nk * HC), n = id / (Nk * HC);
    const int hk = hh / HC, hc = hh % HC;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r = lane & 15, qd = lane >> 4;
    const int dk = a.p.head_dim_qk, dv = a.p.head_dim_v, S = a.p.sinks, W = a.p.window;
    const T *kn = (const T*)a.k + n * a.p.k_stride + (int64_t)hk * dk, *vn = (const T*)a.v + n * a.p.v_stride + (int64_t)hk * dv;
    const int g = hc * 16 + r, head = hk * G + (g < G ? g : G - 1);
    const T* qn = (const T*)a.q + n * a.p.q_stride + (int64_t)head * dk;
    typename Vec<T>::v8 qf[KS];
#pragma unroll
    for (int t = 0; t < KS; ++t) qf[t] = load8<T, VEC, false>(qn, 32 * t + 8 * qd, dk);
    const int len = __builtin_amdgcn_readfirstlane(a.lens[n]), p = len < kMostLen ? len : kMostLen;
    const bool idle = p < 0;
    const int64_t cap = (int64_t)S + W;
    const int rows = (int64_t)p + 1 < cap ? p + 1 : (int)cap, own = p < S ? p : S + (p - S) % W;
    T *kc = (T*)a.kc + (n * cap * Nk + hk) * dk, *vc = (T*)a.vc + (n * cap * Nk + hk) * dv;
    const int64_t kld = (int64_t)Nk * dk, vld = (int64_t)Nk * dv;
    if (!idle && hc == 0 && sp == 0) {
        // nobody reads the token's row of the caches: its old token is out of sight
        for (int d = tid; d < dk; d += 64 * NW) kc[own * kld + d] = kn[d];
        for (int d = tid; d < dv; d += 64 * NW) vc[own * vld + d] = vn[d];
    }
    const float c = a.p.scale * kLog2e;
    const int parts = splits * NW, tiles = idle ? 0 : (rows + 31) / 32, share = (tiles + parts - 1) / parts;
    const int first = (sp * NW + w) * share, last = first + share < tiles ? first + share : tiles;
    f32x4 o[VS];
#pragma unroll
    for (int t = 0; t < VS; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, mc = kNegInf, l = 0.f;
    const lds_c mine_v = lds_of(&Vs[0][0]) + w * 32 * DV * (int)sizeof(T);
    typename Vec<T>::v8 kf[2][KS];
    u32x4 vx[VU];
    auto load_keys = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int row = 32 * tile + 16 * i + r;
            row = row < rows ? row : rows - 1;
            const T* x = row == own ? kn : kc + row * kld;
#pragma unroll
            for (int t = 0; t < KS; ++t) kf[i][t] = load8<T, VEC, ONCE>(x, 32 * t + 8 * qd, dk);
        }
    };
    auto load_values = [&](int tile) {
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int at = lane + 64 * i;
            int row = 32 * tile + at / Tile::UN;
            row = row < rows ? row : rows - 1;
            const T* x = row == own ? vn : vc + row * vld;
            const int d0 = at % Tile::UN * kUnit<T>;
            typename Raw<T, kUnit<T>>::type y;
            if constexpr (VEC) {
                if (d0 < dv) y = load_raw<T, kUnit<T>, ONCE>(x + d0);
                else y = typename Raw<T, kUnit<T>>::type{};
            } else {
#pragma unroll
                for (int e = 0; e < kUnit<T>; ++e) y[e] = d0 + e < dv ? x[d0 + e] : to_t<T>(0.f);
            }
            vx[i] = __builtin_bit_cast(u32x4, y);
        }
    };
    if (first < last) {
        load_keys(first);
        load_values(first);
    }
#pragma unroll 1
    for (int tile = first; tile < last; ++tile) {
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int at = lane + 64 * i, row = at / Tile::UN, unit = at % Tile::UN ^ Tile::swz(row);
            *(lds_p<u32x4>)(mine_v + (row * Tile::UN + unit) * 16) = vx[i];
        }
        const int next = tile + 1 < last ? tile + 1 : tile;
        load_values(next);
        f32x4 s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < KS; ++t) s[i] = mfma_pair(kf[i][t], qf[t], s[i]);
        }
        load_keys(next);
        if (32 * tile + 32 > rows) {
            asm volatile("");
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i >> 2][i & 3] = 32 * tile + 16 * (i >> 2) + 4 * qd + (i & 3) < rows ? s[i >> 2][i & 3] : kNegInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = __builtin_elementwise_maximum(top, s[i >> 2][i & 3]);
        top = quad_max(top);
        const bool grown = (top - m) * c > 8.f;
        if (__any(grown)) {
            const float mn = grown ? top : m, mcn = grown ? mn * c : mc, f = grown ? refer(mc, mcn) : 1.f;
            l *= f;
#pragma unroll
            for (int t = 0; t < VS; ++t) o[t] = o[t] * f;
            m = mn;
            mc = mcn;
        }
        // as in weigh
        float mc0 = m == kNegInf ? 0.f : mc;
        const bool far = fabsf(mc0) > 16777216.f;
        if (__any(far)) {
            asm volatile("");
            const float m0 = far ? m : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] -= m0;
            mc0 = far ? 0.f : mc0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i >> 2][i & 3] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][i & 3], c, -mc0));
            l += s[i >> 2][i & 3];
        }
        const auto wt = acc_to_pair<T>(s[0], s[1]);
#pragma unroll
        for (int t = 0; t < VS; ++t) o[t] = mfma_pair(Tile::operand(mine_v, t), wt, o[t]);
    }
    // join the wavefronts: all their sums in LDS, then a thread an output
    l = quad_sum(l);
    float* mine = reinterpret_cast<float*>(Vs[w]);
    static_assert(32 * DV * sizeof(T) >= 16 * DV * 4, "a wavefront's values make room for its outputs");
#pragma unroll
    for (int t = 0; t < VS; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[(16 * t + 4 * qd + j) * 16 + r] = o[t][j];
    if (lane < 16) {
        ml[w][0][lane] = mc;
        ml[w][1][lane] = l;
    }
    __syncthreads();
    const int cols = G - hc * 16 < HPB ? G - hc * 16 : HPB;
    for (int i = tid; i < dv * cols; i += 64 * NW) {
        const int h = i / dv, d = i - h * dv;
        float mm = kNegInf, ll = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) mm = fmaxf(mm, ml[k][0][h]);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float f = refer(ml[k][0][h], mm);
            ll = __builtin_fmaf(ml[k][1][h], f, ll);
            y = __builtin_fmaf(reinterpret_cast<const float*>(Vs[k])[d * 16 + h], f, y);
        }
        const int64_t row = (int64_t)n * a.p.num_q_heads + hk * G + hc * 16 + h;
        if (splits == 1) {
            store_as<T>(a.o, row * dv + d, idle ? 0.f : y / ll, a.p.out_dtype == GDR_F32);
        } else {
            float* part = a.ws + ((int64_t)sp * a.Ttot * a.p.num_q_heads + row) * (dv + 2);
            part[d] = y;
            if (d == 0) {
                part[dv] = idle ? 0.f : mm;
                part[dv + 1] = idle ? -1.f : ll;
            }
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
// Many rows: 32 a wavefront; few rows: 32 a workgroup, whose wavefronts share the keys.
// Four wavefronts a workgroup for many rows: eight read the keys half as often, but leave
// compute units idle (65,536 tokens of 32 heads the same, 65,536 of 16 heads of 64 over a window of
// 1,024 823 us with four and 1,023 with eight, 8,191 packed ones 55 and 65).
// Shared keys against many rows, 6 heads over 2, us, by blocks of 32 rows:
//   bf16, 128 x 128, window 512     137: 16 23   273: 25 23   546: 42 24   820: 58 24
//                    window 2,048   137: 16 22   273: 31 35   546: 61 54   820: 91 55
//   fp32, 128 x 128, window 512     137: 43 93   273: 58 94   546: 105 95  820: 152 97   1,093: 196 166
//                    window 2,048   273: 81 192  546: 194 306 820: 307 309 1,093: 414 542 1,639: 637 544
//   fp32, 64 x 64, window 512       273: 31 54   546: 48 55   820: 67 55   1,093: 82 89  1,639: 116 91
// In bf16 a compute unit's share of 256 blocks decides, in fp32 sharing pays up to 512 blocks,
// and beyond while n / 256 rounds of tiles / 4 + 5 are less than n / 1,024 rounds of tiles + 2.
constexpr int kRowWaves = 4;
template <typename T> constexpr int kSplitWaves = sizeof(T) == 2 ? 8 : 4;
struct Plan {
    bool split;
    int splits;
    RowBlock rb;
    int64_t nblk, nwork;
};
// behind: there may be cached tokens in front of the call's. A query then sees sinks + window
// keys, else no more than its sequence has (350 pieces of 64 tokens on caches, fp32, 64 x 64, window
// 4,096: shared 356 us, not shared 812; a prompt of 512 tokens, 2 heads of 64 in bf16, under a window
// of 65,536: 9.4 us in a workgroup each and 16.2 in 16, of which 2 have keys).
Plan plan_of(const gdr_attn_problem_t& p, bool behind) {
    Plan x{};
    const int G = group(p);
    const bool bf = p.io_dtype == GDR_BF16, packed = p.batch == 1 && p.num_seqs != 1;
    auto blocks = [&](int rows) {
        x.rb = row_block(rows, G);
        x.nblk = token_blocks(p.batch, p.seq_len, p.num_seqs, packed, x.rb.TPB);
        x.nwork = x.nblk * p.num_kv_heads * x.rb.HC;
    };
    const int64_t all = (int64_t)p.sinks + p.window;
    auto tiles_of = [&](int64_t len) { return ((behind || all < len ? all : len) + 31) / 32; };
    blocks(32);
    x.splits = 1;
    x.split = x.nwork <= (bf ? 256 : 512);
    if (!bf && !x.split && x.nwork < 4096) {
        const int64_t tiles = tiles_of(p.seq_len / (packed && p.num_seqs > 0 ? p.num_seqs : 1));
        x.split = x.nwork * (tiles + 20) < 1024 * ((x.nwork + 1023) / 1024) * (tiles + 2);
    }
    if (x.split) {
        // workgroups share the keys too where a wavefront had 16 tiles of them and more
        const int64_t each = tiles_of(p.seq_len) / (bf ? 8 : 4) / 16;
        const int64_t want = x.nwork > 0 ? 256 / x.nwork : 1, s = want < each ? want : each;
        x.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
    } else {
        blocks(32 * kRowWaves);
    }
    return x;
}

// Single tokens: workgroups that share the rows of a sequence's key head
constexpr int kStepWaves = 8;
// One sequence, 4 key heads, window 4,096: 33 us in one workgroup each, 19 in 8; 4 sequences 42
// and 25. Below 8 tiles a wavefront the second launch costs what sharing saves (window 1,024:
// 14.7 and 15.6).
int step_splits(const gdr_attn_problem_t& p) {
    const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * ((group(p) + 15) / 16);
    const int64_t each = ((int64_t)p.sinks + p.window) / (32 * kStepWaves);       // tiles of a wavefront
    if (each < 8 || units < 1) return 1;
    const int64_t want = 256 / units, s = want < each / 2 ? want : each / 2;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

}  // namespace

size_t attn_fwd_workspace(const gdr_attn_problem_t& p) {
    // the size is asked for without the caches: it does for a call with them and for one without
    const int a = plan_of(p, false).splits, b = plan_of(p, true).splits, splits = a > b ? a : b;
    if (splits <= 1) return 0;
    return (size_t)splits * p.batch * p.seq_len * p.num_q_heads * (p.head_dim_v + 2) * 4;
}

hipError_t launch_attn_step(const AttnArgs& a) {
    if (a.Ttot == 0) return hipSuccess;
    const int splits = step_splits(a.p);
    const int64_t units = (int64_t)a.p.num_seqs * a.p.num_kv_heads * ((group(a.p) + 15) / 16) * splits;
    if (!grid_fits(units, 64 * kStepWaves)) return hipErrorInvalidConfiguration;
    const int64_t rows = (int64_t)a.p.sinks + a.p.window;
    const bool once = beyond_caches(a.p.num_seqs * rows * a.p.num_kv_heads * (a.p.head_dim_qk + a.p.head_dim_v) *
                                    size_of(a.p.io_dtype));
    by_dims(a.p, [&](auto type, auto dk, auto dv) {
        typedef decltype(type) T;
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, NW = kStepWaves;
        const dim3 grid((unsigned)units);
        if (!a.vec) k_window_step<T, DK, DV, NW, false, false><<<grid, 64 * NW, 0, a.stream>>>(a, splits);
        else if (once) k_window_step<T, DK, DV, NW, true, true><<<grid, 64 * NW, 0, a.stream>>>(a, splits);
        else k_window_step<T, DK, DV, NW, true, false><<<grid, 64 * NW, 0, a.stream>>>(a, splits);
        if (splits > 1) {
            const int64_t n = a.Ttot * a.p.num_q_heads;
            k_window_join<T><<<dim3((unsigned)((n + 3) / 4)), 256, 0, a.stream>>>(a, splits);
        }
    });
    return hipGetLastError();
}

size_t attn_step_workspace(const gdr_attn_problem_t& p) {
    const int s = step_splits(p);
    return s > 1 ? (size_t)s * p.num_seqs * p.num_q_heads * (p.head_dim_v + 2) * 4 : 0;
}

hipError_t launch_attn_fwd(const AttnArgs& a) {
    if (a.Ttot == 0) return hipSuccess;
    const Plan x = plan_of(a.p, a.kc && a.lens);
    const int64_t waves = x.split ? (a.p.io_dtype == GDR_BF16 ? kSplitWaves<bf16> : kSplitWaves<float>) : kRowWaves;
    if (x.nwork >= (int64_t)1 << 31 || !grid_fits(x.nwork * x.splits + 8, 64 * (int)waves)) return hipErrorInvalidConfiguration;
    hipError_t e = hipSuccess;
    by_dims(a.p, [&](auto type, auto dk, auto dv) {
        typedef decltype(type) T;
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, NS = kSplitWaves<T>, NR = kRowWaves;
        if (x.split) {
            const dim3 grid((unsigned)(x.nwork * x.splits));
            if (a.vec) k_window_split<T, DK, DV, NS, true><<<grid, 64 * NS, 0, a.stream>>>(a, x.rb, (int)x.nblk, x.splits);
            else k_window_split<T, DK, DV, NS, false><<<grid, 64 * NS, 0, a.stream>>>(a, x.rb, (int)x.nblk, x.splits);
            if (x.splits > 1) {
                const int64_t rows = a.Ttot * a.p.num_q_heads;
                k_window_join<T><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, a.stream>>>(a, x.splits);
            }
        } else {
            const dim3 grid((unsigned)((x.nwork + 7) / 8 * 8));
            auto go = [&](auto tile) {
                constexpr int KT = decltype(tile)::value;
                if (a.vec)
                    k_window_rows<T, DK, DV, NR, KT, true><<<grid, 64 * NR, 0, a.stream>>>(a, x.rb, (int)x.nblk, (int)x.nwork);
                else
                    k_window_rows<T, DK, DV, NR, KT, false><<<grid, 64 * NR, 0, a.stream>>>(a, x.rb, (int)x.nblk, (int)x.nwork);
            };
            // Keys of a tile, bf16, 16 heads over 4, us with 32 and 64. Dims of 64: 8,191 tokens, window 512:
            // 40 48; 65,536, 256: 185 220; 65,536, 2,048: 708 715. Dims of 128 by windows of
            //   65,536 tokens   256: 302 360   1,024: 703 749   2,048: 1,244 1,248   4,096: 2,262 2,197
            //   16,384          512: 108 118   1,024: 172 175   2,048: 303 294       4,096: 547 516
            //   8,191           512: 68 63     1,024: 103 89    2,048: 176 144       4,096: 316 247
            // Tiles of 32 leave less at a window's edges, and registers for three wavefronts a SIMD in
            // place of two, of which up to 1,024 workgroups fill a second round to a third; tiles of 64
            // meet in barriers half as often. v of 64 dims, 65,536 tokens, 4,096: 1,789 1,827; 8,191, 2,048: 134 121.
            if constexpr (sizeof(T) == 2 && DK + DV > 128) {
                const int64_t sight = (int64_t)a.p.sinks + a.p.window;
                if ((x.nwork <= 1024 && sight >= 1024) || (DK + DV == 256 && sight >= 2048)) go(std::integral_constant<int, 64>{});
                else go(std::integral_constant<int, 32>{});
            } else {
                go(std::integral_constant<int, 32>{});
            }
        }
        e = hipGetLastError();
        if (e == hipSuccess && a.kc) {
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
