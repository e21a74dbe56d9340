// Window attention, backward (include/gdr_attn.h; tile conventions in gdr_attn.hpp).
//
//   P_pj = exp(s_pj - lse_p),  dP = d_o v^T,  dS = P (dP - delta),  delta_p = d_o_p . o_p
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T d_o
//
// The scores are formed again, twice: k_window_dq walks the keys of a block of
// queries, k_window_dkv the queries of a block of keys, each summing what it
// owns in registers, so that no sum crosses workgroups and its order is fixed. The
// first also forms delta and leaves it for the second.
// P is exp2(c s - lse log2(e)) with c = scale log2(e). fp32 holds a large lse coarsely: at
// 2^24 an ulp of it is a factor in P, and a row of one key would not weigh one. Where
// |lse log2(e)| is beyond kFarLse, the rounding of lse to fp32 and its few operations (about
// 4 ulps) would cost P more than 2^-12, as much as a score's own rounding does; k_window_dq
// then goes over the row's scores first, as the forward pass did, and P is exp2(c (s - top)
// - log2(sum of exp2(c (s - top)))), in both kernels. A row's own choice, from its lse alone.
// Where no row is far this costs up to 2 % of the gradients' time (4 x 4,096 tokens of 16 heads, 128 x
// 128, 486 us without it, 488 with it; rows that are not 16-byte aligned 5 %), where all are 34 %.
// The first tokens alone are seen by queries of the whole sequence: those behind
// the ones that a key block meets anyway are shared out in runs of tokens,
// whose sums go to slots in memory and are added up by k_window_sinks.
#include "gdr_attn.hpp"

namespace gdr {

namespace {

// Tokens of a run: 64 runs to a sequence, but not too short and not too long ones. By the
// sequence's own length, so that its gradients do not depend on what it is packed with.
__host__ __device__ inline int64_t sink_run(int64_t len) {
    const int64_t n = len / 64;
    return n < 256 ? 256 : n < 4096 ? n : 4096;
}
// First slot of each sequence, by one wavefront: a slot for the own sums of the key blocks
// with sinks, and one for each run of tokens behind a window.
__device__ void count_slots(const AttnArgs& a) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int n0 = 0; n0 <= a.p.num_seqs; n0 += 64) {
        const int n = n0 + lane;
        int m = 0;
        if (n < a.p.num_seqs) {
            int64_t s, e;
            seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
            const int64_t behind = e - s - a.p.window, run = sink_run(e - s);
            if (behind > 0) m = (int)((behind + run - 1) / run) + 1;
        }
        int sum = m;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(sum, d, 64);
            if (lane >= d) sum += x;
        }
        const int first = base + sum - m;
        if (n <= a.p.num_seqs) a.slots[n] = first < a.max_slots ? first : a.max_slots;
        base += __shfl(sum, 63, 64);
    }
}

constexpr float kFarLse = 1024.f;
// a row's scores as exponents refer to them: its largest one (0: they do not) is taken off
__device__ __forceinline__ float below_top(float s, float top) {
    return top != 0.f ? __builtin_elementwise_minimum(s - top, 0.f) : s;
}

// A d_o in fp32 in the io type, 4 elements a thread
template <typename T>
__global__ __launch_bounds__(256) void k_window_round(const float* from, T* to, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * 1024;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += step) {
        if (i + 4 <= n) {
            float x[4];
            unpack<float, 4>(load_raw<float, 4>(from + i), x);
            store_vec<T, 4>(to + i, x);
        } else {
            for (int64_t j = i; j < n; ++j) to[j] = to_t<T>(from[j]);
        }
    }
}

// ---------------------------------------------------------------- dq
// As k_window_rows: 32 rows a wavefront, keys and values of 32 tokens in LDS, two tiles in
// turn. A lane owns a query, so that lse and delta are its own registers. Of the five products
// that gradients need at least, seven are formed in the two kernels (s and dP twice), with no
// sums across workgroups for it. 4 x 4,096 tokens of 16 heads over 4, 128 x 128, window 1,024:
// 231 us here and 293 in k_window_dkv, 600 TFLOP/s of the five; matrix cores busy 42 and 46 % of
// the cycles. fp32, 2 x 2,048 tokens of them: 1,538 us in all, 42 TFLOP/s; 64 x 64 819 us. 128
// rows a workgroup against 256: 240 us and 256, packed prompts of 353 tokens 24 and 29. Tiles of
// 64 keys: 240.
template <typename T, int DK, int DV, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, 2) void k_window_dq(AttnArgs a, RowBlock rb, int nblk, int nwork) {
    constexpr int KT = 32, KF = DK / (2 * kUnit<T>), VF = DV / (2 * kUnit<T>);
    __shared__ __attribute__((aligned(16))) T Ks[2][KT * DK], Vs[2][KT * DV];
    __shared__ int far_rows[NW];
    const lds_c K0 = lds_of(Ks[0]), K1 = lds_of(Ks[1]), V0 = lds_of(Vs[0]), V1 = lds_of(Vs[1]);
    if (blockIdx.x == 0 && threadIdx.x < 64 && a.slots) count_slots(a);
    const int per = (nwork + 7) / 8, id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= nwork) return;
    const int hh = id / nblk, G = a.p.num_q_heads / a.p.num_kv_heads, hk = hh / rb.HC, hc = hh % rb.HC;
    Block b;
    if (!find_block(a.cu, a.p.num_seqs, a.p.seq_len, a.Ttot, rb.TPB, id % nblk, &b)) return;
    const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63, h = lane >> 5;
    const int W = a.p.window, S = a.p.sinks, dk = a.p.head_dim_qk, dv = a.p.head_dim_v;
    const Query q = query_of(b, rb, G, hk, hc, 32 * w + (lane & 31), 0);
    const int pa = __builtin_amdgcn_readlane(q.p, 0), pb = __builtin_amdgcn_readlane(q.p, 31);
    const int64_t row = q.token * a.p.num_q_heads + q.head;
    frag_t<T> qf[KF], gf[VF];
#pragma unroll
    for (int t = 0; t < KF; ++t)
        qf[t] = load_frag_row<T, VEC>((const T*)a.q + q.token * a.p.q_stride + (int64_t)q.head * dk, 2 * t + h, dk, q.live);
#pragma unroll
    for (int t = 0; t < VF; ++t) gf[t] = load_frag_row<T, VEC>((const T*)a.d_o + row * dv, 2 * t + h, dv, q.live);
    // lse in units of log 2, and delta: here for the lane's query, in memory for k_window_dkv
    float lse = a.lse_in[row] * kLog2e, top = 0.f, delta = 0.f;
    const float c = a.p.scale * kLog2e;
    const bool far = fabsf(lse) > kFarLse;
#pragma unroll
    for (int t = 0; t < VF; ++t) {
        const int d0 = (2 * t + h) * kUnit<T>;
        float o[kUnit<T>];
        if (VEC && d0 < dv) {
            load_vec_as<T, kUnit<T>>(a.oin, row * dv + d0, a.p.out_dtype == GDR_F32, o);
        } else {
#pragma unroll
            for (int e = 0; e < kUnit<T>; ++e)
                o[e] = d0 + e < dv ? load_as<T>(a.oin, row * dv + d0 + e, a.p.out_dtype == GDR_F32) : 0.f;
        }
        // rows that are not there have a d_o of zero
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) delta = __builtin_fmaf(q.live ? o[e] : 0.f, to_f(gf[t][e]), delta);
    }
    delta = pair_sum(delta);
    if (lane == 0) far_rows[w] = 0;
    if (far && q.live) far_rows[w] = 1;
    f32x16 acc[DK / 32];
#pragma unroll
    for (int t = 0; t < DK / 32; ++t) acc[t] = zero16();

    Keys keys(b.t0, b.t0 + b.tn - 1, 0, W, S);
    Copy<T, DK, KT, 64 * NW, VEC> ck;
    Copy<T, DV, KT, 64 * NW, VEC> cv;
    int pos, cnt, at;
    bool cached;
    auto fetch = [&](lds_c K, lds_c V) {
        keys.next(KT, &pos, &cnt, &at, &cached);
        if (cnt == 0) return;
        const Source<T> s = source<T>(a, b, hk, at, false);
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
    int some = 0;                                                  // whether a row of the block is far
    auto turn = [&](lds_c K, lds_c V, lds_c Kn, lds_c Vn) {
        const int pos0 = pos, n = cnt;
        const int ro = fresh(row_offset<T, DK>(lane)), rv = DK == DV ? ro : fresh(row_offset<T, DV>(lane)),
                  co = fresh(col_offset<T, DK>(lane));
        fetch(Kn, Vn);
        if (pos0 <= pb && (pos0 < S || pos0 + n - 1 > pa - W)) {
            const bool partial = n < KT || pos0 + KT - 1 > pa || (pos0 <= pb - W && pos0 + KT > S);
            const Sight sees{pos0, n, q.p, W, S};
            f32x16 s = zero16(), g = zero16();
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int t = 0; t < KF; ++t) s = mma(row_frag<T, DK>(K, 0, t, ro), qf[t], s);
            feed<KF, 1, sizeof(T) == 2 ? 1 : 4, 4>();
#pragma unroll
            for (int t = 0; t < VF; ++t) g = mma(row_frag<T, DV>(V, 0, t, rv), gf[t], g);
            feed<VF, 1, sizeof(T) == 2 ? 1 : 4, 4>();
            __builtin_amdgcn_s_setprio(0);
            if (some) {
                asm volatile("");
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = below_top(s[i], top);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse)) * (g[i] - delta);
            if (partial) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = sees(8 * (i >> 2) + 4 * h + (i & 3)) ? s[i] : 0.f;
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto x = acc_frag<T>(s, e);
#pragma unroll
                for (int t = 0; t < DK / 32; ++t) acc[t] = mma(col_frag<T, DK>(K, 16 * e, t, co), x, acc[t]);
            }
            __builtin_amdgcn_s_setprio(0);
        }
        land(Kn, Vn);
    };
    fetch(K0, V0);
    arrived(qf);
    arrived(gf);
    land(K0, V0);
#pragma unroll
    for (int i = 0; i < NW; ++i) some |= far_rows[i];
    some = __builtin_amdgcn_readfirstlane(some);
    if (some) {
        // the largest score and the sum of each row, while the first tile waits in K0 and V0
        Keys all(b.t0, b.t0 + b.tn - 1, 0, W, S);
        Copy<T, DK, KT, 64 * NW, VEC> ca;
        float m = kNegInf, l = 0.f;
        for (;;) {
            int p0, n, r0;
            bool old;
            all.next(KT, &p0, &n, &r0, &old);
            if (n == 0) break;
            const Source<T> x = source<T>(a, b, hk, r0, false);
            ca.start(K1, x.k, x.kld, n, dk, tid);
            ca.finish(K1, tid);
            landed();
            const Sight sees{p0, n, q.p, W, S};
            f32x16 s = zero16();
#pragma unroll
            for (int t = 0; t < KF; ++t) s = mma(row_frag<T, DK>(K1, 0, t, row_offset<T, DK>(lane)), qf[t], s);
            float most = m, sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = sees(8 * (i >> 2) + 4 * h + (i & 3)) ? s[i] : kNegInf;
                most = __builtin_elementwise_maximum(most, s[i]);
            }
            const float ref = most == kNegInf ? 0.f : most;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += __builtin_amdgcn_exp2f((s[i] - ref) * c);
            l = __builtin_fmaf(l, __builtin_amdgcn_exp2f((m - ref) * c), sum);
            m = most;
            __syncthreads();
        }
        const float most = pair_max(m);
        l = pair_sum(l * (m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m - most) * c)));
        if (far) {
            top = most;
            lse = __builtin_amdgcn_logf(l);
        }
    }
    while (cnt > 0) {
        turn(K0, V0, K1, V1);
        if (cnt == 0) break;
        turn(K1, V1, K0, V0);
    }
    if (!q.live) return;
    if (h == 0) {
        a.rows[2 * row] = lse;
        a.rows[2 * row + 1] = delta;
        a.tops[row] = top;
    }
#pragma unroll
    for (int t = 0; t < DK / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = acc[t][4 * i + j] * a.p.scale;
            const int d = 32 * t + 8 * i + 4 * h;
            if (a.p.grad_dtype == GDR_F32) store4((float*)a.dq + row * dk, d, dk, y);
            else store4((T*)a.dq + row * dk, d, dk, y);
        }
}

// ---------------------------------------------------------------- dk, dv
constexpr int kQueryTile = 32;

// A wavefront owns 32 keys (a lane a key), with their k as operand and the sums of dk
// and dv in registers; the queries' tiles go through LDS. v is an operand in registers
// too (fp32), or lies in LDS, so that two wavefronts fit a SIMD (bf16). Work numbers from
// `main` on are the runs of queries that see sinks alone.
// LDS and the matrix cores bound it alike: a tile's 32 rows of q and d_o are read twice each
// and v once, 42 KB to 32 products of 32 cycles for each of eight wavefronts. The loads
// are covered: with tiles in an order in which an XCD's cache serves them (a quarter of the
// bytes from beyond it) the time was the same.
template <typename T, int DK, int DV, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void k_window_dkv(AttnArgs a, RowBlock rb, int nblk,
                                                                                int main, int nwork) {
    constexpr int QT = kQueryTile, KB = 32 * NW, KF = DK / (2 * kUnit<T>), VF = DV / (2 * kUnit<T>);
    constexpr bool VLDS = sizeof(T) == 2;
    __shared__ __attribute__((aligned(16))) T Vb[VLDS ? KB * DV : 1], Qs[2][QT * DK], Gs[2][QT * DV];
    __shared__ __attribute__((aligned(16))) float Rs[2][4 * QT];               // lse of the rows, delta, top, unused
    const lds_c Vk = lds_of(Vb), Q0 = lds_of(Qs[0]), Q1 = lds_of(Qs[1]), G0 = lds_of(Gs[0]), G1 = lds_of(Gs[1]);
    const lds_c R0 = lds_of(Rs[0]), R1 = lds_of(Rs[1]);
    // consecutive key blocks of a head on one XCD; the runs are dealt to all of them
    const int per = (main + 7) / 8, at = (int)(blockIdx.x >> 3);
    const int id = at < per ? (int)(blockIdx.x & 7) * per + at : (int)blockIdx.x - 8 * per + main;
    if (id >= nwork || (at < per && id >= main)) return;
    const int Nk = a.p.num_kv_heads, G = a.p.num_q_heads / Nk, W = a.p.window, S = a.p.sinks;
    const int dk = a.p.head_dim_qk, dv = a.p.head_dim_v;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, h = lane >> 5;
    Block b;
    int hk, slot, ta, te, keys;                // tokens [ta, te) of the sequence, keys from b.t0 on
    if (id < main) {
        hk = id / nblk;
        if (!find_block(a.cu, a.p.num_seqs, a.p.seq_len, a.Ttot, KB, id % nblk, &b)) return;
        keys = b.tn;
        ta = b.t0;
        const int64_t end = (int64_t)b.t0 + b.tn - 1 + W;
        te = end < b.len ? (int)end : b.len;
        slot = b.t0 < S && a.slots && a.slots[b.n + 1] > a.slots[b.n] ? a.slots[b.n] : -1;
    } else {
        const int sb = (S + KB - 1) / KB, i = id - main, u = i / (Nk * sb);
        hk = i / sb % Nk;
        // the sequence whose slots hold u
        int lo = 0, len = a.p.num_seqs;
        while (len > 1) {
            const int step = (len + 63) / 64, at = lo + lane * step;
            const bool before = at < lo + len && a.slots[at] <= u;
            const int k = __popcll(__ballot(before)), x = k > 0 ? (k - 1) * step : 0;
            len = len - x < step ? len - x : step;
            lo += x;
        }
        b.n = __builtin_amdgcn_readfirstlane(lo);
        const int run = u - a.slots[b.n];
        if (run < 1 || u >= a.slots[b.n + 1]) return;
        int64_t s, e;
        seq_range(a.cu, b.n, a.p.seq_len, a.Ttot, &s, &e);
        b.start = s;
        b.len = (int)(e - s);
        b.t0 = i % sb * KB;
        keys = S - b.t0 < KB ? S - b.t0 : KB;
        keys = b.len - b.t0 < keys ? b.len - b.t0 : keys;
        // the key block's own run ends where its last key's window does
        const int own = (b.len - b.t0 < KB ? b.len - b.t0 : KB);
        const int64_t from = (int64_t)b.t0 + own - 1 + W, each = sink_run(b.len), first = W + (run - 1) * each;
        int64_t x = first > from ? first : from, y = first + each;
        // the last run takes what is left; all runs begin behind the first window
        x = x < b.len ? x : b.len;
        y = y < b.len ? y : b.len;
        ta = (int)x;
        te = y > x ? (int)y : (int)x;
        slot = u;
    }
    const int mine = b.t0 + 32 * w + (lane & 31);                  // the lane's key
    const unsigned mine_for = mine < S ? 0x7fffffffu : (unsigned)W; // tokens that see it, itself the first
    const int ja = b.t0 + 32 * w, jb = ja + 31 < b.t0 + keys - 1 ? ja + 31 : b.t0 + keys - 1;
    const bool live = mine < b.t0 + keys;
    const float c = a.p.scale * kLog2e;
    frag_t<T> kf[KF], vf[VLDS ? 1 : VF];
    {
        const int64_t tok = b.start + (live ? mine : b.t0);
        const T* vrow = (const T*)a.v + (int64_t)hk * dv;
#pragma unroll
        for (int t = 0; t < KF; ++t)
            kf[t] = load_frag_row<T, VEC>((const T*)a.k + tok * a.p.k_stride + (int64_t)hk * dk, 2 * t + h, dk, live);
        if constexpr (VLDS) {
            Copy<T, DV, KB, 64 * NW, VEC> cv;
            cv.start(Vk, vrow + (b.start + b.t0) * a.p.v_stride, a.v_ld, keys, dv, tid);
            cv.finish(Vk, tid);
        } else {
#pragma unroll
            for (int t = 0; t < VF; ++t) vf[t] = load_frag_row<T, VEC>(vrow + tok * a.p.v_stride, 2 * t + h, dv, live);
        }
    }
    auto v_frag = [&](int t, int off) {
        if constexpr (VLDS) return row_frag<T, DV>(Vk, 32 * w, t, off);
        else return vf[t];
    };
    f32x16 dK[DK / 32], dV[DV / 32];
#pragma unroll
    for (int t = 0; t < DK / 32; ++t) dK[t] = zero16();
#pragma unroll
    for (int t = 0; t < DV / 32; ++t) dV[t] = zero16();

    // row r of a tile: token r / HPB, head r % HPB. Rows that are not there come as zeros
    // and add nothing.
    const int magic = (65536 + rb.HPB - 1) / rb.HPB;               // r / HPB = r magic / 65536 for r < 256
    const int span = rb.HPB * rb.TPB, Nq = a.p.num_q_heads;
    auto row_at = [&](int r, int ld, int d) {
        const int x = (r * magic) >> 16, g = r - x * rb.HPB;
        return r < span ? (x * ld + g * d) * (int)sizeof(T) : kOutside;
    };
    Copy<T, DK, QT, 64 * NW, VEC> cq;
    Copy<T, DV, QT, 64 * NW, VEC> cg;
    int t = ta, hc = 0, p0 = ta, p1 = ta;
    bool more = true;
    auto fetch = [&](lds_c Q, lds_c Gr, lds_c R) {
        more = t < te;
        if (!more) return;
        const int n = te - t < rb.TPB ? te - t : rb.TPB, heads = G - hc * rb.HPB < rb.HPB ? G - hc * rb.HPB : rb.HPB;
        const int64_t tok = b.start + t;
        const int head = hk * G + hc * rb.HPB, g_ld = Nq * dv;
        cq.start(Q, (const T*)a.q + tok * a.p.q_stride + (int64_t)head * dk,
                 (uint32_t)((n - 1) * a.q_ld + heads * dk) * sizeof(T), [&](int r) { return row_at(r, a.q_ld, dk); }, dk, tid);
        cg.start(Gr, (const T*)a.d_o + (tok * Nq + head) * dv, (uint32_t)((n - 1) * g_ld + heads * dv) * sizeof(T),
                 [&](int r) { return row_at(r, g_ld, dv); }, dv, tid);
        if (w == 0) {
            const int r = lane & 31, x = (r * magic) >> 16, g = r - x * rb.HPB;
            static_assert(QT == 32 && NW > 1, "lse and delta of a tile in 64 lanes, top by the next wavefront");
            copy4_to_lds(raw_rsrc(a.rows + 2 * (tok * Nq + head), (uint32_t)((n - 1) * Nq + heads) * 8), R,
                         r < span ? (x * Nq + g) * 8 + 4 * h : kOutside);
        } else if (w == 1) {
            const int r = lane & 31, x = (r * magic) >> 16, g = r - x * rb.HPB;
            copy4_to_lds(raw_rsrc(a.tops + (tok * Nq + head), (uint32_t)((n - 1) * Nq + heads) * 4), R + 8 * QT,
                         r < span && h == 0 ? (x * Nq + g) * 4 : kOutside);
        }
        p0 = t;
        p1 = t + n - 1;
        if (++hc == rb.HC) {
            hc = 0;
            t += rb.TPB;
        }
    };
    auto land = [&](lds_c Q, lds_c Gr) {
        if (more) {
            cq.finish(Q, tid);
            cg.finish(Gr, tid);
        }
        landed();
    };
    auto turn = [&](lds_c Q, lds_c Gr, lds_c R, lds_c Qn, lds_c Gn, lds_c Rn) {
        const int a0 = p0, a1 = p1;                                // the queries' positions
        const int rq = fresh(row_offset<T, DK>(lane)), rg = DK == DV ? rq : fresh(row_offset<T, DV>(lane));
        const int cq_ = fresh(col_offset<T, DK>(lane)), cg_ = DK == DV ? cq_ : fresh(col_offset<T, DV>(lane));
        fetch(Qn, Gn, Rn);
        if (ja <= jb && a1 >= ja && (ja < S || a0 <= jb + (int64_t)W - 1)) {
            const bool partial = a0 < jb || (a1 - W >= ja && jb >= S);
            // products, vector work and products again, each for itself: what they need in
            // registers leaves room for two wavefronts a SIMD, of which the one with products
            // goes first
            f32x16 s = zero16(), g = zero16();
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int u = 0; u < KF; ++u) s = mma(row_frag<T, DK>(Q, 0, u, rq), kf[u], s);
            feed<KF, 1, sizeof(T) == 2 ? 1 : 4, 4>();
            __builtin_amdgcn_sched_barrier(0);
            const float tops = *(lds_p<float>)(R + 8 * QT + 4 * (lane & 31));
#pragma unroll
            for (int u = 0; u < VF; ++u) g = mma(row_frag<T, DV>(Gr, 0, u, rg), v_frag(u, rg), g);
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            if (__any(tops != 0.f)) {
                asm volatile("");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 M = *(lds_p<f32x4>)(R + 8 * QT + 32 * i + 16 * h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[4 * i + j] = below_top(s[4 * i + j], M[j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 L = *(lds_p<f32x4>)(R + 32 * i + 16 * h), D = *(lds_p<f32x4>)(R + 4 * QT + 32 * i + 16 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * i + j], c, -L[j]));
                    s[4 * i + j] = p;
                    g[4 * i + j] = p * (g[4 * i + j] - D[j]);
                }
            }
            if (partial) {
                asm volatile("");
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = 8 * (i >> 2) + 4 * h + (i & 3), p = a0 + ((r * magic) >> 16);
                    const bool see = (unsigned)(p - mine) < mine_for;
                    s[i] = see ? s[i] : 0.f;
                    g[i] = see ? g[i] : 0.f;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto x = acc_frag<T>(s, e);
#pragma unroll
                for (int u = 0; u < DV / 32; ++u) dV[u] = mma(col_frag<T, DV>(Gr, 16 * e, u, cg_), x, dV[u]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto y = acc_frag<T>(g, e);
#pragma unroll
                for (int u = 0; u < DK / 32; ++u) dK[u] = mma(col_frag<T, DK>(Q, 16 * e, u, cq_), y, dK[u]);
            }
            __builtin_amdgcn_s_setprio(0);
        }
        land(Qn, Gn);
    };
    fetch(Q0, G0, R0);
    arrived(kf);
    if constexpr (!VLDS) arrived(vf);
    land(Q0, G0);
    while (more) {
        turn(Q0, G0, R0, Q1, G1, R1);
        if (!more) break;
        turn(Q1, G1, R1, Q0, G0, R0);
    }
    if (!live) return;
    const bool to_slot = slot >= 0 && mine < S;
    float* part = to_slot ? a.sink_part + (((int64_t)slot * S + mine) * Nk + hk) * (dk + dv) : nullptr;
    const int64_t row = (b.start + mine) * Nk + hk;
#pragma unroll
    for (int u = 0; u < DK / 32; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = dK[u][4 * i + j] * a.p.scale;
            const int d = 32 * u + 8 * i + 4 * h;
            if (to_slot) store4(part, d, dk, y);
            else if (a.p.grad_dtype == GDR_F32) store4((float*)a.dk + row * dk, d, dk, y);
            else store4((T*)a.dk + row * dk, d, dk, y);
        }
#pragma unroll
    for (int u = 0; u < DV / 32; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = dV[u][4 * i + j];
            const int d = 32 * u + 8 * i + 4 * h;
            if (to_slot) store4(part + dk, d, dv, y);
            else if (a.p.grad_dtype == GDR_F32) store4((float*)a.dv + row * dv, d, dv, y);
            else store4((T*)a.dv + row * dv, d, dv, y);
        }
}

// ---------------------------------------------------------------- sums of the sinks' slots
// Workgroups (slot, key head): those of a sequence share its sinks' elements and add up its
// slots in order.
template <typename T>
__global__ __launch_bounds__(256) void k_window_sinks(AttnArgs a) {
    const int Nk = a.p.num_kv_heads, u = blockIdx.x / Nk, hk = blockIdx.x % Nk, S = a.p.sinks;
    int lo = 0, len = a.p.num_seqs;
    while (len > 1) {
        const int step = (len + 63) / 64, at = lo + (int)(threadIdx.x & 63) * step;
        const bool before = at < lo + len && a.slots[at] <= u;
        const int k = __popcll(__ballot(before)), x = k > 0 ? (k - 1) * step : 0;
        len = len - x < step ? len - x : step;
        lo += x;
    }
    const int n = __builtin_amdgcn_readfirstlane(lo), first = a.slots[n], end = a.slots[n + 1];
    if (u >= end) return;
    int64_t s, e;
    seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
    const int dk = a.p.head_dim_qk, dv = a.p.head_dim_v, d = dk + dv;
    const int rows = S < e - s ? S : (int)(e - s);
    const int64_t step = (int64_t)S * Nk * d;
    for (int64_t i = (int64_t)(u - first) * 256 + threadIdx.x; i < (int64_t)rows * d; i += (int64_t)(end - first) * 256) {
        const int j = (int)(i / d), x = (int)(i % d);
        const float* p = a.sink_part + (((int64_t)first * S + j) * Nk + hk) * d + x;
        float sum = 0.f;
#pragma unroll 8
        for (int k = first; k < end; ++k, p += step) sum += *p;
        const int64_t row = (s + j) * Nk + hk;
        if (x < dk) store_as<T>(a.dk, row * dk + x, sum, a.p.grad_dtype == GDR_F32);
        else store_as<T>(a.dv, row * dv + x - dk, sum, a.p.grad_dtype == GDR_F32);
    }
}

struct Plan {
    int64_t slots;
    size_t rows, tops, d_o16, table, part;   // bytes
};
size_t up(size_t n) { return (n + 255) / 256 * 256; }
// A sequence has no more sinks than tokens
int sinks_of(const gdr_attn_problem_t& p) { return p.sinks < p.seq_len ? p.sinks : (int)p.seq_len; }
Plan plan_of(const gdr_attn_problem_t& p) {
    Plan x{};
    const int64_t T = p.batch * p.seq_len, W = p.window;
    x.rows = up((size_t)T * p.num_q_heads * 8);
    x.tops = up((size_t)T * p.num_q_heads * 4);
    if (p.do_dtype != p.io_dtype) x.d_o16 = up((size_t)T * p.num_q_heads * p.head_dim_v * size_of(p.io_dtype));
    if (p.sinks > 0 && T > W) {
        const int64_t most = T / (W + 1), longer = most < p.num_seqs ? most : p.num_seqs;    // than a window
        // runs of 256 tokens at least, and up to 65 to a sequence or runs of 4,096
        const int64_t runs = T / 256 < 65 * longer + T / 4096 ? T / 256 : 65 * longer + T / 4096;
        x.slots = runs + 2 * longer + 1;
        x.table = up(((size_t)p.num_seqs + 1) * 4);
        const double rows = (double)x.slots * sinks_of(p) * p.num_kv_heads;      // more than a launch takes: any number
        x.part = up((rows < 0x1p40 ? (size_t)rows : (size_t)1 << 40) * (p.head_dim_qk + p.head_dim_v) * 4);
    }
    return x;
}

}  // namespace

size_t attn_bwd_workspace(const gdr_attn_problem_t& p) {
    const Plan x = plan_of(p);
    return x.rows + x.tops + x.d_o16 + x.table + x.part;
}

hipError_t launch_attn_bwd(const AttnArgs& in) {
    AttnArgs a = in;
    if (a.Ttot == 0) return hipSuccess;
    const Plan x = plan_of(a.p);
    a.p.sinks = sinks_of(a.p);
    char* ws = reinterpret_cast<char*>(a.ws);
    a.rows = reinterpret_cast<float*>(ws);
    a.tops = reinterpret_cast<float*>(ws += x.rows);
    ws += x.tops;
    a.d_o16 = x.d_o16 ? ws : nullptr;
    ws += x.d_o16;
    a.slots = x.slots ? reinterpret_cast<int32_t*>(ws) : nullptr;
    a.sink_part = x.slots ? reinterpret_cast<float*>(ws + x.table) : nullptr;
    a.max_slots = (int32_t)x.slots;
    const int G = group(a.p), Nk = a.p.num_kv_heads;
    const bool packed = a.cu != nullptr;
    hipError_t e = hipSuccess;
    by_dims(a.p, [&](auto type, auto dk, auto dv) {
        typedef decltype(type) T;
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value, NQ = 4, NK = 4, KB = 32 * NK;
        constexpr int QT = kQueryTile;
        const RowBlock rq = row_block(32 * NQ, G), rk = row_block(QT, G);
        const int64_t bq = token_blocks(a.p.batch, a.p.seq_len, a.p.num_seqs, packed, rq.TPB), wq = bq * Nk * rq.HC;
        const int64_t bk = token_blocks(a.p.batch, a.p.seq_len, a.p.num_seqs, packed, KB), wm = bk * Nk;
        const int64_t wk = wm + x.slots * Nk * (((int64_t)a.p.sinks + KB - 1) / KB);
        if (wq >= (int64_t)1 << 31 || wk >= (int64_t)1 << 31 || !grid_fits(wq + 8, 64 * NQ) || !grid_fits(wk + 8, 64 * NK)) {
            e = hipErrorInvalidConfiguration;
            return;
        }
        if (a.d_o16) {
            const int64_t n = a.Ttot * a.p.num_q_heads * a.p.head_dim_v, need = (n + 1023) / 1024, most = 8192;
            k_window_round<T><<<dim3((unsigned)(need < most ? need : most)), 256, 0, a.stream>>>((const float*)a.d_o,
                                                                                               (T*)a.d_o16, n);
            a.d_o = a.d_o16;
        }
        const dim3 gq((unsigned)((wq + 7) / 8 * 8)), gk((unsigned)((wm + 7) / 8 * 8 + wk - wm));
        auto go = [&](auto vec) {
            constexpr bool VEC = decltype(vec)::value;
            k_window_dq<T, DK, DV, NQ, VEC><<<gq, 64 * NQ, 0, a.stream>>>(a, rq, (int)bq, (int)wq);
            k_window_dkv<T, DK, DV, NK, VEC><<<gk, 64 * NK, 0, a.stream>>>(a, rk, (int)bk, (int)wm, (int)wk);
        };
        a.vec ? go(std::true_type{}) : go(std::false_type{});
        if (x.slots) k_window_sinks<T><<<dim3((unsigned)(x.slots * Nk)), 256, 0, a.stream>>>(a);
        e = hipGetLastError();
    });
    return e;
}

}  // namespace gdr
