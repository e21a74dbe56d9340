// What the scan's forward and backward kernels share.
#pragma once

#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

constexpr int kCh = 16;                                    // channels of a wavefront

// Tokens a wavefront of the forward kernels takes at a time: SPL * piece
// exponentials and as many products stay in registers.
template <int SPL> constexpr int kPiece = SPL <= 4 ? 16 : SPL <= 8 ? 8 : 4;

// A log2 e, finite where A is -inf or near the lowest float: tokens past a
// sequence's end multiply it by a delta of zero. NaN stays.
__device__ __forceinline__ float log2_rate(float A) {
    const float r = A * kLog2e;
    return r < -__FLT_MAX__ ? -__FLT_MAX__ : r;
}
__device__ __forceinline__ void swap32(float& a, float& b) {   // a = {a.lo, b.lo}, b = {a.hi, b.hi} (halves of 32 lanes)
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap16(float& a, float& b) {   // the same with odd and even rows of 16 lanes
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
// v[i] summed over the four rows of 16 lanes; row i keeps the sum of v[i]
__device__ __forceinline__ float rows_sum4(float (&v)[4]) {
    swap32(v[0], v[2]);
    swap32(v[1], v[3]);
    float a = v[0] + v[2], b = v[1] + v[3];
    swap16(a, b);
    return a + b;
}

// the wavefront's number in its workgroup, as a scalar
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// LDS written by some lanes of a wavefront is read by others of the same one:
// its LDS operations complete in order; this keeps the compiler from moving them.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// The sequence of rank r by length, the longest first (the first 64 lengths fit a
// wavefront's lanes; more sequences stay in their order). All lanes call it.
__device__ __forceinline__ int by_length(const int32_t* cu, int N, int r) {
    if (!cu || N > 64) return r;
    const int lane = threadIdx.x & 63;
    const int len = lane < N ? cu[lane + 1] - cu[lane] : -1;
    int rank = 0;
    for (int j = 0; j < N; ++j) {
        const int l = __builtin_amdgcn_readlane(len, j);
        rank += l > len || (l == len && j < lane);
    }
    return __ffsll((unsigned long long)__ballot(lane < N && rank == r)) - 1;
}

// Workgroup -> (sequence, segment, group, channel block). Workgroups are dealt to
// the eight XCDs in turn; kLine consecutive channel blocks, whose rows share
// 128-byte lines, go to the same one, so that the lines meet in one L2 (8,192 tokens
// of 4,096 channels and 16 states: 198 us, dealt one by one 213). Long sequences
// start first: 13 of 4,099 tokens, the longest 1,272, take 82 us instead of 130 in
// their order.
constexpr int kLine = 4;
inline int64_t line_units(int64_t seqs_segments_groups, int cbg) { return seqs_segments_groups * ((cbg + kLine - 1) / kLine); }
inline int64_t unit_blocks(int64_t lines) { return (lines + 7) / 8 * 8 * kLine; }
__device__ __forceinline__ bool unit_of(const ScanArgs& a, int64_t lines, int cbg, int nseg, int* n, int* seg, int* g,
                                        int* cb) {
    const int64_t i = blockIdx.x / (8 * kLine) * 8 + blockIdx.x % 8;
    const int lgs = (cbg + kLine - 1) / kLine;
    *cb = (int)(i % lgs) * kLine + (int)(blockIdx.x / 8 % kLine);
    if (i >= lines || *cb >= cbg) return false;
    const int64_t v = i / lgs;
    *g = (int)(v % a.p.groups);
    *seg = (int)(v / a.p.groups % nseg);
    *n = by_length(a.cu, a.p.num_seqs, (int)(v / a.p.groups / nseg));
    return true;
}

// Slot of a sequence's first tile (or segment) of `tile` tokens: floor(s / tile) + n
// leaves room for the partial ones of the sequences before it.
__device__ __forceinline__ int64_t first_slot(int64_t s, int tile, int n) {
    return (int64_t)((uint32_t)s / (uint32_t)tile) + n;
}

// Rows of a token tensor from token t on, `rows` of them: a buffer whose accesses
// past its end read zero and store nothing, so that the tokens behind a sequence
// need no branches. Offsets inside are bytes, (token - t) * stride + element.
constexpr int kNowhere = 0x7fffffff;                       // an offset past the end of any of them
static_assert(128 * kMostTileStride * 4 <= kNowhere, "a tile of 128 tokens");
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_rows(const void* base, int64_t t, int64_t stride, int64_t rows) {
    return buf_rsrc((const T*)base + t * stride, (uint32_t)(rows * stride * (int64_t)sizeof(T)));
}
template <typename T>
__device__ __forceinline__ T buf_load(__amdgpu_buffer_rsrc_t rs, int off) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0));
    else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
}
template <typename T>
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t rs, int off, float v) {
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, to_t<T>(v)), rs, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, to_t<T>(v)), rs, off, 0, 0);
}

// The rows of B (or C) of a wavefront's L tokens, the first at row `row` of the
// buffer, into LDS as [token][4 SPL] fp32, zero past the sequence and past state_dim.
template <typename T, int SPL, int L>
struct StateRows {
    static constexpr int SP = 4 * SPL, PER = (L * SP + 63) / 64;
    int off[PER];
    T r[PER];
    __device__ __forceinline__ void init(int64_t stride, int first, int S, int row) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = i * 64 + lane, n = idx % SP;
            off[i] = n < S && idx < L * SP ? (int)(((row + idx / SP) * stride + first + n) * (int)sizeof(T)) : kNowhere;
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs) {
#pragma unroll
        for (int i = 0; i < PER; ++i) r[i] = buf_load<T>(rs, off[i]);
    }
    __device__ __forceinline__ void put(float* lds) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (L * SP % 64 == 0 || i * 64 + lane < L * SP) lds[i * 64 + lane] = to_f(r[i]);
    }
};

template <int N>
__device__ __forceinline__ void read_vec(const float* p, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = w[j];
        }
    } else {
        static_assert(N % 2 == 0, "state group");
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const f32x2 w = *reinterpret_cast<const f32x2*>(p + i);
            v[i] = w[0];
            v[i + 1] = w[1];
        }
    }
}
template <int N>
__device__ __forceinline__ void write_vec(float* p, const float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) *reinterpret_cast<f32x2*>(p + i) = f32x2{v[i], v[i + 1]};
    }
}

// Waits for the loads in flight (the next tile's), before this tile's stores join
// them: vector memory completes in order, so a wait at their use would be one for
// the stores too.
__device__ __forceinline__ void loads_arrived() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// v <- P v + x for the pieces [w0, w1) in order (FORWARD) or from the last to the
// first: P and x of piece w at pub + w * stride, + off. The values of
// several pieces are on their way together.
template <int N, bool FORWARD>
__device__ __forceinline__ void join_pieces(const float* pub, int stride, int off, int w0, int w1, float (&v)[N]) {
    constexpr int B = N < 16 ? 16 / N : 1;
    for (int i0 = 0; i0 < w1 - w0; i0 += B) {
        float P[B][N], x[B][N];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (i0 + k >= w1 - w0) break;
            const float* p = pub + (FORWARD ? w0 + i0 + k : w1 - 1 - i0 - k) * stride;
            read_vec(p, P[k]);
            read_vec(p + off, x[k]);
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (i0 + k >= w1 - w0) break;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __builtin_fmaf(P[k][i], v[i], x[k][i]);
        }
    }
}

// Sequences cut into segments of `len` tokens that run side by side (most == 1:
// not cut). A segment's end from a zero state and the sum of its deltas give the
// state behind it, P h + end with P = exp(A sum), so that a first pass over the
// segments lets a second one start each from its true state.
struct Segments {
    int len, most;             // tokens a segment; segments of the longest sequence
    float* end;                // [Ttot / len + N][D][4 SPL]
    float* sum;                // [Ttot / len + N][D]
    // the tokens of segment `seg`; false: the sequence has no such segment (the first one always is)
    __device__ __forceinline__ bool range(int seg, int64_t* s, int64_t* e, bool* last) const {
        *last = true;
        if (most == 1) return true;
        const int64_t b = *s + (int64_t)seg * len;
        if (seg > 0 && b >= *e) return false;
        *last = b + len >= *e;
        *s = b;
        *e = *last ? *e : b + len;
        return true;
    }
    // h: the initial state -> the state before segment `seg` of the sequence that starts at token s
    template <int SPL>
    __device__ __forceinline__ void enter(int n, int seg, int64_t s, int D, int ch, int q, const float (&A2)[SPL],
                                          float (&h)[SPL]) const {
        if (most == 1) return;
        const int64_t slot = first_slot(s, len, n);
#pragma unroll 4
        for (int i = 0; i < seg; ++i) through<SPL>(slot + i, D, ch, q, A2, h);
    }
    // h <- P h + end of one segment
    template <int SPL>
    __device__ __forceinline__ void through(int64_t slot, int D, int ch, int q, const float (&A2)[SPL],
                                            float (&h)[SPL]) const {
        float x[SPL];
        read_vec(end + (slot * D + ch) * 4 * SPL + q * SPL, x);
        const float d = sum[slot * D + ch];
#pragma unroll
        for (int k = 0; k < SPL; ++k) h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[k] * d), h[k], x[k]);
    }
    // Stores a segment's end, which wavefront `holder` has in h, and the sum over the wavefronts of `total`.
    template <int SPL>
    __device__ __forceinline__ void leave(int n, int seg, int64_t s, int D, int ch, int q, bool act, int wave, int nw,
                                          int holder, const float (&h)[SPL], float total, float* lds) const {
        const int lane = threadIdx.x & 63;
        const int64_t slot = first_slot(s, len, n) + seg;
        lds_barrier();
        lds[wave * 64 + lane] = total;
        lds_barrier();
        if (wave != holder || !act) return;
        float v = 0.f;
        for (int w = 0; w < nw; ++w) v += lds[w * 64 + lane];
        write_vec(end + (slot * D + ch) * 4 * SPL + q * SPL, h);
        if (q == 0) sum[slot * D + ch] = v;
    }
};

// The recurrence without outputs. ENDS: over every segment but a sequence's last,
// from a zero state, for `sg`'s ends; else from the initial state (joined from the
// ends), storing the state before every tile of btile tokens.
template <typename T, int SPL, bool SOFT, bool ENDS>
__global__ __launch_bounds__(512) void k_scan_states(ScanArgs a, Segments sg, float* states, int64_t lines, int cbg,
                                                     int btile) {
    constexpr int L = kPiece<SPL>, K = L / 4, SP = 4 * SPL;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    int n, seg, g, cb;
    if (!unit_of(a, lines, cbg, sg.most, &n, &seg, &g, &cb)) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int Dg = a.p.channels / a.p.groups, S = a.p.state_dim;
    const bool act = cb * kCh + c < Dg;
    const int ch = g * Dg + (act ? cb * kCh + c : Dg - 1);
    float* sd = lds + wave * (L * kCh * 2 + L * SP);
    float* sB = sd + L * kCh * 2;
    float* pub = lds + nw * (L * kCh * 2 + L * SP);         // [2][nw][2][64][SPL]
    float* carry = pub + 2 * nw * 128 * SPL;                // [2][64][SPL]
    int64_t s, e;
    seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
    const int64_t seq = s;
    bool last;
    if (!sg.range(seg, &s, &e, &last) || (ENDS && last)) return;
    float A2[SPL], h0[SPL], total = 0.f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const bool in = act && q * SPL + i < S;
        A2[i] = in ? log2_rate(a.A[(int64_t)ch * S + q * SPL + i]) : 0.f;
        h0[i] = !ENDS && in && a.S0 ? a.S0[((int64_t)n * a.p.channels + ch) * S + q * SPL + i] : 0.f;
    }
    if (!ENDS) sg.template enter<SPL>(n, seg, seq, a.p.channels, ch, q, A2, h0);
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f;
    const int row = wave * L, tile = nw * L;
    int ox[K], odt[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t r = row + 4 * k + q;
        ox[k] = act ? (int)((r * a.p.x_stride + ch) * (int)sizeof(T)) : kNowhere;
        odt[k] = act ? (int)((r * a.p.dt_stride + ch) * (int)sizeof(T)) : kNowhere;
    }
    T rx[K], rdt[K];
    StateRows<T, SPL, L> rB;
    rB.init(a.p.b_stride, g * S, S, row);
    auto fetch = [&](int64_t tb) {
        const int64_t rows = e - tb < tile ? (e - tb > 0 ? e - tb : 0) : tile;
        const auto bx = token_rows<T>(a.x, tb, a.p.x_stride, rows), bdt = token_rows<T>(a.dt, tb, a.p.dt_stride, rows);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rx[k] = buf_load<T>(bx, ox[k]);
            rdt[k] = buf_load<T>(bdt, odt[k]);
        }
        rB.load(token_rows<T>(a.B, tb, a.p.b_stride, rows));
    };
    fetch(s);
    const int64_t slot = first_slot(seq, btile, n);
    int buf = 0;
    for (int64_t tb = s; tb < e; tb += tile, buf ^= 1) {
        const int left = (int)(e - tb < tile ? e - tb : tile);
        wave_lds_fence();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float x = to_f(rx[k]);
            float d = to_f(rdt[k]) + bias;
            if (SOFT) d = softplus(d);
            d = row + 4 * k + q < left ? d : 0.f;
            *reinterpret_cast<f32x2*>(sd + ((4 * k + q) * kCh + c) * 2) = f32x2{d, d * x};
        }
        rB.put(sB);
        wave_lds_fence();
        fetch(tb + tile);
        float P[SPL], hl[SPL], sum = 0.f;
#pragma unroll
        for (int i = 0; i < SPL; ++i) hl[i] = 0.f;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const f32x2 d = *reinterpret_cast<const f32x2*>(sd + (j * kCh + c) * 2);
            float Bv[SPL];
            read_vec(sB + j * SP + q * SPL, Bv);
            sum += d[0];
#pragma unroll
            for (int i = 0; i < SPL; ++i)
                hl[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[i] * d[0]), hl[i], d[1] * Bv[i]);
        }
        total += sum;
#pragma unroll
        for (int i = 0; i < SPL; ++i) P[i] = __builtin_amdgcn_exp2f(A2[i] * sum);
        float* all = pub + buf * nw * 128 * SPL + lane * SPL;
        write_vec(all + wave * 128 * SPL, P);
        write_vec(all + wave * 128 * SPL + 64 * SPL, hl);
        lds_barrier();
        if (tb != s) read_vec(carry + (buf ^ 1) * 64 * SPL + lane * SPL, h0);
        join_pieces<SPL, true>(all, 128 * SPL, 64 * SPL, 0, wave, h0);
        loads_arrived();
        // a backward tile starts with this piece (pieces are whole parts of a tile, or the tile is all there is)
        const int at = (int)(tb - seq) + row;
        if (!ENDS && at % btile == 0 && row < left && act)
            write_vec(states + ((slot + at / btile) * a.p.channels + ch) * SP + q * SPL, h0);
        if (wave == nw - 1) {
#pragma unroll
            for (int i = 0; i < SPL; ++i) h0[i] = __builtin_fmaf(P[i], h0[i], hl[i]);
            write_vec(carry + buf * 64 * SPL + lane * SPL, h0);
        }
    }
    if (ENDS) sg.template leave<SPL>(n, seg, seq, a.p.channels, ch, q, act, wave, nw, nw - 1, h0, total, lds);
}

// ---------------------------------------------------------------- host
// Segments where whole sequences leave more than half of 2048 wavefronts idle: as
// many as fill them, of 256 tokens or more. The work of the recurrence is done
// twice then: 16,384 tokens of 512 channels and 16 states take 93 us instead of
// 345, 8,192 of them backward 175 instead of 725. Two segments: 8,192 tokens of
// 2,048 channels 170 instead of 184, backward 654 instead of 746; near the least
// length they cost a little forward (512 tokens 19 instead of 17, backward 64).
constexpr int kMostSegments = 64;
inline int most_segments(int64_t units, int nw) {
    const int64_t want = units > 0 ? 2048 / (units * nw) : 0;
    return (int)(want < 2 ? 1 : want > kMostSegments ? kMostSegments : want);
}
inline Segments segments_for(int64_t units, int nw, int64_t max_len) {
    Segments sg{0, 1, nullptr, nullptr};
    int64_t want = most_segments(units, nw);
    want = want < max_len / 256 ? want : max_len / 256;
    if (want < 2) return sg;
    sg.len = (int)(((max_len + want - 1) / want + 127) / 128 * 128);   // whole tiles of every kernel
    sg.most = (int)((max_len + sg.len - 1) / sg.len);
    return sg;
}
// Slots that the segments of any sequences of these sizes need: at most `most` for
// a sequence and one more left free, and the last sequence's wherever it starts.
inline int64_t segment_slots(int64_t units, int nw, int64_t N) {
    const int most = most_segments(units, nw);
    return most < 2 ? 0 : N * (most + 1) + most;
}

// Wavefronts of a workgroup, a power of two: as many as make `fill` in all units
// together, at least `least`, no more than pieces in the longest sequence or than `most`.
inline int waves_for(int64_t units, int64_t max_len, int piece, int fill, int least, int most) {
    int nw = 1;
    while (nw < most && (int64_t)nw * piece < max_len && (nw < least || units * nw < fill)) nw *= 2;
    return nw;
}

template <int SPL> constexpr size_t states_lds(int nw) {
    return 4 * ((size_t)nw * (kPiece<SPL> * (kCh * 2 + 4 * SPL) + 2 * 128 * SPL) + 2 * 64 * SPL);
}

// f(states a lane). Six of them for 17 to 24 states: 4,099 tokens of 1,540 channels and 24 states take 82 us, padded to
// 32 states 91; 4 x 2,048 tokens of 1,365 channels backward 649 and 1,202.
template <typename F>
auto by_state_dim(int S, F f) {
    if (S <= 8) return f(std::integral_constant<int, 2>{});
    if (S <= 16) return f(std::integral_constant<int, 4>{});
    if (S <= 24) return f(std::integral_constant<int, 6>{});
    if (S <= 32) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}
template <typename F>
hipError_t by_states(const ScanArgs& a, F f) {
    return by_state_dim(a.p.state_dim, [&](auto spl) {
        return a.p.io_dtype == GDR_BF16 ? f(bf16{}, spl) : f(float{}, spl);
    });
}

}  // namespace gdr
