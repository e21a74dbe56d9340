// Selective state space scan with a diagonal transition per channel
// (include/gdr_mixer.h): forward over packed sequences, and one token per
// sequence.
//
//   h_t[d][n] = exp(delta_t[d] A[d][n]) h_{t-1}[d][n] + delta_t[d] B_t[n] x_t[d]
//   y_t[d]    = (sum_n C_t[n] h_t[d][n] + D[d] x_t[d]) silu(z_t[d])
//
// The exponentials bound the forward pass: v_exp_f32 takes 8 cycles of a SIMD
// for a wavefront and every other operation 4, so a (token, channel, state)
// costs at least 24 (two products, exp, two fused multiply-adds) against 1 to 2
// bytes of x, dt, z and y at 16 states. The recurrence is serial in t, and few
// channels would leave the card idle; therefore the wavefronts of a workgroup
// take consecutive pieces of the same channels' time axis: h at the end of a
// piece is P h_in + h_loc with P = exp(A sum(delta)), so each runs its piece
// from a zero state (one more fused multiply-add an element; exp and
// delta B x stay in registers), publishes P and h_loc, and repeats the
// recurrence from the state its predecessors give.
//
// Layout: a wavefront holds 16 channels (lane & 15) by 4 state groups
// (lane >> 4) of SPL states: B and C are then LDS broadcasts, and the sum over
// states ends with three swaps and adds for four tokens, each lane left with
// one token's sum, which it finishes.
#include "gdr_scan.hpp"

namespace gdr {

namespace {

template <int SPL> constexpr int kFwdWaveFloats = kPiece<SPL> * (kCh * 2 + 8 * SPL);       // delta, delta x; B, C
template <int SPL> constexpr int kFwdPubFloats = 64 * 2 * SPL;                             // P and h_loc of a wavefront
template <int SPL> constexpr size_t fwd_lds(int nw) {
    return 4 * ((size_t)nw * (kFwdWaveFloats<SPL> + 2 * kFwdPubFloats<SPL>) + 2 * 64 * SPL);
}

// OT: type of y; GATE: z is there; SOFT: softplus of dt
template <typename T, typename OT, int SPL, bool GATE, bool SOFT>
__global__ __launch_bounds__(512, 2) void k_scan_fwd(ScanArgs a, Segments sg, int64_t lines, int cbg) {
    constexpr int L = kPiece<SPL>, K = L / 4, SP = 4 * SPL;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    int n, seg, g, cb;
    if (!unit_of(a, lines, cbg, sg.most, &n, &seg, &g, &cb)) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int Dg = a.p.channels / a.p.groups, S = a.p.state_dim;
    const bool act = cb * kCh + c < Dg;
    const int ch = g * Dg + (act ? cb * kCh + c : Dg - 1);
    float* sd = lds + wave * kFwdWaveFloats<SPL>;           // [L][16][2]
    float* sB = sd + L * kCh * 2;                           // [L][SP]
    float* sC = sB + L * SP;
    float* pub = lds + nw * kFwdWaveFloats<SPL>;            // [2][nw][2][64][SPL]
    float* carry = pub + 2 * nw * kFwdPubFloats<SPL>;       // [2][64][SPL]

    int64_t s, e;
    seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
    const int64_t seq = s;
    bool last;
    if (!sg.range(seg, &s, &e, &last)) return;
    float A2[SPL], h0[SPL];
    const int64_t st0 = ((int64_t)n * a.p.channels + ch) * S + q * SPL;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const bool in = act && q * SPL + i < S;
        A2[i] = in ? log2_rate(a.A[(int64_t)ch * S + q * SPL + i]) : 0.f;
        h0[i] = in && a.S0 ? a.S0[st0 + i] : 0.f;
    }
    sg.template enter<SPL>(n, seg, seq, a.p.channels, ch, q, A2, h0);
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.D ? a.D[ch] : 0.f;

    // this lane's tokens in a tile are wave L + 4 k + q
    const int row = wave * L, tile = nw * L;
    int ox[K], odt[K], oz[K], oy[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t r = row + 4 * k + q;
        ox[k] = act ? (int)((r * a.p.x_stride + ch) * (int)sizeof(T)) : kNowhere;
        odt[k] = act ? (int)((r * a.p.dt_stride + ch) * (int)sizeof(T)) : kNowhere;
        oz[k] = act ? (int)((r * a.p.z_stride + ch) * (int)sizeof(T)) : kNowhere;
        oy[k] = act ? (int)((r * a.p.channels + ch) * (int)sizeof(OT)) : kNowhere;
    }
    T rx[K], rdt[K], rz[K];
    StateRows<T, SPL, L> rB, rC;
    rB.init(a.p.b_stride, g * S, S, row);
    rC.init(a.p.c_stride, g * S, S, row);
    auto fetch = [&](int64_t tb) {
        const int64_t rows = e - tb < tile ? (e - tb > 0 ? e - tb : 0) : tile;
        const auto bx = token_rows<T>(a.x, tb, a.p.x_stride, rows), bdt = token_rows<T>(a.dt, tb, a.p.dt_stride, rows);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            rx[k] = buf_load<T>(bx, ox[k]);
            rdt[k] = buf_load<T>(bdt, odt[k]);
        }
        if (GATE) {
            const auto bz = token_rows<T>(a.z, tb, a.p.z_stride, rows);
#pragma unroll
            for (int k = 0; k < K; ++k) rz[k] = buf_load<T>(bz, oz[k]);
        }
        rB.load(token_rows<T>(a.B, tb, a.p.b_stride, rows));
        rC.load(token_rows<T>(a.C, tb, a.p.c_stride, rows));
    };
    fetch(s);
    int buf = 0;
    for (int64_t tb = s; tb < e; tb += tile, buf ^= 1) {
        const int left = (int)(e - tb < tile ? e - tb : tile);
        wave_lds_fence();
        float x[K], z[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = to_f(rx[k]);
            if (GATE) z[k] = to_f(rz[k]);
            float d = to_f(rdt[k]) + bias;
            if (SOFT) d = softplus(d);
            d = row + 4 * k + q < left ? d : 0.f;           // past the end: the state stays as it is
            *reinterpret_cast<f32x2*>(sd + ((4 * k + q) * kCh + c) * 2) = f32x2{d, d * x[k]};
        }
        rB.put(sB);
        rC.put(sC);
        wave_lds_fence();
        fetch(tb + tile);

        float ea[L][SPL], b[L][SPL], P[SPL], hl[SPL], sum = 0.f;
#pragma unroll
        for (int i = 0; i < SPL; ++i) hl[i] = 0.f;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const f32x2 d = *reinterpret_cast<const f32x2*>(sd + (j * kCh + c) * 2);
            float Bv[SPL];
            read_vec(sB + j * SP + q * SPL, Bv);
            sum += d[0];
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                ea[j][i] = __builtin_amdgcn_exp2f(A2[i] * d[0]);
                b[j][i] = d[1] * Bv[i];
                hl[i] = __builtin_fmaf(ea[j][i], hl[i], b[j][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < SPL; ++i) P[i] = __builtin_amdgcn_exp2f(A2[i] * sum);
        float* all = pub + buf * nw * kFwdPubFloats<SPL> + lane * SPL;
        write_vec(all + wave * kFwdPubFloats<SPL>, P);
        write_vec(all + wave * kFwdPubFloats<SPL> + 64 * SPL, hl);
        lds_barrier();
        if (tb != s) read_vec(carry + (buf ^ 1) * 64 * SPL + lane * SPL, h0);
        join_pieces<SPL, true>(all, kFwdPubFloats<SPL>, 64 * SPL, 0, wave, h0);
        loads_arrived();
        const auto by = token_rows<OT>(a.y, tb, a.p.channels, left);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float y[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int j = 4 * k + m;
                float Cv[SPL];
                read_vec(sC + j * SP + q * SPL, Cv);
                y[m] = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    h0[i] = __builtin_fmaf(ea[j][i], h0[i], b[j][i]);
                    y[m] = __builtin_fmaf(Cv[i], h0[i], y[m]);
                }
            }
            float v = __builtin_fmaf(skip, x[k], rows_sum4(y));
            if (GATE) v *= silu(z[k]);
            buf_store<OT>(by, oy[k], v);
        }
        if (wave == nw - 1) write_vec(carry + buf * 64 * SPL + lane * SPL, h0);
    }
    if (a.ST && act && last && wave == nw - 1) {
#pragma unroll
        for (int i = 0; i < SPL; ++i)
            if (q * SPL + i < S) a.ST[st0 + i] = h0[i];
    }
}

// One token of every sequence: the state's bytes bound it, so it moves once, 16
// bytes a lane. LC lanes hold the states of a channel, 4 each. WIDE: state_dim is a
// multiple of 4; ONCE: the state moves past the caches.
template <typename T, int LC, bool WIDE, bool ONCE>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a, int64_t nch) {
    const int l = threadIdx.x % LC;
    const int64_t i = (int64_t)blockIdx.x * (256 / LC) + threadIdx.x / LC;     // (sequence, channel)
    if (i >= nch) return;                                  // whole groups of LC lanes
    const int D = a.p.channels, S = a.p.state_dim, Dg = D / a.p.groups;
    const int64_t n = i / D;
    const int ch = (int)(i % D), g = ch / Dg, s0 = l * 4;
    float* st = a.state + i * S + s0;
    const float* Ap = a.A + (int64_t)ch * S + s0;
    const T* Bp = (const T*)a.B + n * a.p.b_stride + (int64_t)g * S + s0;
    const T* Cp = (const T*)a.C + n * a.p.c_stride + (int64_t)g * S + s0;
    float h[4] = {}, A[4] = {}, B[4] = {}, C[4] = {};
    if (WIDE) {
        if (s0 < S) {
            unpack<float, 4>(load_raw<float, 4, ONCE>(st), h);
            unpack<float, 4>(load_raw<float, 4>(Ap), A);
            unpack<T, 4>(load_raw<T, 4>(Bp), B);
            unpack<T, 4>(load_raw<T, 4>(Cp), C);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (s0 + j < S) {
                h[j] = st[j];
                A[j] = Ap[j];
                B[j] = to_f(Bp[j]);
                C[j] = to_f(Cp[j]);
            }
    }
    const float x = to_f(((const T*)a.x)[n * a.p.x_stride + ch]);
    float d = to_f(((const T*)a.dt)[n * a.p.dt_stride + ch]) + (a.dt_bias ? a.dt_bias[ch] : 0.f);
    if (a.p.dt_softplus) d = softplus(d);
    const float dx = d * x;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(log2_rate(A[j]) * d), h[j], dx * B[j]);
        y = __builtin_fmaf(C[j], h[j], y);
    }
    if (WIDE) {
        if (s0 < S) store_vec<float, 4, ONCE>(st, h);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (s0 + j < S) st[j] = h[j];
    }
#pragma unroll
    for (int m = 1; m < LC; m <<= 1) y += __shfl_xor(y, m, 64);
    if (l == 0) {
        y = __builtin_fmaf(a.D ? a.D[ch] : 0.f, x, y);
        if (a.z) y *= silu(to_f(((const T*)a.z)[n * a.p.z_stride + ch]));
        store_as<T>(a.y, i, y, a.p.out_dtype == GDR_F32);
    }
}

// Units of whole sequences.
int64_t units_of(const gdr_scan_problem_t& p) {
    return (int64_t)p.num_seqs * p.groups * ((p.channels / p.groups + kCh - 1) / kCh);
}
template <int SPL> constexpr int kMostWaves = SPL == 16 ? 4 : 8;

template <int SPL>
size_t ends_bytes(const gdr_scan_problem_t& p, size_t* sums) {
    const size_t slots = segment_slots(units_of(p), kMostWaves<SPL>, p.num_seqs);
    *sums = (slots * p.channels * 4 * SPL * 4 + 255) & ~(size_t)255;
    return *sums + slots * p.channels * 4;
}

template <typename T, int SPL>
hipError_t fwd(const ScanArgs& a) {
    constexpr int most = kMostWaves<SPL>;
    static_assert(fwd_lds<SPL>(most) <= 160 * 1024, "LDS of a compute unit");
    const int cbg = (a.p.channels / a.p.groups + kCh - 1) / kCh;
    const int64_t whole = units_of(a.p);
    Segments sg = segments_for(whole, most, a.max_len);
    const int64_t units = whole * sg.most;
    // 2048 wavefronts fill the card at two a SIMD (16 sequences of 512 tokens and 2,048 channels: 95 us, with twice as
    // many 105; 4 of 1,024 tokens and 32 states: 90 and 104); ragged sequences take 4096, for the longest one is a chain
    // that the others do not shorten (13 of 4,099 tokens, the longest 1,272, fp32: 88 us, with 2048 143; 20 of 16,384,
    // the longest 2,523: 108 and 160). Many of few states are the exception (24 of 6,000 tokens, 640 channels and 8
    // states: 37 and 27).
    const int fill = a.max_len * a.p.num_seqs > 2 * a.Ttot ? 4096 : 2048;
    const int nw = waves_for(units, sg.most > 1 ? sg.len : a.max_len, kPiece<SPL>, fill, 1, most);
    const int64_t lines = line_units((int64_t)a.p.num_seqs * a.p.groups * sg.most, cbg), blocks = unit_blocks(lines);
    if (!grid_fits(blocks, 64 * nw)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks);
    hipError_t e = hipSuccess;
    if (sg.most > 1) {
        size_t sums;
        ends_bytes<SPL>(a.p, &sums);
        sg.end = reinterpret_cast<float*>(a.ws);
        sg.sum = reinterpret_cast<float*>(a.ws + sums);
        if (a.p.dt_softplus) k_scan_states<T, SPL, true, true><<<grid, 64 * nw, states_lds<SPL>(nw), a.stream>>>(a, sg, nullptr, lines, cbg, 1);
        else k_scan_states<T, SPL, false, true><<<grid, 64 * nw, states_lds<SPL>(nw), a.stream>>>(a, sg, nullptr, lines, cbg, 1);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    auto go = [&](auto out, auto gate, auto soft) {
        k_scan_fwd<T, decltype(out), SPL, decltype(gate)::value, decltype(soft)::value>
            <<<grid, 64 * nw, fwd_lds<SPL>(nw), a.stream>>>(a, sg, lines, cbg);
    };
    auto by_gate = [&](auto out, auto soft) { a.z ? go(out, std::true_type{}, soft) : go(out, std::false_type{}, soft); };
    auto by_out = [&](auto soft) { a.p.out_dtype == GDR_F32 ? by_gate(float{}, soft) : by_gate(T{}, soft); };
    if (a.p.dt_softplus) by_out(std::true_type{});
    else by_out(std::false_type{});
    return hipGetLastError();
}

template <typename T, bool WIDE>
hipError_t step(const ScanArgs& a) {
    const int64_t nch = (int64_t)a.p.num_seqs * a.p.channels;
    auto go = [&](auto lanes) {
        constexpr int LC = decltype(lanes)::value;
        const int64_t blocks = (nch + 256 / LC - 1) / (256 / LC);
        if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
        if (blocks == 0) return hipSuccess;
        // A state counts twice, read and written, since a model steps several in turn: three of 256 sequences (64 MB each)
        // 30 us from the caches, past them 33, of 520 62 and 58, of 1,024 122 and 113. (One alone would stay in the caches
        // up to 256 MB: 520 sequences 50 and 59, 1,024 123 and 112.)
        if (beyond_caches(8 * nch * a.p.state_dim)) k_scan_step<T, LC, WIDE, true><<<dim3((unsigned)blocks), 256, 0, a.stream>>>(a, nch);
        else k_scan_step<T, LC, WIDE, false><<<dim3((unsigned)blocks), 256, 0, a.stream>>>(a, nch);
        return hipGetLastError();
    };
    const int need = (a.p.state_dim + 3) / 4;
    if (need <= 1) return go(std::integral_constant<int, 1>{});
    if (need <= 2) return go(std::integral_constant<int, 2>{});
    if (need <= 4) return go(std::integral_constant<int, 4>{});
    if (need <= 8) return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 16>{});
}

}  // namespace

size_t scan_fwd_workspace(const gdr_scan_problem_t& p) {
    return by_state_dim(p.state_dim, [&](auto spl) {
        constexpr int SPL = decltype(spl)::value;
        size_t sums;
        return segment_slots(units_of(p), kMostWaves<SPL>, p.num_seqs) ? ends_bytes<SPL>(p, &sums) : (size_t)0;
    });
}

hipError_t launch_scan_fwd(const ScanArgs& a) {
    if (a.p.num_seqs == 0) return hipSuccess;
    return by_states(a, [&](auto type, auto spl) { return fwd<decltype(type), decltype(spl)::value>(a); });
}

hipError_t launch_scan_step(const ScanArgs& a) {
    const bool wide = a.p.state_dim % 4 == 0;
    if (a.p.io_dtype == GDR_BF16) return wide ? step<bf16, true>(a) : step<bf16, false>(a);
    return wide ? step<float, true>(a) : step<float, false>(a);
}

}  // namespace gdr
