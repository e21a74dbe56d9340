// Backward pass of the selective state space scan (include/gdr_mixer.h).
//
// With ds = d_y silu(z) and g_t the gradient of h_t,
//   g_t = ds_t C_t + G_t,   G_{t-1} = exp(delta_t A) g_t   (G behind the last token: d_final_state)
//   dC_t = sum_d ds h,  dB_t = sum_d g delta x,  dx = delta sum_n g B + D ds,
//   d delta = x sum_n g B + sum_n g p A,  dA = sum_t g p delta,  p_t = exp(delta_t A) h_{t-1}.
//
// k_scan_states runs the recurrence once and stores the state before every tile
// of tokens. k_scan_bwd takes the tiles of 16 J channels from the last to the
// first; within a tile the wavefronts take consecutive pieces of L tokens, whose
// exponentials and states stay in registers. Forward, a piece's entering state
// comes from the tile's state and its predecessors' (P, h_loc); in reverse, its
// incoming G from the later tile's and its successors' (P, G_loc): G at the
// start of a piece is P G_in + G_loc.
//
// Layout: state group on lane bits 0 and 1, channel on bits 2 to 5 (and J of them
// in a lane). The sums over channels (dB and dC, 2 SPL values a token) take swaps
// and adds over bits 5 and 4, each halving the values, and row rotations by 4 and
// 8; those over states take quad permutes. (The sums over channels as products
// with columns of an identity on the fp32 matrix cores were slower, 463 us
// against 395 at 4 x 2,048 x 2,048 x 16: eight 32-cycle products a token.)
//
// dB and dC of a token sum over all channels of a group: every workgroup stores
// its channels' sums and k_sum_partials joins them in a fixed order.
#include "gdr_scan.hpp"

namespace gdr {

namespace {

// Variants by states a lane: J channels a lane, L tokens a piece, at most NW
// wavefronts, and at least LEAST of them where a sequence has the pieces (the
// states before the tiles are written and read once more). The exponentials and
// states of a piece take 2 SPL J L registers, and what does not fit goes to
// scratch. 4 x 2,048 tokens, gated, bf16, of 4,096 channels and 8 states, 2,048 and
// 16, 1,365 and 24, 1,024 and 32, 512 and 64: 427, 371, 649, 630 and 897 us. With one
// channel a lane at 8 states 480, two at 16 983; pieces of 8 tokens at 24 and 32
// states 1,112 and 1,178; 64 states at two wavefronts a SIMD 2,743. Still in scratch,
// with a gate: 28 to 36 bytes a lane at up to 8 states (with softplus), 156 to 168 at
// 25 to 32, 52 to 72 at 33 to 64.
template <int SPL> struct Bwd {
    static constexpr int J = SPL <= 2 ? 2 : 1, L = SPL <= 4 ? 8 : 4, NW = SPL <= 8 ? 8 : 4, LEAST = 4;
    static constexpr int EPT = SPL * J, SP = 4 * SPL, CHB = kCh * J;
    static constexpr int TOK = CHB * 4 + 8;                           // floats of a token's row: its 4 writers on other banks
    static constexpr int kWaveFloats = L * TOK + 2 * L * SP;      // (delta, delta x, ds, -); B, C
    static constexpr int kPubFloats = 3 * 64 * EPT;                   // P, h_loc, G_loc
    // Idle lanes' offset, to which the distance of later tokens is added: past the end
    // of the rows of a tile, and within an int after the additions.
    static constexpr int IDLE = 1 << 30;
    static_assert(NW * L * kMostTileStride * 4 <= IDLE, "rows of a tile");
    static_assert(IDLE + (L / 4 - 1) * 4 * kMostTileStride * 4 <= 0x7fffffff, "offsets of the tokens of an idle lane");
    static constexpr size_t lds(int nw) { return 4 * ((size_t)nw * (kWaveFloats + 2 * kPubFloats) + 2 * 64 * EPT); }
};

struct ScanBwdWs {
    float* states;             // [Ttot / tile + N][D][4 SPL] states before the tiles
    float* bc;                 // [channel blocks of a group][2][Ttot][groups][S]: dB, dC
    float* par;                // [N][segments]: dA [D][S], dD [D], ddt_bias [D]
};

// own + x of another lane
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x, float own) {
    return own + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// over lane bits 0 and 1, the state groups
__device__ __forceinline__ float sum_states(float x) {
    x = add_dpp<0x4e>(x, x);
    return add_dpp<0xb1>(x, x);
}
// over lane bits 2 and 3, the last four channels of a row
__device__ __forceinline__ float sum_row(float x) {
    x = add_dpp<0x124>(x, x);
    return add_dpp<0x128>(x, x);
}
// v[i] summed over the four state groups; lanes of group q keep the sum of v[q]
__device__ __forceinline__ float states_sum4(const float (&v)[4], int q) {
    const bool hi = q & 2, odd = q & 1;
    const float a = add_dpp<0x4e>(hi ? v[0] : v[2], hi ? v[2] : v[0]);      // v[0] or v[2] of groups q and q ^ 2
    const float b = add_dpp<0x4e>(hi ? v[1] : v[3], hi ? v[3] : v[1]);
    return add_dpp<0xb1>(odd ? a : b, odd ? b : a);
}

// G at the start of every segment but a sequence's first from zero behind it, and
// the sum of its deltas: the recurrence backwards, G <- exp(delta A) (ds C + G).
template <typename T, int SPL, bool GATE, bool SOFT>
__global__ __launch_bounds__(512) void k_scan_grad_ends(ScanArgs a, Segments sg, int64_t lines, int cbg) {
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
    float* sC = sd + L * kCh * 2;
    float* pub = lds + nw * (L * kCh * 2 + L * SP);         // [2][nw][2][64][SPL]
    float* carry = pub + 2 * nw * 128 * SPL;                // [2][64][SPL]
    int64_t s, e;
    seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
    const int64_t seq = s;
    bool last;
    if (!sg.range(seg, &s, &e, &last) || seg == 0) return;
    float A2[SPL], G[SPL], total = 0.f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = act && q * SPL + i < S ? log2_rate(a.A[(int64_t)ch * S + q * SPL + i]) : 0.f;
        G[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f;
    const int dy32 = a.p.dy_dtype == GDR_F32, row = wave * L, tile = nw * L;
    const int ntiles = (int)((uint32_t)(e - s + tile - 1) / (uint32_t)tile);
    StateRows<T, SPL, L> rC;
    rC.init(a.p.c_stride, g * S, S, row);
    int buf = 0;
    for (int it = ntiles - 1; it >= 0; --it, buf ^= 1) {
        const int64_t tb = s + (int64_t)it * tile;
        const int left = (int)(e - tb < tile ? e - tb : tile);
        rC.load(token_rows<T>(a.C, tb, a.p.c_stride, left));
        wave_lds_fence();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = tb + row + 4 * k + q;
            float d = 0.f, ds = 0.f;
            if (act && row + 4 * k + q < left) {
                d = to_f(((const T*)a.dt)[t * a.p.dt_stride + ch]) + bias;
                if (SOFT) d = softplus(d);
                ds = load_as<T>(a.d_y, t * a.p.channels + ch, dy32);
                if (GATE) ds *= silu(to_f(((const T*)a.z)[t * a.p.z_stride + ch]));
            }
            *reinterpret_cast<f32x2*>(sd + ((4 * k + q) * kCh + c) * 2) = f32x2{d, ds};
        }
        rC.put(sC);
        wave_lds_fence();
        float P[SPL], Gl[SPL], sum = 0.f;
#pragma unroll
        for (int i = 0; i < SPL; ++i) Gl[i] = 0.f;
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const f32x2 d = *reinterpret_cast<const f32x2*>(sd + (j * kCh + c) * 2);
            float Cv[SPL];
            read_vec(sC + j * SP + q * SPL, Cv);
            sum += d[0];
#pragma unroll
            for (int i = 0; i < SPL; ++i)
                Gl[i] = __builtin_amdgcn_exp2f(A2[i] * d[0]) * __builtin_fmaf(d[1], Cv[i], Gl[i]);
        }
        total += sum;
#pragma unroll
        for (int i = 0; i < SPL; ++i) P[i] = __builtin_amdgcn_exp2f(A2[i] * sum);
        float* all = pub + buf * nw * 128 * SPL + lane * SPL;
        write_vec(all + wave * 128 * SPL, P);
        write_vec(all + wave * 128 * SPL + 64 * SPL, Gl);
        lds_barrier();
        if (wave == 0) {
            if (it != ntiles - 1) read_vec(carry + (buf ^ 1) * 64 * SPL + lane * SPL, G);
            join_pieces<SPL, false>(all, 128 * SPL, 64 * SPL, 0, nw, G);
            write_vec(carry + buf * 64 * SPL + lane * SPL, G);
        }
    }
    sg.template leave<SPL>(n, seg, seq, a.p.channels, ch, q, act, wave, nw, 0, G, total, lds);
}

// What a token brings to a lane: (delta, delta x, ds, -) of its channels, B and C of its states.
template <int SPL, int J> struct Operands {
    f32x4 d[J];
    float B[SPL], C[SPL];
    __device__ __forceinline__ void read(const float* pd, const float* pB, const float* pC) {
#pragma unroll
        for (int j = 0; j < J; ++j) d[j] = *reinterpret_cast<const f32x4*>(pd + j * kCh * 4);
        read_vec(pB, B);
        read_vec(pC, C);
    }
};

template <typename T, int SPL, bool GATE, bool SOFT>
__global__ __launch_bounds__(64 * Bwd<SPL>::NW, SPL == 16 ? 1 : 2) void k_scan_bwd(ScanArgs a, ScanBwdWs ws, Segments sg, int64_t lines, int cbg) {
    typedef Bwd<SPL> V;
    constexpr int J = V::J, L = V::L, K = L / 4, SP = V::SP, EPT = V::EPT, CHB = V::CHB, TOK = V::TOK, H2 = SPL / 2;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    int n, seg, g, cb;
    if (!unit_of(a, lines, cbg, sg.most, &n, &seg, &g, &cb)) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int c = lane >> 2, q = lane & 3, l4 = c & 3;
    const int D = a.p.channels, Dg = D / a.p.groups, S = a.p.state_dim;
    float* sd = lds + wave * V::kWaveFloats;                // [L][TOK]: [CHB][4]
    float* sB = sd + L * TOK;                           // [L][SP]
    float* sC = sB + L * SP;
    float* pub = lds + nw * V::kWaveFloats;                 // [2][nw][3][64][EPT]
    float* carry = pub + 2 * nw * V::kPubFloats;            // [2][64][EPT]
    int64_t s, e;
    seq_range(a.cu, n, a.p.seq_len, a.Ttot, &s, &e);
    const int64_t seq = s;
    int nseg = sg.most == 1 || e == s ? 1 : (int)((uint32_t)(e - s + sg.len - 1) / (uint32_t)sg.len);
    nseg = nseg < sg.most ? nseg : sg.most;
    bool last;
    if (!sg.range(seg, &s, &e, &last)) e = s;               // no such segment: its sums are zero

    bool act[J];
    int ch[J];
    float bias[J], skip[J], A2[EPT], dA[EPT], G[EPT], sumD[J], sumT[J];
    int64_t st0[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int cl = cb * CHB + c + kCh * j;
        act[j] = cl < Dg;
        ch[j] = g * Dg + (act[j] ? cl : Dg - 1);
        bias[j] = a.dt_bias ? a.dt_bias[ch[j]] : 0.f;
        skip[j] = a.D ? a.D[ch[j]] : 0.f;
        sumD[j] = sumT[j] = 0.f;
        st0[j] = ((int64_t)n * D + ch[j]) * S + q * SPL;
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const bool in = act[j] && q * SPL + i < S;
            A2[j * SPL + i] = in ? log2_rate(a.A[(int64_t)ch[j] * S + q * SPL + i]) : 0.f;
            G[j * SPL + i] = in && a.dST ? a.dST[st0[j] + i] : 0.f;
            dA[j * SPL + i] = 0.f;
        }
        if (nseg > 1) {                                     // G behind this segment, from the later ones
            float A2j[SPL], Gj[SPL];
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                A2j[i] = A2[j * SPL + i];
                Gj[i] = G[j * SPL + i];
            }
            const int64_t slot = first_slot(seq, sg.len, n);
#pragma unroll 4
            for (int i = nseg - 1; i > seg; --i) sg.template through<SPL>(slot + i, D, ch[j], q, A2j, Gj);
#pragma unroll
            for (int i = 0; i < SPL; ++i) G[j * SPL + i] = Gj[i];
        }
    }
    const bool dy32 = a.p.dy_dtype == GDR_F32 && sizeof(T) == 2, g32 = a.p.grad_dtype == GDR_F32;
    const int dyb = a.p.dy_dtype == GDR_F32 ? 4 : 2, gb = g32 ? 4 : 2;
    const int row = wave * L, tile = nw * L;
    const int ntiles = (int)((uint32_t)(e - s + tile - 1) / (uint32_t)tile);
    float* part = ws.bc + (int64_t)cb * 2 * a.Ttot * a.p.groups * S;
    const float* states = ws.states + (first_slot(seq, tile, n) + (uint32_t)(s - seq) / (uint32_t)tile) * D * SP;
    // this lane's tokens in a tile are wave L + 4 k + q; the offsets of the first, and bytes between k and k + 1
    const int64_t r0 = row + q;
    int ox[J], odt[J], oz[J], ody[J], og[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        ox[j] = act[j] ? (int)((r0 * a.p.x_stride + ch[j]) * (int)sizeof(T)) : V::IDLE;
        odt[j] = act[j] ? (int)((r0 * a.p.dt_stride + ch[j]) * (int)sizeof(T)) : V::IDLE;
        oz[j] = act[j] ? (int)((r0 * a.p.z_stride + ch[j]) * (int)sizeof(T)) : V::IDLE;
        ody[j] = act[j] ? (int)((r0 * D + ch[j]) * dyb) : V::IDLE;
        og[j] = act[j] ? (int)((r0 * D + ch[j]) * gb) : V::IDLE;
    }
    const int kx = (int)(4 * a.p.x_stride * (int)sizeof(T)), kdt = (int)(4 * a.p.dt_stride * (int)sizeof(T));
    const int kz = (int)(4 * a.p.z_stride * (int)sizeof(T)), kdy = 4 * D * dyb, kg = 4 * D * gb;
    // rows [t, t + rows) of a dense [Ttot, D] tensor of elements of `bytes` bytes
    auto dense_rows = [&](const void* p, int64_t t, int rows, int bytes) {
        return buf_rsrc((const char*)p + t * D * bytes, (uint32_t)((int64_t)rows * D * bytes));
    };
    T rx[K][J], rdt[K][J], rz[K][J];
    uint32_t rdy[K][J];
    float rh[J][SPL];
    StateRows<T, SPL, L> rB, rC;
    rB.init(a.p.b_stride, g * S, S, row);
    rC.init(a.p.c_stride, g * S, S, row);
    auto fetch = [&](int it) {                              // it < 0: nothing left
        const int64_t tb = s + (int64_t)it * tile;
        const int rows = it < 0 ? 0 : (int)(e - tb < tile ? e - tb : tile);
        const auto bx = token_rows<T>(a.x, tb, a.p.x_stride, rows), bdt = token_rows<T>(a.dt, tb, a.p.dt_stride, rows);
        const auto bdy = dense_rows(a.d_y, tb, rows, dyb);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                rx[k][j] = buf_load<T>(bx, ox[j] + k * kx);
                rdt[k][j] = buf_load<T>(bdt, odt[j] + k * kdt);
            }
        if (GATE) {
            const auto bz = token_rows<T>(a.z, tb, a.p.z_stride, rows);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < J; ++j) rz[k][j] = buf_load<T>(bz, oz[j] + k * kz);
        }
        // the raw bits, so that nothing waits for them here
        if (sizeof(T) == 4 || dy32) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < J; ++j) rdy[k][j] = __float_as_uint(buf_load<float>(bdy, ody[j] + k * kdy));
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    rdy[k][j] = __builtin_bit_cast(unsigned short, buf_load<bf16>(bdy, ody[j] + k * kdy));
        }
        rB.load(token_rows<T>(a.B, tb, a.p.b_stride, rows));
        rC.load(token_rows<T>(a.C, tb, a.p.c_stride, rows));
        if (rows > 0) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                read_vec(states + ((int64_t)it * D + ch[j]) * SP + q * SPL, rh[j]);
        }
    };
    const int shift = sizeof(T) == 4 || dy32 ? 0 : 16;      // raw bits of d_y to fp32
    if (ntiles > 0) fetch(ntiles - 1);
    int buf = 0;
    for (int it = ntiles - 1; it >= 0; --it, buf ^= 1) {
        const int64_t tb = s + (int64_t)it * tile, t0 = tb + row;
        const int left = (int)(e - tb < tile ? e - tb : tile);
        float h[L + 1][EPT], ea[L][EPT];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < SPL; ++i) h[0][j * SPL + i] = act[j] ? rh[j][i] : 0.f;
        wave_lds_fence();
        // of this lane's tokens: x, delta, d delta / d dt, ds, d_y silu'(z)
        float x[K][J], delta[K][J], slope[K][J], ds[K][J], dyg[K][J];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                x[k][j] = to_f(rx[k][j]);
                ds[k][j] = __uint_as_float(rdy[k][j] << shift);
                if (GATE) {
                    const float z = to_f(rz[k][j]), sg = sigmoid(z);
                    dyg[k][j] = ds[k][j] * silu_slope(z, sg);
                    ds[k][j] *= z * sg;
                }
                const float pre = to_f(rdt[k][j]) + bias[j];
                slope[k][j] = 1.f;
                const float d = SOFT ? softplus(pre, &slope[k][j]) : pre;
                delta[k][j] = act[j] && row + 4 * k + q < left ? d : 0.f;
                *reinterpret_cast<f32x4*>(sd + (4 * k + q) * TOK + (c + kCh * j) * 4) =
                    f32x4{delta[k][j], delta[k][j] * x[k][j], ds[k][j], 0.f};
            }
        rB.put(sB);
        rC.put(sC);
        wave_lds_fence();
        fetch(it - 1);

        // a piece's operands are read from LDS together, ahead of their use
        Operands<SPL, J> op[L];
#pragma unroll
        for (int m = 0; m < L; ++m) op[m].read(sd + m * TOK + c * 4, sB + m * SP + q * SPL, sC + m * SP + q * SPL);

        // the piece from a zero state, and its G from zero behind it
        float P[EPT], hl[EPT], Gl[EPT], sum[J];
#pragma unroll
        for (int i = 0; i < EPT; ++i) hl[i] = Gl[i] = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) sum[j] = 0.f;
#pragma unroll
        for (int m = 0; m < L; ++m)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                sum[j] += op[m].d[j][0];
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const int o = j * SPL + i;
                    ea[m][o] = __builtin_amdgcn_exp2f(A2[o] * op[m].d[j][0]);
                    hl[o] = __builtin_fmaf(ea[m][o], hl[o], op[m].d[j][1] * op[m].B[i]);
                }
            }
#pragma unroll
        for (int m = L - 1; m >= 0; --m)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    const int o = j * SPL + i;
                    Gl[o] = ea[m][o] * __builtin_fmaf(op[m].d[j][2], op[m].C[i], Gl[o]);
                }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < SPL; ++i) P[j * SPL + i] = __builtin_amdgcn_exp2f(A2[j * SPL + i] * sum[j]);
        float* all = pub + buf * nw * V::kPubFloats + lane * EPT;
        write_vec(all + wave * V::kPubFloats, P);
        write_vec(all + wave * V::kPubFloats + 64 * EPT, hl);
        write_vec(all + wave * V::kPubFloats + 128 * EPT, Gl);
        lds_barrier();
        if (it != ntiles - 1) read_vec(carry + (buf ^ 1) * 64 * EPT + lane * EPT, G);
        join_pieces<EPT, true>(all, V::kPubFloats, 64 * EPT, 0, wave, h[0]);
        join_pieces<EPT, false>(all, V::kPubFloats, 128 * EPT, wave + 1, nw, G);
        loads_arrived();
        {
            float Bv[L][SPL], dx[L][J];
#pragma unroll
            for (int m = 0; m < L; ++m) {
                read_vec(sB + m * SP + q * SPL, Bv[m]);
#pragma unroll
                for (int j = 0; j < J; ++j) dx[m][j] = sd[m * TOK + (c + kCh * j) * 4 + 1];
            }
#pragma unroll
            for (int m = 0; m < L; ++m)
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < SPL; ++i) {
                        const int o = j * SPL + i;
                        h[m + 1][o] = __builtin_fmaf(ea[m][o], h[m][o], dx[m][j] * Bv[m][i]);
                    }
        }
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            Operands<SPL, J> o4[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                o4[m].read(sd + (4 * k + m) * TOK + c * 4, sB + (4 * k + m) * SP + q * SPL, sC + (4 * k + m) * SP + q * SPL);
            float gB[J][4], gA[J][4], yC[J][4];
            float u[H2];
#pragma unroll
            for (int i = 0; i < H2; ++i) u[i] = 0.f;
#pragma unroll
            for (int m4 = 3; m4 >= 0; --m4) {
                const int m = 4 * k + m4;
                float dBv[SPL], dCv[SPL];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float tB = 0.f, tA = 0.f, tC = 0.f;
#pragma unroll
                    for (int i = 0; i < SPL; ++i) {
                        const int o = j * SPL + i;
                        const float gr = __builtin_fmaf(o4[m4].d[j][2], o4[m4].C[i], G[o]);
                        const float gp = gr * (ea[m][o] * h[m][o]);
                        tB = __builtin_fmaf(gr, o4[m4].B[i], tB);
                        tA = __builtin_fmaf(gp, A2[o], tA);
                        if (GATE) tC = __builtin_fmaf(o4[m4].C[i], h[m + 1][o], tC);
                        dA[o] = __builtin_fmaf(gp, o4[m4].d[j][0], dA[o]);
                        dBv[i] = j ? __builtin_fmaf(gr, o4[m4].d[j][1], dBv[i]) : gr * o4[m4].d[j][1];
                        dCv[i] = j ? __builtin_fmaf(o4[m4].d[j][2], h[m + 1][o], dCv[i]) : o4[m4].d[j][2] * h[m + 1][o];
                        G[o] = ea[m][o] * gr;
                    }
                    gB[j][m4] = tB;
                    gA[j][m4] = tA;
                    yC[j][m4] = tC;
                }
                // over the channels: lanes below 32 keep dB, the others dC; rows then halve the states
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    swap32(dBv[i], dCv[i]);
                    dBv[i] += dCv[i];
                }
#pragma unroll
                for (int i = 0; i < H2; ++i) {
                    swap16(dBv[i], dBv[i + H2]);
                    const float v = sum_row(dBv[i] + dBv[i + H2]);
                    u[i] = l4 == m4 ? v : u[i];
                }
            }
            const int64_t tk = t0 + 4 * k;
            if (tk + l4 < e) {
                const int64_t at = (((int64_t)(lane >> 5) * a.Ttot + tk + l4) * a.p.groups + g) * S;
                const int n0 = q * SPL + ((lane >> 4) & 1) * H2;
#pragma unroll
                for (int i = 0; i < H2; ++i)
                    if (n0 + i < S) part[at + n0 + i] = u[i];
            }
            const auto bdx = dense_rows(a.dx, tb, left, gb), bddt = dense_rows(a.ddt, tb, left, gb);
            const auto bdz = dense_rows(GATE ? a.dz : a.dx, tb, left, gb);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float gBs = states_sum4(gB[j], q), gAs = states_sum4(gA[j], q);
                const float ddelta = __builtin_fmaf(gAs, kLn2, x[k][j] * gBs);
                float ddt = ddelta * slope[k][j];
                const float dx_ = __builtin_fmaf(skip[j], ds[k][j], delta[k][j] * gBs);
                const float dz_ = GATE ? dyg[k][j] * __builtin_fmaf(skip[j], x[k][j], states_sum4(yC[j], q)) : 0.f;
                const int o = og[j] + k * kg;
                if (g32) {
                    buf_store<float>(bdx, o, dx_);
                    buf_store<float>(bddt, o, ddt);
                    if (GATE) buf_store<float>(bdz, o, dz_);
                } else {
                    buf_store<T>(bdx, o, dx_);
                    buf_store<T>(bddt, o, ddt);
                    if (GATE) buf_store<T>(bdz, o, dz_);
                }
                ddt = row + 4 * k + q < left ? ddt : 0.f;
                sumD[j] = __builtin_fmaf(ds[k][j], x[k][j], sumD[j]);  // x and d_y are zero past the end
                sumT[j] += ddt;
            }
        }
        if (wave == 0) write_vec(carry + buf * 64 * EPT + lane * EPT, G);
    }
    if (a.dS0 && seg == 0 && wave == 0) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < SPL; ++i)
                if (act[j] && q * SPL + i < S) a.dS0[st0[j] + i] = G[j * SPL + i];
    }
    // the wavefronts' sums over their tokens, joined in order
    lds_barrier();
    float* all = lds;                                       // [nw][64][EPT + 2 J]
    constexpr int R = EPT + 2 * J;
#pragma unroll
    for (int i = 0; i < EPT; ++i) all[(wave * R + i) * 64 + lane] = dA[i];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        all[(wave * R + EPT + j) * 64 + lane] = sum_states(sumD[j]);
        all[(wave * R + EPT + J + j) * 64 + lane] = sum_states(sumT[j]);
    }
    lds_barrier();
    if (wave != 0) return;
    float* par = ws.par + ((int64_t)n * sg.most + seg) * D * (S + 2);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float v = 0.f;
        for (int w = 0; w < nw; ++w) v += all[(w * R + i) * 64 + lane];
        const int j = i < EPT ? i / SPL : (i - EPT) % J;
        if (!act[j]) continue;
        if (i < EPT) {
            if (q * SPL + i % SPL < S) par[(int64_t)ch[j] * S + q * SPL + i % SPL] = v;
        } else if (q == 0) {
            par[(int64_t)D * S + (int64_t)((i - EPT) / J) * D + ch[j]] = v;
        }
    }
}

template <typename T> struct StateGradOut {                 // dB, dC in grad_dtype
    void *dB, *dC;
    int64_t half;
    int f32;
    __device__ void operator()(int64_t i, float v) const {
        if (i < half) store_as<T>(dB, i, v, f32);
        else store_as<T>(dC, i - half, v, f32);
    }
};
struct ParameterOut {                                       // dA [D][S], then dD [D], ddt_bias [D]
    float *dA, *dD, *ddt_bias;
    int64_t DS, D;
    __device__ void operator()(int64_t i, float v) const {
        if (i < DS) dA[i] = v;
        else if (i < DS + D) {
            if (dD) dD[i - DS] = v;
        } else if (ddt_bias) {
            ddt_bias[i - DS - D] = v;
        }
    }
};

// Workspace regions. States kept: one a tile of nw L tokens, and one more a
// sequence. With fewer than LEAST wavefronts no sequence is longer than a tile,
// so that T / tile <= N; otherwise the tile has LEAST L tokens or more.
struct BwdPlan {
    size_t states, bc, par, end, sum, gend, gsum, all;
};
template <int SPL> int64_t bwd_units(const gdr_scan_problem_t& p) {
    return (int64_t)p.num_seqs * p.groups * ((p.channels / p.groups + Bwd<SPL>::CHB - 1) / Bwd<SPL>::CHB);
}
template <int SPL>
BwdPlan plan(const gdr_scan_problem_t& p) {
    typedef Bwd<SPL> V;
    const size_t D = p.channels, S = p.state_dim, N = p.num_seqs, T = (size_t)(p.batch * p.seq_len);
    const size_t cbg = (D / p.groups + V::CHB - 1) / V::CHB;
    const size_t slots = segment_slots(bwd_units<SPL>(p), V::NW, N);
    const size_t nseg = slots ? most_segments(bwd_units<SPL>(p), V::NW) : 1;
    BwdPlan b;
    size_t off = 0;
    auto take = [&](size_t floats) { size_t o = off; off = (off + floats * 4 + 255) & ~(size_t)255; return o; };
    const size_t most = N < T ? N : T, tiles = T / (V::LEAST * V::L);
    b.states = take(((tiles > most ? tiles : most) + N) * D * V::SP);
    b.bc = take(cbg * 2 * T * p.groups * S);
    b.par = take(N * nseg * D * (S + 2));
    b.end = take(slots * D * V::SP);
    b.sum = take(slots * D);
    b.gend = take(slots * D * V::SP);
    b.gsum = take(slots * D);
    b.all = off;
    return b;
}

template <typename T, int SPL>
hipError_t bwd(const ScanArgs& a) {
    typedef Bwd<SPL> V;
    static_assert(V::lds(V::NW) <= 160 * 1024, "LDS of a compute unit");
    const BwdPlan pl = plan<SPL>(a.p);
    auto f = [&](size_t off) { return reinterpret_cast<float*>(a.ws + off); };
    const ScanBwdWs ws = {f(pl.states), f(pl.bc), f(pl.par)};
    const int Dg = a.p.channels / a.p.groups;
    const int cbs = (Dg + kCh - 1) / kCh, cbg = (Dg + V::CHB - 1) / V::CHB;
    Segments sg = segments_for(bwd_units<SPL>(a.p), V::NW, a.max_len), gsg = sg;
    sg.end = f(pl.end);
    sg.sum = f(pl.sum);
    gsg.end = f(pl.gend);
    gsg.sum = f(pl.gsum);
    const int64_t NG = (int64_t)a.p.num_seqs * a.p.groups * sg.most, longest = sg.most > 1 ? sg.len : a.max_len;
    const int nw = waves_for(NG * cbg, longest, V::L, 2048, V::LEAST, V::NW);
    const int nws = waves_for(NG * cbs, longest, kPiece<SPL>, 4096, 1, SPL == 16 ? 4 : 8);
    const int64_t slines = line_units(NG, cbs), lines = line_units(NG, cbg);
    hipError_t e = hipSuccess;
    if (!grid_fits(unit_blocks(slines), 64 * (nw > nws ? nw : nws))) return hipErrorInvalidConfiguration;
    if (NG > 0) {
        const size_t lds = states_lds<SPL>(nws);
        const dim3 sgrid((unsigned)unit_blocks(slines)), bgrid((unsigned)unit_blocks(lines));
        auto go = [&](auto gate, auto soft) {
            constexpr bool GATE = decltype(gate)::value, SOFT = decltype(soft)::value;
            if (sg.most > 1) {
                k_scan_states<T, SPL, SOFT, true><<<sgrid, 64 * nws, lds, a.stream>>>(a, sg, nullptr, slines, cbs, 1);
                if ((e = hipGetLastError()) != hipSuccess) return;
                k_scan_grad_ends<T, SPL, GATE, SOFT><<<sgrid, 64 * nws, lds, a.stream>>>(a, gsg, slines, cbs);
                if ((e = hipGetLastError()) != hipSuccess) return;
            }
            k_scan_states<T, SPL, SOFT, false><<<sgrid, 64 * nws, lds, a.stream>>>(a, sg, ws.states, slines, cbs, nw * V::L);
            if ((e = hipGetLastError()) != hipSuccess) return;
            k_scan_bwd<T, SPL, GATE, SOFT><<<bgrid, 64 * nw, V::lds(nw), a.stream>>>(a, ws, gsg, lines, cbg);
        };
        auto by_gate = [&](auto soft) { a.z ? go(std::true_type{}, soft) : go(std::false_type{}, soft); };
        a.p.dt_softplus ? by_gate(std::true_type{}) : by_gate(std::false_type{});
        if (e != hipSuccess) return e;
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t D = a.p.channels, S = a.p.state_dim, half = a.Ttot * a.p.groups * S;
    const int64_t parts = (int64_t)a.p.num_seqs * sg.most;
    e = sum_partials(ws.bc, cbg, 2 * half, StateGradOut<T>{a.dB, a.dC, half, a.p.grad_dtype == GDR_F32}, a.stream);
    if (e == hipSuccess) e = sum_partials(ws.par, parts, D * (S + 2), ParameterOut{a.dA, a.dD, a.ddt_bias, D * S, D}, a.stream);
    return e;
}

}  // namespace

size_t scan_bwd_workspace(const gdr_scan_problem_t& p) {
    return by_state_dim(p.state_dim, [&](auto spl) { return plan<decltype(spl)::value>(p).all; });
}

hipError_t launch_scan_bwd(const ScanArgs& a) {
    return by_states(a, [&](auto type, auto spl) { return bwd<decltype(type), decltype(spl)::value>(a); });
}

}  // namespace gdr
