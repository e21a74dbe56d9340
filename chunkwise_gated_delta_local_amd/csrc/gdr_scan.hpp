// What the scan's forward and backward kernels share.
#pragma once

#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

constexpr int kCh = 16;                                    // channels of a wavefront

// Tokens a wavefront of the forward kernels takes at a time: SPL * piece
// exponentials and as many products stay in registers.
template <int SPL> constexpr int kPiece = SPL <= 4 ? 16 : 64 / SPL;

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

// Workgroup -> (sequence, group, channel block): consecutive blocks of channels
// on the same XCD (workgroups are dealt to the eight XCDs in turn), so that the
// 32-byte pieces of a 128-byte line meet in one L2.
__device__ __forceinline__ bool unit_of(int64_t units, int cbg, int groups, int* n, int* g, int* cb) {
    const int64_t per = (units + 7) / 8, u = (blockIdx.x % 8) * per + blockIdx.x / 8;
    if (u >= units || blockIdx.x / 8 >= per) return false;
    *cb = (int)(u % cbg);
    *g = (int)(u / cbg % groups);
    *n = (int)(u / ((int64_t)cbg * groups));
    return true;
}

// Rows of a token tensor from token t on, `rows` of them: a buffer whose accesses
// past its end read zero and store nothing, so that the tokens behind a sequence
// need no branches. Offsets inside are bytes, (token - t) * stride + element.
constexpr int kNowhere = 0x7fffffff;                       // an offset past the end of any of them
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
    static constexpr int SP = 4 * SPL, PER = L * SP / 64;
    int off[PER];
    T r[PER];
    __device__ __forceinline__ void init(int64_t stride, int first, int S, int row) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = i * 64 + lane, n = idx % SP;
            off[i] = n < S ? (int)(((row + idx / SP) * stride + first + n) * (int)sizeof(T)) : kNowhere;
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs) {
#pragma unroll
        for (int i = 0; i < PER; ++i) r[i] = buf_load<T>(rs, off[i]);
    }
    __device__ __forceinline__ void put(float* lds) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < PER; ++i) lds[i * 64 + lane] = to_f(r[i]);
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
        static_assert(N == 2, "state group");
        const f32x2 w = *reinterpret_cast<const f32x2*>(p);
        v[0] = w[0];
        v[1] = w[1];
    }
}
template <int N>
__device__ __forceinline__ void write_vec(float* p, const float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
        *reinterpret_cast<f32x2*>(p) = f32x2{v[0], v[1]};
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

// ---------------------------------------------------------------- host
// Wavefronts of a workgroup, a power of two: as many as make `fill` in all units
// together, at least `least`, no more than pieces in the longest sequence or than `most`.
inline int waves_for(int64_t units, int64_t max_len, int piece, int fill, int least, int most) {
    int nw = 1;
    while (nw < most && (int64_t)nw * piece < max_len && (nw < least || units * nw < fill)) nw *= 2;
    return nw;
}

template <typename F>
hipError_t by_states(const ScanArgs& a, F f) {
    auto pick = [&](auto type) {
        const int S = a.p.state_dim;
        if (S <= 8) return f(type, std::integral_constant<int, 2>{});
        if (S <= 16) return f(type, std::integral_constant<int, 4>{});
        if (S <= 32) return f(type, std::integral_constant<int, 8>{});
        return f(type, std::integral_constant<int, 16>{});
    };
    return a.p.io_dtype == GDR_BF16 ? pick(bf16{}) : pick(float{});
}

}  // namespace gdr
