// Internal interface of the window attention (include/gdr_attn.h): launch
// arguments, and the device building blocks that its kernels share.
//
// Products run on 32x32 matrix-core tiles. For lane l = 32 h + r of a wavefront
// the operand of 32 rows holds row r, and the accumulator holds column r with
// the rows 8 i + 4 h + j in register 4 i + j. Operand and accumulator then fit
// without moving data between lanes: the scores are formed transposed (keys in
// the accumulator's rows, a query in each lane's column), so that
//  - a query's maximum and sum are a lane's own but for one exchange of halves;
//  - the weights are the operand of the product with v as they lie, contracted
//    over keys in the order 8 i + 4 h + j;
//  - v enters that product by transposing LDS reads of 4 keys at a time (bf16),
//    or by plain ones (fp32).
// The contraction over the head dimension may run in any order that both
// operands share: a step takes 16 bytes of each row, the half h its unit 2 t + h.
#pragma once

#include <type_traits>

#include "gdr_attn.h"
#include "gdr_mixer.hpp"

namespace gdr {

struct AttnArgs {
    gdr_attn_problem_t p;
    int64_t Ttot;              // total tokens
    int32_t q_ld, k_ld, v_ld;  // elements between tokens
    const void *q, *k, *v;
    void *kc, *vc;             // caches or NULL
    const int32_t *lens, *cu;  // NULL: zeros; NULL: batch rows
    void* o;
    float* lse;
    bool vec;                  // rows of q, k, v and the caches in 16-byte pieces at 16-byte addresses
    float* ws;
    // backward
    const void *oin, *d_o;     // d_o: as given, then in the io type
    const float* lse_in;
    void *dq, *dk, *dv;
    float* rows;               // [Ttot][Nq][2]: lse log2(e), sum of d_o o
    float* tops;               // [Ttot][Nq]: the largest score where lse is formed from there, else 0
    void* d_o16;               // d_o rounded to the io type, where it comes in fp32
    int32_t* slots;            // [num_seqs + 1]: first slot of each sequence
    float* sink_part;          // [slots][sinks][Nk][dk + dv]
    int32_t max_slots;
    hipStream_t stream;
};

size_t attn_fwd_workspace(const gdr_attn_problem_t& p);
hipError_t launch_attn_fwd(const AttnArgs& a);
size_t attn_step_workspace(const gdr_attn_problem_t& p);
hipError_t launch_attn_step(const AttnArgs& a);
size_t attn_bwd_workspace(const gdr_attn_problem_t& p);
hipError_t launch_attn_bwd(const AttnArgs& a);

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();

// Tiles in LDS are addressed as LDS, by bytes: a pointer that could point anywhere costs
// a test for NULL wherever an LDS address is made of it.
template <typename T> using lds_p = __attribute__((address_space(3))) T*;
typedef lds_p<char> lds_c;
template <typename T>
__device__ __forceinline__ lds_c lds_of(T* tile) { return (lds_c)(lds_p<T>)tile; }

// elements in 16 bytes
template <typename T> constexpr int kUnit = 16 / (int)sizeof(T);

// ---------------------------------------------------------------- rows of queries
// A block of queries is TPB tokens of one sequence times HPB of the G heads that
// share a key head: row r is token r / HPB, head r % HPB. The keys of a block are
// read once for all its heads, and its window is little longer than one token's.
struct RowBlock {
    int HPB, TPB, HC;          // heads and tokens of a block, blocks to a key head's group
};
__host__ __device__ inline RowBlock row_block(int rows, int G) {
    RowBlock b;
    b.HPB = G < rows ? G : rows;
    b.TPB = rows / b.HPB;
    b.HC = (G + b.HPB - 1) / b.HPB;
    return b;
}
// Blocks of TPB tokens: sequence n has the numbers from start / TPB + n (packed
// sequences; some numbers stay unused) or n ceil(T / TPB) on.
__host__ __device__ inline int64_t token_blocks(int64_t batch, int64_t T, int N, bool packed, int TPB) {
    return packed ? T / TPB + N : batch * ((T + TPB - 1) / TPB);
}

struct Block {
    int n, t0, tn;             // sequence, first token in it, tokens
    int64_t start;             // the sequence's first row of q, k, v
    int len;                   // its tokens
};
// Block number b of tokens; false: unused. All lanes call it alike.
__device__ inline bool find_block(const int32_t* cu, int N, int64_t T, int64_t Ttot, int TPB, int b, Block* x) {
    if (!cu) {
        const int per = (int)((T + TPB - 1) / TPB);
        x->n = b / per;
        x->t0 = (b - x->n * per) * TPB;
        x->start = (int64_t)x->n * T;
        x->len = (int)T;
    } else {
        // the last n with cu[n] / TPB + n <= b; each lane looks at a 64th of what is left
        int lo = 0, len = N;
        while (len > 1) {
            const int step = (len + 63) / 64, i = lo + (int)(threadIdx.x & 63) * step;
            const bool before = i < lo + len && cu[i] / TPB + i <= b;
            const int k = __popcll(__ballot(before));
            const int at = k > 0 ? (k - 1) * step : 0;
            len = len - at < step ? len - at : step;
            lo += at;
        }
        x->n = __builtin_amdgcn_readfirstlane(lo);
        int64_t s, e;
        seq_range(cu, x->n, 0, Ttot, &s, &e);
        s = __builtin_amdgcn_readfirstlane((int)s);
        e = __builtin_amdgcn_readfirstlane((int)e);
        x->start = s;
        x->len = (int)(e - s);
        const int first = (int)s / TPB + x->n;
        if (b < first || b - first > x->len / TPB) return false;
        x->t0 = (b - first) * TPB;
    }
    x->tn = x->len - x->t0 < TPB ? x->len - x->t0 : TPB;
    return x->tn > 0;
}

// The keys that queries at positions p0 .. p1 see (behind len cached tokens), as
// at most five runs of consecutive rows: cached sinks, two pieces of the ring, new
// sinks, new tokens. All members are the same in every lane.
struct Keys {
    int n0, n1, n2, n3, n4;    // keys of the runs that are left, the present one first
    int p0, p1, p2, p3, p4;    // their first positions
    int r0, r1, r2, r3, r4;    // and rows
    int old;                   // runs among them that lie in the cache

    __device__ Keys(int first, int last, int len, int W, int S) : old(3) {
        const int end = last + 1, lo = first - W + 1 > S ? first - W + 1 : S;
        p0 = r0 = 0;
        n0 = len < S ? len : S;
        p1 = lo;
        n1 = n2 = 0;
        r1 = r2 = S;
        if (lo < len) {
            const int n = len - lo, w = (lo - S) % W;
            n1 = n < W - w ? n : W - w;
            n2 = n - n1;
            r1 = S + w;
            if (lo == S) {                       // the ring goes on behind the sinks (and has not turned)
                n0 += n1;
                n1 = 0;
            }
        }
        p2 = p1 + n1;
        const int sink_end = S < end ? S : end;
        p3 = len;
        n3 = len < sink_end ? sink_end - len : 0;
        p4 = lo > len ? lo : len;
        n4 = end > p4 ? end - p4 : 0;
        if (n3 > 0 && p4 == len + n3) {
            n3 += n4;
            n4 = 0;
        }
        r3 = 0;
        r4 = p4 - len;
    }
    __device__ int total() const { return n0 + n1 + n2 + n3 + n4; }
    __device__ void drop() {
        n0 = n1; n1 = n2; n2 = n3; n3 = n4; n4 = 0;
        p0 = p1; p1 = p2; p2 = p3; p3 = p4;
        r0 = r1; r1 = r2; r2 = r3; r3 = r4;
        --old;
    }
    __device__ void cut(int n) {
        n0 -= n;
        p0 += n;
        r0 += n;
    }
    // moves n <= total() keys on
    __device__ void skip(int n) {
#pragma unroll
        for (int i = 0; i < 5; ++i)
            if (n >= n0) {
                n -= n0;
                drop();
            }
        cut(n);
    }
    // the next tile of at most n keys: its first position, keys, first row, whether cached; 0 keys: the end
    __device__ void next(int n, int* pos, int* cnt, int* row, bool* cached) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 == 0) drop();
        *cnt = n0 < n ? n0 : n;
        *pos = p0;
        *row = r0;
        *cached = old > 0;
        cut(*cnt);
    }
};

// ---------------------------------------------------------------- tiles
// Rows of D elements in LDS, in UN 16-byte units; unit u of a row lies at u ^ swz(row).
// The 64 banks give 256 bytes a cycle to accesses that spread over them: 16 rows' reads
// of one unit (16 lanes of 16 bytes) and transposing reads of 4 rows (32 lanes of 8
// bytes). For rows of 256 bytes swz takes 16 rows to 16 units, the 4 rows of a transposing
// read to different groups of 4; of 128 bytes, every other row to 8 units. Cycles an
// instruction with eight wavefronts, so and with 3 bits of the row's number: 16 bytes
// 3.8 and 6.3, transposing 2.3 and 3.5.
template <int UN>
__device__ __forceinline__ int swz(int row) {
    if constexpr (UN == 8) return (row >> 1 & 1) << 2 | (row >> 2 & 3);
    else return (row & 3) << 2 | (row >> 2 & 3);
}

// A row's operand for a contraction over the head dimension
template <typename T> struct Frag;
template <> struct Frag<bf16> {
    typedef Vec<bf16>::v8 type;
};
template <> struct Frag<float> {
    typedef f32x4 type;
};
template <typename T> using frag_t = typename Frag<T>::type;

__device__ __forceinline__ f32x16 mma(const Vec<bf16>::v8& a, const Vec<bf16>::v8& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const f32x4& a, const f32x4& b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// A lane's byte offsets into a tile of rows of D elements, for the operands below: what
// an access adds to them is known when the kernel is compiled, a bitwise sum of unit
// numbers (the swizzle is one) and a number of rows.
template <typename T, int D>
__device__ __forceinline__ int row_offset(int lane) {
    const int row = lane & 31;
    return row * D * (int)sizeof(T) + (((lane >> 5) ^ swz<D / kUnit<T>>(row)) << 4);
}
template <typename T, int D>
__device__ __forceinline__ int col_offset(int lane) {
    const int h = lane >> 5, l = lane & 15;
    if constexpr (sizeof(T) == 2) {
        const int row = 4 * h + (l >> 2), unit = (lane >> 3 & 2) | (l >> 1 & 1);
        return row * D * 2 + ((unit ^ swz<D / 8>(row)) << 4) + 8 * (l & 1);
    } else {
        return 4 * h * D * 4 + (((lane & 31) >> 2 ^ swz<D / 4>(4 * h)) << 4) + 4 * (lane & 3);
    }
}
// A value that the compiler does not know: addresses are then formed where they are used
// and not all kept in registers through a loop.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Operands that were loaded before a loop are waited for here, not in each of its turns
// (where the copies under way would be waited for with them).
template <typename F, int N>
__device__ __forceinline__ void arrived(F (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

// row r0 + lane % 32 (r0 a multiple of 32), step t; off: row_offset
template <typename T, int D>
__device__ __forceinline__ frag_t<T> row_frag(lds_c tile, int r0, int t, int off) {
    return *(lds_p<frag_t<T>>)(tile + (off ^ (t << 5)) + r0 * D * (int)sizeof(T));
}
// Operand of the transpose: row 32 u + lane % 32 (a column of the tile), contracted over
// the 16 tile rows r0 + 8 i + 4 h + j, i < 2 (r0 a multiple of 16); off: col_offset
template <typename T, int D>
__device__ __forceinline__ typename Vec<T>::v8 col_frag(lds_c tile, int r0, int u, int off) {
    if constexpr (sizeof(T) == 2) {
        s16x4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p<s16x4>)(tile + (off ^ (u << 6 | i << 5)) + (r0 + 8 * i) * D * 2));
        return __builtin_bit_cast(typename Vec<T>::v8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        typename Vec<T>::v8 x;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = *(lds_p<float>)(tile + (off ^ (u << 7 ^ (i & 3) << 6 ^ (i >> 2) << 5)) + (r0 + 8 * (i >> 2) + (i & 3)) * D * 4);
        return x;
    }
}
__device__ __forceinline__ f32x16 mma(const Vec<float>::v8& a, const Vec<float>::v8& b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
// rows 16 q .. 16 q + 15 of an accumulator as the other operand of that contraction
template <typename T>
__device__ __forceinline__ typename Vec<T>::v8 acc_frag(const f32x16& s, int q) {
    typename Vec<T>::v8 x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_t<T>(s[8 * q + e]);
    return x;
}

// Order of a run of N operands that are read from LDS in R reads each and used in M
// products each: AHEAD operands are read before the first product.
template <int N, int R, int M, int AHEAD = 6>
__device__ __forceinline__ void feed() {
    constexpr int A = AHEAD < N ? AHEAD : N;
    __builtin_amdgcn_sched_group_barrier(0x100, A * R, 0);
#pragma unroll
    for (int i = 0; i < N - A; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, A * M, 0);
}

constexpr int kOutside = 0x7ffffff0;                       // bytes behind the end of every buffer
// 16 bytes of a row through a range-checked buffer, zero from element d on; VEC:
// rows begin and end at 16-byte addresses
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 load_unit(__amdgpu_buffer_rsrc_t rs, int row_bytes, int unit, int d) {
    constexpr int out = kOutside;
    if constexpr (VEC) {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             rs, unit * kUnit<T> < d ? row_bytes + unit * 16 : out, 0, 0));
    } else if constexpr (sizeof(T) == 4) {
        u32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, unit * 4 + e < d ? row_bytes + unit * 16 + 4 * e : out, 0, 0);
        return x;
    } else {
        u32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                    rs, unit * 8 + 2 * e + i < d ? row_bytes + unit * 16 + 4 * e + 2 * i : out, 0, 0);
            x[e] = v[0] | v[1] << 16;
        }
        return x;
    }
}
// the same of a row in memory (`live`: its address is valid)
template <typename T, bool VEC>
__device__ __forceinline__ frag_t<T> load_frag_row(const T* row, int unit, int d, bool live) {
    frag_t<T> x;
    if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) x[e] = to_t<T>(0.f);
        if (live && unit * kUnit<T> < d) x = *reinterpret_cast<const frag_t<T>*>(row + unit * kUnit<T>);
    } else {
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) {
            const int c = unit * kUnit<T> + e;
            x[e] = live && c < d ? row[c] : to_t<T>(0.f);
        }
    }
    return x;
}

// Copies of 16 or 4 bytes a lane to lds + 16 lane (4 lane), as buffer_to_lds16 and
// buffer_to_lds4 (gdr_device.hpp), which the compiler does not know for ones: it would
// have every transposing read of LDS wait for all copies under way. Whoever reads the data
// waits himself: wait_vmem() in the wavefront that copies, and a barrier. m0, which holds
// the address, is put back; a write of it needs one cycle before its use.
__device__ __forceinline__ void copy16_to_lds(u32x4 rsrc, lds_c lds, int voffset) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds)), "v"(voffset), "s"(rsrc) : "memory");
}
__device__ __forceinline__ void copy4_to_lds(u32x4 rsrc, lds_c lds, int voffset) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, 0 offen lds\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(m0) : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds)), "v"(voffset), "s"(rsrc) : "memory");
}
// the buffer of `bytes` bytes at base (buf_rsrc) as the instruction takes it
__device__ __forceinline__ u32x4 raw_rsrc(const void* base, uint32_t bytes) {
    const uint64_t p = (uint64_t)base;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu)),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

// ROWS rows of a tile on their way from memory to LDS, by NT threads: `start` issues the
// loads; once `finish` has been called and the workgroup has met at `landed`, the rows
// are in LDS. With 16-byte rows they go there directly, else through registers.
template <typename T, int D, int ROWS, int NT, bool VEC>
struct Copy {
    static constexpr int UN = D / kUnit<T>, N = ROWS * UN / NT;
    static_assert(ROWS * UN % NT == 0 && NT % 64 == 0, "whole units a thread");
    u32x4 x[VEC ? 1 : N];
    // row_at(row): its bytes behind base, of which `bytes` are valid
    template <typename F>
    __device__ __forceinline__ void start(lds_c tile, const T* base, uint32_t bytes, F row_at, int d, int tid) {
        const int first = __builtin_amdgcn_readfirstlane(tid) & ~63;
        if constexpr (VEC) {
            const u32x4 rs = raw_rsrc(base, bytes);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int id = tid + i * NT, row = id / UN, unit = (id % UN) ^ swz<UN>(row);
                copy16_to_lds(rs, tile + (first + i * NT) * 16,
                              unit * kUnit<T> < d ? row_at(row) + unit * 16 : kOutside);
            }
        } else {
            const auto rs = buf_rsrc(base, bytes);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int id = tid + i * NT, row = id / UN, unit = (id % UN) ^ swz<UN>(row);
                x[i] = load_unit<T, VEC>(rs, row_at(row), unit, d);
            }
        }
    }
    __device__ __forceinline__ void start(lds_c tile, const T* base, int ld, int rows, int d, int tid) {
        const uint32_t row_bytes = (uint32_t)ld * sizeof(T);
        start(tile, base, rows > 0 ? (rows - 1) * row_bytes + d * (uint32_t)sizeof(T) : 0,
              [&](int row) { return row * (int)row_bytes; }, d, tid);
    }
    __device__ __forceinline__ void finish(lds_c tile, int tid) const {
        if constexpr (!VEC) {
#pragma unroll
            for (int i = 0; i < N; ++i) *(lds_p<u32x4>)(tile + (tid + i * NT) * 16) = x[i];
        }
    }
};
__device__ __forceinline__ void landed() {
    wait_vmem();
    lds_barrier();
}
// The same by one wavefront for itself, through registers: `load` early, `store` when the
// tile before has been read.
template <typename T, int D, int ROWS, bool VEC>
struct OwnCopy {
    static constexpr int UN = D / kUnit<T>, N = ROWS * UN / 64;
    u32x4 x[N];
    __device__ __forceinline__ void load(const T* base, int ld, int rows, int d) {
        const uint32_t row_bytes = (uint32_t)ld * sizeof(T);
        const auto rs = buf_rsrc(base, rows > 0 ? (rows - 1) * row_bytes + d * (uint32_t)sizeof(T) : 0);
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = lane + i * 64, row = id / UN, unit = (id % UN) ^ swz<UN>(row);
            x[i] = load_unit<T, VEC>(rs, row * (int)row_bytes, unit, d);
        }
    }
    __device__ __forceinline__ void store(lds_c tile) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *(lds_p<u32x4>)(tile + ((int)(threadIdx.x & 63) + i * 64) * 16) = x[i];
    }
};

// over the two lanes of a column
__device__ __forceinline__ float pair_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Which of a tile's keys a lane's query sees.
struct Sight {
    int pos0, cnt, p, W, S;
    __device__ bool operator()(int key) const {
        const int pos = pos0 + key;
        return key < cnt && pos <= p && (pos < S || pos > p - W);
    }
};

// ---------------------------------------------------------------- shared set-up
// A wavefront's 32 rows of a block: the lane's row, its query's place and position.
struct Query {
    bool live;
    int64_t token;             // row of q and o
    int head, p;               // head of q; position in the sequence
};
__device__ __forceinline__ Query query_of(const Block& b, const RowBlock& rb, int G, int hk, int hc, int r, int len) {
    const int t = r / rb.HPB, g = hc * rb.HPB + r % rb.HPB;
    Query q;
    q.live = t < b.tn && t < rb.TPB && g < G;
    const int tc = t < b.tn ? t : b.tn - 1;            // rows behind the block follow its last token
    q.token = b.start + b.t0 + tc;
    q.head = hk * G + (g < G ? g : G - 1);
    q.p = len + b.t0 + tc;
    return q;
}
// A single token's position at most; positions and a tile of keys behind them fit 31 bits
constexpr int kMostLen = 0x7fffffff - 65;
__device__ __forceinline__ int past_len(const AttnArgs& a, int n) {
    if (!a.lens) return 0;
    const int len = __builtin_amdgcn_readfirstlane(a.lens[n]), most = kMostLen + 1 - (int)a.p.seq_len;
    return len < 0 ? 0 : len < most ? len : most;
}

template <typename T>
struct Source {                // where a tile's keys and values begin
    const T *k, *v;
    int kld, vld;
};
template <typename T>
__device__ __forceinline__ Source<T> source(const AttnArgs& a, const Block& b, int hk, int row, bool cached) {
    const int dk = a.p.head_dim_qk, dv = a.p.head_dim_v, Nk = a.p.num_kv_heads;
    Source<T> s;
    if (cached) {
        const int64_t at = (int64_t)b.n * ((int64_t)a.p.sinks + a.p.window) + row;
        s.k = (const T*)a.kc + (at * Nk + hk) * dk;
        s.v = (const T*)a.vc + (at * Nk + hk) * dv;
        s.kld = Nk * dk;
        s.vld = Nk * dv;
    } else {
        s.k = (const T*)a.k + (b.start + row) * a.p.k_stride + hk * dk;
        s.v = (const T*)a.v + (b.start + row) * a.p.v_stride + hk * dv;
        s.kld = a.k_ld;
        s.vld = a.v_ld;
    }
    return s;
}

// Four consecutive outputs d .. d + 3 of a row
template <typename OT>
__device__ __forceinline__ void store4(OT* row, int d, int dv, const float (&y)[4]) {
    if (d + 4 <= dv) {
        store_vec<OT, 4>(row + d, y);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (d + j < dv) row[d + j] = to_t<OT>(y[j]);
    }
}

// ---------------------------------------------------------------- launches
inline int group(const gdr_attn_problem_t& p) { return p.num_q_heads / p.num_kv_heads; }

// f(io type, DK, DV)
template <typename F>
void by_dims(const gdr_attn_problem_t& p, F f) {
    auto go = [&](auto type) {
        typedef std::integral_constant<int, 64> d64;
        typedef std::integral_constant<int, 128> d128;
        if (p.head_dim_qk <= 64) p.head_dim_v <= 64 ? f(type, d64{}, d64{}) : f(type, d64{}, d128{});
        else p.head_dim_v <= 64 ? f(type, d128{}, d64{}) : f(type, d128{}, d128{});
    };
    p.io_dtype == GDR_BF16 ? go(bf16{}) : go(float{});
}

}  // namespace gdr
