// Argument checks that the layer operators' entry points share (gdr_mixer_api.hip,
// gdr_attn_api.hip); they set the calling thread's error message.
#pragma once

#include "gdr_mixer.hpp"

namespace gdr {

inline bool is_dtype(int32_t t) { return t == GDR_F32 || t == GDR_BF16; }
// a type that may be the io type or fp32
inline bool io_or_f32(int32_t t, int32_t io) { return t == io || t == GDR_F32; }
inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

struct Ptr {
    const void* p;
    int32_t dtype;
    bool required;
    const char* name;
};
template <int N>
gdr_status_t check_ptrs(const Ptr (&ptrs)[N], bool any) {
    for (const Ptr& t : ptrs) {
        if (t.required && any && !t.p) return fail(GDR_ERR_NULL, "%s is required", t.name);
        if (!aligned(t.p, (size_t)size_of(t.dtype)))
            return fail(GDR_ERR_SHAPE, "%s is not aligned to its element type", t.name);
    }
    return GDR_OK;
}

inline gdr_status_t check_tokens(int64_t batch, int64_t seq_len, int32_t num_seqs, int32_t channels) {
    if (batch < 0 || seq_len < 0 || num_seqs < 0)
        return fail(GDR_ERR_SHAPE, "batch, seq_len and num_seqs must be >= 0");
    if (channels < 1) return fail(GDR_ERR_SHAPE, "channels must be positive (got %d)", channels);
    const int64_t most = ((int64_t)1 << 31) - 1 - 64;
    if (batch > most || seq_len > most || (batch > 0 && seq_len > most / batch))
        return fail(GDR_ERR_SHAPE, "total tokens exceed the int32 token index");
    return GDR_OK;
}

// Sequences of a call; *max_len: the longest (host).
inline gdr_status_t check_seqs(int64_t batch, int64_t seq_len, int32_t num_seqs, const int32_t* cu_dev,
                        const int32_t* cu_host, int64_t* max_len) {
    if ((cu_dev == nullptr) != (cu_host == nullptr))
        return fail(GDR_ERR_NULL, "cu_seqlens_dev and cu_seqlens_host must both be given or both be NULL");
    if (!cu_host) {
        if (num_seqs != batch)
            return fail(GDR_ERR_SHAPE, "num_seqs (%d) must equal batch (%lld) without cu_seqlens", num_seqs,
                        (long long)batch);
        *max_len = seq_len;
        return GDR_OK;
    }
    if (batch != 1) return fail(GDR_ERR_SEQLENS, "cu_seqlens requires batch == 1");
    if (num_seqs < 1) return fail(GDR_ERR_SEQLENS, "cu_seqlens needs num_seqs >= 1");
    if (!aligned(cu_dev, 4)) return fail(GDR_ERR_SHAPE, "cu_seqlens_dev is not aligned to its element type");
    if (cu_host[0] != 0) return fail(GDR_ERR_SEQLENS, "cu_seqlens[0] = %d, expected 0", cu_host[0]);
    *max_len = 0;
    for (int32_t n = 0; n < num_seqs; ++n) {
        if (cu_host[n + 1] < cu_host[n]) return fail(GDR_ERR_SEQLENS, "cu_seqlens decreases at %d", n);
        const int64_t len = (int64_t)cu_host[n + 1] - cu_host[n];
        *max_len = len > *max_len ? len : *max_len;
    }
    if ((int64_t)cu_host[num_seqs] != seq_len)
        return fail(GDR_ERR_SEQLENS, "cu_seqlens[N] = %d but seq_len = %lld", cu_host[num_seqs], (long long)seq_len);
    return GDR_OK;
}

constexpr int64_t kMostStride = (int64_t)1 << 40;
inline gdr_status_t check_stride(const char* name, int64_t stride, int64_t row, int64_t most = kMostStride) {
    if (stride < row || stride > most)
        return fail(GDR_ERR_SHAPE, "%s (%lld) must be at least the row's %lld elements and at most %lld", name,
                    (long long)stride, (long long)row, (long long)most);
    return GDR_OK;
}

inline gdr_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDR_OK;
    if (!ws) return fail(GDR_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(ws, 256)) return fail(GDR_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (have < need) return fail(GDR_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return GDR_OK;
}

inline gdr_status_t done(hipError_t e) {
    if (e == hipErrorInvalidConfiguration) return fail(GDR_ERR_SHAPE, "problem too large for one launch");
    if (e != hipSuccess) return fail(GDR_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    clear_error();
    return GDR_OK;
}

}  // namespace gdr

#define GDR_TRY(expr)                            \
    do {                                         \
        const gdr_status_t st_ = (expr);         \
        if (st_ != GDR_OK) return st_;           \
    } while (0)
