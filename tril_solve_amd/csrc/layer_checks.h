// Host checks of arguments that the layer's calls and their gradients share.
#pragma once

#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "kda_layer.h"
#include "kda_tril.h"

namespace kda {

constexpr int64_t kMaxTokens = (int64_t)INT32_MAX - 64;  // int32 rows in the kernels
constexpr int32_t kMaxHeads = 4096;
// (request, head) pairs of one launch: at most 512 threads each, fewer than
// 2^32 threads in all
constexpr int64_t kMaxPairs = ((int64_t)1 << 23) - 1;
constexpr int64_t kMaxItems = ((int64_t)1 << 24) - 1;  // 256 threads each, likewise
constexpr int64_t kMaxVectors = ((int64_t)1 << 28) - 1;

inline bool valid_dtype(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16 || d == KDA_F16; }
inline size_t dtype_bytes(kda_dtype d) { return d == KDA_F32 ? 4 : 2; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Span {
    const void *p;
    size_t n;
};
inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}
template <size_t N>
inline bool overlaps_any(Span a, const Span (&b)[N]) {
    for (const Span &x : b)
        if (overlap(a, x)) return true;
    return false;
}

inline bool bad_eps(float e) { return !(e >= 0.0f) || e > 1e30f; }  // negative, NaN or infinite

// The requests of a call. dense_T < 0: packed with cu_seqlens.
inline kda_status check_requests(Requests &r, const int32_t *cu, int64_t num_seqs, int64_t tokens,
                          int64_t dense_T) {
    if (num_seqs < 0 || tokens < 0) return KDA_ERR_INVALID_ARG;
    if (num_seqs > kMaxTokens || tokens > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (dense_T < 0 && num_seqs > 0 && (cu == nullptr || !aligned(cu, 4)))
        return KDA_ERR_INVALID_ARG;
    r.cu = dense_T < 0 ? cu : nullptr;
    r.num_seqs = (int32_t)num_seqs;
    r.seq_len = dense_T < 0 ? 0 : (int32_t)dense_T;
    r.total_tokens = (int32_t)tokens;
    return KDA_OK;
}

inline kda_status check_dense(int64_t B, int64_t T) {
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    if (B > 0 && T > kMaxTokens / B) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

inline kda_status check_pool(Pool &p, float *base, const int32_t *slot, const int32_t *init,
                      int64_t num_slots, int64_t num_seqs) {
    memset(&p, 0, sizeof(p));
    if (base == nullptr) return KDA_OK;
    if (num_slots < 0 || !aligned(base, 16) || !aligned(slot, 4) || !aligned(init, 4))
        return KDA_ERR_INVALID_ARG;
    if (num_slots > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (num_slots == 0 || (slot == nullptr && num_slots < num_seqs)))
        return KDA_ERR_INVALID_ARG;
    p.base = base;
    p.slot = slot;
    p.init = init;
    p.num_slots = (int32_t)num_slots;
    return KDA_OK;
}

// rows x H vectors of d channels.
inline kda_status vector_sizes(int64_t rows, int32_t H, int32_t d) {
    if (rows < 0 || H <= 0 || d <= 0) return KDA_ERR_INVALID_ARG;
    if (rows > kMaxTokens || H > kMaxHeads || (d != 64 && d != 128) || rows > kMaxVectors / H)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// Likewise for a launch that takes d / 8 lanes to a vector in workgroups of 256: below
// 2^32 threads in all, the last workgroup's idle ones counted.
inline kda_status vector_launch_sizes(int64_t rows, int32_t H, int32_t d) {
    const kda_status st = vector_sizes(rows, H, d);
    return st == KDA_OK && rows * H * (d / 8) > kMaxItems * 256 ? KDA_ERR_UNSUPPORTED : st;
}

}  // namespace kda
