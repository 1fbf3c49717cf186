// C ABI of the KDA layer's calls (declared in include/kda_tril.h): host
// checks, then one enqueue on the caller's stream. Never allocates, copies or
// synchronises.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kda_layer.h"
#include "kda_tril.h"

using namespace kda;

namespace {

constexpr int64_t kMaxTokens = (int64_t)INT32_MAX - 64;  // int32 rows in the kernels
constexpr int32_t kMaxHeads = 4096;
// (request, head) pairs of one launch: at most 512 threads each, fewer than
// 2^32 threads in all
constexpr int64_t kMaxPairs = ((int64_t)1 << 23) - 1;

bool valid_dtype(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16 || d == KDA_F16; }
size_t dtype_bytes(kda_dtype d) { return d == KDA_F32 ? 4 : 2; }
bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Span {
    const void *p;
    size_t n;
};
bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}
template <size_t N>
bool overlaps_any(Span a, const Span (&b)[N]) {
    for (const Span &x : b)
        if (overlap(a, x)) return true;
    return false;
}

bool bad_eps(float e) { return !(e >= 0.0f) || e > 1e30f; }  // negative, NaN or infinite

// The requests of a call. dense_T < 0: packed with cu_seqlens.
kda_status check_requests(Requests &r, const int32_t *cu, int64_t num_seqs, int64_t tokens,
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

kda_status check_dense(int64_t B, int64_t T) {
    if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
    if (B > 0 && T > kMaxTokens / B) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_pool(Pool &p, float *base, const int32_t *slot, const int32_t *init,
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

struct DeltaArgs {
    const void *q, *k, *v;
    kda_dtype in_dtype;
    const float *g, *beta;
    void *out;
    kda_dtype out_dtype;
    int32_t H, Hk, K, V, gate_dim;
    float *state;
    const int32_t *slot, *init;
    int64_t num_slots;
    float scale;
};

kda_status check_delta(DeltaProblem &p, const DeltaArgs &a, const int32_t *cu, int64_t num_seqs,
                       int64_t tokens, int64_t dense_T) {
    memset(&p, 0, sizeof(p));
    if (!valid_dtype(a.in_dtype) || !valid_dtype(a.out_dtype) || a.H <= 0 || a.Hk <= 0 ||
        a.H % a.Hk != 0 || a.K <= 0 || a.V <= 0 || !isfinite(a.scale))
        return KDA_ERR_INVALID_ARG;
    if (a.gate_dim != 1 && a.gate_dim != a.K) return KDA_ERR_INVALID_ARG;
    if (a.H > kMaxHeads || (a.K != 64 && a.K != 128) || a.V % 32 != 0 || a.V > 256)
        return KDA_ERR_UNSUPPORTED;
    kda_status st = check_requests(p.req, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK) return st;
    if (num_seqs > kMaxPairs / a.H) return KDA_ERR_UNSUPPORTED;
    st = check_pool(p.pool, a.state, a.slot, a.init, a.num_slots, num_seqs);
    if (st != KDA_OK) return st;
    const Span pool = {a.state, p.pool.base ? (size_t)a.num_slots * a.H * a.K * a.V * 4 : 0};
    const Span lists[] = {{cu, (size_t)(num_seqs + 1) * 4},
                          {a.slot, (size_t)num_seqs * 4},
                          {a.init, (size_t)num_seqs * 4}};
    if (overlaps_any(pool, lists)) return KDA_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.out) return KDA_ERR_INVALID_ARG;
        if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.g, 16) ||
            !aligned(a.beta, 4) || !aligned(a.out, 16))
            return KDA_ERR_INVALID_ARG;
        const size_t T = (size_t)tokens, e = dtype_bytes(a.in_dtype);
        const Span in[] = {{a.q, T * a.Hk * a.K * e},       {a.k, T * a.Hk * a.K * e},
                           {a.v, T * a.H * a.V * e},        {a.g, T * a.H * a.gate_dim * 4},
                           {a.beta, T * (size_t)a.H * 4},   lists[0], lists[1], lists[2]};
        const Span out = {a.out, T * a.H * a.V * dtype_bytes(a.out_dtype)};
        if (overlaps_any(out, in) || overlap(out, pool) || overlaps_any(pool, in))
            return KDA_ERR_INVALID_ARG;
    }
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.g = a.g;
    p.beta = a.beta;
    p.out = a.out;
    p.H = a.H;
    p.Hk = a.Hk;
    p.K = a.K;
    p.V = a.V;
    p.gate_stride = a.gate_dim;
    p.out_dt = (int32_t)a.out_dtype;
    p.scale = a.scale;
    return KDA_OK;
}

// Nothing to do: no request, or no token and no state to leave behind.
bool idle(const DeltaProblem &p) {
    return p.req.num_seqs == 0 || (p.req.total_tokens == 0 && p.pool.base == nullptr);
}

// Bytes with which a call cuts its prompts into segments of seg tokens.
size_t prefill_bytes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t K, int32_t V,
                     int32_t seg) {
    if (seg == 0) return 0;
    const size_t segs = (size_t)prefill_max_segments(tokens, num_seqs, seg);
    return (size_t)H * K * 4 * (segs * (V + K) + (size_t)num_seqs * V);
}

kda_status prefill(const DeltaArgs &a, const int32_t *cu, int64_t num_seqs, int64_t tokens,
                   int64_t dense_T, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    DeltaProblem p;
    const kda_status st = check_delta(p, a, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK) return st;
    if ((!workspace && workspace_bytes) || (workspace && !aligned(workspace, 16)))
        return KDA_ERR_INVALID_ARG;
    if (idle(p)) return KDA_OK;
    const int32_t seg = prefill_segments(tokens, num_seqs, a.H, a.V);
    const size_t need = prefill_bytes(tokens, num_seqs, a.H, a.K, a.V, seg);
    if (need && workspace_bytes >= need) {
        const size_t T = (size_t)tokens, e = dtype_bytes(a.in_dtype);
        const Span used[] = {{a.q, T * a.Hk * a.K * e},
                             {a.k, T * a.Hk * a.K * e},
                             {a.v, T * a.H * a.V * e},
                             {a.g, T * a.H * a.gate_dim * 4},
                             {a.beta, T * (size_t)a.H * 4},
                             {a.out, T * a.H * a.V * dtype_bytes(a.out_dtype)},
                             {cu, (size_t)(num_seqs + 1) * 4},
                             {a.slot, (size_t)num_seqs * 4},
                             {a.init, (size_t)num_seqs * 4},
                             {a.state, (size_t)(a.state ? a.num_slots : 0) * a.H * a.K * a.V * 4}};
        if (overlaps_any({workspace, need}, used)) return KDA_ERR_INVALID_ARG;
        p.seg = seg;
        p.segs = (int32_t)prefill_max_segments(tokens, num_seqs, seg);
        const size_t states = (size_t)a.H * a.K * a.V;
        p.seg_state = static_cast<float *>(workspace);
        p.seg_map = p.seg_state + (size_t)p.segs * states;
        p.seg_first = p.seg_map + (size_t)p.segs * a.H * a.K * a.K;
    }
    return launch_prefill(p, (int)a.in_dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status recurrent(const DeltaArgs &a, const int32_t *cu, int64_t num_seqs, int64_t tokens,
                     int64_t dense_T, hipStream_t stream) {
    DeltaProblem p;
    const kda_status st = check_delta(p, a, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK || idle(p)) return st;
    return launch_recurrent(p, (int)a.in_dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status conv(const void *qkv, kda_dtype dtype, const float *conv_w, void *q, void *k, void *v,
                const int32_t *cu, int64_t num_seqs, int64_t tokens, int64_t dense_T, int32_t H,
                int32_t d, int32_t W, float *conv_state, const int32_t *slot, const int32_t *init,
                int64_t num_slots, float eps_l2, hipStream_t stream) {
    ConvProblem p;
    memset(&p, 0, sizeof(p));
    if (!valid_dtype(dtype) || H <= 0 || d <= 0 || W <= 0 || bad_eps(eps_l2))
        return KDA_ERR_INVALID_ARG;
    if (H > kMaxHeads || (d != 64 && d != 128) || W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    kda_status st = check_requests(p.req, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK) return st;
    st = check_pool(p.pool, conv_state, slot, init, num_slots, num_seqs);
    if (st != KDA_OK) return st;
    if (num_seqs == 0 || (tokens == 0 && conv_state == nullptr)) return KDA_OK;
    if (!conv_w || !aligned(conv_w, 16)) return KDA_ERR_INVALID_ARG;
    const Span pool = {conv_state, p.pool.base ? (size_t)num_slots * 3 * H * (W - 1) * d * 4 : 0};
    const Span kept[] = {{conv_w, (size_t)3 * W * H * d * 4},
                         {cu, (size_t)(num_seqs + 1) * 4},
                         {slot, (size_t)num_seqs * 4},
                         {init, (size_t)num_seqs * 4}};
    if (overlaps_any(pool, kept)) return KDA_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!qkv || !q || !k || !v) return KDA_ERR_INVALID_ARG;
        if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))
            return KDA_ERR_INVALID_ARG;
        const size_t each = (size_t)tokens * H * d * dtype_bytes(dtype);
        const Span in[] = {{qkv, 3 * each}, kept[0], kept[1], kept[2], kept[3]};
        const Span out[] = {{q, each}, {k, each}, {v, each}};
        for (const Span &o : out)
            if (overlaps_any(o, in) || overlap(o, pool)) return KDA_ERR_INVALID_ARG;
        if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2]) ||
            overlaps_any(pool, in))
            return KDA_ERR_INVALID_ARG;
    }
    p.qkv = qkv;
    p.conv_w = conv_w;
    p.out[0] = q;
    p.out[1] = k;
    p.out[2] = v;
    p.H = H;
    p.d = d;
    p.W = W;
    p.eps_l2 = eps_l2;
    const hipError_t e = launch_conv(p, (int)dtype, stream);
    return e == hipSuccess                ? KDA_OK
           : e == hipErrorInvalidConfiguration ? KDA_ERR_UNSUPPORTED  // grid too large
                                               : KDA_ERR_HIP;
}

}  // namespace

extern "C" {

kda_status kda_chunk_map(const int32_t *seq_lens, int64_t num_seqs, int64_t total_tokens,
                         int32_t chunk_size, int32_t *cu_seqlens, int32_t *chunk_indices,
                         int64_t max_chunks, int32_t *num_chunks, hipStream_t stream) {
    if (num_seqs < 0 || total_tokens < 0 || max_chunks < 0) return KDA_ERR_INVALID_ARG;
    if (chunk_size != 16 && chunk_size != 32 && chunk_size != 64) return KDA_ERR_INVALID_ARG;
    if ((chunk_indices == nullptr) != (max_chunks == 0)) return KDA_ERR_INVALID_ARG;
    if (num_seqs > kMaxTokens || total_tokens > kMaxTokens || max_chunks > kMaxTokens)
        return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens || (num_seqs > 0 && !seq_lens)) return KDA_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(chunk_indices, 8) ||
        !aligned(num_chunks, 4))
        return KDA_ERR_INVALID_ARG;
    const Span all[] = {{seq_lens, (size_t)num_seqs * 4},
                        {cu_seqlens, (size_t)(num_seqs + 1) * 4},
                        {chunk_indices, (size_t)max_chunks * 8},
                        {num_chunks, 4}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (overlap(all[i], all[j])) return KDA_ERR_INVALID_ARG;
    MapProblem p;
    memset(&p, 0, sizeof(p));
    p.seq_lens = seq_lens;
    p.cu = cu_seqlens;
    p.map = chunk_indices;
    p.count = num_chunks;
    p.num_seqs = (int32_t)num_seqs;
    p.total_tokens = (int32_t)total_tokens;
    p.chunk = chunk_size;
    p.max_chunks = (int32_t)max_chunks;
    return launch_map(p, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_conv_prefill_packed(const void *qkv, kda_dtype dtype, const float *conv_w, void *q,
                                   void *k, void *v, const int32_t *cu_seqlens, int64_t num_seqs,
                                   int64_t total_tokens, int32_t H, int32_t head_dim,
                                   int32_t conv_width, float *conv_state, const int32_t *slot,
                                   const int32_t *init, int64_t num_slots, float eps_l2,
                                   hipStream_t stream) {
    return conv(qkv, dtype, conv_w, q, k, v, cu_seqlens, num_seqs, total_tokens, -1, H, head_dim,
                conv_width, conv_state, slot, init, num_slots, eps_l2, stream);
}

kda_status kda_conv_prefill_dense(const void *qkv, kda_dtype dtype, const float *conv_w, void *q,
                                  void *k, void *v, int64_t B, int64_t T, int32_t H,
                                  int32_t head_dim, int32_t conv_width, float *conv_state,
                                  const int32_t *slot, const int32_t *init, int64_t num_slots,
                                  float eps_l2, hipStream_t stream) {
    const kda_status st = check_dense(B, T);
    if (st != KDA_OK) return st;
    return conv(qkv, dtype, conv_w, q, k, v, nullptr, B, B * T, T, H, head_dim, conv_width,
                conv_state, slot, init, num_slots, eps_l2, stream);
}

kda_status kda_prefill_workspace_size(int64_t total_tokens, int64_t num_seqs, int32_t H, int32_t K,
                                      int32_t V, size_t *bytes) {
    if (!bytes || total_tokens < 0 || num_seqs < 0 || H <= 0 || K <= 0 || V <= 0)
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > kMaxTokens || num_seqs > kMaxTokens || H > kMaxHeads ||
        (K != 64 && K != 128) || V % 32 != 0 || V > 256 || num_seqs > kMaxPairs / H)
        return KDA_ERR_UNSUPPORTED;
    *bytes = prefill_bytes(total_tokens, num_seqs, H, K, V,
                           prefill_segments(total_tokens, num_seqs, H, V));
    return KDA_OK;
}

kda_status kda_prefill_packed(const void *q, const void *k, const void *v, kda_dtype in_dtype,
                              const float *g, const float *beta, void *out, kda_dtype out_dtype,
                              const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens,
                              int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t gate_dim,
                              float *state, const int32_t *slot, const int32_t *init,
                              int64_t num_slots, float scale, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    const DeltaArgs a = {q, k, v, in_dtype, g,     beta, out,  out_dtype, H,
                         Hk, K, V, gate_dim, state, slot, init, num_slots, scale};
    return prefill(a, cu_seqlens, num_seqs, total_tokens, -1, workspace, workspace_bytes, stream);
}

kda_status kda_prefill_dense(const void *q, const void *k, const void *v, kda_dtype in_dtype,
                             const float *g, const float *beta, void *out, kda_dtype out_dtype,
                             int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                             int32_t gate_dim, float *state, const int32_t *slot,
                             const int32_t *init, int64_t num_slots, float scale, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    const kda_status st = check_dense(B, T);
    if (st != KDA_OK) return st;
    const DeltaArgs a = {q, k, v, in_dtype, g,     beta, out,  out_dtype, H,
                         Hk, K, V, gate_dim, state, slot, init, num_slots, scale};
    return prefill(a, nullptr, B, B * T, T, workspace, workspace_bytes, stream);
}

kda_status kda_recurrent_packed(const void *q, const void *k, const void *v, kda_dtype in_dtype,
                                const float *g, const float *beta, void *out, kda_dtype out_dtype,
                                const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens,
                                int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t gate_dim,
                                float *state, const int32_t *slot, const int32_t *init,
                                int64_t num_slots, float scale, hipStream_t stream) {
    const DeltaArgs a = {q, k, v, in_dtype, g,     beta, out,  out_dtype, H,
                         Hk, K, V, gate_dim, state, slot, init, num_slots, scale};
    return recurrent(a, cu_seqlens, num_seqs, total_tokens, -1, stream);
}

kda_status kda_recurrent_dense(const void *q, const void *k, const void *v, kda_dtype in_dtype,
                               const float *g, const float *beta, void *out, kda_dtype out_dtype,
                               int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                               int32_t gate_dim, float *state, const int32_t *slot,
                               const int32_t *init, int64_t num_slots, float scale,
                               hipStream_t stream) {
    const kda_status st = check_dense(B, T);
    if (st != KDA_OK) return st;
    const DeltaArgs a = {q, k, v, in_dtype, g,     beta, out,  out_dtype, H,
                         Hk, K, V, gate_dim, state, slot, init, num_slots, scale};
    return recurrent(a, nullptr, B, B * T, T, stream);
}

kda_status kda_gated_norm(const void *o, const void *z, kda_dtype in_dtype, const float *norm_w,
                          void *out, kda_dtype out_dtype, int64_t rows, int32_t H,
                          int32_t head_dim, float eps_norm, hipStream_t stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || rows < 0 || H <= 0 ||
        head_dim <= 0 || bad_eps(eps_norm))
        return KDA_ERR_INVALID_ARG;
    // 16 lanes per vector at most, fewer than 2^32 threads
    if (rows > kMaxTokens || H > kMaxHeads || (head_dim != 64 && head_dim != 128) ||
        rows > ((int64_t)1 << 28) / H - 1)
        return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!o || !z || !norm_w || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(o, 16) || !aligned(z, 16) || !aligned(out, 16) || !aligned(norm_w, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t e = (size_t)rows * H * head_dim;
    const Span so = {out, e * dtype_bytes(out_dtype)};
    const Span in[] = {{z, e * dtype_bytes(in_dtype)}, {norm_w, (size_t)head_dim * 4}};
    const bool in_place = o == out && in_dtype == out_dtype;
    if (overlaps_any(so, in) || (!in_place && overlap(so, {o, e * dtype_bytes(in_dtype)})))
        return KDA_ERR_INVALID_ARG;
    NormProblem p;
    memset(&p, 0, sizeof(p));
    p.o = o;
    p.z = z;
    p.norm_w = norm_w;
    p.out = out;
    p.vecs = rows * H;
    p.d = head_dim;
    p.eps_norm = eps_norm;
    return launch_norm(p, (int)in_dtype, (int)out_dtype, stream) == hipSuccess ? KDA_OK
                                                                               : KDA_ERR_HIP;
}

}  // extern "C"
