// C ABI of the layer's backward pass and of its activation checkpoints
// (declared in include/kda_tril.h): host checks, then kernels enqueued on the
// caller's stream. Never allocates, copies or synchronises.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kda_tril.h"
#include "layer_checks.h"

using namespace kda;

namespace {

constexpr int64_t kMaxChunks = ((int64_t)1 << 23) - 1;  // 512 threads each

// Writable arguments overlap neither each other nor anything that is read.
template <size_t N, size_t M>
bool clash(const Span (&out)[N], const Span (&in)[M]) {
    for (size_t i = 0; i < N; ++i) {
        if (overlaps_any(out[i], in)) return true;
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

// Both pools of a backward call; they share slot, init and num_slots.
kda_status check_pools(Pool &read, Pool &grad, const float *state, float *dstate,
                       const int32_t *slot, const int32_t *init, int64_t num_slots,
                       int64_t num_seqs) {
    kda_status st = check_pool(read, const_cast<float *>(state), slot, init, num_slots, num_seqs);
    if (st == KDA_OK) st = check_pool(grad, dstate, slot, init, num_slots, num_seqs);
    if (st != KDA_OK) return st;
    if (read.base == nullptr) read = grad, read.base = nullptr;
    if (grad.base == nullptr) grad = read, grad.base = nullptr;
    return KDA_OK;
}

kda_status check_workspace(const void *workspace, size_t bytes, size_t need) {
    if ((!workspace && bytes) || !aligned(workspace, 16)) return KDA_ERR_INVALID_ARG;
    return bytes < need ? KDA_ERR_WORKSPACE : KDA_OK;
}

// ------------------------------------------------------------------ delta rule

kda_status delta_sizes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t Hk, int32_t K,
                       int32_t V) {
    if (tokens < 0 || num_seqs < 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || K <= 0 || V <= 0)
        return KDA_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || num_seqs > kMaxTokens || H > kMaxHeads || (K != 64 && K != 128) ||
        V % 32 != 0 || V > 256 || num_seqs > kMaxPairs / H ||
        grad_slots(tokens, num_seqs) > kMaxChunks / H ||
        num_seqs * H + 8 > kMaxItems / (V / 32))  // walks of 32 columns, in groups of 8
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t delta_chunks_bytes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t K, int32_t V) {
    return (size_t)grad_slots(tokens, num_seqs) * H * grad_chunk_floats(K, V) * 4;
}
size_t delta_bytes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t Hk, int32_t K, int32_t V) {
    if (tokens == 0) return 0;
    return delta_chunks_bytes(tokens, num_seqs, H, K, V) +
           (Hk == H ? 0 : (size_t)2 * tokens * H * K * 4);
}

struct DeltaGradArgs {
    const void *dout;
    kda_dtype out_dtype;
    const void *q, *k, *v;
    kda_dtype in_dtype;
    const float *g, *beta;
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    int32_t H, Hk, K, V, gate_dim;
    const float *state;
    float *dstate;
    const int32_t *slot, *init;
    int64_t num_slots;
    float scale;
    void *workspace;
    size_t workspace_bytes;
};

kda_status delta_backward(const DeltaGradArgs &a, const int32_t *cu, int64_t num_seqs,
                          int64_t tokens, int64_t dense_T, hipStream_t stream) {
    DeltaGradProblem p;
    memset(&p, 0, sizeof(p));
    if (!valid_dtype(a.in_dtype) || !valid_dtype(a.out_dtype) || !isfinite(a.scale))
        return KDA_ERR_INVALID_ARG;
    kda_status st = delta_sizes(tokens, num_seqs, a.H, a.Hk, a.K, a.V);
    if (st == KDA_ERR_INVALID_ARG) return st;
    if (a.gate_dim != 1 && a.gate_dim != a.K) return KDA_ERR_INVALID_ARG;
    if (st != KDA_OK) return st;
    st = check_requests(p.req, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK) return st;
    st = check_pools(p.pool, p.grad, a.state, a.dstate, a.slot, a.init, a.num_slots, num_seqs);
    if (st != KDA_OK) return st;
    if (num_seqs == 0 || (tokens == 0 && a.dstate == nullptr)) return KDA_OK;
    const size_t need = delta_bytes(tokens, num_seqs, a.H, a.Hk, a.K, a.V);
    st = check_workspace(a.workspace, a.workspace_bytes, need);
    if (st == KDA_ERR_INVALID_ARG) return st;
    const size_t T = (size_t)tokens, e = dtype_bytes(a.in_dtype);
    const size_t keys = T * a.Hk * a.K * e, values = T * a.H * a.V, gates = T * a.H * a.gate_dim * 4;
    const size_t pool = (size_t)a.num_slots * a.H * a.K * a.V * 4;
    if (tokens > 0) {
        const void *const all[] = {a.dout, a.q, a.k, a.v, a.g, a.dq, a.dk, a.dv, a.dg};
        for (const void *x : all)
            if (!x || !aligned(x, 16)) return KDA_ERR_INVALID_ARG;
        if (!a.beta || !a.dbeta || !aligned(a.beta, 4) || !aligned(a.dbeta, 4))
            return KDA_ERR_INVALID_ARG;
    }
    const Span in[] = {{a.dout, values * dtype_bytes(a.out_dtype)},
                       {a.q, keys},
                       {a.k, keys},
                       {a.v, values * e},
                       {a.g, gates},
                       {a.beta, T * a.H * 4},
                       {a.state, a.state ? pool : 0},
                       {cu, (size_t)(num_seqs + 1) * 4},
                       {a.slot, (size_t)num_seqs * 4},
                       {a.init, (size_t)num_seqs * 4}};
    const Span out[] = {{a.dq, keys},
                        {a.dk, keys},
                        {a.dv, values * e},
                        {a.dg, gates},
                        {a.dbeta, T * a.H * 4},
                        {a.dstate, a.dstate ? pool : 0},
                        {a.workspace, need}};
    if (clash(out, in)) return KDA_ERR_INVALID_ARG;
    if (st != KDA_OK) return st;
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.dout = a.dout;
    p.g = a.g;
    p.beta = a.beta;
    p.dq = a.dq;
    p.dk = a.dk;
    p.dv = a.dv;
    p.dg = a.dg;
    p.dbeta = a.dbeta;
    p.H = a.H;
    p.Hk = a.Hk;
    p.K = a.K;
    p.V = a.V;
    p.gate_stride = a.gate_dim;
    p.slots = (int32_t)grad_slots(tokens, num_seqs);
    p.scale = a.scale;
    p.work = static_cast<float *>(a.workspace);
    if (a.Hk != a.H && tokens > 0) {
        p.dq_head = p.work + delta_chunks_bytes(tokens, num_seqs, a.H, a.K, a.V) / 4;
        p.dk_head = p.dq_head + T * a.H * a.K;
    }
    return launch_delta_grad(p, (int)a.in_dtype, (int)a.out_dtype, stream) == hipSuccess
               ? KDA_OK : KDA_ERR_HIP;
}

// ----------------------------------------------------------------- convolution

kda_status conv_sizes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t d, int32_t W) {
    if (tokens < 0 || num_seqs < 0 || H <= 0 || d <= 0 || W <= 0) return KDA_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || num_seqs > kMaxItems || H > kMaxHeads || (d != 64 && d != 128) ||
        W < 2 || W > 4)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
size_t conv_part_bytes(int64_t tokens, int32_t H, int32_t d, int32_t W) {
    return (size_t)conv_grad_rows(tokens, conv_grad_segment(tokens, H, d)) * 3 * W * H * d * 4;
}
size_t conv_bytes(int64_t tokens, int64_t num_seqs, int32_t H, int32_t d, int32_t W) {
    return conv_part_bytes(tokens, H, d, W) + (size_t)num_seqs * 3 * H * (W - 1) * d * 4;
}

kda_status conv_backward(const void *dq, const void *dk, const void *dv, kda_dtype dtype,
                         const void *qkv, const float *qkv_scale, const float *conv_w, void *dqkv,
                         float *dconv_w, const int32_t *cu, int64_t num_seqs, int64_t tokens,
                         int64_t dense_T, int32_t H, int32_t d, int32_t W, const float *conv_state,
                         float *dconv_state, const int32_t *slot, const int32_t *init,
                         int64_t num_slots, float eps_l2, void *workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    ConvGradProblem p;
    memset(&p, 0, sizeof(p));
    if (!valid_dtype(dtype) || bad_eps(eps_l2)) return KDA_ERR_INVALID_ARG;
    kda_status st = conv_sizes(tokens, num_seqs, H, d, W);
    if (st != KDA_OK) return st;
    st = check_requests(p.req, cu, num_seqs, tokens, dense_T);
    if (st != KDA_OK) return st;
    st = check_pools(p.pool, p.grad, conv_state, dconv_state, slot, init, num_slots, num_seqs);
    if (st != KDA_OK) return st;
    if (dconv_state != nullptr &&
        num_seqs > (kMaxItems - conv_grad_tap_blocks(H, d, W)) / conv_grad_window_blocks(H, d, W))
        return KDA_ERR_UNSUPPORTED;
    if (!conv_w || !dconv_w || !aligned(conv_w, 16) || !aligned(dconv_w, 16))
        return KDA_ERR_INVALID_ARG;
    const size_t need = conv_bytes(tokens, num_seqs, H, d, W);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st == KDA_ERR_INVALID_ARG) return st;
    const size_t n = (size_t)tokens * H * d, each = n * dtype_bytes(dtype);
    const size_t taps = (size_t)3 * W * H * d * 4, pool = (size_t)num_slots * 3 * H * (W - 1) * d * 4;
    if (tokens > 0) {
        if (!dq || !dk || !dv || !qkv || !dqkv) return KDA_ERR_INVALID_ARG;
        if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dqkv, 16) ||
            !aligned(qkv, qkv_scale ? 8 : 16) || !aligned(qkv_scale, 4))
            return KDA_ERR_INVALID_ARG;
    }
    const Span in[] = {{dq, each},
                       {dk, each},
                       {dv, each},
                       {qkv, qkv_scale ? 3 * n : 3 * each},
                       {qkv_scale, (size_t)tokens * 3 * H * 4},
                       {conv_w, taps},
                       {conv_state, conv_state ? pool : 0},
                       {cu, (size_t)(num_seqs + 1) * 4},
                       {slot, (size_t)num_seqs * 4},
                       {init, (size_t)num_seqs * 4}};
    const Span out[] = {{dqkv, 3 * each},
                        {dconv_w, taps},
                        {dconv_state, dconv_state ? pool : 0},
                        {workspace, need}};
    if (clash(out, in)) return KDA_ERR_INVALID_ARG;
    if (st != KDA_OK) return st;
    p.dout[0] = dq;
    p.dout[1] = dk;
    p.dout[2] = dv;
    p.qkv = qkv;
    p.qkv_scale = qkv_scale;
    p.conv_w = conv_w;
    p.dqkv = dqkv;
    p.dconv_w = dconv_w;
    p.part = static_cast<float *>(workspace);
    p.old = p.part + conv_part_bytes(tokens, H, d, W) / 4;
    p.H = H;
    p.d = d;
    p.W = W;
    p.seg = conv_grad_segment(tokens, H, d);
    p.eps_l2 = eps_l2;
    return launch_conv_grad(p, (int)dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

// --------------------------------------------------------- norm and checkpoints

size_t norm_bytes(int64_t rows, int32_t H, int32_t d) {
    return (size_t)norm_grad_blocks(rows * H, d) * d * 4;
}

}  // namespace

extern "C" {

kda_status kda_prefill_backward_workspace_size(int64_t total_tokens, int64_t num_seqs, int32_t H,
                                               int32_t Hk, int32_t K, int32_t V, size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    const kda_status st = delta_sizes(total_tokens, num_seqs, H, Hk, K, V);
    if (st == KDA_OK) *bytes = delta_bytes(total_tokens, num_seqs, H, Hk, K, V);
    return st;
}

kda_status kda_prefill_backward_packed(
    const void *dout, kda_dtype out_dtype, const void *q, const void *k, const void *v,
    kda_dtype in_dtype, const float *g, const float *beta, void *dq, void *dk, void *dv, float *dg,
    float *dbeta, const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens, int32_t H,
    int32_t Hk, int32_t K, int32_t V, int32_t gate_dim, const float *state, float *dstate,
    const int32_t *slot, const int32_t *init, int64_t num_slots, float scale, void *workspace,
    size_t workspace_bytes, hipStream_t stream) {
    const DeltaGradArgs a = {dout, out_dtype, q, k, v, in_dtype, g, beta, dq, dk, dv, dg, dbeta,
                             H, Hk, K, V, gate_dim, state, dstate, slot, init, num_slots, scale,
                             workspace, workspace_bytes};
    return delta_backward(a, cu_seqlens, num_seqs, total_tokens, -1, stream);
}

kda_status kda_prefill_backward_dense(
    const void *dout, kda_dtype out_dtype, const void *q, const void *k, const void *v,
    kda_dtype in_dtype, const float *g, const float *beta, void *dq, void *dk, void *dv, float *dg,
    float *dbeta, int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
    int32_t gate_dim, const float *state, float *dstate, const int32_t *slot, const int32_t *init,
    int64_t num_slots, float scale, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const kda_status st = check_dense(B, T);
    if (st != KDA_OK) return st;
    const DeltaGradArgs a = {dout, out_dtype, q, k, v, in_dtype, g, beta, dq, dk, dv, dg, dbeta,
                             H, Hk, K, V, gate_dim, state, dstate, slot, init, num_slots, scale,
                             workspace, workspace_bytes};
    return delta_backward(a, nullptr, B, B * T, T, stream);
}

kda_status kda_conv_backward_workspace_size(int64_t total_tokens, int64_t num_seqs, int32_t H,
                                            int32_t head_dim, int32_t conv_width, size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    const kda_status st = conv_sizes(total_tokens, num_seqs, H, head_dim, conv_width);
    if (st == KDA_OK) *bytes = conv_bytes(total_tokens, num_seqs, H, head_dim, conv_width);
    return st;
}

kda_status kda_conv_backward_packed(const void *dq, const void *dk, const void *dv,
                                    kda_dtype dtype, const void *qkv, const float *qkv_scale,
                                    const float *conv_w, void *dqkv, float *dconv_w,
                                    const int32_t *cu_seqlens, int64_t num_seqs,
                                    int64_t total_tokens, int32_t H, int32_t head_dim,
                                    int32_t conv_width, const float *conv_state,
                                    float *dconv_state, const int32_t *slot, const int32_t *init,
                                    int64_t num_slots, float eps_l2, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
    return conv_backward(dq, dk, dv, dtype, qkv, qkv_scale, conv_w, dqkv, dconv_w, cu_seqlens,
                         num_seqs, total_tokens, -1, H, head_dim, conv_width, conv_state,
                         dconv_state, slot, init, num_slots, eps_l2, workspace, workspace_bytes,
                         stream);
}

kda_status kda_conv_backward_dense(const void *dq, const void *dk, const void *dv, kda_dtype dtype,
                                   const void *qkv, const float *qkv_scale, const float *conv_w,
                                   void *dqkv, float *dconv_w, int64_t B, int64_t T, int32_t H,
                                   int32_t head_dim, int32_t conv_width, const float *conv_state,
                                   float *dconv_state, const int32_t *slot, const int32_t *init,
                                   int64_t num_slots, float eps_l2, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    const kda_status st = check_dense(B, T);
    if (st != KDA_OK) return st;
    return conv_backward(dq, dk, dv, dtype, qkv, qkv_scale, conv_w, dqkv, dconv_w, nullptr, B,
                         B * T, T, H, head_dim, conv_width, conv_state, dconv_state, slot, init,
                         num_slots, eps_l2, workspace, workspace_bytes, stream);
}

kda_status kda_gated_norm_backward_workspace_size(int64_t rows, int32_t H, int32_t head_dim,
                                                  size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    const kda_status st = vector_sizes(rows, H, head_dim);
    if (st == KDA_OK) *bytes = norm_bytes(rows, H, head_dim);
    return st;
}

kda_status kda_gated_norm_backward(const void *dout, const void *o, const void *z, kda_dtype dtype,
                                   const float *o_scale, const float *z_scale, const float *norm_w,
                                   void *d_o, void *dz, float *dnorm_w, int64_t rows, int32_t H,
                                   int32_t head_dim, float eps_norm, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    if (!valid_dtype(dtype) || bad_eps(eps_norm) || (o_scale == nullptr) != (z_scale == nullptr))
        return KDA_ERR_INVALID_ARG;
    kda_status st = vector_sizes(rows, H, head_dim);
    if (st != KDA_OK) return st;
    if (!dnorm_w || !aligned(dnorm_w, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = norm_bytes(rows, H, head_dim);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st == KDA_ERR_INVALID_ARG) return st;
    const size_t vecs = (size_t)rows * H, n = vecs * head_dim, e = n * dtype_bytes(dtype);
    if (rows > 0) {
        const size_t least = o_scale ? 8 : 16;
        if (!dout || !o || !z || !norm_w || !d_o || !dz) return KDA_ERR_INVALID_ARG;
        if (!aligned(dout, 16) || !aligned(o, least) || !aligned(z, least) ||
            !aligned(d_o, 16) || !aligned(dz, 16) || !aligned(norm_w, 4) ||
            !aligned(o_scale, 4) || !aligned(z_scale, 4))
            return KDA_ERR_INVALID_ARG;
    }
    const Span in[] = {{dout, e},
                       {o, o_scale ? n : e},
                       {z, o_scale ? n : e},
                       {o_scale, vecs * 4},
                       {z_scale, vecs * 4},
                       {norm_w, (size_t)head_dim * 4}};
    const Span out[] = {{d_o, e}, {dz, e}, {dnorm_w, (size_t)head_dim * 4}, {workspace, need}};
    if (clash(out, in)) return KDA_ERR_INVALID_ARG;
    if (st != KDA_OK) return st;
    NormGradProblem p;
    memset(&p, 0, sizeof(p));
    p.dout = dout;
    p.o = o;
    p.z = z;
    p.o_scale = o_scale;
    p.z_scale = z_scale;
    p.norm_w = norm_w;
    p.d_o = d_o;
    p.dz = dz;
    p.dnorm_w = dnorm_w;
    p.part = static_cast<float *>(workspace);
    p.vecs = rows * H;
    p.d = head_dim;
    p.eps_norm = eps_norm;
    return launch_norm_grad(p, (int)dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_checkpoint(const void *x, kda_dtype dtype, int8_t *codes, float *scale,
                          int64_t rows, int32_t H, int32_t head_dim, hipStream_t stream) {
    if (!valid_dtype(dtype)) return KDA_ERR_INVALID_ARG;
    const kda_status st = vector_launch_sizes(rows, H, head_dim);
    if (st != KDA_OK || rows == 0) return st;
    if (!x || !codes || !scale || !aligned(x, 16) || !aligned(codes, 8) || !aligned(scale, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t vecs = (size_t)rows * H, n = vecs * head_dim;
    const Span in[] = {{x, n * dtype_bytes(dtype)}};
    const Span out[] = {{codes, n}, {scale, vecs * 4}};
    if (clash(out, in)) return KDA_ERR_INVALID_ARG;
    CheckpointProblem p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.codes = codes;
    p.scale = scale;
    p.vecs = rows * H;
    p.d = head_dim;
    return launch_checkpoint(p, (int)dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_checkpoint_load(const int8_t *codes, const float *scale, void *out,
                               kda_dtype out_dtype, int64_t rows, int32_t H, int32_t head_dim,
                               hipStream_t stream) {
    if (!valid_dtype(out_dtype)) return KDA_ERR_INVALID_ARG;
    const kda_status st = vector_launch_sizes(rows, H, head_dim);
    if (st != KDA_OK || rows == 0) return st;
    if (!codes || !scale || !out || !aligned(codes, 8) || !aligned(scale, 4) || !aligned(out, 16))
        return KDA_ERR_INVALID_ARG;
    const size_t vecs = (size_t)rows * H, n = vecs * head_dim;
    const Span in[] = {{codes, n}, {scale, vecs * 4}};
    const Span to[] = {{out, n * dtype_bytes(out_dtype)}};
    if (clash(to, in)) return KDA_ERR_INVALID_ARG;
    CheckpointProblem p;
    memset(&p, 0, sizeof(p));
    p.codes = const_cast<int8_t *>(codes);
    p.scale = const_cast<float *>(scale);
    p.out = out;
    p.vecs = rows * H;
    p.d = head_dim;
    return launch_checkpoint(p, (int)out_dtype, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status kda_gated_norm_checkpoint(const void *o, const void *z, kda_dtype in_dtype,
                                     const float *norm_w, void *out, kda_dtype out_dtype,
                                     int8_t *o_codes, float *o_scale, int8_t *z_codes,
                                     float *z_scale, int64_t rows, int32_t H, int32_t head_dim,
                                     float eps_norm, hipStream_t stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype) || bad_eps(eps_norm))
        return KDA_ERR_INVALID_ARG;
    const kda_status st = vector_launch_sizes(rows, H, head_dim);
    if (st != KDA_OK || rows == 0) return st;
    if (!o || !z || !norm_w || !out || !o_codes || !o_scale || !z_codes || !z_scale ||
        !aligned(o, 16) || !aligned(z, 16) || !aligned(out, 16) || !aligned(norm_w, 4) ||
        !aligned(o_codes, 8) || !aligned(z_codes, 8) || !aligned(o_scale, 4) ||
        !aligned(z_scale, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t vecs = (size_t)rows * H, n = vecs * head_dim, e = n * dtype_bytes(in_dtype);
    const Span in[] = {{o, e}, {z, e}, {norm_w, (size_t)head_dim * 4}};
    const Span to[] = {{out, n * dtype_bytes(out_dtype)},
                       {o_codes, n}, {o_scale, vecs * 4}, {z_codes, n}, {z_scale, vecs * 4}};
    if (clash(to, in)) return KDA_ERR_INVALID_ARG;
    NormCheckpointProblem p;
    memset(&p, 0, sizeof(p));
    p.norm.o = o;
    p.norm.z = z;
    p.norm.norm_w = norm_w;
    p.norm.out = out;
    p.norm.vecs = rows * H;
    p.norm.d = head_dim;
    p.norm.eps_norm = eps_norm;
    p.o_codes = o_codes;
    p.o_scale = o_scale;
    p.z_codes = z_codes;
    p.z_scale = z_scale;
    return launch_norm_checkpoint(p, (int)in_dtype, (int)out_dtype, stream) == hipSuccess
               ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
