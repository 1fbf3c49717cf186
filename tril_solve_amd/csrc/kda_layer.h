// Problem descriptions and launchers of the KDA layer's kernels around the
// solver and the decode step (internal; the public interface is
// include/kda_tril.h).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace kda {

// Requests of one call: packed (cu_seqlens, device memory) or dense rows of
// seq_len tokens each.
struct Requests {
    const int32_t *cu;  // [num_seqs + 1] or null (dense)
    int32_t num_seqs;
    int32_t seq_len;       // dense T
    int32_t total_tokens;  // rows of every token tensor
};

// A pool of per-request state (recurrent states or convolution windows).
struct Pool {
    float *base;          // null: every request starts from zeros, nothing is kept
    const int32_t *slot;  // [num_seqs] or null (request n uses slot n)
    const int32_t *init;  // [num_seqs] or null (every request continues)
    int32_t num_slots;
};

// Gated delta rule, chunked or recurrent; layouts as in the C ABI.
struct DeltaProblem {
    Requests req;
    Pool pool;         // [num_slots, H, K, V]
    const void *q;     // [T, Hk, K]
    const void *k;     // [T, Hk, K]
    const void *v;     // [T, H, V]
    const float *g;    // [T, H, K] or [T, H]
    const float *beta; // [T, H]
    void *out;         // [T, H, V]
    int32_t H, Hk, K, V;
    int32_t gate_stride;  // elements of g per (token, head): K or 1
    int32_t out_dt;       // kda_dtype of out
    float scale;
    // Prompts cut into segments of `seg` tokens (0: not cut), at most `segs` of
    // them over all requests (chunked form only; see prefill_segments)
    int32_t seg, segs;
    float *seg_state;  // [segs, H, K, V] the state behind a segment
    float *seg_map;    // [segs, H, K, K] what a segment makes of the state before it
    float *seg_first;  // [num_seqs, H, K, V] the state before the first segment
};

// Tokens per segment of a call on these sizes, or 0 where cutting does not pay.
int32_t prefill_segments(int64_t total_tokens, int64_t num_seqs, int32_t H, int32_t V);
// Most segments that the requests of a call can have.
inline int64_t prefill_max_segments(int64_t total_tokens, int64_t num_seqs, int32_t seg) {
    return total_tokens / seg + num_seqs;
}

struct ConvProblem {
    Requests req;
    Pool pool;            // [num_slots, 3, H, W - 1, d]
    const void *qkv;      // [T, 3, H, d]
    const float *conv_w;  // [3, W, H, d]
    void *out[3];         // q, k, v: [T, H, d]
    int32_t H, d, W;
    int32_t seg;          // tokens per wavefront
    float eps_l2;
};

struct NormProblem {
    const void *o, *z;    // [rows, H, d]
    const float *norm_w;  // [d]
    void *out;
    int64_t vecs;         // rows * H
    int32_t d;
    float eps_norm;
};

struct MapProblem {
    const int32_t *seq_lens;  // [num_seqs]
    int32_t *cu;              // [num_seqs + 1]
    int32_t *map;             // [max_chunks][2]
    int32_t *count;           // [1] or null
    int32_t num_seqs, total_tokens, chunk, max_chunks;
};

// Gradients of the gated delta rule. Chunks have slots: chunk c of request n,
// which starts at row b, has slot b / kGradChunk + n + c.
constexpr int kGradChunk = 64;
struct DeltaGradProblem {
    Requests req;
    Pool pool;           // states before the forward pass, [num_slots, H, K, V]
    Pool grad;           // gradients of the states, in place (slot, init as in pool)
    const void *q, *k;   // [T, Hk, K]
    const void *v;       // [T, H, V]
    const void *dout;    // [T, H, V]
    const float *g;      // [T, H, K] or [T, H]
    const float *beta;   // [T, H]
    void *dq, *dk;       // [T, Hk, K]
    void *dv;            // [T, H, V]
    float *dg, *dbeta;   // [T, H, K] or [T, H]; [T, H]
    int32_t H, Hk, K, V;
    int32_t gate_stride;  // elements of g per (token, head): K or 1
    int32_t slots;        // chunk slots of the workspace
    float scale;
    float *work;          // [slots, H] chunks of grad_chunk_floats
    float *dq_head, *dk_head;  // [T, H, K] where key heads are shared, else null
};
inline int64_t grad_slots(int64_t total_tokens, int64_t num_seqs) {
    return total_tokens / kGradChunk + num_seqs;
}
// A and its inverse, three operands of C x K, two of C x V, two states, decays,
// beta, the chunk itself.
inline int64_t grad_chunk_floats(int32_t K, int32_t V) {
    return (int64_t)2 * kGradChunk * kGradChunk + 3 * kGradChunk * K + 2 * kGradChunk * V +
           2 * K * V + K + kGradChunk + 4;
}

struct CheckpointProblem {
    const void *x;   // [vecs, d] to be stored, or null: to be read back
    int8_t *codes;   // [vecs, d]
    float *scale;    // [vecs]
    void *out;       // [vecs, d], read back
    int64_t vecs;
    int32_t d;
};
struct NormCheckpointProblem {
    NormProblem norm;
    int8_t *o_codes, *z_codes;
    float *o_scale, *z_scale;
};
struct NormGradProblem {
    const void *dout, *o, *z;         // o, z: codes where o_scale is given
    const float *o_scale, *z_scale;   // [rows, H] or null
    const float *norm_w;
    void *d_o, *dz;
    float *dnorm_w;
    float *part;  // [blocks, d]
    int64_t vecs;
    int32_t d;
    float eps_norm;
};
// Workgroups of the norm's backward pass, each of which leaves a row of dnorm_w:
// enough for every compute unit, and few rows to add.
inline int64_t norm_grad_blocks(int64_t vecs, int32_t d) {
    const int64_t per = 256 / (d / 8), need = (vecs + per - 1) / per;
    return need < 2048 ? need : 2048;
}

struct ConvGradProblem {
    Requests req;
    Pool pool;            // windows before the forward pass, [num_slots, 3, H, W - 1, d]
    Pool grad;            // gradients of the windows, in place
    const void *dout[3];  // of q, k, v: [T, H, d]
    const void *qkv;      // [T, 3, H, d], or codes where qkv_scale is given
    const float *qkv_scale;  // [T, 3, H] or null
    const float *conv_w;  // [3, W, H, d]
    void *dqkv;           // [T, 3, H, d]
    float *dconv_w;       // [3, W, H, d]
    float *part;          // [rows, 3, W, H, d]
    float *old;           // [num_seqs, 3, H, W - 1, d]
    int32_t H, d, W;
    int32_t seg;          // tokens per wavefront
    float eps_l2;
};
// Workgroups of the launch that sums dconv_w and puts the gradients of `windows`
// requests' windows into the pool: kConvGradPart floats each, the taps' first.
constexpr int64_t kConvGradPart = 1024;
inline int64_t conv_grad_tap_blocks(int32_t H, int32_t d, int32_t W) {
    return ((int64_t)3 * W * H * d + kConvGradPart - 1) / kConvGradPart;
}
inline int64_t conv_grad_window_blocks(int32_t H, int32_t d, int32_t W) {  // of one request
    return ((int64_t)3 * (W - 1) * H * d + kConvGradPart - 1) / kConvGradPart;
}
// Rows of dconv_w that the workgroups (four segments each) leave.
inline int64_t conv_grad_rows(int64_t tokens, int32_t seg) {
    return (tokens + 4 * (int64_t)seg - 1) / (4 * (int64_t)seg);
}
// Tokens per wavefront: up to 64 (every segment takes W - 1 rows twice at both
// ends: 8,192 tokens of 64 heads, bf16 308 us with 16, 263 with 32, 248 with 64, 249
// with 128, 256 with 256; from 8-bit codes 311, 261, 242, 239, 236), fewer while a
// compute unit would have less than 12 wavefronts (2,048 tokens of 16 heads 24 us with
// the 16 of this rule, 27 with 32, 35 with 64; 512 tokens of 64 heads 23, 28 with 32).
// With rows of two and a half wavefronts a part of their lanes idles, and it divides
// too far: 7,000 tokens of 9 heads of 64, f32, 49 us with its 16, 42 with 32, 43 with
// 64. Past 32,768 tokens always 512 segments, so that the workspace stays as it is
// however long the call: 131,072 tokens of 4 heads 283 us with its 256 or with 64,
// 65,536 of 16 heads 536 with 128, 511 with 64, 65,536 of one head of 64 channels 79
// and 85, 40,000 of two 57 with 79, 50 with 64.
inline int32_t conv_grad_segment(int64_t tokens, int32_t H, int32_t d) {
    if (tokens > 32768) return (int32_t)((tokens + 511) / 512);
    const int64_t per_segment = ((int64_t)H * d + 255) / 256 * 3;
    int32_t seg = 64;
    while (seg > 4 && tokens / seg * per_segment < 12 * 256) seg /= 2;
    return seg;
}

hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_recurrent(const DeltaProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_conv(const ConvProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_norm(const NormProblem &p, int in_dt, int out_dt, hipStream_t stream);
hipError_t launch_delta_grad(const DeltaGradProblem &p, int in_dt, int dout_dt, hipStream_t stream);
hipError_t launch_conv_grad(const ConvGradProblem &p, int dt, hipStream_t stream);
hipError_t launch_norm_grad(const NormGradProblem &p, int dt, hipStream_t stream);
hipError_t launch_checkpoint(const CheckpointProblem &p, int dt, hipStream_t stream);
hipError_t launch_norm_checkpoint(const NormCheckpointProblem &p, int in_dt, int out_dt,
                                  hipStream_t stream);
hipError_t launch_map(const MapProblem &p, hipStream_t stream);

}  // namespace kda
