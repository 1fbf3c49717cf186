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

hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_recurrent(const DeltaProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_conv(const ConvProblem &p, int in_dt, hipStream_t stream);
hipError_t launch_norm(const NormProblem &p, int in_dt, int out_dt, hipStream_t stream);
hipError_t launch_map(const MapProblem &p, hipStream_t stream);

}  // namespace kda
