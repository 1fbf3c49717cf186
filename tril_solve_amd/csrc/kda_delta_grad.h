// Gradients of the gated delta rule over whole prompts, in chunks of 64
// tokens, for gfx950.
//
// Forward, S the K x V state before a chunk, G_i the decay summed from its
// first token through token i, G its whole decay, B = diag(beta):
//   A_ij = sum_d k_id k_jd e^{G_id - G_jd} (j < i),  P_ij likewise with q_i (j <= i)
//   X = (I + A B)^-1 (V - (k e^G) S),  U = B X,  O = scale ((q e^G) S + P U)
//   S <- e^G S + (k e^{G - G_i})^T U
// Backward, dS the gradient of the state behind the chunk, O' = scale dO:
//   dU = P^T O' + (k e^{G - G_i}) dS,   Y = (I + A B)^-T (B dU) = dV
//   dS <- (q e^G)^T O' + e^G dS - (k e^G)^T Y
//   E = strict(Y X^T),  dA = -E B,  dP = low(O' X^T) B,  dbeta = X.dU - sum_i A_ij E_ij
//   dq_i = e^{G_i} (O' S^T) + sum_j dP_ij k_j e^{G_i - G_j}
//   dk_i = -e^{G_i} (Y S^T) + e^{G - G_i} (U dS^T) + sum_j dA_ij k_j e^{G_i - G_j}
//          + sum_j (dA_ji k_j + dP_ji q_j) e^{G_j - G_i}
//   dg_t = what crosses the border in front of token t: the terms of q dq and
//          k dk of every pair i >= t > j, and those of both states.
//
// Three launches. Chunks are prepared side by side: A, its inverse, W =
// (I + A B)^-1 (k e^G), and X and dU without the states. Then the states walk
// forwards and their gradients backwards, both at once, each workgroup on its
// own value columns:
//   X -= W S,                    S <- e^G S + (k e^{G - G_i})^T B X
//   dU += (k e^{G - G_i}) dS,    dS <- e^G dS + (q e^G)^T O' - W^T B dU.
// Last, the chunks' gradients side by side, each wavefront on its own 16 key
// channels. States and their gradients lie in the workspace between launches, one
// for every 64 tokens: chunks of 32 would double that.
//
// Decays within a chunk never leave [0, 1]: a pair i > j meets at the level
// b = msb(i ^ j) (1, 2, ..., 32) with m the middle of the 2b tokens around both,
// e^{G_i - G_j} = e^{G_i - G_m} e^{G_m - G_j}, both sums of the token's own
// half. A level is a masked product of 16 x 16 (below 16) or of whole tiles, and
// any decay down to e^-inf goes through it exactly. dg is summed the same
// way, level by level, without differences.
//
// Products run on the FP32 matrix instructions, but for those of the chunks' last
// kernel over value columns, which take six bfloat16 products of three parts (see
// bf16_parts.h). FP32 outputs are 1e-7 to 4e-7 of their norm from 64 bits.
//
// What bounds it (16 x 512 tokens of 64 heads, K = V = 128, bf16: 3.02 ms, 0.69 +
// 1.18 + 1.28 in the three kernels under a trace; one sequence of 16,384 tokens and
// 32 heads 3.00 ms, 0.69 + 1.18 + 1.26): the traffic of the workspace (9.9 GB a call,
// 3.5, 3.3 and 2.8 TB/s of a tuned copy's 6.4) and the chains between barriers, which the
// few wavefronts that their registers and LDS leave room for do not cover (two to a
// SIMD). The matrix pipes are busy for 34, 52 and 26% of the cycles, the vector
// units for 34, 10 and 35%.
#pragma once

#include <hip/hip_runtime.h>

#include "bf16_parts.h"
#include "layer_device.h"
#include "tril_launch.h"

namespace kda {

constexpr int kGC = kGradChunk;
constexpr int kMatRow = kGC + 4;  // floats between rows of a 64 x 64 matrix in LDS
constexpr float kGradLog2E = 1.4426950408889634f;
constexpr float kLeastGate = -1024.0f;  // in powers of two; e^-inf and this are 0 alike

// Parts of one chunk-head's workspace.
template <int K>
struct GradWork {
    float *base;
    int V;
    // floats of one chunk and head
    static __device__ __forceinline__ long size(int V) {
        return 2L * kGC * kGC + 3L * kGC * K + 2L * kGC * V + 2L * K * V + K + kGC + 4;
    }
    __device__ __forceinline__ GradWork(float *work, int V, long item)
        : base(work + item * size(V)), V(V) {}
    __device__ __forceinline__ float *A() const { return base; }
    __device__ __forceinline__ float *M() const { return base + kGC * kGC; }       // (I + A B)^-1
    __device__ __forceinline__ float *W() const { return M() + kGC * kGC; }        // [C][K]
    __device__ __forceinline__ float *Kb() const { return W() + kGC * K; }         // k e^{G - G_i}
    __device__ __forceinline__ float *Qt() const { return Kb() + kGC * K; }        // q e^G
    __device__ __forceinline__ float *decay() const { return Qt() + kGC * K; }     // e^G, [K]
    __device__ __forceinline__ float *beta() const { return decay() + K; }         // [C]
    // the first row, the number of rows (0: no such chunk), whether it is padding
    __device__ __forceinline__ int32_t *chunk() const {
        return reinterpret_cast<int32_t *>(beta() + kGC);
    }
    __device__ __forceinline__ float *X() const { return beta() + kGC + 4; }       // [C][V]
    __device__ __forceinline__ float *U() const { return X() + kGC * V; }          // dU, [C][V]
    __device__ __forceinline__ float *S() const { return U() + kGC * V; }          // [K][V]
    __device__ __forceinline__ float *D() const { return S() + K * V; }            // dS, [K][V]
};

// The chunk of a slot: its request, first row and number of rows (0: none).
struct GradChunk {
    int request, row, len;
};
__device__ __forceinline__ int grad_first_row(const Requests &r, int n) {
    return r.cu ? min(max(r.cu[n], 0), r.total_tokens) : n * r.seq_len;
}
// The last request whose first slot is not behind `slot`: 64 spread requests
// are compared at a time (wave-uniform).
__device__ __forceinline__ GradChunk grad_chunk(const Requests &r, int slot, int lane) {
    int lo = 0, hi = r.num_seqs;
    while (lo < hi) {
        const int step = (hi - lo + kWave - 1) / kWave;
        const int i = lo + lane * step;
        const bool upto = i < hi && grad_first_row(r, i) / kGC + i <= slot;
        const int m = __popcll(__ballot(upto));
        if (m == 0) break;
        const int top = lo + m * step;
        lo = lo + (m - 1) * step + 1;
        hi = min(hi, top);
    }
    const int n = lo - 1;
    if (n < 0) return GradChunk{0, 0, 0};
    const int2 rows = request_rows(r, n);
    const int at = (slot - (rows.x / kGC + n));
    const long first = (long)at * kGC;
    if (at < 0 || first >= rows.y) return GradChunk{n, 0, 0};
    return GradChunk{__builtin_amdgcn_readfirstlane(n),
                     __builtin_amdgcn_readfirstlane(rows.x + (int)first),
                     __builtin_amdgcn_readfirstlane(min(kGC, rows.y - (int)first))};
}

// c + a b over 16 of the reduction: lane (x = lane & 15, g = lane >> 4) holds
// elements 4 g .. 4 g + 3 of row x of a and of column x of b; the accumulator
// holds rows 4 g .. 4 g + 3 of column x, so it is itself such an operand b.
__device__ __forceinline__ f4 mm16(f4 a, f4 b, f4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

template <class E>
__device__ __forceinline__ void grad_put(typename E::T *p, float x);
template <>
__device__ __forceinline__ void grad_put<F32>(float *p, float x) { *p = x; }
template <>
__device__ __forceinline__ void grad_put<BF16>(uint16_t *p, float x) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)x);
}
template <>
__device__ __forceinline__ void grad_put<F16>(uint16_t *p, float x) {
    *p = __builtin_bit_cast(uint16_t, (_Float16)x);
}
__device__ __forceinline__ const f4 &as4(const float *p) { return *reinterpret_cast<const f4 *>(p); }
__device__ __forceinline__ f4 &as4(float *p) { return *reinterpret_cast<f4 *>(p); }

// Descriptors: rows row .. row + len - 1 of head h in a tensor [T, heads, width],
// from the first one's element of that head on; n floats.
template <class E>
__device__ __forceinline__ Rsrc grad_rows(const void *base, long row, int h, int heads, int width,
                                          int len) {
    const typename E::T *at =
        static_cast<const typename E::T *>(base) + (row * heads + h) * (long)width;
    const uint32_t n = ((uint32_t)(len - 1) * heads * width + width) * E::kBytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<typename E::T *>(at), 0, n, kRsrcWord3);
}
__device__ __forceinline__ Rsrc grad_floats(float *base, int n) {
    return __builtin_amdgcn_make_buffer_rsrc(base, 0, 4 * n, kRsrcWord3);
}
// An element as loaded, and widened where it is used: a load in flight is not waited
// for before.
template <class E>
__device__ __forceinline__ uint32_t grad_raw1(Rsrc r, uint32_t off) {
    if constexpr (E::kBytes == 4)
        return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}
template <class E>
__device__ __forceinline__ float grad_widen(uint32_t raw) {
    if constexpr (E::kBytes == 4)
        return __builtin_bit_cast(float, raw);
    else
        return Elem<E>::widen(raw);
}
// Stores of 16 lanes fill a part of a line, which the next one completes: they
// go through L2 by its usual policy.
template <class E>
__device__ __forceinline__ void grad_store1(Rsrc r, uint32_t off, float v);
template <>
__device__ __forceinline__ void grad_store1<F32>(Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, 0);
}
template <>
__device__ __forceinline__ void grad_store1<BF16>(Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, off, 0, 0);
}
template <>
__device__ __forceinline__ void grad_store1<F16>(Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (_Float16)v), r, off, 0, 0);
}

template <class E>
__device__ __forceinline__ void grad_store4(Rsrc r, uint32_t off, f4 v) {
    if constexpr (E::kBytes == 4) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(w4, v), r, off, 0, 0);
    } else {
        const w2 o = {Elem<E>::pack(v[0], v[1]), Elem<E>::pack(v[2], v[3])};
        __builtin_amdgcn_raw_buffer_store_b64(o, r, off, 0, 0);
    }
}

// A gate in powers of two. NaN stays (a comparison with it is false).
__device__ __forceinline__ float grad_gate(float g) {
    const float x = g * kGradLog2E;
    return x < kLeastGate ? kLeastGate : x;
}

// One level of 16 tokens in lanes 0..15 of a row: the sums of aligned halves of
// b tokens are joined to 2b. pre: through the token from the half's start;
// suf: behind the token to the half's end; tot: of the half.
template <int CTRL>
__device__ __forceinline__ float grad_dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ void grad_join(float &pre, float &suf, float &tot, bool upper) {
    const float o = grad_dpp<CTRL>(tot);
    pre += upper ? o : 0.0f;
    suf += upper ? 0.0f : o;
    tot += o;
}

// Barrier of the workgroup that orders LDS alone: loads and stores of memory stay
// in flight.
__device__ __forceinline__ void grad_lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---------------------------------------------------------------- preparation

// A workgroup to a chunk and head. The levels are products of 64-token images in
// LDS (16 lanes: 16 tokens, their sums by DPP); the inverse is substitution within
// 16 x 16 and products above; all that the other kernels read is stored as they
// load it, rows of four floats to a lane. Pairs within four tokens are vector
// instructions (as masked products with the others 0.73 instead of 0.69 ms), the values
// are on their way while the inverse is made (0.77 ms without). Bound by what it
// stores and by the latency between its parts: 16 x 512 tokens of 64 heads take 0.69
// ms for 0.8 GB read and 1.6 written.
template <class E, class EO, int K>
__global__ __launch_bounds__(256, 2) void kda_grad_prepare_kernel(DeltaGradProblem p) {
    constexpr int NT = K / 16, KR = K + 4;
    // operands of one level, as the wavefronts hold them; afterwards the
    // matrices M, P, L and, in L's place, the decayed keys
    constexpr int kMat = kGC * kMatRow;
    constexpr int kImages = 6 * NT * 64 * 4, kMats = 2 * kMat + (kMat > kGC * KR ? kMat : kGC * KR);
    __shared__ __align__(16) float lds[kImages > kMats ? kImages : kMats];
    __shared__ __align__(16) float totals[4][K];
    __shared__ float bs[kGC];
    const int lane = threadIdx.x & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    const int h = (int)(blockIdx.x % p.H), slot = (int)(blockIdx.x / p.H);
    const GradChunk ch = grad_chunk(p.req, slot, lane);
    const GradWork<K> ws(p.work, p.V, (long)slot * p.H + h);
    const bool padding =
        ch.len > 0 && p.grad.slot != nullptr && request_slot(p.grad, ch.request) < 0;
    if (threadIdx.x == 0)
        *reinterpret_cast<int4 *>(ws.chunk()) = make_int4(ch.row, ch.len, padding, 0);
    if (ch.len == 0 || padding) return;
    const int V = p.V, tok = 16 * w + x;
    f4 k[NT], q[NT], pre[NT], suf[NT], tot[NT];
    {  // rows behind the last load 0
        const int hk = h / (p.H / p.Hk);
        const Rsrc rk = grad_rows<E>(p.k, ch.row, hk, p.Hk, K, ch.len);
        const Rsrc rq = grad_rows<E>(p.q, ch.row, hk, p.Hk, K, ch.len);
        const Rsrc rg = grad_rows<F32>(p.g, ch.row, h, p.H, p.gate_stride, ch.len);
        const uint32_t at = (uint32_t)(tok * p.Hk * K + 4 * gq) * E::kBytes;
        const uint32_t gat = (uint32_t)tok * p.H * p.gate_stride * 4;
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            k[T] = load4<E>(rk, at + 16 * T * E::kBytes);
            q[T] = load4<E>(rq, at + 16 * T * E::kBytes);
        }
        if (p.gate_stride == K) {
#pragma unroll
            for (int T = 0; T < NT; ++T) tot[T] = load4<F32>(rg, gat + 16 * gq + 64 * T);
        } else {
            const float one = load1<F32>(rg, gat);
#pragma unroll
            for (int T = 0; T < NT; ++T) tot[T] = f4{one, one, one, one};
        }
#pragma unroll
        for (int T = 0; T < NT; ++T) {
#pragma unroll
            for (int s = 0; s < 4; ++s) tot[T][s] = grad_gate(tot[T][s]);
            pre[T] = tot[T];
            suf[T] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // diagonal tiles: the levels below 16, within the wavefront
    f4 dA = {0.0f, 0.0f, 0.0f, 0.0f}, dP = dA;
    float pd = 0.0f;
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) pd = __builtin_fmaf(q[T][s], k[T][s], pd);
    pd = add_rows32(add_rows16(pd));
    auto factor = [&](int T, bool rows) {
        return exp2(rows ? pre[T] : suf[T]);
    };
    auto diagonal = [&](int b) {
        f4 lA = {0.0f, 0.0f, 0.0f, 0.0f}, lP = lA;
        const bool rows = (x & b) != 0;
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            const f4 f = factor(T, rows), kf = k[T] * f, qf = q[T] * f;
            lA = mm16(kf, kf, lA);
            lP = mm16(qf, kf, lP);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int i = 4 * gq + s, d = i ^ x;
            if ((i & b) && d >= b && d < 2 * b) {
                dA[s] = lA[s];
                dP[s] = lP[s];
            }
        }
    };
    // pairs within four tokens: y holds the key of 1, 2, 3 tokens before, decayed to
    // this one; lanes whose pair crosses the four do not count
    {
        float sA[3] = {0.0f, 0.0f, 0.0f}, sP[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            const f4 e = exp2(tot[T]);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float y = k[T][s];
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                    y = e[s] * grad_dpp<0x111>(y);  // row_shr:1
                    sA[d] = __builtin_fmaf(k[T][s], y, sA[d]);
                    sP[d] = __builtin_fmaf(q[T][s], y, sP[d]);
                }
            }
        }
        auto put4 = [&](f4 &to, const float (&sum)[3]) {
            float v[3];
#pragma unroll
            for (int d = 0; d < 3; ++d) v[d] = add_rows32(add_rows16(sum[d]));
            const float a1 = grad_dpp<0x55>(v[0]), a2 = grad_dpp<0xAA>(v[0]),
                        b2 = grad_dpp<0xAA>(v[1]), a3 = grad_dpp<0xFF>(v[0]),
                        b3 = grad_dpp<0xFF>(v[1]), c3 = grad_dpp<0xFF>(v[2]);
            const int at = gq == x >> 2 ? x & 3 : 4;
            to[1] = at == 0 ? a1 : to[1];
            to[2] = at == 1 ? a2 : at == 0 ? b2 : to[2];
            to[3] = at == 2 ? a3 : at == 1 ? b3 : at == 0 ? c3 : to[3];
        };
        put4(dA, sA);
        put4(dP, sP);
    }
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float a = pre[T][s], c = suf[T][s], t = tot[T][s];
            grad_join<0xB1>(a, c, t, x & 1);
            pre[T][s] = a, suf[T][s] = c, tot[T][s] = t;
        }
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float a = pre[T][s], c = suf[T][s], t = tot[T][s];
            grad_join<0x4E>(a, c, t, x & 2);
            pre[T][s] = a, suf[T][s] = c, tot[T][s] = t;
        }
    diagonal(4);
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float a = pre[T][s], c = suf[T][s], t = tot[T][s];
            grad_join<0x141>(a, c, t, x & 4);
            pre[T][s] = a, suf[T][s] = c, tot[T][s] = t;
        }
    diagonal(8);
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float a = pre[T][s], c = suf[T][s], t = tot[T][s];
            grad_join<0x140>(a, c, t, x & 8);
            pre[T][s] = a, suf[T][s] = c, tot[T][s] = t;
        }
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (4 * gq + s == x) dP[s] = pd;

    // levels 16 and 32: tiles of two wavefronts, whose operands pass through LDS
    float *imK = lds, *imQ = lds + 4 * NT * 256;  // [4][NT][64] f4, [2][NT][64] f4
    auto image = [&](float *im, int slot_, int T) -> f4 & {
        return as4(im + ((slot_ * NT + T) * 64 + lane) * 4);
    };
    if (threadIdx.x < kGC) {
        const Rsrc rb = grad_rows<F32>(p.beta, ch.row, h, p.H, 1, ch.len);
        const float one = load1<F32>(rb, threadIdx.x * p.H * 4);
        bs[threadIdx.x] = one;
        ws.beta()[threadIdx.x] = one;
    }
    if (x == 0)
#pragma unroll
        for (int T = 0; T < NT; ++T) as4(&totals[w][16 * T + 4 * gq]) = tot[T];
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        const f4 f = factor(T, w & 1);
        image(imK, w, T) = k[T] * f;
        if (w & 1) image(imQ, w >> 1, T) = q[T] * f;
    }
    grad_lds_barrier();
    f4 o16 = {0.0f, 0.0f, 0.0f, 0.0f}, oA = o16, oP = o16;
    {  // wavefronts 0, 1: A and P of tile (1, 0); 2, 3: of tile (3, 2)
        const int pair = w >> 1;
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            const f4 a = (w & 1) ? image(imQ, pair, T) : image(imK, 2 * pair + 1, T);
            o16 = mm16(a, image(imK, 2 * pair, T), o16);
        }
    }
    grad_lds_barrier();
    // 1 for wavefronts from 1, 2, 3 on and up to 0, 1, 2 (branches on them would cut
    // the code into pieces)
    const float u1 = w >= 1, u2 = w >= 2, u3 = w >= 3, d0 = w < 1, d1 = w < 2, d2 = w < 3;
    const float a32 = w == 0, b32 = w == 3;
    f4 kg[NT];  // k e^G
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        f4 t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = as4(&totals[j][16 * T + 4 * gq]);
        const f4 half = exp2((w >= 2 ? pre[T] : suf[T]) + (a32 * t[1] + b32 * t[2]));
        image(imK, w, T) = k[T] * half;
        if (w >= 2) image(imQ, w - 2, T) = q[T] * half;
        const f4 before = u1 * t[0] + u2 * t[1] + u3 * t[2];
        const f4 behind = d2 * t[3] + d1 * t[2] + d0 * t[1];
        // operands of the walks, by tokens: k e^{G - G_i}, q e^G
        const f4 eg = exp2(pre[T] + before), kb = k[T] * exp2(suf[T] + behind), qg = q[T] * eg;
        kg[T] = k[T] * eg;
        as4(ws.Kb() + tok * K + 16 * T + 4 * gq) = kb;
        as4(ws.Qt() + tok * K + 16 * T + 4 * gq) = qg;
        if (w == 0 && x == 0) as4(ws.decay() + 16 * T + 4 * gq) = exp2(t[0] + t[1] + t[2] + t[3]);
    }
    grad_lds_barrier();
    const int ti = 2 + (w >> 1), tj = w & 1;  // this wavefront's tile of level 32
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        const f4 b = image(imK, tj, T);
        oA = mm16(image(imK, ti, T), b, oA);
        oP = mm16(image(imQ, ti - 2, T), b, oP);
    }

    grad_lds_barrier();  // the images are read

    // the values' first columns, on their way until the inverse is there
    const Rsrc rv = grad_rows<E>(p.v, ch.row, h, p.H, V, ch.len);
    const Rsrc ro = grad_rows<EO>(p.dout, ch.row, h, p.H, V, ch.len);
    const uint32_t vstep = (uint32_t)p.H * V;
    uint32_t vraw[4][4], oraw[4][4];
    auto load_values = [&](int n) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t at =
                    n < V / 16 ? (16 * t + 4 * gq + s) * vstep + 16 * n + x : kOffMasked / 4;
                vraw[t][s] = grad_raw1<E>(rv, at * E::kBytes);
                oraw[t][s] = grad_raw1<EO>(ro, at * EO::kBytes);
            }
    };
    load_values(w);

    // the matrices: A to memory, L = A B and P to LDS
    float *Mm = lds, *Pm = lds + kMat, *Lm = lds + 2 * kMat;
    auto put = [&](int bi, int bj, f4 a, bool isA, bool isP) {
        const int col = 16 * bj + x;
        const float beta = bs[col];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * bi + 4 * gq + s;
            if (isA) {
                ws.A()[r * kGC + col] = a[s];
                Lm[r * kMatRow + col] = a[s] * beta;
            }
            if (isP) Pm[r * kMatRow + col] = a[s];
        }
    };
    put(w, w, dA, true, false);
    put(w, w, dP, false, true);
    put(2 * (w >> 1) + 1, 2 * (w >> 1), o16, !(w & 1), w & 1);
    put(ti, tj, oA, true, false);
    put(ti, tj, oP, false, true);
    grad_lds_barrier();

    // M = (I + L)^-1: diagonal blocks by substitution, then merged twice
    {
        float a[16], m[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f4 l = as4(&Lm[(16 * w + x) * kMatRow + 16 * w + 4 * c]);
#pragma unroll
            for (int s = 0; s < 4; ++s) a[4 * c + s] = -l[s];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) m[r] = r == x ? 1.0f : 0.0f;
        substitute(a, m);
        if (gq == 0)
#pragma unroll
            for (int r = 0; r < 16; ++r) Mm[(16 * w + r) * kMatRow + 16 * w + x] = m[r];
    }
    grad_lds_barrier();
    auto left = [&](const float *mat, int bi, int bj) {  // operand a: rows of a tile
        return as4(mat + (16 * bi + x) * kMatRow + 16 * bj + 4 * gq);
    };
    auto right = [&](const float *mat, int bi, int bj) {  // operand b: columns of a tile
        f4 v;
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = mat[(16 * bi + 4 * gq + s) * kMatRow + 16 * bj + x];
        return v;
    };
    auto keep = [&](int bi, int bj, f4 v) {
#pragma unroll
        for (int s = 0; s < 4; ++s) Mm[(16 * bi + 4 * gq + s) * kMatRow + 16 * bj + x] = v[s];
    };
    const f4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    if (w < 2) {
        const int a = 2 * w + 1, b = 2 * w;
        const f4 t = mm16(left(Lm, a, b), right(Mm, b, b), zero4);
        keep(a, b, -mm16(left(Mm, a, a), t, zero4));
    }
    grad_lds_barrier();
    if (w < 2) {
        f4 t2 = zero4, t3 = zero4;
        for (int c = w; c < 2; ++c) {
            const f4 m = right(Mm, c, w);
            t2 = mm16(left(Lm, 2, c), m, t2);
            t3 = mm16(left(Lm, 3, c), m, t3);
        }
        keep(2, w, -mm16(left(Mm, 2, 2), t2, zero4));
        keep(3, w, -mm16(left(Mm, 3, 3), t3, mm16(left(Mm, 3, 2), t2, zero4)));
    }
    grad_lds_barrier();

    // k e^G by tokens, in L's place; M to memory
    float *Kg = Lm;
#pragma unroll
    for (int T = 0; T < NT; ++T) as4(&Kg[tok * KR + 16 * T + 4 * gq]) = kg[T];
    for (int e = threadIdx.x; e < kGC * kGC / 4; e += 256) {
        const int r = e / (kGC / 4), c = e % (kGC / 4) * 4;
        if (c / 16 <= r / 16) as4(ws.M() + r * kGC + c) = as4(&Mm[r * kMatRow + c]);
    }
    grad_lds_barrier();

    // W = M (k e^G); the transposed accumulators hold four adjacent channels of a row
    for (int n = w; n < NT; n += 4) {
        f4 b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) b[t][s] = Kg[(16 * t + 4 * gq + s) * KR + 16 * n + x];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 acc = zero4;
#pragma unroll
            for (int t = 0; t <= i; ++t) acc = mm16(b[t], left(Mm, i, t), acc);
            as4(ws.W() + (16 * i + x) * K + 16 * n + 4 * gq) = acc;
        }
    }
    // X = M V, dU = P^T O', still without the states
    for (int n = w; n < V / 16; n += 4) {
        f4 b[4], o[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                b[t][s] = grad_widen<E>(vraw[t][s]);
                o[t][s] = grad_widen<EO>(oraw[t][s]) * p.scale;
            }
        load_values(n + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 acc = zero4, up = zero4;
#pragma unroll
            for (int t = 0; t <= i; ++t) acc = mm16(b[t], left(Mm, i, t), acc);
#pragma unroll
            for (int t = i; t < 4; ++t) {  // column i of P's tiles, read across
                f4 a;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    a[s] = Pm[(16 * t + 4 * gq + s) * kMatRow + 16 * i + x];
                up = mm16(o[t], a, up);
            }
            const int at = (16 * i + x) * V + 16 * n + 4 * gq;
            as4(ws.X() + at) = acc;
            as4(ws.U() + at) = up;
        }
    }
}

// -------------------------------------------------------------------- the walks

// A workgroup's columns of a request and head: CT tiles of 16. Each of its four
// wavefronts owns a quarter of the state's channels and adds its part of W S (or
// of (k e^{G - G_i}) dS); wavefront i joins the parts of tile row i in LDS and
// makes X (or dU) of it, and every wavefront updates its channels with the whole
// U. So one step of the chain is a quarter of the products, two exchanges in LDS
// and another quarter, and the operands of the next chunk are on their way
// meanwhile, a tile row behind the products that read it: all of them at once hold the
// wavefront up (one sequence of 16,384 tokens and 32 heads 1.45 ms, 1.18 so; loads
// spread evenly between the products, or the states' stores among them, 1.18 to
// 1.28). One wavefront with all channels made that call 15.4 ms instead of 5.3. Six
// bfloat16 products, 0.75 of the matrix time of FP32's, lost: the splits are vector
// instructions in the chain (1.92 ms then, for 1.48).
// Bound by the chain with one sequence (256 steps of 4.6 us, 2.9 of them products of the
// longer way), by the states' traffic with many (16 x 512 tokens: 3.9 GB in 1.18 ms;
// the products alone take 0.76).
template <int CT>
struct GradWalkLds {
    float part[4][4 * CT][kWave * 4];  // [wavefront][tile row, column tile]
    float u[4 * CT][kWave * 4], o[4 * CT][kWave * 4];
    // a wavefront's state by rows, on its way to memory in whole lines
    float rows[4][32][16 * CT + 4];
};
template <class EO, int K, int CT, bool BACK>
__device__ __forceinline__ void grad_walk(const DeltaGradProblem &p, int n, int h, int part,
                                          GradWalkLds<CT> &lds) {
    constexpr int NT = K / 64;  // tiles of 16 channels to a wavefront
    const int lane = threadIdx.x & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    // (copies: captured by reference, the arguments would be read from scratch)
    float *const work = p.work;
    const void *const dout = p.dout;
    const float scale = p.scale;
    const int V = p.V, H = p.H, col = part * 16 * CT + x, c0 = 16 * NT * w;
    int2 rows = request_rows(p.req, n);
    rows.x = __builtin_amdgcn_readfirstlane(rows.x);  // (descriptors are made of them)
    rows.y = __builtin_amdgcn_readfirstlane(rows.y);
    const Pool pool = BACK ? p.grad : p.pool;
    const int at = __builtin_amdgcn_readfirstlane(
        p.grad.slot != nullptr || pool.base != nullptr ? request_slot(pool, n) : 0);
    if (at < 0) return;  // padding
    const int chunks = (rows.y + kGC - 1) / kGC, slot0 = rows.x / kGC + n;
    const bool from_pool = pool.base != nullptr && (BACK || request_continues(pool, n));
    float *state = pool.base + ((long)at * p.H + h) * K * V;
    const f4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    f4 S[NT][CT];
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                S[T][c][s] =
                    from_pool ? state[(c0 + 16 * T + 4 * gq + s) * V + col + 16 * c] : 0.0f;

    f4 lhs[4][NT], rhs[NT][4], qt[NT][4], x0[CT], beta, decay[NT];
    uint32_t o[CT][4];
    // Operands are loaded tile row by tile row, each right behind the products that
    // read its predecessor: 32 loads at once would hold the wavefront up.
    auto load_first = [&](const GradWork<K> &ws, int i) {  // for W S or (k e^{G - G_i}) dS
        const Rsrc r = grad_floats(BACK ? ws.Kb() : ws.W(), kGC * K);
#pragma unroll
        for (int T = 0; T < NT; ++T)
            lhs[i][T] = load4<F32>(r, 4 * ((16 * i + x) * K + c0 + 16 * T + 4 * gq));
    };
    auto load_join = [&](const GradWork<K> &ws) {
        const Rsrc r = grad_floats(BACK ? ws.U() : ws.X(), kGC * V);
        beta = load4<F32>(grad_floats(ws.beta(), kGC), 4 * (16 * w + 4 * gq));
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                x0[c][s] = load1<F32>(r, 4 * ((16 * w + 4 * gq + s) * V + col + 16 * c));
    };
    auto load_dout = [&](int j) {
        if constexpr (BACK) {
            const Rsrc ro = grad_rows<EO>(dout, rows.x + j * kGC, h, H, V,
                                          min(kGC, rows.y - j * kGC));
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    o[c][s] = grad_raw1<EO>(ro, ((uint32_t)(16 * w + 4 * gq + s) * H * V + col +
                                                 16 * c) * EO::kBytes);
        }
    };
    auto load_decay = [&](const GradWork<K> &ws) {
        const Rsrc rd = grad_floats(ws.decay(), K);
#pragma unroll
        for (int T = 0; T < NT; ++T) decay[T] = load4<F32>(rd, 4 * (c0 + 16 * T + 4 * gq));
    };
    auto load_rows = [&](float *rows, f4 (&to)[NT][4], int t) {  // as a left operand, across
        const Rsrc r = grad_floats(rows, kGC * K);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int T = 0; T < NT; ++T)
                to[T][t][s] = load1<F32>(r, 4 * ((16 * t + 4 * gq + s) * K + c0 + 16 * T + x));
    };
    auto load_middle = [&](const GradWork<K> &ws, int t) {
        if constexpr (BACK) load_rows(ws.Qt(), qt, t);
    };
    auto load_last = [&](const GradWork<K> &ws, int t) {
        load_rows(BACK ? ws.W() : ws.Kb(), rhs, t);
    };
    auto chunk_of = [&](int j) { return BACK ? chunks - 1 - j : j; };
    if (chunks > 0) {
        const GradWork<K> ws(work, V, (long)(slot0 + chunk_of(0)) * H + h);
        load_dout(chunk_of(0));
#pragma unroll
        for (int i = 0; i < 4; ++i) load_first(ws, i);
        load_join(ws);
        load_decay(ws);
#pragma unroll
        for (int t = 0; t < 4; ++t) load_middle(ws, t);
#pragma unroll
        for (int t = 0; t < 4; ++t) load_last(ws, t);
    }
    for (int j = 0; j < chunks; ++j) {
        const GradWork<K> ws(work, V, (long)(slot0 + chunk_of(j)) * H + h);
        const int jn = chunk_of(min(j + 1, chunks - 1));
        const GradWork<K> next(work, V, (long)(slot0 + jn) * H + h);
        if constexpr (BACK)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                f4 v;
#pragma unroll
                for (int s = 0; s < 4; ++s) v[s] = scale * grad_widen<EO>(o[c][s]);
                as4(&lds.o[w * CT + c][lane * 4]) = v;
            }
        load_dout(jn);
        f4 acc[4][CT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                acc[i][c] = zero4;
#pragma unroll
                for (int T = 0; T < NT; ++T) acc[i][c] = mm16(lhs[i][T], S[T][c], acc[i][c]);
            }
            load_first(next, i);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < CT; ++c) as4(&lds.part[w][i * CT + c][lane * 4]) = acc[i][c];
        {
            const Rsrc r = grad_floats(BACK ? ws.D() : ws.S(), K * V);
#pragma unroll
            for (int T = 0; T < NT; ++T)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        lds.rows[w][16 * T + 4 * gq + s][16 * c + x] = S[T][c][s];
            constexpr int kLanes = 4 * CT;  // to a row
#pragma unroll
            for (int e = 0; e < NT * CT; ++e) {
                const int row = (e * kWave + lane) / kLanes, at = lane % kLanes * 4;
                const f4 v = as4(&lds.rows[w][row][at]);
                grad_store4<F32>(r, 4 * ((c0 + row) * V + part * 16 * CT + at), v);
            }
        }
        grad_lds_barrier();
        {
            const Rsrc r = grad_floats(BACK ? ws.U() : ws.X(), kGC * V);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int e = w * CT + c;
                const f4 sum =
                    (as4(&lds.part[0][e][lane * 4]) + as4(&lds.part[1][e][lane * 4])) +
                    (as4(&lds.part[2][e][lane * 4]) + as4(&lds.part[3][e][lane * 4]));
                const f4 y = BACK ? x0[c] + sum : x0[c] - sum;
                as4(&lds.u[e][lane * 4]) = (BACK ? -beta : beta) * y;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    grad_store1<F32>(r, 4 * ((16 * w + 4 * gq + s) * V + col + 16 * c), y[s]);
            }
        }
        load_join(next);
#pragma unroll
        for (int T = 0; T < NT; ++T)
#pragma unroll
            for (int c = 0; c < CT; ++c) S[T][c] *= decay[T];
        load_decay(next);
        // S += tile column t of the operand, times tile row t of u
        auto add = [&](const f4 (&to)[NT][4], const float (*u)[kWave * 4], int t) {
            f4 b[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) b[c] = as4(&u[t * CT + c][lane * 4]);
#pragma unroll
            for (int T = 0; T < NT; ++T)
#pragma unroll
                for (int c = 0; c < CT; ++c) S[T][c] = mm16(to[T][t], b[c], S[T][c]);
        };
        if constexpr (BACK)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                add(qt, lds.o, t);
                load_middle(next, t);
                __builtin_amdgcn_sched_barrier(0);
            }
        grad_lds_barrier();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            add(rhs, lds.u, t);
            load_last(next, t);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (BACK && pool.base != nullptr) {
        const bool cont = request_continues(pool, n);
#pragma unroll
        for (int T = 0; T < NT; ++T)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    state[(c0 + 16 * T + 4 * gq + s) * V + col + 16 * c] =
                        cont ? S[T][c][s] : 0.0f;
    }
}

// blockIdx.y: 0 the states forwards, 1 their gradients backwards. The workgroups
// of a request and head (`parts`) read the same operands: their numbers are 8
// apart, which puts them on one XCD and its L2.
template <class EO, int K, int CT>
__global__ __launch_bounds__(256, 2) void kda_grad_walk_kernel(DeltaGradProblem p, int parts) {
    __shared__ __align__(16) GradWalkLds<CT> lds;
    const int group = blockIdx.x / (8u * parts), in = blockIdx.x % (8u * parts);
    const int walk = group * 8 + in % 8;
    if (walk >= p.req.num_seqs * p.H) return;
    const int part = in / 8, h = __builtin_amdgcn_readfirstlane(walk % p.H);
    const int n = __builtin_amdgcn_readfirstlane(walk / p.H);
    if (blockIdx.y == 0)
        grad_walk<EO, K, CT, false>(p, n, h, part, lds);
    else
        grad_walk<EO, K, CT, true>(p, n, h, part, lds);
}

// ------------------------------------------------------------ gradients of a chunk

// LDS of the last kernel (bytes): parts of Y and X of up to VB value columns (rows
// 16 bytes apart in their banks), dout if it is kept (bfloat16, one part), the
// inverse and then dA in its place, dP in X's place, and per token beta, X.dU, the
// column sums of A * E by tile rows and, with one gate per head, dg by wavefronts.
template <int K, int VB, bool DOUT>
struct GradLds {
    static constexpr int RS = 2 * VB + 16, PART = kGC * RS, kMat = kGC * kMatRow * 4;
    static constexpr int Y = 0, X = Y + kParts * PART, O = X + kParts * PART;
    static constexpr int A = O + (DOUT ? PART : 0), P = X, BETA = A + kMat;
    static constexpr int XDU = BETA + kGC * 4, COLS = XDU + kGC * 4, DG = COLS + 4 * kGC * 4;
    static constexpr int kBytes = DG + K / 16 * kGC * 4;
    static_assert(kMat <= kParts * PART && kBytes <= (VB == 64 ? 80 : 160) * 1024);
};
// Eight adjacent elements of dout as an operand (bfloat16: all in its first part).
template <class EO>
__device__ __forceinline__ Operand grad_operand(Rsrc r, uint32_t off) {
    const f4 a = load4<EO>(r, off), b = load4<EO>(r, off + 4 * EO::kBytes);
    return join(split4(a), split4(b));
}

// A wavefront to every 16 key channels, one workgroup to a compute unit (160 KB of
// LDS): Y, X and dout are there for all of them, and S and dS are read once. FP32
// products over the value columns instead of six bfloat16 ones made a call of 16 x
// 512 tokens of 64 heads 3.6 ms instead of 3.3. Levels 1 and 2, pairs within a
// lane's four tokens, are vector instructions (1.39 -> 1.31 ms for this kernel with
// the operands of E taken as they lie); from 4 on a level is one product of
// masked tiles. ONE: all value columns at once (up to 128; with a loop over them the
// sums take registers from what is loaded ahead). With K = 64 and up to 64 columns
// two workgroups of four wavefronts share a unit (8,161 tokens of 8 heads, f32: 124 -> 88
// us). Two wavefronts to a SIMD leave 256 registers, which are not quite enough: 24 bytes
// a lane go through scratch with K = 128, 76 to 92 with a loop over the columns, 8 with
// K = 64 and up to 64 columns; K = 64 with more has one wavefront to a SIMD, and none.
template <class E, class EO, int K, int VB, bool ONE>
__global__ __launch_bounds__(K * 4, K == 128 || VB == 64 ? 2 : 1) void kda_grad_chunk_kernel(
    DeltaGradProblem p) {
    constexpr int NW = K / 16;
    // dout is one bfloat16 part (which two workgroups' LDS does not hold)
    constexpr bool kExact = VB == 128 && EO::kBytes == 2 && !__is_same(EO, F16);
    typedef GradLds<K, VB, kExact> L;
    __shared__ __align__(16) char lds[L::kBytes];
    const int lane = threadIdx.x & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    const int h = (int)(blockIdx.x % p.H), slot = (int)(blockIdx.x / p.H);
    const GradWork<K> ws(p.work, p.V, (long)slot * p.H + h);
    float *Am = reinterpret_cast<float *>(lds + L::A), *Pm = reinterpret_cast<float *>(lds + L::P);
    float *bs = reinterpret_cast<float *>(lds + L::BETA);
    float *xdu = reinterpret_cast<float *>(lds + L::XDU);
    float *cols = reinterpret_cast<float *>(lds + L::COLS);
    float *dgs = reinterpret_cast<float *>(lds + L::DG);
    const f4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    const int V = p.V, hk = h / (p.H / p.Hk);
    const int c = 16 * w + x;  // this lane's key channel
    // what does not depend on the chunk is loaded before it is known (of slots
    // without a chunk, whatever lies there)
    const Rsrc rX = grad_floats(ws.X(), kGC * V), rU = grad_floats(ws.U(), kGC * V);
    const Rsrc rS = grad_floats(ws.S(), 2 * K * V);  // and dS behind it
    const Rsrc rM = grad_floats(ws.M(), kGC * kGC);
    // this wavefront's rows of S and dS, 32 columns to a step
    f4 s4[VB / 32][2], d4[VB / 32][2];
    auto load_rows = [&](f4 (&to)[VB / 32][2], int row, int vb) {
#pragma unroll
        for (int t = 0; t < VB / 32; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = vb + 32 * t + 8 * gq + 4 * e;
                to[t][e] = load4<F32>(rS, vb + 32 * t < V ? 4 * (row * V + v) : kOffMasked);
            }
    };
    // this thread's part of X and dU for LDS, and this wavefront's columns of dU
    constexpr int NS = VB / (4 * NW);
    f4 xs[NS], us[NS], ub[4];
    auto load_columns = [&](int vb) {
#pragma unroll
        for (int e = 0; e < NS; ++e) {
            const int col = vb + 4 * (threadIdx.x % NW) + 4 * NW * e;
            const uint32_t at = col < V ? 4 * (threadIdx.x / NW * V + col) : kOffMasked;
            xs[e] = load4<F32>(rX, at);
            us[e] = load4<F32>(rU, at);
        }
    };
    auto load_tile = [&](int vb, int n) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int col = vb + 16 * n + x;
                ub[t][s] = load1<F32>(
                    rU, col < V ? 4 * ((16 * t + 4 * gq + s) * V + col) : kOffMasked);
            }
    };
    const int4 where = *reinterpret_cast<const int4 *>(ws.chunk());
    if constexpr (ONE) load_columns(0);
    f4 minv[1024 / (K * 4)];
#pragma unroll
    for (int e = 0; e < 1024 / (K * 4); ++e)
        minv[e] = load4<F32>(rM, 16 * (threadIdx.x + e * K * 4));
    const float my_beta =
        threadIdx.x < kGC ? load1<F32>(grad_floats(ws.beta(), kGC), 4 * threadIdx.x) : 0.0f;
    if constexpr (ONE) {
        load_tile(0, w);
        load_rows(s4, c, 0);
    }
    const int len = __builtin_amdgcn_readfirstlane(where.y);
    if (len == 0) return;
    struct {
        int row;
    } ch = {__builtin_amdgcn_readfirstlane(where.x)};
    typedef typename E::T T_;
    if (__builtin_amdgcn_readfirstlane(where.z)) {  // padding: zeros
        for (int r = w; r < len; r += NW) {
            const long row = ch.row + r, at = row * p.H + h;
            for (int c = lane; c < V; c += kWave)
                grad_put<E>(static_cast<T_ *>(p.dv) + at * V + c, 0.0f);
            for (int c = lane; c < K; c += kWave) {
                if (p.dq_head) {
                    p.dq_head[at * K + c] = 0.0f;
                    p.dk_head[at * K + c] = 0.0f;
                } else {
                    grad_put<E>(static_cast<T_ *>(p.dq) + (row * p.Hk + hk) * K + c, 0.0f);
                    grad_put<E>(static_cast<T_ *>(p.dk) + (row * p.Hk + hk) * K + c, 0.0f);
                }
                if (c < p.gate_stride) p.dg[at * p.gate_stride + c] = 0.0f;
            }
            if (lane == 0) p.dbeta[at] = 0.0f;
        }
        return;
    }
    // rows of this chunk and head; loads behind the last give 0, stores are dropped
    const Rsrc rdout = grad_rows<EO>(p.dout, ch.row, h, p.H, V, len);
    const Rsrc rdv = grad_rows<E>(p.dv, ch.row, h, p.H, V, len);
    const uint32_t dstep = (uint32_t)p.H * V * EO::kBytes;  // bytes between rows of dout
    const uint32_t vstep = (uint32_t)p.H * V * E::kBytes;
#pragma unroll
    for (int e = 0; e < 1024 / (K * 4); ++e) {  // (its upper tiles are not read)
        const int at = threadIdx.x + e * K * 4;
        as4(&Am[at / 16 * kMatRow + at % 16 * 4]) = minv[e];
    }
    if (threadIdx.x < kGC) bs[threadIdx.x] = my_beta;

    // O' S^T, Y S^T, X dS^T, the rows of S * dS, and tile rows of Y X^T and O' X^T:
    // row w & 3 of one of them, or, with four wavefronts, row w of both
    constexpr int NJ = 8 / NW;
    f4 dq[4], dk[4], ke[4], ex[NJ][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        dq[i] = dk[i] = ke[i] = zero4;
#pragma unroll
        for (int j = 0; j < NJ; ++j) ex[j][i] = zero4;
    }
    float both = 0.0f;
    const int tr = w & 3;
#pragma unroll 1
    for (int vb = 0; vb < (ONE ? 1 : V); vb += VB) {
        const int nv = min(VB, V - vb);
        if constexpr (!ONE) {
            if (vb > 0) __syncthreads();
            load_columns(vb);
            load_tile(vb, w);
            load_rows(s4, c, vb);
        }
        {  // X and dout to LDS; X.dU, NW lanes to a row
            const int r = threadIdx.x / NW, c0 = 4 * (threadIdx.x % NW);
            w2 os[NS];
            if constexpr (kExact)
#pragma unroll
                for (int e = 0; e < NS; ++e)
                    os[e] = __builtin_bit_cast(
                        w2, __builtin_amdgcn_raw_buffer_load_b64(
                                rdout, r * dstep + 2 * (vb + c0 + 4 * NW * e), 0, 0));
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < NS; ++e) {
#pragma unroll
                for (int s = 0; s < 4; ++s) sum = __builtin_fmaf(xs[e][s], us[e][s], sum);
                const Half parts = split4(xs[e]);
                char *at = lds + L::X + r * L::RS + 2 * (c0 + 4 * NW * e);
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    *reinterpret_cast<w2 *>(at + i * L::PART) = parts.p[i];
            }
            sum = lane_add<0x4E>(lane_add<0xB1>(sum));
            if (NW == 8) sum = lane_add<0x141>(sum);
            if (threadIdx.x % NW == 0) xdu[r] = vb > 0 ? xdu[r] + sum : sum;
            if constexpr (kExact)
#pragma unroll
                for (int e = 0; e < NS; ++e)
                    *reinterpret_cast<w2 *>(lds + L::O + r * L::RS + 2 * (c0 + 4 * NW * e)) = os[e];
        }
        if (vb == 0) __syncthreads();  // the inverse and beta
        // Y = M^T (B dU), its transpose in the accumulators: columns of four
        auto gradients_of_v = [&](int n) {
            f4 b[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) b[t] = as4(&bs[16 * t + 4 * gq]) * ub[t];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f4 acc = zero4;
#pragma unroll
                for (int t = i; t < 4; ++t) {
                    f4 a;
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        a[s] = Am[(16 * t + 4 * gq + s) * kMatRow + 16 * i + x];
                    acc = mm16(b[t], a, acc);
                }
                const int r = 16 * i + x, col = 16 * n + 4 * gq;
                const Half parts = split4(acc);
                char *at = lds + L::Y + r * L::RS + 2 * col;
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    *reinterpret_cast<w2 *>(at + j * L::PART) = parts.p[j];
                grad_store4<E>(rdv, r * vstep + (uint32_t)(vb + col) * E::kBytes, acc);
            }
        };
        if (w < nv / 16) gradients_of_v(w);
        if (NW == 4 && w + NW < nv / 16) {
            load_tile(vb, w + NW);
            gradients_of_v(w + NW);
        }
        load_rows(d4, K + c, vb);  // (not earlier: registers)
        __syncthreads();
        auto rows_of = [&](int base, int i, int t) {  // tile row i, columns 32 t ..
            const char *at = lds + base + (16 * i + x) * L::RS + 64 * t + 16 * gq;
            Operand o;
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                o.p[j] = *reinterpret_cast<const w4 *>(at + j * L::PART);
            return o;
        };
        // O' tile rows times b's parts
        auto dout_mul = [&](int i, int t, const Operand &b, f4 acc) {
            if constexpr (kExact) {
                const w4 a = *reinterpret_cast<const w4 *>(lds + L::O + (16 * i + x) * L::RS +
                                                           64 * t + 16 * gq);
                return mfma(a, b.p[0], mfma(a, b.p[1], mfma(a, b.p[2], acc)));
            } else {
                const Operand a = grad_operand<EO>(
                    rdout,
                    (16 * i + x) * dstep + (uint32_t)(vb + 32 * t + 8 * gq) * EO::kBytes);
#pragma unroll
                for (int j = 0; j < 6; ++j) acc = mfma(a.p[part_a(j)], b.p[part_b(j)], acc);
                return acc;
            }
        };
#pragma unroll
        for (int t = 0; t < VB / 32; ++t) {
            if (32 * t >= nv) break;
            // the states' products
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int s = 0; s < 4; ++s) both = __builtin_fmaf(s4[t][e][s], d4[t][e][s], both);
            {
                const Operand S = join(split4(s4[t][0]), split4(s4[t][1]));
#pragma unroll
                for (int i = 0; i < 4; i += 2) {  // (four at a time lack registers)
                    const Operand a[2] = {rows_of(L::Y, i, t), rows_of(L::Y, i + 1, t)};
#pragma unroll
                    for (int m = 0; m < 6; ++m)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            dk[i + e] = mfma(a[e].p[part_a(m)], S.p[part_b(m)], dk[i + e]);
                    dq[i] = dout_mul(i, t, S, dq[i]);
                    dq[i + 1] = dout_mul(i + 1, t, S, dq[i + 1]);
                }
            }
            {
                const Operand D = join(split4(d4[t][0]), split4(d4[t][1]));
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const Operand a[2] = {rows_of(L::X, i, t), rows_of(L::X, i + 1, t)};
#pragma unroll
                    for (int m = 0; m < 6; ++m)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            ke[i + e] = mfma(a[e].p[part_a(m)], D.p[part_b(m)], ke[i + e]);
                    // E, dP, whose columns are the same rows of X
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const bool isP = NW == 8 ? w >= 4 : j == 1;
                        if (i > tr) continue;
                        if (isP) {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                ex[j][i + e] = dout_mul(tr, t, a[e], ex[j][i + e]);
                        } else {
                            const Operand y = rows_of(L::Y, tr, t);
#pragma unroll
                            for (int m = 0; m < 6; ++m)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    ex[j][i + e] =
                                        mfma(y.p[part_a(m)], a[e].p[part_b(m)], ex[j][i + e]);
                        }
                    }
                }
            }
        }
    }
    const bool per_channel = p.gate_stride == K;
    const Rsrc rk = grad_rows<E>(p.k, ch.row, hk, p.Hk, K, len);
    const Rsrc rq = grad_rows<E>(p.q, ch.row, hk, p.Hk, K, len);
    const Rsrc rg = grad_rows<F32>(p.g, ch.row, h, p.H, p.gate_stride, len);
    const uint32_t kstep = (uint32_t)p.Hk * K, gstep = (uint32_t)p.H * p.gate_stride;
    uint32_t kraw[4][4], qraw[4][4];
    f4 g[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t r = 16 * t + 4 * gq + s, at = r * kstep + c;
            kraw[t][s] = grad_raw1<E>(rk, at * E::kBytes);
            qraw[t][s] = grad_raw1<E>(rq, at * E::kBytes);
            g[t][s] = load1<F32>(rg, 4 * (r * gstep + (per_channel ? c : 0)));
        }
    both = add_rows32(add_rows16(both));
#pragma unroll
    for (int i = 0; i < 4; ++i) ke[i] *= as4(&bs[16 * i + 4 * gq]);
    __syncthreads();

    // E and dP: both halves of dA and dP to LDS; of a tile on the diagonal only
    // what is below it
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const bool isP = NW == 8 ? w >= 4 : j == 1;
        float *mat = isP ? Pm : Am;
        const float factor = isP ? p.scale : -1.0f;
        const Rsrc rA = grad_floats(ws.A(), kGC * kGC);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i <= tr) {
                const int col = 16 * i + x, r0 = 16 * tr + 4 * gq;
                f4 v = ex[j][i];
                if (!isP) {
                    float sum = 0.0f;
                    f4 a;
#pragma unroll
                    for (int s = 0; s < 4; ++s) a[s] = load1<F32>(rA, 4 * ((r0 + s) * kGC + col));
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        sum = __builtin_fmaf(r0 + s > col ? a[s] : 0.0f, v[s], sum);
                    sum = add_rows32(add_rows16(sum));
                    if (gq == 0) cols[tr * kGC + col] = sum;
                }
                v *= factor * bs[col];
                if (i < tr) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) mat[(r0 + s) * kMatRow + col] = v[s];
                    as4(&mat[col * kMatRow + r0]) = v;
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int r = r0 + s;
                        if (r > col) mat[col * kMatRow + r] = v[s];
                        if (r >= col) mat[r * kMatRow + col] = isP || r > col ? v[s] : 0.0f;
                    }
                }
            }
    }
    __syncthreads();
    if ((int)threadIdx.x < len) {
        const int r = threadIdx.x;
        float sum = xdu[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum -= i >= r / 16 ? cols[i * kGC + r] : 0.0f;
        p.dbeta[(long)(ch.row + r) * p.H + h] = sum;
    }

    // the rest by key channels, in registers
    {
        f4 k[4], q[4], pre[4], suf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                k[t][s] = grad_widen<E>(kraw[t][s]);
                q[t][s] = grad_widen<E>(qraw[t][s]);
                g[t][s] = grad_gate(g[t][s]);
            }
        // In registers, tokens 4 g .. 4 g + 3 of a tile: sums through the token
        // (in) and behind it (out) over 4, 16 and more tokens.
        auto in4 = [](f4 v) {
            const float a = v[0] + v[1], b = a + v[2];
            return f4{v[0], a, b, b + v[3]};
        };
        auto out4 = [](f4 v) {
            const float a = v[2] + v[3];
            return f4{v[1] + a, a, v[3], 0.0f};
        };
        auto from4 = [](f4 v) {
            const float a = v[2] + v[3], b = v[1] + a;
            return f4{v[0] + b, b, a, v[3]};
        };
        auto before4 = [](f4 v) {
            const float a = v[0] + v[1];
            return f4{0.0f, v[0], a, a + v[2]};
        };
        // a sum of four tokens, of each group of lanes
        auto groups = [&](float v, float (&part)[4]) {
            float a = v, b = v;
            lane_swap32(a, b);
            part[0] = part[1] = a;
            part[2] = part[3] = b;
            lane_swap16(part[0], part[1]);
            lane_swap16(part[2], part[3]);
        };
        // (by factors of 0 and 1: selections become branches)
        const float u1 = gq >= 1, u2 = gq >= 2, u3 = gq >= 3, l0 = gq < 1, l1 = gq < 2, l2 = gq < 3;
        const float is0 = gq == 0, is1 = gq == 1, is2 = gq == 2, is3 = gq == 3;
        auto earlier = [&](const float (&o)[4]) {
            return __builtin_fmaf(u3, o[2], __builtin_fmaf(u2, o[1], u1 * o[0]));
        };
        auto later = [&](const float (&o)[4]) {
            return __builtin_fmaf(l0, o[1], __builtin_fmaf(l1, o[2], l2 * o[3]));
        };
        float total[4], next8[4];  // next8: of the other group in the token's half of 16
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f4 in = in4(g[t]);
            float o[4];
            groups(in[3], o);
            next8[t] = __builtin_fmaf(is3, o[2], is0 * o[1]);
            pre[t] = in + earlier(o);
            suf[t] = out4(g[t]) + later(o);
            total[t] = (o[0] + o[1]) + (o[2] + o[3]);
        }
        f4 dg[4];
        auto from16 = [&](f4 v, float &sum) {
            float o[4];
            const f4 in = from4(v);
            groups(in[0], o);
            sum = (o[0] + o[1]) + (o[2] + o[3]);
            return in + later(o);
        };
        auto before16 = [&](f4 v, float &sum) {
            float o[4];
            const f4 in = before4(v);
            groups(in[3] + v[3], o);
            sum = (o[0] + o[1]) + (o[2] + o[3]);
            return in + earlier(o);
        };
        // Forms the sums here: the compiler else moves them behind everything,
        // and keeps all of their terms till there.
        auto now = [&](int t) { asm volatile("" : "+v"(dq[t]), "+v"(dk[t]), "+v"(dg[t])); };
        // the states' terms: decays from the chunk's start and to its end
        {
            const float whole = (total[0] + total[1]) + (total[2] + total[3]);
            const float all = __builtin_amdgcn_exp2f(whole) * both;
            float head = 0.0f, rs[4], es[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 eg = exp2(pre[t] + head);
                float tail = 0.0f;
#pragma unroll
                for (int j = 3; j > t; --j) tail += total[j];
                const f4 ez = exp2(suf[t] + tail);
                head += total[t];
                dq[t] = eg * dq[t] * p.scale;
                const f4 r = -eg * dk[t], e = ez * ke[t];
                dk[t] = r + e;
                dg[t] = from16(q[t] * dq[t] + k[t] * r, rs[t]);
                dg[t] += before16(k[t] * e, es[t]);
                now(t);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float more = all;
#pragma unroll
                for (int j = 0; j < 4; ++j) more += j > t ? rs[j] : j < t ? es[j] : 0.0f;
                dg[t] += more;
            }
        }
        // pairs of tokens, level by level: z holds queries of the upper half
        // and keys of the lower, so one product serves rows and columns
        auto level = [&](int t, f4 f, const bool (&upper)[4], f4 e1, f4 e2) {
            f4 term;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float a = f[s] * (upper[s] ? e2[s] : e1[s] + e2[s]);
                const float b = upper[s] ? f[s] * e1[s] : 0.0f;
                dq[t][s] += b;
                dk[t][s] += a;
                term[s] = __builtin_fmaf(q[t][s], b, k[t][s] * a);
            }
            return term;
        };
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            asm volatile("" : "+v"(g[t]));  // its sums are not worth registers till here
            const f4 a = as4(&Am[(16 * t + x) * kMatRow + 16 * t + 4 * gq]);
            const f4 b = as4(&Pm[(16 * t + x) * kMatRow + 16 * t + 4 * gq]);
            // levels 4 and 8
            f4 f[2], e1[2], e2[2], z[2], kf[2], am[2], bm[2];
            bool upper[2][4];
            f[0] = exp2((gq & 1) ? in4(g[t]) : out4(g[t]));
            f[1] = exp2(((gq & 2) ? in4(g[t]) : out4(g[t])) + next8[t]);
#pragma unroll
            for (int l = 0; l < 2; ++l) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int d = (4 * gq + s) ^ x;
                    const bool here = d >= (4 << l) && d < (8 << l);
                    am[l][s] = here ? a[s] : 0.0f;
                    bm[l][s] = here ? b[s] : 0.0f;
                    upper[l][s] = gq & (1 << l);
                    kf[l][s] = k[t][s] * f[l][s];
                    z[l][s] = upper[l][s] ? q[t][s] * f[l][s] : kf[l][s];
                }
                e1[l] = e2[l] = zero4;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    e2[l] = __builtin_amdgcn_mfma_f32_16x16x4f32(am[l][s], kf[l][s], e2[l], 0, 0, 0);
                    e1[l] = __builtin_amdgcn_mfma_f32_16x16x4f32(bm[l][s], z[l][s], e1[l], 0, 0, 0);
                }
            {  // levels 1 and 2, and the diagonal of P: pairs within a lane's four tokens
                f4 A4[4], P4[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int at = (16 * t + 4 * gq + s) * kMatRow + 16 * t + 4 * gq;
                    A4[s] = as4(&Am[at]);
                    P4[s] = as4(&Pm[at]);
                }
                const float f1 = __builtin_amdgcn_exp2f(g[t][1]);
                const float f2 = __builtin_amdgcn_exp2f(g[t][2]);
                const float f3 = __builtin_amdgcn_exp2f(g[t][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    dq[t][i] = __builtin_fmaf(P4[i][i], k[t][i], dq[t][i]);
                    dk[t][i] = __builtin_fmaf(P4[i][i], q[t][i], dk[t][i]);
                    float fall = 1.0f;
#pragma unroll
                    for (int j = i - 1; j >= 0; --j) {
                        fall *= j == 2 ? f3 : j == 1 ? f2 : f1;
                        const float kj = k[t][j] * fall;
                        const float row = A4[i][j] * k[t][i] + P4[i][j] * q[t][i];
                        dq[t][i] = __builtin_fmaf(P4[i][j], kj, dq[t][i]);
                        dk[t][i] = __builtin_fmaf(A4[i][j], kj, dk[t][i]);
                        dk[t][j] = __builtin_fmaf(fall, row, dk[t][j]);
                        const float term = kj * row;
#pragma unroll
                        for (int m = j + 1; m <= i; ++m) dg[t][m] += term;
                    }
                }
            }
            {
                const f4 r4 = level(t, f[0], upper[0], e1[0], e2[0]);
                dg[t] += (gq & 1) ? from4(r4) : before4(r4);
                const f4 r8 = level(t, f[1], upper[1], e1[1], e2[1]);
                float o[4];
                groups((r8[0] + r8[1]) + (r8[2] + r8[3]), o);
                const float more = __builtin_fmaf(is2, o[3], is1 * o[0]);
                dg[t] += ((gq & 2) ? from4(r8) : before4(r8)) + more;
            }
            now(t);
        }
        auto tiles = [&](const float *m, int i, int j) {
            return as4(m + (16 * i + x) * kMatRow + 16 * j + 4 * gq);
        };
#pragma unroll
        for (int pair = 0; pair < 4; pair += 2) {  // level 16: tiles 0 and 1, 2 and 3
            f4 f[2], kf[2], z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = pair + i;
                f[i] = exp2(i ? pre[t] : suf[t]);
                kf[i] = k[t] * f[i];
                z[i] = i ? q[t] * f[i] : kf[i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = pair + i;
                const f4 e2 = mm16(tiles(Am, t, t ^ 1), kf[1 - i], zero4);
                const f4 e1 = mm16(tiles(Pm, t, t ^ 1), z[1 - i], zero4);
                const bool upper[4] = {i == 1, i == 1, i == 1, i == 1};
                const f4 r = level(t, f[i], upper, e1, e2);
                float sum;
                dg[t] += i ? from16(r, sum) : before16(r, sum);
                now(t);
            }
        }
        {  // level 32
            f4 kf[4], z[4];
            float sum[4];
            auto factor = [&](int t) {
                return exp2(t == 0   ? suf[0] + total[1]
                            : t == 1 ? suf[1]
                            : t == 2 ? pre[2]
                                     : pre[3] + total[2]);
            };
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 f = factor(t);
                kf[t] = k[t] * f;
                z[t] = t >= 2 ? q[t] * f : kf[t];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int y = t >= 2 ? 0 : 2;
                const f4 e2 = mm16(tiles(Am, t, y + 1), kf[y + 1],
                                   mm16(tiles(Am, t, y), kf[y], zero4));
                const f4 e1 = mm16(tiles(Pm, t, y + 1), z[y + 1],
                                   mm16(tiles(Pm, t, y), z[y], zero4));
                const bool upper[4] = {t >= 2, t >= 2, t >= 2, t >= 2};
                const f4 r = level(t, factor(t), upper, e1, e2);
                dg[t] += t >= 2 ? from16(r, sum[t]) : before16(r, sum[t]);
                now(t);
            }
            dg[1] += sum[0];
            dg[2] += sum[3];
        }
        const Rsrc rdq = p.dq_head ? grad_rows<F32>(p.dq_head, ch.row, h, p.H, K, len)
                                   : grad_rows<E>(p.dq, ch.row, hk, p.Hk, K, len);
        const Rsrc rdk = p.dq_head ? grad_rows<F32>(p.dk_head, ch.row, h, p.H, K, len)
                                   : grad_rows<E>(p.dk, ch.row, hk, p.Hk, K, len);
        const Rsrc rdg = grad_rows<F32>(p.dg, ch.row, h, p.H, p.gate_stride, len);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t r = 16 * t + 4 * gq + s;
                if (p.dq_head) {
                    grad_store1<F32>(rdq, 4 * (r * p.H * K + c), dq[t][s]);
                    grad_store1<F32>(rdk, 4 * (r * p.H * K + c), dk[t][s]);
                } else {
                    grad_store1<E>(rdq, (r * kstep + c) * E::kBytes, dq[t][s]);
                    grad_store1<E>(rdk, (r * kstep + c) * E::kBytes, dk[t][s]);
                }
                if (per_channel) grad_store1<F32>(rdg, 4 * (r * gstep + c), dg[t][s]);
            }
        if (!per_channel)  // summed over the channels: 16 lanes, then the wavefronts
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float sum = sum16(dg[t][s]);
                    if (x == 0) dgs[w * kGC + 16 * t + 4 * gq + s] = sum;
                }
    }
    if (!per_channel) {
        __syncthreads();
        const int r = threadIdx.x;
        if (r < len) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NW; ++i) sum += dgs[i * kGC + r];
            p.dg[(long)(ch.row + r) * p.H + h] = sum;
        }
    }
}

template <class E>
__device__ __forceinline__ void grad_put4(typename E::T *p, f4 v) {
    if constexpr (E::kBytes == 4)
        *reinterpret_cast<f4 *>(p) = v;
    else
        *reinterpret_cast<w2 *>(p) = w2{Elem<E>::pack(v[0], v[1]), Elem<E>::pack(v[2], v[3])};
}

// Gradients of shared key heads: the sum over the value heads that read them, in
// order, so its bits are the same every time. Bound by memory: it reads FP32 rows
// of every value head (18 us on 8,161 tokens, 8 heads over 4 of 64).
template <class E, int K>
__global__ __launch_bounds__(256) void kda_grad_shared_kernel(DeltaGradProblem p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int hk = (int)(blockIdx.x % p.Hk), slot = (int)(blockIdx.x / p.Hk);
    const GradChunk ch = grad_chunk(p.req, slot, lane);
    const int group = p.H / p.Hk;
    for (int e = threadIdx.x; e < ch.len * (K / 4); e += 256) {  // four channels to a lane
        const long row = ch.row + e / (K / 4);
        const int c = e % (K / 4) * 4;
        const long from = (row * p.H + (long)hk * group) * K + c;
        f4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
        for (int i = 0; i < group; ++i) {
            a += as4(p.dq_head + from + (long)i * K);
            b += as4(p.dk_head + from + (long)i * K);
        }
        const long to = (row * p.Hk + hk) * K + c;
        grad_put4<E>(static_cast<typename E::T *>(p.dq) + to, a);
        grad_put4<E>(static_cast<typename E::T *>(p.dk) + to, b);
    }
}

template <class E, class EO, int K>
hipError_t launch_delta_grad_with(const DeltaGradProblem &p, hipStream_t stream) {
    const unsigned items = (unsigned)((long)p.slots * p.H);
    if (p.req.total_tokens > 0) {
        hipLaunchKernelGGL((kda_grad_prepare_kernel<E, EO, K>), dim3(items), dim3(256), 0, stream,
                           p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    const long walks = (long)p.req.num_seqs * p.H, groups = (walks + 7) / 8;
    // 32 columns to a workgroup halve what the operands cost in L2, 16 columns the
    // work of a step: one sequence of 4,096 tokens takes 170 us in 16 and 243 in
    // 32 with 8 heads (128 and 64 workgroups), 411 and 294 with 32 heads. With K = 64
    // the rule holds, too (the whole call, 4,096 tokens, V = 64: 8 heads 150 and 209, 32
    // heads 348 and 390, 64 heads 685 and 642; V = 128: 16 heads 273 and 327, 32 heads
    // 578 and 535), but not for every set of requests (8,161 tokens in 20, 8 heads, f32
    // 218 and the 232 of this rule: there four workgroups of 16 columns share a unit, two
    // of 32).
    if (2 * walks * (p.V / 16) > device_cus()) {
        const int parts = p.V / 32;
        hipLaunchKernelGGL((kda_grad_walk_kernel<EO, K, 2>), dim3((unsigned)(groups * 8 * parts), 2),
                           dim3(256), 0, stream, p, parts);
    } else {
        const int parts = p.V / 16;
        hipLaunchKernelGGL((kda_grad_walk_kernel<EO, K, 1>), dim3((unsigned)(groups * 8 * parts), 2),
                           dim3(256), 0, stream, p, parts);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (p.req.total_tokens > 0) {
        auto fn = p.V <= 128 ? kda_grad_chunk_kernel<E, EO, K, 128, true>
                             : kda_grad_chunk_kernel<E, EO, K, 128, false>;
        if constexpr (K == 64)
            if (p.V <= 64) fn = kda_grad_chunk_kernel<E, EO, K, 64, true>;
        hipLaunchKernelGGL(fn, dim3(items), dim3(K * 4), 0, stream, p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        if (p.Hk != p.H)
            hipLaunchKernelGGL((kda_grad_shared_kernel<E, K>), dim3((unsigned)(p.slots * p.Hk)),
                               dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

template <class E>
hipError_t launch_delta_grad_of(const DeltaGradProblem &p, int dout_dt, hipStream_t stream) {
    auto with_k = [&]<class EO>() {
        return p.K == 64 ? launch_delta_grad_with<E, EO, 64>(p, stream)
                         : launch_delta_grad_with<E, EO, 128>(p, stream);
    };
    return dout_dt == 0   ? with_k.template operator()<F32>()
           : dout_dt == 1 ? with_k.template operator()<BF16>()
                          : with_k.template operator()<F16>();
}

}  // namespace kda
