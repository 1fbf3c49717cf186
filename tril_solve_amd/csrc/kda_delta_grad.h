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
// Three launches. Chunks are prepared side by side (A, its inverse, W =
// (I + A B)^-1 (k e^G), X and dU without the states). Then the states walk
// forwards, X -= W S, and their gradients backwards, both at once, each
// wavefront on its own value columns:
//   S <- e^G S + (k e^{G - G_i})^T U,  dS <- e^G dS + (q e^G)^T O' - W^T B dU.
// Last, the chunks' gradients side by side, each wavefront on its own key
// channels. States and their gradients lie in the workspace between launches.
//
// Decays within a chunk never leave [0, 1]: a pair i > j meets at the level
// b = msb(i ^ j) (1, 2, ..., 32) with m the middle of the 2b tokens around both,
// e^{G_i - G_j} = e^{G_i - G_m} e^{G_m - G_j}, both sums of the token's own
// half. A level is a masked product of 16 x 16 (below 16) or of whole tiles, and
// any decay down to e^-inf goes through it exactly. dg is summed the same
// way, level by level, without differences.
//
// All products run on the FP32 matrix instructions: gradients are sums of long
// chains, and FP32 outputs (dg, dbeta, states) are wanted to FP32.
#pragma once

#include <hip/hip_runtime.h>

#include "layer_device.h"
#include "tril_launch.h"

namespace kda {

constexpr int kGC = kGradChunk;
constexpr int kMatRow = kGC + 4;  // floats between rows of a 64 x 64 matrix in LDS
constexpr float kGradLog2E = 1.4426950408889634f;
constexpr float kGradLn2 = 0.6931471805599453f;
constexpr float kLeastGate = -1024.0f;  // in powers of two; e^-inf and this are 0 alike

// Parts of one chunk-head's workspace.
template <int K>
struct GradWork {
    float *base;
    int V;
    __device__ __forceinline__ GradWork(const DeltaGradProblem &p, int slot, int h)
        : base(p.work + ((long)slot * p.H + h) *
                            (2L * kGC * kGC + 5L * kGC * K + 2L * kGC * p.V + 2L * K * p.V + K)),
          V(p.V) {}
    __device__ __forceinline__ float *A() const { return base; }
    __device__ __forceinline__ float *M() const { return base + kGC * kGC; }       // (I + A B)^-1
    __device__ __forceinline__ float *W() const { return M() + kGC * kGC; }        // [C][K]
    __device__ __forceinline__ float *Wt() const { return W() + kGC * K; }         // [K][C]
    __device__ __forceinline__ float *Kb() const { return Wt() + kGC * K; }        // k e^{G - G_i}
    __device__ __forceinline__ float *Kbt() const { return Kb() + kGC * K; }       // [K][C]
    __device__ __forceinline__ float *Qt() const { return Kbt() + kGC * K; }       // q e^G, [K][C]
    __device__ __forceinline__ float *decay() const { return Qt() + kGC * K; }     // e^G, [K]
    __device__ __forceinline__ float *X() const { return decay() + K; }            // [C][V]
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
__device__ __forceinline__ f4 grad_load4(const typename E::T *p);
template <>
__device__ __forceinline__ f4 grad_load4<F32>(const float *p) {
    return *reinterpret_cast<const f4 *>(p);
}
template <>
__device__ __forceinline__ f4 grad_load4<BF16>(const uint16_t *p) {
    const w2 w = *reinterpret_cast<const w2 *>(p);
    return f4{bf16_to_f32(w[0] & 0xFFFFu), bf16_to_f32(w[0] >> 16), bf16_to_f32(w[1] & 0xFFFFu),
              bf16_to_f32(w[1] >> 16)};
}
template <>
__device__ __forceinline__ f4 grad_load4<F16>(const uint16_t *p) {
    const w2 w = *reinterpret_cast<const w2 *>(p);
    return f4{Elem<F16>::widen(w[0] & 0xFFFFu), Elem<F16>::widen(w[0] >> 16),
              Elem<F16>::widen(w[1] & 0xFFFFu), Elem<F16>::widen(w[1] >> 16)};
}
__device__ __forceinline__ void grad_store(float *p, float x) { *p = x; }
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

// A gate in powers of two. NaN stays (a comparison with it is false).
__device__ __forceinline__ float grad_gate(float g) {
    const float x = g * kGradLog2E;
    return x < kLeastGate ? kLeastGate : x;
}

// One level of 16 tokens in lanes 0..15 of a row: the sums of aligned halves of
// b tokens are joined to 2b. pre: through the token from the half's start;
// suf: behind the token to the half's end; tot: of the half.
template <int CTRL>
__device__ __forceinline__ void grad_join(float &pre, float &suf, float &tot, bool upper) {
    const float o = __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, tot), CTRL, 0xF, 0xF, true));
    pre += upper ? o : 0.0f;
    suf += upper ? 0.0f : o;
    tot += o;
}

// ---------------------------------------------------------------- preparation

template <class E, class EO, int K>
__global__ __launch_bounds__(256, 2) void kda_grad_prepare_kernel(DeltaGradProblem p) {
    constexpr int NT = K / 16, KR = K + 4;
    // operands of one level, as the wavefronts hold them; afterwards the
    // matrices M, P, L and, in L's place, the decayed keys
    constexpr int kMat = kGC * kMatRow;
    constexpr int kImages = 6 * NT * 64 * 4, kMats = 2 * kMat + (kMat > kGC * KR ? kMat : kGC * KR);
    __shared__ __align__(16) float lds[kImages > kMats ? kImages : kMats];
    __shared__ __align__(16) float totals[4][K];
    const int lane = threadIdx.x & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    const int h = (int)(blockIdx.x % p.H), slot = (int)(blockIdx.x / p.H);
    const GradChunk ch = grad_chunk(p.req, slot, lane);
    if (ch.len == 0) return;
    if (p.grad.slot != nullptr && request_slot(p.grad, ch.request) < 0) return;
    const GradWork<K> ws(p, slot, h);
    const int V = p.V, tok = 16 * w + x;
    const bool on = tok < ch.len;
    const long row = ch.row + min(tok, ch.len - 1);

    f4 k[NT], q[NT], pre[NT], suf[NT], tot[NT];
    {
        const long at = (row * p.Hk + h / (p.H / p.Hk)) * K + 4 * gq;
        const typename E::T *kp = static_cast<const typename E::T *>(p.k) + at;
        const typename E::T *qp = static_cast<const typename E::T *>(p.q) + at;
        const float *gp = p.g + (row * p.H + h) * p.gate_stride;
        const bool per_channel = p.gate_stride == K;
        const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            k[T] = grad_load4<E>(kp + 16 * T);
            q[T] = grad_load4<E>(qp + 16 * T);
            f4 gg;
            if (per_channel) {
                gg = as4(gp + 16 * T + 4 * gq);
            } else {
                const float one = *gp;
                gg = f4{one, one, one, one};
            }
            if (!on) k[T] = q[T] = gg = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s) gg[s] = grad_gate(gg[s]);
            pre[T] = tot[T] = gg;
            suf[T] = zero;
        }
    }

    // diagonal tiles: the levels below 16 within the wavefront
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
    diagonal(1);
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            float a = pre[T][s], c = suf[T][s], t = tot[T][s];
            grad_join<0xB1>(a, c, t, x & 1);
            pre[T][s] = a, suf[T][s] = c, tot[T][s] = t;
        }
    diagonal(2);
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
    if (x == 0)
#pragma unroll
        for (int T = 0; T < NT; ++T) as4(&totals[w][16 * T + 4 * gq]) = tot[T];
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        const f4 f = factor(T, w & 1);
        image(imK, w, T) = k[T] * f;
        if (w & 1) image(imQ, w >> 1, T) = q[T] * f;
    }
    __syncthreads();
    f4 o16 = {0.0f, 0.0f, 0.0f, 0.0f}, oA = o16, oP = o16;
    {  // wavefronts 0, 1: A and P of tile (1, 0); 2, 3: of tile (3, 2)
        const int pair = w >> 1;
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            const f4 a = (w & 1) ? image(imQ, pair, T) : image(imK, 2 * pair + 1, T);
            o16 = mm16(a, image(imK, 2 * pair, T), o16);
        }
    }
    __syncthreads();
    f4 eg[NT], es[NT];  // e^G from the chunk's start through the token, and from it to the end
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        f4 t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = as4(&totals[j][16 * T + 4 * gq]);
        f4 half = w == 0 ? suf[T] + t[1] : w == 1 ? suf[T] : w == 2 ? pre[T] : pre[T] + t[2];
        half = exp2(half);
        image(imK, w, T) = k[T] * half;
        if (w >= 2) image(imQ, w - 2, T) = q[T] * half;
        const f4 before = w == 0 ? f4{0.0f, 0.0f, 0.0f, 0.0f} : w == 1 ? t[0]
                          : w == 2 ? t[0] + t[1] : t[0] + t[1] + t[2];
        const f4 behind = w == 3 ? f4{0.0f, 0.0f, 0.0f, 0.0f} : w == 2 ? t[3]
                          : w == 1 ? t[2] + t[3] : t[1] + t[2] + t[3];
        eg[T] = exp2(pre[T] + before);
        es[T] = exp2(suf[T] + behind);
        if (w == 0 && x == 0) as4(ws.decay() + 16 * T + 4 * gq) = exp2(t[0] + t[1] + t[2] + t[3]);
    }
    __syncthreads();
    const int ti = 2 + (w >> 1), tj = w & 1;  // this wavefront's tile of level 32
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        const f4 b = image(imK, tj, T);
        oA = mm16(image(imK, ti, T), b, oA);
        oP = mm16(image(imQ, ti - 2, T), b, oP);
    }

    // operands of the walks: k e^{G - G_i} both ways, q e^G by channels
#pragma unroll
    for (int T = 0; T < NT; ++T) {
        const f4 kb = k[T] * es[T], qg = q[T] * eg[T];
        as4(ws.Kb() + tok * K + 16 * T + 4 * gq) = kb;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            ws.Kbt()[(16 * T + 4 * gq + s) * kGC + tok] = kb[s];
            ws.Qt()[(16 * T + 4 * gq + s) * kGC + tok] = qg[s];
        }
    }
    __syncthreads();  // the images are read

    // the matrices: A to memory, L = A B and P to LDS
    float *Mm = lds, *Pm = lds + kMat, *Lm = lds + 2 * kMat;
    auto put = [&](int bi, int bj, f4 a, bool isA, bool isP) {
        const int col = 16 * bj + x;
        const float beta = col < ch.len ? p.beta[(long)(ch.row + col) * p.H + h] : 0.0f;
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
    __syncthreads();

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
    __syncthreads();
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
    __syncthreads();
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
    __syncthreads();

    // k e^G by tokens, in L's place; M to memory
    float *Kg = Lm;
#pragma unroll
    for (int T = 0; T < NT; ++T) as4(&Kg[tok * KR + 16 * T + 4 * gq]) = k[T] * eg[T];
    for (int e = threadIdx.x; e < kGC * kGC / 4; e += 256) {
        const int r = e / (kGC / 4), c = e % (kGC / 4) * 4;
        if (c / 16 <= r / 16) as4(ws.M() + r * kGC + c) = as4(&Mm[r * kMatRow + c]);
    }
    __syncthreads();

    // W = M (k e^G)
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
            for (int t = 0; t <= i; ++t) acc = mm16(left(Mm, i, t), b[t], acc);
            as4(ws.Wt() + (16 * n + x) * kGC + 16 * i + 4 * gq) = acc;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                ws.W()[(16 * i + 4 * gq + s) * K + 16 * n + x] = acc[s];
        }
    }
    // X = M V, dU = P^T O', still without the states
    for (int n = w; n < V / 16; n += 4) {
        f4 b[4], o[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * t + 4 * gq + s;
                const long at = ((long)(ch.row + min(r, ch.len - 1)) * p.H + h) * V + 16 * n + x;
                const float vv = Elem<E>::one(static_cast<const typename E::T *>(p.v) + at);
                const float oo = Elem<EO>::one(static_cast<const typename EO::T *>(p.dout) + at);
                b[t][s] = r < ch.len ? vv : 0.0f;
                o[t][s] = r < ch.len ? p.scale * oo : 0.0f;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 acc = zero4, up = zero4;
#pragma unroll
            for (int t = 0; t <= i; ++t) acc = mm16(left(Mm, i, t), b[t], acc);
#pragma unroll
            for (int t = i; t < 4; ++t) {  // column i of P's tiles, read across
                f4 a;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    a[s] = Pm[(16 * t + 4 * gq + s) * kMatRow + 16 * i + x];
                up = mm16(a, o[t], up);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int at = (16 * i + 4 * gq + s) * V + 16 * n + x;
                ws.X()[at] = acc[s];
                ws.U()[at] = up[s];
            }
        }
    }
}

// -------------------------------------------------------------------- the walks

// A wavefront's columns of a request and head: CT tiles of 16. blockIdx.y: 0
// the states forwards, 1 their gradients backwards.
template <class EO, int K, int CT>
__global__ __launch_bounds__(CT == 1 ? 64 : 512) void kda_grad_walk_kernel(DeltaGradProblem p,
                                                                             int per_head) {
    constexpr int NT = K / 16;
    const int lane = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    const int waves = blockDim.x / kWave;
    const int part = (int)(blockIdx.x % per_head), rest = (int)(blockIdx.x / per_head);
    const int h = rest % p.H, n = rest / p.H;
    const int V = p.V, col = (part * waves + wv) * 16 * CT + x;
    const int2 rows = request_rows(p.req, n);
    const bool back = blockIdx.y != 0;
    const Pool &pool = back ? p.grad : p.pool;
    const int at = p.grad.slot != nullptr || pool.base != nullptr ? request_slot(pool, n) : 0;
    if (at < 0) return;  // padding
    const int chunks = (rows.y + kGC - 1) / kGC, slot0 = rows.x / kGC + n;
    const bool from_pool = pool.base != nullptr && (back || request_continues(pool, n));
    float *state = pool.base + ((long)at * p.H + h) * K * V;
    f4 S[NT][CT];
#pragma unroll
    for (int T = 0; T < NT; ++T)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                S[T][c][s] = from_pool ? state[(16 * T + 4 * gq + s) * V + col + 16 * c] : 0.0f;
    for (int j = 0; j < chunks; ++j) {
        const int c0 = back ? chunks - 1 - j : j;
        const GradWork<K> ws(p, slot0 + c0, h);
        const int row0 = rows.x + c0 * kGC, len = min(kGC, rows.y - c0 * kGC);
        float *kept = back ? ws.D() : ws.S();
        const float *lhs = back ? ws.Kb() : ws.W();
        float *io = back ? ws.U() : ws.X();
#pragma unroll
        for (int T = 0; T < NT; ++T)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    kept[(16 * T + 4 * gq + s) * V + col + 16 * c] = S[T][c][s];
        // X - W S, or dU + (k e^{G - G_i}) dS
        f4 u[4][CT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 acc[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int T = 0; T < NT; ++T) {
                const f4 a = as4(lhs + (16 * i + x) * K + 16 * T + 4 * gq);
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[c] = mm16(a, S[T][c], acc[c]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * i + 4 * gq + s;
                const long row = (long)(row0 + min(r, len - 1)) * p.H + h;
                const float beta = r < len ? p.beta[row] : 0.0f;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    float *e = io + r * V + col + 16 * c;
                    const float y = back ? *e + acc[c][s] : *e - acc[c][s];
                    *e = y;
                    u[i][c][s] = back ? -beta * y : beta * y;
                }
            }
        }
        // e^G S + (k e^{G - G_i})^T U, or e^G dS - W^T B dU + (q e^G)^T O'
        const float *rhs = back ? ws.Wt() : ws.Kbt();
#pragma unroll
        for (int T = 0; T < NT; ++T) {
            const f4 d = as4(ws.decay() + 16 * T + 4 * gq);
#pragma unroll
            for (int c = 0; c < CT; ++c) S[T][c] *= d;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 a = as4(rhs + (16 * T + x) * kGC + 16 * t + 4 * gq);
#pragma unroll
                for (int c = 0; c < CT; ++c) S[T][c] = mm16(a, u[t][c], S[T][c]);
            }
        }
        if (back) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * t + 4 * gq + s;
                    const long row = ((long)(row0 + min(r, len - 1)) * p.H + h) * V + col;
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const float o = Elem<EO>::one(
                            static_cast<const typename EO::T *>(p.dout) + row + 16 * c);
                        u[t][c][s] = r < len ? p.scale * o : 0.0f;
                    }
                }
#pragma unroll
            for (int T = 0; T < NT; ++T)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const f4 a = as4(ws.Qt() + (16 * T + x) * kGC + 16 * t + 4 * gq);
#pragma unroll
                    for (int c = 0; c < CT; ++c) S[T][c] = mm16(a, u[t][c], S[T][c]);
                }
        }
    }
    if (back && pool.base != nullptr) {
        const bool cont = request_continues(pool, n);
#pragma unroll
        for (int T = 0; T < NT; ++T)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    state[(16 * T + 4 * gq + s) * V + col + 16 * c] = cont ? S[T][c][s] : 0.0f;
    }
}

// ------------------------------------------------------------ gradients of a chunk

template <class E, class EO, int K>
__global__ __launch_bounds__(256, 2) void kda_grad_chunk_kernel(DeltaGradProblem p) {
    constexpr int NT = K / 16;
    extern __shared__ __align__(16) float lds[];
    const int lane = threadIdx.x & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int x = lane & 15, gq = lane >> 4;
    const int h = (int)(blockIdx.x % p.H), slot = (int)(blockIdx.x / p.H);
    const GradChunk ch = grad_chunk(p.req, slot, lane);
    if (ch.len == 0) return;
    const int V = p.V, VR = V + 4, len = ch.len;
    const int hk = h / (p.H / p.Hk);
    typedef typename E::T T_;
    if (p.grad.slot != nullptr && request_slot(p.grad, ch.request) < 0) {  // padding: zeros
        for (int r = w; r < len; r += 4) {
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
    const GradWork<K> ws(p, slot, h);
    constexpr int kMat = kGC * kMatRow;
    float *Am = lds, *Pm = lds + kMat;  // dA and dP, both halves (first M, in Am)
    float *Ys = lds + 2 * kMat;         // [C][V + 4]
    float *bs = Ys + kGC * VR;          // beta [C], X.dU [C], column sums [2][C]
    float *xdu = bs + kGC, *cols = xdu + kGC;
    float *dgs = cols + 2 * kGC;        // [4][C] per wavefront (one gate per head)
    const f4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};

    for (int e = threadIdx.x; e < kGC * kGC / 4; e += 256) {
        const int r = e / (kGC / 4), c = e % (kGC / 4) * 4;
        if (c / 16 <= r / 16) as4(&Am[r * kMatRow + c]) = as4(ws.M() + r * kGC + c);
    }
    if (threadIdx.x < kGC)
        bs[threadIdx.x] = (int)threadIdx.x < len
                              ? p.beta[(long)(ch.row + threadIdx.x) * p.H + h] : 0.0f;
    {  // X.dU: four lanes to a row
        const int r = threadIdx.x >> 2;
        float sum = 0.0f;
        for (int c = 4 * (threadIdx.x & 3); c < V; c += 16) {
            const f4 a = as4(ws.X() + r * V + c), b = as4(ws.U() + r * V + c);
#pragma unroll
            for (int s = 0; s < 4; ++s) sum = __builtin_fmaf(a[s], b[s], sum);
        }
        sum = lane_add<0x4E>(lane_add<0xB1>(sum));
        if ((threadIdx.x & 3) == 0) xdu[r] = sum;
    }
    __syncthreads();

    // Y = M^T (B dU)
    for (int n = w; n < V / 16; n += 4) {
        f4 b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * t + 4 * gq + s;
                b[t][s] = bs[r] * ws.U()[r * V + 16 * n + x];
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f4 acc = zero4;
#pragma unroll
            for (int t = i; t < 4; ++t) {
                f4 a;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    a[s] = Am[(16 * t + 4 * gq + s) * kMatRow + 16 * i + x];
                acc = mm16(a, b[t], acc);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * i + 4 * gq + s;
                Ys[r * VR + 16 * n + x] = acc[s];
                if (r < len)
                    grad_put<E>(static_cast<T_ *>(p.dv) +
                                    ((long)(ch.row + r) * p.H + h) * V + 16 * n + x, acc[s]);
            }
        }
    }
    __syncthreads();

    auto dout4 = [&](int r, int c) {
        const long at = ((long)(ch.row + min(r, len - 1)) * p.H + h) * V + c;
        const f4 o = grad_load4<EO>(static_cast<const typename EO::T *>(p.dout) + at);
        return r < len ? o * p.scale : f4{0.0f, 0.0f, 0.0f, 0.0f};
    };

    // E = strict(Y X^T) (even wavefronts) and low(O' X^T) (odd): tile rows 3 and 0
    // (0, 1) or 2 and 1 (2, 3)
    {
        const bool isP = w & 1;
        const int hi = w < 2 ? 3 : 2, lo = w < 2 ? 0 : 1;
        f4 up[4], dn[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) up[j] = zero4;
        dn[0] = dn[1] = zero4;
        for (int T = 0; T < V / 16; ++T) {
            const int c = 16 * T + 4 * gq;
            const f4 a = isP ? dout4(16 * hi + x, c) : as4(&Ys[(16 * hi + x) * VR + c]);
            const f4 b = isP ? dout4(16 * lo + x, c) : as4(&Ys[(16 * lo + x) * VR + c]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= hi) {
                    const f4 xv = as4(ws.X() + (16 * j + x) * V + c);
                    up[j] = mm16(a, xv, up[j]);
                    if (j < 2 && j <= lo) dn[j] = mm16(b, xv, dn[j]);
                }
        }
        float colsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        auto place = [&](int i, int j, f4 v) {
            const int c = 16 * j + x;
            const float beta = bs[c];
            float *mat = isP ? Pm : Am;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * i + 4 * gq + s;
                float e = v[s];
                if (isP) {
                    if (r >= c) mat[r * kMatRow + c] = mat[c * kMatRow + r] = e * beta;
                } else {
                    e = r > c ? e : 0.0f;
                    colsum[j] = __builtin_fmaf(r > c ? ws.A()[r * kGC + c] : 0.0f, e, colsum[j]);
                    if (r > c) mat[r * kMatRow + c] = mat[c * kMatRow + r] = -e * beta;
                    if (r == c) mat[r * kMatRow + c] = 0.0f;
                }
            }
        };
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= hi) place(hi, j, up[j]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j <= lo) place(lo, j, dn[j]);
        if (!isP)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float sum = add_rows32(add_rows16(colsum[j]));
                if (gq == 0) cols[(w >> 1) * kGC + 16 * j + x] = sum;
            }
    }
    __syncthreads();
    if ((int)threadIdx.x < len)
        p.dbeta[(long)(ch.row + threadIdx.x) * p.H + h] =
            xdu[threadIdx.x] - cols[threadIdx.x] - cols[kGC + threadIdx.x];

    // the rest by key channels: 16 to a wavefront at a time
    const bool per_channel = p.gate_stride == K;
    f4 dg_head[4] = {zero4, zero4, zero4, zero4};
    for (int n = w; n < NT; n += 4) {
        const int c = 16 * n + x;
        // O' S^T, Y S^T, U dS^T and the rows of S * dS
        f4 dq[4], dk[4], ke[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[i] = dk[i] = ke[i] = zero4;
        float both = 0.0f;
        for (int T = 0; T < V / 16; ++T) {
            const int v = 16 * T + 4 * gq;
            const f4 s4 = as4(ws.S() + c * V + v), d4 = as4(ws.D() + c * V + v);
#pragma unroll
            for (int s = 0; s < 4; ++s) both = __builtin_fmaf(s4[s], d4[s], both);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * i + x;
                dq[i] = mm16(dout4(r, v), s4, dq[i]);
                dk[i] = mm16(as4(&Ys[r * VR + v]), s4, dk[i]);
                ke[i] = mm16(as4(ws.X() + r * V + v) * bs[r], d4, ke[i]);
            }
        }
        both = add_rows32(add_rows16(both));

        f4 k[4], q[4], pre[4], suf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * t + 4 * gq + s;
                const long row = ch.row + min(r, len - 1);
                const long at = (row * p.Hk + hk) * K + c;
                const float kk = Elem<E>::one(static_cast<const T_ *>(p.k) + at);
                const float qq = Elem<E>::one(static_cast<const T_ *>(p.q) + at);
                const float gg = p.g[(row * p.H + h) * p.gate_stride + (per_channel ? c : 0)];
                k[t][s] = r < len ? kk : 0.0f;
                q[t][s] = r < len ? qq : 0.0f;
                pre[t][s] = grad_gate(r < len ? gg : 0.0f);
            }
        // In registers, tokens 4 g .. 4 g + 3 of a tile: sums before (through
        // the token) and behind it, over 2, 4, 8, 16 and more tokens. fac(b): the
        // factor of level b.
        f4 fac[4][4];  // levels 1, 2, 4, 8 of each tile
        float total[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f4 g = pre[t];
            fac[0][t] = exp2(f4{0.0f, g[1], 0.0f, g[3]});
            fac[1][t] = exp2(f4{g[1], 0.0f, g[2], g[2] + g[3]});
            const f4 in = {g[0], g[0] + g[1], g[0] + g[1] + g[2], g[0] + g[1] + g[2] + g[3]};
            const f4 out = {g[1] + g[2] + g[3], g[2] + g[3], g[3], 0.0f};
            fac[2][t] = exp2((gq & 1) ? in : out);
            f4 part[4];  // totals of the four groups of lanes
            gather_groups<4>(f4{in[3], 0.0f, 0.0f, 0.0f}, part);
            const float t0 = part[0][0], t1 = part[1][0], t2 = part[2][0], t3 = part[3][0];
            const float e8 = gq == 3 ? t2 : gq == 0 ? t1 : 0.0f;
            fac[3][t] = exp2((gq & 2) ? in + e8 : out + e8);
            const float b16 = gq == 0 ? 0.0f : gq == 1 ? t0 : gq == 2 ? t0 + t1 : t0 + t1 + t2;
            const float a16 = gq == 3 ? 0.0f : gq == 2 ? t3 : gq == 1 ? t2 + t3 : t1 + t2 + t3;
            pre[t] = in + b16;
            suf[t] = out + a16;
            total[t] = t0 + t1 + t2 + t3;
        }
        f4 dg[4];
        // sums of x over the tokens of a tile from this one on, or before it
        auto groups = [&](f4 v, float (&part)[4]) {
            f4 o[4];
            gather_groups<4>(f4{v[0] + v[1] + v[2] + v[3], 0.0f, 0.0f, 0.0f}, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) part[i] = o[i][0];
        };
        auto from4 = [](f4 v) {
            return f4{v[0] + v[1] + v[2] + v[3], v[1] + v[2] + v[3], v[2] + v[3], v[3]};
        };
        auto before4 = [](f4 v) { return f4{0.0f, v[0], v[0] + v[1], v[0] + v[1] + v[2]}; };
        auto from16 = [&](f4 v, float &sum) {
            float o[4];
            groups(v, o);
            sum = o[0] + o[1] + o[2] + o[3];
            return from4(v) + (gq == 3 ? 0.0f : gq == 2 ? o[3] : gq == 1 ? o[2] + o[3]
                                                              : o[1] + o[2] + o[3]);
        };
        auto before16 = [&](f4 v, float &sum) {
            float o[4];
            groups(v, o);
            sum = o[0] + o[1] + o[2] + o[3];
            return before4(v) + (gq == 0 ? 0.0f : gq == 1 ? o[0] : gq == 2 ? o[0] + o[1]
                                                                : o[0] + o[1] + o[2]);
        };
        // the states' terms: decays from the chunk's start and to its end
        {
            const float whole = total[0] + total[1] + total[2] + total[3];
            const float all = __builtin_amdgcn_exp2f(whole) * both;
            float head = 0.0f, rs[4], es[4];
            f4 er[4], rr[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 eg = exp2(pre[t] + head);
                float tail = 0.0f;
#pragma unroll
                for (int j = 3; j > t; --j) tail += total[j];
                const f4 ez = exp2(suf[t] + tail);
                head += total[t];
                dq[t] = eg * dq[t];
                const f4 r = -eg * dk[t], e = ez * ke[t];
                dk[t] = r + e;
                rr[t] = from16(q[t] * dq[t] + k[t] * r, rs[t]);
                er[t] = before16(k[t] * e, es[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float more = all;
#pragma unroll
                for (int j = 0; j < 4; ++j) more += j > t ? rs[j] : j < t ? es[j] : 0.0f;
                dg[t] = rr[t] + er[t] + more;
            }
        }
        // pairs of tokens, level by level: z holds queries of the upper half
        // and keys of the lower, so one product serves rows and columns
        auto level = [&](int t, f4 f, bool upper[4], f4 e1, f4 e2) {
            f4 term;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float kf = k[t][s] * f[s], qf = q[t][s] * f[s];
                if (upper[s]) {
                    dq[t][s] = __builtin_fmaf(f[s], e1[s], dq[t][s]);
                    dk[t][s] = __builtin_fmaf(f[s], e2[s], dk[t][s]);
                    term[s] = qf * e1[s] + kf * e2[s];
                } else {
                    dk[t][s] = __builtin_fmaf(f[s], e1[s] + e2[s], dk[t][s]);
                    term[s] = kf * (e1[s] + e2[s]);
                }
            }
            return term;
        };
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f4 a = as4(&Am[(16 * t + x) * kMatRow + 16 * t + 4 * gq]);
            const f4 b = as4(&Pm[(16 * t + x) * kMatRow + 16 * t + 4 * gq]);
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                f4 am, bm, z, kf;
                bool upper[4];
                const f4 f = fac[l][t];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int d = (4 * gq + s) ^ x;
                    const bool here = d >= (1 << l) && d < (2 << l);
                    am[s] = here ? a[s] : 0.0f;
                    bm[s] = here ? b[s] : 0.0f;
                    upper[s] = (4 * gq + s) & (1 << l);
                    kf[s] = k[t][s] * f[s];
                    z[s] = upper[s] ? q[t][s] * f[s] : kf[s];
                }
                const f4 e2 = mm16(am, kf, zero4), e1 = mm16(bm, z, zero4);
                const f4 r = level(t, f, upper, e1, e2);
                if (l == 0) {
                    dg[t][1] += r[1];
                    dg[t][3] += r[3];
                } else if (l == 1) {
                    dg[t][1] += r[0];
                    dg[t][2] += r[2] + r[3];
                    dg[t][3] += r[3];
                } else if (l == 2) {
                    dg[t] += (gq & 1) ? from4(r) : before4(r);
                } else {
                    float o[4];
                    groups(r, o);
                    dg[t] += (gq & 2) ? from4(r) + (gq == 2 ? o[3] : 0.0f)
                                      : before4(r) + (gq == 1 ? o[0] : 0.0f);
                }
            }
            // the diagonal of P
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * t + 4 * gq + s;
                const float d = Pm[r * kMatRow + r];
                dq[t][s] = __builtin_fmaf(d, k[t][s], dq[t][s]);
                dk[t][s] = __builtin_fmaf(d, q[t][s], dk[t][s]);
            }
        }
        auto tiles = [&](const float *m, int i, int j) {
            return as4(m + (16 * i + x) * kMatRow + 16 * j + 4 * gq);
        };
        {  // level 16
            f4 f[4], kf[4], z[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f[t] = exp2((t & 1) ? pre[t] : suf[t]);
                kf[t] = k[t] * f[t];
                z[t] = (t & 1) ? q[t] * f[t] : kf[t];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 e2 = mm16(tiles(Am, t, t ^ 1), kf[t ^ 1], zero4);
                const f4 e1 = mm16(tiles(Pm, t, t ^ 1), z[t ^ 1], zero4);
                bool upper[4] = {(t & 1) != 0, (t & 1) != 0, (t & 1) != 0, (t & 1) != 0};
                const f4 r = level(t, f[t], upper, e1, e2);
                float sum;
                dg[t] += (t & 1) ? from16(r, sum) : before16(r, sum);
            }
        }
        {  // level 32
            f4 f[4], kf[4], z[4], term[4];
            float sum[4];
            f[0] = exp2(suf[0] + total[1]);
            f[1] = exp2(suf[1]);
            f[2] = exp2(pre[2]);
            f[3] = exp2(pre[3] + total[2]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                kf[t] = k[t] * f[t];
                z[t] = t >= 2 ? q[t] * f[t] : kf[t];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int y = t >= 2 ? 0 : 2;
                const f4 e2 = mm16(tiles(Am, t, y + 1), kf[y + 1],
                                   mm16(tiles(Am, t, y), kf[y], zero4));
                const f4 e1 = mm16(tiles(Pm, t, y + 1), z[y + 1],
                                   mm16(tiles(Pm, t, y), z[y], zero4));
                bool upper[4] = {t >= 2, t >= 2, t >= 2, t >= 2};
                const f4 r = level(t, f[t], upper, e1, e2);
                term[t] = t >= 2 ? from16(r, sum[t]) : before16(r, sum[t]);
            }
            dg[0] += term[0];
            dg[1] += term[1] + sum[0];
            dg[2] += term[2] + sum[3];
            dg[3] += term[3];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * t + 4 * gq + s;
                if (r < len) {
                    const long row = ch.row + r, at = row * p.H + h;
                    if (p.dq_head) {
                        p.dq_head[at * K + c] = dq[t][s];
                        p.dk_head[at * K + c] = dk[t][s];
                    } else {
                        grad_put<E>(static_cast<T_ *>(p.dq) + (row * p.Hk + hk) * K + c, dq[t][s]);
                        grad_put<E>(static_cast<T_ *>(p.dk) + (row * p.Hk + hk) * K + c, dk[t][s]);
                    }
                    if (per_channel) p.dg[at * K + c] = dg[t][s];
                }
            }
#pragma unroll
        for (int t = 0; t < 4; ++t) dg_head[t] += dg[t];
    }
    if (!per_channel) {  // summed over the channels: 16 lanes, then the wavefronts
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float sum = sum16(dg_head[t][s]);
                if (x == 0) dgs[w * kGC + 16 * t + 4 * gq + s] = sum;
            }
        __syncthreads();
        const int r = threadIdx.x;
        if (r < len)
            p.dg[(long)(ch.row + r) * p.H + h] =
                (dgs[r] + dgs[kGC + r]) + (dgs[2 * kGC + r] + dgs[3 * kGC + r]);
    }
}

// Gradients of shared key heads: the sum over the value heads that read them.
template <class E, int K>
__global__ __launch_bounds__(256) void kda_grad_shared_kernel(DeltaGradProblem p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int hk = (int)(blockIdx.x % p.Hk), slot = (int)(blockIdx.x / p.Hk);
    const GradChunk ch = grad_chunk(p.req, slot, lane);
    const int group = p.H / p.Hk;
    for (int e = threadIdx.x; e < ch.len * K; e += 256) {
        const long row = ch.row + e / K;
        const int c = e % K;
        const long from = (row * p.H + (long)hk * group) * K + c;
        float a = 0.0f, b = 0.0f;
        for (int i = 0; i < group; ++i) {
            a += p.dq_head[from + (long)i * K];
            b += p.dk_head[from + (long)i * K];
        }
        const long to = (row * p.Hk + hk) * K + c;
        grad_put<E>(static_cast<typename E::T *>(p.dq) + to, a);
        grad_put<E>(static_cast<typename E::T *>(p.dk) + to, b);
    }
}

constexpr size_t grad_chunk_lds(int V) {
    return sizeof(float) * (2 * kGC * kMatRow + kGC * (V + 4) + 8 * kGC);
}

template <class E, class EO, int K>
hipError_t launch_delta_grad_with(const DeltaGradProblem &p, hipStream_t stream) {
    const unsigned items = (unsigned)((long)p.slots * p.H);
    if (p.req.total_tokens > 0) {
        hipLaunchKernelGGL((kda_grad_prepare_kernel<E, EO, K>), dim3(items), dim3(256), 0, stream,
                           p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    const long walks = (long)p.req.num_seqs * p.H;
    if (walks * (p.V / 16) > 2048) {
        const int waves = p.V / 32;
        hipLaunchKernelGGL((kda_grad_walk_kernel<EO, K, 2>), dim3((unsigned)walks, 2),
                           dim3(waves * kWave), 0, stream, p, 1);
    } else {
        hipLaunchKernelGGL((kda_grad_walk_kernel<EO, K, 1>),
                           dim3((unsigned)(walks * (p.V / 16)), 2), dim3(kWave), 0, stream, p,
                           p.V / 16);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (p.req.total_tokens > 0) {
        const auto fn = kda_grad_chunk_kernel<E, EO, K>;
        const size_t lds = grad_chunk_lds(p.V);
        if (lds > 64 * 1024) {
            const hipError_t e = hipFuncSetAttribute(
                reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                (int)lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(fn, dim3(items), dim3(256), lds, stream, p);
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
