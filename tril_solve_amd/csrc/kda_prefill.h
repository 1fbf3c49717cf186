// Gated delta rule over whole prompts, in chunks of 32 tokens, for gfx950.
//
// Per request and value head, S the K x V FP32 state, G_i the decay summed
// from the chunk's first token through token i (per key channel):
//   L_ij = beta_i sum_d k_id k_jd e^{G_id - G_jd} (j < i)
//   P_ij = scale sum_d q_id k_jd e^{G_id - G_jd}  (j <= i)
//   (I + L) U = beta (V - (k e^G) S)
//   O = scale (q e^G) S + P U
//   S <- diag(e^{G_32}) S + (k e^{G_32 - G})^T U
// which is the recurrence S <- diag(e^g) S, u = beta (v - S^T k), S += k u^T,
// o = scale S^T q of 32 tokens at once (the decode step's recurrence).
//
// One workgroup of four wavefronts per request, value head and 128 value
// columns walks the request's chunks. Every product runs on the bfloat16
// matrix cores with FP32 accumulators, each FP32 factor taken as a sum of
// bfloat16 parts (hi = bf16(x), mid = bf16(x - hi), lo = bf16(x - hi - mid)):
//   6 products (hi hi, hi mid, mid hi, mid mid, hi lo, lo hi; about 2^-24 of
//     each term) for what the state is summed from, (k e^{G_32 - G})^T U and
//     the inverse times the right-hand side, and for everything an FP32
//     output is summed from;
//   3 products (hi hi, hi mid, mid hi; about 2^-17) where the result enters
//     only as a correction (L and (k e^G) S: 5e-7 and 1e-7 of the state), and
//     for what a 16-bit output is summed from.
// Against FP32 matrix instructions (16 x 16 x 32 in eight of 32 cycles) that
// is 6 or 3 of 16 cycles. Sums, the state and the decays stay FP32.
//
//   * Each wavefront owns 32 value columns of the state in registers
//     (accumulator layout). With the reduction index of a 16 x 16 x 32
//     product permuted as 8 g + 4 b + s <-> 16 b + 4 g + s, two accumulator
//     tiles are the B operand of the next product as they stand, so the chain
//     k S -> U -> O, S stays inside the wavefront's registers.
//   * The A operands (decayed keys and queries, the inverse of I + L, P) are
//     the same for all columns: the wavefronts prepare them together in LDS,
//     8 tokens each.
//   * Decays enter as factors relative to the middle of each 16-token block,
//     e^{G_i - G_j} = e^{G_i - m} e^{m - G_j}, so that no factor leaves FP32's
//     range while the decay of 8 adjacent tokens stays within e^{+-64}. A
//     chunk that has a steeper channel (or a gate that is not finite) forms
//     its L and P from running products of the decays instead, every factor
//     of which is the decay between two tokens.
#pragma once

#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

constexpr int kPreC = 32;  // tokens per chunk
constexpr int kPreWaves = 4;
constexpr int kPreThreads = kWave * kPreWaves;
constexpr int kPreCols = 32;  // value columns per wavefront
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kSteep = 64.0f * kLog2E;  // in powers of two

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// Position of index x (0..31) of a 32-long reduction in operand order.
__device__ __forceinline__ constexpr int operand_pos(int x) {
    return 8 * ((x & 15) >> 2) + 4 * (x >> 4) + (x & 3);
}

// The first N bfloat16 parts of two floats, packed in pairs.
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t w = Elem<BF16>::pack(a, b);
        part[i] = w;
        if (i + 1 < N) {
            a -= __builtin_bit_cast(float, w << 16);
            b -= __builtin_bit_cast(float, w & 0xFFFF0000u);
        }
    }
}
// An operand half: four values (one accumulator tile), N parts.
template <int N>
struct Half {
    w2 p[N];
};
template <int N>
__device__ __forceinline__ Half<N> split4(f4 x) {
    uint32_t a[N], b[N];
    split2<N>(x[0], x[1], a);
    split2<N>(x[2], x[3], b);
    Half<N> h;
#pragma unroll
    for (int i = 0; i < N; ++i) h.p[i] = w2{a[i], b[i]};
    return h;
}
template <int N>
__device__ __forceinline__ Half<N> zero_half() {
    Half<N> h;
#pragma unroll
    for (int i = 0; i < N; ++i) h.p[i] = w2{0u, 0u};
    return h;
}
// An operand: eight values, N parts.
template <int N>
struct Operand {
    w4 p[N];
};
template <int N>
__device__ __forceinline__ Operand<N> join(const Half<N> &a, const Half<N> &b) {
    Operand<N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.p[i] = w4{a.p[i][0], a.p[i][1], b.p[i][0], b.p[i][1]};
    return o;
}
__device__ __forceinline__ f4 mfma(w4 a, w4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                   __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// c + a b in M = 1, 3 or 6 products, the smallest first.
template <int M, int NA, int NB>
__device__ __forceinline__ f4 mul(const Operand<NA> &a, const Operand<NB> &b, f4 c) {
    static_assert(NA >= (M == 6 ? 3 : M == 3 ? 2 : 1) && NB >= (M == 6 ? 3 : M == 3 ? 2 : 1));
    if constexpr (M == 6) {
        c = mfma(a.p[2], b.p[0], c);
        c = mfma(a.p[0], b.p[2], c);
        c = mfma(a.p[1], b.p[1], c);
    }
    if constexpr (M >= 3) {
        c = mfma(a.p[1], b.p[0], c);
        c = mfma(a.p[0], b.p[1], c);
    }
    return mfma(a.p[0], b.p[0], c);
}

// A lane's CPL adjacent channels of one token as loaded (no conversion).
template <class E, int N>
struct RawC;
template <class E>
struct RawC<E, 2> {
    uint32_t w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    }
    __device__ __forceinline__ float at(int i) const {
        return Elem<E>::widen(i ? w >> 16 : w & 0xFFFFu);
    }
};
template <class E>
struct RawC<E, 1> {
    uint32_t w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    }
    __device__ __forceinline__ float at(int) const { return Elem<E>::widen(w); }
};
template <>
struct RawC<F32, 2> {
    f2 w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(f2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
    __device__ __forceinline__ void load_same(Rsrc r, uint32_t off) {
        const float x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
        w = f2{x, x};
    }
    __device__ __forceinline__ float at(int i) const { return w[i]; }
};
template <>
struct RawC<F32, 1> {
    float w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    }
    __device__ __forceinline__ void load_same(Rsrc r, uint32_t off) { load(r, off); }
    __device__ __forceinline__ float at(int) const { return w; }
};

// LDS layout (bytes). Operands lie in rows of 2 K bytes (reduced over
// channels) or 64 bytes (over tokens); the 16-byte pieces of a row are
// exchanged by an exclusive or with the row number so that the 16 rows that an
// operand read touches fall in different banks without padding.
// OUT: kda_dtype of the output.
template <int K, int OUT>
struct PreLds {
    static constexpr int RS = 2 * K, TS = 2 * kPreC;
    static constexpr int R32 = kPreC * RS, R16 = R32 / 2, T32 = kPreC * TS, KTP = K * TS;
    static constexpr int NQ = OUT == 0 ? 3 : 2;  // parts of P's factors, P and q e^G
    // first half of a chunk: keys, queries (relative to their block's middle)
    // against keys; block 0's keys relative to block 1's middle
    static constexpr int KR = 0, QR = KR + 2 * R32, KL = QR + NQ * R32, KO = KL + NQ * R32;
    static constexpr int kFirst = KO + NQ * R16;
    // the steep form: keys, queries, decays FP32, then L / beta and P
    static constexpr int SK = 0, SQ = SK + kPreC * K * 4, SA = SQ + kPreC * K * 4;
    static constexpr int SM = SA + kPreC * K * 4, SP = SM + kPreC * kPreC * 4;
    static constexpr int kSteepBytes = SP + kPreC * kPreC * 4;
    // second half: k e^G, q e^G, (k e^{G_32 - G})^T
    static constexpr int KS = 0, QS = KS + 2 * R32, KT = QS + NQ * R32;
    static constexpr int kSecond = KT + 3 * KTP;
    static constexpr int kMax1 = kFirst > kSteepBytes ? kFirst : kSteepBytes;
    static constexpr int kShared = kMax1 > kSecond ? kMax1 : kSecond;
    // kept apart: diagonal blocks of the inverse and -L_10; P
    static constexpr int TM = kShared, PM = TM + 3 * T32;
    static constexpr int PATCH = PM + NQ * T32;
    static constexpr int TOT = PATCH + 2 * 16 * 17 * 4;
    static constexpr int DEC = TOT + kPreWaves * K * 4;
    static constexpr int BETA = DEC + K * 4;
    static constexpr int FLAG = BETA + 2 * kPreC * 4;
    static constexpr int kBytes = FLAG + kPreWaves * 4;
    // exchange of 16-byte pieces
    static __device__ __forceinline__ int swz_row(int row) {
        return (K == 128 ? row & 15 : (row >> 1) & 7) << 4;
    }
    static __device__ __forceinline__ int swz_tok(int row) { return ((row >> 2) & 3) << 4; }
};

template <int I, int N>
__device__ __forceinline__ void substitute(const float (&arow)[16], float (&x)[16], int c) {
    if constexpr (I < N) {
        subst_row<I>(arow, x, c);
        substitute<I + 1, N>(arow, x, c);
    }
}

template <class EI, int K, int OUT>
__global__ __launch_bounds__(kPreThreads, 2) void kda_prefill_kernel(DeltaProblem p) {
    typedef PreLds<K, OUT> L;
    constexpr int CPL = K / kWave;  // channels per lane
    constexpr int NT = K / 16;      // state row tiles
    constexpr int NQ = L::NQ;
    constexpr int MQ = OUT == 0 ? 6 : 3;  // products for P, P U and (q e^G) S
    constexpr int OE = OUT == 0 ? 4 : 2;  // bytes of an output element
    __shared__ __align__(16) char lds[L::kBytes];

    const int lane0 = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = blockIdx.x / p.H, h = blockIdx.x - n * p.H;
    const int hk = h / (p.H / p.Hk);
    const int2 rows = request_rows(p.req, n);
    const int len_all = __builtin_amdgcn_readfirstlane(rows.y);
    const long row_first = __builtin_amdgcn_readfirstlane(rows.x);
    const bool keep = p.pool.base != nullptr;
    const int slot = __builtin_amdgcn_readfirstlane(keep ? request_slot(p.pool, n) : 0);

    // this wavefront's columns: tile ct holds column col + ct of each lane
    const int col0 = (blockIdx.y * kPreWaves + wv) * kPreCols;
    const bool cols = col0 < p.V;  // V is a multiple of 32
    const int col = (cols ? col0 : 0) + 2 * (lane0 & 15);

    // Token tensors from the request's first row and this head on, and the
    // bytes between their rows (fewer than 2^21).
    const long first_k = (row_first * p.Hk + hk) * K;
    const long first_v = (row_first * p.H + h) * p.V;
    const int gd = p.gate_stride;
    const uint32_t ks = (uint32_t)(p.Hk * K) * EI::kBytes, gs = (uint32_t)(p.H * gd) * 4;
    const uint32_t vs = (uint32_t)(p.H * p.V) * EI::kBytes, os = (uint32_t)(p.H * p.V) * OE;
    const char *kb = static_cast<const char *>(p.k) + first_k * EI::kBytes;
    const char *qb = static_cast<const char *>(p.q) + first_k * EI::kBytes;
    const char *gb = reinterpret_cast<const char *>(p.g + (row_first * p.H + h) * gd);
    const char *vb = static_cast<const char *>(p.v) + first_v * EI::kBytes;
    char *ob = static_cast<char *>(p.out) + first_v * OE;
    // `len` rows from `base` on as a buffer: rows past them read as 0 and are
    // not written
    auto rows_of = [](const char *base, uint32_t stride, int width, int len) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0,
                                                 (len - 1) * stride + width, kRsrcWord3);
    };
    auto put_out = [&](Rsrc r, uint32_t off, float a, float b) {
        if constexpr (OUT == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(w2, f2{a, b}), r, off, 0,
                                                  kNontemporal);
        else
            __builtin_amdgcn_raw_buffer_store_b32(
                OUT == 1 ? Elem<BF16>::pack(a, b) : Elem<F16>::pack(a, b), r, off, 0,
                kNontemporal);
    };
    if (slot < 0) {  // padding: zero outputs, no state
        if (cols)
            for (int t = lane0 >> 4; t < len_all; t += 4)
#pragma unroll
                for (int c = 0; c < 2 * OE; c += 4)
                    *reinterpret_cast<uint32_t *>(ob + (long)t * os + col * OE + c) = 0u;
        return;
    }

    // the state
    f4 S[NT][2];
    float *pool = p.pool.base + (((long)slot * p.H + h) * K + 4 * (lane0 >> 4)) * p.V + col;
    if (cols && request_continues(p.pool, n)) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const f2 v = __builtin_nontemporal_load(
                    reinterpret_cast<const f2 *>(pool + (long)(16 * rt + s) * p.V));
                S[rt][0][s] = v[0];
                S[rt][1][s] = v[1];
            }
    } else {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
            S[rt][0] = S[rt][1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // entries of the inverse and of P that no chunk writes are zero
    for (int i = threadIdx.x; i < (3 + NQ) * L::T32 / 4; i += kPreThreads)
        reinterpret_cast<uint32_t *>(lds + L::TM)[i] = 0;

    // this wavefront's 8 tokens of the next chunk, as loaded
    RawC<EI, CPL> kraw[8], qraw[8];
    RawC<F32, CPL> graw[8];
    auto load_rows = [&](int t0) {
        const int len = min(kPreC, len_all - t0);
        const Rsrc rk = rows_of(kb + (long)t0 * ks, ks, K * EI::kBytes, len);
        const Rsrc rq = rows_of(qb + (long)t0 * ks, ks, K * EI::kBytes, len);
        const Rsrc rg = rows_of(gb + (long)t0 * gs, gs, gd * 4, len);
        const int lane = opaque_lane(lane0);
        const uint32_t ok = 8 * wv * ks + CPL * lane * EI::kBytes;
        if (gd == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) graw[i].load_same(rg, (8 * wv + i) * gs);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) graw[i].load(rg, 8 * wv * gs + CPL * lane * 4 + i * gs);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            kraw[i].load(rk, ok + i * ks);
            qraw[i].load(rq, ok + i * ks);
        }
    };
    if (len_all > 0) load_rows(0);

    for (int t0 = 0, buf = 0; t0 < len_all; t0 += kPreC, buf ^= 1) {
        const int len = min(kPreC, len_all - t0);
        // the lane made opaque: the many addresses derived from it are formed
        // where they are used instead of being kept (and spilled) across chunks
        const int lane = opaque_lane(lane0);
        const int g4 = lane >> 4, n16 = lane & 15;
        const int ch = CPL * lane;
        // byte of this lane's channels in a row reduced over channels, and of its
        // operand piece
        const int cpos = 2 * (32 * (ch >> 5) + operand_pos(ch & 31));
        const int rpos = n16 * L::RS + ((g4 << 4) ^ L::swz_row(n16));
        const int tpos = n16 * L::TS + ((g4 << 4) ^ L::swz_tok(n16));

        auto put_row = [&]<int N>(int at, int row, int size, const float (&x)[CPL]) {
            char *d = lds + at + row * L::RS + (cpos ^ L::swz_row(row));
            uint32_t part[N];
            split2<N>(x[0], x[CPL - 1], part);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if constexpr (CPL == 2)
                    *reinterpret_cast<uint32_t *>(d + i * size) = part[i];
                else
                    *reinterpret_cast<uint16_t *>(d + i * size) = (uint16_t)part[i];
        };
        // rows 16 I + n16 of an operand
        auto row_operand = [&]<int N>(int at, int kk, int size) -> Operand<N> {
            Operand<N> o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o.p[i] = *reinterpret_cast<const w4 *>(lds + at + i * size + (rpos ^ (64 * kk)));
            return o;
        };
        auto tok_operand = [&]<int N>(int at, int size) -> Operand<N> {
            Operand<N> o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o.p[i] = *reinterpret_cast<const w4 *>(lds + at + i * size + tpos);
            return o;
        };
        // one entry of an operand reduced over tokens
        auto put_entry = [&]<int N>(int at, int row, int c, float x) {
            char *d = lds + at + row * L::TS + ((2 * operand_pos(c)) ^ L::swz_tok(row));
            uint32_t part[N];
            split2<N>(x, 0.0f, part);
#pragma unroll
            for (int i = 0; i < N; ++i)
                *reinterpret_cast<uint16_t *>(d + i * L::T32) = (uint16_t)part[i];
        };

        // ---- 1. decays of this wavefront's 8 tokens
        float tot[CPL];
        float steep = 0.0f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float x = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x += graw[i].at(c) * kLog2E;
                steep = !(__builtin_fabsf(x) <= kSteep) ? 1.0f : steep;
            }
            tot[c] = x;
        }
        float *tots = reinterpret_cast<float *>(lds + L::TOT);
#pragma unroll
        for (int c = 0; c < CPL; ++c) tots[wv * K + ch + c] = tot[c];
        int *flag = reinterpret_cast<int *>(lds + L::FLAG);
        const bool any = __ballot(steep != 0.0f) != 0;
        if (lane == 0) flag[wv] = any;
        float *beta = reinterpret_cast<float *>(lds + L::BETA) + buf * kPreC;
        if (wv == 3 && lane < kPreC)
            beta[lane] =
                lane < len ? p.beta[(row_first + t0 + lane) * p.H + h] : 0.0f;
        __syncthreads();  // totals; every read of the previous chunk's operands is done

        const bool far = (flag[0] | flag[1] | flag[2] | flag[3]) != 0;
        float wt[kPreWaves][CPL];
#pragma unroll
        for (int w = 0; w < kPreWaves; ++w)
#pragma unroll
            for (int c = 0; c < CPL; ++c) wt[w][c] = tots[w * K + ch + c];
        if (wv == 0) {
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                reinterpret_cast<float *>(lds + L::DEC)[ch + c] =
                    __builtin_amdgcn_exp2f(wt[0][c] + wt[1][c] + wt[2][c] + wt[3][c]);
        }
        // e^{G - middle of the block} of every token (or, of a steep chunk, e^G
        // from step 3 on)
        float er[8][CPL];
        if (!far) {
            float ko[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                float x = wv & 1 ? 0.0f : -tot[c];
                ko[c] = __builtin_amdgcn_exp2f(wt[1][c] + wt[2][c]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x += graw[i].at(c) * kLog2E;
                    er[i][c] = __builtin_amdgcn_exp2f(x);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * wv + i;
                float a[CPL], b[CPL], d[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    a[c] = kraw[i].at(c) * er[i][c];
                    b[c] = qraw[i].at(c) * (er[i][c] * p.scale);
                    d[c] = kraw[i].at(c) * __builtin_amdgcn_rcpf(er[i][c]);
                }
                put_row.template operator()<2>(L::KR, r, L::R32, a);
                put_row.template operator()<NQ>(L::QR, r, L::R32, b);
                put_row.template operator()<NQ>(L::KL, r, L::R32, d);
            }
            if (wv < 2) {  // block 0's keys relative to block 1's middle
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float d[CPL];
#pragma unroll
                    for (int c = 0; c < CPL; ++c)
                        d[c] = kraw[i].at(c) * (__builtin_amdgcn_rcpf(er[i][c]) * ko[c]);
                    put_row.template operator()<NQ>(L::KO, 8 * wv + i, L::R16, d);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const int at = (8 * wv + i) * K + ch + c;
                    reinterpret_cast<float *>(lds + L::SK)[at] = kraw[i].at(c);
                    reinterpret_cast<float *>(lds + L::SQ)[at] = qraw[i].at(c) * p.scale;
                    reinterpret_cast<float *>(lds + L::SA)[at] =
                        __builtin_amdgcn_exp2f(graw[i].at(c) * kLog2E);
                }
        }
        __syncthreads();

        // ---- 2. L / beta and P, one 16 x 16 block per wavefront: (0, 0),
        // (1, 1), (1, 0)
        const int bi = wv == 0 ? 0 : 1, bj = wv == 1 ? 1 : 0;
        f4 m = {0.0f, 0.0f, 0.0f, 0.0f}, pp = m;
        if (!far) {
            if (wv < 3) {
                const int kl = wv == 2 ? L::KO : L::KL + 16 * bj * L::RS;
                const int size = wv == 2 ? L::R16 : L::R32;
#pragma unroll
                for (int kk = 0; kk < K / 32; ++kk) {
                    const auto d = row_operand.template operator()<NQ>(kl, kk, size);
                    m = mul<3>(row_operand.template operator()<2>(L::KR + 16 * bi * L::RS, kk,
                                                                  L::R32),
                               d, m);
                    pp = mul<MQ>(row_operand.template operator()<NQ>(L::QR + 16 * bi * L::RS, kk,
                                                                     L::R32),
                                 d, pp);
                }
            }
        } else {
            // running products of the decays from token j on
            const float *sk = reinterpret_cast<const float *>(lds + L::SK);
            const float *sq = reinterpret_cast<const float *>(lds + L::SQ);
            const float *sa = reinterpret_cast<const float *>(lds + L::SA);
            float *sm = reinterpret_cast<float *>(lds + L::SM);
            float *sp = reinterpret_cast<float *>(lds + L::SP);
#pragma unroll 1
            for (int j = wv; j < kPreC; j += kPreWaves) {
                float f[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) f[c] = sk[j * K + ch + c];
#pragma unroll 1
                for (int i = j; i < kPreC; ++i) {
                    float a = 0.0f, b = 0.0f;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        if (i > j) f[c] *= sa[i * K + ch + c];
                        a = __builtin_fmaf(f[c], sk[i * K + ch + c], a);
                        b = __builtin_fmaf(f[c], sq[i * K + ch + c], b);
                    }
                    a = sum64(a);
                    b = sum64(b);
                    if (lane == 0) {
                        sm[i * kPreC + j] = a;
                        sp[i * kPreC + j] = b;
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int at = (16 * bi + 4 * g4 + s) * kPreC + 16 * bj + n16;
                m[s] = sm[at];
                pp[s] = sp[at];
            }
        }
        // the inverse's diagonal blocks and -L_10, and P, as A operands
        if (wv < 3) {
            const f4 b4 = *reinterpret_cast<const f4 *>(beta + 16 * bi + 4 * g4);
            if (wv == 2) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    put_entry.template operator()<2>(L::TM, 16 + 4 * g4 + s, n16, -b4[s] * m[s]);
                    put_entry.template operator()<NQ>(L::PM, 16 + 4 * g4 + s, n16, pp[s]);
                }
            } else {
                float *patch = reinterpret_cast<float *>(lds + L::PATCH) + wv * 16 * 17;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 4 * g4 + s;
                    patch[r * 17 + n16] = n16 < r ? b4[s] * m[s] : 0.0f;
                    put_entry.template operator()<NQ>(L::PM, 16 * wv + r, 16 * wv + n16,
                                                      n16 <= r ? pp[s] : 0.0f);
                }
                wave_sync();
                // forward substitution, one lane per column (every 16-lane row
                // of the wavefront the same)
                float arow[16], x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    arow[j] = patch[n16 * 17 + j];
                    x[j] = j == n16 ? 1.0f : 0.0f;
                }
                substitute<1, 16>(arow, x, n16);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float y = g4 == 0 ? x[s] : g4 == 1 ? x[4 + s]
                                                : g4 == 2   ? x[8 + s]
                                                            : x[12 + s];
                    put_entry.template operator()<3>(L::TM, 16 * wv + 4 * g4 + s, 16 * wv + n16,
                                                     y);
                }
            }
        }
        __syncthreads();

        // ---- 3. k e^G, q e^G and (k e^{G_32 - G})^T
        {
            // k e^{G_32 - G} first, while er is relative to the block's middle
            float kh[8][CPL];
            if (!far) {
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const float before = wv < 2 ? wt[0][c] : wt[0][c] + wt[1][c] + wt[2][c];
                    const float after = wv < 2 ? wt[1][c] + wt[2][c] + wt[3][c] : wt[3][c];
                    const float eb = __builtin_amdgcn_exp2f(before);
                    const float ea = __builtin_amdgcn_exp2f(after);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        kh[i][c] = kraw[i].at(c) * (__builtin_amdgcn_rcpf(er[i][c]) * ea);
                        er[i][c] *= eb;
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    float x = 0.0f, y = 0.0f;
#pragma unroll
                    for (int w = 0; w < kPreWaves; ++w) {
                        x += w < wv ? wt[w][c] : 0.0f;
                        y += w > wv ? wt[w][c] : 0.0f;
                    }
#pragma unroll
                    for (int i = 7; i >= 0; --i) {
                        kh[i][c] = kraw[i].at(c) * __builtin_amdgcn_exp2f(y);
                        y += graw[i].at(c) * kLog2E;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x += graw[i].at(c) * kLog2E;
                        er[i][c] = __builtin_amdgcn_exp2f(x);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const Half<3> hx = split4<3>(
                        f4{kh[4 * j][c], kh[4 * j + 1][c], kh[4 * j + 2][c], kh[4 * j + 3][c]});
                    char *d = lds + L::KT + (ch + c) * L::TS +
                              ((2 * operand_pos(8 * wv + 4 * j)) ^ L::swz_tok(ch + c));
#pragma unroll
                    for (int i = 0; i < 3; ++i) *reinterpret_cast<w2 *>(d + i * L::KTP) = hx.p[i];
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float a[CPL], b[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    a[c] = kraw[i].at(c) * er[i][c];
                    b[c] = qraw[i].at(c) * (er[i][c] * p.scale);
                }
                put_row.template operator()<2>(L::KS, 8 * wv + i, L::R32, a);
                put_row.template operator()<NQ>(L::QS, 8 * wv + i, L::R32, b);
            }
        }
        // the next chunk's rows, and the values of this wavefront's columns
        __syncthreads();
        RawC<EI, 2> vraw[2][4];
        {
            const Rsrc rv = rows_of(vb + (long)t0 * vs, vs, p.V * EI::kBytes, len);
            const uint32_t at = 4 * g4 * vs + col * EI::kBytes;
#pragma unroll
            for (int I = 0; I < 2; ++I)
#pragma unroll
                for (int s = 0; s < 4; ++s) vraw[I][s].load(rv, at + (16 * I + s) * vs);
        }
        if (t0 + kPreC < len_all) load_rows(t0 + kPreC);

        // ---- 4. this wavefront's columns
        if (!cols) continue;
        const f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        f4 ks[2][2] = {{z, z}, {z, z}}, o[2][2] = {{z, z}, {z, z}};
#pragma unroll
        for (int kk = 0; kk < K / 32; ++kk) {
            Operand<NQ> b[2];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
                b[ct] = join(split4<NQ>(S[2 * kk][ct]), split4<NQ>(S[2 * kk + 1][ct]));
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                const auto a =
                    row_operand.template operator()<2>(L::KS + 16 * I * L::RS, kk, L::R32);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) ks[I][ct] = mul<3>(a, b[ct], ks[I][ct]);
                const auto q =
                    row_operand.template operator()<NQ>(L::QS + 16 * I * L::RS, kk, L::R32);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) o[I][ct] = mul<MQ>(q, b[ct], o[I][ct]);
            }
        }
        // U, 16 rows at a time: U_0 = X_00 R_0, U_1 = X_11 (R_1 - L_10 U_0)
        f4 R[2][2];
#pragma unroll
        for (int I = 0; I < 2; ++I) {
            const f4 b4 = *reinterpret_cast<const f4 *>(beta + 16 * I + 4 * g4);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
                    R[I][ct][s] = b4[s] * (vraw[I][s].at(ct) - ks[I][ct][s]);
        }
        Operand<3> u[2];
        {
            const auto x0 = tok_operand.template operator()<3>(L::TM, L::T32);
            const auto x1 = tok_operand.template operator()<3>(L::TM + 16 * L::TS, L::T32);
            const auto p0 = tok_operand.template operator()<NQ>(L::PM, L::T32);
            const auto p1 = tok_operand.template operator()<NQ>(L::PM + 16 * L::TS, L::T32);
            const Half<3> none = zero_half<3>();
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const f4 u0 = mul<6>(x0, join(split4<3>(R[0][ct]), none), z);
                const Half<3> h0 = split4<3>(u0);
                const Operand<3> first = join(h0, none);
                const f4 r1 = mul<3>(x1, first, R[1][ct]);
                const f4 u1 = mul<6>(x1, join(none, split4<3>(r1)), z);
                u[ct] = join(h0, split4<3>(u1));
                o[0][ct] = mul<MQ>(p0, first, o[0][ct]);
                o[1][ct] = mul<MQ>(p1, u[ct], o[1][ct]);
            }
        }
        {
            const Rsrc ro = rows_of(ob + (long)t0 * os, os, p.V * OE, len);
            const uint32_t at = 4 * g4 * os + col * OE;
#pragma unroll
            for (int I = 0; I < 2; ++I)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    put_out(ro, at + (16 * I + s) * os, o[I][0][s], o[I][1][s]);
        }
        // the state
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
            const f4 d = *reinterpret_cast<const f4 *>(lds + L::DEC + (16 * rt + 4 * g4) * 4);
            const auto a = tok_operand.template operator()<3>(L::KT + 16 * rt * L::TS, L::KTP);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) S[rt][ct] = mul<6>(a, u[ct], S[rt][ct] * d);
        }
    }
    if (keep && cols) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                __builtin_nontemporal_store(
                    f2{S[rt][0][s], S[rt][1][s]},
                    reinterpret_cast<f2 *>(pool + (long)(16 * rt + s) * p.V));
    }
}

template <class EI>
hipError_t launch_prefill_of(const DeltaProblem &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.req.num_seqs * p.H),
                    (unsigned)((p.V + kPreWaves * kPreCols - 1) / (kPreWaves * kPreCols)));
    auto go = [&]<int K, int OUT>() {
        hipLaunchKernelGGL((kda_prefill_kernel<EI, K, OUT>), grid, dim3(kPreThreads), 0, stream, p);
        return hipGetLastError();
    };
    auto with_k = [&]<int OUT>() {
        return p.K == 64 ? go.template operator()<64, OUT>() : go.template operator()<128, OUT>();
    };
    return p.out_dt == 0   ? with_k.template operator()<0>()
           : p.out_dt == 1 ? with_k.template operator()<1>()
                           : with_k.template operator()<2>();
}

hipError_t launch_prefill_f32(const DeltaProblem &p, hipStream_t stream);
hipError_t launch_prefill_bf16(const DeltaProblem &p, hipStream_t stream);
hipError_t launch_prefill_f16(const DeltaProblem &p, hipStream_t stream);

}  // namespace kda
