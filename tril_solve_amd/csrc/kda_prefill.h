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
// A workgroup per request, value head and 128 (or 64) value columns walks the
// request's chunks. Every product runs on the bfloat16 matrix cores with FP32
// accumulators, each FP32 factor taken as a sum of three bfloat16 parts
// (hi = bf16(x), mid = bf16(x - hi), lo = bf16(x - hi - mid)), in six products
// (hi hi, hi mid, mid hi, mid mid, hi lo, lo hi; about 2^-24 of each term). That
// is 6 of 16 cycles against FP32 matrix instructions' eight of 32 (16 x 16 x 32).
// Sums, the state and the decays stay FP32. State and FP32 outputs are 1e-7 to
// 4e-7 of their norm from 64 bits, and a 16-bit output differs from the rounded
// exact one as often as FP32 arithmetic does (bf16: 2e-5 to 5e-5 of the norm).
// Fewer products were faster, but lost bits: three in L and (k e^G) S 2e-6 of the
// state where decays are slow, three in the correction L_10 U_0 7e-6 where keys
// have a common direction; three in P and what 16-bit outputs are summed from
// (16 x 512 tokens 398 us instead of 462 on one card) four times as many
// outputs rounded to the other neighbour.
//
//   * Each wavefront owns 32 (or 16) value columns of the state in registers
//     (accumulator layout). Two accumulator tiles b = 0, 1 are the B operand of
//     the next product as they stand when its reduction index 8 g + 4 b + s
//     means row 4 g + s of tile b: tokens 16 b + 4 g + s of U, and, for the
//     state, tile 2 i + b holding channels 32 i + 8 g + 4 b + s, so that keys
//     and queries keep their order. The chain k S -> U -> O, S thus stays
//     inside the wavefront's registers.
//   * The A operands (decayed keys and queries, the inverse of I + L times
//     beta, P) are the same for all columns: four wavefronts prepare them
//     together in LDS, 8 tokens each.
//   * Decays enter as factors relative to the chunk's middle, G_16 =: m:
//     e^{G_i - G_j} = e^{G_i - m} e^{m - G_j}, and with S' = e^m S
//       (k e^G) S = (k e^{G - m}) S',  (q e^G) S likewise,
//       e^{G_32} S + (k e^{G_32 - G})^T U = e^{G_32 - m} (S' + (k e^{m - G})^T U),
//     so three operands serve all six products, and the last one is the keys
//     of L and P read transposed from LDS. No factor leaves FP32's range while
//     the decay of 16 adjacent tokens stays within e^{-64}. A chunk that has a
//     steeper channel (or a gate that is not finite) forms its L and P from
//     running products of the decays instead, every factor of which is the
//     decay between two tokens, and takes the left-hand forms above. The factor
//     e^{G_32 - m} is left owing and taken together with the next chunk's e^m.
//     Sums of decays past 2^8 over 16 tokens are formed in fixed point: in FP32
//     they keep 2^-17 of a power of two at 2^-74, which neighbours far from the
//     middle lose between them (state 1.6e-6 off, then 4e-7).
//
// Two forms. With many workgroups, four wavefronts prepare a chunk and then
// walk their columns through it, two workgroups to a compute unit (79 KB of
// LDS each). With at most 256, wavefronts of either kind work side by side, one
// chunk apart, on twice the LDS: 64 walks of 2,048 tokens 567 -> 416 us, 32
// of 16,384 tokens 4.47 -> 3.23 ms; but 1,024 walks of 512 tokens, four rounds
// of workgroups whose beginnings and ends nothing covers, 453 -> 465 us.
//
// What bounds it: instruction issue and, with all units at work, power (1.6 to
// 1.8 of 2.4 GHz). A wavefront's chunk is 384 matrix instructions and 2,020
// vector instructions, 16 and 4 cycles each, most of them the splits into
// parts; 16 x 512 tokens of 64 heads, K = V = 128, bf16, take 432 to 470 us on
// three cards: 2.0 TB/s of the 6.4 that a tuned copy reaches, 0.95 of 2.5 PFLOP/s of
// the products as run.
#pragma once

#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

constexpr int kPreC = 32;  // tokens per chunk
constexpr int kPreWaves = 4;  // that prepare a chunk
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kSteep = 64.0f * kLog2E;  // in powers of two
constexpr float kFine = 8.0f;             // likewise
constexpr float kFixed = 16777216.0f;     // units of 2^-24 of a power of two

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// Position of token x (0..31) in an operand reduced over tokens.
__device__ __forceinline__ constexpr int operand_pos(int x) {
    return 8 * ((x & 15) >> 2) + 4 * (x >> 4) + (x & 3);
}

constexpr int kParts = 3;  // bfloat16 parts of an FP32 factor
// The parts of two floats, packed in pairs.
__device__ __forceinline__ void split2(float a, float b, uint32_t (&part)[kParts]) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        uint32_t w = Elem<BF16>::pack(a, b);
        asm("" : "+v"(w));  // else a's own conversion is made a second time
        part[i] = w;
        if (i + 1 < kParts) {
            a -= __builtin_bit_cast(float, w << 16);
            b -= __builtin_bit_cast(float, w & 0xFFFF0000u);
        }
    }
}
// The parts of an operand half: four values (one accumulator tile).
struct Half {
    w2 p[kParts];
};
__device__ __forceinline__ Half split4(f4 x) {
    uint32_t a[kParts], b[kParts];
    split2(x[0], x[1], a);
    split2(x[2], x[3], b);
    Half h;
#pragma unroll
    for (int i = 0; i < kParts; ++i) h.p[i] = w2{a[i], b[i]};
    return h;
}
// The parts of an operand: eight values.
struct Operand {
    w4 p[kParts];
};
__device__ __forceinline__ Operand join(const Half &a, const Half &b) {
    Operand o;
#pragma unroll
    for (int i = 0; i < kParts; ++i) o.p[i] = w4{a.p[i][0], a.p[i][1], b.p[i][0], b.p[i][1]};
    return o;
}
__device__ __forceinline__ Half half_of(const Operand &o, int which) {
    Half h;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
        h.p[i] = which ? w2{o.p[i][2], o.p[i][3]} : w2{o.p[i][0], o.p[i][1]};
    return h;
}
__device__ __forceinline__ f4 mfma(w4 a, w4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                   __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// c + a b over one half (16 of the reduction) of an operand.
__device__ __forceinline__ f4 mfma(w2 a, w2 b, f4 c) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s4, a),
                                                     __builtin_bit_cast(s4, b), c, 0, 0, 0);
}
// c + a b in six products, the smallest first; several such sums are formed
// product by product, since a product that waits for the one before it takes 21
// cycles instead of 16. part_a, part_b: the parts of product i.
constexpr int part_a(int i) {
    constexpr int a[] = {2, 0, 1, 1, 0, 0};
    return a[i];
}
constexpr int part_b(int i) {
    constexpr int b[] = {0, 2, 1, 0, 1, 0};
    return b[i];
}
template <int CT, class A, class B>
__device__ __forceinline__ void mul_columns(const A &a, const B (&b)[CT], f4 (&c)[CT]) {
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) c[ct] = mfma(a.p[part_a(i)], b[ct].p[part_b(i)], c[ct]);
}

// Shapes the schedule of the code around it: N times one matrix instruction
// followed by up to V vector instructions, which run in its shadow.
template <int N, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
        __builtin_amdgcn_sched_group_barrier(0x002, V, 0);  // vector
    }
}

// Two registers of 16-bit values, transposed among 16 lanes (see its use).
__device__ __forceinline__ w2 read_transposed(const char *p) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 *Lds;
    return __builtin_bit_cast(w2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                      (Lds)(__attribute__((address_space(3))) char *)p));
}

// Barrier among the wavefronts that add to `count`, which starts at zero; `sum`
// is what it holds once all of them have come here. (s_barrier takes the whole
// workgroup.) All of a workgroup's wavefronts are resident, so the wait ends.
__device__ __forceinline__ void meet(int *count, int sum) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    if ((threadIdx.x & (kWave - 1)) == 0)
        __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    while (__builtin_amdgcn_readfirstlane(__hip_atomic_load(
               count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) < sum)
        __builtin_amdgcn_s_sleep(1);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// N adjacent elements of one row as loaded (no conversion).
template <class E, int N>
struct RawC;
template <class E>
struct RawC<E, 4> {
    w2 w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(w2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
    __device__ __forceinline__ f4 all() const {
        return f4{Elem<E>::widen(w[0] & 0xFFFFu), Elem<E>::widen(w[0] >> 16),
                  Elem<E>::widen(w[1] & 0xFFFFu), Elem<E>::widen(w[1] >> 16)};
    }
};
template <>
struct RawC<F32, 4> {
    f4 w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    }
    __device__ __forceinline__ f4 all() const { return w; }
};
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
    uint16_t w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    }
    __device__ __forceinline__ float at(int) const { return Elem<E>::widen(w); }
};
template <>
struct RawC<F32, 1> {
    float w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    }
    __device__ __forceinline__ float at(int) const { return w; }
};
template <>
struct RawC<F32, 2> {
    f2 w;
    __device__ __forceinline__ void load(Rsrc r, uint32_t off) {
        w = __builtin_bit_cast(f2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
    __device__ __forceinline__ float at(int i) const { return w[i]; }
};

__device__ __forceinline__ f4 exp2(f4 x) {
    return f4{__builtin_amdgcn_exp2f(x[0]), __builtin_amdgcn_exp2f(x[1]),
              __builtin_amdgcn_exp2f(x[2]), __builtin_amdgcn_exp2f(x[3])};
}
// Powers of two in units of 2^-24, as integers: sums of them are exact.
typedef int i4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i4 fixed(f4 x, float unit) {
    return i4{(int)__builtin_rintf(x[0] * unit), (int)__builtin_rintf(x[1] * unit),
              (int)__builtin_rintf(x[2] * unit), (int)__builtin_rintf(x[3] * unit)};
}
// 2^(x 2^-24) for |x| < 125 2^24: 2^(1 + fraction), its exponent moved by the
// integer part less one.
__device__ __forceinline__ f4 exp2(i4 x) {
    f4 e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = x[i] >> 1;
        const float y = __builtin_amdgcn_exp2f(
            __builtin_bit_cast(float, (s & 0x7FFFFF) | 0x3F800000));
        e[i] = __builtin_bit_cast(float, __builtin_bit_cast(int, y) + (s & (int)0xFF800000) -
                                             0x800000);
    }
    return e;
}
__device__ __forceinline__ f4 rcp(f4 x) {
    return f4{__builtin_amdgcn_rcpf(x[0]), __builtin_amdgcn_rcpf(x[1]),
              __builtin_amdgcn_rcpf(x[2]), __builtin_amdgcn_rcpf(x[3])};
}
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }
// The largest magnitude, or NaN where there is one.
__device__ __forceinline__ float largest(float a, f4 x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) a = __builtin_elementwise_maximum(a, __builtin_fabsf(x[e]));
    return a;
}
// out[g] = x of the lane at the same place in group g, G groups of 64 / G lanes.
template <int G>
__device__ __forceinline__ void gather_groups(f4 x, f4 (&out)[G]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = x[e], b = x[e];
        lane_swap32(a, b);
        if constexpr (G == 2) {
            out[0][e] = a;
            out[1][e] = b;
        } else {
            float a1 = a, b1 = b;
            lane_swap16(a, a1);
            lane_swap16(b, b1);
            out[0][e] = a;
            out[1][e] = a1;
            out[2][e] = b;
            out[3][e] = b1;
        }
    }
}

// LDS layout (bytes). Operands lie in rows of 2 K bytes (reduced over
// channels) or of 32 and 64 bytes (over 16 and 32 tokens); the 16-byte pieces
// of a row are exchanged by an exclusive or with the row number so that the 16
// rows of one operand read, and the 4 rows of 4 adjacent pieces of a transposed
// one, fall in different banks without padding.
// N: chunks whose operands are held at once.
template <int K, int N>
struct PreLds {
    static constexpr int RS = 2 * K, TS = 2 * kPreC;
    static constexpr int kPatch = 20;  // floats between rows of a block of L
    static constexpr int R32 = kPreC * RS;
    // Three parts of the queries do not fit beside those of the keys with K =
    // 128: they lie there in FP32, in the room of two parts, and are split by
    // the wavefronts that read them.
    static constexpr bool kSplitLate = K == 128;
    static constexpr int kRawQ = kSplitLate ? 2 : kParts;  // pieces of a queries' operand
    // N chunks' operands, each:
    // keys and queries times e^{G - m} (steep: e^G), keys times e^{m - G}
    // (steep: e^{G_32 - G})
    static constexpr int KR = 0, QR = KR + kParts * R32, KL = QR + kRawQ * R32;
    static constexpr int kOperands = KL + kParts * R32;
    // a steep chunk's first half: keys, queries, decays FP32, then L / beta and P
    static constexpr int SK = 0, SQ = SK + kPreC * K * 4, SA = SQ + kPreC * K * 4;
    static constexpr int SM = SA + kPreC * K * 4, SP = SM + kPreC * kPreC * 4;
    // (and each wavefront's first token that is not finite)
    static constexpr int STOP = SP + kPreC * kPreC * 4, kSteepBytes = STOP + kPreWaves * 4;
    // a lower triangle of 32 x 32: the block of rows 0..15 (16 tokens), then
    // rows 16..31 (32 tokens)
    static constexpr int LOW = 16 * TS / 2, T32 = LOW + 16 * TS;
    // diagonal blocks of the inverse and -L_10; P
    static constexpr int TM = kOperands > kSteepBytes ? kOperands : kSteepBytes;
    static constexpr int PM = TM + kParts * T32;
    static constexpr int kBuffer = PM + kParts * T32;
    static_assert(kBuffer % 256 == 0);
    // per channel: what S' is of the state in registers (steep: 1), what that
    // state owes (see `apart`), and for a steep chunk e^{G_32}; N chunks'
    static constexpr int FACTORS = N * kBuffer, kFactors = 3 * K * 4;
    static constexpr int EM = 0, EG = K * 4, EF = 2 * K * 4;
    static constexpr int TOT = FACTORS + N * kFactors, kTot = kPreWaves * K * 4;
    static constexpr int PATCH = TOT + N * kTot;
    static constexpr int BETA = PATCH + 2 * 16 * kPatch * 4;
    static constexpr int FLAGS = BETA + N * kPreC * 4;
    static constexpr int kBytes = FLAGS + 16;
    // exchange of 16-byte pieces
    static __device__ __forceinline__ int swz_row(int row) {
        // bits 1, 0 of the row move it by 4 pieces, bits 2, 3 within them; (K =
        // 64: two rows to a line, bit 0 picks the half)
        const int low = ((row >> 2 ^ row >> 3) & 1) * 2 + (row >> 3 & 1);
        const int high = K == 128 ? (row >> 1 & 1) * 2 + (row & 1) : row >> 1 & 1;
        return (high * 4 + low) << 4;
    }
    static __device__ __forceinline__ int swz_tok(int row) { return ((row >> 2) & 3) << 4; }
    // 16 rows of the queries' operand as loaded: its parts, or the two halves of
    // this lane's eight FP32 values.
    struct Queries {
        w4 p[kRawQ];
        __device__ __forceinline__ Operand parts() const {
            if constexpr (kSplitLate)
                return join(split4(__builtin_bit_cast(f4, p[0])),
                            split4(__builtin_bit_cast(f4, p[1])));
            else
                return Operand{p[0], p[1], p[kRawQ - 1]};
        }
    };
};

// x = (I + L)^-1, one lane per column of a 16 x 16 block in every 16-lane row:
// lane i of the row holds row i of -L in a (0 on and above the diagonal), x
// starts as the identity's column, and once x_j is final every x_i below takes
// a_ij x_j, with a_ij read from lane i by a DPP broadcast inside the
// multiply-add (the compiler spends a move on each). The updates of one j do
// not depend on each other. The DPP source must not have been written by the
// two instructions before: s_nop 1.
#define KDA_FMAC(i, o, a, x) \
    "v_fmac_f32_dpp %" #o ", %" #a ", %" #x " row_newbcast:" #i " row_mask:0xf bank_mask:0xf\n\t"
__device__ __forceinline__ void substitute(const float (&a)[16], float (&x)[16]) {
    asm("s_nop 1\n\t"
        KDA_FMAC(1, 0, 15, 16) KDA_FMAC(2, 1, 15, 16) KDA_FMAC(3, 2, 15, 16)
        KDA_FMAC(4, 3, 15, 16) KDA_FMAC(5, 4, 15, 16) KDA_FMAC(6, 5, 15, 16)
        KDA_FMAC(7, 6, 15, 16) KDA_FMAC(8, 7, 15, 16) KDA_FMAC(9, 8, 15, 16)
        KDA_FMAC(10, 9, 15, 16) KDA_FMAC(11, 10, 15, 16) KDA_FMAC(12, 11, 15, 16)
        KDA_FMAC(13, 12, 15, 16) KDA_FMAC(14, 13, 15, 16) KDA_FMAC(15, 14, 15, 16)
        : "+v"(x[1]), "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]),
          "+v"(x[6]), "+v"(x[7]), "+v"(x[8]), "+v"(x[9]), "+v"(x[10]),
          "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[0]), "v"(x[0]));
    asm("s_nop 1\n\t"
        KDA_FMAC(2, 0, 14, 15) KDA_FMAC(3, 1, 14, 15) KDA_FMAC(4, 2, 14, 15)
        KDA_FMAC(5, 3, 14, 15) KDA_FMAC(6, 4, 14, 15) KDA_FMAC(7, 5, 14, 15)
        KDA_FMAC(8, 6, 14, 15) KDA_FMAC(9, 7, 14, 15) KDA_FMAC(10, 8, 14, 15)
        KDA_FMAC(11, 9, 14, 15) KDA_FMAC(12, 10, 14, 15) KDA_FMAC(13, 11, 14, 15)
        KDA_FMAC(14, 12, 14, 15) KDA_FMAC(15, 13, 14, 15)
        : "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]), "+v"(x[6]),
          "+v"(x[7]), "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]),
          "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[1]), "v"(x[1]));
    asm("s_nop 1\n\t"
        KDA_FMAC(3, 0, 13, 14) KDA_FMAC(4, 1, 13, 14) KDA_FMAC(5, 2, 13, 14)
        KDA_FMAC(6, 3, 13, 14) KDA_FMAC(7, 4, 13, 14) KDA_FMAC(8, 5, 13, 14)
        KDA_FMAC(9, 6, 13, 14) KDA_FMAC(10, 7, 13, 14) KDA_FMAC(11, 8, 13, 14)
        KDA_FMAC(12, 9, 13, 14) KDA_FMAC(13, 10, 13, 14) KDA_FMAC(14, 11, 13, 14)
        KDA_FMAC(15, 12, 13, 14)
        : "+v"(x[3]), "+v"(x[4]), "+v"(x[5]), "+v"(x[6]), "+v"(x[7]),
          "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]), "+v"(x[12]),
          "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[2]), "v"(x[2]));
    asm("s_nop 1\n\t"
        KDA_FMAC(4, 0, 12, 13) KDA_FMAC(5, 1, 12, 13) KDA_FMAC(6, 2, 12, 13)
        KDA_FMAC(7, 3, 12, 13) KDA_FMAC(8, 4, 12, 13) KDA_FMAC(9, 5, 12, 13)
        KDA_FMAC(10, 6, 12, 13) KDA_FMAC(11, 7, 12, 13) KDA_FMAC(12, 8, 12, 13)
        KDA_FMAC(13, 9, 12, 13) KDA_FMAC(14, 10, 12, 13) KDA_FMAC(15, 11, 12, 13)
        : "+v"(x[4]), "+v"(x[5]), "+v"(x[6]), "+v"(x[7]), "+v"(x[8]),
          "+v"(x[9]), "+v"(x[10]), "+v"(x[11]), "+v"(x[12]), "+v"(x[13]),
          "+v"(x[14]), "+v"(x[15])
        : "v"(a[3]), "v"(x[3]));
    asm("s_nop 1\n\t"
        KDA_FMAC(5, 0, 11, 12) KDA_FMAC(6, 1, 11, 12) KDA_FMAC(7, 2, 11, 12)
        KDA_FMAC(8, 3, 11, 12) KDA_FMAC(9, 4, 11, 12) KDA_FMAC(10, 5, 11, 12)
        KDA_FMAC(11, 6, 11, 12) KDA_FMAC(12, 7, 11, 12) KDA_FMAC(13, 8, 11, 12)
        KDA_FMAC(14, 9, 11, 12) KDA_FMAC(15, 10, 11, 12)
        : "+v"(x[5]), "+v"(x[6]), "+v"(x[7]), "+v"(x[8]), "+v"(x[9]),
          "+v"(x[10]), "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]),
          "+v"(x[15])
        : "v"(a[4]), "v"(x[4]));
    asm("s_nop 1\n\t"
        KDA_FMAC(6, 0, 10, 11) KDA_FMAC(7, 1, 10, 11) KDA_FMAC(8, 2, 10, 11)
        KDA_FMAC(9, 3, 10, 11) KDA_FMAC(10, 4, 10, 11) KDA_FMAC(11, 5, 10, 11)
        KDA_FMAC(12, 6, 10, 11) KDA_FMAC(13, 7, 10, 11) KDA_FMAC(14, 8, 10, 11)
        KDA_FMAC(15, 9, 10, 11)
        : "+v"(x[6]), "+v"(x[7]), "+v"(x[8]), "+v"(x[9]), "+v"(x[10]),
          "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[5]), "v"(x[5]));
    asm("s_nop 1\n\t"
        KDA_FMAC(7, 0, 9, 10) KDA_FMAC(8, 1, 9, 10) KDA_FMAC(9, 2, 9, 10)
        KDA_FMAC(10, 3, 9, 10) KDA_FMAC(11, 4, 9, 10) KDA_FMAC(12, 5, 9, 10)
        KDA_FMAC(13, 6, 9, 10) KDA_FMAC(14, 7, 9, 10) KDA_FMAC(15, 8, 9, 10)
        : "+v"(x[7]), "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]),
          "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[6]), "v"(x[6]));
    asm("s_nop 1\n\t"
        KDA_FMAC(8, 0, 8, 9) KDA_FMAC(9, 1, 8, 9) KDA_FMAC(10, 2, 8, 9)
        KDA_FMAC(11, 3, 8, 9) KDA_FMAC(12, 4, 8, 9) KDA_FMAC(13, 5, 8, 9)
        KDA_FMAC(14, 6, 8, 9) KDA_FMAC(15, 7, 8, 9)
        : "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]), "+v"(x[12]),
          "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[7]), "v"(x[7]));
    asm("s_nop 1\n\t"
        KDA_FMAC(9, 0, 7, 8) KDA_FMAC(10, 1, 7, 8) KDA_FMAC(11, 2, 7, 8)
        KDA_FMAC(12, 3, 7, 8) KDA_FMAC(13, 4, 7, 8) KDA_FMAC(14, 5, 7, 8)
        KDA_FMAC(15, 6, 7, 8)
        : "+v"(x[9]), "+v"(x[10]), "+v"(x[11]), "+v"(x[12]), "+v"(x[13]),
          "+v"(x[14]), "+v"(x[15])
        : "v"(a[8]), "v"(x[8]));
    asm("s_nop 1\n\t"
        KDA_FMAC(10, 0, 6, 7) KDA_FMAC(11, 1, 6, 7) KDA_FMAC(12, 2, 6, 7)
        KDA_FMAC(13, 3, 6, 7) KDA_FMAC(14, 4, 6, 7) KDA_FMAC(15, 5, 6, 7)
        : "+v"(x[10]), "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]),
          "+v"(x[15])
        : "v"(a[9]), "v"(x[9]));
    asm("s_nop 1\n\t"
        KDA_FMAC(11, 0, 5, 6) KDA_FMAC(12, 1, 5, 6) KDA_FMAC(13, 2, 5, 6)
        KDA_FMAC(14, 3, 5, 6) KDA_FMAC(15, 4, 5, 6)
        : "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[10]), "v"(x[10]));
    asm("s_nop 1\n\t"
        KDA_FMAC(12, 0, 4, 5) KDA_FMAC(13, 1, 4, 5) KDA_FMAC(14, 2, 4, 5)
        KDA_FMAC(15, 3, 4, 5)
        : "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[11]), "v"(x[11]));
    asm("s_nop 1\n\t"
        KDA_FMAC(13, 0, 3, 4) KDA_FMAC(14, 1, 3, 4) KDA_FMAC(15, 2, 3, 4)
        : "+v"(x[13]), "+v"(x[14]), "+v"(x[15])
        : "v"(a[12]), "v"(x[12]));
    asm("s_nop 1\n\t"
        KDA_FMAC(14, 0, 2, 3) KDA_FMAC(15, 1, 2, 3)
        : "+v"(x[14]), "+v"(x[15])
        : "v"(a[13]), "v"(x[13]));
    asm("s_nop 1\n\t"
        KDA_FMAC(15, 0, 1, 2)
        : "+v"(x[15])
        : "v"(a[14]), "v"(x[14]));
}
#undef KDA_FMAC

// Segment j of all requests' segments in order (every wavefront finds it by
// itself; at most kWave requests). A request without tokens has one segment.
// Segments past `segs`, which only a malformed cu_seqlens can have, do not
// exist.
constexpr int kMaxCutRequests = kWave;
struct Segment {
    int request, first, count, at;  // segments [first, first + count) of the request; at < count
};
__device__ __forceinline__ int lane_prefix(int x) {  // inclusive sum over the wavefront
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int y = __shfl_up(x, d, kWave);
        if (lane >= d) x += y;
    }
    return x;
}
__device__ __forceinline__ int segments_to_lane(const DeltaProblem &p, int &own) {
    const int lane = threadIdx.x & (kWave - 1);
    own = 0;
    if (lane < p.req.num_seqs) own = 1 + max(request_rows(p.req, lane).y - 1, 0) / p.seg;
    return lane_prefix(own);
}
__device__ __forceinline__ Segment find_segment(const DeltaProblem &p, int j) {
    int own;
    const int upto = segments_to_lane(p, own);
    const uint64_t past = __ballot(upto > j);
    if (past == 0) return Segment{-1, 0, 0, 0};
    const int n = __builtin_ctzll(past);
    Segment s;
    s.request = n;
    s.count = __builtin_amdgcn_readlane(own, n);
    s.first = __builtin_amdgcn_readlane(upto, n) - s.count;
    s.at = j - s.first;
    return s;
}

// SUM: instead of outputs, what the segments but every request's last one do
// to the state, S_after = M S_before + B, as the columns [B | M] of a V + K
// columns wide state: B starts from zero (a first segment's from the request's
// state, and then is S_after), M from the identity and with V = 0.
// ROLES: four wavefronts prepare the next chunk while others (kCols) take their
// columns of this one through it; else four wavefronts do both in turn.
// CT: tiles of 16 columns to a wavefront.
enum class PrePass { whole, roles, narrow, sums };
template <bool SUM, bool ROLES, int CT>
struct PreShape {
    static constexpr int kCols = SUM ? 8 : 4;  // wavefronts with columns
    static constexpr int kWidth = kCols * 16 * CT;  // columns of a workgroup
    static constexpr int kThreads = kWave * (ROLES ? kCols + kPreWaves : kCols);
    // wavefronts, by their registers (three of whole K = 64: 16 x 512 tokens, 64
    // heads, V = 64, 205 -> 197 us)
    static constexpr int per_simd(int K) { return SUM || (K == 64 && !ROLES && CT == 1) ? 3 : 2; }
    static_assert(ROLES || kCols == kPreWaves);
};
template <class EI, int K, int OUT, bool SUM, bool ROLES, int CT>
__global__
__launch_bounds__((PreShape<SUM, ROLES, CT>::kThreads), (PreShape<SUM, ROLES, CT>::per_simd(K)))
void kda_prefill_kernel(DeltaProblem p) {
    typedef PreLds<K, ROLES ? 2 : 1> L;
    typedef PreShape<SUM, ROLES, CT> Shape;
    constexpr int CW = Shape::kCols;
    constexpr int NT = K / 16;  // state row tiles
    // A wavefront prepares 8 tokens: K / 4 lanes of 4 channels to a token, in
    // GRP groups of lanes with TPL tokens each.
    constexpr int GRP = 4 * kWave / K, TPL = 8 / GRP;
    constexpr int OE = OUT == 0 ? 4 : 2;  // bytes of an output element
    __shared__ __align__(16) char lds[L::kBytes];

    const int lane0 = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool prepares = !ROLES || wv >= CW, walks = !ROLES || wv < CW;
    const int pw = ROLES ? wv - CW : wv;  // a preparing wavefront's number
    const int j = blockIdx.x / p.H, h = blockIdx.x - j * p.H;
    Segment sg = {j, j, 1, 0};
    if (p.seg != 0) {
        sg = find_segment(p, j);
        if (sg.request < 0 || (SUM && sg.at + 1 == sg.count)) return;
        if (SUM && sg.at == 0 && (int)(blockIdx.y * Shape::kWidth) >= p.V) return;
    }
    const int n = sg.request;
    const int hk = h / (p.H / p.Hk);
    const int2 rows = request_rows(p.req, n);
    const int skip = sg.at * p.seg;  // the request's tokens before the segment
    const int len_all = __builtin_amdgcn_readfirstlane(
        sg.at + 1 < sg.count ? p.seg : rows.y - skip);
    const long row_first = __builtin_amdgcn_readfirstlane(rows.x + skip);
    const bool keep = p.pool.base != nullptr;
    const int slot = __builtin_amdgcn_readfirstlane(keep ? request_slot(p.pool, n) : 0);

    // this wavefront's columns: tile ct holds column col + ct of each lane
    const int col0 = (blockIdx.y * CW + wv) * 16 * CT;
    const bool map = SUM && col0 >= p.V;  // V is a multiple of 32
    const bool cols = walks && (SUM ? col0 < p.V + (sg.at ? K : 0) : col0 < p.V);
    const int col = (cols ? map ? col0 - p.V : col0 : 0) + CT * (lane0 & 15);

    // Token tensors from the request's first row and this head on, and the
    // bytes between their rows (at most 2^22: 32 rows' offsets fit 32 bits).
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
    auto put_out = [&](Rsrc r, uint32_t off, const f4 (&o)[CT], int s) {
        if constexpr (OUT == 0 && CT == 2)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(w2, f2{o[0][s], o[1][s]}), r,
                                                  off, 0, kNontemporal);
        else if constexpr (OUT == 0)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)o[0][s]), r,
                                                  off, 0, kNontemporal);
        else {
            const float a = o[0][s], b = o[CT - 1][s];
            const uint32_t w = OUT == 1 ? Elem<BF16>::pack(a, b) : Elem<F16>::pack(a, b);
            if constexpr (CT == 2)
                __builtin_amdgcn_raw_buffer_store_b32(w, r, off, 0, kNontemporal);
            else
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w, r, off, 0, kNontemporal);
        }
    };
    if (slot < 0) {  // padding: zero outputs, no state
        if (!SUM && cols)
            for (int t = lane0 >> 4; t < len_all; t += 4)
#pragma unroll
                for (int c = 0; c < CT * OE; c += 2)
                    *reinterpret_cast<uint16_t *>(ob + (long)t * os + col * OE + c) = 0;
        return;
    }

    // the state: lane group g4's rows of tile rt are channels
    // 32 (rt / 2) + 8 g4 + 4 (rt % 2) + s
    auto state_row = [](int rt, int s) { return 32 * (rt >> 1) + 4 * (rt & 1) + s; };
    // ======== preparing a chunk: 8 tokens to a wavefront
    // this wavefront's tokens as loaded and (wavefront 3) the chunk's write
    // strengths
    struct Rows {
        RawC<EI, 4> k[TPL], q[TPL];
        f4 g[TPL];
        float beta;
    };
    Rows now;
    now.beta = 0.0f;
    auto load_rows = [&](int t0, Rows &to) {
        const int len = min(kPreC, len_all - t0);
        const Rsrc rk = rows_of(kb + (long)t0 * ks, ks, K * EI::kBytes, len);
        const Rsrc rq = rows_of(qb + (long)t0 * ks, ks, K * EI::kBytes, len);
        const Rsrc rg = rows_of(gb + (long)t0 * gs, gs, gd * 4, len);
        const int lane = opaque_lane(lane0);
        const uint32_t first = 8 * pw + lane / (K / 4) * TPL, c4 = lane % (K / 4) * 4;
        if (gd == 1) {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const float x = load1<F32>(rg, (first + i) * gs);
                to.g[i] = f4{x, x, x, x};
            }
        } else {
#pragma unroll
            for (int i = 0; i < TPL; ++i) to.g[i] = load4<F32>(rg, (first + i) * gs + c4 * 4);
        }
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
            to.k[i].load(rk, (first + i) * ks + c4 * EI::kBytes);
            if constexpr (!SUM) to.q[i].load(rq, (first + i) * ks + c4 * EI::kBytes);
        }
        if (pw == 3)
            to.beta = lane < len ? p.beta[(row_first + t0 + lane) * p.H + h] : 0.0f;
    };
    // Decays of a lane's tokens, summed from its wavefront's first token on,
    // and the totals of the wavefront's groups of lanes.
    f4 er[TPL], sums[GRP];
    auto sum_decays = [&](int buf) {
        const int lane = opaque_lane(lane0), grp = lane / (K / 4), ch = lane % (K / 4) * 4;
        float *tots = reinterpret_cast<float *>(lds + L::TOT + buf * L::kTot);
        {
            f4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __builtin_fmaf(now.g[i][e], kLog2E, x[e]);
                er[i] = x;
            }
            // a key or write strength that is not finite shows in the totals
            // (and the chunk takes the steep path, which looks for its token)
            float most = pw == 3 ? __builtin_fabsf(now.beta) : 0.0f;
#pragma unroll
            for (int i = 0; i < TPL; ++i) most = largest(most, now.k[i].all());
            x[0] = __builtin_fmaf(most, 0.0f, x[0]);
            gather_groups<GRP>(x, sums);
            f4 all = sums[0];
#pragma unroll
            for (int g = 1; g < GRP; ++g) all += sums[g];
            if (grp == 0) *reinterpret_cast<f4 *>(tots + pw * K + ch) = all;
        }
        if (pw == 3 && lane < kPreC)
            reinterpret_cast<float *>(lds + L::BETA)[buf * kPreC + lane] = now.beta;
    };
    // the decay (of this lane's channels, a power of two) that the state in
    // registers still has to take: G_32 - m of the chunk before
    f4 owed = {0.0f, 0.0f, 0.0f, 0.0f};
    i4 owed_i = {0, 0, 0, 0};  // (in fixed point; the first wavefront's)
    // a barrier of the preparing wavefronts
    int *count = reinterpret_cast<int *>(lds + L::FLAGS) + 2, met = 0;
    auto meet_all = [&] {
        if constexpr (ROLES)
            meet(count, met += kPreWaves);
        else
            __syncthreads();
    };
    // What the chunk at t0 puts into buffer `buf`, from its loaded rows and the
    // wavefronts' totals; far, apart: see there; stop: the first token with a
    // key, decay or write strength that is not finite.
    auto prepare = [&](int buf, bool &far, bool &apart, int &stop) {
        // the lane made opaque: the many addresses derived from it are formed
        // where they are used instead of being kept (and spilled) across chunks
        const int lane = opaque_lane(lane0);
        const int g4 = lane >> 4, n16 = lane & 15;
        // this lane's group, channels and first token of the wavefront's 8
        const int grp = lane / (K / 4), ch = lane % (K / 4) * 4, tok = 8 * pw + TPL * grp;
        char *op = lds + buf * L::kBuffer, *fac = lds + L::FACTORS + buf * L::kFactors;
        const float *tots = reinterpret_cast<const float *>(lds + L::TOT + buf * L::kTot);
        const float *beta = reinterpret_cast<const float *>(lds + L::BETA) + buf * kPreC;

        auto put_row = [&](int at, int row, f4 x) {
            char *d = op + at + row * L::RS + ((2 * ch) ^ L::swz_row(row));
            const Half hx = split4(x);
#pragma unroll
            for (int i = 0; i < kParts; ++i) *reinterpret_cast<w2 *>(d + i * L::R32) = hx.p[i];
        };
        auto put_query = [&](int row, f4 x) {
            if constexpr (L::kSplitLate)  // channels 8 i + 4 e .. + 3 to the half e
                *reinterpret_cast<f4 *>(op + L::QR + (ch >> 2 & 1) * L::R32 + row * L::RS +
                                        ((2 * (ch & ~7)) ^ L::swz_row(row))) = x;
            else
                put_row(L::QR, row, x);
        };
        // entries (row, c) and (row + 1, c), row even, of an operand reduced
        // over tokens; low: rows 16..31
        auto put_pair = [&](int at, bool low, int row, int c, float x, float y) {
            char *d = op + at + (low ? L::LOW + row * L::TS +
                                           ((2 * operand_pos(c)) ^ L::swz_tok(row))
                                     : row * (L::TS / 2) + 2 * c);
            uint32_t part[kParts];
            split2(x, y, part);
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                *reinterpret_cast<uint16_t *>(d + i * L::T32) = (uint16_t)part[i];
                *reinterpret_cast<uint16_t *>(d + i * L::T32 + (low ? L::TS : L::TS / 2)) =
                    (uint16_t)(part[i] >> 16);
            }
        };
        // ---- 1. the operands reduced over channels
        f4 wt[kPreWaves];  // every wavefront's 8 tokens
#pragma unroll
        for (int w = 0; w < kPreWaves; ++w)
            wt[w] = *reinterpret_cast<const f4 *>(tots + w * K + ch);
        const f4 first = wt[0] + wt[1], second = wt[2] + wt[3];  // m, G_32 - m
        const f4 both = owed + first;
        bool steep = false, deep = false, wide = false;  // (steep: also where not finite)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            steep |= !(__builtin_fabsf(first[e]) <= kSteep) |
                     !(__builtin_fabsf(second[e]) <= kSteep);
            deep |= __builtin_fabsf(both[e]) > 124.0f;
            wide |= !(__builtin_fabsf(first[e]) <= kFine) | !(__builtin_fabsf(second[e]) <= kFine);
        }
        far = __ballot(steep) != 0;  // the same in every wavefront
        apart = far | (__ballot(deep) != 0);
        stop = kPreC;
        // m and G_32 - m in fixed point (the first wavefront's)
        i4 first_i = {0, 0, 0, 0}, second_i = first_i;
        // the factor of token i of this lane's: keys, queries and their inverse
        auto put_token = [&](int i, f4 e) {
            const f4 k = now.k[i].all();
            put_row(L::KR, tok + i, k * e);
            if constexpr (!SUM) put_query(tok + i, now.q[i].all() * (e * p.scale));
            put_row(L::KL, tok + i, k * rcp(e));
        };
        // from the chunk's middle to this lane's first token, of the wavefronts'
        // totals and this one's groups
        auto from_middle = [&](const auto &w, const auto &own) {
            auto mid = w[0] - w[0];
            if (pw >= 2) {
                if (pw == 3) mid = w[2];
#pragma unroll
                for (int g = 0; g + 1 < GRP; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (g < grp) mid[e] += own[g][e];
            } else {
                mid = -own[GRP - 1];
                if (pw == 0) mid -= w[1];
#pragma unroll
                for (int g = 0; g + 1 < GRP; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (g >= grp) mid[e] -= own[g][e];
            }
            return mid;
        };
        if (!far && __ballot(wide) == 0) {
            if (pw == 0) {
                first_i = fixed(first, kFixed);
                second_i = fixed(second, kFixed);
            }
            const f4 mid = from_middle(wt, sums);
#pragma unroll
            for (int i = 0; i < TPL; ++i) put_token(i, exp2(er[i] + mid));
        } else if (!far) {
            // Far from the middle the FP32 sums of steep decays keep too few bits
            // of a power of two (2^-17 of 2^74), and adjacent tokens would lose
            // them: the sums once more in fixed point, where they are exact.
            i4 x = {0, 0, 0, 0}, ei[TPL], own[GRP], wi[kPreWaves];
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                x += fixed(now.g[i], kLog2E * kFixed);
                ei[i] = x;
            }
            f4 parts[GRP];
            gather_groups<GRP>(__builtin_bit_cast(f4, x), parts);
            i4 all = {0, 0, 0, 0};
#pragma unroll
            for (int g = 0; g < GRP; ++g) {
                own[g] = __builtin_bit_cast(i4, parts[g]);
                all += own[g];
            }
            // (the inverse's place: written after the next barrier)
            int *totals = reinterpret_cast<int *>(op + L::TM);
            if (grp == 0) *reinterpret_cast<i4 *>(totals + pw * K + ch) = all;
            meet_all();
#pragma unroll
            for (int w = 0; w < kPreWaves; ++w)
                wi[w] = *reinterpret_cast<const i4 *>(totals + w * K + ch);
            first_i = wi[0] + wi[1];
            second_i = wi[2] + wi[3];
            const i4 mid = from_middle(wi, own);
#pragma unroll
            for (int i = 0; i < TPL; ++i) put_token(i, exp2(ei[i] + mid));
        } else {
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const int at = 4 * ((tok + i) * K + ch);
                *reinterpret_cast<f4 *>(op + L::SK + at) = now.k[i].all();
                if constexpr (!SUM)
                    *reinterpret_cast<f4 *>(op + L::SQ + at) = now.q[i].all() * p.scale;
                *reinterpret_cast<f4 *>(op + L::SA + at) = exp2(now.g[i] * kLog2E);
            }
            int mine = pw == 3 && lane < kPreC && !finite(now.beta) ? lane : kPreC;
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                const f4 k = now.k[i].all();
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    bad |= !finite(k[e]) | !(now.g[i][e] < __builtin_inff());
                mine = min(mine, bad ? tok + i : kPreC);
            }
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) mine = min(mine, __shfl_xor(mine, d));
            reinterpret_cast<int *>(op + L::STOP)[pw] = mine;
        }
        if (pw == 0 && grp == 0) {
            const f4 one = {1.0f, 1.0f, 1.0f, 1.0f};
            *reinterpret_cast<f4 *>(fac + L::EM + 4 * ch) =
                far ? one : exp2(apart ? first_i : owed_i + first_i);
            *reinterpret_cast<f4 *>(fac + L::EG + 4 * ch) = exp2(owed_i);
            *reinterpret_cast<f4 *>(fac + L::EF + 4 * ch) = exp2(first + second);
        }
        if (ROLES && pw == 0 && lane0 == 0 && !far)  // (else below)
            reinterpret_cast<int *>(lds + L::FLAGS)[buf] = (apart ? 2 : 0) | kPreC << 2;
        owed = far ? f4{0.0f, 0.0f, 0.0f, 0.0f} : second;
        owed_i = far ? i4{0, 0, 0, 0} : second_i;
        meet_all();

        const int rpos = n16 * L::RS + ((g4 << 4) ^ L::swz_row(n16));
        // 16 rows of an operand reduced over channels, k-step kk
        auto row_operand = [&]<class O>(int at, int kk) -> O {
            O o;
#pragma unroll
            for (int i = 0; i < (int)(sizeof(O) / sizeof(w4)); ++i)
                o.p[i] = *reinterpret_cast<const w4 *>(op + at + i * L::R32 + (rpos ^ (64 * kk)));
            return o;
        };
        // ---- 2. 16 x 16 blocks of L / beta and P: wavefronts 0 and 1 a
        // diagonal block of L each (and its inverse), 2 those of P, 3 the two
        // blocks below
        f4 m[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        if (!far) {
            // rows 16 bi .. of the keys or queries against rows 16 bj .. of the keys
            auto block = [&]<bool Q>(int bi, int bj) -> f4 {
                f4 c[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
                for (int kk = 0; kk < K / 32; kk += 2) {
                    Operand l[2], r[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if constexpr (Q)
                            l[e] = row_operand
                                       .template operator()<typename L::Queries>(
                                           L::QR + 16 * bi * L::RS, kk + e)
                                       .parts();
                        else
                            l[e] = row_operand.template operator()<Operand>(
                                L::KR + 16 * bi * L::RS, kk + e);
                        r[e] = row_operand.template operator()<Operand>(L::KL + 16 * bj * L::RS,
                                                                        kk + e);
                    }
#pragma unroll
                    for (int i = 0; i < 6; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            c[e] = mfma(l[e].p[part_a(i)], r[e].p[part_b(i)], c[e]);
                    // (all of them read ahead spill where the state is held, too)
                    if constexpr (!ROLES) __builtin_amdgcn_sched_barrier(0);
                }
                return c[0] + c[1];
            };
            if (pw < 2) {
                m[0] = block.template operator()<false>(pw, pw);
            } else if (pw == 3) {
                m[0] = block.template operator()<false>(1, 0);
                if constexpr (!SUM) m[1] = block.template operator()<true>(1, 0);
            } else if constexpr (!SUM) {
                m[0] = block.template operator()<true>(0, 0);
                m[1] = block.template operator()<true>(1, 1);
            }
        } else {
            // running products of the decays from token j on
            const float *sk = reinterpret_cast<const float *>(op + L::SK);
            const float *sq = reinterpret_cast<const float *>(op + L::SQ);
            const float *sa = reinterpret_cast<const float *>(op + L::SA);
            float *sm = reinterpret_cast<float *>(op + L::SM);
            float *sp = reinterpret_cast<float *>(op + L::SP);
            const int *stops = reinterpret_cast<const int *>(op + L::STOP);
            stop = __builtin_amdgcn_readfirstlane(
                min(min(stops[0], stops[1]), min(stops[2], stops[3])));
            if (pw == 3 && lane >= stop && lane < kPreC)
                reinterpret_cast<float *>(lds + L::BETA)[buf * kPreC + lane] = 0.0f;
            if (ROLES && pw == 0 && lane == 0)
                reinterpret_cast<int *>(lds + L::FLAGS)[buf] = 3 | stop << 2;
#pragma unroll 1
            for (int j = pw; j < kPreC; j += kPreWaves) {
                constexpr int CPL = K / kWave;  // channels per lane, 64 apart
                float f[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) f[c] = sk[j * K + lane + 64 * c];
#pragma unroll 1
                for (int i = j; i < kPreC; ++i) {
                    float a = 0.0f, b = 0.0f;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        const int at = i * K + lane + 64 * c;
                        if (i > j) f[c] *= sa[at];
                        a = __builtin_fmaf(f[c], sk[at], a);
                        if constexpr (!SUM) b = __builtin_fmaf(f[c], sq[at], b);
                    }
                    a = sum64(a);
                    if constexpr (!SUM) b = sum64(b);
                    if (lane == 0) {
                        sm[i * kPreC + j] = a;
                        sp[i * kPreC + j] = b;
                    }
                }
            }
            meet_all();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int top = (4 * g4 + s) * kPreC + n16, low = top + 16 * kPreC;
                // (L stops there, as if the tokens from there on were none)
                if (pw < 2) {
                    m[0][s] = 16 * pw + 4 * g4 + s < stop ? sm[pw == 0 ? top : low + 16] : 0.0f;
                }
                if (pw == 2) {
                    m[0][s] = sp[top];
                    m[1][s] = sp[low + 16];
                }
                if (pw == 3) {
                    m[0][s] = 16 + 4 * g4 + s < stop ? sm[low] : 0.0f;
                    m[1][s] = sp[low];
                }
            }
        }
        // the inverse's diagonal blocks times beta (of their column), -L_10 /
        // beta (of the row) and P, as A operands
        if (pw < 2) {
            float *patch = reinterpret_cast<float *>(lds + L::PATCH) + pw * 16 * L::kPatch;
            const f4 b4 = *reinterpret_cast<const f4 *>(beta + 16 * pw + 4 * g4);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 4 * g4 + s;
                patch[r * L::kPatch + n16] = n16 < r ? -b4[s] * m[0][s] : 0.0f;
            }
            float arow[16], x[16];  // every 16-lane row the same
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = j == n16 ? 1.0f : 0.0f;
            wave_sync();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 v = *reinterpret_cast<const f4 *>(&patch[n16 * L::kPatch + 4 * j]);
#pragma unroll
                for (int s = 0; s < 4; ++s) arow[4 * j + s] = v[s];
            }
            substitute(arow, x);
            const float bc = beta[16 * pw + n16];
            f4 y;  // rows 4 g4 .. + 3 (two opaque bits: selects, not a switch on g4)
            const bool odd = opaque_lane(g4 & 1), high = opaque_lane(g4 >> 1);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float a = odd ? x[4 + s] : x[s], b = odd ? x[12 + s] : x[8 + s];
                y[s] = (high ? b : a) * bc;
            }
#pragma unroll
            for (int s = 0; s < 4; s += 2)
                put_pair(L::TM, pw == 1, 4 * g4 + s, 16 * pw + n16, y[s],
                                                y[s + 1]);
        } else if (pw == 2) {
            if constexpr (!SUM)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int s = 0; s < 4; s += 2) {
                        const int r = 4 * g4 + s;
                        put_pair(L::PM, b == 1, r, 16 * b + n16,
                                                         n16 <= r ? m[b][s] : 0.0f,
                                                         n16 <= r + 1 ? m[b][s + 1] : 0.0f);
                    }
        } else {
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
                put_pair(L::TM, true, 4 * g4 + s, n16, -m[0][s],
                                                -m[0][s + 1]);
                if constexpr (!SUM)
                    put_pair(L::PM, true, 4 * g4 + s, n16, m[1][s],
                                                     m[1][s + 1]);
            }
        }
        if (far) {
            // k e^G, q e^G and k e^{G_32 - G} over the FP32 copies; sums from
            // the chunk's ends, so that no difference of large sums is taken
            // (formed anew from the loaded gates, through copies that the
            // compiler cannot tell from new values, so that nothing is held in
            // registers for this branch)
            f4 before = {0.0f, 0.0f, 0.0f, 0.0f}, after = before, g2[TPL], ends[GRP], x = before;
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float g = now.g[i][e];
                    asm("" : "+v"(g));
                    g2[i][e] = g * kLog2E;
                }
                x += g2[i];
            }
            gather_groups<GRP>(x, ends);
#pragma unroll 1
            for (int w = 0; w < kPreWaves; ++w) {
                const f4 y = *reinterpret_cast<const f4 *>(tots + w * K + ch);
                if (w < pw) before += y;
                if (w > pw) after += y;
            }
#pragma unroll
            for (int g = 0; g < GRP; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    before[e] += g < grp ? ends[g][e] : 0.0f;
                    after[e] += g > grp ? ends[g][e] : 0.0f;
                }
            meet_all();  // the copies (and L and P) have been read
#pragma unroll
            for (int i = 0; i < TPL; ++i) {
                before += g2[i];
                const f4 e = exp2(before);
                put_row(L::KR, tok + i, now.k[i].all() * e);
                if constexpr (!SUM) put_query(tok + i, now.q[i].all() * (e * p.scale));
            }
#pragma unroll
            for (int i = TPL - 1; i >= 0; --i) {
                put_row(L::KL, tok + i, now.k[i].all() * exp2(after));
                after += g2[i];
            }
        }
    };

    // ======== this wavefront's columns
    f4 S[NT][CT];
    // [K, V] of this head in slot `at` of a tensor [.., H, K, V], this lane's part
    auto state_at = [&](float *base, int at) {
        return base + (((long)at * p.H + h) * K + 8 * (lane0 >> 4)) * p.V + col;
    };
    auto load_state = [&](const float *src) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float *at = src + (long)state_row(rt, s) * p.V;
                if constexpr (CT == 2) {
                    const f2 v = __builtin_nontemporal_load(reinterpret_cast<const f2 *>(at));
                    S[rt][0][s] = v[0];
                    S[rt][1][s] = v[1];
                } else {
                    S[rt][0][s] = __builtin_nontemporal_load(at);
                }
            }
    };
    auto store_state = [&](float *dst, int stride) {
#pragma unroll
        for (int rt = 0; rt < NT; ++rt)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float *at = dst + (long)state_row(rt, s) * stride;
                if constexpr (CT == 2) {
                    const f2 v = {S[rt][0][s], S[rt][1][s]};
                    if (SUM)  // read next
                        *reinterpret_cast<f2 *>(at) = v;
                    else
                        __builtin_nontemporal_store(v, reinterpret_cast<f2 *>(at));
                } else {
                    __builtin_nontemporal_store((float)S[rt][0][s], at);
                }
            }
    };
    auto start_state = [&] {
        if (!SUM && sg.count > 1 && cols) {
            load_state(sg.at == 0 ? state_at(p.seg_first, n) : state_at(p.seg_state, j - 1));
        } else if (cols && sg.at == 0 && request_continues(p.pool, n)) {
            load_state(state_at(p.pool.base, slot));
        } else {
#pragma unroll
            for (int rt = 0; rt < NT; ++rt)
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        S[rt][ct][s] =
                            map && 8 * (lane0 >> 4) + state_row(rt, s) == col + ct ? 1.0f : 0.0f;
        }
        // the last segment of the later pass overwrites the pool's state
        if (SUM && sg.at == 0 && cols) store_state(state_at(p.seg_first, n), p.V);
    };
    // the values of this wavefront's columns
    RawC<EI, CT> vraw[2][4];
    auto load_values = [&](int t0) {
        const int len = min(kPreC, len_all - t0);
        // (no row at all for M's columns: V = 0)
        const Rsrc rv = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(vb + (long)t0 * vs), 0,
            map ? 0 : (len - 1) * vs + p.V * EI::kBytes, kRsrcWord3);
        const uint32_t at = 4 * (opaque_lane(lane0) >> 4) * vs + col * EI::kBytes;
#pragma unroll
        for (int I = 0; I < 2; ++I)
#pragma unroll
            for (int s = 0; s < 4; ++s) vraw[I][s].load(rv, at + (16 * I + s) * vs);
    };
    auto use = [&](int t0, int buf, bool far, bool apart, int stop) {
        const int len = min(kPreC, len_all - t0);
        const int lane = opaque_lane(lane0);
        const int g4 = lane >> 4, n16 = lane & 15;
        const int rpos = n16 * L::RS + ((g4 << 4) ^ L::swz_row(n16));
        const char *op = lds + buf * L::kBuffer, *fac = lds + L::FACTORS + buf * L::kFactors;
        // 16 rows of an operand reduced over channels, k-step kk
        auto row_operand = [&]<class O>(int at, int kk) -> O {
            O o;
#pragma unroll
            for (int i = 0; i < (int)(sizeof(O) / sizeof(w4)); ++i)
                o.p[i] = *reinterpret_cast<const w4 *>(op + at + i * L::R32 + (rpos ^ (64 * kk)));
            return o;
        };
        // a lower triangle's rows 0..15, and 16..31
        auto top_operand = [&](int at) {
            Half o;
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                o.p[i] = *reinterpret_cast<const w2 *>(op + at + i * L::T32 + n16 * (L::TS / 2) +
                                                       8 * g4);
            return o;
        };
        auto low_operand = [&](int at) {
            Operand o;
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                o.p[i] = *reinterpret_cast<const w4 *>(op + at + i * L::T32 + L::LOW +
                                                       n16 * L::TS + ((g4 << 4) ^ L::swz_tok(n16)));
            return o;
        };
        // The operands of each group of products are read from LDS one group
        // ahead, and the state's next rows are scaled and split in the
        // products' shadow.
        const f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        f4 kS[2][CT], o[2][CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) kS[0][ct] = kS[1][ct] = o[0][ct] = o[1][ct] = z;
        Operand ka_op[2];
        typename L::Queries qa_op[2];
        Operand b[2][CT];
        f4 em[2];
        auto read_rows = [&](int j) {  // k-step j / 2, row tile j % 2
            const int at = 16 * (j & 1) * L::RS;
            ka_op[j & 1] = row_operand.template operator()<Operand>(L::KR + at, j >> 1);
            if constexpr (!SUM)
                qa_op[j & 1] =
                    row_operand.template operator()<typename L::Queries>(L::QR + at, j >> 1);
        };
        auto read_em = [&](int kk) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                em[t] = *reinterpret_cast<const f4 *>(fac + L::EM +
                                                      4 * (8 * g4 + state_row(2 * kk + t, 0)));
        };
        auto split_state = [&](int kk, int ct) {  // S' (also of a steep chunk, where it is S)
#pragma unroll
            for (int t = 0; t < 2; ++t) S[2 * kk + t][ct] *= em[t];
            b[kk & 1][ct] = join(split4(S[2 * kk][ct]), split4(S[2 * kk + 1][ct]));
        };
        if (apart) {
#pragma unroll
            for (int rt = 0; rt < NT; ++rt) {
                const f4 e =
                    *reinterpret_cast<const f4 *>(fac + L::EG + 4 * (8 * g4 + state_row(rt, 0)));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[rt][ct] *= e;
            }
        }
        // (no room for the next operands beside 32 columns and the preparation's
        // registers, 16 x 512 tokens 552 -> 470 us, or with three wavefronts to a
        // SIMD; elsewhere 1 to 2% faster)
        constexpr bool kNext = K == 64 || (!SUM && (ROLES || CT == 1));
        read_em(0);
        read_rows(0);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) split_state(0, ct);
        read_em(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < K / 16; ++j) {
            const int kk = j >> 1, I = j & 1;
            if (kNext && j + 1 < K / 16) read_rows(j + 1);
            if (!kNext && j > 0) read_rows(j);
            if (kk + 1 < K / 32 && I < CT) split_state(kk + 1, I);
            if (I == 1 && kk + 2 < K / 32) read_em(kk + 2);
            if constexpr (SUM) {
                mul_columns<CT>(ka_op[I], b[kk & 1], kS[I]);
            } else {
                const Operand qa = qa_op[I].parts();
#pragma unroll
                for (int i = 0; i < 6; ++i)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        const auto &bc = b[kk & 1][ct];
                        kS[I][ct] = mfma(ka_op[I].p[part_a(i)], bc.p[part_b(i)], kS[I][ct]);
                        o[I][ct] = mfma(qa.p[part_a(i)], bc.p[part_b(i)], o[I][ct]);
                    }
            }
            __builtin_amdgcn_sched_group_barrier(0x100, SUM ? 3 : 3 + L::kRawQ, 0);  // LDS reads
            interleave<SUM ? 6 * CT : 12 * CT, SUM ? 5 : 3>();
            __builtin_amdgcn_sched_barrier(0);
        }
        // U, 16 rows at a time, X the inverse's diagonal blocks times beta:
        // R = V - (k e^G) S, U_0 = X_00 R_0, U_1 = X_11 (R_1 - (L_10 / beta) U_0)
        f4 R[2][CT];
#pragma unroll
        for (int I = 0; I < 2; ++I)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) R[I][ct][s] = vraw[I][s].at(ct) - kS[I][ct][s];
        if (ROLES && t0 + kPreC < len_all) load_values(t0 + kPreC);
        // A value that is not finite may only reach its column's outputs from its
        // token on, but the products with zeros above the diagonals would take it
        // to earlier ones: the column is then without tokens from there on, and
        // its outputs from there on and its state are NaN.
        int first[CT];
        bool broken = stop < kPreC;
        if constexpr (!SUM) {
            float most = 0.0f;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) most = largest(largest(most, R[0][ct]), R[1][ct]);
            broken |= __ballot(!finite(most)) != 0;
            if (broken) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    first[ct] = stop;
#pragma unroll
                    for (int I = 0; I < 2; ++I)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            if (!finite(R[I][ct][s]))
                                first[ct] = min(first[ct], 16 * I + 4 * g4 + s);
                    first[ct] = min(first[ct], __shfl_xor(first[ct], 16));
                    first[ct] = min(first[ct], __shfl_xor(first[ct], 32));
#pragma unroll
                    for (int I = 0; I < 2; ++I)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            if (16 * I + 4 * g4 + s >= first[ct]) R[I][ct][s] = 0.0f;
                }
            }
        }
        Operand u[CT];
        {
            const auto x0 = top_operand(L::TM);
            const auto x1 = low_operand(L::TM);
            const auto p0 = top_operand(L::PM);
            const auto p1 = low_operand(L::PM);
            Half r[CT], h0[CT];
            f4 x[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                r[ct] = split4(R[0][ct]);
                x[ct] = z;
            }
            mul_columns<CT>(x0, r, x);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) h0[ct] = split4(x[ct]);
            mul_columns<CT>(half_of(x1, 0), h0, R[1]);
            if constexpr (!SUM) mul_columns<CT>(p0, h0, o[0]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                r[ct] = split4(R[1][ct]);
                x[ct] = z;
            }
            mul_columns<CT>(half_of(x1, 1), r, x);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) u[ct] = join(h0[ct], split4(x[ct]));
            if constexpr (!SUM) mul_columns<CT>(p1, u, o[1]);
        }
        if constexpr (!SUM) {
            if (broken)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int I = 0; I < 2; ++I)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            if (16 * I + 4 * g4 + s >= first[ct]) o[I][ct][s] = __builtin_nanf("");
            const Rsrc ro = rows_of(ob + (long)t0 * os, os, p.V * OE, len);
            const uint32_t at = 4 * g4 * os + col * OE;
#pragma unroll
            for (int I = 0; I < 2; ++I)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    put_out(ro, at + (16 * I + s) * os, o[I], s);
        }
        // the state: S' + (k e^{m - G})^T U, which owes e^{G_32 - m}; of a steep
        // chunk e^{G_32} S + (k e^{G_32 - G})^T U
        Operand kt[2];
        // rows of tile rt are channels, reduced over tokens: 4 x 16 blocks of
        // the keys' rows, transposed by the read (lane 4 r + c of 16 gives the
        // address of 4 channels of token r, lane j gets channel j's 4 tokens).
        // Of a row's bytes, bits 4 and 5 are c, 6 and 7 are rt / 2.
        const int trow = 4 * g4 + (n16 >> 2);
        int tpiece[2];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
            tpiece[hb] = (trow + 16 * hb) * L::RS +
                         ((16 * (n16 & 3)) ^ L::swz_row(trow + 16 * hb));
        auto read_state = [&](int rt) {
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
                const char *at = op + (tpiece[hb] ^ (64 * (rt >> 1)));
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const w2 x = read_transposed(at + L::KL + i * L::R32 + 8 * (rt & 1));
                    kt[rt & 1].p[i][2 * hb] = x[0];
                    kt[rt & 1].p[i][2 * hb + 1] = x[1];
                }
            }
        };
        if (far) {
#pragma unroll
            for (int rt = 0; rt < NT; ++rt) {
                const f4 e =
                    *reinterpret_cast<const f4 *>(fac + L::EF + 4 * (8 * g4 + state_row(rt, 0)));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[rt][ct] *= e;
            }
        }
        read_state(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
            if (rt + 1 < NT) read_state(rt + 1);
            mul_columns<CT>(kt[rt & 1], u, S[rt]);
            __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
            interleave<6 * CT, 1>();
            __builtin_amdgcn_sched_barrier(0);
        }
        if (broken)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                if (SUM || first[ct] < kPreC)
#pragma unroll
                    for (int rt = 0; rt < NT; ++rt)
#pragma unroll
                        for (int s = 0; s < 4; ++s) S[rt][ct][s] = __builtin_nanf("");
    };

    // ======== the walk over the chunks
    if constexpr (ROLES) {
        if (prepares) {
            // (16,384 tokens, 32 heads, cut: 900 -> 890 us; in the sums, too, where
            // eight other wavefronts would wait: 914 us)
            if (!SUM) __builtin_amdgcn_s_setprio(2);
            Rows next;
            next.beta = 0.0f;
            if (len_all > 0) {
                if (pw == 0 && lane0 == 0) *count = 0;
                load_rows(0, now);
                sum_decays(0);
                __syncthreads();
            }
            for (int t0 = 0, buf = 0; t0 < len_all; t0 += kPreC, buf ^= 1) {
                const bool more = t0 + kPreC < len_all;
                bool far, apart;
                int stop;
                if (more) load_rows(t0 + kPreC, next);
                prepare(buf, far, apart, stop);
                if (more) {
                    now = next;
                    sum_decays(buf ^ 1);
                }
                __syncthreads();  // this chunk's operands, the next one's totals
            }
            if (len_all > 0) {
                // what the last chunk owes (nothing reads the totals now)
                if (pw == 0 && lane0 < K / 4)
                    *reinterpret_cast<f4 *>(lds + L::TOT + 16 * lane0) = exp2(owed_i);
                __syncthreads();
            }
            return;
        }
        start_state();
        if (len_all > 0) {
            if (cols) load_values(0);
            __syncthreads();  // totals
            __syncthreads();  // the first chunk's operands
        }
        for (int t0 = 0, buf = 0; t0 < len_all; t0 += kPreC, buf ^= 1) {
            const int flags = __builtin_amdgcn_readfirstlane(
                reinterpret_cast<const int *>(lds + L::FLAGS)[buf]);
            if (cols) use(t0, buf, flags & 1, flags & 2, flags >> 2);
            __syncthreads();
        }
    } else {
        start_state();
        if (len_all > 0) load_rows(0, now);
        for (int t0 = 0; t0 < len_all; t0 += kPreC) {
            bool far, apart;
            int stop;
            // The other workgroup of the compute unit gives way to a walk (8 x 2,048
            // tokens, 64 heads: 922 -> 865 us; 16 x 512, K = 64: 282 -> 267 us).
            __builtin_amdgcn_s_setprio(0);
            sum_decays(0);
            __syncthreads();  // totals; nothing reads the chunk before any more
            prepare(0, far, apart, stop);
            if (cols) load_values(t0);
            __syncthreads();
            __builtin_amdgcn_s_setprio(2);
            if (t0 + kPreC < len_all) load_rows(t0 + kPreC, now);
            if (cols) use(t0, 0, far, apart, stop);
        }
        if (len_all > 0) {
            if (pw == 0 && lane0 < K / 4)
                *reinterpret_cast<f4 *>(lds + L::TOT + 16 * lane0) = exp2(owed_i);
            __syncthreads();
        }
    }
    if (len_all > 0) {  // what the last chunk owes
        const float *left = reinterpret_cast<const float *>(lds + L::TOT);
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) {
            const f4 e =
                *reinterpret_cast<const f4 *>(left + 8 * (lane0 >> 4) + state_row(rt, 0));
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[rt][ct] *= e;
        }
    }
    if (SUM && cols) {
        if (map)
            store_state(p.seg_map + (((long)j * p.H + h) * K + 8 * (lane0 >> 4)) * K + col, K);
        else
            store_state(state_at(p.seg_state, j), p.V);
    } else if (keep && cols && sg.at + 1 == sg.count) {
        store_state(state_at(p.pool.base, slot), p.V);
    }
}

template <class EI>
hipError_t launch_prefill_of(const DeltaProblem &p, PrePass pass, hipStream_t stream) {
    const int64_t parts = p.seg != 0 ? p.segs : p.req.num_seqs;
    auto go = [&]<int K, int OUT, bool SUM, bool ROLES, int CT>() {
        typedef PreShape<SUM, ROLES, CT> Shape;
        const int cols = p.V + (SUM ? K : 0);
        const dim3 grid((unsigned)(parts * p.H),
                        (unsigned)((cols + Shape::kWidth - 1) / Shape::kWidth));
        hipLaunchKernelGGL((kda_prefill_kernel<EI, K, OUT, SUM, ROLES, CT>), grid,
                           dim3(Shape::kThreads), 0, stream, p);
        return hipGetLastError();
    };
    // Columns of 16 to a wavefront halve its part of a chunk: while that still
    // takes at most a workgroup per compute unit (64 walks of 64 tokens 21.2 ->
    // 17.5 us, 128 walks of 300 tokens 76 -> 64 us), and for up to 64 columns in
    // all, which 32 to a wavefront would leave to two of four wavefronts (1,024
    // walks of 512 tokens, K = 128, V = 64, 358 -> 330 us; K = V = 64 236 -> 193).
    auto with_out = [&]<int K, int OUT>() {
        // FP32 rows on their way leave a wavefront that does both without
        // registers: it spills (f32, 40 requests of 1 to 2,000 tokens, 16 heads
        // 761 -> 835 us; 64 of 64 tokens, 64 heads 374 and 334)
        constexpr bool kRoles = K == 128 && EI::kBytes == 4;
        if (pass == PrePass::narrow) return go.template operator()<K, OUT, false, true, 1>();
        if (pass == PrePass::roles) return go.template operator()<K, OUT, false, true, 2>();
        return p.V <= 64 ? go.template operator()<K, OUT, false, kRoles, 1>()
                         : go.template operator()<K, OUT, false, kRoles, 2>();
    };
    auto with_k = [&]<int K>() {
        // (the sums have no outputs: OUT does not matter)
        return pass == PrePass::sums ? go.template operator()<K, 1, true, true, 2>()
               : p.out_dt == 0       ? with_out.template operator()<K, 0>()
               : p.out_dt == 1       ? with_out.template operator()<K, 1>()
                                     : with_out.template operator()<K, 2>();
    };
    return p.K == 64 ? with_k.template operator()<64>() : with_k.template operator()<128>();
}

hipError_t launch_prefill_f32(const DeltaProblem &p, PrePass pass, hipStream_t stream);
hipError_t launch_prefill_bf16(const DeltaProblem &p, PrePass pass, hipStream_t stream);
hipError_t launch_prefill_f16(const DeltaProblem &p, PrePass pass, hipStream_t stream);

}  // namespace kda
