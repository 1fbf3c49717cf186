// Device helpers shared by the KDA layer's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_layer.h"
#include "tril_device.h"

namespace kda {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t w2 __attribute__((ext_vector_type(2)));
typedef uint32_t w4 __attribute__((ext_vector_type(4)));

// Elements widened to float (exact) and pairs packed back (round to nearest even).
template <class E>
struct Elem;
template <>
struct Elem<F32> {
    static __device__ __forceinline__ float one(const float *p) { return *p; }
};
template <>
struct Elem<BF16> {
    static __device__ __forceinline__ float widen(uint32_t b) { return bf16_to_f32(b); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        const b2 v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return widen(*p); }
};
template <>
struct Elem<F16> {
    static __device__ __forceinline__ float widen(uint32_t b) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return widen(*p); }
};

// Eight consecutive elements (16 or 32 bytes, 16-byte aligned).
template <class E>
struct Raw8 {
    w4 w;
    __device__ __forceinline__ void load(const typename E::T *p) {
        w = *reinterpret_cast<const w4 *>(p);
    }
    __device__ __forceinline__ void load_stream(const typename E::T *p) {  // read once
        w = __builtin_nontemporal_load(reinterpret_cast<const w4 *>(p));
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = Elem<E>::widen(w[i] & 0xFFFFu);
            x[2 * i + 1] = Elem<E>::widen(w[i] >> 16);
        }
    }
    static __device__ __forceinline__ void store(typename E::T *p, const float (&x)[8]) {
        w4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = Elem<E>::pack(x[2 * i], x[2 * i + 1]);
        __builtin_nontemporal_store(o, reinterpret_cast<w4 *>(p));
    }
};
template <>
struct Raw8<F32> {
    f4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const f4 *>(p)[0];
        b = reinterpret_cast<const f4 *>(p)[1];
    }
    __device__ __forceinline__ void load_stream(const float *p) {
        a = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p));
        b = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p) + 1);
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8]) {
        const f4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
        __builtin_nontemporal_store(lo, reinterpret_cast<f4 *>(p));
        __builtin_nontemporal_store(hi, reinterpret_cast<f4 *>(p) + 1);
    }
};

// First row and length of request n, clamped to the rows of the tensors so
// that a malformed cu_seqlens cannot address memory outside them.
__device__ __forceinline__ int2 request_rows(const Requests &r, int n) {
    if (r.cu == nullptr) return make_int2(n * r.seq_len, r.seq_len);
    const int b = min(max(r.cu[n], 0), r.total_tokens);
    const int e = min(max(r.cu[n + 1], b), r.total_tokens);
    return make_int2(b, e - b);
}

// Pool slot of request n: -1 for padding (outside the pool).
__device__ __forceinline__ int request_slot(const Pool &p, int n) {
    const int s = p.slot ? p.slot[n] : n;
    return s >= 0 && s < p.num_slots ? s : -1;
}
__device__ __forceinline__ bool request_continues(const Pool &p, int n) {
    return p.base != nullptr && (p.init == nullptr || p.init[n] != 0);
}

// Sums over groups of lanes on DPP moves and lane swaps; partners are paired
// both ways, so every lane of a group ends with the same bits.
template <int CTRL>
__device__ __forceinline__ float lane_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL,
                                                                  0xF, 0xF, true));
}
__device__ __forceinline__ float sum8(float v) {  // 8 adjacent lanes
    return lane_add<0x141>(lane_add<0x4E>(lane_add<0xB1>(v)));
}
__device__ __forceinline__ float sum16(float v) { return lane_add<0x140>(sum8(v)); }
__device__ __forceinline__ float add_rows16(float v) {  // 16-lane rows 0 + 1, 2 + 3
    float a = v, b = v;
    lane_swap16(a, b);
    return a + b;
}
__device__ __forceinline__ float add_rows32(float v) {  // lanes 0..31 + 32..63
    float a = v, b = v;
    lane_swap32(a, b);
    return a + b;
}
__device__ __forceinline__ float sum64(float v) { return add_rows32(add_rows16(sum16(v))); }

__device__ __forceinline__ f4 exp2(f4 x) {
    return f4{__builtin_amdgcn_exp2f(x[0]), __builtin_amdgcn_exp2f(x[1]),
              __builtin_amdgcn_exp2f(x[2]), __builtin_amdgcn_exp2f(x[3])};
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

}  // namespace kda
