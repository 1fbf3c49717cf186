// FP32 products on the bfloat16 matrix cores: every factor as a sum of three
// bfloat16 parts.
#pragma once

#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

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

}  // namespace kda
