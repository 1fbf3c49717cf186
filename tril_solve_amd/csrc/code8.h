// Vectors of d channels held in 8 bits: int8 codes and one FP32 scale, the
// largest magnitude being 127 steps. Eight channels to a lane.
#pragma once

#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

struct I8 {
    typedef int8_t T;
    static constexpr int kBytes = 1;
};
template <>
struct Raw8<I8> {
    w2 w;
    __device__ __forceinline__ void load(const int8_t *p) { w = *reinterpret_cast<const w2 *>(p); }
    __device__ __forceinline__ void load_stream(const int8_t *p) {
        w = __builtin_nontemporal_load(reinterpret_cast<const w2 *>(p));
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(w[i >> 2] >> 8 * (i & 3));
    }
    static __device__ __forceinline__ void store(int8_t *p, const int (&c)[8]) {
        w2 o = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i >> 2] |= (uint32_t)(c[i] & 0xFF) << 8 * (i & 3);
        *reinterpret_cast<w2 *>(p) = o;
    }
};

template <int CTRL>
__device__ __forceinline__ float lane_max(float v) {
    return __builtin_elementwise_maximum(
        v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF,
                                                              0xF, true)));
}
// The largest of L = 8 or 16 adjacent lanes, NaN where there is one.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    v = lane_max<0x141>(lane_max<0x4E>(lane_max<0xB1>(v)));
    return L == 16 ? lane_max<0x140>(v) : v;
}

// Largest magnitudes below this are stored as zeros: their steps would leave
// FP32's normal range.
constexpr float kLeast8 = 0x1p-110f;
// The largest step of which 127 are finite in FP32: the quotient of the largest
// float (and of no other) rounds to the one above and would read back as infinity.
constexpr float kMost8 = 0x1.020406p+121f;

// Codes of x and the vector's scale: the integer nearest x / scale, halves to
// even, found exactly. x / scale is first taken by 127 / max, off by less
// than 2^-14, so the integer next to it is at most one off, and only where the
// quotient is near a half; the remainder x - c scale of that integer is then exact
// in FP32 (both are multiples of half the scale's last place, and it is near
// half the scale) and says which side x is on. Hardly any wavefront has such a
// value: the rest skip that (4 of 14 vector instructions a value are left). A
// vector that is not finite keeps a scale of NaN and reads back as NaN.
template <int L>
__device__ __forceinline__ float encode8(const float (&x)[8], int (&c)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_elementwise_maximum(top, __builtin_fabsf(x[i]));
    top = lanes_max<L>(top);
    const bool fine = top < __builtin_inff(), some = top >= kLeast8;
    const float scale = __builtin_fminf(top / 127.0f, kMost8), half = 0.5f * scale;
    const float inv = fine && some ? 127.0f / top : 0.0f;
    float n[8], worst = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        n[i] = __builtin_rintf((fine ? x[i] : 0.0f) * inv);
        worst = __builtin_fmaxf(worst, __builtin_fabsf(__builtin_fmaf(-n[i], scale, x[i])));
    }
    if (__any(worst >= half && inv > 0.0f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = __builtin_fmaf(-n[i], scale, x[i]);
            const bool odd = (int)n[i] & 1;
            if (inv > 0.0f && (r > half || (r == half && odd))) n[i] += 1.0f;
            if (inv > 0.0f && (r < -half || (r == -half && odd))) n[i] -= 1.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = (int)n[i];
    return !fine ? __builtin_nanf("") : some ? scale : 0.0f;
}

}  // namespace kda
