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

}  // namespace kda
