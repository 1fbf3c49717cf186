// Activation checkpoints in 8 bits for gfx950: vectors of d channels as int8
// codes with one FP32 scale each, their reading back, and the gated RMSNorm
// that stores both of its inputs so on its way.
//
// Bound by memory: each element is read and written once, and a vector takes
// d / 8 lanes, so its largest magnitude is a DPP maximum over 8 or 16 lanes.
// 8,192 x 64 vectors of 3 x 128, bf16: into codes 112 us and back 85 (5.4 and 7.2
// TB/s, some of it in the last-level cache); the norm with its two checkpoints 105 us
// on vectors of 128.
#include <hip/hip_runtime.h>

#include "code8.h"
#include "tril_launch.h"

namespace kda {

constexpr int kCodeThreads = 256;

template <class E, int D>
__global__ __launch_bounds__(kCodeThreads) void kda_checkpoint_kernel(CheckpointProblem p) {
    constexpr int L = D / 8;
    const long first = (long)blockIdx.x * kCodeThreads + threadIdx.x;
    const long vec = first / L;
    if (vec >= p.vecs) return;
    const int c = (int)(threadIdx.x % L) * 8;
    Raw8<E> raw;
    raw.load_stream(static_cast<const typename E::T *>(p.x) + vec * D + c);
    float x[8];
    int code[8];
    raw.widen(x);
    const float scale = encode8<L>(x, code);
    Raw8<I8>::store(p.codes + vec * D + c, code);
    if (c == 0) p.scale[vec] = scale;
}

template <class E, int D>
__global__ __launch_bounds__(kCodeThreads) void kda_checkpoint_load_kernel(CheckpointProblem p) {
    constexpr int L = D / 8;
    const long first = (long)blockIdx.x * kCodeThreads + threadIdx.x;
    const long vec = first / L;
    if (vec >= p.vecs) return;
    const int c = (int)(threadIdx.x % L) * 8;
    Raw8<I8> raw;
    raw.load_stream(p.codes + vec * D + c);
    const float scale = p.scale[vec];
    float x[8];
    raw.widen(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= scale;
    Raw8<E>::store(static_cast<typename E::T *>(p.out) + vec * D + c, x);
}

// kda_gated_norm_kernel with both inputs' checkpoints.
template <class E, class EO, int D>
__global__ __launch_bounds__(kCodeThreads) void kda_norm_checkpoint_kernel(
    NormCheckpointProblem p) {
    constexpr int L = D / 8;
    const long first = (long)blockIdx.x * kCodeThreads + threadIdx.x;
    const long vec = first / L;
    if (vec >= p.norm.vecs) return;
    const int c = (int)(threadIdx.x % L) * 8;
    float w[8], o[8], z[8];
    Raw8<E> ro, rz;
    ro.load_stream(static_cast<const typename E::T *>(p.norm.o) + vec * D + c);
    rz.load_stream(static_cast<const typename E::T *>(p.norm.z) + vec * D + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p.norm.norm_w[c + i];
    ro.widen(o);
    rz.widen(z);
    int code[8];
    const float so = encode8<L>(o, code);
    Raw8<I8>::store(p.o_codes + vec * D + c, code);
    const float sz = encode8<L>(z, code);
    Raw8<I8>::store(p.z_codes + vec * D + c, code);
    if (c == 0) {
        p.o_scale[vec] = so;
        p.z_scale[vec] = sz;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(o[i], o[i], ss);
    ss = L == 16 ? sum16(ss) : sum8(ss);
    const float rn = 1.0f / __builtin_sqrtf(ss * (1.0f / D) + p.norm.eps_norm);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * rn * w[i] / (1.0f + __expf(-z[i]));
    Raw8<EO>::store(static_cast<typename EO::T *>(p.norm.out) + vec * D + c, o);
}

hipError_t launch_checkpoint(const CheckpointProblem &p, int dt, hipStream_t stream) {
    const long threads = p.vecs * (p.d / 8);
    const dim3 grid((unsigned)((threads + kCodeThreads - 1) / kCodeThreads));
    return dispatch_dtypes<F32, BF16, F16>(dt, 0, [&]<class E, class EO>() {
        const bool save = p.x != nullptr;
        const auto fn = p.d == 64 ? (save ? kda_checkpoint_kernel<E, 64>
                                          : kda_checkpoint_load_kernel<E, 64>)
                                  : (save ? kda_checkpoint_kernel<E, 128>
                                          : kda_checkpoint_load_kernel<E, 128>);
        hipLaunchKernelGGL(fn, grid, dim3(kCodeThreads), 0, stream, p);
        return hipGetLastError();
    });
}

hipError_t launch_norm_checkpoint(const NormCheckpointProblem &p, int in_dt, int out_dt,
                                  hipStream_t stream) {
    const long threads = p.norm.vecs * (p.norm.d / 8);
    const dim3 grid((unsigned)((threads + kCodeThreads - 1) / kCodeThreads));
    return dispatch_dtypes<F32, BF16, F16>(in_dt, out_dt, [&]<class E, class EO>() {
        const auto fn = p.norm.d == 64 ? kda_norm_checkpoint_kernel<E, EO, 64>
                                       : kda_norm_checkpoint_kernel<E, EO, 128>;
        hipLaunchKernelGGL(fn, grid, dim3(kCodeThreads), 0, stream, p);
        return hipGetLastError();
    });
}

}  // namespace kda
