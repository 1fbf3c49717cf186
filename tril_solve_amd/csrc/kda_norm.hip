// Gated RMSNorm of a prompt's outputs for gfx950 (the decode step's last
// stage, for many tokens): out = o / sqrt(mean(o^2) + eps) * w * sigmoid(z).
//
// Bound by memory: every element of o and z is read once and of out written
// once. A vector of d channels takes d / 8 lanes of 8 channels each (16-byte
// loads of 16-bit elements), so the sum of squares is a DPP sum over 8 or 16
// lanes and nothing goes through LDS. 16 x 512 tokens, 64 heads of 128, bf16:
// 62 us, 6.5 TB/s of its 403 MB (some of it served by the last-level cache; a
// tuned copy reaches 6.4); 64 tokens: 2.6 us.
#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

constexpr int kNormThreads = 256;

template <class E, class EO, int D>
__global__ __launch_bounds__(kNormThreads) void kda_gated_norm_kernel(NormProblem p) {
    constexpr int L = D / 8;  // lanes per vector
    const long first = (long)blockIdx.x * kNormThreads + threadIdx.x;
    const int c = (int)(threadIdx.x % L) * 8;
    const long vec = first / L;
    if (vec >= p.vecs) return;  // whole groups of L lanes leave together
    float w[8], o[8], z[8];
    Raw8<E> ro, rz;
    ro.load_stream(static_cast<const typename E::T *>(p.o) + vec * D + c);
    rz.load_stream(static_cast<const typename E::T *>(p.z) + vec * D + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p.norm_w[c + i];
    ro.widen(o);
    rz.widen(z);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(o[i], o[i], ss);
    ss = L == 16 ? sum16(ss) : sum8(ss);
    const float rn = 1.0f / __builtin_sqrtf(ss * (1.0f / D) + p.eps_norm);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * rn * w[i] / (1.0f + __expf(-z[i]));
    Raw8<EO>::store(static_cast<typename EO::T *>(p.out) + vec * D + c, o);
}

hipError_t launch_norm(const NormProblem &p, int in_dt, int out_dt, hipStream_t stream) {
    return dispatch_dtypes<F32, BF16, F16>(in_dt, out_dt, [&]<class E, class EO>() {
        const long threads = p.vecs * (p.d / 8);
        const dim3 grid((unsigned)((threads + kNormThreads - 1) / kNormThreads));
        if (p.d == 64)
            hipLaunchKernelGGL((kda_gated_norm_kernel<E, EO, 64>), grid, dim3(kNormThreads), 0,
                               stream, p);
        else
            hipLaunchKernelGGL((kda_gated_norm_kernel<E, EO, 128>), grid, dim3(kNormThreads), 0,
                               stream, p);
        return hipGetLastError();
    });
}

}  // namespace kda
