// Gradients of the gated RMSNorm for gfx950. With n = o / sqrt(mean(o^2) + eps),
// s = sigmoid(z), dout the gradient of out = n w s:
//   do = (dn - n mean(dn n)) / sqrt(mean(o^2) + eps),  dn = dout w s
//   dz = dout w n s (1 - s),   dw = sum over all vectors of dout n s
// o and z are tensors or 8-bit checkpoints.
//
// Bound by memory: three streams in, two out (8,192 x 64 vectors of 128, bf16 from
// 8-bit codes: 98 us, 5.5 TB/s of a tuned copy's 6.4). A vector takes d / 8 lanes of 8
// channels; a workgroup walks its share of the vectors with its part of dw in
// registers, joins it over its vectors in LDS and leaves one row in the
// workspace, and a second launch adds those rows in order, so dw has the same
// bits every time.
#include <hip/hip_runtime.h>

#include "code8.h"
#include "tril_launch.h"

namespace kda {

constexpr int kNgThreads = 256;

template <class E, class EX, int D>
__global__ __launch_bounds__(kNgThreads) void kda_norm_grad_kernel(NormGradProblem p) {
    constexpr int L = D / 8, kVecs = kNgThreads / L;
    constexpr bool kCoded = sizeof(typename EX::T) == 1;
    __shared__ float rows[kVecs][D];
    const int c = (int)(threadIdx.x % L) * 8, at = threadIdx.x / L;
    float w[8], dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = p.norm_w[c + i];
        dw[i] = 0.0f;
    }
    for (long vec = (long)blockIdx.x * kVecs + at; vec < p.vecs; vec += (long)gridDim.x * kVecs) {
        Raw8<E> rd;
        Raw8<EX> ro, rz;
        rd.load_stream(static_cast<const typename E::T *>(p.dout) + vec * D + c);
        ro.load_stream(static_cast<const typename EX::T *>(p.o) + vec * D + c);
        rz.load_stream(static_cast<const typename EX::T *>(p.z) + vec * D + c);
        float d[8], o[8], z[8];
        rd.widen(d);
        ro.widen(o);
        rz.widen(z);
        if constexpr (kCoded) {
            const float so = p.o_scale[vec], sz = p.z_scale[vec];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] *= so;
                z[i] *= sz;
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(o[i], o[i], ss);
        ss = L == 16 ? sum16(ss) : sum8(ss);
        const float rn = 1.0f / __builtin_sqrtf(ss * (1.0f / D) + p.eps_norm);
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __expf(-z[i]), s = __builtin_amdgcn_rcpf(1.0f + e);
            const float n = o[i] * rn, ds = d[i] * s, dn = ds * w[i];
            dw[i] = __builtin_fmaf(ds, n, dw[i]);
            // 1 - s = e s, without its cancellation; 0 where e overflows (s = 0)
            z[i] = dn * n * (e < __builtin_inff() ? e * s : 1.0f);
            o[i] = n;
            d[i] = dn;
            mean = __builtin_fmaf(dn, n, mean);
        }
        mean = (L == 16 ? sum16(mean) : sum8(mean)) * (1.0f / D);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rn * (d[i] - o[i] * mean);
        Raw8<E>::store(static_cast<typename E::T *>(p.d_o) + vec * D + c, o);
        Raw8<E>::store(static_cast<typename E::T *>(p.dz) + vec * D + c, z);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) rows[at][c + i] = dw[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kVecs; ++r) sum += rows[r][threadIdx.x];
        p.part[(long)blockIdx.x * D + threadIdx.x] = sum;
    }
}

// dw from the workgroups' rows: a workgroup per 16 channels, 16 lanes add every
// 64th row.
__global__ __launch_bounds__(1024) void kda_norm_grad_sum_kernel(NormGradProblem p, int rows) {
    __shared__ float part[64][17];
    const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    float sum = 0.0f;
#pragma unroll 8
    for (int r = r0; r < rows; r += 64) sum += p.part[(long)r * p.d + blockIdx.x * 16 + c];
    part[r0][c] = sum;
    __syncthreads();
    if (threadIdx.x < 16) {
        sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 64; ++r) sum += part[r][c];
        p.dnorm_w[blockIdx.x * 16 + c] = sum;
    }
}

hipError_t launch_norm_grad(const NormGradProblem &p, int dt, hipStream_t stream) {
    const unsigned blocks = (unsigned)norm_grad_blocks(p.vecs, p.d);
    const hipError_t e = blocks == 0 ? hipSuccess : dispatch_dtypes<F32, BF16, F16>(dt, 0, [&]<class E, class EO>() {
        const bool coded = p.o_scale != nullptr;
        const auto fn = p.d == 64 ? (coded ? kda_norm_grad_kernel<E, I8, 64>
                                           : kda_norm_grad_kernel<E, E, 64>)
                                  : (coded ? kda_norm_grad_kernel<E, I8, 128>
                                           : kda_norm_grad_kernel<E, E, 128>);
        hipLaunchKernelGGL(fn, dim3(blocks), dim3(kNgThreads), 0, stream, p);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kda_norm_grad_sum_kernel, dim3(p.d / 16), dim3(1024), 0, stream,
                       p, (int)blocks);
    return hipGetLastError();
}

}  // namespace kda
