// Launch of the gated delta rule over whole prompts, and the walk over the
// segments of prompts that are cut.
#include "kda_prefill.h"

namespace kda {

namespace {

// The states between a request's segments, S_{s + 1} = M_s S_s + B_s, in place
// of the B_s: one workgroup per request, head and 16 value columns, a quarter
// of the rows to a wavefront, on the FP32 matrix cores. The rows of the next
// M_s, which do not depend on the state, are loaded during a step; the state
// goes from one step's accumulators to the next one's operands through LDS.
// Reduction index 4 (4 a + e) + g of a 16 x 16 x 4 product means channel
// 16 a + 4 g + e, which is row e of lane group g in accumulator tile a.
template <int K>
__global__ __launch_bounds__(256) void kda_prefill_join_kernel(DeltaProblem p) {
    constexpr int NT = K / 16, TPW = NT / 4;  // row tiles, those of a wavefront
    __shared__ f4 st[2][NT][kWave];
    const int lane = threadIdx.x & (kWave - 1), g4 = lane >> 4, n16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = blockIdx.x / p.H, h = blockIdx.x - n * p.H;
    int own;
    const int upto = segments_to_lane(p, own);
    const int count = __builtin_amdgcn_readlane(own, n);
    const int first = __builtin_amdgcn_readlane(upto, n) - count;
    const int end = min(first + count, p.segs) - 1;  // the last segment has no M and B
    if (first + 1 >= end || (p.pool.base != nullptr && request_slot(p.pool, n) < 0)) return;

    const int col = blockIdx.y * 16 + n16;
    auto states = [&](int j, int t) {  // rows 16 (TPW wv + t) + 4 g4 ..
        return p.seg_state +
               (((long)j * p.H + h) * K + 16 * (TPW * wv + t) + 4 * g4) * p.V + col;
    };
    f4 x[TPW], m[TPW][NT], b[TPW];
    auto load = [&](int j) {
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            const float *row = p.seg_map +
                (((long)j * p.H + h) * K + 16 * (TPW * wv + t) + n16) * K + 4 * g4;
#pragma unroll
            for (int a = 0; a < NT; ++a) m[t][a] = *reinterpret_cast<const f4 *>(row + 16 * a);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[t][e] = states(j, t)[(long)e * p.V];
        }
    };
    load(first + 1);
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] = states(first, t)[(long)e * p.V];
    for (int j = first + 1, buf = 0; j < end; ++j, buf ^= 1) {
#pragma unroll
        for (int t = 0; t < TPW; ++t) st[buf][TPW * wv + t][lane] = x[t];
        f4 m_now[TPW][NT];
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            x[t] = b[t];
#pragma unroll
            for (int a = 0; a < NT; ++a) m_now[t][a] = m[t][a];
        }
        __syncthreads();  // (the reads of the step before the last are done, too)
        if (j + 1 < end) load(j + 1);
#pragma unroll
        for (int a = 0; a < NT; ++a) {
            const f4 s = st[buf][a][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < TPW; ++t)
                    x[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(m_now[t][a][e], s[e], x[t], 0, 0,
                                                                0);
        }
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) states(j, t)[(long)e * p.V] = x[t][e];
    }
}

// Workgroups per request and head.
int column_blocks(int V) {
    constexpr int each = PreShape<false, true>::kCols * kPreCols;
    return (V + each - 1) / each;
}

hipError_t launch_pass(const DeltaProblem &p, int in_dt, PrePass pass, hipStream_t stream) {
    return in_dt == 0   ? launch_prefill_f32(p, pass, stream)
           : in_dt == 1 ? launch_prefill_bf16(p, pass, stream)
                        : launch_prefill_f16(p, pass, stream);
}

}  // namespace

// A request's walk over its chunks is serial, so a few (request, head, 128
// columns) workgroups leave most of the 256 compute units idle; a cut prompt
// takes the chunks of its segments at once, for about 2.4 times the work.
int32_t prefill_segments(int64_t total_tokens, int64_t num_seqs, int32_t H, int32_t V) {
    const int64_t walks = num_seqs * H * column_blocks(V);
    const int64_t chunks = total_tokens / kPreC;
    if (num_seqs < 1 || num_seqs > kMaxCutRequests || walks > 64 || chunks < 16 * num_seqs)
        return 0;
    const int64_t parts = 256 * num_seqs / walks;  // a workgroup per compute unit
    const int64_t seg = (chunks + parts - 1) / parts;
    return (int32_t)(kPreC * (seg < 4 ? 4 : seg));
}

hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream) {
    if (p.seg != 0) {
        hipError_t e = launch_pass(p, in_dt, PrePass::sums, stream);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)(p.req.num_seqs * p.H), (unsigned)(p.V / 16));
        if (p.K == 64)
            hipLaunchKernelGGL((kda_prefill_join_kernel<64>), grid, dim3(256), 0, stream, p);
        else
            hipLaunchKernelGGL((kda_prefill_join_kernel<128>), grid, dim3(256), 0, stream, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t walks = (p.seg != 0 ? p.segs : p.req.num_seqs) * (int64_t)p.H * column_blocks(p.V);
    return launch_pass(p, in_dt, walks <= 256 ? PrePass::roles : PrePass::whole, stream);
}

}  // namespace kda
