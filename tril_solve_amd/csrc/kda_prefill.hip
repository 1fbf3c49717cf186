// Launch of the gated delta rule over whole prompts, and the walk over the
// segments of prompts that are cut.
#include "kda_prefill.h"

namespace kda {

namespace {

// The states between a request's segments, S_{s + 1} = M_s S_s + B_s, in place
// of the B_s: one workgroup per request, head and 16 value columns, 16 rows to
// a wavefront, on the FP32 matrix cores. What bounds it is a compute unit's
// loads of M, 64 KB a step (2.3 us). It forms S^T = S^T M^T +
// B^T, whose accumulators hold four adjacent columns of a row, so that B and S
// move 16 bytes at a time. The rows of the next two M_s, which do not depend
// on the state, are on their way during a step; the state goes from one step's
// accumulators to the next one's operands through LDS. Reduction index
// 4 (4 a + e) + g of the 16 x 16 x 4 products means channel 16 a + 4 g + e.
constexpr int kAhead = 2;  // steps whose M is loaded ahead (even: two LDS buffers in turn)
template <int K>
__global__ __launch_bounds__(4 * K, 2) void kda_prefill_join_kernel(DeltaProblem p) {
    constexpr int NT = K / 16;  // wavefronts
    constexpr int kRow = K + 4;  // floats between columns of the state in LDS
    __shared__ __align__(16) float st[2][16 * kRow];
    const int lane = threadIdx.x & (kWave - 1), g4 = lane >> 4, n16 = lane & 15;
    const int row = threadIdx.x / kWave * 16 + n16;  // of M and the state
    const int n = blockIdx.x / p.H, h = blockIdx.x - n * p.H;
    int own;
    const int upto = segments_to_lane(p, own);
    const int count = __builtin_amdgcn_readlane(own, n);
    const int first = __builtin_amdgcn_readlane(upto, n) - count;
    const int end = min(first + count, p.segs) - 1;  // the last segment has no M and B
    if (first + 1 >= end || (p.pool.base != nullptr && request_slot(p.pool, n) < 0)) return;

    auto state = [&](int j) -> f4 & {
        return *reinterpret_cast<f4 *>(p.seg_state + (((long)j * p.H + h) * K + row) * p.V +
                                       blockIdx.y * 16 + 4 * g4);
    };
    struct Step {
        f4 m[NT], b;
    };
    Step ahead[kAhead];
    auto load = [&](int j, Step &to) {
        const float *m = p.seg_map + (((long)j * p.H + h) * K + row) * K + 4 * g4;
#pragma unroll
        for (int a = 0; a < NT; ++a) to.m[a] = *reinterpret_cast<const f4 *>(m + 16 * a);
        to.b = state(j);
    };
    f4 x;
    auto step = [&](int j, Step &at, float *buf) {
#pragma unroll
        for (int e = 0; e < 4; ++e) buf[(4 * g4 + e) * kRow + row] = x[e];
        __syncthreads();  // (the reads of the step before the last are done, too)
        f4 s[NT];
#pragma unroll
        for (int a = 0; a < NT; ++a)
            s[a] = *reinterpret_cast<const f4 *>(buf + n16 * kRow + 16 * a + 4 * g4);
        f4 y = {0.0f, 0.0f, 0.0f, 0.0f};  // two sums: neither waits for itself
        x = at.b;
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                x = __builtin_amdgcn_mfma_f32_16x16x4f32(s[a][e], at.m[a][e], x, 0, 0, 0);
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(s[a][e + 1], at.m[a][e + 1], y, 0, 0, 0);
            }
        load(min(j + kAhead, end - 1), at);
        x += y;
        state(j) = x;
    };
    x = state(first);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(min(first + 1 + i, end - 1), ahead[i]);
    // (left from within: with steps or loads under conditions the compiler
    // would wait for every load in flight)
    for (int j = first + 1;;)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            step(j, ahead[i], st[i & 1]);
            if (++j == end) return;
        }
}

// Workgroups per request and head, wavefronts having CT tiles of 16 columns.
template <int CT>
int column_blocks(int V) {
    constexpr int each = PreShape<false, true, CT>::kWidth;
    return (V + each - 1) / each;
}

hipError_t launch_pass(const DeltaProblem &p, int in_dt, PrePass pass, hipStream_t stream) {
    return in_dt == 0   ? launch_prefill_f32(p, pass, stream)
           : in_dt == 1 ? launch_prefill_bf16(p, pass, stream)
                        : launch_prefill_f16(p, pass, stream);
}

}  // namespace

// MI355X's compute units. The rules below and the workspace query, which runs
// without a device, have to agree.
constexpr int64_t kUnits = 256;

// A request's walk over its chunks is serial, so a few (request, head, 128
// columns) workgroups leave most compute units idle; a cut prompt takes the
// chunks of its segments at once, for about twice the work: 32 walks of 16,384
// tokens 2,440 -> 870 us, of 768 tokens 121 -> 91 us, of 512 tokens 82 -> 72 us, 64
// walks of 2,048 tokens 312 -> 253 us, of 1,280 tokens 198 -> 169 us; but of 1,024
// tokens 160 and 154 us, 96 walks of 2,048 tokens 313 -> 376 us.
int32_t prefill_segments(int64_t total_tokens, int64_t num_seqs, int32_t H, int32_t V) {
    const int64_t walks = num_seqs * H * column_blocks<2>(V);
    const int64_t chunks = total_tokens / kPreC;
    if (num_seqs < 1 || num_seqs > kMaxCutRequests || walks > 64 ||
        chunks < (walks > 32 ? 40 : 16) * num_seqs)
        return 0;
    const int64_t parts = kUnits * num_seqs / walks;  // a workgroup per compute unit
    int64_t seg = (chunks + parts - 1) / parts;
    // A chunk more per segment takes 11 us of both passes, a segment more 2 us of
    // the walk over them: at least four chunks, and about the square root of a
    // third of a request's (one request of 512 chunks, 2 heads: 9 chunks a segment
    // 235 us, 13 242 us, 18 274 us, 26 342 us).
    while (seg < 4 || 3 * seg * seg * num_seqs < chunks) ++seg;
    return (int32_t)(kPreC * seg);
}

hipError_t launch_prefill(const DeltaProblem &p, int in_dt, hipStream_t stream) {
    if (p.seg != 0) {
        hipError_t e = launch_pass(p, in_dt, PrePass::sums, stream);
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)(p.req.num_seqs * p.H), (unsigned)(p.V / 16));
        if (p.K == 64)
            hipLaunchKernelGGL((kda_prefill_join_kernel<64>), grid, dim3(256), 0, stream, p);
        else
            hipLaunchKernelGGL((kda_prefill_join_kernel<128>), grid, dim3(512), 0, stream, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // Up to a workgroup per compute unit (of the segments, p.segs - num_seqs at
    // least exist): 256 walks of 512 tokens 127 us with roles and 152 without,
    // 320 walks 221 and 190, 1,024 walks 465 and 453 (K = 128, bf16).
    const int64_t parts = p.seg != 0 ? p.segs - p.req.num_seqs : p.req.num_seqs;
    const int64_t walks = parts * p.H;
    const PrePass pass = walks * column_blocks<1>(p.V) <= kUnits   ? PrePass::narrow
                         : walks * column_blocks<2>(p.V) <= kUnits ? PrePass::roles
                                                                : PrePass::whole;
    return launch_pass(p, in_dt, pass, stream);
}

}  // namespace kda
