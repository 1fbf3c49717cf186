// Gradients of a prompt's causal convolution for gfx950. With a the taps' sum,
// y = a sigmoid(a), n = y / sqrt(|y|^2 + eps) (queries, keys; v = y):
//   dy = (dn - n (n.dn)) / sqrt(|y|^2 + eps) (values: dy = dv)
//   da = dy s (1 + a (1 - s)),  s = sigmoid(a)
//   dx[t] = sum_w taps[w] da[t + W - 1 - w],   dtaps[w] = sum_t da[t] x[t - W + 1 + w]
// over a request's own tokens; x before its first token is its window in the
// pool, whose gradient takes the terms that reach it, and the window left
// behind hands its gradient to the last W - 1 inputs. Inputs are a tensor or an
// 8-bit checkpoint.
//
// Bound by memory: two streams in, one out. A wavefront owns 512 adjacent
// channels of one projection (lane: 8) and walks `seg` tokens forwards with the
// last W - 1 inputs and the unfinished dx of W - 1 rows in registers; it takes
// W - 1 rows more on both sides, which its neighbours take, too. The four
// wavefronts of a workgroup walk adjacent segments, join their dtaps in LDS and
// leave one row in the workspace; a second launch adds the rows in order and
// puts the windows' gradients into the pool (which the first one still reads).
#include <hip/hip_runtime.h>

#include "code8.h"
#include "tril_launch.h"

namespace kda {

constexpr int kCgThreads = 256;
constexpr int kCgWaves = kCgThreads / kWave;

// Number of requests that end at or before row t (wave-uniform).
__device__ __forceinline__ int requests_ended(const Requests &r, int t, int lane) {
    if (r.cu == nullptr) return r.seq_len > 0 ? t / r.seq_len : r.num_seqs;
    int lo = 0, hi = r.num_seqs;
    while (lo < hi) {
        const int step = (hi - lo + kWave - 1) / kWave;
        const int i = lo + lane * step;
        const bool ended = i < hi && r.cu[i + 1] <= t;
        const int m = __popcll(__ballot(ended));
        if (m == 0) break;
        const int top = lo + m * step;
        lo = lo + (m - 1) * step + 1;
        hi = min(hi, top);
    }
    return lo;
}

template <class E, class EX, int D, int W>
__global__ __launch_bounds__(kCgThreads) void kda_conv_grad_kernel(ConvGradProblem p) {
    typedef typename E::T T;
    constexpr bool kCoded = sizeof(typename EX::T) == 1;
    __shared__ float joined[kCgWaves][8 * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int width = p.H * D;
    const int groups = (width + 8 * kWave - 1) / (8 * kWave);
    const int proj = (int)(blockIdx.x % 3);
    const int grp = (int)(blockIdx.x / 3 % groups);
    const long block = blockIdx.x / 3 / groups;
    const long t_first = (block * kCgWaves + wv) * p.seg;
    const int T_all = p.req.total_tokens;
    const int t0 = (int)min(t_first, (long)T_all), t1 = (int)min(t_first + p.seg, (long)T_all);
    const int ch = grp * 8 * kWave + lane * 8;
    const bool live = ch < width;  // whole heads: width is a multiple of D
    const int c = live ? ch : 0;   // other lanes read valid channels and store nothing
    const bool unit = proj < 2;

    const T *dout = static_cast<const T *>(p.dout[proj]) + c;
    const typename EX::T *xin = static_cast<const typename EX::T *>(p.qkv) + (long)proj * width + c;
    T *dx = static_cast<T *>(p.dqkv) + (long)proj * width + c;
    const long xrow = 3L * width;
    float tap[W][8], dtap[W][8];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            tap[w][e] = p.conv_w[((long)proj * W + w) * width + c + e];
            dtap[w][e] = 0.0f;
        }
    auto row_in = [&](int t, float (&v)[8]) {
        Raw8<EX> r;
        r.load(xin + (long)t * xrow);
        r.widen(v);
        if constexpr (kCoded) {
            const float s = p.qkv_scale[((long)t * 3 + proj) * p.H + c / D];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= s;
        }
    };
    auto window = [&](long slot, int w) {
        return ((slot * 3 + proj) * p.H + c / D) * (W - 1) * D + (long)w * D + c % D;
    };

    for (int n = t0 < t1 ? requests_ended(p.req, t0, lane) : p.req.num_seqs; n < p.req.num_seqs;
         ++n) {
        const int2 rows = request_rows(p.req, n);
        const int b = rows.x, end = rows.x + rows.y;
        if (b >= t1) break;
        const int s = max(b, t0), f = min(end, t1);
        if (s >= f) continue;
        const int slot = p.grad.slot != nullptr || p.pool.base != nullptr || p.grad.base != nullptr
                             ? request_slot(p.grad, n) : 0;
        if (slot < 0) {  // padding
            float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (live)
                for (int t = s; t < f; ++t) Raw8<E>::store(dx + (long)t * xrow, zero);
            continue;
        }
        const bool cont = request_continues(p.pool, n);
        float win[W][8], acc[W][8];  // inputs t - W + 1 .. t; dx of rows t - W + 1 .. t
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) win[w][e] = acc[w][e] = 0.0f;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int t = s - (W - 1) + w;
            if (t >= b) {
                row_in(t, win[w]);
            } else if (cont) {
                const float *old = p.pool.base + window(slot, t - b + W - 1);
#pragma unroll
                for (int e = 0; e < 8; ++e) win[w][e] = old[e];
            }
        }
        // row r is complete: to dx, or, in front of the request, to its window
        auto leave = [&](int r, float (&v)[8]) {
            if (!live) return;
            const bool mine = r >= s && r < f, before = s == b && r < b;
            if (!mine && !before) return;
            const int j = r - (end - (W - 1));
            if (p.grad.base != nullptr && j >= 0) {
                const float *d = p.grad.base + window(slot, j);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += d[e];
            }
            if (mine) {
                Raw8<E>::store(dx + (long)r * xrow, v);
            } else if (p.grad.base != nullptr) {
                float *d = p.old + window(n, r - b + W - 1);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = v[e];
            }
        };
        const int stop = min(end, f + W - 1);
        for (int t = s; t < stop; ++t) {
            float dn[8], y[8], a[8];
            Raw8<E> rd;
            rd.load(dout + (long)t * width);
            row_in(t, win[W - 1]);
            rd.widen(dn);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) sum = __builtin_fmaf(tap[w][e], win[w][e], sum);
                const float em = __expf(-sum), sg = 1.0f / (1.0f + em);
                y[e] = sum * sg;
                // the slope s (1 + a (1 - s)), with 1 - s = em s
                a[e] = em < __builtin_inff() ? sg * (1.0f + sum * (em * sg)) : sum * 0.0f;
                ss = __builtin_fmaf(y[e], y[e], ss);
                dot = __builtin_fmaf(y[e], dn[e], dot);
            }
            if (unit) {
                ss = D == 128 ? sum16(ss) : sum8(ss);
                dot = D == 128 ? sum16(dot) : sum8(dot);
                const float r = 1.0f / __builtin_sqrtf(ss + p.eps_l2), rr = r * r * dot;
#pragma unroll
                for (int e = 0; e < 8; ++e) dn[e] = r * (dn[e] - y[e] * rr);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] *= dn[e];
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (t < f) dtap[w][e] = __builtin_fmaf(a[e], win[w][e], dtap[w][e]);
                    acc[w][e] = __builtin_fmaf(tap[w][e], a[e], acc[w][e]);
                }
            leave(t - (W - 1), acc[0]);
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    win[w][e] = win[w + 1][e];
                    acc[w][e] = acc[w + 1][e];
                }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[W - 1][e] = 0.0f;
        }
        if (stop == end) {  // the last rows, which no later token adds to
#pragma unroll
            for (int w = 0; w < W - 1; ++w) leave(end - (W - 1) + w, acc[w]);
        }
    }

    // dtaps of the workgroup's segments
#pragma unroll
    for (int w = 0; w < W; ++w) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) joined[wv][lane * 8 + e] = dtap[w][e];
        __syncthreads();
        for (int e = threadIdx.x; e < 8 * kWave; e += kCgThreads) {
            const int at = grp * 8 * kWave + e;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kCgWaves; ++i) sum += joined[i][e];
            if (at < width) p.part[(block * 3 + proj) * (long)W * width + (long)w * width + at] = sum;
        }
    }
}

// dtaps: the sum of the workgroups' rows. Windows: what the first launch left,
// or zeros where a request starts from zeros.
__global__ __launch_bounds__(kCgThreads) void kda_conv_grad_sum_kernel(ConvGradProblem p,
                                                                        long rows, long taps,
                                                                        unsigned tap_blocks) {
    if (blockIdx.x < tap_blocks) {
        const long e = (long)blockIdx.x * kCgThreads + threadIdx.x;
        if (e >= taps) return;
        float sum = 0.0f;
        for (long r = 0; r < rows; ++r) sum += p.part[r * taps + e];
        p.dconv_w[e] = sum;
        return;
    }
    const int n = (int)(blockIdx.x - tap_blocks);
    const int slot = request_slot(p.grad, n);
    if (slot < 0) return;
    const bool cont = request_continues(p.grad, n);
    const long size = 3L * p.H * (p.W - 1) * p.d;
    if (cont && request_rows(p.req, n).y == 0) return;  // handed on as it is
    for (long e = threadIdx.x; e < size; e += kCgThreads)
        p.grad.base[slot * size + e] = cont ? p.old[n * size + e] : 0.0f;
}

hipError_t launch_conv_grad(const ConvGradProblem &p, int dt, hipStream_t stream) {
    const long groups = ((long)p.H * p.d + 8 * kWave - 1) / (8 * kWave);
    const long rows = conv_grad_rows(p.req.total_tokens, p.seg);
    const long taps = 3L * p.W * p.H * p.d;
    if (rows > 0) {
        const dim3 grid((unsigned)(rows * groups * 3));
        auto with_w = [&]<class E, class EX, int D>() {
            const auto fn = p.W == 2   ? kda_conv_grad_kernel<E, EX, D, 2>
                            : p.W == 3 ? kda_conv_grad_kernel<E, EX, D, 3>
                                       : kda_conv_grad_kernel<E, EX, D, 4>;
            hipLaunchKernelGGL(fn, grid, dim3(kCgThreads), 0, stream, p);
            return hipGetLastError();
        };
        const hipError_t e = dispatch_dtypes<F32, BF16, F16>(dt, 0, [&]<class E, class EO>() {
            if (p.qkv_scale != nullptr)
                return p.d == 64 ? with_w.template operator()<E, I8, 64>()
                                 : with_w.template operator()<E, I8, 128>();
            return p.d == 64 ? with_w.template operator()<E, E, 64>()
                             : with_w.template operator()<E, E, 128>();
        });
        if (e != hipSuccess) return e;
    }
    const unsigned tap_blocks = (unsigned)((taps + kCgThreads - 1) / kCgThreads);
    const unsigned windows = p.grad.base != nullptr ? (unsigned)p.req.num_seqs : 0u;
    hipLaunchKernelGGL(kda_conv_grad_sum_kernel, dim3(tap_blocks + windows), dim3(kCgThreads), 0,
                       stream, p, rows, taps, tap_blocks);
    return hipGetLastError();
}

}  // namespace kda
