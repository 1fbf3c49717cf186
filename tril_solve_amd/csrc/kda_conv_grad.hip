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
// A wavefront owns 256 adjacent channels of one projection (lane: 4) and walks
// `seg` tokens forwards with the last W - 1 inputs and the unfinished dx of W - 1
// rows in registers; it takes W - 1 rows more on both sides, which its neighbours
// take, too. W tokens are unrolled, so the rings are registers; rows are loaded
// ahead by buffer loads whose row is a scalar. The four
// wavefronts of a workgroup walk adjacent segments, join their dtaps in LDS and
// leave one row in the workspace; a second launch adds the rows in order and
// puts the windows' gradients into the pool (which the first one still reads).
//
// Bound by the vector units: the silu, its derivative, 2 W products and the
// normalisation are 34 instructions to an element, and 84% of the cycles issue
// one. 16 x 512 tokens of 64 heads of 128, bf16 from 8-bit codes: 242 to 252 us (4.1 TB/s;
// one channel to a lane 431). 7,000 tokens of 9 heads of 64, f32: 50 us (2.9 TB/s).
#include <hip/hip_runtime.h>

#include "code8.h"
#include "tril_launch.h"

namespace kda {

constexpr int kCgThreads = 256;
constexpr int kCgWaves = kCgThreads / kWave;
constexpr int kCgChans = 4;  // channels of a lane

// Four adjacent elements.
template <class E>
struct Quad {
    w2 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const w2 *>(p); }
    __device__ __forceinline__ void widen(float (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = Elem<E>::widen(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&x)[4]) {
        const w2 o = {Elem<E>::pack(x[0], x[1]), Elem<E>::pack(x[2], x[3])};
        __builtin_nontemporal_store(o, reinterpret_cast<w2 *>(p));
    }
};
template <>
struct Quad<F32> {
    f4 w;
    __device__ __forceinline__ void load(const float *p) { w = *reinterpret_cast<const f4 *>(p); }
    __device__ __forceinline__ void widen(float (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = w[i];
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
        __builtin_nontemporal_store(f4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f4 *>(p));
    }
};
template <>
struct Quad<I8> {
    uint32_t w;
    __device__ __forceinline__ void load(const int8_t *p) {
        w = *reinterpret_cast<const uint32_t *>(p);
    }
    __device__ __forceinline__ void widen(float (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> 8 * i);
    }
};

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
__global__ __launch_bounds__(kCgThreads, 2) void kda_conv_grad_kernel(ConvGradProblem p) {
    typedef typename E::T T;
    constexpr bool kCoded = sizeof(typename EX::T) == 1;
    __shared__ float joined[kCgWaves][kCgChans * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int width = p.H * D;
    const int groups = (width + kCgChans * kWave - 1) / (kCgChans * kWave);
    const int proj = (int)(blockIdx.x % 3);
    const int grp = (int)(blockIdx.x / 3 % groups);
    const long block = blockIdx.x / 3 / groups;
    const long t_first = (block * kCgWaves + wv) * p.seg;
    const int T_all = p.req.total_tokens;
    const int t0 = (int)min(t_first, (long)T_all), t1 = (int)min(t_first + p.seg, (long)T_all);
    const int ch = grp * kCgChans * kWave + lane * kCgChans;
    const bool live = ch < width;  // whole heads: width is a multiple of D
    const int c = live ? ch : 0;   // other lanes read valid channels and store nothing
    const bool unit = proj < 2;

    // (rows are found in scalar registers, a lane adds its channel)
    const uint32_t lc = c;
    const T *dout = static_cast<const T *>(p.dout[proj]);
    const typename EX::T *xin = static_cast<const typename EX::T *>(p.qkv) + (long)proj * width;
    T *dx = static_cast<T *>(p.dqkv) + (long)proj * width;
    const float *scales = p.qkv_scale + (kCoded ? (long)proj * p.H : 0);
    const uint32_t head = lc / D;
    const long xrow = 3L * width;
    float tap[W][kCgChans], dtap[W][kCgChans];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int e = 0; e < kCgChans; ++e) {
            tap[w][e] = p.conv_w[((long)proj * W + w) * width + c + e];
            dtap[w][e] = 0.0f;
        }
    struct Row {  // an input and the gradient of its output, as loaded
        Quad<EX> x;
        Quad<E> d;
        float scale;
    };
    auto load_x = [&](int t, Row &r) {
        r.x.load(xin + (long)t * xrow + lc);
        r.scale = kCoded ? (scales + (long)t * 3 * p.H)[head] : 1.0f;
    };
    auto load_row = [&](int t, Row &r) {
        load_x(t, r);
        r.d.load(dout + (long)t * width + lc);
    };
    auto widen_x = [&](const Row &r, float (&v)[kCgChans]) {
        r.x.widen(v);
        if constexpr (kCoded)
#pragma unroll
            for (int e = 0; e < kCgChans; ++e) v[e] *= r.scale;
    };
    auto window = [&](long slot, int w) {
        return ((slot * 3 + proj) * p.H + c / D) * (W - 1) * D + (long)w * D + c % D;
    };

    for (int n = t0 < t1 ? requests_ended(p.req, t0, lane) : p.req.num_seqs; n < p.req.num_seqs;
         ++n) {
        int2 rows = request_rows(p.req, n);
        rows.x = __builtin_amdgcn_readfirstlane(rows.x);
        rows.y = __builtin_amdgcn_readfirstlane(rows.y);
        const int b = rows.x, end = rows.x + rows.y;
        if (b >= t1) break;
        const int s = max(b, t0), f = min(end, t1);
        if (s >= f) continue;
        const int slot = p.grad.slot != nullptr || p.pool.base != nullptr || p.grad.base != nullptr
                             ? request_slot(p.grad, n) : 0;
        if (slot < 0) {  // padding
            float zero[kCgChans] = {0, 0, 0, 0};
            if (live)
                for (int t = s; t < f; ++t) Quad<E>::store(dx + (long)t * xrow + lc, zero);
            continue;
        }
        const bool cont = request_continues(p.pool, n);
        float win[W][kCgChans], acc[W][kCgChans];  // inputs t - W + 1 .. t; dx of rows t - W + 1 .. t
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int e = 0; e < kCgChans; ++e) win[w][e] = acc[w][e] = 0.0f;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int t = s - (W - 1) + w;
            if (t >= b) {
                Row r;
                load_x(t, r);
                widen_x(r, win[w]);
            } else if (cont) {
                const float *old = p.pool.base + window(slot, t - b + W - 1);
#pragma unroll
                for (int e = 0; e < kCgChans; ++e) win[w][e] = old[e];
            }
        }
        // row r is complete: to dx, or, in front of the request, to its window
        auto leave = [&](int r, float (&v)[kCgChans]) {
            if (!live) return;
            const bool mine = r >= s && r < f, before = s == b && r < b;
            if (!mine && !before) return;
            const int j = r - (end - (W - 1));
            if (p.grad.base != nullptr && j >= 0) {
                const float *d = p.grad.base + window(slot, j);
#pragma unroll
                for (int e = 0; e < kCgChans; ++e) v[e] += d[e];
            }
            if (mine) {
                Quad<E>::store(dx + (long)r * xrow + lc, v);
            } else if (p.grad.base != nullptr) {
                float *d = p.old + window(n, r - b + W - 1);
#pragma unroll
                for (int e = 0; e < kCgChans; ++e) d[e] = v[e];
            }
        };
        // Token t, whose window's oldest entry and unfinished row are at place R of
        // the rings; in the segment itself also its share of dtaps.
        auto token = [&]<int R, bool OWN>(int t, const Row &row) {
            float dn[kCgChans], y[kCgChans], a[kCgChans];
            float(&xt)[kCgChans] = win[(R + W - 1) % W];
            widen_x(row, xt);
            row.d.widen(dn);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int e = 0; e < kCgChans; ++e) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    sum = __builtin_fmaf(tap[w][e], win[(R + w) % W][e], sum);
                const float em = __expf(-sum), sg = __builtin_amdgcn_rcpf(1.0f + em);
                y[e] = sum * sg;
                a[e] = sg + __builtin_fmaf(-y[e], sg, y[e]);  // the slope s + a s (1 - s)
                ss = __builtin_fmaf(y[e], y[e], ss);
                dot = __builtin_fmaf(y[e], dn[e], dot);
            }
            if (unit) {
                ss = D == 128 ? add_rows16(sum16(ss)) : sum16(ss);
                dot = D == 128 ? add_rows16(sum16(dot)) : sum16(dot);
                const float r = __builtin_amdgcn_rsqf(ss + p.eps_l2), rr = r * r * dot;
#pragma unroll
                for (int e = 0; e < kCgChans; ++e) dn[e] = r * __builtin_fmaf(-y[e], rr, dn[e]);
            }
#pragma unroll
            for (int e = 0; e < kCgChans; ++e) a[e] *= dn[e];
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int e = 0; e < kCgChans; ++e) {
                    if constexpr (OWN)
                        dtap[w][e] = __builtin_fmaf(a[e], win[(R + w) % W][e], dtap[w][e]);
                    float &to = acc[(R + w) % W][e];
                    to = w == W - 1 ? tap[w][e] * a[e] : __builtin_fmaf(tap[w][e], a[e], to);
                }
            leave(t - (W - 1), acc[R]);
        };
        // W tokens at a time, whose places in the rings are known; their successors
        // are loaded meanwhile
        int t = s;
        if (t + W <= f) {
            Row rows_[W];
#pragma unroll
            for (int i = 0; i < W; ++i) load_row(t + i, rows_[i]);
            for (; t + W <= f; t += W) {
                Row next[W];
#pragma unroll
                for (int i = 0; i < W; ++i) load_row(min(t + W + i, end - 1), next[i]);
                token.template operator()<0, true>(t, rows_[0]);
                token.template operator()<1, true>(t + 1, rows_[1]);
                if constexpr (W > 2) token.template operator()<2, true>(t + 2, rows_[2]);
                if constexpr (W > 3) token.template operator()<3, true>(t + 3, rows_[3]);
#pragma unroll
                for (int i = 0; i < W; ++i) rows_[i] = next[i];
            }
        }
        const int stop = min(end, f + W - 1);
        for (; t < stop; ++t) {
            Row row;
            load_row(t, row);
            if (t < f)
                token.template operator()<0, true>(t, row);
            else
                token.template operator()<0, false>(t, row);
#pragma unroll
            for (int e = 0; e < kCgChans; ++e) {
                const float w0 = win[0][e], a0 = acc[0][e];
#pragma unroll
                for (int w = 0; w < W - 1; ++w) {
                    win[w][e] = win[w + 1][e];
                    acc[w][e] = acc[w + 1][e];
                }
                win[W - 1][e] = w0;
                acc[W - 1][e] = a0;
            }
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
        for (int e = 0; e < kCgChans; ++e) joined[wv][lane * kCgChans + e] = dtap[w][e];
        __syncthreads();
        for (int e = threadIdx.x; e < kCgChans * kWave; e += kCgThreads) {
            const int at = grp * kCgChans * kWave + e;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kCgWaves; ++i) sum += joined[i][e];
            if (at < width) p.part[(block * 3 + proj) * (long)W * width + (long)w * width + at] = sum;
        }
    }
}

// dtaps: the sum of the workgroups' rows, four floats to a lane. Windows: what the
// first launch left, or zeros where a request starts from zeros; a workgroup to
// kConvGradPart floats.
static_assert(kConvGradPart == 4 * kCgThreads);
__global__ __launch_bounds__(kCgThreads) void kda_conv_grad_sum_kernel(ConvGradProblem p, int rows,
                                                                        long taps,
                                                                        unsigned tap_blocks,
                                                                        unsigned parts) {
    if (blockIdx.x < tap_blocks) {
        const long e = ((long)blockIdx.x * kCgThreads + threadIdx.x) * 4;
        if (e >= taps) return;
        f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int r = 0; r < rows; ++r) sum += *reinterpret_cast<const f4 *>(p.part + r * taps + e);
        *reinterpret_cast<f4 *>(p.dconv_w + e) = sum;
        return;
    }
    const int n = (int)((blockIdx.x - tap_blocks) / parts);
    const long at = (blockIdx.x - tap_blocks) % parts * kConvGradPart + threadIdx.x * 4L;
    const long size = 3L * p.H * (p.W - 1) * p.d;  // a multiple of 4
    const int slot = request_slot(p.grad, n);
    if (slot < 0 || at >= size) return;
    const bool cont = request_continues(p.grad, n);
    if (cont && request_rows(p.req, n).y == 0) return;  // handed on as it is
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (cont) v = *reinterpret_cast<const f4 *>(p.old + n * size + at);
    *reinterpret_cast<f4 *>(p.grad.base + slot * size + at) = v;
}

hipError_t launch_conv_grad(const ConvGradProblem &p, int dt, hipStream_t stream) {
    const long groups = ((long)p.H * p.d + kCgChans * kWave - 1) / (kCgChans * kWave);
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
    const unsigned tap_blocks = (unsigned)conv_grad_tap_blocks(p.H, p.d, p.W);
    const unsigned parts = (unsigned)conv_grad_window_blocks(p.H, p.d, p.W);
    const unsigned windows = p.grad.base != nullptr ? (unsigned)p.req.num_seqs : 0u;
    hipLaunchKernelGGL(kda_conv_grad_sum_kernel, dim3(tap_blocks + windows * parts),
                       dim3(kCgThreads), 0, stream, p, (int)rows, taps, tap_blocks, parts);
    return hipGetLastError();
}

}  // namespace kda
