// Causal convolution of a prompt's queries, keys and values for gfx950 (the
// decode step's first stage, for whole packed requests):
//   y_p[t] = silu(sum_{w<W} conv_w[p][w] x_p[t - (W - 1) + w]),  p = q, k, v
//   q, k: y / sqrt(|y|^2 + eps) over the d channels of a head;  v: y
// with x before a request's first token taken from its window in the pool (or
// zero), and the window left holding the last W - 1 inputs.
//
// Bound by memory: every input is read once, every output written once. A
// wavefront owns 512 adjacent channels of one projection (lane: 8 channels, a
// 16-byte access of 16-bit elements) and walks `seg` tokens of the packed
// batch with the last W - 1 inputs in registers, so a segment reads W - 1
// rows besides its own. The norms are DPP sums over the d / 8 lanes of a head.
// 16 x 512 tokens, 64 heads of 128, W = 4, bf16: 148 us, 5.4 TB/s of its 805 MB
// (a tuned copy reaches 6.4); 64 tokens: 6.5 us, a launch and two dependent loads.
//
// The window of a request is read and written by the wavefront whose segment
// holds the request's first token, in that order and each channel by one
// lane; it also computes the request's first W - 1 rows where they reach into
// the next segment, so no other wavefront needs the old window and no read
// can meet the write. Requests of no tokens belong to the segment in which
// they would start.
#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

constexpr int kConvThreads = 256;
constexpr float kLog2E = 1.4426950408889634f;
constexpr int kConvWaves = kConvThreads / kWave;

// Number of requests that start before row t (wave-uniform t and result):
// the wave compares 64 spread entries of cu_seqlens at a time and narrows the
// range to one of 65 parts, two rounds for 4,096 requests.
__device__ __forceinline__ int requests_before(const int32_t *cu, int n, int t, int lane) {
    int lo = 0, hi = n;  // cu[i] < t for i < lo; cu[i] >= t for i >= hi
    while (lo < hi) {
        const int step = (hi - lo + kWave - 1) / kWave;
        const int i = lo + lane * step;
        const bool before = i < hi && cu[i] < t;
        const int m = __popcll(__ballot(before));  // entries lo, lo + step, ... below t
        if (m == 0) return lo;
        const int top = lo + m * step;
        lo = lo + (m - 1) * step + 1;
        hi = min(hi, top);
    }
    return lo;
}

template <class E, int D, int W>
__global__ __launch_bounds__(kConvThreads) void kda_conv_prefill_kernel(ConvProblem p) {
    typedef typename E::T T;
    const int lane = threadIdx.x & (kWave - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int width = p.H * D;  // channels of one projection
    const int groups = (width + 8 * kWave - 1) / (8 * kWave);
    const long item = (long)blockIdx.x * kConvWaves + wv;
    const int proj = (int)(item % 3);
    const long rest = item / 3;
    const int grp = (int)(rest % groups);
    const long t_first = rest / groups * p.seg;
    const int T_all = p.req.total_tokens;
    if (t_first >= T_all && t_first > 0) return;  // one segment stays for requests of no tokens
    const int t0 = (int)t_first, t1 = (int)min(t_first + p.seg, (long)T_all);
    const int ch = grp * 8 * kWave + lane * 8;
    const bool live = ch < width;  // whole heads: width is a multiple of D
    const int c = live ? ch : 0;   // other lanes read valid channels and store nothing

    const T *x = static_cast<const T *>(p.qkv) + (long)proj * width + c;
    const long xrow = 3L * width;
    T *out = static_cast<T *>(p.out[proj]) + c;
    float tap[W][8];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            tap[w][e] = p.conv_w[((long)proj * W + w) * width + c + e];

    const bool keep = p.pool.base != nullptr;
    const int N = p.req.num_seqs;
    float win[W - 1][8];  // the W - 1 inputs before the next token, oldest first
    bool pad = false;

    auto row_in = [&](int t, float (&v)[8]) {
        Raw8<E> r;
        r.load(x + (long)t * xrow);
        r.widen(v);
    };
    auto pool_at = [&](int slot, int w) {
        return p.pool.base + ((((long)slot * 3 + proj) * p.H) * (W - 1)) * (long)D +
               ((long)(c / D) * (W - 1) + w) * D + c % D;
    };
    // the window before the first token of request n
    auto past_window = [&](int n, int slot) {
        const bool cont = slot >= 0 && request_continues(p.pool, n);
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) win[w][e] = cont ? pool_at(slot, w)[e] : 0.0f;
    };
    // request n starts here: its window, and the one it leaves in the pool
    auto begin = [&](int n) {
        const int2 rows = request_rows(p.req, n);
        const int slot = keep ? request_slot(p.pool, n) : -1;
        pad = keep && slot < 0;
        past_window(n, slot);
        if (slot < 0 || !live) return;
        float left[W - 1][8];
        if (rows.y >= W - 1) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w) row_in(rows.x + rows.y - (W - 1) + w, left[w]);
        } else {  // the old window, shifted by the few rows there are
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) left[w][e] = win[w][e];
            for (int i = 0; i < rows.y; ++i) {
                float v[8];
                row_in(rows.x + i, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int w = 0; w + 1 < W - 1; ++w) left[w][e] = left[w + 1][e];
                    left[W - 2][e] = v[e];
                }
            }
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            f4 *dst = reinterpret_cast<f4 *>(pool_at(slot, w));
            dst[0] = f4{left[w][0], left[w][1], left[w][2], left[w][3]};
            dst[1] = f4{left[w][4], left[w][5], left[w][6], left[w][7]};
        }
    };

    auto start_of = [&](int n) {
        return p.req.cu ? min(max(p.req.cu[n], 0), T_all) : n * p.req.seq_len;
    };
    auto end_of = [&](int n) {
        const int2 rows = request_rows(p.req, n);
        return rows.x + rows.y;
    };
    // Rows a .. b - 1 of the current request, U at a time, the next U loaded
    // before the present ones are used.
    constexpr int U = 4;
    Raw8<E> blk[U];
    int ready = t0;  // the first row in blk
    auto load_rows = [&](Raw8<E>(&r)[U], int t, int last) {
#pragma unroll
        for (int i = 0; i < U; ++i) r[i].load(x + (long)min(t + i, last) * xrow);
    };
    auto run = [&](int a, int b) {
        if (ready != a) load_rows(blk, a, b - 1);
        for (int t = a; t < b; t += U) {
            float v[U][8];
#pragma unroll
            for (int i = 0; i < U; ++i) blk[i].widen(v[i]);
            if (t + U < b) load_rows(blk, t + U, b - 1);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (t + i >= b) break;
                // inputs i - (W - 1) .. i: from the window while negative
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float s = tap[W - 1][e] * v[i][e];
#pragma unroll
                    for (int w = 0; w < W - 1; ++w) {
                        const int at = i - (W - 1) + w;
                        s = __builtin_fmaf(tap[w][e], at < 0 ? win[W - 1 + at][e] : v[at][e], s);
                    }
                    // silu (rcp, exp2 and rsq below are within 1 ulp)
                    y[e] = s * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s * -kLog2E));
                }
                if (proj < 2) {
                    float ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(y[e], y[e], ss);
                    ss = D == 128 ? sum16(ss) : sum8(ss);
                    const float r = __builtin_amdgcn_rsqf(ss + p.eps_l2);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= r;
                }
                if (pad) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
                }
                if (live) Raw8<E>::store(out + (long)(t + i) * width, y);
            }
            // the window behind a whole block (after a part of one the run ends:
            // another run begins with another request, or there is none)
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) win[w][e] = v[U - (W - 1) + w][e];
        }
        ready = -1;
    };

    // the first rows, of whatever request, while their request is looked up
    Raw8<E> halo[W - 1];
    const bool any_row = T_all > 0;
    if (any_row) {
        load_rows(blk, t0, T_all - 1);
#pragma unroll
        for (int w = 0; w < W - 1; ++w) halo[w].load(x + (long)max(t0 - (W - 1) + w, 0) * xrow);
    }
    // the request that row t0 lies in, and the next one to start
    int t = t0, cur_bos = 0, cur_end = 0;  // rows [cur_bos, cur_end) of the current request
    int next = 0;  // (dense requests of no tokens all start at row 0)
    if (p.req.cu)
        next = requests_before(p.req.cu, N, t0, lane);
    else if (p.req.seq_len > 0)
        next = (t0 + p.req.seq_len - 1) / p.req.seq_len;
    next = __builtin_amdgcn_readfirstlane(next);
    if (next > 0 && end_of(next - 1) > t0) {  // inside request next - 1
        cur_bos = start_of(next - 1);
        cur_end = end_of(next - 1);
        pad = keep && request_slot(p.pool, next - 1) < 0;
        // its first W - 1 rows need the window of the pool: they belong to
        // the wavefront that begins the request (below)
        t = max(t0, min(cur_bos + W - 1, cur_end));
        if (t == t0) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w) halo[w].widen(win[w]);
        } else if (t < cur_end) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w) row_in(t - (W - 1) + w, win[w]);
        }
        cur_bos = INT32_MIN / 2;  // not begun here
    }
    while (t < t1) {
        while (next < N && start_of(next) <= t) {
            begin(next);
            cur_bos = start_of(next);
            cur_end = end_of(next);
            ++next;
        }
        if (t < cur_end) {
            // to the segment's end, or through the first W - 1 rows of a
            // request that begins here
            const int stop = min(cur_end, max(t1, cur_bos + W - 1));
            run(t, stop);
            t = stop;
        } else {
            t = next < N ? min(t1, start_of(next)) : t1;  // no request's rows
        }
    }
    if (t1 == T_all)  // requests of no tokens behind the last row
        while (next < N) begin(next++);
}

hipError_t launch_conv(const ConvProblem &p0, int in_dt, hipStream_t stream) {
    ConvProblem p = p0;
    const long groups = ((long)p.H * p.d + 8 * kWave - 1) / (8 * kWave);
    const long tokens = p.req.total_tokens > 0 ? p.req.total_tokens : 1;
    // Tokens per wavefront: 16 (W - 1 rows read twice in 16: 8,192 tokens, 64
    // heads, bf16 150 us; 8: 157, 32: 162), fewer while the launch would leave
    // the compute units short of wavefronts (512 tokens 13.2 us with 8, 14.1
    // with 16; 64 tokens 7.0 with 4, 10.4 with 16).
    const long want = 8 * device_cus();
    p.seg = 16;
    while (p.seg > 4 && (tokens + p.seg - 1) / p.seg * groups * 3 < want) p.seg /= 2;
    const long waves = (tokens + p.seg - 1) / p.seg * groups * 3;
    const long blocks = (waves + kConvWaves - 1) / kConvWaves;
    if (blocks > (long)(UINT32_MAX / kConvThreads)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks);
    auto with_w = [&]<class E, int D>() {
        if (p.W == 2)
            hipLaunchKernelGGL((kda_conv_prefill_kernel<E, D, 2>), grid, dim3(kConvThreads), 0,
                               stream, p);
        else if (p.W == 3)
            hipLaunchKernelGGL((kda_conv_prefill_kernel<E, D, 3>), grid, dim3(kConvThreads), 0,
                               stream, p);
        else
            hipLaunchKernelGGL((kda_conv_prefill_kernel<E, D, 4>), grid, dim3(kConvThreads), 0,
                               stream, p);
        return hipGetLastError();
    };
    auto with_d = [&]<class E>() {
        return p.d == 64 ? with_w.template operator()<E, 64>()
                         : with_w.template operator()<E, 128>();
    };
    return in_dt == 0   ? with_d.template operator()<F32>()
           : in_dt == 1 ? with_d.template operator()<BF16>()
                        : with_d.template operator()<F16>();
}

}  // namespace kda
