// Gated delta rule, token by token, for a few tokens per request (decoding,
// drafted tokens, short extensions of a prompt), on gfx950.
//
// Per request and value head, with S the K x V FP32 state:
//   S <- diag(exp(g_t)) S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T
//   o_t = scale * S^T q_t = scale * ((decayed S)^T q_t + (k_t . q_t) u)
// so one pass over the state per token gives both products.
//
// The state rules the traffic (64 KiB read and written per request and head
// at K = V = 128, against about 1.3 KiB per token), and its value columns are
// independent of each other: each wavefront keeps 32 columns of all K rows in
// registers from the first token to the last (lane l: columns 4 (l % 8) .. +3
// of rows (K / 8)(l / 8) .. ), and a workgroup holds the V / 32 wavefronts of
// one (request, head), which share the staged keys, queries and decays.
// 32 requests of one token, 32 heads, K = V = 128, bf16: 21.2 us, 6.4 TB/s of
// its 136 MB. 24 requests of up to 8 tokens, 16 heads: 17.2 us, of which 10 are
// the state's traffic and the rest the chain of 8 tokens (about 1 us each;
// 16-byte reads of the staged rows did not shorten it).
#include <hip/hip_runtime.h>

#include "layer_device.h"

namespace kda {

constexpr int kRecTokens = 8;  // tokens staged in LDS at a time

template <class EI, int K>
__global__ __launch_bounds__(512) void kda_recurrent_kernel(DeltaProblem p) {
    constexpr int R = K / 8;       // state rows per lane
    constexpr int KP = K + K / R;  // padded rows: the 8 rows read at once in distinct banks
    __shared__ float kq[kRecTokens][3][KP];  // key, query, decay of each staged token
    __shared__ __align__(16) float vs[kRecTokens][256];
    __shared__ float bt[kRecTokens], dot[kRecTokens];
    typedef typename EI::T T;

    const int n = blockIdx.x / p.H, h = blockIdx.x - n * p.H;
    const int hk = h / (p.H / p.Hk);
    const int tid = threadIdx.x, l = tid & (kWave - 1), nt = blockDim.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave), nw = nt / kWave;
    const int2 rows = request_rows(p.req, n);
    const bool keep = p.pool.base != nullptr;
    const int slot = keep ? request_slot(p.pool, n) : 0;
    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k);
    const T *v = static_cast<const T *>(p.v);
    const int col = 32 * wv + 4 * (l & 7), r0 = R * (l >> 3);

    auto store_out = [&](long row, f4 o) {
        const long at = (row * p.H + h) * p.V + col;
        if (p.out_dt == 0) {
            *reinterpret_cast<f4 *>(static_cast<float *>(p.out) + at) = o;
        } else {
            const w2 w = p.out_dt == 1
                             ? w2{Elem<BF16>::pack(o[0], o[1]), Elem<BF16>::pack(o[2], o[3])}
                             : w2{Elem<F16>::pack(o[0], o[1]), Elem<F16>::pack(o[2], o[3])};
            *reinterpret_cast<w2 *>(static_cast<uint16_t *>(p.out) + at) = w;
        }
    };
    if (slot < 0) {  // padding: zero outputs, no state
        if (l < 8)
            for (int t = 0; t < rows.y; ++t) store_out(rows.x + t, f4{0.0f, 0.0f, 0.0f, 0.0f});
        return;
    }
    float *S = p.pool.base + (((long)slot * p.H + h) * K + r0) * p.V + col;
    f4 s[R];
    if (request_continues(p.pool, n)) {
        // the small inputs of the first tokens are loaded below while the
        // state is in flight
#pragma unroll
        for (int i = 0; i < R; ++i)
            s[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(S + (long)i * p.V));
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    for (int t0 = 0; t0 < rows.y; t0 += kRecTokens) {
        const int cnt = min(kRecTokens, rows.y - t0);
        const long row0 = rows.x + t0;
        if (t0) __syncthreads();  // the previous tokens' reads are done
        for (int i = tid; i < cnt * K; i += nt) {
            const int t = i / K, c = i - t * K, at = c + c / R;
            const long rk = ((row0 + t) * p.Hk + hk) * K + c;
            kq[t][0][at] = Elem<EI>::one(k + rk);
            kq[t][1][at] = Elem<EI>::one(q + rk);
            kq[t][2][at] = __expf(p.g[((row0 + t) * p.H + h) * (long)p.gate_stride +
                                      (p.gate_stride == 1 ? 0 : c)]);
        }
        for (int i = tid; i < cnt * p.V; i += nt) {
            const int t = i / p.V, c = i - t * p.V;
            vs[t][c] = Elem<EI>::one(v + ((row0 + t) * p.H + h) * p.V + c);
        }
        if (tid < cnt) bt[tid] = p.beta[(row0 + tid) * p.H + h];
        __syncthreads();
        for (int t = wv; t < cnt; t += nw) {
            float d = 0.0f;
#pragma unroll
            for (int c = l; c < K; c += kWave) d += kq[t][0][c + c / R] * kq[t][1][c + c / R];
            d = sum64(d);
            if (l == 0) dot[t] = d;
        }
        __syncthreads();
        for (int t = 0; t < cnt; ++t) {
            const float *kt = kq[t][0] + r0 + (l >> 3), *qt = kq[t][1] + r0 + (l >> 3);
            const float *at = kq[t][2] + r0 + (l >> 3);
            f4 pa = {0.0f, 0.0f, 0.0f, 0.0f}, pb = pa;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                s[i] *= at[i];
                pa += s[i] * kt[i];
                pb += s[i] * qt[i];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // over the 8 lanes with the same l % 8
                pa[j] = add_rows32(add_rows16(lane_add<0x128>(pa[j])));
                pb[j] = add_rows32(add_rows16(lane_add<0x128>(pb[j])));
            }
            const f4 u = bt[t] * (*reinterpret_cast<const f4 *>(&vs[t][col]) - pa);
#pragma unroll
            for (int i = 0; i < R; ++i) s[i] += kt[i] * u;
            if (l < 8) store_out(row0 + t, (pb + dot[t] * u) * p.scale);
        }
    }
    if (keep) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            __builtin_nontemporal_store(s[i], reinterpret_cast<f4 *>(S + (long)i * p.V));
    }
}

hipError_t launch_recurrent(const DeltaProblem &p, int in_dt, hipStream_t stream) {
    const dim3 grid((unsigned)(p.req.num_seqs * p.H)), block((unsigned)(2 * p.V));
    auto go = [&](auto e) {
        using EI = decltype(e);
        if (p.K == 64)
            hipLaunchKernelGGL((kda_recurrent_kernel<EI, 64>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((kda_recurrent_kernel<EI, 128>), grid, block, 0, stream, p);
        return hipGetLastError();
    };
    return in_dt == 0 ? go(F32{}) : in_dt == 1 ? go(BF16{}) : go(F16{});
}

}  // namespace kda
