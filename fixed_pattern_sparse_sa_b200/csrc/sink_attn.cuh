// sink_attn.cuh -- sliding-window attention with sinks: the first `sinks` keys
// of a sequence stay visible beside the last `window` ones.
//
//   V(p) = { j <= min(p, n_k - 1) : p - j < window or j < sinks }
//   z_j = scale q.k_j,  lse = log sum exp z,  out = sum exp(z_j - lse) v_j
//   P = exp(z - lse), D = dout.out, dS = P (dout.v - D)
//   dq = scale sum_j dS k_j,  dk_j = scale sum dS q,  dv_j = sum P dout
#pragma once

#include <cuda_fp16.h>

#include "sa_common.cuh"

namespace sa {

struct SinkParams {
    const void *q, *k, *v, *dout, *o;
    long long q_s[3], k_s[3], v_s[3], o_s[3], do_s[3], lse_s[3];   // batch, token, head strides (elements)
    const int32_t *cu_q, *cu_k;                  // packed: [B + 1] each; NULL: dense
    int B, Hq, Hkv, G;
    int window, sinks;
    long long Tq, L;                             // dense: per sequence; packed: rows of the batch
    long long q_pos0, max_q, max_k;
    float scale, scale_log2;
    void *out;
    float *lse;                                  // the forward's result
    const float *lse_in;                         // the backward's input
    void *dq, *dk, *dv;
    float2 *stat;                                // [rows of q, Hq] lse in base 2 and D = dout . out
    unsigned *err;
};

// Rows of one sequence: queries [q0, q0 + nq) and keys [k0, k0 + nk) of the
// batch, the position of its first query.  A cu that decreases, leaves the
// batch or gives a length above its bound is clamped and reported.
struct SinkSeq {
    long long q0, k0, pos0;
    int nq, nk;
};
__device__ __forceinline__ SinkSeq sink_seq(const SinkParams &p, int b) {
    SinkSeq s;
    if (!p.cu_q) {
        s.q0 = s.k0 = 0;
        s.nq = (int)p.Tq;
        s.nk = (int)p.L;
        s.pos0 = p.q_pos0;
        return s;
    }
    auto ends = [&](const int32_t *cu, long long rows, long long bound, long long &lo) -> int {
        const long long a = __ldg(cu + b), e = __ldg(cu + b + 1);
        long long c = a < 0 ? 0 : a > rows ? rows : a;
        long long f = e < c ? c : e > rows ? rows : e;
        if (bound > 0 && f - c > bound) f = c + bound;
        if (c != a || f != e) raise_error(p.err, ERR_BAD_INDEX);
        lo = c;
        return (int)(f - c);
    };
    s.nq = ends(p.cu_q, p.Tq, p.max_q, s.q0);
    s.nk = ends(p.cu_k, p.L, p.max_k, s.k0);
    s.pos0 = (long long)s.nk - s.nq;
    return s;
}
// Reports the sequences whose rows had to be clamped (by the first CTA).
__device__ __forceinline__ void sink_report(const SinkParams &p) {
    if (p.cu_q && blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) (void)sink_seq(p, b);
}
// Visible keys of position pos: [0, s1) and [lo, hi), s1 <= lo.
__device__ __forceinline__ void sink_visible(const SinkParams &p, int nk, long long pos, int &s1, int &lo, int &hi) {
    hi = pos < 0 ? 0 : (int)(pos + 1 < nk ? pos + 1 : nk);
    const long long w0 = pos - p.window + 1;
    lo = w0 <= 0 ? 0 : w0 < hi ? (int)w0 : hi;
    s1 = min(p.sinks, lo);
}
// The sequence that holds row r of the batch (-1: none), by bisection.
__device__ __forceinline__ int sink_find(const int32_t *cu, int B, long long r) {
    if (r < __ldg(cu) || r >= __ldg(cu + B)) return -1;
    int lo = 0, hi = B;                          // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (__ldg(cu + m) <= r) lo = m; else hi = m;
    }
    return lo;
}

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half(x); }

// two values as a packed pair, the first in the low half
template <typename T>
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return pack_bf16(lo, hi);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<unsigned *>(&h);
    }
}

// Per row and head: the lse in base 2 and D = dout . out.
template <typename T, int D>
__global__ void __launch_bounds__(128) sink_bwd_prep_kernel(const SinkParams p) {
    grid_dependency_sync();
    sink_report(p);
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long rows = (p.cu_q ? 1 : p.B) * p.Tq * p.Hq;
    for (long long w = blockIdx.x * 4ll + (threadIdx.x >> 5); w < rows; w += gridDim.x * 4ll) {
        const int h = (int)(w % p.Hq);
        const long long r = w / p.Hq, b = p.cu_q ? 0 : r / p.Tq, t = p.cu_q ? r : r % p.Tq;
        const T *g = (const T *)p.dout + b * p.do_s[0] + t * p.do_s[1] + h * p.do_s[2] + lane * E;
        const T *o = (const T *)p.o + b * p.o_s[0] + t * p.o_s[1] + h * p.o_s[2] + lane * E;
        float x = 0.f;
        for (int e = 0; e < E; ++e) x += to_f(g[e]) * to_f(o[e]);
        x = warp_sum(x);
        if (lane == 0)
            p.stat[w] = make_float2(p.lse_in[b * p.lse_s[0] + t * p.lse_s[1] + h * p.lse_s[2]] * kLog2e, x);
    }
}

// dq: one warp per query row and head.
template <typename T, int D>
__global__ void __launch_bounds__(128) sink_dq_rows_kernel(const SinkParams p) {
    grid_dependency_sync();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long rows = (p.cu_q ? 1 : p.B) * p.Tq * p.Hq;
    for (long long w = blockIdx.x * 4ll + (threadIdx.x >> 5); w < rows; w += gridDim.x * 4ll) {
        const int h = (int)(w % p.Hq), g = h / p.G;
        const long long r = w / p.Hq;
        const int b = p.cu_q ? sink_find(p.cu_q, p.B, r) : (int)(r / p.Tq);
        if (b < 0) continue;
        const SinkSeq s = sink_seq(p, b);
        const long long t = p.cu_q ? r - s.q0 : r % p.Tq;
        if (t < 0 || t >= s.nq) continue;
        const long long bq = p.cu_q ? 0 : b;
        const T *q = (const T *)p.q + bq * p.q_s[0] + (s.q0 + t) * p.q_s[1] + h * p.q_s[2] + lane * E;
        const T *dp = (const T *)p.dout + bq * p.do_s[0] + (s.q0 + t) * p.do_s[1] + h * p.do_s[2] + lane * E;
        const T *kb = (const T *)p.k + bq * p.k_s[0] + s.k0 * p.k_s[1] + g * p.k_s[2] + lane * E;
        const T *vb = (const T *)p.v + bq * p.v_s[0] + s.k0 * p.v_s[1] + g * p.v_s[2] + lane * E;
        float qf[E], gf[E], dq[E] = {};
        for (int e = 0; e < E; ++e) { qf[e] = to_f(q[e]); gf[e] = to_f(dp[e]); }
        const float l2 = p.stat[w].x, Dr = p.stat[w].y;
        int s1, lo, hi;
        sink_visible(p, s.nk, s.pos0 + t, s1, lo, hi);
        for (int j = s1 > 0 ? 0 : lo; j < hi; j = j + 1 == s1 ? lo : j + 1) {
            float z = 0.f, dP = 0.f;
            for (int e = 0; e < E; ++e) {
                z += qf[e] * to_f(kb[j * p.k_s[1] + e]);
                dP += gf[e] * to_f(vb[j * p.v_s[1] + e]);
            }
            const float dS = exp2f(warp_sum(z) * p.scale_log2 - l2) * (warp_sum(dP) - Dr);
            for (int e = 0; e < E; ++e) dq[e] += dS * to_f(kb[j * p.k_s[1] + e]);
        }
        T *out = (T *)p.dq + w * D + lane * E;
        for (int e = 0; e < E; ++e) out[e] = from_f<T>(dq[e] * p.scale);
    }
}

// dk, dv: one warp per key row and KV head, over the queries that see it.
template <typename T, int D>
__global__ void __launch_bounds__(128) sink_dkv_rows_kernel(const SinkParams p) {
    grid_dependency_sync();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long rows = (p.cu_q ? 1 : p.B) * p.L * p.Hkv;
    for (long long w = blockIdx.x * 4ll + (threadIdx.x >> 5); w < rows; w += gridDim.x * 4ll) {
        const int g = (int)(w % p.Hkv);
        const long long r = w / p.Hkv;
        const int b = p.cu_q ? sink_find(p.cu_k, p.B, r) : (int)(r / p.L);
        if (b < 0) continue;
        const SinkSeq s = sink_seq(p, b);
        const long long j = p.cu_q ? r - s.k0 : r % p.L;
        if (j < 0 || j >= s.nk) continue;
        const long long bq = p.cu_q ? 0 : b;
        const T *k = (const T *)p.k + bq * p.k_s[0] + (s.k0 + j) * p.k_s[1] + g * p.k_s[2] + lane * E;
        const T *v = (const T *)p.v + bq * p.v_s[0] + (s.k0 + j) * p.v_s[1] + g * p.v_s[2] + lane * E;
        float kf[E], vf[E], dk[E] = {}, dv[E] = {};
        for (int e = 0; e < E; ++e) { kf[e] = to_f(k[e]); vf[e] = to_f(v[e]); }
        // queries with j <= p, and p - j < window unless j is a sink
        const long long t0 = j > s.pos0 ? j - s.pos0 : 0;
        const long long end = j < p.sinks ? s.nq : j + p.window - s.pos0;
        const long long t1 = end < s.nq ? end : s.nq;
        for (long long t = t0; t < t1; ++t)
            for (int h = g * p.G; h < (g + 1) * p.G; ++h) {
                const T *q = (const T *)p.q + bq * p.q_s[0] + (s.q0 + t) * p.q_s[1] + h * p.q_s[2] + lane * E;
                const T *dp = (const T *)p.dout + bq * p.do_s[0] + (s.q0 + t) * p.do_s[1] + h * p.do_s[2] + lane * E;
                const long long row = (p.cu_q ? s.q0 + t : b * p.Tq + t) * p.Hq + h;
                float qf[E], gf[E], z = 0.f, dP = 0.f;
                for (int e = 0; e < E; ++e) {
                    qf[e] = to_f(q[e]); gf[e] = to_f(dp[e]);
                    z += qf[e] * kf[e];
                    dP += gf[e] * vf[e];
                }
                const float P = exp2f(warp_sum(z) * p.scale_log2 - p.stat[row].x);
                const float dS = P * (warp_sum(dP) - p.stat[row].y);
                for (int e = 0; e < E; ++e) { dk[e] += dS * qf[e]; dv[e] += P * gf[e]; }
            }
        T *dko = (T *)p.dk + w * D + lane * E, *dvo = (T *)p.dv + w * D + lane * E;
        for (int e = 0; e < E; ++e) { dko[e] = from_f<T>(dk[e] * p.scale); dvo[e] = from_f<T>(dv[e]); }
    }
}

}  // namespace sa
