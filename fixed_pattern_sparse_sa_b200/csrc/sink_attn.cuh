// sink_attn.cuh -- sliding-window attention with sinks: the first `sinks` keys
// of a sequence stay visible beside the last `window` ones.
//
//   V(p) = { j <= min(p, n_k - 1) : p - j < window or j < sinks }
//   z_j = scale q.k_j,  lse = log sum exp z,  out = sum exp(z_j - lse) v_j
//   P = exp(z - lse), D = sum_j P dout.v, dS = P (dout.v - D)
//   dq = scale sum_j dS k_j,  dk_j = scale sum dS q,  dv_j = sum P dout
#pragma once

#include <cuda_fp16.h>

#include "sa_common.cuh"

namespace sa {

struct SinkParams {
    const void *q, *k, *v, *dout;
    long long q_s[3], k_s[3], v_s[3], do_s[3], lse_s[3];   // batch, token, head strides (elements)
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
    float2 *stat;                                // [rows of q, Hq] lse in base 2 and D, from the query-major pass
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

}  // namespace sa
