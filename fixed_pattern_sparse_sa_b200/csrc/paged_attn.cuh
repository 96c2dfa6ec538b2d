// paged_attn.cuh -- attention of one new token per sequence over a paged
// key/value cache, split over the cache's length and joined.
//
// With n tokens held, p = n - 1 and V(p) the visible keys (all, or the last
// `window` and the first `sinks`):
//   z_j = scale q.k_j,  lse = log sum exp z,  out = sum exp(z_j - lse) v_j
// Bound by the visible K and V rows, each read once (4 d bytes a key and KV
// head against 4 d G flops).
//
// The visible keys of a sequence are numbered 0 .. n_vis-1 (sinks first) and
// cut into chunks of 16.  All chunks of all (sequence, KV head) items form
// one list; it is cut evenly over the CTAs and each CTA's share evenly over
// its warps, so ragged lengths cost nothing and the split follows the
// lengths on the device.  A warp streams its chunks through its own ring of
// cp.async stages (no block barrier in the loop) with the group's heads as
// the 16 rows of mma.sync: S = Q K^T, an online softmax, O += P V.  An item
// that lies within one warp is written by it; a CTA whose whole share is
// one item merges its warps in shared memory; what remains spans several
// warps or CTAs and is joined by paged_join_kernel from fp32 partials.
//
// P enters the second product as two values of the caches' type, rounded
// towards zero and what that leaves (16 to 22 bits), so that a row of few keys
// is as exact as its output's type; the bytes bind, not the products.  Both
// parts are above 0, so an infinity in a visible V stays one (0 * inf, or
// parts of different signs, would make it NaN).  All sums are fp32.
//
// Measured on one B200: 32 sequences of 128K, 16 heads on one KV head, 386 us =
// 5.6 TB/s (85 % of a copy's rate; 358 us on another); 192 ragged sequences,
// window 4096 and 64 sinks, 64 heads on 8, 353 us = 5.1 TB/s.
#pragma once

#include "sa_common.cuh"
#include "sink_attn.cuh"

namespace sa {

constexpr int PD_NW = 12;                 // warps per CTA
constexpr int PD_NK = 16;                 // keys per chunk
constexpr int PD_STAGES = 2;              // ring stages per warp: one chunk in flight, one in use
constexpr int PD_THREADS = PD_NW * 32;
constexpr int PD_MIN_CHUNKS = 2;          // chunks per warp below which fewer CTAs share the list
constexpr float PD_RAISE = 8.f;           // log2 headroom before the accumulators are rescaled
// log2 of the largest weight when it is taken.  fp16 holds nothing below 2^-24:
// at 2^7 to 2^15 of its 2^16 a weight of 2^-17 of the largest still has 14 bits.
template <typename T> constexpr float PD_TOP = std::is_same<T, __half>::value ? 7.f : 0.f;

template <int D>
struct PdSmem {
    static constexpr int TILE = PD_NK * D * 2;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int RING = PD_STAGES * STAGE;            // per warp
    static constexpr int OFF_ML = PD_NW * RING;               // [NW][16] m, [NW][16] l
    static constexpr int OFF_SCAN = OFF_ML + PD_NW * 32 * 4;
    static constexpr int TOTAL = OFF_SCAN + 256;
    static_assert((2 * 8 + 4) * PD_NW <= 256, "scan area");
    static_assert(RING >= 16 * D * 4, "a warp's ring holds its fp32 accumulators at the merge");
};

struct PagedParams {
    const void *q, *k, *v;
    long long q_s[2], k_s[3], v_s[3];     // q: batch, head; caches: page, slot, head (elements)
    const int32_t *table, *lens;
    int B, Hq, Hkv, G, HT;                // HT: tiles of 16 heads per group
    int page, max_pages, window, sinks;
    long long n_pages;
    float scale_log2;
    void *out;
    float *lse;
    // workspace
    long long *c0;                        // [B + 1]: chunks (of one item) of the sequences before b; [B] = all
    float *part;                          // [CTAs][2 NW][16 (D + 2)]: o, m, l
    unsigned *err;
};

struct PdSeq {
    int ns, lo, n_vis, nch;               // sinks, first window key, visible keys, chunks
};
__device__ __forceinline__ PdSeq pd_seq(const PagedParams &p, int b, bool report) {
    const int raw = __ldg(p.lens + b);
    const long long cap = (long long)p.max_pages * p.page;
    const int n = raw < 0 ? 0 : raw > cap ? (int)cap : raw;
    if (report && n != raw) raise_error(p.err, ERR_BAD_INDEX);
    PdSeq s;
    s.lo = p.window > 0 && n > p.window ? n - p.window : 0;
    s.ns = min(p.sinks, s.lo);
    s.n_vis = s.ns + n - s.lo;
    s.nch = (s.n_vis + PD_NK - 1) / PD_NK;
    return s;
}
// CTAs that share a list of `total` chunks.
__device__ __forceinline__ int pd_ctas(long long total, int grid) {
    const long long want = (total + PD_NW * PD_MIN_CHUNKS - 1) / (PD_NW * PD_MIN_CHUNKS);
    return want < grid ? (int)want : grid;
}
// First chunk of share i of n.
__device__ __forceinline__ long long pd_cut(long long total, int i, int n) { return total * i / n; }

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        mma_bf16_16816(d, a, b0, b1);
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}
// Two weights >= 0 as packed pairs a + b: a rounded towards zero, b what that
// leaves, but no less than the type's least (normal bf16, fp16) value.
template <typename T>
__device__ __forceinline__ void split_up(float x, float y, unsigned &a, unsigned &b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const unsigned xi = __float_as_uint(x), yi = __float_as_uint(y);
        a = __byte_perm(xi, yi, 0x7632);
        b = pack2<T>(fmaxf(x - __uint_as_float(xi & 0xffff0000u), 0x1p-126f),
                     fmaxf(y - __uint_as_float(yi & 0xffff0000u), 0x1p-126f));
    } else {
        const __half xh = __float2half_rz(x), yh = __float2half_rz(y);
        const __half2 h = __halves2half2(xh, yh);
        a = *reinterpret_cast<const unsigned *>(&h);
        b = pack2<T>(fmaxf(x - to_f(xh), 0x1p-24f), fmaxf(y - to_f(yh), 0x1p-24f));
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(PD_THREADS) paged_decode_kernel(const PagedParams p) {
    grid_dependency_sync();
    using L = PdSmem<D>;
    constexpr int U = D / 8;                  // 16-byte units per row
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H2 = p.Hkv * p.HT;
    long long *scan = reinterpret_cast<long long *>(smem + L::OFF_SCAN);   // [NW] warp sums, [NW] start prefixes
    int *start_b = reinterpret_cast<int *>(scan + 2 * PD_NW);              // [NW]

    // --- the chunk list: total, then the sequence in which each warp starts
    auto block_scan = [&](int b, long long carry, long long &excl) -> long long {
        const long long n = b < p.B ? pd_seq(p, b, false).nch : 0;
        long long x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < PD_NW; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
        excl = carry + before + x - n;
        return carry + all;
    };
    long long total1 = 0, excl = 0;           // chunks of one head item over the sequences
    for (int b0 = 0; b0 < p.B; b0 += PD_THREADS) {
        const int b = b0 + tid;
        total1 = block_scan(b, total1, excl);
        if (blockIdx.x == 0 && b < p.B) p.c0[b] = excl;
    }
    if (blockIdx.x == 0 && tid == 0) p.c0[p.B] = total1;
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B; b += PD_THREADS) (void)pd_seq(p, b, true);
    const long long total = total1 * H2;
    const int C = pd_ctas(total, gridDim.x);
    if ((int)blockIdx.x >= C) return;         // the whole CTA: nothing below is shared with it
    const long long ca = pd_cut(total, blockIdx.x, C), ce = pd_cut(total, blockIdx.x + 1, C);
    const long long wa = ca + pd_cut(ce - ca, warp, PD_NW), we = ca + pd_cut(ce - ca, warp + 1, PD_NW);
    {
        long long carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += PD_THREADS) {
            const int b = b0 + tid;
            long long ex = excl;
            if (p.B > PD_THREADS) carry = block_scan(b, carry, ex);
            const long long n = b < p.B ? pd_seq(p, b, false).nch : 0;
            for (int w = 0; w < PD_NW; ++w) {
                const long long x = ca + pd_cut(ce - ca, w, PD_NW);
                if (n > 0 && x >= ex * H2 && x < (ex + n) * H2) {
                    start_b[w] = b;
                    scan[PD_NW + w] = ex;
                }
            }
        }
        __syncthreads();
    }

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    unsigned qa[D / 16][4];
    unsigned char *ring = smem + warp * L::RING;
    const uint32_t ring_a = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    // does this CTA's share lie within one item?
    bool single = false;
    const bool busy = we > wa;
    float *part_cta = p.part + (size_t)blockIdx.x * (2 * PD_NW) * 16 * (D + 2);

    struct Pos { int b, h2, c; PdSeq s; };
    auto start = [&](Pos &x) {
        x.b = start_b[warp];
        x.s = pd_seq(p, x.b, false);
        const long long rel = wa - scan[PD_NW + warp] * H2;
        x.h2 = (int)(rel / x.s.nch);
        x.c = (int)(rel % x.s.nch);
    };
    auto next = [&](Pos &x) {                 // to the chunk after x; only called while one remains
        if (++x.c < x.s.nch) return;
        x.c = 0;
        if (++x.h2 < H2) return;
        x.h2 = 0;
        do {
            ++x.b;
            x.s = pd_seq(p, x.b, false);
        } while (x.s.nch == 0);
    };
    unsigned vmask[PD_STAGES];                // visible, well-paged keys of the chunk in each stage
    // chunk x into ring stage st: lanes i and i + 16 find key i's page and slot, one for K, one for V
    const long long page_s = lane < 16 ? p.k_s[0] : p.v_s[0], slot_s = lane < 16 ? p.k_s[1] : p.v_s[1];
    auto load = [&](const Pos &x, int st) -> unsigned {
        const int i = x.c * PD_NK + (lane & 15);
        bool ok = i < x.s.n_vis;
        int pg = 0, slot = 0;
        if (ok) {
            const int j = i < x.s.ns ? i : i - x.s.ns + x.s.lo;
            const int e = j / p.page;
            slot = j - e * p.page;
            pg = __ldg(p.table + (size_t)x.b * p.max_pages + e);
            if (pg < 0 || pg >= p.n_pages) {
                raise_error(p.err, ERR_BAD_INDEX);
                ok = false;
                pg = 0;
            }
        }
        const unsigned mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        const long long row = pg * page_s + slot * slot_s;
        const int hk = x.h2 / p.HT;
        const T *kb = (const T *)p.k + hk * p.k_s[2], *vb = (const T *)p.v + hk * p.v_s[2];
        const uint32_t dst = ring_a + st * L::STAGE;
        constexpr int RPI = 32 / U;           // rows per warp instruction
        const int u = lane % U;
#pragma unroll
        for (int r0 = 0; r0 < PD_NK; r0 += RPI) {
            const int r = r0 + lane / U;
            const long long kr = __shfl_sync(0xffffffffu, row, r), vr = __shfl_sync(0xffffffffu, row, r + 16);
            const int bytes = (mask >> r) & 1 ? 16 : 0;
            const uint32_t at = dst + r * (D * 2) + ((u ^ (r & 7)) * 16);
            cp_async16_at<0, 0>(at, kb + kr + u * 8, bytes);
            cp_async16_at<L::TILE, 0>(at, vb + vr + u * 8, bytes);
        }
        return mask;
    };
    // Q of item (b, h2) as A fragments, rows past the group 0
    auto load_q = [&](const Pos &x) {
        const int hk = x.h2 / p.HT, ht = x.h2 % p.HT;
        const int r0 = lane >> 2, c0 = (lane & 3) * 2;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int h = ht * 16 + r0 + (e & 1) * 8, c = ks * 16 + c0 + (e >> 1) * 8;
                qa[ks][e] = h < p.G ? __ldg(reinterpret_cast<const unsigned *>(
                                          (const T *)p.q + x.b * p.q_s[0] + (hk * p.G + h) * p.q_s[1] + c))
                                    : 0u;
            }
    };
    auto reset = [&]() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    };
    auto sum_l = [&]() {                      // row sums over the four lanes that share a row
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }
    };
    // final rows of an item held by this warp alone
    auto write_out = [&](const Pos &x) {
        const int hk = x.h2 / p.HT, ht = x.h2 % p.HT;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = ht * 16 + (lane >> 2) + e * 8;
            if (h >= p.G) continue;
            const long long row = (long long)x.b * p.Hq + hk * p.G + h;
            const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
            T *dst = (T *)p.out + row * D + (lane & 3) * 2;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<unsigned *>(dst + i * 8) = pack2<T>(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
            if ((lane & 3) == 0) p.lse[row] = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * kLn2;
        }
    };
    auto write_part = [&](float *dst) {       // [16][D] o, [16] m, [16] l
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = (lane >> 2) + e * 8;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(dst + r * D + i * 8 + (lane & 3) * 2) =
                    make_float2(o[i][2 * e], o[i][2 * e + 1]);
            if ((lane & 3) == 0) {
                dst[16 * D + r] = m[e];
                dst[16 * D + 16 + r] = l[e];
            }
        }
    };

    Pos cur{};
    if (busy) {
        Pos pro;
        start(pro);
        cur = pro;
        {
            const long long i0 = scan[PD_NW + warp] * H2 + (long long)cur.h2 * cur.s.nch;
            single = ca >= i0 && ce <= i0 + cur.s.nch;
        }
        long long left = we - wa;             // chunks still to load
        load_q(cur);
#pragma unroll
        for (int st = 0; st < PD_STAGES - 1; ++st) {
            vmask[st] = 0;
            if (left > 0) {
                vmask[st] = load(pro, st);
                if (--left > 0) next(pro);
            }
            cp_async_commit();
        }
        bool first_seg = true;
        int seg_c0 = cur.c;                   // first chunk of the current segment
        int st = 0;
        for (long long n = we - wa; n > 0; --n) {
            const int ahead = st == 0 ? PD_STAGES - 1 : st - 1;
            unsigned nm = 0;
            if (left > 0) {
                nm = load(pro, ahead);
                if (--left > 0) next(pro);
            }
            cp_async_commit();
            cp_async_wait<PD_STAGES - 1>();
            __syncwarp();
            unsigned mask = vmask[0];
#pragma unroll
            for (int i = 0; i + 2 < PD_STAGES; ++i) vmask[i] = vmask[i + 1];
            vmask[PD_STAGES - 2] = nm;
            const uint32_t kt = ring_a + st * L::STAGE, vt = kt + L::TILE;
            float s[2][4] = {};
            {
                // K: matrices (keys 0-7, c 0-7), (keys 0-7, c 8-15), (keys 8-15, c 0-7), (keys 8-15, c 8-15)
                const int r = (lane & 7) + (lane >> 4) * 8, ub = (lane >> 3) & 1;
                const uint32_t row = kt + r * (D * 2);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    unsigned b0, b1, b2, b3;
                    ldsm_x4_a(b0, b1, b2, b3, row + (((ks * 2 + ub) ^ (r & 7)) * 16));
                    mma_16816<T>(s[0], qa[ks], b0, b1);
                    mma_16816<T>(s[1], qa[ks], b2, b3);
                }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = t * 8 + (lane & 3) * 2 + (e & 1);
                    s[t][e] = (mask >> key) & 1 ? s[t][e] * p.scale_log2 : -INFINITY;
                    mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
                }
            bool raise = false;
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                mx[e] -= PD_TOP<T>;
                alpha[e] = 1.f;
                if (mx[e] > m[e] + (m[e] == -INFINITY ? 0.f : PD_RAISE)) {
                    alpha[e] = m[e] == -INFINITY ? 0.f : ex2_fast(m[e] - mx[e]);
                    m[e] = mx[e];
                    raise = true;
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) l[e] *= alpha[e];
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
            }
            const float mb[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[t][e] = ex2_fast(s[t][e] - mb[e >> 1]);
                    l[e >> 1] += s[t][e];
                }
            unsigned pa[4], pb[4];                // P = pa + pb
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split_up<T>(s[t][2 * e], s[t][2 * e + 1], pa[2 * t + e], pb[2 * t + e]);
            {
                // V transposed: (keys 0-7, c 0-7), (keys 8-15, c 0-7), (keys 0-7, c 8-15), (keys 8-15, c 8-15)
                const int r = (lane & 15), ub = lane >> 4;
                const uint32_t row = vt + r * (D * 2);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    unsigned b0, b1, b2, b3;
                    ldsm_x4_ta(b0, b1, b2, b3, row + (((i * 2 + ub) ^ (r & 7)) * 16));
                    mma_16816<T>(o[2 * i], pa, b0, b1);
                    mma_16816<T>(o[2 * i + 1], pa, b2, b3);
                    mma_16816<T>(o[2 * i], pb, b0, b1);
                    mma_16816<T>(o[2 * i + 1], pb, b2, b3);
                }
            }
            __syncwarp();                     // every lane has read the stage before it is loaded again
            st = st + 1 == PD_STAGES ? 0 : st + 1;
            // the end of the item, or of this warp's share
            if ((cur.c + 1 == cur.s.nch || n == 1) && !single) {
                sum_l();
                if (seg_c0 == 0 && cur.c + 1 == cur.s.nch)
                    write_out(cur);
                else
                    write_part(part_cta + (size_t)(2 * warp + (first_seg ? 0 : 1)) * 16 * (D + 2));
                first_seg = false;
                if (n > 1) reset();
            }
            if (n > 1) {
                next(cur);
                if (cur.c == 0) {
                    load_q(cur);
                    seg_c0 = 0;
                }
            }
        }
        if (single) sum_l();
    }
    // --- one item for the whole CTA: merge the warps in shared memory
    const bool merge = __syncthreads_or(single && busy);
    if (!merge) return;
    cp_async_wait<0>();
    float *sm = reinterpret_cast<float *>(smem + L::OFF_ML), *sl = sm + PD_NW * 16;
    if ((lane & 3) == 0)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sm[warp * 16 + (lane >> 2) + e * 8] = m[e];
            sl[warp * 16 + (lane >> 2) + e * 8] = l[e];
        }
    __syncwarp();
    float *mine = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2 *>(mine + ((lane >> 2) + e * 8) * D + i * 8 + (lane & 3) * 2) =
                make_float2(o[i][2 * e], o[i][2 * e + 1]);
    __syncthreads();
    // 16 rows over the first 256 threads
    if (tid >= 256) return;
    constexpr int TPR = 16, CPT = D / TPR;
    const int r = tid / TPR, c = (tid % TPR) * CPT;
    float M = -INFINITY, Ls = 0.f, acc[CPT] = {};
    for (int w = 0; w < PD_NW; ++w) M = fmaxf(M, sm[w * 16 + r]);
    const float Mb = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < PD_NW; ++w) {
        const float f = ex2_fast(sm[w * 16 + r] - Mb);
        Ls += f * sl[w * 16 + r];
        const float *src = reinterpret_cast<const float *>(smem + w * L::RING) + r * D + c;
#pragma unroll
        for (int e = 0; e < CPT; ++e) acc[e] += f * src[e];
    }
    // the CTA's one item
    const int b = start_b[PD_NW - 1];         // the last warp's share is never empty
    const PdSeq s = pd_seq(p, b, false);
    const long long i0 = (ca - scan[2 * PD_NW - 1] * H2) / s.nch;
    const int h2 = (int)i0, hk = h2 / p.HT, h = (h2 % p.HT) * 16 + r;
    if (ce - ca == s.nch) {
        if (h < p.G) {
            const long long row = (long long)b * p.Hq + hk * p.G + h;
            const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
            T *dst = (T *)p.out + row * D + c;
#pragma unroll
            for (int e = 0; e < CPT; ++e) dst[e] = from_f<T>(acc[e] * inv);
            if (c == 0) p.lse[row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
        }
    } else {
#pragma unroll
        for (int e = 0; e < CPT; ++e) part_cta[r * D + c + e] = acc[e];
        if (c == 0) {
            part_cta[16 * D + r] = M;
            part_cta[16 * D + 16 + r] = Ls;
        }
    }
}

// Joins the partials of the items that span several warps or CTAs (in the
// order of the list, so the result does not depend on timing) and writes the
// rows of empty sequences.  grid: (B * Hkv * HT, ceil(min(G, 16) / 4)), 4 rows
// per CTA; gx is the decode kernel's grid.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p, int gx) {
    grid_dependency_sync();
    __shared__ int slots[2 * PD_NW + 1024];
    __shared__ int n_slots;
    const int H2 = p.Hkv * p.HT;
    const int b = blockIdx.x / H2, h2 = blockIdx.x % H2, hk = h2 / p.HT;
    const PdSeq s = pd_seq(p, b, false);
    const int r = blockIdx.y * 4 + threadIdx.x / 64, h = (h2 % p.HT) * 16 + r;
    constexpr int E = D / 64;
    const int c = (threadIdx.x % 64) * E;
    const long long row = (long long)b * p.Hq + hk * p.G + h;
    if (s.nch == 0) {
        if (h < p.G) {
            for (int e = 0; e < E; ++e) ((T *)p.out)[row * D + c + e] = from_f<T>(0.f);
            if (c == 0) p.lse[row] = -INFINITY;
        }
        return;
    }
    const long long total = p.c0[p.B] * H2, i0 = p.c0[b] * H2 + (long long)h2 * s.nch, i1 = i0 + s.nch;
    const int C = pd_ctas(total, gx);
    auto owner = [&](long long x) -> int { return (int)(((x + 1) * C + total - 1) / total) - 1; };
    const int cf = owner(i0), cl = owner(i1 - 1);
    // warps of CTA ci that hold chunks of the item
    auto inside = [&](int ci) -> bool {
        return pd_cut(total, ci, C) >= i0 && pd_cut(total, ci + 1, C) <= i1;
    };
    if (cf == cl && inside(cf)) return;                       // written by that CTA
    if (threadIdx.x == 0) {
        int n = 0;
        auto ends = [&](int ci) {
            if (inside(ci)) {
                slots[n++] = ci * 2 * PD_NW;
                return;
            }
            const long long ca = pd_cut(total, ci, C), ce = pd_cut(total, ci + 1, C);
            for (int w = 0; w < PD_NW; ++w) {
                const long long wa = ca + pd_cut(ce - ca, w, PD_NW), we = ca + pd_cut(ce - ca, w + 1, PD_NW);
                if (we <= wa || we <= i0 || wa >= i1) continue;
                if (wa <= i0 && we >= i1) { n = -1; return; }     // the whole item in one warp: written
                slots[n++] = (ci * PD_NW + w) * 2 + (wa >= i0 ? 0 : 1);
            }
        };
        ends(cf);
        if (n >= 0 && cl > cf) {
            for (int ci = cf + 1; ci < cl; ++ci) slots[n++] = ci * 2 * PD_NW;
            ends(cl);
        }
        n_slots = n;
    }
    __syncthreads();
    const int n = n_slots;
    if (n < 0 || h >= p.G) return;
    constexpr size_t SZ = 16 * (D + 2);
    float M = -INFINITY;
    for (int i = 0; i < n; ++i) M = fmaxf(M, p.part[slots[i] * SZ + 16 * D + r]);
    const float Mb = M == -INFINITY ? 0.f : M;
    float Ls = 0.f, acc[E] = {};
    for (int i = 0; i < n; ++i) {
        const float *x = p.part + slots[i] * SZ;
        const float f = ex2_fast(x[16 * D + r] - Mb);
        Ls += f * x[16 * D + 16 + r];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * x[r * D + c + e];
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
#pragma unroll
    for (int e = 0; e < E; ++e) ((T *)p.out)[row * D + c + e] = from_f<T>(acc[e] * inv);
    if (c == 0) p.lse[row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
}

}  // namespace sa
