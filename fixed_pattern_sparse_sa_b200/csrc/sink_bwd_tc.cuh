// sink_bwd_tc.cuh -- backward of the sink-window attention on the tcgen05
// tensor cores.
//
//   P = exp(z - lse), dP = dout.v, D = sum_j P dP, dS = P (dP - D)
//   dq = scale sum_j dS k_j,  dk_j = scale sum dS q,  dv_j = sum P dout
//
// D equals dout.out, but out is stored rounded: where a row's attention lies
// on few keys that rounding is as large as dS's own (two visible keys: dq off
// by 2^-8.7 more than rounding it costs), so D is summed here, in fp32.
//
// Two passes, each with its sums in tensor memory from first to last, so
// nothing is added up in global memory and the result does not depend on the
// order of the blocks: query-major for dq, key-major for dk and dv.  The
// price is that S and dP are formed three times (9 products instead of 5): in
// the query-major pass once for D and once for dq, and in the key-major one;
// adding dq up from the key-major pass would move 4 bytes per element of dq
// and key tile through L2 atomics instead, in varying order.
//
// P and dS are rounded to bf16 for the second products (with SPLIT what that
// leaves enters as another product); sums are fp32 and rounded once.
//
// Measured on one B200: 16K tokens, 64 heads on 4 KV heads, window 512, 16
// sinks 1.94 ms = 359 TFLOP/s of the formulas' 10 d flops a pair (dq 1.0 ms,
// dk and dv 0.8 ms, 990 W at 1660 MHz); 2 x 1000 tokens, 8 heads, 29 us.
#pragma once

#include "sink_fwd_tc.cuh"

namespace sa {

constexpr int SB_THREADS = 384;
constexpr int SB_REGS_SCORE = 208, SB_REGS_ISSUE = 88;     // as in the forward: 2 x 208 + 88 = 3 x 168

// ------------------------------------------------------------------- dq --
// A work item is one tile of 128 rows (queries x heads, as in the forward)
// and the key tiles its rows see.  Per key tile
//   S = Q K^T,  dP = dO V^T  (N = 128),  dS = P (dP - D),  dq += dS K.
// Tensor memory holds S twice, dP once and dq: S of the next tile runs while
// the score warps work on this one, dP of the next as soon as they have read
// dP into registers.  dS replaces S and is the A operand of the last product.
// The item's key tiles are walked twice: for D (S and dP only), then for dq.
//
// Warps: 0-7 score and epilogue (thread = row; warps 0-3 the first 64 keys of
// a tile, 4-7 the rest), 8 TMA producer, 9 MMA issuer of S and dP and TMEM
// owner, 10 MMA issuer of dq, 11 TMA producer of V.
// beside the forward's tile facts: a tile of the walk for D, the first of the walk for dq
enum : uint32_t { TI_SUM = 512u, TI_START = 1024u };
constexpr uint32_t DQT_S = 0, DQT_DP = 256, DQT_DQ = 384;

template <int D>
struct SqSmem {
    static constexpr int TILE = 128 * D * 2;
    static constexpr int OFF_Q = 0;                        // 2 x (Q | dO); the staged dq of the item, afterwards
    static constexpr int OFF_K = OFF_Q + 4 * TILE;         // 2
    static constexpr int OFF_V = OFF_K + 2 * TILE;         // 1
    static constexpr int OFF_BAR = OFF_V + TILE;
    // q_full[2], q_empty[2], k_full[2], k_empty[2], v_full, v_empty, dp_full, dp_free, ds_full[2],
    // dq_full, drain[2], item_full[2], item_empty[2], d_full
    static constexpr int N_BAR = 24;                       // 22, to keep the items on 16 bytes
    static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;   // tmem slot, abort flag, -, -, tile info[2]
    static constexpr int OFF_ITEM = OFF_MISC + 32;
    static constexpr int OFF_D = OFF_ITEM + 2 * 64;        // [2][128] halves of D
    static constexpr int TOTAL = OFF_D + 1024;
    static constexpr int ALLOC = TOTAL + 1024;
    static_assert(OFF_ITEM % 16 == 0 && ALLOC <= 232448, "items are copied by 16 bytes; 227 KB per CTA");
    static_assert(8 * 32 * D <= 2 * TILE, "the staged rows fit the item's Q and dO");
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(SB_THREADS, 1)
    sink_dq_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                      const __grid_constant__ KeyMaps kmap, const __grid_constant__ KeyMaps vmap,
                      const __grid_constant__ SinkParams p, const __grid_constant__ SinkTiles tl, int *counter) {
    grid_dependency_sync();
    using T = __nv_bfloat16;
    using L = SqSmem<D>;
    constexpr int HALVES = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *q_full = bars, *q_empty = bars + 2, *k_full = bars + 4, *k_empty = bars + 6, *v_full = bars + 8;
    uint64_t *v_empty = bars + 9, *dp_full = bars + 10, *dp_free = bars + 11, *ds_full = bars + 12;
    uint64_t *dq_full = bars + 14, *drain = bars + 15, *item_full = bars + 17, *item_empty = bars + 19;
    uint64_t *d_full = bars + 21;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    volatile uint32_t *info_s = reinterpret_cast<volatile uint32_t *>(smem + L::OFF_MISC + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    sink_report(p);
    if (tid == 0) {
        if (blockIdx.x == 0) *counter = 0;            // the key-major pass's next item
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + i, 1); tc::mbar_init(q_empty + i, 8);
            tc::mbar_init(k_full + i, 1); tc::mbar_init(k_empty + i, 1);
            tc::mbar_init(ds_full + i, 8);
            tc::mbar_init(drain + i, 1);
            tc::mbar_init(item_full + i, 1); tc::mbar_init(item_empty + i, 8);
        }
        tc::mbar_init(v_full, 1); tc::mbar_init(v_empty, 1);
        tc::mbar_init(dp_full, 1); tc::mbar_init(dp_free, 8);
        tc::mbar_init(dq_full, 1); tc::mbar_init(d_full, 8);
        *abort_flag = 0;
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        raise_error(p.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp >= 8) {
        regs_dec<SB_REGS_ISSUE>();
        if (warp == 8 && lane == 0 && !debug_stall()) {      // (test hook: nothing is loaded)
            // -------------------------------------------------- TMA producer
            bool ok = true;
            int qn = 0, t = 0, in = 0;                // items with keys, key tiles, items handed over
            auto hand_over = [&](const SfItem &y) -> bool {
                if (!atc::wait(item_empty + (in & 1), ((in >> 1) & 1) ^ 1, abort_flag)) return false;
                const int4 *src = reinterpret_cast<const int4 *>(&y);
                int4 *dst = reinterpret_cast<int4 *>(smem + L::OFF_ITEM + (in & 1) * sizeof(SfItem));
#pragma unroll
                for (int c = 0; c < 4; ++c) dst[c] = src[c];
                atc::arrive(item_full + (in & 1));
                ++in;
                return true;
            };
            for (int it = blockIdx.x; it < tl.items && ok; it += gridDim.x) {
                SinkItem x;
                if (!sink_item<1>(p, tl, it, x)) continue;
                ok = hand_over(SfItem{x.nt, {x.nq_i[0], 0}, (int)x.s.pos0 + x.t0, x.band_lo, x.band_hi, x.s_end,
                                      x.n_sink | x.head / SF_HEAD << 28,
                                      {0, 0}, {0, 0}, 0, 0, x.h0 | x.nh << 20,
                                      (int)((p.cu_q ? 0 : x.b * p.Tq) + x.s.q0) + x.t0});
                if (!ok) break;
                if (x.nt == 0) continue;
                const int cb = p.cu_q ? 0 : x.b, qb = qn & 1;
                if (!(ok = atc::wait(q_empty + qb, ((qn >> 1) & 1) ^ 1, abort_flag))) break;
                atc::expect_tx(q_full + qb, 2 * HALVES * 128 * tl.HB * tl.TPT);
                for (int h = 0; h < HALVES; ++h) {
                    unsigned char *dst = smem + L::OFF_Q + qb * 2 * L::TILE + h * (128 * 128);
                    load_4d(dst, &qmap, h * 64, x.h0, (int)(x.s.q0 + x.t0), cb, q_full + qb);
                    load_4d(dst + L::TILE, &domap, h * 64, x.h0, (int)(x.s.q0 + x.t0), cb, q_full + qb);
                }
                ++qn;
                for (int i = 0; i < 2 * x.nt && ok; ++i, ++t) {
                    const bool sum = i < x.nt;
                    const int j = sum ? i : i - x.nt, sl = t & 1;
                    int k0, n;
                    x.tile(j, k0, n);
                    if (!(ok = atc::wait(k_empty + sl, ((t >> 1) & 1) ^ 1, abort_flag))) break;
                    info_s[sl] = (uint32_t)((n + 15) / 16) | (i == 0 ? TI_FIRST : 0u) | (sum ? TI_SUM : 0u) |
                                 (i == x.nt ? TI_START : 0u) | (i + 1 == 2 * x.nt ? TI_LAST : 0u) | TI_TILE;
                    atc::expect_tx(k_full + sl, L::TILE);
                    load_keys<D>(smem + L::OFF_K + sl * L::TILE, kmap, x, j, k0, cb, k_full + sl);
                }
            }
            if (ok) ok = hand_over(SfItem{-1});
            if (ok) ok = atc::wait(k_empty + (t & 1), ((t >> 1) & 1) ^ 1, abort_flag);
            if (ok) {
                info_s[t & 1] = 0u;
                atc::arrive(k_full + (t & 1));
                ++t;
            }
            if (!ok) fail();
            // let the copies land before the CTA exits
            for (int i = 1; i <= 2 && i <= qn; ++i)
                tc::mbar_wait_bounded(q_full + ((qn - i) & 1), ((qn - i) >> 1) & 1, ATC_WAIT);
            for (int i = 1; i <= 2 && i <= t; ++i)
                tc::mbar_wait_bounded(k_full + ((t - i) & 1), ((t - i) >> 1) & 1, ATC_WAIT);
        } else if (warp == 11 && lane == 0 && !debug_stall()) {
            // ---------------------------------------------------- V producer
            // its one buffer is free as soon as dP is formed, long before K's: a producer that
            // waited for both in turn would hold the next K back
            bool ok = true;
            int t = 0;
            for (int it = blockIdx.x; it < tl.items && ok; it += gridDim.x) {
                SinkItem x;
                if (!sink_item<1>(p, tl, it, x)) continue;
                for (int i = 0; i < 2 * x.nt; ++i, ++t) {
                    const int j = i < x.nt ? i : i - x.nt;
                    int k0, n;
                    x.tile(j, k0, n);
                    if (!(ok = atc::wait(v_empty, (t & 1) ^ 1, abort_flag))) break;
                    atc::expect_tx(v_full, L::TILE);
                    load_keys<D>(smem + L::OFF_V, vmap, x, j, k0, p.cu_q ? 0 : x.b, v_full);
                }
            }
            if (!ok) fail();
            if (t > 0) tc::mbar_wait_bounded(v_full, (t - 1) & 1, ATC_WAIT);
        } else if (warp == 9) {
            // ----------------------------------------------- S and dP issuer
            const bool leader = elect_one();
            const uint64_t qd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_Q), 16, 1024);
            const uint64_t kd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_K), 16, 1024);
            const uint64_t vd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_V), 16, 1024);
            constexpr uint32_t TSTEP = L::TILE >> 4;
            bool ok = true;
            int qn = 0;
            for (int t = 0;; ++t) {
                const int sl = t & 1;
                if (!(ok = wait_warp(k_full + sl, (t >> 1) & 1, abort_flag))) break;
                const uint32_t info = info_s[sl];
                if (!(info & TI_TILE)) break;
                if (info & TI_FIRST) {
                    if (!(ok = wait_warp(q_full + (qn & 1), (qn >> 1) & 1, abort_flag))) break;
                    ++qn;
                }
                // S buffer sl is free: this K tile was loaded after tile t - 2 was done with
                const uint64_t a = qd + (((qn - 1) & 1) * 2) * TSTEP, b = kd + sl * TSTEP;
                const uint32_t id = tc::make_idesc(1, 1, 128, 0) | ((info & TI_STEPS) << 18);
                tc::fence_after_sync();
                if (leader) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int off = ((c / 4) * (128 * 128) + (c % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + DQT_S + sl * 128, a + off, b + off, id, c > 0 ? 1u : 0u);
                    }
                }
                if (!(ok = wait_warp(v_full, t & 1, abort_flag) && wait_warp(dp_free, (t & 1) ^ 1, abort_flag))) break;
                tc::fence_after_sync();
                if (leader) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int off = ((c / 4) * (128 * 128) + (c % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + DQT_DP, a + TSTEP + off, vd + off, id, c > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(dp_full);          // S and dP
                    tc::mma_commit(v_empty);
                }
            }
            if (lane == 0 && !ok) fail();
            if (leader) {
                tc::mma_commit(drain);
                tc::mbar_wait_bounded(drain, 0, ATC_WAIT);
            }
        } else if (warp == 10) {
            // ----------------------------------------------------- dq issuer
            constexpr uint32_t ID_Q = tc::make_idesc(1, 1, 128, D) | (1u << 16);    // B (K) MN-major
            const bool leader = elect_one();
            const uint64_t kd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_K), 128 * 128, 1024);
            bool ok = true;
            for (int t = 0;; ++t) {
                const int sl = t & 1;
                if (!(ok = wait_warp(k_full + sl, (t >> 1) & 1, abort_flag))) break;
                const uint32_t info = info_s[sl];
                if (!(info & TI_TILE)) break;
                // the score warps write an item's first dS after they have read the dq of the item before
                if (!(ok = wait_warp(ds_full + sl, (t >> 1) & 1, abort_flag))) break;
                if (info & TI_SUM) {
                    if (leader) atc::arrive(k_empty + sl);
                    continue;
                }
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t b = kd + sl * (L::TILE >> 4);
                    const int steps = info & TI_STEPS;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c < steps)
                            tc::mma_bf16_ts(tmem + DQT_DQ, tmem + DQT_S + sl * 128 + (c / 4) * 64 + (c % 4) * 8, b + c * 128,
                                            ID_Q, c > 0 ? 1u : (info & TI_START ? 0u : 1u));
                    if constexpr (SPLIT) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c < steps)
                                tc::mma_bf16_ts(tmem + DQT_DQ, tmem + DQT_S + sl * 128 + (c / 4) * 64 + 32 + (c % 4) * 8,
                                                b + c * 128, ID_Q, 1u);
                    }
                    tc::mma_commit(k_empty + sl);
                    if (info & TI_LAST) tc::mma_commit(dq_full);
                }
            }
            if (lane == 0 && !ok) fail();
            if (leader) {
                tc::mma_commit(drain + 1);
                tc::mbar_wait_bounded(drain + 1, 0, ATC_WAIT);
            }
        }
        __syncwarp();
    } else {
        regs_inc<SB_REGS_SCORE>();
        // ------------------------------------------------- score, epilogue
        const int w = warp >> 2, r = (warp & 3) * 32 + lane;      // column half, row
        const uint32_t lrow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int tt = r / tl.HB, hh = r - tt * tl.HB;
        constexpr int CW = D / 2;                                 // dq columns of this warp
        bool ok = true;
        int t = 0, qn = 0;
        for (uint32_t in = 0;; ++in) {
            if (!wait_warp(item_full + (in & 1), (in >> 1) & 1, abort_flag)) { ok = false; break; }
            SfItem x;
            {
                const int4 *src = reinterpret_cast<const int4 *>(smem + L::OFF_ITEM + (in & 1) * sizeof(SfItem));
                int4 *dst = reinterpret_cast<int4 *>(&x);
#pragma unroll
                for (int c = 0; c < 4; ++c) dst[c] = src[c];
            }
            arrive_warp(item_empty + (in & 1));
            if (x.nt < 0) break;
            const bool row_ok = tt < x.nq[0] && hh < (x.heads >> 20);
            const int row_at = row_ok ? tt * p.Hq + hh : -1;
            const long long row0 = (long long)x.row * p.Hq + (x.heads & 0xfffff);
            int s1 = 0, lo = -(1 << 30), hi = 1 << 30;    // rows of nobody: anything, never written
            float nl = -INFINITY, Dr = 0.f;
            if (row_ok) {
                const int pos = x.pos + tt;
                hi = min(max(pos + 1, 0), x.band_hi);
                lo = min(max(pos - p.window + 1, 0), hi);
                s1 = min(p.sinks, lo);
                const int b = p.cu_q ? 0 : x.row / (int)p.Tq, tok = x.row - b * (int)p.Tq + tt;
                nl = -kLog2e * __ldg(p.lse_in + b * p.lse_s[0] + tok * p.lse_s[1] + ((x.heads & 0xfffff) + hh) * p.lse_s[2]);
            }
            uint64_t dsum[2] = {0ull, 0ull};
            const int n_sink = x.sinks & 0xfffffff, head = (x.sinks >> 28) * SF_HEAD;
            const int base = x.band_lo - (head ? head : n_sink * SF_KT);
            for (int i = 0; i < 2 * x.nt; ++i, ++t) {
                const bool sum = i < x.nt;
                const int j = sum ? i : i - x.nt;
                if (i == x.nt) {
                    // D from the two halves of the row
                    float *xd = reinterpret_cast<float *>(smem + L::OFF_D), d0, d1;
                    f2_unpack(f2_add(dsum[0], dsum[1]), d0, d1);
                    xd[w * 128 + r] = d0 + d1;
                    // (an mbarrier: a warp that gave up must not leave the others waiting without a limit)
                    arrive_warp(d_full);
                    if (!wait_warp(d_full, qn & 1, abort_flag)) { ok = false; break; }
                    Dr = xd[r] + xd[128 + r];
                    if (w == 0 && row_ok) p.stat[row0 + row_at] = make_float2(-nl, Dr);
                }
                const bool apart = head == 0 && j < n_sink;
                const int k0 = (apart ? 0 : base) + j * SF_KT, sh = j == 0 ? head : 0;
                const int n = min(SF_KT, (apart ? x.s_end : x.band_hi) - k0), sb = t & 1;
                if (!wait_warp(dp_full, t & 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                uint32_t s[64], dp[64];
                const uint32_t tS = lrow + DQT_S + sb * 128 + w * 64, tP = lrow + DQT_DP + w * 64;
                const int c0 = w * 64;
#pragma unroll
                for (int c = 0; c < 64; c += 32)
                    if (c0 + c < n) {
                        tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(s + c));
                        tmem_ld32(tP + c, *reinterpret_cast<uint32_t(*)[32]>(dp + c));
                    }
                tc::tmem_ld_wait();
                tc::fence_before_sync();
                arrive_warp(dp_free);
                if (sum) {
                    arrive_warp(ds_full + sb);            // S has been read
                } else if ((n & 15) || sh > x.s_end) {
                    // rows n .. of the last 16 keys, and those between the sinks and the band, hold whatever lies
                    // there: 0 * inf must not reach dq
                    constexpr int U = D / 8;
                    const int gap = max(0, sh - x.s_end), rows = gap + ((n + 15) & ~15) - n;
#pragma unroll 1
                    for (int u = tid; u < rows * U; u += 256) {
                        const int e = u / U, key = e < gap ? x.s_end + e : n + e - gap, c = u % U;
                        *reinterpret_cast<uint4 *>(smem + L::OFF_K + sb * L::TILE + (c / 8) * (128 * 128) + key * 128 +
                                                   (((c & 7) ^ (key & 7)) * 16)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_proxy_async_smem();
                }
                const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(nl, nl), nD2 = f2_pack(-Dr, -Dr);
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    if (c0 + c < n) {
                        uint32_t pk[16], pr[16];
                        const int k = k0 + c0 + c;
                        const bool whole = c0 + c + 32 <= n && ((k >= lo && k + 32 <= hi) || k + 32 <= s1) && c0 + c >= sh;
                        uint32_t vis = 0xffffffffu;
                        if (!__all_sync(0xffffffffu, whole))
                            vis = (bit_range(lo - k, hi - k) | bit_range(sh - c0 - c, s1 - k) |
                                   bit_range(-c0 - c, (sh ? min(s1, x.s_end) : 0) - c0 - c)) & bit_range(0, n - c0 - c);
                        const bool all = __all_sync(0xffffffffu, vis == 0xffffffffu);
                        if (sum) {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a, b;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), sc2, nl2),
                                          a, b);
                                a = ex2_fast(a);
                                b = ex2_fast(b);
                                float u = __uint_as_float(dp[c + e]), v = __uint_as_float(dp[c + e + 1]);
                                if (!all) {               // both factors: dP of an unseen key may be anything
                                    const bool v0 = (vis >> e) & 1u, v1 = (vis >> (e + 1)) & 1u;
                                    a = v0 ? a : 0.f; u = v0 ? u : 0.f;
                                    b = v1 ? b : 0.f; v = v1 ? v : 0.f;
                                }
                                dsum[(e >> 1) & 1] = f2_fma(f2_pack(a, b), f2_pack(u, v), dsum[(e >> 1) & 1]);
                            }
                            continue;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b, u, v;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), sc2, nl2), a,
                                      b);
                            const uint64_t P2 = f2_pack(ex2_fast(a), ex2_fast(b));
                            const uint64_t d2 =
                                f2_add(f2_pack(__uint_as_float(dp[c + e]), __uint_as_float(dp[c + e + 1])), nD2);
                            f2_unpack(f2_mul(P2, d2), u, v);
                            if (!all) {
                                u = (vis >> e) & 1u ? u : 0.f;
                                v = (vis >> (e + 1)) & 1u ? v : 0.f;
                            }
                            pk[e / 2] = pack_bf16(u, v);
                            if constexpr (SPLIT) pr[e / 2] = pack2_rest<T>(u, v, pk[e / 2]);
                        }
                        atc::tmem_st16(tS + c / 2, pk);
                        if constexpr (SPLIT) atc::tmem_st16(tS + 32 + c / 2, pr);
                    }
                }
                if (!sum) {
                    atc::tmem_st_wait();
                    tc::fence_before_sync();
                    arrive_warp(ds_full + sb);
                }
            }
            if (!ok) break;
            // ------------------------------------------------------ epilogue
            T *out0 = (T *)p.dq + row0 * D + w * CW;
            uint32_t o[CW];
            if (x.nt > 0) {
                if (!wait_warp(dq_full, qn & 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < CW; c += 32)
                    tmem_ld32(lrow + DQT_DQ + w * CW + c, *reinterpret_cast<uint32_t(*)[32]>(o + c));
                tc::tmem_ld_wait();
                tc::fence_before_sync();
            } else {
#pragma unroll
                for (int c = 0; c < CW; ++c) o[c] = 0u;
            }
            if (x.nt == 0) {
                if (row_ok)
#pragma unroll
                    for (int u = 0; u < CW / 8; ++u)
                        *reinterpret_cast<uint4 *>(out0 + (long long)row_at * D + u * 8) = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            // through the item's Q and dO, which no product reads any more, so that whole lines are written
            constexpr int UR = CW / 8, RPI = 32 / UR;             // units per row, rows per step
            unsigned char *stage = smem + L::OFF_Q + (qn & 1) * 2 * L::TILE + warp * (32 * CW * 2);
#pragma unroll
            for (int u = 0; u < UR; ++u) {
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    pk[e] = pack_bf16(__uint_as_float(o[8 * u + 2 * e]) * p.scale,
                                      __uint_as_float(o[8 * u + 2 * e + 1]) * p.scale);
                *reinterpret_cast<uint4 *>(stage + lane * (CW * 2) + ((u ^ (lane & (UR - 1))) * 16)) =
                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 32 / RPI; ++k) {
                const int rr = k * RPI + lane / UR, u = lane % UR;
                const int to = __shfl_sync(0xffffffffu, row_at, rr);
                const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * (CW * 2) + ((u ^ (rr & (UR - 1))) * 16));
                if (to >= 0) *reinterpret_cast<uint4 *>(out0 + (long long)to * D + u * 8) = v;
            }
            tc::fence_proxy_async_smem();
            arrive_warp(q_empty + (qn & 1));
            ++qn;
        }
        if (!ok) fail();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------- dk, dv --
// A work item is 128 keys of one KV head (the tensor-memory lanes) and a run
// of the queries that see them, walked in units of 64 rows: TPT queries x HB
// heads of the group (HB = min(G, 64), TPT = 64 / HB).  Per unit
//   S^T = K Q^T,  dP^T = V dO^T  (N = 64),  P^T and dS^T over them in place,
//   dV += P^T dO,  dK += dS^T Q.
// Two buffers of S^T and dP^T, each with its own four score warps, so a
// unit's first products overlap the other's scores.
//
// Keys [sinks, nk) form band items: the queries of their windows.  The sinks
// are seen by every later query; their keys form items of their own, cut over
// the queries into pieces whose fp32 sums sink_dkv_join_kernel adds up in
// order.  (Where no query is past the window the sinks are plain keys.)
//
// Warps: 0-3 and 4-7 score warps of the even and odd units (thread = key),
// then the epilogue of dv and dk; 8 TMA producer, 9 MMA issuer of S^T and
// dP^T and TMEM owner, 10 MMA issuer of dV and dK.
constexpr int KVT_STAGES = 3;
constexpr uint32_t KVT_S = 0, KVT_V = 256, KVT_K = 384;    // buffer g: S^T at 128 g, dP^T at 128 g + 64

struct SinkKvTiles {
    int HB, HC, TPT;         // heads per unit, head chunks, queries per unit
    int per_seq, band;       // dense: band tiles per sequence; band tile slots of the batch
    int n_kt, n_split, tps;  // sink key tiles, pieces of each, queries per piece
    int items;               // (band + B * n_kt * n_split) * Hkv
    float *part;             // [B, Hkv, n_split, sinks, {dv, dk}, D] when n_split > 1
    int *counter;            // next item
};
// Sinks of a sequence that queries past the window still see.
__device__ __forceinline__ int sink_apart(const SinkParams &p, const SinkSeq &s) {
    return s.pos0 + s.nq > p.window ? min(p.sinks, s.nk) : 0;
}
// Queries [ta, te) of piece sp for the sink keys from j0 on.
__device__ __forceinline__ void sink_piece(const SinkSeq &s, int tps, int sp, int j0, int &ta, int &te) {
    const long long a = (long long)sp * tps, v = j0 - s.pos0;
    ta = (int)min((long long)s.nq, max(a, max(v, 0ll)));
    te = (int)min((long long)s.nq, a + tps);
}
struct alignas(16) KvItem {
    int units;               // 0: nothing sees the keys; -1 ends the stream
    int j_rel, n_keys;       // first key less the position of query 0, keys
    int ta, te;              // queries
    int q_row, k_row;        // query 0's row and the first key's row of the whole batch
    int hk, sink;
    int part;                // piece to write fp32 sums to, -1 = dk and dv themselves
    int j0;
    int pad[5];
};
struct KvWhere { int b; long long q0, k0; };
__device__ __forceinline__ bool kv_item(const SinkParams &p, const SinkKvTiles &tl, int it, KvItem &x, KvWhere &at) {
    x.hk = it % p.Hkv;
    int r = it / p.Hkv, local;
    SinkSeq s;
    x.part = -1;
    if (r < tl.band) {
        if (!p.cu_k) {
            at.b = r / tl.per_seq;
            local = r - at.b * tl.per_seq;
        } else {
            sink_slot(p.cu_k, p.B, (int)p.L, 128u, r, at.b, local);
        }
        s = sink_seq(p, at.b);
        const int se = sink_apart(p, s);
        if (local < 0 || (long long)local * 128 + se >= s.nk) return false;
        x.j0 = se + local * 128;
        x.n_keys = min(128, s.nk - x.j0);
        x.sink = 0;
        const long long ta = x.j0 - s.pos0, te = (long long)x.j0 + x.n_keys - 1 + p.window - s.pos0;
        x.ta = (int)min((long long)s.nq, max(ta, 0ll));
        x.te = (int)max(0ll, min((long long)s.nq, te));
    } else {
        r -= tl.band;
        const int sp = r % tl.n_split;
        r /= tl.n_split;
        const int kt = r % tl.n_kt;
        at.b = r / tl.n_kt;
        s = sink_seq(p, at.b);
        const int se = sink_apart(p, s);
        x.j0 = kt * 128;
        if (x.j0 >= se) return false;
        x.n_keys = min(128, se - x.j0);
        x.sink = 1;
        sink_piece(s, tl.tps, sp, x.j0, x.ta, x.te);
        if (tl.n_split > 1) {
            if (x.ta >= x.te) return false;                   // the join skips it too
            x.part = (at.b * p.Hkv + x.hk) * tl.n_split + sp;
        }
    }
    x.j_rel = (int)(x.j0 - s.pos0);
    x.units = x.ta < x.te ? ((x.te - x.ta + tl.TPT - 1) / tl.TPT) * tl.HC : 0;
    const int bb = p.cu_q ? 0 : at.b;
    x.q_row = (int)(bb * p.Tq + s.q0);
    x.k_row = (int)(bb * p.L + s.k0) + x.j0;
    at.q0 = s.q0;
    at.k0 = s.k0;
    return true;
}

template <int D>
struct SkSmem {
    static constexpr int TILE = 128 * D * 2;               // K or V
    static constexpr int UNIT = 64 * D * 2;                // Q or dO of a unit
    static constexpr int OFF_K = 0;                        // K | V
    static constexpr int OFF_Q = OFF_K + 2 * TILE;         // stages of Q | dO
    static constexpr int OFF_STAGE = OFF_Q + KVT_STAGES * 2 * UNIT;       // outputs: 32 rows x 128 B per score warp
    static constexpr int OFF_STAT = OFF_STAGE + 8 * 4096;  // [group][2][64] lse, D
    static constexpr int OFF_BAR = OFF_STAT + 4 * 64 * 8;
    // kv_full, kv_empty, q_full[S], q_empty[S], sd_full[2], pd_full[2], pd_done[2], acc_full, acc_free, drain[2],
    // item_full[2], item_empty[2], stat_full[2]
    static constexpr int N_BAR = 18 + 2 * KVT_STAGES;
    static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;   // tmem slot, abort flag, -, -, unit info[S]
    static constexpr int OFF_ITEM = OFF_MISC + 32;
    static constexpr int TOTAL = OFF_ITEM + 2 * 64;
    static constexpr int ALLOC = TOTAL + 1024;
    static_assert(OFF_ITEM % 16 == 0 && ALLOC <= 232448, "items are copied by 16 bytes; 227 KB per CTA");
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(SB_THREADS, 1)
    sink_dkv_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap domap,
                       const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ SinkParams p, const __grid_constant__ SinkKvTiles tl) {
    grid_dependency_sync();
    using T = __nv_bfloat16;
    using L = SkSmem<D>;
    constexpr int HALVES = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *kv_full = bars, *kv_empty = bars + 1, *q_full = bars + 2, *q_empty = q_full + KVT_STAGES;
    uint64_t *sd_full = q_empty + KVT_STAGES, *pd_full = sd_full + 2, *pd_done = pd_full + 2, *acc_full = pd_done + 2;
    uint64_t *acc_free = acc_full + 1, *drain = acc_free + 1, *item_full = drain + 2, *item_empty = item_full + 2;
    uint64_t *stat_full = item_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    volatile uint32_t *info_s = reinterpret_cast<volatile uint32_t *>(smem + L::OFF_MISC + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(kv_full, 1); tc::mbar_init(kv_empty, 1);
        for (int i = 0; i < KVT_STAGES; ++i) { tc::mbar_init(q_full + i, 1); tc::mbar_init(q_empty + i, 1); }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(sd_full + i, 1); tc::mbar_init(pd_full + i, 4); tc::mbar_init(pd_done + i, 1);
            tc::mbar_init(stat_full + i, 4);
            tc::mbar_init(drain + i, 1);
            tc::mbar_init(item_full + i, 1); tc::mbar_init(item_empty + i, 8);
        }
        tc::mbar_init(acc_full, 1); tc::mbar_init(acc_free, 8);
        *abort_flag = 0;
        tc::mbar_fence_init();
    }
    // rows of a unit that no copy writes (64 is not a multiple of HB) are 0 for good
    for (int u = tid; u < KVT_STAGES * 2 * L::UNIT / 16; u += SB_THREADS)
        reinterpret_cast<uint4 *>(smem + L::OFF_Q)[u] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        raise_error(p.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp >= 8) {
        regs_dec<SB_REGS_ISSUE>();
        if (warp == 8 && lane == 0 && !debug_stall()) {      // (test hook: nothing is loaded)
            // -------------------------------------------------- TMA producer
            bool ok = true;
            int kn = 0, u = 0, in = 0;                // items with units, units, items handed over
            auto hand_over = [&](const KvItem &y) -> bool {
                if (!atc::wait(item_empty + (in & 1), ((in >> 1) & 1) ^ 1, abort_flag)) return false;
                const int4 *src = reinterpret_cast<const int4 *>(&y);
                int4 *dst = reinterpret_cast<int4 *>(smem + L::OFF_ITEM + (in & 1) * sizeof(KvItem));
#pragma unroll
                for (int c = 0; c < 3; ++c) dst[c] = src[c];
                atc::arrive(item_full + (in & 1));
                ++in;
                return true;
            };
            int it = atomicAdd(tl.counter, 1);
            while (it < tl.items && ok) {
                const int it_next = atomicAdd(tl.counter, 1);
                KvItem x;
                KvWhere at;
                const bool any = kv_item(p, tl, it, x, at);
                it = it_next;
                if (!any) continue;
                if (!(ok = hand_over(x))) break;
                if (x.units == 0) continue;
                const int cb = p.cu_q ? 0 : at.b;
                if (!(ok = atc::wait(kv_empty, (kn & 1) ^ 1, abort_flag))) break;
                atc::expect_tx(kv_full, 2 * L::TILE);
                for (int h = 0; h < HALVES; ++h) {
                    load_4d(smem + L::OFF_K + h * (128 * 128), &kmap, h * 64, x.hk, (int)at.k0 + x.j0, cb, kv_full);
                    load_4d(smem + L::OFF_K + L::TILE + h * (128 * 128), &vmap, h * 64, x.hk, (int)at.k0 + x.j0, cb,
                            kv_full);
                }
                ++kn;
                int t0 = x.ta, hc = 0;
                for (int i = 0; i < x.units; ++i, ++u) {
                    const int st = u % KVT_STAGES;
                    if (!(ok = atc::wait(q_empty + st, ((u / KVT_STAGES) & 1) ^ 1, abort_flag))) break;
                    info_s[st] = TI_TILE | (i == 0 ? TI_FIRST : 0u) | (i + 1 == x.units ? TI_LAST : 0u);
                    atc::expect_tx(q_full + st, 2 * HALVES * 128 * tl.HB * tl.TPT);
                    for (int h = 0; h < HALVES; ++h) {
                        unsigned char *dst = smem + L::OFF_Q + st * 2 * L::UNIT + h * (64 * 128);
                        load_4d(dst, &qmap, h * 64, x.hk * p.G + hc * tl.HB, (int)at.q0 + t0, cb, q_full + st);
                        load_4d(dst + L::UNIT, &domap, h * 64, x.hk * p.G + hc * tl.HB, (int)at.q0 + t0, cb, q_full + st);
                    }
                    if (++hc == tl.HC) {
                        hc = 0;
                        t0 += tl.TPT;
                    }
                }
            }
            if (ok) ok = hand_over(KvItem{-1});
            if (ok) ok = atc::wait(q_empty + u % KVT_STAGES, ((u / KVT_STAGES) & 1) ^ 1, abort_flag);
            if (ok) {
                info_s[u % KVT_STAGES] = 0u;
                atc::arrive(q_full + u % KVT_STAGES);
                ++u;
            }
            if (!ok) fail();
            // let the copies land before the CTA exits
            if (kn > 0) tc::mbar_wait_bounded(kv_full, (kn - 1) & 1, ATC_WAIT);
            for (int i = 1; i <= KVT_STAGES && i <= u; ++i)
                tc::mbar_wait_bounded(q_full + (u - i) % KVT_STAGES, ((u - i) / KVT_STAGES) & 1, ATC_WAIT);
        } else if (warp == 9) {
            // ------------------------------------------- S^T and dP^T issuer
            constexpr uint32_t ID_S = tc::make_idesc(1, 1, 128, 64);
            constexpr uint32_t USTEP = L::UNIT >> 4, TSTEP = L::TILE >> 4;
            const bool leader = elect_one();
            const uint64_t kd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_K), 16, 1024);
            const uint64_t qd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_Q), 16, 1024);
            bool ok = true;
            int st = 0;
            uint32_t qpar = 0, kpar = 0;
            for (int u = 0;; ++u) {
                if (!(ok = wait_warp(q_full + st, qpar, abort_flag))) break;
                const uint32_t info = info_s[st];
                if (!(info & TI_TILE)) break;
                if (info & TI_FIRST) {
                    if (!(ok = wait_warp(kv_full, kpar, abort_flag))) break;
                    kpar ^= 1;
                }
                const int g = u & 1;
                // buffer g is free once the products of unit u - 2 have read its P^T and dS^T
                if (!(ok = wait_warp(pd_done + g, ((u >> 1) & 1) ^ 1, abort_flag))) break;
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t b = qd + st * 2 * USTEP;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int ao = ((c / 4) * (128 * 128) + (c % 4) * 32) >> 4;
                        const int bo = ((c / 4) * (64 * 128) + (c % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + KVT_S + g * 128, kd + ao, b + bo, ID_S, c > 0 ? 1u : 0u);
                    }
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int ao = ((c / 4) * (128 * 128) + (c % 4) * 32) >> 4;
                        const int bo = ((c / 4) * (64 * 128) + (c % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + KVT_S + g * 128 + 64, kd + TSTEP + ao, b + USTEP + bo, ID_S, c > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(sd_full + g);
                    if (info & TI_LAST) tc::mma_commit(kv_empty);
                }
                if (++st == KVT_STAGES) { st = 0; qpar ^= 1; }
            }
            if (lane == 0 && !ok) fail();
            if (leader) {
                tc::mma_commit(drain);
                tc::mbar_wait_bounded(drain, 0, ATC_WAIT);
            }
        } else if (warp == 10) {
            // --------------------------------------------- dV and dK issuer
            constexpr uint32_t ID_O = tc::make_idesc(1, 1, 128, D) | (1u << 16);    // B (dO, Q) MN-major
            constexpr uint32_t USTEP = L::UNIT >> 4;
            const bool leader = elect_one();
            const uint64_t qd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_Q), 64 * 128, 1024);
            bool ok = true;
            int st = 0;
            uint32_t qpar = 0, apar = 1;
            for (int u = 0;; ++u) {
                if (!(ok = wait_warp(q_full + st, qpar, abort_flag))) break;
                const uint32_t info = info_s[st];
                if (!(info & TI_TILE)) break;
                const int g = u & 1;
                if (info & TI_FIRST) {
                    // the item before has been read out of the accumulators
                    if (!(ok = wait_warp(acc_free, apar, abort_flag))) break;
                    apar ^= 1;
                }
                if (!(ok = wait_warp(pd_full + g, (u >> 1) & 1, abort_flag))) break;
                tc::fence_after_sync();
                if (leader) {
                    const uint64_t b = qd + st * 2 * USTEP;
                    const uint32_t acc = info & TI_FIRST ? 0u : 1u;
#pragma unroll
                    for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tc::mma_bf16_ts(tmem + KVT_V, tmem + KVT_S + g * 128 + part * 32 + c * 8, b + USTEP + c * 128, ID_O,
                                            c + part > 0 ? 1u : acc);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tc::mma_bf16_ts(tmem + KVT_K, tmem + KVT_S + g * 128 + 64 + part * 32 + c * 8, b + c * 128, ID_O,
                                            c + part > 0 ? 1u : acc);
                    }
                    tc::mma_commit(pd_done + g);
                    tc::mma_commit(q_empty + st);
                    if (info & TI_LAST) tc::mma_commit(acc_full);
                }
                if (++st == KVT_STAGES) { st = 0; qpar ^= 1; }
            }
            if (lane == 0 && !ok) fail();
            if (leader) {
                tc::mma_commit(drain + 1);
                tc::mbar_wait_bounded(drain + 1, 0, ATC_WAIT);
            }
        }
        __syncwarp();
    } else {
        regs_inc<SB_REGS_SCORE>();
        // ------------------------------------------------- score, epilogue
        const int g = warp >> 2, r = (warp & 3) * 32 + lane;      // unit parity, key
        const uint32_t lrow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lrow + KVT_S + g * 128, tP = tS + 64;
        float2 *stat_s = reinterpret_cast<float2 *>(smem + L::OFF_STAT) + g * 128;
        // the unit's row whose lse and D this thread brings (threads 0 .. 63 of the group)
        const int col = tid & 127, ct = col / tl.HB, ch = col - ct * tl.HB;
        const bool brings = col < 64 && ct < tl.TPT;
        bool ok = true;
        int u0 = 0, kn = 0;                           // units of the stream before this item, items with units
        for (uint32_t in = 0;; ++in) {
            if (!wait_warp(item_full + (in & 1), (in >> 1) & 1, abort_flag)) { ok = false; break; }
            KvItem x;
            {
                const int4 *src = reinterpret_cast<const int4 *>(smem + L::OFF_ITEM + (in & 1) * sizeof(KvItem));
                int4 *dst = reinterpret_cast<int4 *>(&x);
#pragma unroll
                for (int c = 0; c < 3; ++c) dst[c] = src[c];
            }
            arrive_warp(item_empty + (in & 1));
            if (x.units < 0) break;
            const bool key_ok = r < x.n_keys;
            // queries that see this key
            const int tlo = x.j_rel + r, thi = x.sink ? INT_MAX : tlo + p.window;
            // own units: i, i + 2, ...; their lse and D are loaded one unit ahead
            auto fetch = [&](int i) -> float2 {
                const int tu = tl.HC == 1 ? i : i / tl.HC, hc = tl.HC == 1 ? 0 : i - tu * tl.HC;
                const int t = x.ta + tu * tl.TPT + ct, h = hc * tl.HB + ch;
                if (!brings || i >= x.units || t >= x.te || h >= p.G) return make_float2(INFINITY, 0.f);
                return __ldg(p.stat + (long long)(x.q_row + t) * p.Hq + x.hk * p.G + h);
            };
            int i = (g ^ u0) & 1;
            float2 mine = fetch(i);
            for (; i < x.units; i += 2) {
                const int u = u0 + i;
                float2 *sm = stat_s + ((u >> 1) & 1) * 64;
                if (col < 64) sm[col] = make_float2(-mine.x, -mine.y);
                arrive_warp(stat_full + g);           // bounded, as every wait between warps here
                if (!wait_warp(stat_full + g, (u >> 1) & 1, abort_flag)) { ok = false; break; }
                mine = fetch(i + 2);
                const int t0 = x.ta + (tl.HC == 1 ? i : i / tl.HC) * tl.TPT;
                if (!wait_warp(sd_full + g, (u >> 1) & 1, abort_flag)) { ok = false; break; }
                tc::fence_after_sync();
                const int n_t = min(tl.TPT, x.te - t0);          // queries of the unit
                const bool whole = !key_ok || (t0 >= tlo && t0 + tl.TPT <= thi);
                // columns of no query row (past HB * TPT, heads past the group) have lse = inf: P = dS = 0
                const bool clear = __all_sync(0xffffffffu, whole && n_t == tl.TPT);
                // columns of the queries [tlo, thi) among the unit's
                const int ca = max(tlo - t0, 0), cb = min(n_t, thi - t0);
                const int va = min(ca, 64) * tl.HB, vb = max(cb, 0) * tl.HB;
                if (n_t < tl.TPT) {
                    // rows past the last query hold whatever lies behind: 0 * inf must not reach the sums
                    constexpr int U = D / 8;
                    const int first = n_t * tl.HB, st = u % KVT_STAGES;
#pragma unroll 1
                    for (int e = r; e < (64 - first) * U * 2; e += 128) {
                        const int which = e / ((64 - first) * U), f = e - which * (64 - first) * U;
                        const int row = first + f / U, c = f % U;
                        *reinterpret_cast<uint4 *>(smem + L::OFF_Q + (st * 2 + which) * L::UNIT + (c / 8) * (64 * 128) +
                                                   row * 128 + (((c & 7) ^ (row & 7)) * 16)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_proxy_async_smem();
                }
                const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
                uint32_t s1[SPLIT ? 32 : 1], dp1[SPLIT ? 32 : 1];
                if constexpr (SPLIT) {                    // the rests of the first columns go over these
                    tmem_ld32(tS + 32, s1);
                    tmem_ld32(tP + 32, dp1);
                }
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t s[32], dp[32], pk[16], dk[16], pr[16], dr[16];
                    if (SPLIT && c > 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            s[e] = s1[SPLIT ? e : 0];
                            dp[e] = dp1[SPLIT ? e : 0];
                        }
                    } else {
                        tmem_ld32(tS + c, s);
                        tmem_ld32(tP + c, dp);
                        tc::tmem_ld_wait();
                    }
                    const uint32_t vis = clear ? 0xffffffffu : bit_range(va - c, vb - c);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float4 st = *reinterpret_cast<const float4 *>(sm + c + e);     // -lse, -D of two rows
                        float a, b, x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, f2_pack(st.x, st.z)),
                                  a, b);
                        a = ex2_fast(a);
                        b = ex2_fast(b);
                        f2_unpack(f2_mul(f2_pack(a, b), f2_add(f2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])),
                                                               f2_pack(st.y, st.w))),
                                  x0, x1);
                        if (!clear) {
                            const bool v0 = (vis >> e) & 1u, v1 = (vis >> (e + 1)) & 1u;
                            a = v0 ? a : 0.f; x0 = v0 ? x0 : 0.f;
                            b = v1 ? b : 0.f; x1 = v1 ? x1 : 0.f;
                        }
                        pk[e / 2] = pack_bf16(a, b);
                        dk[e / 2] = pack_bf16(x0, x1);
                        if constexpr (SPLIT) {
                            pr[e / 2] = pack2_rest<T>(a, b, pk[e / 2]);
                            dr[e / 2] = pack2_rest<T>(x0, x1, dk[e / 2]);
                        }
                    }
                    atc::tmem_st16(tS + c / 2, pk);
                    atc::tmem_st16(tP + c / 2, dk);
                    if constexpr (SPLIT) {
                        atc::tmem_st16(tS + 32 + c / 2, pr);
                        atc::tmem_st16(tP + 32 + c / 2, dr);
                    }
                }
                atc::tmem_st_wait();
                tc::fence_before_sync();
                arrive_warp(pd_full + g);
            }
            if (!ok) break;
            u0 += x.units;
            // ---------------------------- epilogue: group 0 dv, group 1 dk
            if (x.units > 0) {
                if (!wait_warp(acc_full, kn & 1, abort_flag)) { ok = false; break; }
                ++kn;
                tc::fence_after_sync();
            }
            const float f = g ? p.scale : 1.f;
            const uint32_t tA = lrow + (g ? KVT_K : KVT_V);
            unsigned char *stage = smem + L::OFF_STAGE + warp * 4096;
            T *out0 = (T *)(g ? p.dk : p.dv) + ((long long)x.k_row * p.Hkv + x.hk) * D;
            const int n_rows = x.n_keys - (warp & 3) * 32;        // of this warp's 32
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 64) {
                uint32_t o[64];
                if (x.units > 0) {
                    tmem_ld32(tA + c0, *reinterpret_cast<uint32_t(*)[32]>(o));
                    tmem_ld32(tA + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = 0u;
                }
                if (x.part >= 0) {
                    if (key_ok) {
                        float4 *dst = reinterpret_cast<float4 *>(
                            tl.part + (((long long)x.part * p.sinks + x.j0 + r) * 2 + g) * D + c0);
#pragma unroll
                        for (int e = 0; e < 64; e += 4)
                            dst[e / 4] = make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                                     __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                    }
                    continue;
                }
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16(__uint_as_float(o[8 * v + 2 * e]) * f, __uint_as_float(o[8 * v + 2 * e + 1]) * f);
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((v ^ (lane & 7)) * 16)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = k * 4 + lane / 8, v = lane % 8;
                    const uint4 y = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((v ^ (rr & 7)) * 16));
                    if (rr < n_rows)
                        *reinterpret_cast<uint4 *>(out0 + (long long)((warp & 3) * 32 + rr) * p.Hkv * D + c0 + v * 8) = y;
                }
                __syncwarp();
            }
            if (x.units > 0) {
                tc::fence_before_sync();
                arrive_warp(acc_free);
            }
        }
        if (!ok) fail();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

// dk and dv of the sinks that lie apart: the pieces' fp32 sums, one CTA per
// key and KV head; warp w takes pieces w, w + 8, ..., then the eight partial
// sums are added in order.
template <int D>
__global__ void __launch_bounds__(256) sink_dkv_join_kernel(const SinkParams p, const SinkKvTiles tl) {
    grid_dependency_sync();
    constexpr int E = 2 * D / 32;
    __shared__ float sums[8][2 * D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long rows = (long long)p.B * p.Hkv * p.sinks;
    for (long long w = blockIdx.x; w < rows; w += gridDim.x) {
        const int j = (int)(w % p.sinks);
        const long long bh = w / p.sinks;
        const int hk = (int)(bh % p.Hkv), b = (int)(bh / p.Hkv);
        const SinkSeq s = sink_seq(p, b);
        if (j >= sink_apart(p, s)) continue;
        float x[E] = {};
#pragma unroll 4
        for (int sp = warp; sp < tl.n_split; sp += 8) {
            int ta, te;
            sink_piece(s, tl.tps, sp, j / 128 * 128, ta, te);
            if (ta >= te) continue;
            const float4 *src = reinterpret_cast<const float4 *>(tl.part + ((bh * tl.n_split + sp) * p.sinks + j) * 2 * D +
                                                                 lane * E);
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 v = src[e / 4];
                x[e] += v.x; x[e + 1] += v.y; x[e + 2] += v.z; x[e + 3] += v.w;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = x[e];
        __syncthreads();
        // columns 0 .. D-1 are dv, the rest dk
        const int c = threadIdx.x;
        if (c < 2 * D) {
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y += sums[i][c];
            const long long row = (((p.cu_k ? 0 : b * p.L) + s.k0 + j) * p.Hkv + hk) * D;
            ((__nv_bfloat16 *)(c < D ? p.dv : p.dk))[row + c % D] = __float2bfloat16(y);
        }
        __syncthreads();
    }
}

}  // namespace sa
