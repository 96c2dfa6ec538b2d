// sink_fwd_tc.cuh -- forward of the sink-window attention on the tcgen05
// tensor cores.
//
// A work item is two row tiles (A, B) of 128 rows: TPT consecutive queries x
// the HB heads of a KV group (HB = min(G, 128), TPT = 128 / HB), row =
// query * HB + head, so both tiles read the same keys.  What any of the rows
// sees is two contiguous key ranges, [0, s_end) of the sinks and [band_lo,
// band_hi) of the windows, walked in tiles of up to 128 keys.  Per tile and
// row tile
//   S = Q K^T (tcgen05.mma, fp32 in tensor memory),  P = 2^(S c - m),  O += P V
// with the running maximum m and sum of a row held by one thread; P replaces
// S in tensor memory and is the A operand of the second product.  m is raised
// (and O rescaled) only when a tile exceeds it by more than 2^8.  P is
// rounded to the inputs' type (half a step a weight, as the output is); with
// SPLIT what that leaves enters as a second product, so that the output's own
// rounding is all that remains.
//
// The tensor cores and the softmax alternate between A and B: while one
// tile's scores are turned into weights the other's products run.  S and P of
// a row tile are held in two halves of 64 keys: while the softmax warps work on
// one, the product of the other and its next S run.  Each row tile's queue is
// S(0), S(1), then P.V(u), S(u + 2), ... over the halves u, across items.
// A tile of n < 128 keys costs N = n (rounded up to 16) columns in the first
// product and n rows in the second, but the softmax warps' way around a tile
// costs much the same: up to 16 sinks therefore share their tile with the
// first 112 keys of the band.  A row tile skips key
// tiles that none of its rows sees.
//
// Rows of V that not every row of the item sees are cleaned in shared memory
// first: 0 * inf would put NaN into rows that must not see them.  What is not
// finite there is added back, at the end, to the rows that do see it.  (With
// SPLIT every row is: the two parts of a weight times inf are inf - inf.)
//
// Warps: 0-3 softmax and epilogue of A (thread = row), 4-7 of B, 8 TMA
// producer, 9 and 10 MMA issuers of A and B (9 also owns the TMEM).
//
// Measured on one B200: 64K tokens, 16 heads on one KV head, window 2048, 128
// sinks 1.23 ms = 933 TFLOP/s (990 W, 1860 MHz); 7 ragged fp16 prompts, 8000
// tokens, 16 heads on 4, window 512, 73 us = 403 TFLOP/s.  Every wait is bounded; a timeout
// sets ERR_TIMEOUT and the CTA drains and exits.
#pragma once

#include "attn_tc.cuh"
#include "sink_attn.cuh"

namespace sa {

constexpr int SF_KT = 128;               // keys per tile
constexpr int SF_SLOTS = 4;              // ring of tiles: K, V of even key tiles, K, V of odd ones
constexpr int SF_THREADS = 384;          // 3 warpgroups; warp 11 only gives its registers away
// registers a thread: launched with 168 (384 x 168 = 64512); 2 x 208 + 88 = 3 x 168
constexpr int SF_REGS_SOFTMAX = 208, SF_REGS_ISSUE = 88;
constexpr uint32_t SF_TM_S = 0;          // S / P of A, B: 128 columns each
constexpr uint32_t SF_TM_O = 256;        // O of A, B: 128 columns each
constexpr uint32_t SF_TM_COLS = 512;
constexpr float SF_RAISE = 8.f;
constexpr int SF_HEAD = 16;              // sinks up to here share their tile with the band

template <int D>
struct SfSmem {
    static constexpr int TILE = 128 * D * 2;               // Q, K or V tile: D / 64 halves of 128 rows x 128 B
    static constexpr int OFF_Q = 0;                        // A, B
    static constexpr int OFF_KV = OFF_Q + 2 * TILE;
    static constexpr int OFF_STAGE = OFF_KV + SF_SLOTS * TILE;      // outputs: 32 rows x 128 B per softmax warp
    static constexpr int OFF_BAR = OFF_STAGE + 8 * 4096;
    // q_full[2], q_empty[2], kv_full[S], kv_empty[S], s_full[2][2], p_full[2][2], pv_done[2][2],
    // o_full[2], drain[2], item_full[2], item_empty[2]
    static constexpr int N_BAR = 4 + 2 * SF_SLOTS + 12 + 4 + 4;
    static constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;   // tmem slot, abort flag, dirty flag, tile info[2]
    static constexpr int OFF_ITEM = OFF_MISC + 32;         // two work items of the softmax warps
    static constexpr int TOTAL = OFF_ITEM + 2 * 64;
    static constexpr int ALLOC = TOTAL + 1024;
    static_assert(OFF_ITEM % 16 == 0 && ALLOC <= 232448, "items are copied by 16 bytes; 227 KB per CTA");
};

struct SinkTiles {
    int HB, HC, TPT;         // heads per row tile, head chunks per group, queries per row tile
    int per_seq;             // dense: query blocks of TPT * (row tiles per item) per sequence
    int items;               // query blocks (packed: an upper bound) * Hkv * HC
};

// One work item: its sequence, rows and key tiles.
struct SinkItem {
    SinkSeq s;
    int b, hk, h0, nh;       // h0: first head, nh: heads of the tile that belong to the group
    int t0, nq_i[2];         // first query; queries of A and B
    int band_lo, band_hi, s_end, nt;
    int n_sink;              // tiles that hold sinks; every row tile uses them
    int head;                // SF_HEAD: the sinks take these rows of a tile that they share with the band; 0: they
                             // have tiles of their own
    int base;                // tile j >= n_sink (and the shared one) starts at key base + 128 j
    int ja[2], jb[2];        // key tiles that A and B use: the sinks' and [ja, jb) (none: nq_i = 0)
    int clean_lo, clean_hi;  // keys of [band_lo, clean_lo) and [clean_hi, band_hi) are not seen by every row

    __device__ __forceinline__ void tile(int j, int &k0, int &n) const {
        const bool apart = j < n_sink && head == 0;
        k0 = (apart ? 0 : base) + j * SF_KT;
        n = min(SF_KT, (apart ? s_end : band_hi) - k0);
    }
    __device__ __forceinline__ bool active(int i, int j) const {
        return (i ? nq_i[1] : nq_i[0]) > 0 && (j < n_sink || (j >= (i ? ja[1] : ja[0]) && j < (i ? jb[1] : jb[0])));
    }
};
// Block blk of a packed batch in blocks of TI rows: its sequence and the
// block's number there.  Sequence b starts at block cu[b] / TI + b, so there
// is room for every sequence's last, partial block; blocks past it are empty.
__device__ __forceinline__ void sink_slot(const int32_t *cu, int B, int rows, unsigned TI, int blk, int &b, int &local) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        const unsigned c = (unsigned)min(max(__ldg(cu + m), 0), rows);
        if ((long long)(c / TI) + m <= blk) lo = m; else hi = m;
    }
    b = lo;
    local = blk - (int)((unsigned)min(max(__ldg(cu + lo), 0), rows) / TI + lo);
}
// Work item `it` of NT row tiles; false: it lies past its sequence.
template <int NT>
__device__ __forceinline__ bool sink_item(const SinkParams &p, const SinkTiles &tl, int it, SinkItem &x) {
    const int H2 = p.Hkv * tl.HC, blk = it / H2, hh = it - blk * H2;
    const int hc = tl.HC == 1 ? 0 : hh % tl.HC;
    const unsigned TI = NT * tl.TPT;
    x.hk = tl.HC == 1 ? hh : hh / tl.HC;
    x.h0 = x.hk * p.G + hc * tl.HB;
    x.nh = min(tl.HB, p.G - hc * tl.HB);
    int local;
    if (!p.cu_q) {
        x.b = blk / tl.per_seq;
        local = blk - x.b * tl.per_seq;
    } else {
        sink_slot(p.cu_q, p.B, (int)p.Tq, TI, blk, x.b, local);
    }
    x.s = sink_seq(p, x.b);
    if (local < 0 || (long long)local * TI >= x.s.nq) return false;
    x.t0 = local * TI;
    int s1, lo, hi;
    sink_visible(p, x.s.nk, x.s.pos0 + x.t0, s1, lo, hi);
    x.band_lo = lo;
    x.clean_hi = hi;
    x.s_end = min(p.sinks, lo);
    x.clean_lo = lo;
    x.band_hi = hi;
    int lo_min[2], hi_max[2], s1_max[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int ta = x.t0 + i * tl.TPT;
        x.nq_i[i] = i < NT ? max(0, min(tl.TPT, x.s.nq - ta)) : 0;
        lo_min[i] = hi_max[i] = s1_max[i] = 0;
        if (x.nq_i[i] == 0) continue;
        sink_visible(p, x.s.nk, x.s.pos0 + ta, s1, lo, hi);
        lo_min[i] = lo;
        sink_visible(p, x.s.nk, x.s.pos0 + ta + x.nq_i[i] - 1, s1, lo, hi);
        hi_max[i] = hi;
        s1_max[i] = s1;
        x.band_hi = hi;
        x.clean_lo = lo;
    }
    x.n_sink = (x.s_end + SF_KT - 1) / SF_KT;
    x.head = x.s_end > 0 && x.s_end <= SF_HEAD && x.band_hi > x.band_lo ? SF_HEAD : 0;
    x.base = x.band_lo - (x.head ? x.head : x.n_sink * SF_KT);
    x.nt = x.band_hi > x.band_lo ? (x.band_hi - x.base + SF_KT - 1) / SF_KT : x.n_sink;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // a row that still sees sinks inside the band needs the band from its start
        x.ja[i] = max(x.n_sink, s1_max[i] > x.band_lo ? 0 : (lo_min[i] - x.base) / SF_KT);
        x.jb[i] = hi_max[i] > x.band_lo ? (hi_max[i] - x.base + SF_KT - 1) / SF_KT : 0;
    }
    return true;
}

// 32 lanes x 32 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// box of a 4-D tensor map at (x, y, z, w)
__device__ __forceinline__ void load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
        : "memory");
}
// Maps of K or V: boxes of 128 rows, of SF_HEAD and of the rest.
struct KeyMaps { CUtensorMap all, head, rest; };
// Key tile j of item x (K or V: 128 rows) into dst.
template <int D>
__device__ __forceinline__ void load_keys(unsigned char *dst, const KeyMaps &m, const SinkItem &x, int j, int k0, int batch,
                                          uint64_t *bar) {
    const int row = (int)x.s.k0;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        unsigned char *to = dst + h * (SF_KT * 128);
        if (j > 0 || x.head == 0) {
            load_4d(to, &m.all, h * 64, x.hk, row + k0, batch, bar);
        } else {
            load_4d(to, &m.head, h * 64, x.hk, row, batch, bar);
            load_4d(to + SF_HEAD * 128, &m.rest, h * 64, x.hk, row + k0 + SF_HEAD, batch, bar);
        }
    }
}
// kind::f16 instruction descriptor operand format of T
template <typename T>
__host__ __device__ constexpr uint32_t ab_format() { return std::is_same<T, __nv_bfloat16>::value ? 1u : 0u; }
// Does a pair of 16-bit values hold an infinity or NaN (exponent all ones)?
template <typename T>
__device__ __forceinline__ bool not_finite16(uint32_t x) {
    constexpr uint32_t E = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    return (x & E) == E;
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// What rounding two values to T leaves, as a packed pair.
template <typename T>
__device__ __forceinline__ unsigned pack2_rest(float lo, float hi, unsigned packed) {
    const T *q = reinterpret_cast<const T *>(&packed);
    return pack2<T>(lo - to_f(q[0]), hi - to_f(q[1]));
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
// a wait of a whole warp, with one verdict
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, atc::wait(bar, parity, abort_flag)) != 0;
}
// one arrival for a warp, after all its lanes
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) atc::arrive(bar);
}
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
// bits [lo, hi) of a 32-bit word, bounds clamped
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    const uint32_t a = lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : 0xffffffffu << lo;
    const uint32_t b = hi <= 0 ? 0u : hi >= 32 ? 0xffffffffu : ~(0xffffffffu << hi);
    return a & b;
}

// What the softmax warps have to know of a work item (16 words).
struct alignas(16) SfItem {
    int nt;                  // key tiles; -1 ends the stream
    int nq[2];               // queries of A and B
    int pos;                 // position of the first query
    int band_lo, band_hi, s_end;
    int sinks;               // head / SF_HEAD << 28 | n_sink
    int ja[2], jb[2];
    int clean_lo, clean_hi;
    int heads;               // first head | heads of the tile << 20
    int row;                 // first query's row of the whole batch
};
// What the issuing warp has to know of a key tile, written by the producer
// beside it: columns / 16, who uses it, where its item begins and ends.
enum : uint32_t { TI_STEPS = 15u, TI_A = 16u, TI_B = 32u, TI_FIRST = 64u, TI_LAST = 128u, TI_TILE = 256u };

template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(SF_THREADS, 1)
    sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ KeyMaps kmap,
                       const __grid_constant__ KeyMaps vmap, const __grid_constant__ SinkParams p,
                       const __grid_constant__ SinkTiles tl) {
    grid_dependency_sync();
    using L = SfSmem<D>;
    constexpr int HALVES = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *q_full = bars, *q_empty = bars + 2, *kv_full = bars + 4, *kv_empty = kv_full + SF_SLOTS;
    uint64_t *s_full = kv_empty + SF_SLOTS, *p_full = s_full + 4, *pv_done = p_full + 4, *o_full = pv_done + 4;
    uint64_t *drain = o_full + 2;
    uint64_t *item_full = drain + 2, *item_empty = item_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    volatile int *dirty = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 8);
    volatile uint32_t *info_s = reinterpret_cast<volatile uint32_t *>(smem + L::OFF_MISC + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, SF_TM_COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + i, 1); tc::mbar_init(q_empty + i, 1);
            tc::mbar_init(o_full + i, 1);
            for (int h = 0; h < 2; ++h) {
                tc::mbar_init(s_full + 2 * i + h, 1); tc::mbar_init(p_full + 2 * i + h, 4);
                tc::mbar_init(pv_done + 2 * i + h, 1);
            }
            tc::mbar_init(drain + i, 1);
            tc::mbar_init(item_full + i, 1); tc::mbar_init(item_empty + i, 8);
        }
        for (int i = 0; i < SF_SLOTS; ++i) { tc::mbar_init(kv_full + i, 1); tc::mbar_init(kv_empty + i, 2); }
        *abort_flag = 0;
        *dirty = 0;
        tc::mbar_fence_init();
    }
    sink_report(p);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        raise_error(p.err, ERR_TIMEOUT);
        *abort_flag = 1;
    };

    // ------------------------------------------------------------------- MMA
    // One warp per row tile walks the tile stream (uniform control flow and
    // operands); one lane issues.  Its instructions run one after the other at
    // their latency, so what it has to know of a tile comes ready from the
    // producer, and two warps share the issuing.
    auto issue = [&](auto which) {
        constexpr int I = decltype(which)::value;
        constexpr uint32_t F = ab_format<T>();
        constexpr uint32_t ID_O = tc::make_idesc(1, F, 128, D) | (1u << 16);    // B (V) MN-major
        constexpr uint32_t TSTEP = L::TILE >> 4;      // descriptor step between tiles
        constexpr uint32_t USES = I == 0 ? TI_A : TI_B;
        const bool leader = elect_one();
        const uint64_t qd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_Q + I * L::TILE), 16, 1024);
        const uint64_t kd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_KV), 16, 1024);
        // V: MN-major, 64-column atoms SF_KT * 128 B apart, 8-key groups 1 KB apart
        const uint64_t vd = atc::desc_sw128(tc::smem_u32(smem + L::OFF_KV), SF_KT * 128, 1024);
        const uint32_t tS = tmem + SF_TM_S + I * 128, tO = tmem + SF_TM_O + I * 128;
        bool ok = true;
        uint32_t qpar = 1;                            // parity of the current item's Q
        uint32_t ppar = 0;                            // parities of P's halves in bits 0, 1
        uint32_t begun = 0;                           // O holds a product of the current item
        // S over half h of the key tile in K slot k
        auto issue_s = [&](uint32_t info, int k, int h) {
            const int steps = (int)(info & TI_STEPS) - 4 * h;      // 16-key steps of this half
            if ((info & USES) && steps > 0 && leader) {
                const uint32_t id = tc::make_idesc(1, F, 128, 0) | ((uint32_t)min(steps, 4) << 18);   // N / 8 at bit 17
                const uint64_t b = kd + k * TSTEP + h * (64 * 128 >> 4);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const int off = ((c / 4) * (128 * 128) + (c % 4) * 32) >> 4;
                    tc::mma_bf16(tS + h * 64, qd + off, b + off, id, c > 0 ? 1u : 0u);
                }
                tc::mma_commit(s_full + 2 * I + h);
            }
        };
        ok = wait_warp(kv_full + 0, 0, abort_flag);
        uint32_t info = ok ? info_s[0] : 0u;
        if (info & TI_TILE) {
            qpar ^= 1;
            ok = wait_warp(q_full + I, qpar, abort_flag);
            if (ok) {
                tc::fence_after_sync();
                issue_s(info, 0, 0);
                issue_s(info, 0, 1);
                if (leader) {
                    tc::mma_commit(kv_empty + 0);
                    if (info & TI_LAST) tc::mma_commit(q_empty + I);
                }
            }
        }
        uint32_t t = 0;                               // key tile; K of tile t in slot 2 (t & 1), V in the next
        while (ok && (info & TI_TILE)) {
            const int vs = 2 * (t & 1) + 1, ks = 2 * ((t + 1) & 1);
            if (!(ok = wait_warp(kv_full + vs, (t >> 1) & 1, abort_flag) &&
                       wait_warp(kv_full + ks, ((t + 1) >> 1) & 1, abort_flag)))
                break;
            const uint32_t next = info_s[ks / 2];
            if (next & TI_FIRST) {
                qpar ^= 1;
                if (!(ok = wait_warp(q_full + I, qpar, abort_flag))) break;
            }
            const uint64_t v = vd + vs * TSTEP;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int steps = (int)(info & TI_STEPS) - 4 * h;
                if ((info & USES) && steps > 0) {
                    // the softmax warps write an item's first P after they have read the O of the item before
                    if (!(ok = wait_warp(p_full + 2 * I + h, (ppar >> h) & 1, abort_flag))) break;
                    tc::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (c < steps)
                                tc::mma_bf16_ts(tO, tS + h * 64 + c * 8, v + (4 * h + c) * 128, ID_O, c > 0 ? 1u : begun);
                        if constexpr (SPLIT) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c < steps)
                                    tc::mma_bf16_ts(tO, tS + h * 64 + 32 + c * 8, v + (4 * h + c) * 128, ID_O, 1u);
                        }
                        tc::mma_commit(pv_done + 2 * I + h);
                    }
                    ppar ^= 1u << h;
                    begun = 1;
                }
                if ((info & TI_LAST) && begun && h == ((info & TI_STEPS) > 4 ? 1 : 0) && leader)
                    tc::mma_commit(o_full + I);       // the item's last product
                tc::fence_after_sync();
                issue_s(next, ks, h);                 // into the half whose P this product has read
            }
            if (!ok) break;
            if (leader) {
                tc::mma_commit(kv_empty + vs);
                if (next & TI_TILE) tc::mma_commit(kv_empty + ks);
                if (next & TI_LAST) tc::mma_commit(q_empty + I);
            }
            if (info & TI_LAST) begun = 0;
            info = next;
            ++t;
        }
        if (lane == 0 && !ok) fail();
        if (leader) {
            tc::mma_commit(drain + I);
            tc::mbar_wait_bounded(drain + I, 0, ATC_WAIT);
        }
    };

    if (warp >= 8) {
        regs_dec<SF_REGS_ISSUE>();
        if (warp == 8 && lane == 0 && !debug_stall()) {      // (test hook: nothing is loaded)
            // -------------------------------------------------- TMA producer
            // ring order K 0, V 0, K 1, V 1, ... over all items' tiles, then an empty K that ends the stream
            bool ok = true;
            int qn = 0, kv = 0, in = 0;               // items with keys and ring tiles loaded, items handed over
            int q_loads[2] = {0, 0};
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
                if (!sink_item<2>(p, tl, it, x)) continue;
                ok = hand_over(SfItem{x.nt, {x.nq_i[0], x.nq_i[1]}, (int)x.s.pos0 + x.t0, x.band_lo, x.band_hi, x.s_end,
                                      x.n_sink | x.head / SF_HEAD << 28, {x.ja[0], x.ja[1]}, {x.jb[0], x.jb[1]}, x.clean_lo, x.clean_hi,
                                      x.h0 | x.nh << 20,
                                      (int)((p.cu_q ? 0 : x.b * p.Tq) + x.s.q0) + x.t0});
                if (!ok) break;
                if (x.nt == 0) continue;
                const int qb = p.cu_q ? 0 : x.b;
                auto load_q = [&](int i) -> bool {
                    if (!atc::wait(q_empty + i, (qn & 1) ^ 1, abort_flag)) return false;
                    atc::expect_tx(q_full + i, HALVES * 128 * tl.HB * tl.TPT);
                    for (int h = 0; h < HALVES; ++h)
                        load_4d(smem + L::OFF_Q + i * L::TILE + h * (128 * 128), &qmap, h * 64, x.h0,
                                (int)(x.s.q0 + x.t0 + i * tl.TPT), qb, q_full + i);
                    ++q_loads[i];
                    return true;
                };
                for (int j = 0; j < x.nt && ok; ++j) {
                    int k0, n;
                    x.tile(j, k0, n);
                    for (int v = 0; v < 2 && ok; ++v, ++kv) {
                        const int sl = kv % SF_SLOTS;
                        ok = atc::wait(kv_empty + sl, ((kv / SF_SLOTS) & 1) ^ 1, abort_flag);
                        if (!ok) break;
                        if (v == 0)
                            info_s[sl / 2] = (uint32_t)((n + 15) / 16) | (x.active(0, j) ? TI_A : 0u) |
                                             (x.active(1, j) ? TI_B : 0u) | (j == 0 ? TI_FIRST : 0u) |
                                             (j + 1 == x.nt ? TI_LAST : 0u) | TI_TILE;
                        atc::expect_tx(kv_full + sl, L::TILE);
                        load_keys<D>(smem + L::OFF_KV + sl * L::TILE, v ? vmap : kmap, x, j, k0, qb, kv_full + sl);
                        if (j == 0 && v == 0) ok = load_q(0) && load_q(1);
                    }
                }
                ++qn;
            }
            if (ok) {
                const int sl = kv % SF_SLOTS;
                ok = atc::wait(kv_empty + sl, ((kv / SF_SLOTS) & 1) ^ 1, abort_flag);
                if (ok) ok = hand_over(SfItem{-1});
                if (ok) {
                    info_s[sl / 2] = 0u;
                    atc::arrive(kv_full + sl);
                    ++kv;
                }
            }
            if (!ok) fail();
            // let the copies land before the CTA exits
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (q_loads[i] > 0) tc::mbar_wait_bounded(q_full + i, (q_loads[i] - 1) & 1, ATC_WAIT);
            for (int i = 0; i < SF_SLOTS && i < kv; ++i) {
                const int t = kv - 1 - i;
                tc::mbar_wait_bounded(kv_full + t % SF_SLOTS, (t / SF_SLOTS) & 1, ATC_WAIT);
            }
        } else if (warp == 9) {
            issue(std::integral_constant<int, 0>{});
        } else if (warp == 10) {
            issue(std::integral_constant<int, 1>{});
        }
        __syncwarp();
    } else {
        regs_inc<SF_REGS_SOFTMAX>();
        // --------------------------------------------- softmax and epilogue
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;      // row tile, row of it
        const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lrow + SF_TM_S + i * 128, tO = tmem + lrow + SF_TM_O + i * 128;
        const int tt = r / tl.HB, hh = r - tt * tl.HB;
        unsigned char *stage = smem + L::OFF_STAGE + warp * 4096;
        bool ok = true;
        uint32_t spar = 0, opar = 0;                  // parities of S's halves in bits 0, 1; of o_full
        uint32_t kt0 = 0;                             // key tiles of the stream before this item
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
            const int nqi = i ? x.nq[1] : x.nq[0], ja = i ? x.ja[1] : x.ja[0], jb = i ? x.jb[1] : x.jb[0];
            const bool row_ok = tt < nqi && hh < (x.heads >> 20);
            int s1 = 0, lo = -(1 << 30), hi = 1 << 30;    // rows of nobody: anything, never written
            if (row_ok) {
                const int pos = x.pos + i * tl.TPT + tt;
                hi = min(max(pos + 1, 0), x.band_hi);     // the last row of the item sees up to band_hi
                lo = min(max(pos - p.window + 1, 0), hi);
                s1 = min(p.sinks, lo);
            }
            float m = -INFINITY, l = 0.f;
            bool first = true;
            uint32_t used = 0;                        // halves with a product into this item's O
            // the sinks' tiles, then [ja, jb): next tile j at key k0, the range's end, the range to clean
            const int n_sink = x.sinks & 0xfffffff, head = (x.sinks >> 28) * SF_HEAD;
            const int base = x.band_lo - (head ? head : n_sink * SF_KT);
            bool in_sink = n_sink > 0;
            int j = in_sink ? 0 : ja, jend = in_sink ? n_sink : jb;
            const bool apart = in_sink && head == 0;
            int k0 = (apart ? 0 : base) + j * SF_KT, kend = apart ? x.s_end : x.band_hi;
            int cl = apart ? 0 : x.clean_lo, ch = apart ? x.s_end : x.clean_hi;
            if (nqi > 0) for (;; ++j, k0 += SF_KT) {
                if (j >= jend) {
                    if (!in_sink || ja >= jb) break;
                    in_sink = false;
                    j = ja; jend = jb; k0 = base + ja * SF_KT; kend = x.band_hi;
                    cl = x.clean_lo; ch = x.clean_hi;
                }
                const int n = min(SF_KT, kend - k0), n16 = (n + 15) & ~15;
                const int sh = in_sink ? head : 0;         // rows of the tile that the sinks share
                // clean the rows of V that not every row of the item sees.  Both row tiles do, each before its own
                // P: their products are issued by different warps, and cleaning twice changes nothing
                if (SPLIT || k0 + sh < cl || k0 + n16 > ch || sh > x.s_end) {
                    const uint32_t kt = kt0 + j;
                    const int sl = 2 * (kt & 1) + 1, ca = SPLIT ? n : min(n, max(0, cl - k0)), cb = min(n, max(0, ch - k0));
                    if (!wait_warp(kv_full + sl, (kt >> 1) & 1, abort_flag)) { ok = false; break; }
                    // 16-byte units of the rows [0, ca) and [cb, n16)
                    constexpr int U = D / 8;
                    const int gap = max(cb, ca) - ca, rows = n16 - gap;
#pragma unroll 1
                    for (int u = r; u < rows * U; u += 128) {
                        int key = u / U;
                        const int c = u % U;
                        if (key >= ca) key += gap;
                        if (!SPLIT && key < sh && key < x.s_end) continue;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + L::OFF_KV + sl * L::TILE + (c / 8) * (SF_KT * 128) +
                                                              key * 128 + (((c & 7) ^ (key & 7)) * 16));
                        if (key >= n || (key < sh && key >= x.s_end)) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        uint4 v = *at;
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        bool bad = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (not_finite16<T>(w[e])) { w[e] &= 0xffff0000u; bad = true; }
                            if (not_finite16<T>(w[e] >> 16)) { w[e] &= 0xffffu; bad = true; }
                        }
                        if (bad) {
                            *dirty = 1;               // first: the other row tile may find the unit clean
                            __threadfence_block();
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    tc::fence_proxy_async_smem();
                }
                // sinks: the columns [sh, v1), and of a shared tile [0, sees)
                const int v1 = s1 - k0, sees = sh ? min(s1, x.s_end) : 0;
                const bool row_whole = ((k0 >= lo && k0 + n <= hi) || k0 + n <= s1) && sh == 0;
                const bool whole = __all_sync(0xffffffffu, row_whole);
#pragma unroll 1
                for (int h = 0; h * 64 < n; ++h) {
                    // S of this half; the other half's was issued before, its P.V may still run
                    if (!wait_warp(s_full + 2 * i + h, (spar >> h) & 1, abort_flag)) { ok = false; break; }
                    tc::fence_after_sync();
                    const int c0 = h * 64, nh = n - c0;
                    uint32_t s[64];
                    tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(s));
                    tmem_ld32(tS + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                    tc::tmem_ld_wait();
                    if (!whole || nh < 64) {
#pragma unroll
                        for (int c = 0; c < 64; c += 32) {
                            const int q = c0 + c;
                            const uint32_t vis = (bit_range(lo - k0 - q, hi - k0 - q) | bit_range(sh - q, v1 - q) |
                                                  bit_range(-q, sees - q)) & bit_range(0, n - q);
                            if (__any_sync(0xffffffffu, vis != 0xffffffffu)) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!((vis >> e) & 1u)) s[c + e] = __float_as_uint(-INFINITY);
                            }
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                    const bool raise = mt > m + (m == -INFINITY ? 0.f : SF_RAISE);
                    float alpha = 1.f;
                    if (raise) {
                        alpha = m == -INFINITY ? 0.f : ex2_fast(m - mt);
                        m = mt;
                        l *= alpha;
                    }
                    if (!first && __any_sync(0xffffffffu, raise)) {
                        // every product into O so far: the last one of each half (one of them is older and done)
                        bool got = true;
                        if (used & 1u) got = wait_warp(pv_done + 2 * i, ((spar & 1) ^ 1), abort_flag);
                        if (used & 2u) got = wait_warp(pv_done + 2 * i + 1, ((spar >> 1) & 1) ^ 1, abort_flag) && got;
                        if (!got) { ok = false; break; }
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o16[16];
                            tc::tmem_ld16(tO + c, o16);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o16[e] = __float_as_uint(__uint_as_float(o16[e]) * alpha);
                            atc::tmem_st16(tO + c, o16);
                        }
                    }
                    first = false;
                    used |= 1u << h;
                    spar ^= 1u << h;
                    const float nb = m == -INFINITY ? 0.f : -m;
                    const uint64_t nb2 = f2_pack(nb, nb), sc2 = f2_pack(p.scale_log2, p.scale_log2);
                    uint64_t rs[2] = {0ull, 0ull};
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t pk[16], pr[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float p0, p1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), sc2, nb2),
                                      p0, p1);
                            p0 = ex2_fast(p0);
                            p1 = ex2_fast(p1);
                            rs[(e >> 1) & 1] = f2_add(rs[(e >> 1) & 1], f2_pack(p0, p1));
                            pk[e / 2] = pack2<T>(p0, p1);
                            if constexpr (SPLIT) pr[e / 2] = pack2_rest<T>(p0, p1, pk[e / 2]);
                        }
                        atc::tmem_st16(tS + c0 + c / 2, pk);
                        if constexpr (SPLIT) atc::tmem_st16(tS + c0 + 32 + c / 2, pr);
                    }
                    float r0, r1;
                    f2_unpack(f2_add(rs[0], rs[1]), r0, r1);
                    l += r0 + r1;
                    atc::tmem_st_wait();
                    tc::fence_before_sync();
                    arrive_warp(p_full + 2 * i + h);
                }
                if (!ok) break;
            }
            if (!ok) break;
            kt0 += x.nt;
            // ------------------------------------------------------ epilogue
            if (nqi == 0) continue;
            // rows of the output relative to the tile's first; -1: nobody's
            const int row_at = row_ok ? tt * p.Hq + hh : -1;
            const long long row0 = (long long)(x.row + i * tl.TPT) * p.Hq + (x.heads & 0xfffff);
            T *out0 = (T *)p.out + row0 * D;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (row_ok) p.lse[row0 + row_at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            if (!first) {
                if (!wait_warp(o_full + i, opar, abort_flag)) { ok = false; break; }
                opar ^= 1;
                tc::fence_after_sync();
            }
            const bool patch = *dirty != 0 && row_ok;  // set once, for every later item of this CTA
            const uint64_t inv2 = f2_pack(inv, inv);
            // 64 columns at a time through the warp's own shared memory, so that whole lines are written
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 64) {
                uint32_t o[64];
                if (first) {                          // no key tile: O holds nothing of this item
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = 0u;
                } else {
                    tmem_ld32(tO + c0, *reinterpret_cast<uint32_t(*)[32]>(o));
                    tmem_ld32(tO + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        float a, b;
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), inv2), a, b);
                        o[e] = __float_as_uint(a);
                        o[e + 1] = __float_as_uint(b);
                    }
                }
                if (__any_sync(0xffffffffu, patch)) {
                    if (patch) {
                        const long long qr = x.row;
                        const int b = p.cu_q ? sink_find(p.cu_q, p.B, qr) : (int)(qr / p.Tq);
                        const SinkSeq sq = sink_seq(p, max(b, 0));
                        const T *vb = (const T *)p.v + (p.cu_q ? 0 : b) * p.v_s[0] + sq.k0 * p.v_s[1] +
                                      (x.heads & 0xfffff) / p.G * p.v_s[2] + c0;
#pragma unroll 1
                        for (int k = SPLIT ? 0 : x.band_lo; k < x.band_hi; ++k) {
                            if (SPLIT) {
                                if (k >= x.s_end && k < x.band_lo) k = x.band_lo;
                            } else if (k == x.clean_lo && k < x.clean_hi) {
                                k = x.clean_hi;
                            }
                            if (k >= x.band_hi) break;
                            if (!(k < s1 || (k >= lo && k < hi))) continue;
#pragma unroll
                            for (int e = 0; e < 64; ++e) {
                                const float v = to_f(vb[k * p.v_s[1] + e]);
                                if (!isfinite(v)) o[e] = __float_as_uint(__uint_as_float(o[e]) + v);
                            }
                        }
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack2<T>(__uint_as_float(o[8 * u + 2 * e]), __uint_as_float(o[8 * u + 2 * e + 1]));
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((u ^ (lane & 7)) * 16)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                // 8 lanes per row, 4 rows at a time
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = k * 4 + lane / 8, u = lane % 8;
                    const int to = __shfl_sync(0xffffffffu, row_at, rr);
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((u ^ (rr & 7)) * 16));
                    if (to >= 0) *reinterpret_cast<uint4 *>(out0 + (long long)to * D + c0 + u * 8) = v;
                }
                __syncwarp();
            }
            tc::fence_before_sync();
        }
        if (!ok) fail();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) tc::tmem_dealloc(tmem, SF_TM_COLS);
}

}  // namespace sa
