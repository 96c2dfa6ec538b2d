// paged_books.cuh -- the pages of a cache: handing them out, writing new
// tokens, forking, freeing, compacting.
//
// The books (block_table, seq_lens, refcount) are small; what they cost is
// latency, so each call is one kernel of one cluster of 8 CTAs, whose 256
// warps each own a run of page ids: count what is looked for (ballots),
// exchange the counts through distributed shared memory, and walk the run
// again with the rank of every page known.  Ranks follow the page ids and the
// list order, so the books do not depend on timing.  The pages themselves
// move in a second kernel at copy bandwidth (paged_copy_kernel: 1.5 GB read and
// written by a compaction in 258 us = 5.8 TB/s, 89 % of a copy's rate).
#pragma once

#include <cooperative_groups.h>

#include "sa_common.cuh"

namespace sa {

namespace cg = cooperative_groups;

constexpr int PB_CTAS = 8;
constexpr int PB_THREADS = 1024;
constexpr int PB_WARPS = PB_CTAS * PB_THREADS / 32;
constexpr int PB_ENDS = 4096;               // list entries whose page counts are kept in shared memory

struct BooksParams {
    int32_t *table, *lens, *refcount;
    int S, max_pages, page;
    long long n_pages;
    const int32_t *a, *c;                   // extend: seqs, n_new; fork: src, dst
    int n;
    int32_t *result;                        // start / done / n_live
    // workspace
    int32_t *owner;                         // [S] first list entry that names the sequence as its own
    int32_t *srcmark;                       // fork, [S]: the sequence is a src of the list
    int32_t *ends;                          // [n] pages needed by entries 0 .. i (capped above n_pages)
    int32_t *seq;                           // [n] sequence served by entry i, -1 = none
    int32_t *from, *to;                     // page moves
    int32_t *n_moves;                       // compact: {moves, first src rank}
    int32_t *map;                           // compact: [n_pages] new id of a moved page
    unsigned *err;
};

// Pages per warp of the cluster, a multiple of 32.
__device__ __forceinline__ long long pb_run(long long n_pages) {
    return ((n_pages + PB_WARPS - 1) / PB_WARPS + 31) / 32 * 32;
}
// Number of matching pages in this warp's run, for every warp of the cluster:
// returns the count before this warp; total over all.  Ends with a cluster
// barrier, so what any thread wrote before it is visible after it.
template <bool LIVE>
__device__ __forceinline__ int pb_rank(const BooksParams &p, int *counts, int &total) {
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, gw = (int)cl.block_rank() * 32 + (threadIdx.x >> 5);
    const long long run = pb_run(p.n_pages), lo = gw * run, hi = min(p.n_pages, lo + run);
    int n = 0;
    for (long long i = lo + lane; i < hi; i += 32) n += (p.refcount[i] > 0) == LIVE;
    n = warp_sum_int(n);
    if (lane == 0) counts[threadIdx.x >> 5] = n;
    cl.sync();
    int before = 0, all = 0;
#pragma unroll
    for (int r = 0; r < PB_CTAS; ++r) {
        const int x = cl.map_shared_rank(counts, r)[lane];
        all += x;
        if (r * 32 + lane < gw) before += x;
    }
    total = warp_sum_int(all);
    before = warp_sum_int(before);
    cl.sync();
    return before;
}
// Calls f(page id, rank) for the matching pages of this warp's run.
template <bool LIVE, typename F>
__device__ __forceinline__ void pb_walk(const BooksParams &p, int before, int limit, F &&f) {
    const int lane = threadIdx.x & 31;
    const int gw = (int)cg::this_cluster().block_rank() * 32 + (threadIdx.x >> 5);
    const long long run = pb_run(p.n_pages), lo = gw * run, hi = min(p.n_pages, lo + run);
    for (long long i0 = lo; i0 < hi && before < limit; i0 += 32) {
        const long long i = i0 + lane;
        const bool hit = i < hi && (p.refcount[i] > 0) == LIVE;
        const unsigned b = __ballot_sync(0xffffffffu, hit);
        const int r = before + __popc(b & ((1u << lane) - 1u));
        if (hit && r < limit) f((int)i, r);
        before += __popc(b);
    }
}
// First entry whose end lies above rank r.
__device__ __forceinline__ int pb_entry(const int32_t *ends, int n, int r) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int m = (lo + hi) / 2;
        if (ends[m] > r) hi = m; else lo = m + 1;
    }
    return lo;
}
// Running sums of need(i) over the list, written to ends; by CTA 0 of the
// cluster.  Capped at n_pages + 1: no comparison with a number of free pages
// tells larger values apart.  Two neighbours at the cap do look alike, so
// whether an entry needs pages is never read off a difference of ends.
template <typename F>
__device__ __forceinline__ void pb_ends(const BooksParams &p, int *warp_sums, F &&need) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long carry = 0;
    for (int i0 = 0; i0 < p.n; i0 += PB_THREADS) {
        const int i = i0 + tid;
        int x = i < p.n ? need(i) : 0;
        // an entry needs at most max_pages < 2^26 pages (checked by the host): a warp's sum fits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        long long before = carry, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += warp_sums[w];
            all += warp_sums[w];
        }
        __syncthreads();
        if (i < p.n) p.ends[i] = (int32_t)min(before + x, p.n_pages + 1);
        carry = min(carry + all, p.n_pages + 1);
    }
}

// Pages that `add` tokens behind the first `old` take beyond those of the first.
__device__ __forceinline__ int pb_more(int page, int old, int add) {
    return (int)(((long long)old + add + page - 1) / page - ((long long)old + page - 1) / page);
}

__global__ void __cluster_dims__(PB_CTAS, 1, 1) __launch_bounds__(PB_THREADS) paged_extend_kernel(const BooksParams p) {
    grid_dependency_sync();
    __shared__ int counts[32], warp_sums[32];
    __shared__ int ends_s[PB_ENDS];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x;
    const long long cap = (long long)p.max_pages * p.page;
    if (cl.block_rank() == 0) {
        // a sequence belongs to the first entry that names it
        for (int i = tid; i < p.n; i += PB_THREADS)
            if (p.a[i] >= 0 && p.a[i] < p.S) p.owner[p.a[i]] = INT_MAX;
        __syncthreads();
        for (int i = tid; i < p.n; i += PB_THREADS)
            if (p.a[i] >= 0 && p.a[i] < p.S) atomicMin(&p.owner[p.a[i]], i);
        __syncthreads();
        pb_ends(p, warp_sums, [&](int i) -> int {
            const int s = p.a[i], add = p.c[i];
            int old = 0;
            const bool ok = s >= 0 && s < p.S && p.owner[s] == i && add >= 0 && (old = p.lens[s]) >= 0 &&
                            (long long)old <= cap;
            const bool fits = ok && (long long)old + add <= cap;
            if (!ok) raise_error(p.err, ERR_BAD_INDEX);
            p.seq[i] = fits ? s : -1;
            return fits ? pb_more(p.page, old, add) : 0;
        });
    }
    int n_free;
    const int before = pb_rank<false>(p, counts, n_free);      // its barrier publishes ends and seq
    const int need = p.n > 0 ? p.ends[p.n - 1] : 0;
    const bool in_smem = p.n <= PB_ENDS;
    if (in_smem) {
        for (int i = tid; i < p.n; i += PB_THREADS) ends_s[i] = p.ends[i];
        __syncthreads();
    }
    const int32_t *ends = in_smem ? ends_s : p.ends;
    pb_walk<false>(p, before, min(need, n_free), [&](int id, int r) {
        const int i = pb_entry(ends, p.n, r);
        if (ends[i] > n_free) return;                          // the pool does not hold this entry's pages
        const int s = p.seq[i], first = i > 0 ? ends[i - 1] : 0;
        const int have = (int)(((long long)p.lens[s] + p.page - 1) / p.page);
        p.table[(size_t)s * p.max_pages + have + (r - first)] = id;
        p.refcount[id] = 1;
    });
    cl.sync();                                                 // every length has been read
    if (cl.block_rank() == 0)
        for (int i = tid; i < p.n; i += PB_THREADS) {
            const int s = p.seq[i];
            int st = -1;
            if (s >= 0) {
                const int old = p.lens[s], add = p.c[i];
                if (ends[i] <= n_free || pb_more(p.page, old, add) == 0) {
                    st = old;
                    p.lens[s] = old + add;
                }
            }
            p.result[i] = st;
        }
}

__global__ void __cluster_dims__(PB_CTAS, 1, 1) __launch_bounds__(PB_THREADS) paged_fork_kernel(const BooksParams p) {
    grid_dependency_sync();
    __shared__ int counts[32], warp_sums[32];
    __shared__ int ends_s[PB_ENDS];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31;
    auto in = [&](int s) { return s >= 0 && s < p.S; };
    auto held = [&](int s, int &len) -> bool {                // a sequence whose length its row can hold
        len = in(s) ? p.lens[s] : -1;
        return len >= 0 && (long long)len <= (long long)p.max_pages * p.page;
    };
    // an entry whose row names a page outside the pool is refused before any page is counted for it: a warp per
    // entry looks its row over (to[i] = 1 where it does)
    for (int i = (int)cl.block_rank() * 32 + (tid >> 5); i < p.n; i += PB_WARPS) {
        const int s = p.a[i];
        int len;
        bool out = false;
        if (held(s, len)) {
            const int32_t *row = p.table + (size_t)s * p.max_pages;
            const int pages = (int)(((long long)len + p.page - 1) / p.page);
#pragma unroll 8
            for (int k = lane; k < pages; k += 32) out |= row[k] >= p.n_pages;
        }
        out = __any_sync(0xffffffffu, out);
        if (lane == 0) p.to[i] = out;
    }
    cl.sync();
    if (cl.block_rank() == 0) {
        for (int i = tid; i < p.n; i += PB_THREADS) {
            if (in(p.c[i])) { p.owner[p.c[i]] = INT_MAX; p.srcmark[p.c[i]] = 0; }
            if (in(p.a[i])) p.owner[p.a[i]] = INT_MAX;
        }
        __syncthreads();
        for (int i = tid; i < p.n; i += PB_THREADS) {
            if (in(p.c[i])) atomicMin(&p.owner[p.c[i]], i);
            if (in(p.a[i])) p.srcmark[p.a[i]] = 1;
        }
        __syncthreads();
        pb_ends(p, warp_sums, [&](int i) -> int {
            const int s = p.a[i], d = p.c[i];
            int len, need = 0;
            bool ok = held(s, len) && in(d) && p.owner[d] == i && p.owner[s] == INT_MAX && p.srcmark[d] == 0 &&
                      p.lens[d] == 0 && p.to[i] == 0;
            if (ok && len % p.page) need = ok = p.table[(size_t)s * p.max_pages + len / p.page] >= 0;
            if (!ok) raise_error(p.err, ERR_BAD_INDEX);
            p.seq[i] = ok ? s : -1;
            p.from[i] = p.to[i] = -1;
            return need;
        });
    }
    int n_free;
    const int before = pb_rank<false>(p, counts, n_free);
    const int need = p.n > 0 ? p.ends[p.n - 1] : 0;
    const bool in_smem = p.n <= PB_ENDS;
    if (in_smem) {
        for (int i = tid; i < p.n; i += PB_THREADS) ends_s[i] = p.ends[i];
        __syncthreads();
    }
    const int32_t *ends = in_smem ? ends_s : p.ends;
    // fresh pages for the last, partly filled ones
    pb_walk<false>(p, before, min(need, n_free), [&](int id, int r) {
        const int i = pb_entry(ends, p.n, r), s = p.seq[i], d = p.c[i], full = p.lens[s] / p.page;
        p.from[i] = p.table[(size_t)s * p.max_pages + full];
        p.to[i] = id;
        p.table[(size_t)d * p.max_pages + full] = id;
        p.refcount[id] = 1;
    });
    // the shared pages: one warp per entry; the fresh page's place is the walk's
    for (int i = (int)cl.block_rank() * 32 + (tid >> 5); i < p.n; i += PB_WARPS) {
        const int s = p.seq[i];
        if (s < 0) continue;
        const int d = p.c[i], len = p.lens[s], full = len / p.page;
        const bool tail = len % p.page != 0;
        if (tail && ends[i] > n_free) continue;
        for (int k = lane; k < p.max_pages; k += 32) {
            if (tail && k == full) continue;
            int id = -1;
            if (k < full) {
                id = p.table[(size_t)s * p.max_pages + k];
                if (id >= 0 && atomicAdd(&p.refcount[id], 1) <= 0) raise_error(p.err, ERR_BAD_INDEX);
            }
            p.table[(size_t)d * p.max_pages + k] = id;
        }
    }
    // dst lengths: no dst is a src, so nothing above reads them
    if (cl.block_rank() == 0)
        for (int i = tid; i < p.n; i += PB_THREADS) {
            const int s = p.seq[i], len = s >= 0 ? p.lens[s] : 0;
            const bool ok = s >= 0 && (len % p.page == 0 || ends[i] <= n_free);
            if (ok) p.lens[p.c[i]] = len;
            p.result[i] = ok;
        }
}

// One thread per table entry of a listed sequence: the exchange and the count
// are two dependent trips to L2, so they go side by side (a warp per sequence
// that walked its row took 36 us for 192 rows of 1025 entries).  An entry is
// taken out by an exchange, so a sequence that is listed twice gives each page
// back once.
__global__ void __launch_bounds__(256) paged_free_kernel(const BooksParams p, int window, int sinks) {
    grid_dependency_sync();
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int s = p.a[i];
        if (s < 0 || s >= p.S) {
            if (blockIdx.y == 0 && threadIdx.x == 0) raise_error(p.err, ERR_BAD_INDEX);
            continue;
        }
        const long long gone = window > 0 ? (long long)p.lens[s] - window : 0;
        for (int k = blockIdx.y * 256 + threadIdx.x; k < p.max_pages; k += gridDim.y * 256) {
            const long long lo = (long long)k * p.page;
            if (window > 0 && (lo < sinks || lo + p.page > gone)) continue;
            int *at = &p.table[(size_t)s * p.max_pages + k];
            if (*at == -1) continue;
            const int id = atomicExch(at, -1);
            if (id < 0) continue;
            if (id >= p.n_pages) { raise_error(p.err, ERR_BAD_INDEX); continue; }
            if (atomicSub(&p.refcount[id], 1) <= 0) {
                atomicAdd(&p.refcount[id], 1);
                raise_error(p.err, ERR_BAD_INDEX);
            }
        }
        if (window == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.lens[s] = 0;
    }
}

__global__ void __cluster_dims__(PB_CTAS, 1, 1) __launch_bounds__(PB_THREADS) paged_compact_kernel(const BooksParams p) {
    grid_dependency_sync();
    __shared__ int counts[32];
    cg::cluster_group cl = cg::this_cluster();
    int n_live;
    const int before = pb_rank<true>(p, counts, n_live);
    const int lane = threadIdx.x & 31, gw = (int)cl.block_rank() * 32 + (threadIdx.x >> 5);
    const long long run = pb_run(p.n_pages), lo = gw * run, hi = min(p.n_pages, lo + run);
    int r0 = before;
    for (long long i0 = lo; i0 < hi; i0 += 32) {
        const long long i = i0 + lane;
        const bool live = i < hi && p.refcount[i] > 0;
        const unsigned b = __ballot_sync(0xffffffffu, live);
        const int r = r0 + __popc(b & ((1u << lane) - 1u));       // live pages below i
        if (i < hi) {
            if (i == n_live) p.n_moves[1] = r;                    // live pages that stay
            if (i < n_live) {
                if (!live) p.to[i - r] = (int)i;                  // the (i - r)-th free id below n_live
            } else {
                p.map[i] = (int)i;
                if (live) p.from[r] = (int)i;
            }
        }
        r0 += __popc(b);
    }
    if (gw == 0 && lane == 0) {
        p.result[0] = n_live;
        if (n_live >= p.n_pages) p.n_moves[1] = n_live;
    }
    cl.sync();
    const int stay = p.n_moves[1], moves = n_live - stay;
    if (gw == 0 && lane == 0) p.n_moves[0] = moves;
    for (int r = gw * 32 + lane; r < moves; r += PB_WARPS * 32) {
        const int s = p.from[stay + r], d = p.to[r];
        p.map[s] = d;
        p.refcount[d] = p.refcount[s];
        p.refcount[s] = 0;
    }
}

// ------------------------------------------------------------------- copies --
constexpr int PC_MAX_CACHES = 128;           // caches per launch
struct PageCache {
    char *base;
    long long page_stride, slot_stride;      // bytes
};
struct CopyParams {
    const int32_t *from, *to;                // page moves; to < 0: none
    const int32_t *n_moves;                  // {moves, first src} on the device, or NULL: n moves from 0
    int n, n_caches, slots;                  // slots per page (1 where a page is contiguous)
    long long slot_bytes;                    // contiguous bytes per slot
    const int32_t *n_live, *map;             // compact: remap of the table, by the first launch
    int32_t *table;
    long long table_n, n_pages;
    unsigned *err;
    PageCache caches[PC_MAX_CACHES];
};

// Units of up to 32 * NV vectors of one slot run of one page in one cache; a
// warp moves a unit with all its loads in flight.
template <typename V>
__global__ void __launch_bounds__(256) paged_copy_kernel(const __grid_constant__ CopyParams p) {
    grid_dependency_sync();
    constexpr int NV = 8;
    const int lane = threadIdx.x & 31;
    const int moves = p.n_moves ? p.n_moves[0] : p.n, skip = p.n_moves ? p.n_moves[1] : 0;
    const long long vecs = p.slot_bytes / (long long)sizeof(V);
    const long long per_slot = (vecs + 32 * NV - 1) / (32 * NV), per_page = per_slot * p.slots;
    const long long units = (long long)moves * p.n_caches * per_page;
    for (long long w = blockIdx.x * 8ll + (threadIdx.x >> 5); w < units; w += gridDim.x * 8ll) {
        const long long pc = w / per_page, in = w - pc * per_page;
        const int c = (int)(pc % p.n_caches);
        const long long mv = pc / p.n_caches;
        const int d = p.to[mv];
        if (d < 0) continue;
        const long long s = p.from[mv + skip], slot = in / per_slot, part = in - slot * per_slot;
        const PageCache &x = p.caches[c];
        const V *src = reinterpret_cast<const V *>(x.base + s * x.page_stride + slot * x.slot_stride);
        V *dst = reinterpret_cast<V *>(x.base + d * x.page_stride + slot * x.slot_stride);
        V v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const long long at = (part * NV + i) * 32 + lane;
            if (at < vecs) v[i] = src[at];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const long long at = (part * NV + i) * 32 + lane;
            if (at < vecs) dst[at] = v[i];
        }
    }
    if (p.map) {
        const int n_live = p.n_live[0];
        for (long long i = blockIdx.x * 256ll + threadIdx.x; i < p.table_n; i += gridDim.x * 256ll) {
            const int id = p.table[i];
            if (id < n_live) continue;
            if (id >= p.n_pages) raise_error(p.err, ERR_BAD_INDEX);
            else p.table[i] = p.map[id];
        }
    }
}

struct PagedWriteParams {
    const char *src[2];
    char *dst[2];
    long long src_s[2][2];                   // token, head (bytes)
    long long dst_s[2][3];                   // page, slot, head (bytes)
    const int32_t *table, *seqs, *start, *cu;
    int n, S, max_pages, page, Hkv, row_bytes;
    long long N, n_pages;
    unsigned *err;
};
// One warp per new row: its place by bisection of cu, then all heads of K and V.
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedWriteParams p) {
    grid_dependency_sync();
    const int lane = threadIdx.x & 31;
    const int per_head = p.row_bytes / 16, units = 2 * p.Hkv * per_head;
    for (long long r = blockIdx.x * 8ll + (threadIdx.x >> 5); r < p.N; r += gridDim.x * 8ll) {
        int i = (int)r;
        long long off = 0;
        if (p.cu) {
            if (r < __ldg(p.cu) || r >= __ldg(p.cu + p.n)) continue;
            int lo = 0, hi = p.n;
            while (hi - lo > 1) {
                const int m = (lo + hi) / 2;
                if (__ldg(p.cu + m) <= r) lo = m; else hi = m;
            }
            i = lo;
            off = r - __ldg(p.cu + i);
        }
        const int st = __ldg(p.start + i), s = __ldg(p.seqs + i);
        if (st < 0) continue;
        const long long pos = st + off, e = pos / p.page;
        int pg = -1;
        if (s >= 0 && s < p.S && e < p.max_pages) pg = __ldg(p.table + (size_t)s * p.max_pages + e);
        if (pg < 0 || pg >= p.n_pages) {
            if (lane == 0) raise_error(p.err, ERR_BAD_INDEX);
            continue;
        }
        const long long slot = pos - e * p.page;
        for (int u = lane; u < units; u += 32) {
            const int kv = u / (p.Hkv * per_head), w = u - kv * (p.Hkv * per_head), h = w / per_head, c = w % per_head;
            const uint4 x = *reinterpret_cast<const uint4 *>(p.src[kv] + r * p.src_s[kv][0] + h * p.src_s[kv][1] + c * 16);
            *reinterpret_cast<uint4 *>(p.dst[kv] + pg * p.dst_s[kv][0] + slot * p.dst_s[kv][1] + h * p.dst_s[kv][2] +
                                       c * 16) = x;
        }
    }
}

}  // namespace sa
