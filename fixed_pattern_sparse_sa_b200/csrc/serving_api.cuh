// serving_api.cuh -- C ABI entry points of the sink-window attention, the
// paged decode attention and the pages of a cache (declared in include/sa.h).
// Included at the end of sa_api.cu, whose launch, error and alignment helpers
// it uses.
#pragma once

#include "paged_attn.cuh"
#include "paged_books.cuh"
#include "sink_attn.cuh"
#include "sink_bwd_tc.cuh"
#include "sink_fwd_tc.cuh"

// ---------------------------------------------------- sink-window attention --
// set_smem once per device: `done` (one bit a device) belongs to one kernel.
template <typename K>
static int set_smem_once(std::atomic<unsigned long long> &done, K kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return fail(SA_ERR_CUDA, "cudaGetDevice: device %d", dev);
    const unsigned long long bit = 1ull << dev;
    if (done.load(std::memory_order_relaxed) & bit) return SA_OK;
    const int rc = set_smem(kernel, bytes);
    if (rc == SA_OK) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}
static bool strides_ok(const int64_t *s, int n, long long mul) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] % mul) return false;
    return true;
}

static int sink_check(const char *what, const sa_sink_shape *s, const void *q, const void *k, const void *v,
                      const int32_t *cu_q, const int32_t *cu_k, bool bwd) {
    if (!s) return fail(SA_ERR_INVALID_ARG, "%s: shape is null", what);
    if (s->B <= 0 || s->Tq < 0 || s->L < 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Hq % s->Hkv || s->q_pos0 < 0 ||
        s->max_q < 0 || s->max_k < 0)
        return fail(SA_ERR_INVALID_ARG, "%s: bad sizes (Hq a multiple of Hkv)", what);
    if (s->window < 1 || s->sinks < 0) return fail(SA_ERR_INVALID_ARG, "%s: window >= 1, sinks >= 0", what);
    if (!std::isfinite(s->scale) || s->scale <= 0.f) return fail(SA_ERR_INVALID_ARG, "%s: scale must be positive", what);
    if (s->weight_parts < 0 || s->weight_parts > 2)
        return fail(SA_ERR_INVALID_ARG, "%s: weight_parts %d (0, 1 or 2)", what, s->weight_parts);
    if (s->d != 64 && s->d != 128) return fail(SA_ERR_UNSUPPORTED, "%s: head dim %d (64 or 128)", what, s->d);
    if (s->dtype != SA_BF16 && (bwd || s->dtype != SA_FP16))
        return fail(SA_ERR_UNSUPPORTED, "%s: dtype %d", what, s->dtype);
    // positions, row numbers and key tiles are 32-bit
    if (s->Tq >= INT_MAX / 2 || s->L >= INT_MAX / 2 || s->q_pos0 >= INT_MAX / 2)
        return fail(SA_ERR_UNSUPPORTED, "%s: lengths above 2^30", what);
    // so are the work items: at most one per query, KV head and 128 heads of its group, and one more per sequence
    // (a step beyond the last may be formed)
    if (((cu_q ? 1ll : s->B) * s->Tq + s->B) * s->Hkv * ((s->Hq / s->Hkv + 127) / 128) >= INT_MAX / 2 ||
        s->Hq >= (1 << 20) || (bwd && (cu_q ? 1ll : s->B) * s->L * s->Hkv >= INT_MAX / 2))
        return fail(SA_ERR_UNSUPPORTED, "%s: too many rows", what);
    if ((cu_q == nullptr) != (cu_k == nullptr)) return fail(SA_ERR_INVALID_ARG, "%s: cu_q and cu_k go together", what);
    const bool no_q = s->Tq == 0, no_k = s->L == 0;       // an empty tensor may have a null pointer
    if ((!no_q && (!q || !aligned16(q))) || (!no_k && (!k || !v || !aligned16(k) || !aligned16(v))) ||
        (cu_q && (!aligned4(cu_q) || !aligned4(cu_k))))
        return fail(SA_ERR_INVALID_ARG, "%s: null or misaligned pointer", what);
    if (!strides_ok(s->q_stride, 3, 8) || !strides_ok(s->k_stride, 3, 8) || !strides_ok(s->v_stride, 3, 8))
        return fail(SA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements, not negative", what);
    // rows that share memory (a broadcast input) are not taken: the copy engine's maps want a step
    const int nb = cu_q ? 1 : s->B;
    for (int i = 0; i < 3; ++i) {
        const bool many_q = i == 0 ? nb > 1 : i == 1 ? s->Tq > 1 : s->Hq > 1;
        const bool many_k = i == 0 ? nb > 1 : i == 1 ? s->L > 1 : s->Hkv > 1;
        if ((many_q && s->q_stride[i] == 0) || (many_k && (s->k_stride[i] == 0 || s->v_stride[i] == 0)) ||
            (bwd && many_q && s->dout_stride[i] == 0))
            return fail(SA_ERR_INVALID_ARG, "%s: a stride of 0 (a broadcast input) is not supported", what);
    }
    return SA_OK;
}

static SinkParams sink_params(const sa_sink_shape *s, const void *q, const void *k, const void *v,
                              const int32_t *cu_q, const int32_t *cu_k) {
    SinkParams p{};
    p.q = q; p.k = k; p.v = v;
    for (int i = 0; i < 3; ++i) {
        p.q_s[i] = s->q_stride[i]; p.k_s[i] = s->k_stride[i]; p.v_s[i] = s->v_stride[i];
        p.do_s[i] = s->dout_stride[i]; p.lse_s[i] = s->lse_stride[i];
    }
    p.cu_q = cu_q; p.cu_k = cu_k;
    p.B = s->B; p.Hq = s->Hq; p.Hkv = s->Hkv; p.G = s->Hq / s->Hkv;
    // a window past the last position and sinks past the last key say no more than these do
    const int64_t last = cu_q ? s->L : s->q_pos0 + s->Tq;
    p.window = (int)std::min<int64_t>(s->window, std::max<int64_t>(last, 1));
    p.sinks = (int)std::min<int64_t>(s->sinks, s->L);
    p.Tq = s->Tq; p.L = s->L; p.q_pos0 = s->q_pos0; p.max_q = s->max_q; p.max_k = s->max_k;
    p.scale = s->scale; p.scale_log2 = s->scale * kLog2e;
    return p;
}

// 4-D map over [batch, token, head, d] rows with the given strides (elements);
// box = 64 columns (128 bytes) x box_heads x box_tokens, 128-byte swizzle.  A
// dimension of size 1 is never stepped over, so its stride only has to be valid.
template <typename T>
static int rows_tensor_map(CUtensorMap *m, const void *base, int d, long long heads, long long tokens, long long batch,
                           const long long *st, int box_heads, int box_tokens) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return fail(SA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
    cuuint64_t strides[3] = {(cuuint64_t)(heads > 1 ? st[2] : d) * 2, (cuuint64_t)(tokens > 1 ? st[1] : d) * 2,
                             (cuuint64_t)(batch > 1 ? st[0] : d) * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1u};
    cuuint32_t es[4] = {1u, 1u, 1u, 1u};
    const CUresult r = enc(m, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           4, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(SA_ERR_INVALID_ARG, "a tensor of %lld x %lld x %lld rows with strides %lld, %lld, %lld cannot be "
                    "described to the copy engine (%d)", batch, tokens, heads, st[0], st[1], st[2], (int)r);
    return SA_OK;
}

// Weights in two parts (SPLIT) or one.  Measured over 1500 rows, in output
// roundings: one part 1.07 (two visible keys) to 1.40 (1024) in out, 1.40 to
// 1.43 in the gradients, single rows up to 3.5; two parts 1.00 throughout.
// The number of keys seen does not decide it, the number of rows that the
// caller sees does: 36 rows came out at 1.9.  Two parts cost, one -> two in us
// (window 512 unless named):
//   forward   2048 rows (window 32) 8.4 -> 8.5, 8192 rows 14.7 -> 24.2,
//             65536 rows 31 -> 51, 64K x 16 heads (window 2048) 1083 -> 2182
//   backward  2048 rows (window 32) 25 -> 31, 8192 rows 137 -> 229,
//             16K x 64 heads 1862 -> 2390, 64K x 16 heads (2048) 5958 -> 7535
// So the caller chooses; left open, calls of up to 8192 rows take two (there
// 0.01 ms more in a forward, 0.09 ms in a backward).
static bool sink_split(const sa_sink_shape *s, const SinkParams &p) {
    if (s->weight_parts) return s->weight_parts == 2;
    return (p.cu_q ? 1 : p.B) * p.Tq * p.Hq <= 8192;
}

template <typename T>
static int key_maps(KeyMaps &m, const void *base, int d, int heads, long long L, long long batch, const long long *st) {
    L = std::max(L, 1ll);
    int rc = rows_tensor_map<T>(&m.all, base, d, heads, L, batch, st, 1, SF_KT);
    if (!rc) rc = rows_tensor_map<T>(&m.head, base, d, heads, L, batch, st, 1, SF_HEAD);
    if (!rc) rc = rows_tensor_map<T>(&m.rest, base, d, heads, L, batch, st, 1, SF_KT - SF_HEAD);
    return rc;
}

static SinkTiles sink_tiles(const SinkParams &p, int row_tiles) {
    SinkTiles t{};
    t.HB = std::min(p.G, 128);
    t.HC = (p.G + 127) / 128;
    t.TPT = 128 / t.HB;
    const long long TI = (long long)row_tiles * t.TPT;
    t.per_seq = (int)((p.Tq + TI - 1) / TI);
    t.items = (int)((p.cu_q ? p.Tq / TI + p.B : (long long)p.B * t.per_seq) * p.Hkv * t.HC);
    return t;
}

template <typename T, int D, bool SPLIT>
static int sink_fwd_launch(const SinkParams &p, cudaStream_t st) {
    const SinkTiles t = sink_tiles(p, 2);
    const long long nb = p.cu_q ? 1 : p.B;
    CUtensorMap qm;
    KeyMaps km, vm;
    // without keys nothing is loaded; the maps only have to be valid
    const void *k = p.L ? p.k : p.q, *v = p.L ? p.v : p.q;
    int rc = rows_tensor_map<T>(&qm, p.q, D, p.Hq, p.Tq, nb, p.q_s, t.HB, t.TPT);
    if (!rc) rc = key_maps<T>(km, k, D, p.Hkv, p.L, nb, p.k_s);
    if (!rc) rc = key_maps<T>(vm, v, D, p.Hkv, p.L, nb, p.v_s);
    static std::atomic<unsigned long long> done{0};
    if (!rc) rc = set_smem_once(done, sink_fwd_tc_kernel<T, D, SPLIT>, SfSmem<D>::ALLOC);
    if (rc) return rc;
    const unsigned grid = (unsigned)std::min<long long>(t.items, sm_count());
    launch_k("sink_fwd_tc_kernel", sink_fwd_tc_kernel<T, D, SPLIT>, grid, SF_THREADS, SfSmem<D>::ALLOC, st, qm, km, vm, p, t);
    SA_CHECK_LAUNCH("sink_fwd_tc_kernel");
    return SA_OK;
}

extern "C" int sa_sink_attn_fwd(const sa_sink_shape *shape, const void *q, const void *k, const void *v,
                                const int32_t *cu_q, const int32_t *cu_k, void *out, float *lse, void *stream) {
    SA_TRACE("sa_sink_attn_fwd");
    int rc = sink_check("sink_attn_fwd", shape, q, k, v, cu_q, cu_k, false);
    if (rc) return rc;
    if (shape->Tq == 0) return SA_OK;
    if (!out || !lse || !aligned16(out) || !aligned4(lse))
        return fail(SA_ERR_INVALID_ARG, "sink_attn_fwd: null or misaligned output");
    SinkParams p = sink_params(shape, q, k, v, cu_q, cu_k);
    rc = device_error_word(&p.err);
    if (rc) return rc;
    p.out = out; p.lse = lse;
    cudaStream_t st = as_stream(stream);
    using B = __nv_bfloat16;
    using H = __half;
    const bool bf = shape->dtype == SA_BF16;
    if (sink_split(shape, p))
        return shape->d == 64 ? (bf ? sink_fwd_launch<B, 64, true>(p, st) : sink_fwd_launch<H, 64, true>(p, st))
                              : (bf ? sink_fwd_launch<B, 128, true>(p, st) : sink_fwd_launch<H, 128, true>(p, st));
    return shape->d == 64 ? (bf ? sink_fwd_launch<B, 64, false>(p, st) : sink_fwd_launch<H, 64, false>(p, st))
                          : (bf ? sink_fwd_launch<B, 128, false>(p, st) : sink_fwd_launch<H, 128, false>(p, st));
}

// Key-major items of the backward and how the sinks' are cut: pieces of a
// quarter of a band item, so that they fill the last wave, but of 4 units at
// least (one piece of 32 units made a call on 512 tokens 33 us long), 64
// pieces at most, and no more than four waves of them in all.
static SinkKvTiles sink_kv_tiles(const SinkParams &p) {
    SinkKvTiles t{};
    t.HB = std::min(p.G, 64);
    t.HC = (p.G + 63) / 64;
    t.TPT = 64 / t.HB;
    const long long nq = p.cu_q ? (p.max_q ? std::min(p.max_q, p.Tq) : p.Tq) : p.Tq;
    const long long nk = p.cu_q ? (p.max_k ? std::min(p.max_k, p.L) : p.L) : p.L;
    const bool apart = p.cu_q ? nk > p.window : p.q_pos0 + p.Tq > p.window;
    const long long se = apart ? std::min<long long>(p.sinks, nk) : 0;
    t.per_seq = (int)((p.L - se + 127) / 128);                     // dense: every sequence's
    t.band = (int)(p.cu_q ? p.L / 128 + p.B : (long long)p.B * t.per_seq);
    t.n_kt = (int)((se + 127) / 128);
    t.n_split = 1;
    t.tps = (int)std::max<long long>(nq, 1);
    if (t.n_kt && nq) {
        const long long want = std::max({(4ll * t.TPT + t.HC - 1) / t.HC, (p.window + 131ll) / 4, (nq + 63) / 64});
        const long long most = std::max<long long>(1, 4ll * sm_count() / ((long long)p.B * p.Hkv * t.n_kt));
        t.n_split = (int)std::min(most, (nq + want - 1) / want);
        t.tps = (int)((nq + t.n_split - 1) / t.n_split);
    }
    t.items = (int)std::min<long long>((t.band + (long long)p.B * t.n_kt * t.n_split) * p.Hkv, INT_MAX);
    return t;
}
struct SinkBwdLayout { size_t counter, part, total; };
static SinkBwdLayout sink_bwd_layout(const SinkParams &p, int d) {
    const SinkKvTiles t = sink_kv_tiles(p);
    SinkBwdLayout l{};
    l.counter = round_up((size_t)(p.cu_q ? 1 : p.B) * p.Tq * p.Hq * 8, 256);
    l.part = l.counter + 256;
    l.total = l.part + (t.n_split > 1 ? (size_t)p.B * p.Hkv * t.n_split * p.sinks * 2 * d * 4 : 0);
    return l;
}

extern "C" size_t sa_sink_attn_bwd_workspace_size(const sa_sink_shape *s, int packed) {
    if (!s || s->B <= 0 || s->Tq < 0 || s->L < 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Hq % s->Hkv || s->window < 1 ||
        s->sinks < 0)
        return 0;
    const int32_t *cu = packed ? reinterpret_cast<const int32_t *>(s) : nullptr;       // only whether it is there counts
    return sink_bwd_layout(sink_params(s, nullptr, nullptr, nullptr, cu, cu), s->d).total;
}

template <int D, bool SPLIT>
static int sink_bwd_launch(const SinkParams &p, void *ws, cudaStream_t st) {
    using T = __nv_bfloat16;
    const long long nb = p.cu_q ? 1 : p.B;
    const SinkBwdLayout lay = sink_bwd_layout(p, D);
    SinkKvTiles kt = sink_kv_tiles(p);
    kt.counter = reinterpret_cast<int *>(static_cast<char *>(ws) + lay.counter);
    kt.part = reinterpret_cast<float *>(static_cast<char *>(ws) + lay.part);
    // an empty side is never loaded: its maps only have to be valid
    const void *any = p.Tq ? p.q : p.k, *q = any, *g = p.Tq ? p.dout : any, *k = p.L ? p.k : any, *v = p.L ? p.v : any;
    const long long Tq = std::max(p.Tq, 1ll), L = std::max(p.L, 1ll);
    CUtensorMap qm, gm;
    KeyMaps km, vm;
    int rc = key_maps<T>(km, k, D, p.Hkv, L, nb, p.k_s);
    if (!rc) rc = key_maps<T>(vm, v, D, p.Hkv, L, nb, p.v_s);
    if (rc) return rc;
    // first: it also writes the rows' lse and D for the key-major pass, and resets its counter
    if (p.Tq > 0) {
        const SinkTiles t = sink_tiles(p, 1);
        rc = rows_tensor_map<T>(&qm, q, D, p.Hq, Tq, nb, p.q_s, t.HB, t.TPT);
        if (!rc) rc = rows_tensor_map<T>(&gm, g, D, p.Hq, Tq, nb, p.do_s, t.HB, t.TPT);
        static std::atomic<unsigned long long> done{0};
        if (!rc) rc = set_smem_once(done, sink_dq_tc_kernel<D, SPLIT>, SqSmem<D>::ALLOC);
        if (rc) return rc;
        const unsigned grid = (unsigned)std::min(t.items, sm_count());
        launch_k("sink_dq_tc_kernel", sink_dq_tc_kernel<D, SPLIT>, grid, SB_THREADS, SqSmem<D>::ALLOC, st, qm, gm, km, vm, p, t,
                 kt.counter);
        SA_CHECK_LAUNCH("sink_dq_tc_kernel");
    } else {
        const cudaError_t e = cudaMemsetAsync(kt.counter, 0, sizeof(int), st);
        if (e != cudaSuccess) return fail(SA_ERR_CUDA, "sink_attn_bwd memset: %s", cudaGetErrorString(e));
    }
    if (p.L > 0) {
        rc = rows_tensor_map<T>(&qm, q, D, p.Hq, Tq, nb, p.q_s, kt.HB, kt.TPT);
        if (!rc) rc = rows_tensor_map<T>(&gm, g, D, p.Hq, Tq, nb, p.do_s, kt.HB, kt.TPT);
        static std::atomic<unsigned long long> done{0};
        if (!rc) rc = set_smem_once(done, sink_dkv_tc_kernel<D, SPLIT>, SkSmem<D>::ALLOC);
        if (rc) return rc;
        const unsigned grid = (unsigned)std::min(std::max(kt.items, 1), sm_count());
        launch_k("sink_dkv_tc_kernel", sink_dkv_tc_kernel<D, SPLIT>, grid, SB_THREADS, SkSmem<D>::ALLOC, st, qm, gm, km.all, vm.all, p,
                 kt);
        SA_CHECK_LAUNCH("sink_dkv_tc_kernel");
        if (kt.n_split > 1) {
            const long long jr = (long long)p.B * p.Hkv * p.sinks;
            launch_k("sink_dkv_join_kernel", sink_dkv_join_kernel<D>, (unsigned)std::min<long long>(jr, 1 << 20), 256, 0, st,
                     p, kt);
            SA_CHECK_LAUNCH("sink_dkv_join_kernel");
        }
    }
    return SA_OK;
}

extern "C" int sa_sink_attn_bwd(const sa_sink_shape *shape, const void *q, const void *k, const void *v,
                                const void *out, const float *lse, const void *dout, const int32_t *cu_q,
                                const int32_t *cu_k, void *dq, void *dk, void *dv, void *workspace,
                                size_t workspace_bytes, void *stream) {
    SA_TRACE("sa_sink_attn_bwd");
    int rc = sink_check("sink_attn_bwd", shape, q, k, v, cu_q, cu_k, true);
    if (rc) return rc;
    if (!strides_ok(shape->dout_stride, 3, 8) || !strides_ok(shape->lse_stride, 3, 1))
        return fail(SA_ERR_INVALID_ARG, "sink_attn_bwd: strides must be multiples of 8 elements, not negative");
    (void)out;
    if (shape->Tq > 0 && (!lse || !dout || !dq || !aligned4(lse) || !aligned16(dout) || !aligned16(dq)))
        return fail(SA_ERR_INVALID_ARG, "sink_attn_bwd: null or misaligned pointer");
    if (shape->L > 0 && (!dk || !dv || !aligned16(dk) || !aligned16(dv)))
        return fail(SA_ERR_INVALID_ARG, "sink_attn_bwd: null or misaligned pointer");
    const size_t need = sa_sink_attn_bwd_workspace_size(shape, cu_q != nullptr);
    if (workspace_bytes < need || (need && !workspace))
        return fail(SA_ERR_WORKSPACE, "sink_attn_bwd: workspace %zu < %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SA_ERR_INVALID_ARG, "sink_attn_bwd: workspace alignment");
    SinkParams p = sink_params(shape, q, k, v, cu_q, cu_k);
    rc = device_error_word(&p.err);
    if (rc) return rc;
    if (sink_kv_tiles(p).items >= INT_MAX / 2)
        return fail(SA_ERR_UNSUPPORTED, "sink_attn_bwd: too many sequences for so many sinks (give max_k)");
    p.lse_in = lse; p.dout = dout;
    p.dq = dq; p.dk = dk; p.dv = dv; p.stat = static_cast<float2 *>(workspace);
    if (shape->Tq == 0 && shape->L == 0) return SA_OK;
    cudaStream_t st = as_stream(stream);
    if (sink_split(shape, p))
        return shape->d == 64 ? sink_bwd_launch<64, true>(p, workspace, st) : sink_bwd_launch<128, true>(p, workspace, st);
    return shape->d == 64 ? sink_bwd_launch<64, false>(p, workspace, st) : sink_bwd_launch<128, false>(p, workspace, st);
}

// ------------------------------------------------- paged decode attention --
template <int D>
static int pd_grid() { return sm_count() * (D == 64 ? 2 : 1); }   // CTAs that fit with their rings at once

static size_t pd_part_floats(int d) {
    return (size_t)(d == 64 ? pd_grid<64>() : pd_grid<128>()) * 2 * PD_NW * 16 * (d + 2);
}

extern "C" size_t sa_paged_attn_decode_workspace_size(int B, int Hq, int Hkv, int d) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 128)) return 0;
    return round_up((size_t)(B + 1) * 8, 256) + pd_part_floats(d) * 4;
}

template <typename T, int D>
static int pd_launch(const PagedParams &p, cudaStream_t st) {
    const int smem = PdSmem<D>::TOTAL, gx = pd_grid<D>();
    static std::atomic<unsigned long long> done{0};
    int rc = set_smem_once(done, paged_decode_kernel<T, D>, smem);
    if (rc) return rc;
    launch_k("paged_decode_kernel", paged_decode_kernel<T, D>, gx, PD_THREADS, smem, st, p);
    SA_CHECK_LAUNCH("paged_decode_kernel");
    const dim3 gj((unsigned)((long long)p.B * p.Hkv * p.HT), (unsigned)((std::min(p.G, 16) + 3) / 4));
    launch_k("paged_join_kernel", paged_join_kernel<T, D>, gj, 256, 0, st, p, gx);
    SA_CHECK_LAUNCH("paged_join_kernel");
    return SA_OK;
}

extern "C" int sa_paged_attn_decode(const sa_paged_shape *s, const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_table, const int32_t *seq_lens, void *out, float *lse,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    SA_TRACE("sa_paged_attn_decode");
    if (!s) return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: shape is null");
    if (s->B < 0 || s->Hq <= 0 || s->Hkv <= 0 || s->Hq % s->Hkv || s->page <= 0 || s->max_pages < 0 || s->n_pages < 0 ||
        s->window < 0 || s->sinks < 0)
        return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: bad sizes (Hq a multiple of Hkv)");
    if (!std::isfinite(s->scale) || s->scale <= 0.f)
        return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: scale must be positive");
    if (s->d != 64 && s->d != 128) return fail(SA_ERR_UNSUPPORTED, "paged_attn_decode: head dim %d (64 or 128)", s->d);
    if (s->dtype != SA_BF16 && s->dtype != SA_FP16)
        return fail(SA_ERR_UNSUPPORTED, "paged_attn_decode: dtype %d", s->dtype);
    if ((long long)s->max_pages * s->page >= INT_MAX / 2)
        return fail(SA_ERR_UNSUPPORTED, "paged_attn_decode: %d pages of %d tokens (below 2^30 tokens)", s->max_pages,
                    s->page);
    if ((long long)s->B * s->Hq >= INT_MAX / 2 || s->n_pages > INT_MAX)
        return fail(SA_ERR_UNSUPPORTED, "paged_attn_decode: too many rows or pages");
    if (s->B == 0) return SA_OK;
    const bool no_kv = s->n_pages == 0 || s->max_pages == 0;      // an empty pool may have null pointers
    if (!q || !seq_lens || !out || !lse || !aligned16(q) || !aligned4(seq_lens) || !aligned16(out) || !aligned4(lse) ||
        (!no_kv && (!k_cache || !v_cache || !block_table)) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(block_table))
        return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: null or misaligned pointer");
    if (!strides_ok(s->q_stride, 2, 8) || !strides_ok(s->k_stride, 3, 8) || !strides_ok(s->v_stride, 3, 8))
        return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: strides must be multiples of 8 elements, not negative");
    const size_t need = sa_paged_attn_decode_workspace_size(s->B, s->Hq, s->Hkv, s->d);
    if (!workspace || workspace_bytes < need)
        return fail(SA_ERR_WORKSPACE, "paged_attn_decode: workspace %zu < %zu", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(SA_ERR_INVALID_ARG, "paged_attn_decode: workspace alignment");
    PagedParams p{};
    int rc = device_error_word(&p.err);
    if (rc) return rc;
    p.q = q; p.k = k_cache; p.v = v_cache;
    for (int i = 0; i < 2; ++i) p.q_s[i] = s->q_stride[i];
    for (int i = 0; i < 3; ++i) { p.k_s[i] = s->k_stride[i]; p.v_s[i] = s->v_stride[i]; }
    p.table = block_table; p.lens = seq_lens;
    p.B = s->B; p.Hq = s->Hq; p.Hkv = s->Hkv; p.G = s->Hq / s->Hkv; p.HT = (p.G + 15) / 16;
    p.page = s->page; p.max_pages = no_kv ? 0 : s->max_pages; p.window = s->window; p.sinks = s->sinks;
    p.n_pages = s->n_pages; p.scale_log2 = s->scale * kLog2e;
    p.out = out; p.lse = lse;
    p.c0 = static_cast<long long *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up((size_t)(s->B + 1) * 8, 256));
    cudaStream_t st = as_stream(stream);
    if (s->dtype == SA_BF16)
        return s->d == 64 ? pd_launch<__nv_bfloat16, 64>(p, st) : pd_launch<__nv_bfloat16, 128>(p, st);
    return s->d == 64 ? pd_launch<__half, 64>(p, st) : pd_launch<__half, 128>(p, st);
}

// --------------------------------------------------------- pages of a cache --
struct BooksLayout {
    size_t owner, mark, ends, seq, from, to, moves, map, total;
};
static BooksLayout books_layout(int S, int n, int64_t n_pages) {
    BooksLayout l{};
    size_t at = 0;
    auto take = [&](size_t ints) { const size_t o = at; at += round_up(ints * 4, 256); return o; };
    l.owner = take(S); l.mark = take(S);
    l.ends = take(n); l.seq = take(n);
    const size_t moves = std::max<size_t>(n, n_pages);
    l.from = take(moves); l.to = take(moves);
    l.moves = take(2); l.map = take(n_pages);
    l.total = at;
    return l;
}

extern "C" size_t sa_paged_books_workspace_size(int S, int n, int64_t n_pages) {
    if (S < 0 || n < 0 || n_pages < 0) return 0;
    return books_layout(S, n, n_pages).total;
}

static int books_check(const char *what, const void *table, const void *lens, const void *refcount, int S,
                       int max_pages, int64_t n_pages, int page, int n) {
    if (S < 0 || max_pages < 0 || n_pages < 0 || page <= 0 || n < 0)
        return fail(SA_ERR_INVALID_ARG, "%s: bad sizes", what);
    if (n_pages >= INT_MAX || max_pages >= (1 << 26) || (long long)max_pages * page >= INT_MAX / 2)
        return fail(SA_ERR_UNSUPPORTED, "%s: %d pages of %d tokens per sequence, %lld in all (below 2^30 tokens)", what,
                    max_pages, page, (long long)n_pages);
    if ((S > 0 && (!lens || (max_pages > 0 && !table))) || (n_pages > 0 && !refcount) || !aligned4(table) ||
        !aligned4(lens) || !aligned4(refcount))
        return fail(SA_ERR_INVALID_ARG, "%s: null or misaligned pointer", what);
    return SA_OK;
}

static int books_params(const char *what, BooksParams &p, int32_t *table, int32_t *lens, int32_t *refcount, int S,
                        int max_pages, int64_t n_pages, int page, const int32_t *a, const int32_t *c, int n,
                        int32_t *result, void *ws, size_t ws_bytes) {
    const BooksLayout l = books_layout(S, n, n_pages);
    if (ws_bytes < l.total || (l.total && !ws))
        return fail(SA_ERR_WORKSPACE, "%s: workspace %zu < %zu", what, ws_bytes, l.total);
    if (!aligned16(ws)) return fail(SA_ERR_INVALID_ARG, "%s: workspace alignment", what);
    char *w = static_cast<char *>(ws);
    auto at = [&](size_t o) { return reinterpret_cast<int32_t *>(w + o); };
    p.table = table; p.lens = lens; p.refcount = refcount;
    p.S = S; p.max_pages = max_pages; p.page = page; p.n_pages = n_pages;
    p.a = a; p.c = c; p.n = n; p.result = result;
    p.owner = at(l.owner); p.srcmark = at(l.mark); p.ends = at(l.ends); p.seq = at(l.seq);
    p.from = at(l.from); p.to = at(l.to); p.n_moves = at(l.moves); p.map = at(l.map);
    return device_error_word(&p.err);
}

// Checks the caches (of an empty pool a base may be null); vec: bytes of the widest vector that all of them allow.
static int caches_check(const char *what, const sa_page_cache *caches, int n_caches, int64_t slot_bytes, int64_t n_pages,
                        int &vec) {
    if (n_caches < 0 || slot_bytes < 0 || (n_caches > 0 && !caches))
        return fail(SA_ERR_INVALID_ARG, "%s: bad caches", what);
    vec = slot_bytes % 16 ? 4 : 16;
    if (n_caches > 0 && slot_bytes % 4) return fail(SA_ERR_UNSUPPORTED, "%s: slots of %lld bytes (a multiple of 4)", what,
                                                    (long long)slot_bytes);
    for (int i = 0; i < n_caches; ++i) {
        const sa_page_cache &c = caches[i];
        if ((!c.base && n_pages > 0) || c.page_stride < 0 || c.slot_stride < 0)
            return fail(SA_ERR_INVALID_ARG, "%s: cache %d", what, i);
        const unsigned long long bits = reinterpret_cast<uintptr_t>(c.base) | (unsigned long long)c.page_stride |
                                        (unsigned long long)c.slot_stride;
        if (bits % 4) return fail(SA_ERR_INVALID_ARG, "%s: cache %d is not aligned to 4 bytes", what, i);
        if (bits % 16) vec = 4;
    }
    return SA_OK;
}

static int copy_pages(const BooksParams &b, const sa_page_cache *caches, int n_caches, int64_t slot_bytes, int vec,
                      bool compact, cudaStream_t st) {
    bool remap = compact;
    for (int c0 = 0; c0 < n_caches || remap; c0 += PC_MAX_CACHES) {
        CopyParams p{};
        p.from = b.from; p.to = b.to; p.n = b.n; p.n_moves = compact ? b.n_moves : nullptr;
        p.n_caches = std::max(0, std::min(n_caches - c0, PC_MAX_CACHES));
        bool whole = true;                            // pages are contiguous in every cache
        for (int i = 0; i < p.n_caches; ++i) {
            const sa_page_cache &c = caches[c0 + i];
            p.caches[i] = PageCache{static_cast<char *>(c.base), c.page_stride, c.slot_stride};
            whole = whole && c.slot_stride == slot_bytes;
        }
        p.slots = whole ? 1 : b.page;
        p.slot_bytes = whole ? slot_bytes * b.page : slot_bytes;
        if (p.slot_bytes == 0) p.n_caches = 0;
        if (remap) {
            p.map = b.map; p.n_live = b.result; p.table = b.table; p.table_n = (long long)b.S * b.max_pages;
            p.n_pages = b.n_pages; p.err = b.err;
        }
        remap = false;
        const unsigned grid = (unsigned)sm_count() * 4;
        if (vec == 16) launch_k("paged_copy_kernel<16>", paged_copy_kernel<uint4>, grid, 256, 0, st, p);
        else launch_k("paged_copy_kernel<4>", paged_copy_kernel<uint32_t>, grid, 256, 0, st, p);
        SA_CHECK_LAUNCH("paged_copy_kernel");
    }
    return SA_OK;
}

extern "C" int sa_paged_extend(int32_t *block_table, int32_t *seq_lens, int32_t *refcount, int S, int max_pages,
                               int64_t n_pages, int page, const int32_t *seqs, const int32_t *n_new, int n,
                               int32_t *start, void *workspace, size_t workspace_bytes, void *stream) {
    SA_TRACE("sa_paged_extend");
    int rc = books_check("paged_extend", block_table, seq_lens, refcount, S, max_pages, n_pages, page, n);
    if (rc) return rc;
    if (n == 0) return SA_OK;
    if (!seqs || !n_new || !start || !aligned4(seqs) || !aligned4(n_new) || !aligned4(start))
        return fail(SA_ERR_INVALID_ARG, "paged_extend: null or misaligned pointer");
    BooksParams p{};
    rc = books_params("paged_extend", p, block_table, seq_lens, refcount, S, max_pages, n_pages, page, seqs, n_new, n,
                      start, workspace, workspace_bytes);
    if (rc) return rc;
    launch_k("paged_extend_kernel", paged_extend_kernel, PB_CTAS, PB_THREADS, 0, as_stream(stream), p);
    SA_CHECK_LAUNCH("paged_extend_kernel");
    return SA_OK;
}

extern "C" int sa_paged_write(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                              const int32_t *block_table, const int32_t *seqs, const int32_t *start,
                              const int32_t *cu_new, int n, int64_t N, int S, int max_pages, int64_t n_pages, int page,
                              int Hkv, int d, int elem_bytes, const int64_t *strides, void *stream) {
    SA_TRACE("sa_paged_write");
    if (n < 0 || N < 0 || S < 0 || max_pages < 0 || n_pages < 0 || page <= 0 || Hkv <= 0 || d <= 0 || elem_bytes <= 0 ||
        !strides || (!cu_new && N != n))
        return fail(SA_ERR_INVALID_ARG, "paged_write: bad sizes (without cu_new one row per entry)");
    if ((long long)d * elem_bytes % 16 || (long long)Hkv * d * elem_bytes >= (1 << 28))
        return fail(SA_ERR_UNSUPPORTED, "paged_write: rows of %lld bytes (a multiple of 16)", (long long)d * elem_bytes);
    if (n == 0 || N == 0) return SA_OK;
    if (!k_new || !v_new || !seqs || !start || !aligned16(k_new) || !aligned16(v_new) || !aligned4(seqs) ||
        !aligned4(start) || !aligned4(cu_new) || !aligned4(block_table) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (S > 0 && max_pages > 0 && !block_table) || (n_pages > 0 && (!k_cache || !v_cache)))
        return fail(SA_ERR_INVALID_ARG, "paged_write: null or misaligned pointer");
    PagedWriteParams p{};
    const void *src[2] = {k_new, v_new};
    void *dst[2] = {k_cache, v_cache};
    const int64_t *ss[2] = {strides, strides + 2}, *ds[2] = {strides + 4, strides + 7};
    for (int i = 0; i < 2; ++i) {
        p.src[i] = static_cast<const char *>(src[i]);
        p.dst[i] = static_cast<char *>(dst[i]);
        for (int j = 0; j < 2; ++j) p.src_s[i][j] = ss[i][j] * elem_bytes;
        for (int j = 0; j < 3; ++j) p.dst_s[i][j] = ds[i][j] * elem_bytes;
        for (int j = 0; j < 3; ++j)
            if (p.dst_s[i][j] < 0 || p.dst_s[i][j] % 16 || (j < 2 && (p.src_s[i][j] < 0 || p.src_s[i][j] % 16)))
                return fail(SA_ERR_INVALID_ARG, "paged_write: strides must be multiples of 16 bytes, not negative");
    }
    int rc = device_error_word(&p.err);
    if (rc) return rc;
    p.table = block_table; p.seqs = seqs; p.start = start; p.cu = cu_new;
    p.n = n; p.S = S; p.max_pages = max_pages; p.page = page; p.Hkv = Hkv; p.row_bytes = d * elem_bytes;
    p.N = N; p.n_pages = n_pages;
    const unsigned grid = (unsigned)std::min<long long>((N + 7) / 8, sm_count() * 8);
    launch_k("paged_write_kernel", paged_write_kernel, grid, 256, 0, as_stream(stream), p);
    SA_CHECK_LAUNCH("paged_write_kernel");
    return SA_OK;
}

extern "C" int sa_paged_fork(int32_t *block_table, int32_t *seq_lens, int32_t *refcount, int S, int max_pages,
                             int64_t n_pages, int page, const int32_t *src, const int32_t *dst, int n,
                             const sa_page_cache *caches, int n_caches, int64_t slot_bytes, int32_t *done,
                             void *workspace, size_t workspace_bytes, void *stream) {
    SA_TRACE("sa_paged_fork");
    int rc = books_check("paged_fork", block_table, seq_lens, refcount, S, max_pages, n_pages, page, n), vec = 16;
    if (rc == SA_OK) rc = caches_check("paged_fork", caches, n_caches, slot_bytes, n_pages, vec);
    if (rc) return rc;
    if (n == 0) return SA_OK;
    if (!src || !dst || !done || !aligned4(src) || !aligned4(dst) || !aligned4(done))
        return fail(SA_ERR_INVALID_ARG, "paged_fork: null or misaligned pointer");
    BooksParams p{};
    rc = books_params("paged_fork", p, block_table, seq_lens, refcount, S, max_pages, n_pages, page, src, dst, n, done,
                      workspace, workspace_bytes);
    if (rc) return rc;
    cudaStream_t st = as_stream(stream);
    launch_k("paged_fork_kernel", paged_fork_kernel, PB_CTAS, PB_THREADS, 0, st, p);
    SA_CHECK_LAUNCH("paged_fork_kernel");
    return copy_pages(p, caches, n_caches, slot_bytes, vec, false, st);
}

extern "C" int sa_paged_free(int32_t *block_table, int32_t *seq_lens, int32_t *refcount, int S, int max_pages,
                             int64_t n_pages, int page, const int32_t *seqs, int n, int window, int sinks,
                             void *stream) {
    SA_TRACE("sa_paged_free");
    if (window < 0 || sinks < 0) return fail(SA_ERR_INVALID_ARG, "paged_free: window and sinks >= 0");
    int rc = books_check("paged_free", block_table, seq_lens, refcount, S, max_pages, n_pages, page, n);
    if (rc) return rc;
    if (n == 0) return SA_OK;
    if (!seqs || !aligned4(seqs)) return fail(SA_ERR_INVALID_ARG, "paged_free: null or misaligned pointer");
    BooksParams p{};
    rc = device_error_word(&p.err);
    if (rc) return rc;
    p.table = block_table; p.lens = seq_lens; p.refcount = refcount;
    p.S = S; p.max_pages = max_pages; p.page = page; p.n_pages = n_pages; p.a = seqs; p.n = n;
    const dim3 grid((unsigned)std::min(n, 1 << 20), (unsigned)std::min(std::max((max_pages + 255) / 256, 1), 64));
    launch_k("paged_free_kernel", paged_free_kernel, grid, 256, 0, as_stream(stream), p, window, sinks);
    SA_CHECK_LAUNCH("paged_free_kernel");
    return SA_OK;
}

extern "C" int sa_paged_compact(int32_t *block_table, int32_t *refcount, int S, int max_pages, int64_t n_pages,
                                int page, const sa_page_cache *caches, int n_caches, int64_t slot_bytes,
                                int32_t *n_live, void *workspace, size_t workspace_bytes, void *stream) {
    SA_TRACE("sa_paged_compact");
    int vec = 16;
    int rc = books_check("paged_compact", block_table, block_table ? (void *)block_table : (void *)n_live, refcount, S,
                         max_pages, n_pages, page, 0);
    if (rc == SA_OK) rc = caches_check("paged_compact", caches, n_caches, slot_bytes, n_pages, vec);
    if (rc) return rc;
    if (!n_live || !aligned4(n_live)) return fail(SA_ERR_INVALID_ARG, "paged_compact: null or misaligned pointer");
    BooksParams p{};
    rc = books_params("paged_compact", p, block_table, nullptr, refcount, S, max_pages, n_pages, page, nullptr, nullptr,
                      0, n_live, workspace, workspace_bytes);
    if (rc) return rc;
    cudaStream_t st = as_stream(stream);
    launch_k("paged_compact_kernel", paged_compact_kernel, PB_CTAS, PB_THREADS, 0, st, p);
    SA_CHECK_LAUNCH("paged_compact_kernel");
    return copy_pages(p, caches, n_caches, slot_bytes, vec, true, st);
}
