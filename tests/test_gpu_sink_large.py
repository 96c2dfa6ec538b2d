"""GPU tests of the sink-window attention on calls of more than 8192 rows
(batch x queries x heads), which small calls do not reach: head dims, types,
head groups, sinks and packed batches against the plain 64-bit form, unseen
infinities and NaN, captured graphs."""
import math

import pytest
import torch

import _sink_ref as ref
from fixed_pattern_sparse_sa_b200 import api
from test_gpu_sink_attn import BF, HF, _dense, _packed, _rand

pytestmark = pytest.mark.gpu

#         B  Tq    L     Hq  Hkv  d  window sinks type fused
LARGE = [(1, 1100, 1100, 8, 2, 64, 33, 5, BF, True),           # few sinks beside a narrow window
         (1, 1100, 1100, 8, 2, 64, 33, 5, HF, True),
         (2, 701, 701, 6, 2, 128, 100, 130, BF, False),        # groups of 3, more sinks than a tile of keys
         (2, 701, 701, 6, 2, 128, 100, 130, HF, False),
         (1, 1700, 1700, 5, 1, 128, 257, 16, BF, False),       # groups of 5
         (1, 1700, 1700, 5, 1, 64, 257, 17, HF, False),
         (1, 60, 300, 160, 1, 64, 20, 40, BF, False),          # 160 heads on one KV head, a longer cache
         (1, 60, 300, 160, 1, 128, 20, 40, HF, False),
         (1, 8300, 8300, 1, 1, 64, 17, 300, BF, False),
         (1, 600, 1500, 16, 1, 128, 128, 0, BF, False),
         (3, 400, 400, 8, 8, 64, 1000, 0, HF, False),          # a window longer than the sequence
         (3, 400, 400, 8, 8, 128, 1000, 9, BF, False),
         (1, 513, 513, 32, 2, 64, 4, 0, BF, True),
         (1, 513, 513, 32, 2, 128, 1, 1, BF, False),           # the token itself and one sink
         (9000, 1, 3, 1, 1, 64, 2, 1, BF, False),              # one query each
         (1, 512, 512, 16, 4, 128, 70, 20, BF, False),         # 8192 rows
         (1, 513, 513, 16, 4, 128, 70, 20, BF, False)]         # and the next


@pytest.mark.parametrize("B,Tq,L,Hq,Hkv,d,window,sinks,dt,fused", LARGE)
def test_dense(cuda_ok, B, Tq, L, Hq, Hkv, d, window, sinks, dt, fused):
    q, k, v = _dense(B, Tq, L, Hq, Hkv, d, dt, 41, fused)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks)
    api.check_device_status()
    some = range(B) if B < 10 else range(0, B, 997)
    for b in some:
        ro, rl, bo = ref.fwd(q[b], k[b], v[b], L - Tq, window, sinks)
        ref.close(out[b], ro, bo, f"out[{b}]")
        ref.close_lse(lse[b], rl, f"lse[{b}]")
    if dt != BF:
        return
    dout = _rand(torch.Generator(device="cuda").manual_seed(42), q.shape, dt)
    grads = api.sink_attn_bwd(q, k, v, out, lse, dout, window, sinks)
    api.check_device_status()
    for b in some:
        want, bounds = ref.bwd(q[b], k[b], v[b], dout[b], L - Tq, window, sinks)
        for g, w, e, n in zip(grads, want, bounds, ("dq", "dk", "dv")):
            ref.close(g[b], w, e, f"{n}[{b}]")


#          query lengths                   key lengths                     Hq Hkv d  window sinks type
PACKED = [([5, 0, 1, 300, 1400, 64], [5, 7, 1, 300, 1400, 200], 8, 2, 64, 50, 3, BF),
          ([129, 1, 0, 657], [129, 400, 0, 657], 16, 1, 128, 128, 130, BF),
          ([1200, 900, 31], [1000, 900, 31], 4, 4, 128, 60, 2, BF),     # more queries than keys: the first see nothing
          ([1] * 1700, [1 + i % 270 for i in range(1700)], 5, 1, 64, 31, 4, HF),
          ([700, 3, 800], [700, 900, 800], 6, 2, 128, 77, 0, HF)]


@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,window,sinks,dt", PACKED)
def test_packed(cuda_ok, ql, kl, Hq, Hkv, d, window, sinks, dt):
    q, k, v, cu_q, cu_k = _packed(ql, kl, Hq, Hkv, d, dt, 43, before=3, behind=70)
    lens = dict(cu_q=cu_q, cu_k=cu_k, max_q=max(ql), max_k=max(kl))
    dout = _rand(torch.Generator(device="cuda").manual_seed(44), q.shape, dt)
    for t, cu in ((q, cu_q), (k, cu_k), (v, cu_k), (dout, cu_q)):         # rows outside every sequence hold anything
        t[: int(cu[0])] = float("nan")
        t[int(cu[-1]):] = float("inf")
    res = [torch.full_like(x, 7.0) for x in (q, q, k, v)] + [torch.full(q.shape[:2], 7.0, device="cuda")]
    out, dq, dk, dv, lse = res
    api.sink_attn_fwd(q, k, v, window, sinks, **lens, out=out, lse=lse)
    if dt == BF:
        api.sink_attn_bwd(q, k, v, out, lse, dout, window, sinks, **lens, dq=dq, dk=dk, dv=dv)
    api.check_device_status()
    for x, cu in zip(res, (cu_q, cu_q, cu_k, cu_k, cu_q)):
        assert (x[: int(cu[0])] == 7).all() and (x[int(cu[-1]):] == 7).all()
    for b in range(0, len(ql), 1 if len(ql) < 50 else 61):
        sq, sk = (slice(*cu[b:b + 2].tolist()) for cu in (cu_q, cu_k))
        ro, rl, bo = ref.fwd(q[sq], k[sk], v[sk], kl[b] - ql[b], window, sinks)
        ref.close(out[sq], ro, bo, f"out[{b}]")
        ref.close_lse(lse[sq], rl, f"lse[{b}]")
        if dt == BF:
            want, bounds = ref.bwd(q[sq], k[sk], v[sk], dout[sq], kl[b] - ql[b], window, sinks)
            for g, w, e, n in zip((dq[sq], dk[sk], dv[sk]), want, bounds, ("dq", "dk", "dv")):
                ref.close(g, w, e, f"{n}[{b}]")


def test_q_pos0(cuda_ok):
    # a preallocated cache: the keys behind the last query hold NaN
    q, k, v = _dense(1, 533, 900, 16, 1, 128, BF, 45)
    k[:, 633:], v[:, 633:] = float("nan"), float("inf")
    out, lse = api.sink_attn_fwd(q, k, v, 140, 4, q_pos0=100)
    ro, rl, bo = ref.fwd(q[0], k[0, :633], v[0, :633], 100, 140, 4)
    ref.close(out[0], ro, bo, "out")
    ref.close_lse(lse[0], rl, "lse")
    dout = torch.ones_like(q)
    dq, dk, dv = api.sink_attn_bwd(q, k, v, out, lse, dout, 140, 4, q_pos0=100)
    want, bounds = ref.bwd(q[0], k[0, :633], v[0, :633], dout[0], 100, 140, 4)
    for g, w, e, n in zip((dq[0], dk[0, :633], dv[0, :633]), want, bounds, ("dq", "dk", "dv")):
        ref.close(g, w, e, n)
    assert (dk[:, 633:] == 0).all() and (dv[:, 633:] == 0).all()
    # positions beyond the cache: the window runs out of keys, then only the sinks are left, or nothing
    q, k, v = _dense(1, 2600, 1050, 4, 2, 64, BF, 46)
    for sinks in (0, 3, 140):
        out, lse = api.sink_attn_fwd(q, k, v, 20, sinks, q_pos0=30)
        ro, rl, bo = ref.fwd(q[0], k[0], v[0], 30, 20, sinks)
        ref.close(out[0], ro, bo, "out")
        ref.close_lse(lse[0], rl, "lse")
        g = api.sink_attn_bwd(q, k, v, out, lse, torch.ones_like(q), 20, sinks, q_pos0=30)
        want, bounds = ref.bwd(q[0], k[0], v[0], torch.ones_like(q[0]), 30, 20, sinks)
        for x, w, e, n in zip(g, want, bounds, ("dq", "dk", "dv")):
            ref.close(x[0], w, e, n)
    api.check_device_status()


@pytest.mark.parametrize("T,Hq,Hkv,d,dt", [(1100, 8, 2, 128, HF), (1100, 16, 1, 64, BF), (2800, 3, 1, 128, BF),
                                           (560, 16, 1, 128, BF), (1100, 12, 4, 64, HF)])
@pytest.mark.parametrize("window,sinks", [(70, 5), (400, 5), (300, 40), (333, 140), (90, 0)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_unseen_values_reach_no_row(cuda_ok, T, Hq, Hkv, d, dt, window, sinks, bad):
    q, k, v = _dense(1, T, T, Hq, Hkv, d, dt, 47)
    clean = api.sink_attn_fwd(q, k, v, window, sinks)
    other = [c for c in range(d) if c not in (3, d - 1)]
    for j in (150, 2, T - 1):                                     # in the band, in the sinks or the first keys, the last key
        k2, v2 = k.clone(), v.clone()
        v2[0, j, :, 3] = v2[0, j, :, d - 1] = bad
        out, lse = api.sink_attn_fwd(q, k2, v2, window, sinks)
        t = torch.arange(T, device="cuda")
        seen = (t >= j) & ((t - j < window) | (j < sinks))
        assert torch.equal(out[0, ~seen], clean[0][0, ~seen]) and torch.equal(lse, clean[1])
        for c in (3, d - 1):
            x = out[0, seen][..., c]
            assert torch.isnan(x).all() if math.isnan(bad) else (x == bad).all()
        assert torch.equal(out[0, seen][..., other], clean[0][0, seen][..., other])
        k2[0, j] = bad                                            # a bad key: its rows are lost, no other
        out, _ = api.sink_attn_fwd(q, k2, v, window, sinks)
        assert torch.equal(out[0, ~seen], clean[0][0, ~seen])
    api.check_device_status()


def test_graph_and_repeats(cuda_ok):
    q, k, v = _dense(1, 1200, 1200, 8, 2, 64, BF, 48)
    dout = torch.randn(q.shape, device="cuda").to(BF)

    def step():
        out, lse = api.sink_attn_fwd(q, k, v, 130, 20)
        return out, lse, *api.sink_attn_bwd(q, k, v, out, lse, dout, 130, 20)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    q.copy_(q.flip(1).clone())
    want = step()
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    api.check_device_status()
