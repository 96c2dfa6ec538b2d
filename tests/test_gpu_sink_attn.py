"""GPU tests of the sink-window attention against its plain 64-bit form:
values and gradients over dense and packed batches, odd sizes, head groups,
strided inputs, rows that see nothing, unseen infinities and NaN, refusals,
streams and captured graphs.  The bounds are derived in _sink_ref.py."""
import math

import pytest
import torch

import _sink_ref as ref
from fixed_pattern_sparse_sa_b200 import _lib, api

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _rand(gen, shape, dt):
    return torch.randn(shape, generator=gen, device="cuda").to(dt)


def _dense(B, Tq, L, Hq, Hkv, d, dt, seed, fused=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        qkv = _rand(gen, (B, L, Hq + 2 * Hkv, d), dt)
        return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    return _rand(gen, (B, Tq, Hq, d), dt), _rand(gen, (B, L, Hkv, d), dt), _rand(gen, (B, L, Hkv, d), dt)


#        B  Tq   L    Hq Hkv  d  window sinks  type fused
DENSE = [(1, 1, 1, 1, 1, 64, 1, 0, BF, False),
         (1, 1, 300, 4, 1, 128, 64, 4, BF, False),           # one new token
         (2, 257, 257, 8, 2, 64, 33, 5, BF, True),           # odd length, views of one projection
         (1, 130, 513, 16, 1, 128, 100, 130, HF, False),     # more sinks than a tile of keys, a longer cache
         (3, 100, 100, 3, 3, 128, 1000, 0, HF, False),       # a window longer than the sequence
         (1, 515, 515, 10, 2, 128, 1, 1, BF, True),          # groups of 5, the token itself and one sink
         (1, 400, 400, 12, 4, 64, 128, 16, HF, False),       # groups of 3
         (2, 190, 200, 1, 1, 64, 17, 300, BF, False),        # sinks past the whole sequence
         (1, 700, 700, 32, 2, 128, 256, 64, BF, False),
         (1, 5, 40, 160, 1, 128, 9, 2, BF, False),           # 160 heads on one KV head
         (1, 2, 90, 1, 1, 128, 90, 0, BF, False)]


@pytest.mark.parametrize("B,Tq,L,Hq,Hkv,d,window,sinks,dt,fused", DENSE)
def test_dense_forward(cuda_ok, B, Tq, L, Hq, Hkv, d, window, sinks, dt, fused):
    q, k, v = _dense(B, Tq, L, Hq, Hkv, d, dt, 1, fused)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks)
    api.check_device_status()
    assert out.dtype == dt and out.shape == q.shape and lse.shape == q.shape[:-1]
    for b in range(B):
        ro, rl, bo = ref.fwd(q[b], k[b], v[b], L - Tq, window, sinks)
        ref.close(out[b], ro, bo, f"out[{b}]")
        ref.close_lse(lse[b], rl, f"lse[{b}]")


@pytest.mark.parametrize("B,Tq,L,Hq,Hkv,d,window,sinks,dt,fused", [c for c in DENSE if c[8] == BF])
def test_dense_backward(cuda_ok, B, Tq, L, Hq, Hkv, d, window, sinks, dt, fused):
    q, k, v = _dense(B, Tq, L, Hq, Hkv, d, dt, 2, fused)
    dout = _rand(torch.Generator(device="cuda").manual_seed(3), (B, Hq, Tq, d), dt).transpose(1, 2)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks)
    # out and lse are read through strides too
    grads = api.sink_attn_bwd(q, k, v, torch.cat([out, out], 2)[:, :, Hq:], torch.cat([lse, lse], 1)[:, Tq:], dout,
                              window, sinks)
    api.check_device_status()
    for b in range(B):
        want, bounds = ref.bwd(q[b], k[b], v[b], dout[b], L - Tq, window, sinks)
        for g, w, e, n in zip(grads, want, bounds, ("dq", "dk", "dv")):
            ref.close(g[b], w, e, f"{n}[{b}]")


def _packed(ql, kl, Hq, Hkv, d, dt, seed, before=0, behind=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cu = [torch.tensor([before, *x], device="cuda").cumsum(0).to(torch.int32) for x in (ql, kl)]
    q = _rand(gen, (before + sum(ql) + behind, Hq, d), dt)
    k, v = (_rand(gen, (before + sum(kl) + behind, Hkv, d), dt) for _ in range(2))
    return q, k, v, cu[0], cu[1]


#          query lengths        key lengths           Hq Hkv d  window sinks type
PACKED = [([5, 0, 1, 300, 64], [5, 7, 1, 300, 200], 8, 2, 64, 50, 3, BF),
          ([129, 1, 0, 257], [129, 400, 0, 257], 16, 1, 128, 128, 130, BF),
          ([20, 9], [12, 9], 4, 4, 128, 6, 2, BF),            # more queries than keys: the first ones see nothing
          ([1] * 40, [1 + 7 * i for i in range(40)], 5, 1, 64, 31, 4, HF),
          ([333], [333], 6, 2, 128, 77, 0, BF)]


@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,window,sinks,dt", PACKED)
def test_packed(cuda_ok, ql, kl, Hq, Hkv, d, window, sinks, dt):
    q, k, v, cu_q, cu_k = _packed(ql, kl, Hq, Hkv, d, dt, 4, before=3, behind=70)
    for t, cu in ((q, cu_q), (k, cu_k), (v, cu_k)):               # rows outside every sequence hold anything
        t[: int(cu[0])] = float("nan")
        t[int(cu[-1]):] = float("inf")
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    api.sink_attn_fwd(q, k, v, window, sinks, cu_q=cu_q, cu_k=cu_k, max_q=max(ql), max_k=max(kl), out=out, lse=lse)
    api.check_device_status()
    a, e = int(cu_q[0]), int(cu_q[-1])
    assert (out[:a] == 7).all() and (out[e:] == 7).all() and (lse[:a] == 7).all() and (lse[e:] == 7).all()
    seqs = [(slice(*cu_q[b:b + 2].tolist()), slice(*cu_k[b:b + 2].tolist())) for b in range(len(ql))]
    for (sq, sk), n, m in zip(seqs, ql, kl):
        ro, rl, bo = ref.fwd(q[sq], k[sk], v[sk], m - n, window, sinks)
        ref.close(out[sq], ro, bo, "out")
        ref.close_lse(lse[sq], rl, "lse")
    if dt != BF:
        return
    dout = _rand(torch.Generator(device="cuda").manual_seed(5), q.shape, dt)
    dout[e:] = float("nan")
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    api.sink_attn_bwd(q, k, v, out, lse, dout, window, sinks, cu_q=cu_q, cu_k=cu_k, max_q=max(ql), max_k=max(kl),
                      dq=dq, dk=dk, dv=dv)
    api.check_device_status()
    ka, ke = int(cu_k[0]), int(cu_k[-1])
    assert (dq[:a] == 7).all() and (dq[e:] == 7).all()
    assert all((g[:ka] == 7).all() and (g[ke:] == 7).all() for g in (dk, dv))
    for (sq, sk), n, m in zip(seqs, ql, kl):
        want, bounds = ref.bwd(q[sq], k[sk], v[sk], dout[sq], m - n, window, sinks)
        for g, w, b_, name in zip((dq[sq], dk[sk], dv[sk]), want, bounds, ("dq", "dk", "dv")):
            ref.close(g, w, b_, name)


def test_lengths_unknown_and_all_empty(cuda_ok):
    q, k, v, cu_q, cu_k = _packed([40, 3], [40, 10], 4, 2, 64, BF, 6)
    a = api.sink_attn_fwd(q, k, v, 9, 2, cu_q=cu_q, cu_k=cu_k)
    b = api.sink_attn_fwd(q, k, v, 9, 2, cu_q=cu_q, cu_k=cu_k, max_q=40, max_k=64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = api.sink_attn_fwd(q, k, v, 9, 2, cu_q=z, cu_k=z, out=torch.full_like(q, 3.0))
    assert (out == 3).all()
    empty = q[:0]
    o, l = api.sink_attn_fwd(empty, k, v, 9, 2, cu_q=z, cu_k=z)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)
    dq, dk, dv = api.sink_attn_bwd(empty, k, v, o, l, empty, 9, 2, cu_q=z, cu_k=cu_k.new_tensor([0, 9, 9, 50]))
    assert dq.numel() == 0 and (dk == 0).all() and (dv == 0).all()
    api.check_device_status()


def test_q_pos0_past_the_queries_and_past_the_cache(cuda_ok):
    # a preallocated cache: the keys behind the last query hold NaN
    q, k, v = _dense(1, 33, 400, 8, 1, 128, BF, 7)
    k[:, 133:], v[:, 133:] = float("nan"), float("inf")
    out, lse = api.sink_attn_fwd(q, k, v, 40, 4, q_pos0=100)
    ro, rl, bo = ref.fwd(q[0], k[0, :133], v[0, :133], 100, 40, 4)
    ref.close(out[0], ro, bo, "out")
    ref.close_lse(lse[0], rl, "lse")
    dout = torch.ones_like(q)
    dq, dk, dv = api.sink_attn_bwd(q, k, v, out, lse, dout, 40, 4, q_pos0=100)
    want, bounds = ref.bwd(q[0], k[0, :133], v[0, :133], dout[0], 100, 40, 4)
    for g, w, e, n in zip((dq[0], dk[0, :133], dv[0, :133]), want, bounds, ("dq", "dk", "dv")):
        ref.close(g, w, e, n)
    assert (dk[:, 133:] == 0).all() and (dv[:, 133:] == 0).all()
    # positions beyond the cache: the window runs out of keys, then only the sinks are left, or nothing
    q, k, v = _dense(1, 60, 50, 4, 2, 64, BF, 8)
    for sinks in (0, 3):
        out, lse = api.sink_attn_fwd(q, k, v, 20, sinks, q_pos0=30)
        ro, rl, bo = ref.fwd(q[0], k[0], v[0], 30, 20, sinks)
        ref.close(out[0], ro, bo, "out")
        ref.close_lse(lse[0], rl, "lse")
        g = api.sink_attn_bwd(q, k, v, out, lse, torch.ones_like(q), 20, sinks, q_pos0=30)
        want, bounds = ref.bwd(q[0], k[0], v[0], torch.ones_like(q[0]), 30, 20, sinks)
        for x, w, e, n in zip(g, want, bounds, ("dq", "dk", "dv")):
            ref.close(x[0], w, e, n)
    api.check_device_status()


@pytest.mark.parametrize("Hq,Hkv,d,dt", [(1, 1, 128, BF), (16, 1, 128, HF), (6, 2, 64, BF)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_unseen_values_reach_no_row(cuda_ok, Hq, Hkv, d, dt, bad):
    T, window, sinks = 300, 70, 5
    q, k, v = _dense(1, T, T, Hq, Hkv, d, dt, 9)
    clean = api.sink_attn_fwd(q, k, v, window, sinks)
    j = 150                                                       # seen by the queries 150 .. 219
    k2, v2 = k.clone(), v.clone()
    v2[0, j, :, 3] = bad
    out, lse = api.sink_attn_fwd(q, k2, v2, window, sinks)
    unseen = torch.ones(T, dtype=torch.bool, device="cuda")
    unseen[j:j + window] = False
    assert torch.equal(out[0, unseen], clean[0][0, unseen]) and torch.equal(lse, clean[1])
    seen = out[0, ~unseen]
    assert torch.isnan(seen[..., 3]).all() if math.isnan(bad) else (seen[..., 3] == math.inf).all()
    other = [c for c in range(d) if c != 3]
    assert torch.equal(seen[..., other], clean[0][0, ~unseen][..., other])
    k2[0, j] = bad                                                # a bad key: its rows are lost, no other
    out, _ = api.sink_attn_fwd(q, k2, v, window, sinks)
    assert torch.equal(out[0, unseen], clean[0][0, unseen])
    api.check_device_status()


def test_repeats_bit_for_bit(cuda_ok):
    q, k, v = _dense(2, 500, 500, 16, 2, 128, BF, 10)
    dout = torch.randn(q.shape, device="cuda").to(BF)
    first = None
    for _ in range(3):
        out, lse = api.sink_attn_fwd(q, k, v, 100, 20)
        got = (out, lse, *api.sink_attn_bwd(q, k, v, out, lse, dout, 100, 20))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_gradient_is_the_slope(cuda_ok):
    # sum(out * dout) along a direction of each input, by central differences of the 64-bit form
    q, k, v = _dense(1, 40, 40, 4, 2, 64, BF, 11)
    gen = torch.Generator(device="cuda").manual_seed(12)
    dout = _rand(gen, q.shape, BF)
    out, lse = api.sink_attn_fwd(q, k, v, 12, 3)
    grads = api.sink_attn_bwd(q, k, v, out, lse, dout, 12, 3)
    _, bounds = ref.bwd(q[0], k[0], v[0], dout[0], 0, 12, 3)
    for i, (g, b) in enumerate(zip(grads, bounds)):
        x = [t[0].double() for t in (q, k, v)]
        dirn = torch.randn(x[i].shape, generator=gen, device="cuda", dtype=torch.float64)

        def f(h):
            y = list(x)
            y[i] = y[i] + h * dirn
            return (ref.fwd(*y, 0, 12, 3)[0] * dout[0].double()).sum().item()

        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        # the kernel's gradient is within b of the formula's; the difference quotient is off by about 1e-10 / 1e-5
        assert abs((g[0].double() * dirn).sum().item() - slope) <= (b * dirn.abs()).sum().item() + 1e-4


def test_stream_and_graph(cuda_ok):
    q, k, v = _dense(1, 200, 200, 8, 2, 64, BF, 13)
    dout = torch.randn(q.shape, device="cuda").to(BF)
    want = api.sink_attn_fwd(q, k, v, 30, 4)
    wantg = api.sink_attn_bwd(q, k, v, *want, dout, 30, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = api.sink_attn_fwd(q, k, v, 30, 4)
        got = api.sink_attn_bwd(q, k, v, out, lse, dout, 30, 4)
    side.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(a, b) for a, b in zip(got, wantg))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = api.sink_attn_fwd(q, k, v, 30, 4)
        got = api.sink_attn_bwd(q, k, v, out, lse, dout, 30, 4)
    q.copy_(q.flip(1).clone())
    want = api.sink_attn_fwd(q, k, v, 30, 4)
    wantg = api.sink_attn_bwd(q, k, v, *want, dout, 30, 4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(a, b) for a, b in zip(got, wantg))


def test_bad_lengths_are_reported(cuda_ok):
    q, k, v, cu_q, cu_k = _packed([40, 30], [40, 30], 4, 2, 64, BF, 14)
    for cu in ([0, 50, 40], [-5, 40, 70], [0, 40, 900]):
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = api.sink_attn_fwd(q, k, v, 9, 2, cu_q=bad, cu_k=bad)
        with pytest.raises(api.SAError) as e:
            api.check_device_status()
        assert e.value.status == _lib.SA_ERR_DEVICE_ASSERT
        api.sink_attn_bwd(q, k, v, out, lse, q, 9, 2, cu_q=bad, cu_k=bad)
        with pytest.raises(api.SAError):
            api.check_device_status()


def test_refusals(cuda_ok):
    q, k, v = _dense(1, 32, 32, 4, 2, 64, BF, 15)
    cu = torch.tensor([0, 32], dtype=torch.int32, device="cuda")
    f = api.sink_attn_fwd
    with pytest.raises(TypeError):
        f(q.float(), k.float(), v.float(), 4)
    with pytest.raises(TypeError):
        f(q, k.half(), v, 4)
    with pytest.raises(ValueError):
        f(q.cpu(), k, v, 4)
    with pytest.raises(ValueError):
        f(q, k[:, :16], v, 4)
    with pytest.raises(ValueError):
        f(q, k, v, 4, cu_q=cu)
    with pytest.raises(ValueError):
        f(q, k[:, :16], v[:, :16], 4)                             # more queries than keys without q_pos0
    with pytest.raises(ValueError):
        f(q[0], k[0], v[0], 4, cu_q=cu, cu_k=cu, q_pos0=1)
    with pytest.raises(ValueError):
        f(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, 4)
    wide = torch.zeros(1, 32, 4, 65, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        f(wide[..., 1:], k, v, 4)
    with pytest.raises(ValueError):
        f(q, k, v, 4, out=torch.empty(1, 32, 4, 32, dtype=BF, device="cuda"))
    for kw in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, scale=math.inf)):
        with pytest.raises(api.SAError):
            f(q, k, v, **kw)
    q96, k96, v96 = _dense(1, 8, 8, 4, 2, 96, BF, 1)
    with pytest.raises(api.SAError, match="head dim"):
        f(q96, k96, v96, 4)
    with pytest.raises(api.SAError):
        f(q[:, :, :3], k, v, 4)                                   # 3 heads on 2
    out, lse = f(q, k, v, 4)
    with pytest.raises(TypeError):
        api.sink_attn_bwd(q.half(), k.half(), v.half(), out, lse, q, 4)
    with pytest.raises(ValueError):
        api.sink_attn_bwd(q, k, v, out, lse[:, :16], q, 4)
    api.check_device_status()


def test_a_wait_that_runs_out_is_reported(cuda_ok):
    # the stall hook keeps the kernels from loading anything: their first waits run out after the spin limit
    q, k, v = _dense(1, 600, 600, 8, 2, 128, BF, 16)
    dout = torch.randn(q.shape, device="cuda").to(BF)
    want = api.sink_attn_fwd(q, k, v, 100, 4)
    wantg = api.sink_attn_bwd(q, k, v, *want, dout, 100, 4)
    api.check_device_status()
    for call in (lambda: api.sink_attn_fwd(q, k, v, 100, 4), lambda: api.sink_attn_bwd(q, k, v, *want, dout, 100, 4)):
        try:
            api.debug_set_spin_limit(20_000_000)                  # about 10 ms
            api.debug_inject_stall(True)
            call()
            with pytest.raises(api.SAError) as e:
                api.check_device_status()
            assert e.value.status == _lib.SA_ERR_TIMEOUT
        finally:
            api.debug_inject_stall(False)
            api.debug_set_spin_limit(0)
        got = api.sink_attn_fwd(q, k, v, 100, 4)
        gotg = api.sink_attn_bwd(q, k, v, *got, dout, 100, 4)
        api.check_device_status()
        assert all(torch.equal(a, b) for a, b in zip((*want, *wantg), (*got, *gotg)))
