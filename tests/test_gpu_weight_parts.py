"""GPU tests of the sink-window attention with its weights in one and in two
parts, at sizes on both sides of the default's threshold: bounds that only two
parts meet, the error of many outputs against that of rounding them, unseen
values, and results that do not depend on the batch."""
import math

import pytest
import torch

import _sink_ref as ref
import _tight_ref as tight
from fixed_pattern_sparse_sa_b200 import _lib, api
from test_gpu_sink_attn import BF, DENSE, HF, _dense, _packed, _rand
from test_gpu_sink_attn import PACKED as SMALL_PACKED
from test_gpu_sink_large import LARGE
from test_gpu_sink_large import PACKED as LARGE_PACKED

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("B,Tq,L,Hq,Hkv,d,window,sinks,dt,fused", DENSE + LARGE)
def test_dense(cuda_ok, B, Tq, L, Hq, Hkv, d, window, sinks, dt, fused, parts):
    q, k, v = _dense(B, Tq, L, Hq, Hkv, d, dt, 61, fused)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks, weight_parts=parts)
    api.check_device_status()
    some = range(B) if B < 10 else range(0, B, 997)
    for b in some:
        ro, rl, bo = tight.fwd(q[b], k[b], v[b], L - Tq, window, sinks, parts=parts)
        ref.close(out[b], ro, bo, f"out[{b}]")
        ref.close_lse(lse[b], rl, f"lse[{b}]")
    if dt != BF:
        return
    dout = _rand(torch.Generator(device="cuda").manual_seed(62), q.shape, dt)
    grads = api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, weight_parts=parts)
    api.check_device_status()
    for b in some:
        want, bounds = tight.bwd(q[b], k[b], v[b], dout[b], L - Tq, window, sinks, parts=parts)
        for g, w, e, n in zip(grads, want, bounds, ("dq", "dk", "dv")):
            ref.close(g[b], w, e, f"{n}[{b}]")


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("ql,kl,Hq,Hkv,d,window,sinks,dt", SMALL_PACKED + LARGE_PACKED)
def test_packed(cuda_ok, ql, kl, Hq, Hkv, d, window, sinks, dt, parts):
    q, k, v, cu_q, cu_k = _packed(ql, kl, Hq, Hkv, d, dt, 63, before=3, behind=70)
    lens = dict(cu_q=cu_q, cu_k=cu_k, max_q=max(ql), max_k=max(kl), weight_parts=parts)
    dout = _rand(torch.Generator(device="cuda").manual_seed(64), q.shape, dt)
    for t, cu in ((q, cu_q), (k, cu_k), (v, cu_k), (dout, cu_q)):
        t[: int(cu[0])] = float("nan")
        t[int(cu[-1]):] = float("inf")
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks, **lens)
    grads = api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, **lens) if dt == BF else ()
    api.check_device_status()
    for b in range(0, len(ql), 1 if len(ql) < 50 else 61):
        sq, sk = (slice(*cu[b:b + 2].tolist()) for cu in (cu_q, cu_k))
        ro, rl, bo = tight.fwd(q[sq], k[sk], v[sk], kl[b] - ql[b], window, sinks, parts=parts)
        ref.close(out[sq], ro, bo, f"out[{b}]")
        ref.close_lse(lse[sq], rl, f"lse[{b}]")
        if grads:
            want, bounds = tight.bwd(q[sq], k[sk], v[sk], dout[sq], kl[b] - ql[b], window, sinks, parts=parts)
            for g, at, w, e, n in zip(grads, (sq, sk, sk), want, bounds, ("dq", "dk", "dv")):
                ref.close(g[at], w, e, f"{n}[{b}]")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("window,sinks", [(2, 1), (4, 0), (64, 16), (600, 130)])
def test_the_error_against_that_of_rounding(cuda_ok, window, sinks, dt):
    """2-norms over 2^17 values and more.  Two parts leave the outputs' own rounding; with one, every weight's rounding,
    independent of it and of the same size, stands beside it: sqrt(2) times at most where many terms meet."""
    T, Hq, Hkv, d = 1200, 8, 2, 128
    q, k, v = _dense(1, T, T, Hq, Hkv, d, dt, 65)
    dout = _rand(torch.Generator(device="cuda").manual_seed(66), q.shape, dt)
    exact = [ref.fwd(q[0], k[0], v[0], 0, window, sinks)[0]]
    if dt == BF:
        exact += ref.bwd(q[0], k[0], v[0], dout[0], 0, window, sinks)[0]
    for parts, most in ((2, 1.1), (1, 1.5)):
        out, lse = api.sink_attn_fwd(q, k, v, window, sinks, weight_parts=parts)
        got = [out]
        if dt == BF:
            got += api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, weight_parts=parts)
        for g, x, n in zip(got, exact, ("out", "dq", "dk", "dv")):
            own, least = ((y.double() - x).norm().item() for y in (g[0], x.to(dt)))
            assert own <= most * least, f"{n}: {own / least:.3f} times a rounding with {parts} part(s)"


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("T", [300, 1100])
@pytest.mark.parametrize("Hq,Hkv,d,dt", [(16, 1, 128, HF), (6, 2, 64, BF)])
@pytest.mark.parametrize("window,sinks", [(70, 5), (200, 40)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_unseen_values_reach_no_row(cuda_ok, T, Hq, Hkv, d, dt, window, sinks, bad, parts):
    q, k, v = _dense(1, T, T, Hq, Hkv, d, dt, 67)
    clean = api.sink_attn_fwd(q, k, v, window, sinks, weight_parts=parts)
    for j in (150, 2):
        k2, v2 = k.clone(), v.clone()
        v2[0, j, :, 3] = bad
        out, lse = api.sink_attn_fwd(q, k2, v2, window, sinks, weight_parts=parts)
        t = torch.arange(T, device="cuda")
        seen = (t >= j) & ((t - j < window) | (j < sinks))
        assert torch.equal(out[0, ~seen], clean[0][0, ~seen]) and torch.equal(lse, clean[1])
        x = out[0, seen][..., 3]
        assert torch.isnan(x).all() if math.isnan(bad) else (x == math.inf).all()
        k2[0, j] = bad
        out, _ = api.sink_attn_fwd(q, k2, v, window, sinks, weight_parts=parts)
        assert torch.equal(out[0, ~seen], clean[0][0, ~seen])
    api.check_device_status()


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("d,window,sinks", [(64, 50, 0), (128, 100, 9), (128, 40, 140)])
def test_a_sequence_alone_and_in_a_batch(cuda_ok, d, window, sinks, parts):
    lens, Hq, Hkv = [333, 40, 700, 1], 8, 2
    q, k, v, cu, _ = _packed(lens, lens, Hq, Hkv, d, BF, 68)
    dout = _rand(torch.Generator(device="cuda").manual_seed(69), q.shape, BF)
    kw = dict(cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens), weight_parts=parts)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks, **kw)
    grads = api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, **kw)
    for b in range(len(lens)):
        s = slice(*cu[b:b + 2].tolist())
        one = [x[s][None].contiguous() for x in (q, k, v, dout)]
        o, l = api.sink_attn_fwd(*one[:3], window, sinks, weight_parts=parts)
        dq, dk, dv = api.sink_attn_bwd(*one[:3], None, l, one[3], window, sinks, weight_parts=parts)
        assert torch.equal(o[0], out[s]) and torch.equal(l[0], lse[s]) and torch.equal(dq[0], grads[0][s])
        at = slice(sinks, None)                                   # (the sinks' sums are cut by the size of the batch)
        assert torch.equal(dk[0, at], grads[1][s][at]) and torch.equal(dv[0, at], grads[2][s][at])
    api.check_device_status()


def test_refusals(cuda_ok):
    q, k, v = _dense(1, 32, 32, 4, 2, 64, BF, 70)
    for bad in (0, 3, -1, "2"):
        with pytest.raises(ValueError, match="weight_parts"):
            api.sink_attn_fwd(q, k, v, 4, weight_parts=bad)
    out, lse = api.sink_attn_fwd(q, k, v, 4)
    with pytest.raises(ValueError, match="weight_parts"):
        api.sink_attn_bwd(q, k, v, out, lse, q, 4, weight_parts=3)
    assert torch.equal(out, api.sink_attn_fwd(q, k, v, 4, weight_parts=2)[0])


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(cuda_ok, d, parts):
    # the stall hook keeps the kernels from loading anything: their first waits run out after the spin limit
    q, k, v = _dense(1, 1100, 1100, 8, 2, d, BF, 71)
    dout = torch.randn(q.shape, device="cuda").to(BF)

    def step():
        out, lse = api.sink_attn_fwd(q, k, v, 100, 20, weight_parts=parts)
        return out, lse, *api.sink_attn_bwd(q, k, v, None, lse, dout, 100, 20, weight_parts=parts)

    want = step()
    api.check_device_status()
    try:
        api.debug_set_spin_limit(20_000_000)                      # about 10 ms
        api.debug_inject_stall(True)
        step()
        with pytest.raises(api.SAError) as e:
            api.check_device_status()
        assert e.value.status == _lib.SA_ERR_TIMEOUT
    finally:
        api.debug_inject_stall(False)
        api.debug_set_spin_limit(0)
    got = step()
    api.check_device_status()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
