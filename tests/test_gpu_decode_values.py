"""GPU tests of the paged decode's values: outputs as exact as their type's
rounding (the bounds are derived in _tight_ref.py), and infinities and NaN in
visible and unseen keys."""
import math

import pytest
import torch

import _sink_ref as ref
import _tight_ref as tight
from fixed_pattern_sparse_sa_b200 import api
from test_gpu_paged import BF, HF, _pool

pytestmark = pytest.mark.gpu


def _case(lens, Hq, Hkv, d, page, dt, seed, lean=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table, lt, rc = _pool(lens, page, -(-max(lens) // page) + 1, 2, gen)
    kc, vc = (torch.randn((rc.shape[0], page, Hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    q = torch.randn((len(lens), Hq, d), generator=gen, device="cuda").to(dt)
    if lean:                                                      # the first key of each sequence takes most of the weight
        kc[table[:, 0].long(), 0] = (lean * q.view(len(lens), Hkv, -1, d)[:, :, 0].float()).to(dt)
    return q, kc, vc, table, lt


def _visible(n, window, sinks):
    j = torch.arange(n, device="cuda")
    return j if window is None else j[(j > n - 1 - window) | (j < sinks)]


#        lengths            Hq Hkv d  page window sinks type lean
TIGHT = [([1, 2, 3, 5, 9], 4, 1, 64, 16, None, 0, BF, 0.0),
         ([1, 2, 3, 5, 9], 4, 1, 64, 16, None, 0, HF, 0.0),
         ([777, 16, 2000], 16, 2, 128, 64, None, 0, BF, 0.0),
         ([777, 16, 2000], 16, 2, 128, 64, None, 0, HF, 0.0),
         ([3000] * 3, 8, 8, 128, 24, 90, 7, BF, 0.0),
         ([20000], 6, 2, 64, 128, None, 0, HF, 0.0),
         ([30000, 70], 8, 1, 128, 64, None, 0, HF, 0.9),          # one key against many small weights
         ([30000, 70], 8, 1, 128, 64, None, 0, BF, 0.9),
         ([1500] * 50, 16, 1, 64, 16, 400, 4, HF, 0.5)]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,sinks,dt,lean", TIGHT)
def test_as_exact_as_the_type(cuda_ok, lens, Hq, Hkv, d, page, window, sinks, dt, lean):
    q, kc, vc, table, lt = _case(lens, Hq, Hkv, d, page, dt, 51, lean)
    out, lse = api.paged_attn_decode(q, kc, vc, table, lt, window=window, sinks=sinks)
    api.check_device_status()
    for b in range(0, len(lens), 1 if len(lens) < 10 else 7):
        j = _visible(lens[b], window, sinks)
        pg = table[b, j // page].long()
        ro, rl, bo = tight.fwd(q[b:b + 1], kc[pg, j % page], vc[pg, j % page], len(j) - 1, len(j), 0)
        ref.close(out[b:b + 1], ro, bo, f"out[{b}]")
        ref.close_lse(lse[b:b + 1], rl, f"lse[{b}]")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("n,window,sinks", [(3, None, 0), (40, None, 0), (900, None, 0), (5000, 300, 5)])
def test_the_error_is_the_outputs_rounding(cuda_ok, n, window, sinks, dt):
    """Over 2^16 outputs: the error's 2-norm is that of rounding the exact outputs, 1.41 times that with weights of one
    part.  Two parts leave 2^-16 a weight at most against the 2^-9 (bf16) or 2^-12 (fp16) of a rounding's mean."""
    page = 32
    q, kc, vc, table, lt = _case([n] * 32, 16, 4, 128, page, dt, 53)
    out, lse = api.paged_attn_decode(q, kc, vc, table, lt, window=window, sinks=sinks)
    j = _visible(n, window, sinks)
    at = [(table[b, j // page].long(), j % page) for b in range(32)]
    exact = torch.cat([ref.fwd(q[b:b + 1], kc[a], vc[a], len(j) - 1, len(j), 0)[0] for b, a in enumerate(at)])
    own, least = ((x.double() - exact).norm().item() for x in (out, exact.to(dt)))
    assert own <= 1.2 * least, f"{own / least:.3f} times an output rounding"


@pytest.mark.parametrize("Hq,Hkv,d,dt", [(1, 1, 64, BF), (8, 2, 128, HF), (16, 1, 128, BF), (40, 2, 64, HF)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_visible_value_that_is_not_finite_stays_in_its_column(cuda_ok, Hq, Hkv, d, dt, bad):
    lens, page, window, sinks = [1, 40, 700, 2500], 16, 300, 5
    q, kc, vc, table, lt = _case(lens, Hq, Hkv, d, page, dt, 52)
    clean = api.paged_attn_decode(q, kc, vc, table, lt, window=window, sinks=sinks)
    for back in (0, 1, 37, 200, 299, 300, 650, 2499):             # keys from the newest on; the last ones are unseen or sinks
        v2 = vc.clone()
        hit = torch.zeros(len(lens), dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            j = n - 1 - back
            if j < 0:
                continue
            v2[int(table[b, j // page]), j % page, :, 3] = bad
            hit[b] = back < window or j < sinks
        out, lse = api.paged_attn_decode(q, kc, v2, table, lt, window=window, sinks=sinks)
        api.check_device_status()
        assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])
        other = [c for c in range(d) if c != 3]
        assert torch.equal(out[..., other], clean[0][..., other])
        x = out[hit][..., 3]
        assert torch.isnan(x).all() if math.isnan(bad) else (x == bad).all(), back
