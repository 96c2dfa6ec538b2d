"""GPU tests of the sink-window attention and the paged decode when calls
follow and overlap each other: long runs of the same backward, and two streams
at once."""
import pytest
import torch

from fixed_pattern_sparse_sa_b200 import api
from test_gpu_decode_values import _case
from test_gpu_sink_attn import BF, HF, _dense, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("T,Hq,Hkv,d,window,sinks", [(16384, 16, 1, 128, 2048, 128), (4096, 24, 8, 64, 300, 16)])
def test_a_long_run_of_the_same_backward(cuda_ok, T, Hq, Hkv, d, window, sinks, parts):
    q, k, v = _dense(1, T, T, Hq, Hkv, d, BF, 81)
    dout = _rand(torch.Generator(device="cuda").manual_seed(82), q.shape, BF)
    out, lse = api.sink_attn_fwd(q, k, v, window, sinks, weight_parts=parts)
    want = api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, weight_parts=parts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            got = api.sink_attn_bwd(q, k, v, None, lse, dout, window, sinks, weight_parts=parts)
    for _ in range(5):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    api.check_device_status()


def test_two_streams_at_once(cuda_ok):
    jobs = []
    for seed, dt in ((83, BF), (84, HF)):
        q, k, v = _dense(2, 1500, 1500, 16, 2, 128, dt, seed)
        dout = _rand(torch.Generator(device="cuda").manual_seed(seed), q.shape, dt)
        qd, kc, vc, table, lt = _case([4000, 77, 900, 1] * 8, 16, 4, 64, 16, dt, seed)

        def job(q=q, k=k, v=v, dout=dout, qd=qd, kc=kc, vc=vc, table=table, lt=lt, dt=dt):
            out, lse = api.sink_attn_fwd(q, k, v, 200, 30)
            grads = api.sink_attn_bwd(q, k, v, None, lse, dout, 200, 30) if dt == BF else ()
            return out, lse, *grads, *api.paged_attn_decode(qd, kc, vc, table, lt, window=500, sinks=3)
        jobs.append((job, job()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, (s, (job, _)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i].append(job())
    torch.cuda.synchronize()
    api.check_device_status()
    for results, (_, want) in zip(got, jobs):
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
