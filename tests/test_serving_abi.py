"""CPU checks of the sink-window and paged-cache entry points: arguments that
the host must refuse before anything is enqueued (the pointers are never
dereferenced), workspace sizes, and the binding's refusal of CPU tensors."""
import ctypes

import pytest
import torch

from fixed_pattern_sparse_sa_b200 import _lib, api, build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
N = None


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _sink(**kw):
    s = _lib.sa_sink_shape()
    base = dict(dtype=0, B=2, Hq=4, Hkv=2, d=64, window=8, sinks=2, scale=0.1, Tq=16, L=16, q_pos0=0)
    for k, v in {**base, **{a: b for a, b in kw.items() if not a.endswith("stride")}}.items():
        setattr(s, k, v)
    for name, heads in (("q_stride", 4), ("k_stride", 2), ("v_stride", 2), ("dout_stride", 4)):
        for i, x in enumerate(kw.get(name, (16 * heads * 64, heads * 64, 64))):
            getattr(s, name)[i] = x
    return ctypes.byref(s)


def _fwd(lib, s, q=P, k=P, v=P, cu_q=N, cu_k=N, out=P, lse=P):
    return lib.sa_sink_attn_fwd(s, q, k, v, cu_q, cu_k, out, lse, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(Tq=-1), INVALID), (dict(q_pos0=-1), INVALID), (dict(max_q=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(d=96), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED),
    (dict(L=1 << 31), UNSUPPORTED), (dict(Tq=1 << 31), UNSUPPORTED), (dict(q_pos0=1 << 31), UNSUPPORTED),
    (dict(q_stride=(1024, 256, 63)), INVALID), (dict(k_stride=(-8, 128, 64)), INVALID)])
def test_sink_shapes(lib, kw, code):
    assert _fwd(lib, _sink(**kw)) == code
    ws = 1 << 40
    assert lib.sa_sink_attn_bwd(_sink(**kw), P, P, P, P, P, P, N, N, P, P, P, P, ws, None) == code


def test_sink_pointers_and_workspace(lib):
    s = _sink()
    assert _fwd(lib, None) == INVALID
    for name in ("q", "k", "v", "out", "lse"):
        assert _fwd(lib, s, **{name: N}) == INVALID
        assert _fwd(lib, s, **{name: ODD}) == INVALID
    assert _fwd(lib, s, cu_q=P) == INVALID
    assert _fwd(lib, _sink(Tq=0), q=N, out=N, lse=N) == OK                 # nothing to do
    assert lib.sa_sink_attn_bwd(_sink(dtype=1), P, P, P, P, P, P, N, N, P, P, P, P, 1 << 40, None) == UNSUPPORTED
    assert lib.sa_sink_attn_bwd(s, P, P, P, P, P, P, N, N, P, P, P, P, 16, None) == WORKSPACE
    assert lib.sa_sink_attn_bwd(s, P, P, P, P, P, P, N, N, P, P, P, N, 1 << 40, None) == WORKSPACE
    assert lib.sa_sink_attn_bwd(s, P, P, P, P, P, N, N, N, P, P, P, P, 1 << 40, None) == INVALID
    assert lib.sa_sink_attn_bwd(s, P, P, P, P, P, P, N, N, P, N, P, P, 1 << 40, None) == INVALID
    assert lib.sa_sink_attn_bwd(_sink(dout_stride=(1, 1, 1)), P, P, P, P, P, P, N, N, P, P, P, P, 1 << 40,
                                None) == INVALID
    n = lib.sa_sink_attn_bwd_workspace_size(s, 0)
    assert n >= 2 * 16 * 4 * 4 and n % 256 == 0
    assert lib.sa_sink_attn_bwd_workspace_size(None, 0) == 0


def _paged(**kw):
    s = _lib.sa_paged_shape()
    base = dict(dtype=0, B=2, Hq=4, Hkv=2, d=64, page=16, max_pages=4, window=0, sinks=0, scale=0.1, n_pages=9)
    for k, v in {**base, **{a: b for a, b in kw.items() if not a.endswith("stride")}}.items():
        setattr(s, k, v)
    for name, val in (("q_stride", (256, 64)), ("k_stride", (2048, 128, 64)), ("v_stride", (2048, 128, 64))):
        for i, x in enumerate(kw.get(name, val)):
            getattr(s, name)[i] = x
    return ctypes.byref(s)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(Hq=3), INVALID), (dict(page=0), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED),
    (dict(n_pages=1 << 40), UNSUPPORTED), (dict(q_stride=(256, 4)), INVALID), (dict(k_stride=(2048, 128, -64)), INVALID)])
def test_decode_shapes(lib, kw, code):
    assert lib.sa_paged_attn_decode(_paged(**kw), P, P, P, P, P, P, P, P, 1 << 40, None) == code


def test_decode_pointers_and_workspace(lib):
    f = lib.sa_paged_attn_decode
    for i in range(7):
        args = [P] * 7
        args[i] = N
        assert f(_paged(), *args, P, 1 << 40, None) == INVALID, i
        args[i] = ODD
        assert f(_paged(), *args, P, 1 << 40, None) == INVALID, i
    assert f(_paged(), *[P] * 7, P, 64, None) == WORKSPACE
    assert f(_paged(), *[P] * 7, N, 1 << 40, None) == WORKSPACE
    assert f(_paged(), *[P] * 7, ODD, 1 << 40, None) == INVALID
    assert f(_paged(B=0), *[N] * 7, N, 0, None) == OK
    assert lib.sa_paged_attn_decode_workspace_size(4, 16, 1, 96) == 0
    assert lib.sa_paged_attn_decode_workspace_size(4, 16, 1, 128) > 0


def test_books(lib):
    size = lib.sa_paged_books_workspace_size(4, 3, 100)
    assert size >= (4 + 4 + 3 + 3 + 300) * 4 and lib.sa_paged_books_workspace_size(-1, 0, 0) == 0

    def extend(table=P, lens=P, rc=P, S=4, width=8, pages=100, page=16, seqs=P, n_new=P, n=3, start=P, ws=P, nb=size):
        return lib.sa_paged_extend(table, lens, rc, S, width, pages, page, seqs, n_new, n, start, ws, nb, None)
    for kw in (dict(table=N), dict(lens=N), dict(rc=ODD), dict(S=-1), dict(page=0), dict(n=-1), dict(seqs=N),
               dict(n_new=ODD), dict(start=N), dict(pages=-1), dict(ws=ODD)):
        assert extend(**kw) == INVALID, kw
    assert extend(width=1 << 27) == UNSUPPORTED and extend(pages=1 << 31) == UNSUPPORTED
    assert extend(nb=size - 1) == WORKSPACE and extend(ws=N) == WORKSPACE
    assert extend(n=0, seqs=N, n_new=N, start=N, ws=N, nb=0) == OK

    caches = (_lib.sa_page_cache * 2)()
    for c in caches:
        c.base, c.page_stride, c.slot_stride = 1 << 20, 4096, 256

    def fork(src=P, dst=P, n=3, caches=caches, nc=2, slot=256, done=P, nb=size):
        return lib.sa_paged_fork(P, P, P, 4, 8, 100, 16, src, dst, n, caches, nc, slot, done, P, nb, None)
    for kw in (dict(src=N), dict(dst=N), dict(done=N), dict(nc=-1), dict(caches=N), dict(slot=-4)):
        assert fork(**kw) == INVALID, kw
    assert fork(slot=6) == UNSUPPORTED and fork(nb=8) == WORKSPACE
    caches[1].base = None
    assert fork() == INVALID
    caches[1].base = (1 << 20) + 2
    assert fork() == INVALID
    caches[1].base = 1 << 20

    def free(table=P, page=16, seqs=P, n=3, window=0, sinks=0):
        return lib.sa_paged_free(table, P, P, 4, 8, 100, page, seqs, n, window, sinks, None)
    for kw in (dict(table=N), dict(page=0), dict(seqs=N), dict(window=-1), dict(sinks=-1), dict(n=-1)):
        assert free(**kw) == INVALID, kw
    assert free(n=0) == OK
    cs = lib.sa_paged_books_workspace_size(4, 0, 100)
    assert lib.sa_paged_compact(P, P, 4, 8, 100, 16, caches, 2, 256, N, P, cs, None) == INVALID
    assert lib.sa_paged_compact(P, N, 4, 8, 100, 16, caches, 2, 256, P, P, cs, None) == INVALID
    assert lib.sa_paged_compact(P, P, 4, 8, 100, 16, caches, 2, 256, P, P, cs - 1, None) == WORKSPACE
    assert lib.sa_paged_compact(P, P, 4, 8, 100, 16, caches, 2, 2, P, P, cs, None) == UNSUPPORTED


def test_write(lib):
    good = (ctypes.c_int64 * 10)(128, 64, 128, 64, 2048, 128, 64, 2048, 128, 64)
    odd = (ctypes.c_int64 * 10)(128, 64, 128, 64, 2048, 4, 64, 2048, 128, 64)

    def write(kn=P, kc=P, table=P, seqs=P, start=P, cu=N, n=3, rows=3, page=16, d=64, es=2, strides=good):
        return lib.sa_paged_write(kn, P, kc, P, table, seqs, start, cu, n, rows, 4, 8, 100, page, 2, d, es, strides, None)
    for kw in (dict(kn=N), dict(kc=ODD), dict(table=N), dict(seqs=N), dict(start=ODD), dict(cu=ODD), dict(rows=4),
               dict(page=0), dict(n=-1), dict(strides=odd), dict(strides=None)):
        assert write(**kw) == INVALID, kw
    assert write(d=4) == UNSUPPORTED
    assert write(n=0, rows=0, kn=N, seqs=N, start=N) == OK


def test_binding_refuses_cpu_tensors(lib):
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: api.sink_attn_fwd(q, q, q, 4), lambda: api.sink_attn_bwd(q, q, q, q, q, q, 4),
                 lambda: api.paged_attn_decode(q[0], q, q, t, t[0]), lambda: api.paged_extend(t, t[0], t[0], t[0], t[0], 4),
                 lambda: api.paged_write(q[0], q[0], q, q, t, t[0], t[0]),
                 lambda: api.paged_fork(t, t[0], t[0], t[0], t[0], 4), lambda: api.paged_free(t, t[0], t[0], t[0]),
                 lambda: api.paged_compact(t, t[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
