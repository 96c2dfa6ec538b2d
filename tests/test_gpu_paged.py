"""GPU tests of the paged cache: decode attention against its plain 64-bit
form (bounds of _sink_ref.py), the page operations against a plain model of
the books on the host, and a run of them together as a server would make it."""
import math

import pytest
import torch

import _sink_ref as ref
from fixed_pattern_sparse_sa_b200 import _lib, api

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda").reshape(-1)


def _pool(lens, page, width, spare, gen, share=1):
    """Random tables over a pool: block_table, seq_lens, refcount."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=gen, device="cuda").tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    rc = torch.zeros(len(order), dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        ids = order[at:at + n]
        at += n
        table[s, :n] = torch.tensor(ids, dtype=torch.int32)
        rc[ids] = share
    return table.cuda(), _i32(lens), rc.cuda()


def _decode_check(q, kc, vc, table, lens, page, window, sinks, out, lse, scale=None):
    B = q.shape[0]
    for b in range(B):
        n = int(lens[b])
        j = torch.arange(n, device="cuda")
        if window is not None:
            j = j[(j > n - 1 - window) | (j < sinks)]
        if len(j) == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        pg, sl = table[b, j // page].long(), j % page
        # the visible keys as a sequence of their own
        ro, rl, bo = ref.fwd(q[b:b + 1], kc[pg, sl], vc[pg, sl], len(j) - 1, len(j), 0, scale)
        ref.close(out[b:b + 1], ro, bo, f"out[{b}]")
        ref.close_lse(lse[b:b + 1], rl, f"lse[{b}]")


#          lengths                              Hq Hkv d  page window sinks type interleaved
DECODE = [([1], 1, 1, 64, 1, None, 0, BF, False),
          ([17, 0, 1, 300, 64, 63, 65], 16, 1, 128, 16, None, 0, BF, False),
          ([2000], 8, 8, 128, 24, None, 0, HF, True),
          ([5, 1000, 77, 4096, 129], 8, 2, 64, 64, 100, 4, BF, True),
          ([33, 900, 31], 12, 4, 128, 8, 32, 100, HF, False),           # sinks inside, across and past the window
          ([700, 701], 40, 2, 128, 128, 64, 0, BF, False),              # 20 heads per KV head: two tiles
          ([9000], 6, 2, 64, 256, None, 0, HF, False),
          ([1 + 37 * (i % 50) for i in range(600)], 4, 1, 64, 16, None, 0, BF, False),   # more sequences than threads
          ([3000] * 40, 16, 8, 128, 64, 2048, 64, BF, True)]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,sinks,dt,inter", DECODE)
def test_decode(cuda_ok, lens, Hq, Hkv, d, page, window, sinks, dt, inter):
    gen = torch.Generator(device="cuda").manual_seed(1)
    width = -(-max(lens) // page) + 2
    table, lt, rc = _pool(lens, page, width, 3, gen)
    n_pages = rc.shape[0]
    kv = torch.full((n_pages, 2, page, Hkv, d) if inter else (2, n_pages, page, Hkv, d), float("nan"), dtype=dt,
                    device="cuda")
    kc, vc = (kv[:, 0], kv[:, 1]) if inter else (kv[0], kv[1])
    for b, n in enumerate(lens):                                        # only written slots hold numbers
        j = torch.arange(n, device="cuda")
        at = (table[b, j // page].long(), j % page)
        kc[at] = torch.randn((n, Hkv, d), generator=gen, device="cuda").to(dt)
        vc[at] = torch.randn((n, Hkv, d), generator=gen, device="cuda").to(dt)
    if window is not None:                                              # pages without a visible key are gone
        lo = torch.arange(width, device="cuda")[None] * page
        table[(lo >= sinks) & (lo + page <= (lt - window)[:, None])] = -1
    q = torch.randn((len(lens), Hq, d), generator=gen, device="cuda").to(dt)
    out, lse = api.paged_attn_decode(q, kc, vc, table, lt, window=window, sinks=sinks)
    api.check_device_status()
    assert out.dtype == dt and lse.dtype == torch.float32
    _decode_check(q, kc, vc, table, lens, page, window, sinks, out, lse)
    again = api.paged_attn_decode(q, kc, vc, table, lt, window=window, sinks=sinks)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_decode_views_scale_stream_and_graph(cuda_ok):
    gen = torch.Generator(device="cuda").manual_seed(2)
    lens, page, Hkv, d = [200, 31, 500], 16, 2, 128
    table, lt, rc = _pool(lens, page, 40, 2, gen)
    kv = torch.randn((rc.shape[0], page, 2, Hkv, d), generator=gen, device="cuda").to(BF)
    kc, vc = kv[:, :, 0], kv[:, :, 1]                                   # K and V interleaved by slot
    proj = torch.randn((3, 8 + 5, d), generator=gen, device="cuda").to(BF)
    q = proj[:, :8]
    out, lse = api.paged_attn_decode(q, kc, vc, table, lt, scale=0.3)
    _decode_check(q, kc, vc, table, lens, page, None, 0, out, lse, 0.3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = api.paged_attn_decode(q, kc, vc, table, lt, scale=0.3)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # one captured step serves any lengths
    ws = torch.empty(api.paged_attn_decode_workspace_bytes(3, 8, Hkv, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = api.paged_attn_decode(q, kc, vc, table, lt, workspace=ws)
    for new in ([200, 31, 500], [1, 0, 333], [0, 0, 0], [128, 16, 17]):
        lt.copy_(_i32(new))
        graph.replay()
        _decode_check(q, kc, vc, table, new, page, None, 0, o3, l3)
    api.check_device_status()


def test_decode_reports_bad_pages_and_lengths(cuda_ok):
    gen = torch.Generator(device="cuda").manual_seed(3)
    table, lt, rc = _pool([100], 16, 8, 0, gen)
    kc, vc = (torch.randn((rc.shape[0], 16, 1, 64), generator=gen, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((1, 4, 64), generator=gen, device="cuda").to(BF)
    for bad in (-1, rc.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out, lse = api.paged_attn_decode(q, kc, vc, t, lt)
        with pytest.raises(api.SAError):
            api.check_device_status()
        keep = torch.cat([torch.arange(32), torch.arange(48, 100)]).cuda()    # the other keys count
        pg = table[0, keep // 16].long()
        ro, rl, bo = ref.fwd(q, kc[pg, keep % 16], vc[pg, keep % 16], 83, 84, 0)
        ref.close(out, ro, bo, "out")
    for n in (-3, 129, 2 ** 31 - 1):
        api.paged_attn_decode(q, kc, vc, torch.zeros_like(table), _i32([n]))
        with pytest.raises(api.SAError):
            api.check_device_status()


def test_decode_refusals(cuda_ok):
    gen = torch.Generator(device="cuda").manual_seed(4)
    table, lt, rc = _pool([40], 16, 4, 1, gen)
    kc = torch.zeros((rc.shape[0], 16, 2, 64), dtype=BF, device="cuda")
    q = torch.zeros((1, 4, 64), dtype=BF, device="cuda")
    f = api.paged_attn_decode
    with pytest.raises(TypeError):
        f(q.float(), kc, kc, table, lt)
    with pytest.raises(TypeError):
        f(q.half(), kc, kc, table, lt)
    with pytest.raises(TypeError):
        f(q, kc, kc, table.long(), lt)
    with pytest.raises(ValueError):
        f(q, kc, kc[:1], table, lt)
    with pytest.raises(ValueError):
        f(q, kc, kc, table, lt, window=0)
    with pytest.raises(ValueError):
        f(q, kc, kc, table[:0], lt)
    with pytest.raises(ValueError):
        f(q[0], kc, kc, table, lt)
    with pytest.raises(api.SAError):
        f(q[:, :3], kc, kc, table, lt)
    with pytest.raises(api.SAError):
        f(q, kc, kc, table, lt, sinks=-1)
    with pytest.raises(api.SAError, match="workspace"):
        f(q, kc, kc, table, lt, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    out, lse = f(q[:0], kc, kc, table[:0], lt[:0])
    assert out.shape == (0, 4, 64)


# ------------------------------------------------------------------- books --
class Books:
    """The books on the host, one entry at a time."""

    def __init__(self, table, lens, rc, page):
        self.t, self.n, self.rc, self.page = table.tolist(), lens.tolist(), rc.tolist(), page

    def same(self, table, lens, rc):
        assert table.tolist() == self.t and rc.tolist() == self.rc
        assert lens is None or lens.tolist() == self.n

    def extend(self, seqs, n_new):
        free = [i for i, c in enumerate(self.rc) if c == 0]
        pos, start, served = 0, [], set()
        for s, add in zip(seqs, n_new):
            width = len(self.t[0]) * self.page
            if not 0 <= s < len(self.n) or s in served or add < 0 or self.n[s] + add > width:
                start.append(-1)
                served.add(s)
                continue
            served.add(s)
            have, want = -(-self.n[s] // self.page), -(-(self.n[s] + add) // self.page)
            got = free[pos:pos + want - have]
            pos += want - have
            if len(got) < want - have:
                start.append(-1)
                continue
            for i, g in enumerate(got):
                self.t[s][have + i] = g
                self.rc[g] = 1
            start.append(self.n[s])
            self.n[s] += add
        return start

    def fork(self, src, dst):
        free = [i for i, c in enumerate(self.rc) if c == 0]
        pos, done, moves, taken = 0, [], [], set()
        for s, d in zip(src, dst):
            S = len(self.n)
            if not (0 <= s < S and 0 <= d < S) or d in taken or d in src or s in dst or self.n[d]:
                done.append(0)
                taken.add(d)
                continue
            taken.add(d)
            full, part = divmod(self.n[s], self.page)
            if part:
                pos += 1
                if pos > len(free):
                    done.append(0)
                    continue
            row = [-1] * len(self.t[d])
            for i in range(full):
                row[i] = self.t[s][i]
                if row[i] >= 0:
                    self.rc[row[i]] += 1
            if part:
                row[full] = free[pos - 1]
                self.rc[row[full]] = 1
                moves.append((self.t[s][full], row[full]))
            self.t[d], self.n[d] = row, self.n[s]
            done.append(1)
        return done, moves

    def free(self, seqs, window=None, sinks=0):
        for s in seqs:
            for i, g in enumerate(self.t[s]):
                lo = i * self.page
                if g < 0 or window is not None and (lo < sinks or lo + self.page > self.n[s] - window):
                    continue
                self.rc[g] -= 1
                self.t[s][i] = -1
            if window is None:
                self.n[s] = 0

    def compact(self):
        live = sum(c > 0 for c in self.rc)
        src = [i for i, c in enumerate(self.rc) if c > 0 and i >= live]
        dst = [i for i, c in enumerate(self.rc) if c == 0 and i < live]
        new = dict(zip(src, dst))
        for s, d in new.items():
            self.rc[d], self.rc[s] = self.rc[s], 0
        self.t = [[new.get(g, g) for g in row] for row in self.t]
        return live, list(new.items())


def _books(lens, page, width, spare, seed, share=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table, lt, rc = _pool(lens, page, width, spare, gen, share)
    return table, lt, rc, Books(table, lt, rc, page)


@pytest.mark.parametrize("lens,page,width,spare,n_new", [
    ([0, 1, 16, 31, 32], 16, 4, 20, [1, 1, 1, 1, 0]),
    ([5] * 30, 1, 40, 3000, [7, 0, 33, 3, 50, 1] * 5),                # rows that are too short, whole pages of one token
    ([100, 200, 300], 64, 10, 3, [64, 400, 64]),                      # not enough pages for all
    ([9], 8, 4, 0, [8]),                                              # an empty pool
    ([16 * (i % 3) + 1 for i in range(5000)], 16, 5, 9000, [17] * 5000)])
def test_extend(cuda_ok, lens, page, width, spare, n_new):
    table, lt, rc, model = _books(lens, page, width, spare, 5)
    seqs = torch.randperm(len(lens), generator=torch.Generator().manual_seed(6)).tolist()
    start = api.paged_extend(table, lt, rc, _i32(seqs), _i32(n_new), page)
    api.check_device_status()
    assert start.tolist() == model.extend(seqs, n_new)
    model.same(table, lt, rc)
    start = api.paged_extend(table, lt, rc, _i32(seqs[:1]), _i32([1]), page)      # and again on what it left
    assert start.tolist() == model.extend(seqs[:1], [1])
    model.same(table, lt, rc)


def test_extend_wrong_entries(cuda_ok):
    table, lt, rc, model = _books([10, 20, 30], 8, 9, 12, 7)
    seqs, n_new = [1, 1, -1, 3, 0, 2], [9, 9, 1, 1, -2, 30]
    start = api.paged_extend(table, lt, rc, _i32(seqs), _i32(n_new), 8)
    with pytest.raises(api.SAError) as e:
        api.check_device_status()
    assert e.value.status == _lib.SA_ERR_DEVICE_ASSERT
    assert start.tolist() == model.extend(seqs, n_new) == [20, -1, -1, -1, -1, 30]
    model.same(table, lt, rc)
    assert api.paged_extend(table, lt, rc, _i32([]), _i32([]), 8).numel() == 0


@pytest.mark.parametrize("pages", [1, 31, 33, 8191, 70001])
def test_extend_takes_the_lowest_free_pages(cuda_ok, pages):
    gen = torch.Generator(device="cuda").manual_seed(pages)
    rc = (torch.rand(pages, generator=gen, device="cuda") < 0.7).to(torch.int32)
    base = torch.zeros(pages + 3, dtype=torch.int32, device="cuda")[3:]           # only 4-byte aligned
    base.copy_(rc)
    free = (rc == 0).nonzero().flatten().tolist()
    n = min(len(free), 500)
    table = torch.full((1, 600), -1, dtype=torch.int32, device="cuda")
    lt = _i32([0])
    start = api.paged_extend(table, lt, base, _i32([0]), _i32([n * 4]), 4)
    assert start.item() == 0 and table[0, :n].tolist() == free[:n] and (table[0, n:] == -1).all()
    assert base.sum().item() == int(rc.sum()) + n


@pytest.mark.parametrize("dt,d", [(BF, 128), (torch.float8_e4m3fn, 64), (torch.float32, 20)])
@pytest.mark.parametrize("packed", [False, True])
def test_write(cuda_ok, dt, d, packed):
    gen = torch.Generator(device="cuda").manual_seed(8)
    page, Hkv, lens = 8, 3, [3, 16, 0, 40]
    table, lt, rc, _ = _books([n + 30 for n in lens], page, 12, 2, 9)
    seqs, start = [3, 0, 2, 1], [40, 3, -1, 16]
    n_new = [1, 1, 1, 1] if not packed else [5, 0, 2, 17]
    N = sum(n_new) + (3 if packed else 0)
    proj = torch.randn((N, 2 * Hkv + 1, d), generator=gen, device="cuda").to(dt)
    kn, vn = proj[:, :Hkv], proj[:, Hkv + 1:]
    kv = torch.zeros((rc.shape[0], 2, page, Hkv, d), device="cuda").to(dt)
    want = kv.clone()
    off = [sum(n_new[:i]) + (1 if packed else 0) for i in range(5)]      # a row before the list belongs to nobody
    for i, s in enumerate(seqs):
        for t in range(n_new[i]):
            if start[i] >= 0:
                pos = start[i] + t
                g = int(table[s, pos // page])
                want[g, 0, pos % page], want[g, 1, pos % page] = kn[off[i] + t], vn[off[i] + t]
    api.paged_write(kn, vn, kv[:, 0], kv[:, 1], table, _i32(seqs), _i32(start), cu_new=_i32(off) if packed else None)
    api.check_device_status()
    assert torch.equal(kv.view(torch.uint8), want.view(torch.uint8))


def test_write_bad_places_and_refusals(cuda_ok):
    table, lt, rc, _ = _books([20], 8, 4, 1, 10)
    kc = torch.zeros((rc.shape[0], 8, 2, 64), dtype=BF, device="cuda")
    new = torch.ones((1, 2, 64), dtype=BF, device="cuda")
    for seq, st in ((0, 32), (0, 27), (5, 0), (-1, 0), (0, 2 ** 31 - 1)):          # past the row, no page, no sequence
        api.paged_write(new, new, kc, kc, table, _i32([seq]), _i32([st]))
        with pytest.raises(api.SAError):
            api.check_device_status()
        assert (kc == 0).all()
    with pytest.raises(ValueError):
        api.paged_write(new, new, kc, kc, table, _i32([0, 0]), _i32([0, 0]))
    with pytest.raises(TypeError):
        api.paged_write(new, new.half(), kc, kc, table, _i32([0]), _i32([0]))
    with pytest.raises(ValueError):
        api.paged_write(new, new[:, :1], kc, kc, table, _i32([0]), _i32([0]))
    with pytest.raises(ValueError):
        thin = torch.zeros((rc.shape[0], 8, 2, 4), dtype=BF, device="cuda")
        api.paged_write(thin[0, :1], thin[0, :1], thin, thin, table, _i32([0]), _i32([0]))


@pytest.mark.parametrize("n_caches,row,page", [(0, (2, 64), 16), (5, (1, 64), 16), (140, (1, 8), 4), (2, (3,), 24)])
def test_fork(cuda_ok, n_caches, row, page):
    lens = [0, 1, page, 3 * page + 5 % page, 50, 0, 0, 0, 0, 0, 0]
    table, lt, rc, model = _books(lens, page, 60, 6, 11)
    if 50 // page > 1:
        table[4, 1] = -1                                               # a trimmed middle
        model.t[4][1] = -1
    src, dst = [3, 1, 4, 2, 3, 0], [5, 6, 7, 8, 9, 10]
    caches = [torch.randn((rc.shape[0], page, *row), device="cuda").to(BF if row[-1] % 2 == 0 else torch.float32)
              for _ in range(n_caches)]
    want = [c.clone() for c in caches]
    done = api.paged_fork(table, lt, rc, _i32(src), _i32(dst), page, caches)
    api.check_device_status()
    ok, moves = model.fork(src, dst)
    assert done.tolist() == ok
    model.same(table, lt, rc)
    for s, d in moves:
        for c in want:
            c[d] = c[s]
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_fork_wrong_entries_and_an_empty_pool(cuda_ok):
    table, lt, rc, model = _books([20, 9, 16, 0, 0, 0, 0], 8, 5, 1, 12)
    src, dst = [0, 1, 2], [3, 4, 5]                                     # one fresh page for two tails
    done = api.paged_fork(table, lt, rc, _i32(src), _i32(dst), 8)
    api.check_device_status()
    assert done.tolist() == model.fork(src, dst)[0] == [1, 0, 1]
    model.same(table, lt, rc)
    src, dst = [2, 2, 2, 9, 2, 6], [6, 6, 0, 4, -1, 6]                  # twice, in use, no sequence, a src as dst
    done = api.paged_fork(table, lt, rc, _i32(src), _i32(dst), 8)
    with pytest.raises(api.SAError):
        api.check_device_status()
    assert done.tolist() == model.fork(src, dst)[0]
    model.same(table, lt, rc)


def test_free_whole_windowed_and_twice(cuda_ok):
    table, lt, rc, model = _books([100, 33, 64, 7], 8, 14, 3, 13, share=2)
    api.paged_free(table, lt, rc, _i32([0, 1]), page=8, window=20, sinks=9)
    model.free([0, 1], 20, 9)
    model.same(table, lt, rc)
    api.paged_free(table, lt, rc, _i32([1, 3, 1]))
    model.free([1, 3])
    model.same(table, lt, rc)
    api.check_device_status()
    table[2, 0], table[2, 1] = 2 ** 31 - 1, table[2, 2]                 # a page outside the pool, one held too often
    rc[int(table[2, 2])] = 1
    api.paged_free(table, lt, rc, _i32([2, 77]))
    with pytest.raises(api.SAError):
        api.check_device_status()
    assert (rc >= 0).all() and (table[2] == -1).all()
    with pytest.raises(ValueError):
        api.paged_free(table, lt, rc, _i32([0]), window=4)
    with pytest.raises(ValueError):
        api.paged_free(table, lt[:1], rc, _i32([0]))


@pytest.mark.parametrize("pages,live,page", [(1, 1, 8), (1, 0, 8), (40, 13, 8), (40, 40, 1), (9000, 2500, 4),
                                             (20011, 19000, 2)])
def test_compact(cuda_ok, pages, live, page):
    gen = torch.Generator(device="cuda").manual_seed(pages + live)
    ids = torch.randperm(pages, generator=gen, device="cuda")[:live].to(torch.int32)
    table = torch.full((3, live + 2), -1, dtype=torch.int32, device="cuda")
    table[0, :live] = ids
    table[2, 1:1 + live // 2] = ids[: live // 2]                        # shared pages
    rc = torch.zeros(pages, dtype=torch.int32, device="cuda")
    rc[ids.long()] = 1
    rc[ids[: live // 2].long()] = 2
    model = Books(table, _i32([0, 0, 0]), rc, page)
    caches = [torch.randn((pages, page, 2, 8), generator=gen, device="cuda").to(BF) for _ in range(3)]
    pair = torch.randn((pages, 2, page, 2, 8), generator=gen, device="cuda").to(BF)
    caches += [pair[:, 0], pair[:, 1]]
    want = [c.clone() for c in caches]
    n = api.paged_compact(table, rc, caches)
    api.check_device_status()
    count, moves = model.compact()
    assert n.tolist() == [count] == [live]
    model.same(table, None, rc)
    if moves:
        s, d = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for c in want:
            c[d] = c[s]
    held = rc > 0
    assert all(torch.equal(a[held], b[held]) for a, b in zip(caches, want))


def test_compact_refusals(cuda_ok):
    table, lt, rc, _ = _books([20], 8, 4, 1, 14)
    kc = torch.zeros((rc.shape[0], 8, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        api.paged_compact(table, rc, [kc[:1]])
    with pytest.raises(ValueError):
        api.paged_compact(table, rc, [kc, kc[..., :32].contiguous()])
    with pytest.raises(ValueError):
        api.paged_compact(table, rc, [kc[..., :32]])
    with pytest.raises(ValueError):
        api.paged_fork(table, lt, rc, _i32([0]), _i32([0]), 4, [kc])
    with pytest.raises(TypeError):
        api.paged_compact(table.long(), rc)


# ---------------------------------------------------------------- together --
@pytest.mark.parametrize("window,sinks", [(None, 0), (48, 5)])
def test_a_server_run(cuda_ok, window, sinks):
    """Prefill with the packed forward, its keys written to pages; forks; decode
    steps; trimming what the window has passed; a compaction between steps;
    every step against the dense form of each sequence."""
    gen = torch.Generator(device="cuda").manual_seed(20)
    page, Hq, Hkv, d, S = 16, 8, 2, 64, 8
    prompts = [70, 1, 33, 16]
    table = torch.full((S, 16), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    rc = torch.zeros(60, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((60, page, Hkv, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    N = sum(prompts)
    q = torch.randn((N, Hq, d), generator=gen, device="cuda").to(BF)
    k, v = (torch.randn((N, Hkv, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    cu = _i32([0, *torch.tensor(prompts).cumsum(0).tolist()])
    w = window if window is not None else 1000
    out, lse = api.sink_attn_fwd(q, k, v, w, sinks, cu_q=cu, cu_k=cu, max_q=max(prompts), max_k=max(prompts))
    seqs = _i32([0, 1, 2, 3])
    start = api.paged_extend(table, lens, rc, seqs, _i32(prompts), page)
    api.paged_write(k, v, kc, vc, table, seqs, start, cu_new=cu)
    hist = {s: [k[int(cu[s]):int(cu[s + 1])], v[int(cu[s]):int(cu[s + 1])]] for s in range(4)}
    # the last prompt row of the prefill equals a decode step over the pages
    last = q[(cu[1:] - 1).long()]
    o, l = api.paged_attn_decode(last, kc, vc, table[:4], lens[:4], window=window, sinks=sinks)
    for s in range(4):
        ro, rl, bo = ref.fwd(last[s:s + 1], *hist[s], prompts[s] - 1, w, sinks)
        ref.close(o[s:s + 1], ro, bo, "decode after prefill")
        ref.close(out[int(cu[s + 1]) - 1][None], ro, bo, "prefill")
    assert api.paged_fork(table, lens, rc, _i32([0, 0, 3]), _i32([4, 5, 6]), page, [kc, vc]).tolist() == [1, 1, 1]
    for s, d_ in ((0, 4), (0, 5), (3, 6)):
        hist[d_] = list(hist[s])
    alive = [0, 1, 2, 3, 4, 5, 6]
    for step in range(40):
        sq = _i32(alive)
        n = len(alive)
        kn, vn = (torch.randn((n, Hkv, d), generator=gen, device="cuda").to(BF) for _ in range(2))
        start = api.paged_extend(table, lens, rc, sq, torch.ones(n, dtype=torch.int32, device="cuda"), page)
        assert (start >= 0).all()
        api.paged_write(kn, vn, kc, vc, table, sq, start)
        for i, s in enumerate(alive):
            hist[s] = [torch.cat([hist[s][0], kn[i:i + 1]]), torch.cat([hist[s][1], vn[i:i + 1]])]
        qn = torch.randn((n, Hq, d), generator=gen, device="cuda").to(BF)
        o, l = api.paged_attn_decode(qn, kc, vc, table[sq.long()], lens[sq.long()], window=window, sinks=sinks)
        for i, s in enumerate(alive):
            m = hist[s][0].shape[0]
            ro, rl, bo = ref.fwd(qn[i:i + 1], *hist[s], m - 1, w, sinks)
            ref.close(o[i:i + 1], ro, bo, f"step {step} sequence {s}")
            ref.close_lse(l[i:i + 1], rl, "lse")
        if window is not None:
            api.paged_free(table, lens, rc, sq, page=page, window=window, sinks=sinks)
        if step == 11:
            api.paged_free(table, lens, rc, _i32([0, 2]))
            alive = [1, 3, 4, 5, 6]
        if step in (12, 30):
            n_live = api.paged_compact(table, rc, [kc, vc])
            assert (rc[: n_live.item()] > 0).all() and (rc[n_live.item():] == 0).all()
    api.check_device_status()
    api.paged_free(table, lens, rc, _i32(alive))
    assert (rc == 0).all() and (table == -1).all() and (lens == 0).all()


def test_two_captured_steps_share_a_workspace(cuda_ok):
    gen = torch.Generator(device="cuda").manual_seed(21)
    page, Hkv, d = 16, 1, 64
    table, lens, rc, model = _books([40, 7], page, 20, 30, 22)
    kc, vc = (torch.randn((rc.shape[0], page, Hkv, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((2, 4, d), generator=gen, device="cuda").to(BF)
    new = torch.randn((2, Hkv, d), generator=gen, device="cuda").to(BF)
    sq, one = _i32([0, 1]), _i32([1, 1])
    ws = torch.empty(max(api.paged_attn_decode_workspace_bytes(2, 4, Hkv, d), 1 << 20), dtype=torch.uint8,
                     device="cuda")

    def step():
        start = api.paged_extend(table, lens, rc, sq, one, page, workspace=ws)
        api.paged_write(new, new, kc, vc, table, sq, start)
        return api.paged_attn_decode(q, kc, vc, table, lens, workspace=ws)

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res))
    for i in range(30):
        g, (o, l) = graphs[i % 2]
        g.replay()
        model.extend([0, 1], [1, 1])
        model.same(table, lens, rc)
        _decode_check(q, kc, vc, table, lens.tolist(), page, None, 0, o, l)
    api.check_device_status()
