"""GPU tests of the page operations on pools that are asked for more than they
hold, and on tables that name pages outside the pool, against the plain model
of the books."""
import pytest
import torch

from fixed_pattern_sparse_sa_b200 import _lib, api
from test_gpu_paged import BF, _books, _i32

pytestmark = pytest.mark.gpu


def _equal(got, want, what):
    """Lists of thousands of entries, compared without a report of all of them."""
    bad = [i for i, (a, b) in enumerate(zip(got, want)) if a != b]
    n = len(bad) + abs(len(got) - len(want))
    assert n == 0, f"{what}: {n} of {len(want)} differ, first {[(i, got[i], want[i]) for i in bad[:3]]}"


def _same(model, table, lt, rc):
    _equal(rc.tolist(), model.rc, "refcount")
    _equal(lt.tolist(), model.n, "seq_lens")
    _equal(table.tolist(), model.t, "block_table")


def _extend(table, lt, rc, model, seqs, n_new, page):
    start = api.paged_extend(table, lt, rc, _i32(seqs), _i32(n_new), page)
    api.check_device_status()
    _equal(start.tolist(), model.extend(seqs, n_new), "start")
    _same(model, table, lt, rc)


@pytest.mark.parametrize("lens,page,spare,n_new", [
    ([0, 0, 0], 1, 4, [3, 3, 3]),                                 # 9 pages of a pool of 4
    ([1, 1, 0, 0, 0, 0, 0, 0], 1, 2, [0, 0, 1, 1, 1, 1, 1, 1]),   # 2 free pages of 4 for six entries
    ([0] * 64, 16, 1000, [640] * 64),                             # 64 prompts of 40 pages, a pool of 1000
    ([5] * 8, 8, 0, [3, 2, 4, 0, 12, 1, 30, 3]),                  # no free page; entries that need none are served
    ([7, 8, 0, 16] * 6, 8, 3, [1, 1, 40, 0] * 6),                 # both kinds in turn, past the pool's size
    ([0] * 5000, 4, 3000, [9, 0, 4, 1, 0] * 1000),                # a list longer than what shared memory holds
    ([3] * 5000, 4, 3000, [1, 6, 1, 14, 2] * 1000)])
def test_extend_asks_for_more_than_the_pool(cuda_ok, lens, page, spare, n_new):
    table, lt, rc, model = _books(lens, page, max(-(-(a + b) // page) for a, b in zip(lens, n_new)) + 1, spare, 31)
    seqs = list(range(len(lens)))
    _extend(table, lt, rc, model, seqs, n_new, page)
    _extend(table, lt, rc, model, seqs[::-1], [1] * len(seqs), page)      # and on what that left
    _extend(table, lt, rc, model, seqs, [page] * len(seqs), page)


@pytest.mark.parametrize("tails,whole,spare", [(1, 0, 1), (9, 4, 3), (40, 7, 0), (40, 7, 2), (4500, 600, 11),
                                               (4500, 600, 5000)])
def test_fork_asks_for_more_than_the_pool(cuda_ok, tails, whole, spare):
    page, lens = 4, [6, 8, 3]                                     # a tail behind a full page, two full pages, a tail alone
    n = tails + whole
    table, lt, rc, model = _books(lens + [0] * n, page, 4, spare, 32)
    src = [1 if i % (n // whole) == 1 else 2 * (i % 2) for i in range(n)] if whole else [0] * n
    dst = list(range(3, 3 + n))
    cache = torch.randn((rc.shape[0], page, 8), device="cuda").to(BF)
    want = cache.clone()
    done = api.paged_fork(table, lt, rc, _i32(src), _i32(dst), page, [cache])
    api.check_device_status()
    ok, moves = model.fork(src, dst)
    _equal(done.tolist(), ok, "done")
    _same(model, table, lt, rc)
    if moves:
        s, d = (torch.tensor(x, device="cuda") for x in zip(*moves))
        want[d] = want[s]
    assert torch.equal(cache, want)


@pytest.mark.parametrize("at", [0, 1, 70, 71])                       # the last one: the partly filled page
@pytest.mark.parametrize("bad", [0, 5, 2 ** 31 - 1])
def test_fork_of_a_row_that_names_a_page_outside_the_pool(cuda_ok, at, bad):
    # the entry is refused as a whole: its row, length, counts and pages stay, and its page goes to no other
    page, lens = 4, [70 * 4 + 7, 9, 6, 0, 0, 0, 0]
    table, lt, rc, model = _books(lens, page, 80, 3, 33)
    bad = min(rc.shape[0] + bad, 2 ** 31 - 1)
    table[0, at] = model.t[0][at] = bad
    cache = torch.randn((rc.shape[0], page, 8), device="cuda").to(BF)
    want = cache.clone()
    src, dst = [1, 0, 2, 0], [3, 4, 5, 6]
    done = api.paged_fork(table, lt, rc, _i32(src), _i32(dst), page, [cache])
    with pytest.raises(api.SAError) as e:
        api.check_device_status()
    assert e.value.status == _lib.SA_ERR_DEVICE_ASSERT
    ok, moves = model.fork([1, 2], [3, 5])
    assert ok == [1, 1] and done.tolist() == [1, 0, 1, 0]
    _same(model, table, lt, rc)
    for s, d in moves:
        want[d] = want[s]
    assert torch.equal(cache, want)


def test_an_empty_pool_with_caches(cuda_ok):
    page = 8
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lt, rc = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    caches = [torch.zeros((0, page, 2, 64), dtype=BF, device="cuda") for _ in range(2)]
    assert api.paged_compact(table, rc, caches).tolist() == [0]
    assert api.paged_fork(table, lt, rc, _i32([0]), _i32([1]), page, caches).tolist() == [1]     # nothing of nothing
    assert api.paged_extend(table, lt, rc, _i32([0, 2]), _i32([1, 0]), page).tolist() == [-1, 0]
    api.check_device_status()
    assert (table == -1).all() and (lt == 0).all()
