"""Workspaces of the paged entry points: their sizes, and the refusal of one
that the device cannot reach, before anything is enqueued."""
import pytest
import torch

from fixed_pattern_sparse_sa_b200 import api, build


class _OnDevice:
    """Stands for a tensor of device 0 where there is none."""
    device = torch.device("cuda", 0)


@pytest.mark.parametrize("ws", [torch.empty(1 << 16, dtype=torch.uint8), 1 << 20, b"bytes",
                                torch.empty(1 << 16, dtype=torch.uint8, device="meta")])
def test_a_workspace_off_the_device(ws):
    with pytest.raises(ValueError, match="workspace must be a tensor on cuda:0"):
        api._scratch(ws, _OnDevice, lambda: 64)


def test_a_workspace_given_and_made():
    like = torch.zeros(3, dtype=torch.int32)
    own = torch.empty(40, dtype=torch.float32)
    ws, have = api._scratch(own, like, lambda: 64)
    assert ws is own and have == 160
    ws, have = api._scratch(None, like, lambda: 64)
    assert ws.numel() * ws.element_size() == have == 64 and ws.device == like.device
    with pytest.raises(ValueError, match="contiguous"):
        api._scratch(torch.empty(8, 8)[:, ::2], like, lambda: 64)


def test_sizes():
    build.build()
    assert api.paged_books_workspace_bytes(4, 3, 100) >= (4 + 4 + 3 + 3 + 300) * 4
    assert api.paged_books_workspace_bytes(0, 0, 0) < 4096
    assert api.paged_attn_decode_workspace_bytes(4, 16, 1, 128) > 0


@pytest.mark.gpu
def test_the_calls_refuse_and_take_it(cuda_ok):
    S, page, pages = 3, 8, 20
    table = torch.full((S, 4), -1, dtype=torch.int32, device="cuda")
    lens, rc = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    kc = torch.zeros((pages, page, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((S, 4, 64), dtype=torch.bfloat16, device="cuda")
    a, b, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0], [1], [9]))
    calls = [(lambda ws: api.paged_extend(table, lens, rc, a, n, page, workspace=ws), api.paged_books_workspace_bytes(S, 1, pages)),
             (lambda ws: api.paged_fork(table, lens, rc, a, b, page, [kc], workspace=ws), api.paged_books_workspace_bytes(S, 1, pages)),
             (lambda ws: api.paged_compact(table, rc, [kc], workspace=ws), api.paged_books_workspace_bytes(S, 0, pages)),
             (lambda ws: api.paged_attn_decode(q, kc, kc, table, lens, workspace=ws),
              api.paged_attn_decode_workspace_bytes(S, 4, 1, 64))]
    for call, nbytes in calls:
        with pytest.raises(ValueError, match="workspace"):
            call(torch.empty(1 << 20, dtype=torch.uint8))
        with pytest.raises(api.SAError, match="workspace"):
            call(torch.empty(nbytes - 1, dtype=torch.uint8, device="cuda"))
        with pytest.raises(api.SAError, match="alignment"):
            call(torch.empty(nbytes + 8, dtype=torch.uint8, device="cuda")[8:])
        call(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
    api.check_device_status()
    assert lens.tolist() == [9, 9, 0]
