"""Fields of tv_page_params: what a call does not use may hold anything, the
result is the same; and which pages `sinks` keeps."""
import ctypes as C

import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def pointers(*tensors):
    return [C.c_void_p(t.data_ptr()) for t in tensors]


@pytest.mark.parametrize("new_rows, sinks", [(2000, 0), (2 ** 31 - 1, -1), (-5, 7)])
def test_allocation_and_compaction(new_rows, sinks):
    lib = ensure_built()
    results = []
    for n, k in ((0, 0), (new_rows, sinks)):
        prm = tv.PageParams(3, n, 16, 5, 40, k)
        table = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
        table[1, 0], table[2, 1] = 7, 39
        refs = torch.zeros(40, dtype=torch.int32, device="cuda")
        refs[7], refs[39] = 1, 2
        end = torch.tensor([20, 70, 0], dtype=torch.int32, device="cuda")
        status, out, counts = torch.full_like(end, 9), torch.empty_like(table), torch.empty_like(refs)
        to, moves, count = torch.empty_like(refs), torch.zeros(20, 3, dtype=torch.int32, device="cuda"), torch.empty_like(end[:2])
        ws = torch.empty(int(lib.tv_pages_workspace_size(C.byref(prm))), dtype=torch.uint8, device="cuda")
        t, r, e, s, o, c, p, m, x, w = pointers(table, refs, end, status, out, counts, to, moves, count, ws)
        stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert lib.tv_alloc_pages(C.byref(prm), t, r, None, e, s, w, ws.numel(), stream) == tv.TV_OK
        assert lib.tv_compact_pages(C.byref(prm), t, r, o, c, p, m, x, s, stream) == tv.TV_OK
        results.append([y.tolist() for y in (table, refs, status, out, counts, to, moves, count[:2])])
    assert results[0] == results[1]


def test_sinks_stay_below_the_kept_tokens_only():
    """The first tokens' pages stay when a window moves on, and go with an ended row."""
    ensure_built()
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    refs = torch.ones(12, dtype=torch.int32, device="cuda")
    begin, end = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([33, 64, 0], [64, 0, 16]))
    status = tv.free_pages(table, refs, keep_begin=begin, keep_end=end, sinks=20)
    assert status.tolist() == [0, 0, 0]
    assert table.tolist() == [[0, 1, 2, 3], [-1] * 4, [8, -1, -1, -1]]
    assert refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0, 1, 0, 0, 0]
