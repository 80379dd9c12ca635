"""Calls of host threads at once, each on its own stream with its own workspace and
outputs: every one succeeds, whatever sizes the other threads' calls have."""
import ctypes as C
import threading

import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def together(calls, times):
    """Each call (of a stream handle) `times` times by a thread of its own, on a stream of
    its own; the codes that are not TV_OK."""
    codes, start = [], threading.Barrier(len(calls))
    torch.cuda.synchronize()  # (inputs are there)

    def body(call):
        stream = torch.cuda.Stream()
        start.wait()
        for i in range(times):
            rc = call(stream.cuda_stream)
            if rc != tv.TV_OK:
                codes.append(rc)
            if i % 256 == 255:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=body, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return codes


def pointers(*tensors):
    return [C.c_void_p(t.data_ptr()) for t in tensors]


def beams(lib, logits):
    """A call on rows that are dead (little to do on the GPU, so that host calls meet)."""
    rows, vocab = logits.shape
    prm = tv.BeamParams(rows, 1, 2, vocab, 1 if logits.dtype is torch.float32 else 0, -1, 0.0, 0)
    scores = torch.full((rows,), -float("inf"), device="cuda")
    tokens, parents, status = (torch.full((rows, 2), 7, dtype=torch.int32, device="cuda") for _ in range(3))
    best = torch.zeros(rows, 2, device="cuda")
    ws = torch.empty(int(lib.tv_beam_select_workspace_size(C.byref(prm))), dtype=torch.uint8, device="cuda")
    x, s, t, p, b, st, w = pointers(logits, scores, tokens, parents, best, status, ws)
    keep = (scores, tokens, parents, best, status, ws)
    return (lambda stream: lib.tv_beam_select(C.byref(prm), x, s, None, None, t, p, b, None, None, st, w, ws.numel(),
                                              C.c_void_p(stream))), keep


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_of_less_and_more_shared_memory(dtype):
    """Rows of the largest vocabulary by one CTA each, and a few of them by several."""
    lib = ensure_built()
    logits = torch.randn(400, 262143, device="cuda", dtype=dtype)
    calls = [beams(lib, logits), beams(lib, logits[:2]), beams(lib, logits), beams(lib, logits[:2])]
    assert together([c for c, _ in calls], 3000) == []
    for _, (_, tokens, parents, best, status, _) in calls:
        assert (tokens == -1).all() and (parents == -1).all() and (best == -float("inf")).all()
        assert (status.flatten()[:status.shape[0]] == 0).all()


def pages(lib, rows, width, pool):
    """Allocations that find nothing lacking."""
    table = torch.zeros(rows, width, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    refs[0] = rows * width
    end = torch.full((rows,), 16 * width, dtype=torch.int32, device="cuda")
    status = torch.full_like(end, 7)
    prm = tv.PageParams(rows, 0, 16, width, pool, 0)
    ws = torch.empty(int(lib.tv_pages_workspace_size(C.byref(prm))), dtype=torch.uint8, device="cuda")
    t, r, e, st, w = pointers(table, refs, end, status, ws)
    return (lambda stream: lib.tv_alloc_pages(C.byref(prm), t, r, None, e, st, w, ws.numel(),
                                              C.c_void_p(stream))), (table, refs, status, end, ws)


@pytest.mark.parametrize("pool", [9000, 140000])
def test_allocations_of_many_and_of_few_rows(pool):
    lib = ensure_built()
    calls = [pages(lib, rows, 1, pool) for rows in (65536, 30000, 65536, 30000)]
    assert together([c for c, _ in calls], 2000) == []
    for _, (table, refs, status, _, _) in calls:
        assert (table == 0).all() and int(refs.sum()) == table.shape[0] and (status == 0).all()
