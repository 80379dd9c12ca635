"""The order that a fork and a compaction ask for: their copies first, then the calls that
give out or write pages.  The copies' sources may be free by then: an allocation behind
the copies takes them, and what is written there leaves the copied rows alone."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def pools(pages, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(2, pages, 3, 16, 64, device="cuda", generator=g).to(torch.bfloat16)
    return k, -k


def rows_of(pool, row, tokens):
    """The first `tokens` cached rows of a sequence, [layers, heads, tokens, D]."""
    got = pool[:, row[:-(-tokens // 16)]]
    return got.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :tokens]


@pytest.mark.parametrize("parents", [[0, 1], [0, -1], [-1, 1], [1, 0], [0, 1, 1, 0]])
def test_rows_that_share_a_half_filled_page(parents):
    """Two rows that share a full page and the first 7 tokens of the next one."""
    ensure_built()
    table, refs, lens = [[2, 0, -1, -1], [2, 0, -1, -1]], [0] * 9, [23, 23]
    refs[2] = refs[0] = 2
    k, v = pools(9, 1)
    want = [x[:, :, :23].clone() for x in (rows_of(k, [2, 0], 23), rows_of(v, [2, 0], 23))]
    t, r = i32(table), i32(refs)
    out, ends, copies, st = tv.fork_pages(t, i32(lens), i32(parents), r)
    new, _, cp, _ = oracle.fork_pages(table, lens, parents, refs)
    assert (st == 0).all() and copies.tolist() == [list(c) for c in cp] and r.tolist() == refs
    assert refs[0] == 0  # every sharer has its own page now, or none
    tv.copy_pages(copies, k, v)
    # the next pages go to everybody, the shared one among them, and are written over
    st = tv.alloc_pages(out, r, i32([16 * 3 if p >= 0 else 0 for p in parents]))
    given = [e for a, b in zip(out.tolist(), new) for e, old in zip(a, b) if e >= 0 and old < 0]
    assert (st == 0).all() and 0 in given  # (the lowest free one)
    k[:, given] = 77.0
    v[:, given] = 78.0
    for row, p, n in zip(out.tolist(), parents, ends.tolist()):
        assert n == (23 if p >= 0 else 0)
        if p >= 0:
            assert torch.equal(rows_of(k, row, 23), want[0]) and torch.equal(rows_of(v, row, 23), want[1])


def test_sources_of_a_compaction_are_given_out_behind_its_copies():
    ensure_built()
    table, refs = [[8, 1, -1], [5, 7, -1]], [0, 1, 0, 0, 0, 1, 0, 1, 1]
    k, v = pools(9, 2)
    want = [[rows_of(x, row[:2], 32).clone() for x in (k, v)] for row in table]
    r = tv.compact_pages(i32(table), i32(refs))
    tv.copy_pages(r["moves"], k, v, count=r["count"][1:])
    out = r["block_table"]
    st = tv.alloc_pages(out, r["ref_counts"], i32([48, 48]))
    given = [row[2] for row in out.tolist()]
    assert (st == 0).all() and given == [4, 5]  # (5 was a source)
    k[:, given] = 77.0
    v[:, given] = 78.0
    for row, (a, b) in zip(out.tolist(), want):
        assert torch.equal(rows_of(k, row[:2], 32), a) and torch.equal(rows_of(v, row[:2], 32), b)
