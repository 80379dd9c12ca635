"""GPU parity of the page calls (tv_alloc_pages, tv_free_pages, tv_fork_pages,
tv_compact_pages, tv_copy_pages) with a list-by-list model: tables, counts, copies
and statuses match exactly, whatever the sizes, and also of malformed rows."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def same(t, x):
    np.testing.assert_array_equal(t.cpu().numpy(), np.array(x, np.int32).reshape(t.shape))


def sequences(rows, width, pages, seed, fill=0.5):
    """Tables of random lengths over shuffled pages, some shared, and their counts."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, 16 * width + 1, rows)
    need = -(-lens // 16)
    while need.sum() > pages * fill:
        lens = lens * 3 // 4
        need = -(-lens // 16)
    ids = g.permutation(pages)
    table, at = [], 0
    for b in range(rows):
        row = ids[at:at + need[b]].tolist()
        if b and g.random() < 0.4:  # a prefix shared with the row before
            n = g.integers(0, min(lens[b], lens[b - 1]) // 16 + 1)
            row[:n] = table[b - 1][:n]
        at += need[b]
        table.append(row + [-1] * (width - len(row)))
    refs = [0] * pages
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return table, refs, lens.tolist(), g


def consistent(table, refs):
    t, r = table.cpu().numpy(), refs.cpu().numpy()
    want = np.bincount(t[t >= 0], minlength=len(r))
    np.testing.assert_array_equal(r, want)


SIZES = [  # rows, entries a row, pages
    (1, 1, 1), (1, 3, 5), (3, 7, 40), (16, 257, 3000), (70, 33, 1025), (5, 2100, 127), (300, 40, 9001),
    (9, 130, 100003), (1100, 9, 16384), (2500, 3, 70000),
    (40, 2500, 300001), (600, 30, 700000), (700, 500, 200000)]


@pytest.mark.parametrize("rows, width, pages", SIZES)
def test_alloc(rows, width, pages):
    ensure_built()
    for seed, fill in ((1, 0.3), (2, 0.8)):
        table, refs, lens, g = sequences(rows, width, pages, seed, fill)
        end = [int(min(16 * width, n + x)) for n, x in zip(lens, g.integers(0, 200, rows))]
        begin = [int(x) for x in np.where(g.random(rows) < 0.5, lens, 0)]
        if rows > 2:
            end[0], begin[2] = 0, 16 * width
        # holes in front, as a window leaves them
        oracle.free_pages(table[::3], refs, [n // 2 for n in lens[::3]], [16 * width] * len(lens[::3]))
        t, r = i32(table), i32(refs)
        st = tv.alloc_pages(t, r, i32(end), begin=i32(begin))
        want = oracle.alloc_pages(table, refs, begin, end)
        same(st, want)
        same(t, table)
        same(r, refs)
        st = tv.alloc_pages(t, r, i32(end))
        same(st, oracle.alloc_pages(table, refs, [0] * rows, end))
        same(t, table)
        same(r, refs)


def test_alloc_runs_out_and_malformed_rows():
    ensure_built()
    table = [[-1] * 6 for _ in range(8)]
    table[3][1] = 20           # of a pool of 20 pages
    table[5][:2] = [4, 17]
    refs = [0] * 20
    refs[4] = refs[17] = 1
    end = [90, -1, 97, 40, 96, 33, 70, 16]  # 6, bad, bad, bad, 6, 1, 5, 1 pages
    t, r = i32(table), i32(refs)
    st = tv.alloc_pages(t, r, i32(end))
    want = oracle.alloc_pages(table, refs, [0] * 8, end)
    assert want == [0, 5, 5, 5, 0, 0, 0, 7]  # 18 free: 6 + 6 + 1 + 5, and one that does not fit
    same(st, want)
    same(t, table)
    same(r, refs)
    # a row that does not fit counts all the same; an empty one behind it is served
    table, refs = [[-1] * 4, [-1] * 4, [-1] * 4, [-1] * 4], [0] * 3
    t, r = i32(table), i32(refs)
    st = tv.alloc_pages(t, r, i32([32, 33, 0, 1]))
    same(st, [0, 7, 0, 7])
    same(r, [1, 1, 0])
    begin = i32([-1, 0, 0, 0])
    same(tv.alloc_pages(t, r, i32([1, 0, 0, 1]), begin=begin), [5, 0, 0, 0])
    same(t, [[0, 1, -1, -1], [-1] * 4, [-1] * 4, [2, -1, -1, -1]])


@pytest.mark.parametrize("rows, width, pages", SIZES)
def test_free(rows, width, pages):
    ensure_built()
    table, refs, lens, g = sequences(rows, width, pages, 3)
    keep_end = [int(x) for x in g.integers(0, 16 * width + 1, rows) * (g.random(rows) < 0.7)]
    keep_begin = [int(x) for x in g.integers(0, 16 * width + 1, rows) * (g.random(rows) < 0.5)]
    for kw in (dict(keep_begin=keep_begin, sinks=20), dict(keep_end=keep_end), dict(keep_begin=keep_begin, keep_end=keep_end)):
        a, b = [list(x) for x in table], list(refs)
        t, r = i32(a), i32(b)
        st = tv.free_pages(t, r, **{k: v if k == "sinks" else i32(v) for k, v in kw.items()})
        want = oracle.free_pages(a, b, kw.get("keep_begin", [0] * rows), kw.get("keep_end", [2 ** 31 - 1] * rows), kw.get("sinks", 0))
        same(st, want)
        same(t, a)
        same(r, b)
        consistent(t, r)
    t, r = i32(table), i32(refs)
    tv.free_pages(t, r, keep_end=i32([0] * rows))
    assert (t == -1).all() and (r == 0).all()


def test_free_malformed():
    ensure_built()
    table, refs = [[0, 1, 9], [2, 10 ** 9, -5], [3, -1, 4], [3, 3, 3]], [1, 1, 1, 4, 1]
    t, r = i32(table), i32(refs)
    end = [16, 5, -1, 0]
    st = tv.free_pages(t, r, keep_end=i32(end))
    same(st, oracle.free_pages(table, refs, [0] * 4, end))
    same(st, [5, 5, 5, 0])
    same(t, [[0, -1, -1], [2, -1, -5], [3, -1, 4], [-1, -1, -1]])
    same(r, [1, 0, 1, 1, 1])
    begin = i32([0, -3, 2 ** 31 - 1, 0])
    same(tv.free_pages(t, r, keep_begin=begin, sinks=2 ** 31 - 1), [0, 5, 0, 0])
    same(r, [1, 0, 1, 1, 1])


@pytest.mark.parametrize("rows, width, pages", SIZES)
def test_fork(rows, width, pages):
    ensure_built()
    for seed in (4, 5):
        table, refs, lens, g = sequences(rows, width, pages, seed, 0.4)
        for b in range(0, rows, 3):  # pages given ahead
            oracle.alloc_pages(table[b:b + 1], refs, [0], [min(16 * width, lens[b] + 40)])
        new = int(rows * (1 if seed == 4 else 1.7)) + (seed == 5)
        parents = g.integers(0, rows, new)
        parents = np.where(g.random(new) < 0.1, -1, np.where(g.random(new) < 0.5, np.arange(new) % rows, parents)).tolist()
        t, r = i32(table), i32(refs)
        out, ends, copies, st = tv.fork_pages(t, i32(lens), i32(parents), r)
        want = oracle.fork_pages(table, lens, parents, refs)
        same(t, table)
        same(out, want[0])
        same(ends, want[1])
        same(copies, want[2])
        same(st, want[3])
        same(r, refs)
        consistent(out, r)


def test_fork_runs_out_and_malformed_rows():
    ensure_built()
    #        full, part     shared part    too long  spare pages    bad entry, bad spare    no page  no count
    table = [[0, 1, -1, -1], [2, 3, -1, -1], [4, 1, -1, -1], [5, 6, 7, 8], [9, 30, 11, -1], [12, -1, -1, -1], [13, 14, -1, -1]]
    lens = [20, 32, 20, 17, 33, 17, 20]
    refs = [1, 2, 1, 1, 1, 1, 1, 1, 1, 1, 0, 1, 1, 1, 0, 0, 0, 0]
    for free in (4, 1, 0):
        a = list(refs)
        for p in range(14 + free, 18):
            a[p] = 3  # the caller's own
        a[10] = 3 if free < 4 else 0
        for parents in ([0, 0, 1, 2, 3, 3, 4, 5, 6, 7, -2, -1], [3, 3, 3], [0], [2, 0, 0], [4, 4], [-1], [1] * 30, [6, 5, 0, 1, 2, 3, 4]):
            b, rows = list(a), [list(x) for x in table]
            t, r = i32(rows), i32(b)
            out, ends, copies, st = tv.fork_pages(t, i32(lens), i32(parents), r)
            want = oracle.fork_pages(rows, lens, parents, b)
            same(out, want[0])
            same(ends, want[1])
            same(copies, want[2])
            same(st, want[3])
            same(r, b)
    lens = [65, -1, 64, 0, 0, 0, 0]
    t, r = i32(table), i32(refs)
    out, ends, copies, st = tv.fork_pages(t, i32(lens), i32([0, 1, 3, 3]), r)
    same(st, [5, 5, 0, 0])
    same(out, [[-1] * 4, [-1] * 4, [5, 6, 7, 8], [-1] * 4])
    same(ends, [0, 0, 0, 0])


@pytest.mark.parametrize("rows, width, pages", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(rows, width, pages, in_place):
    ensure_built()
    for seed, fill in ((6, 0.2), (7, 0.5), (8, 0.95)):
        table, refs, lens, g = sequences(rows, width, pages, seed, fill)
        for p in g.integers(0, pages, 3):
            refs[p] += 5  # pages that the caller holds
        t, r = i32(table), i32(refs)
        moves = torch.full((max(1, pages // 2), 3), -77, dtype=torch.int32, device="cuda")
        kw = dict(block_table_out=t, ref_counts_out=r) if in_place else {}
        got = tv.compact_pages(t, r, moves=moves, **kw)
        new, counts, to, want_moves, n, status = oracle.compact_pages(table, refs)
        if not in_place:
            same(t, table)
            same(r, refs)
        same(got["block_table"], new)
        same(got["ref_counts"], counts)
        same(got["page_map"], to)
        same(got["count"], [n, len(want_moves)])
        same(got["moves"][:len(want_moves)], want_moves)
        assert (got["moves"][len(want_moves):] == -77).all()
        same(got["status"], status)


def test_compact_full_empty_and_malformed():
    ensure_built()
    table = [[3, 7, -9], [8, 2, 9], [5, -1, -1]]
    refs = [0, 0, 1, 1, 0, 0, 0, 1]
    got = tv.compact_pages(i32(table), i32(refs))
    same(got["status"], [0, 5, 5])
    same(got["block_table"], [[0, 1, -1], [-1, 2, -1], [-1, -1, -1]])
    same(got["count"], [3, 2])
    same(got["moves"][:2], [[3, 0, 16], [7, 1, 16]])
    same(got["page_map"], oracle.compact_pages(table, refs)[2])
    for refs in ([1] * 37, [0] * 37, [0] * 36 + [1], [1] + [0] * 36):
        got = tv.compact_pages(i32([[-1] * 5] * 2), i32(refs))
        want = oracle.compact_pages([[-1] * 5] * 2, refs)
        same(got["ref_counts"], want[1])
        same(got["page_map"], want[2])
        same(got["count"], [want[4], len(want[3])])
        same(got["moves"][:len(want[3])], want[3])


COPIES = [  # layers, pages, heads, D, fp8
    (1, 9, 1, 64, False), (1, 40, 8, 128, False), (3, 40, 5, 128, True), (2, 33, 4, 64, True), (1, 300, 3, 128, False)]


@pytest.mark.parametrize("layers, pages, heads, d, fp8", COPIES)
def test_copy(layers, pages, heads, d, fp8):
    ensure_built()
    g = np.random.default_rng(pages)
    shape = (layers, pages, heads, 16, d)
    ids = g.permutation(pages)
    n = pages // 2
    copies = np.stack([ids[:n], ids[n:2 * n], g.integers(0, 17, n)], 1).astype(np.int32)
    copies[0], copies[1, 2], copies[2, 1] = (-1, -1, 0), 16, copies[2, 0]
    status = np.zeros(n, np.int32)
    for i, bad in ((3, (pages, copies[3, 1], 4)), (-1, (copies[-1, 0], copies[-1, 1], 17)), (-2, (copies[-2, 0], -1, 3)) if n > 6 else (3, (pages, copies[3, 1], 4))):
        copies[i] = bad
        status[i] = 7
    pool = [torch.randint(0, 120, shape, dtype=torch.uint8).cuda() if fp8 else torch.randn(shape).to(torch.bfloat16).cuda() for _ in range(2)]
    scale = [torch.rand(shape[:4]).cuda() for _ in range(2)] if fp8 else []
    for count in (None, n // 2, 0, n + 100, -3):
        done = n if count is None else min(max(count, 0), n)
        want = [x.cpu().clone() for x in pool + scale]
        for i, (s, t, k) in enumerate(copies.tolist()):
            if i < done and status[i] == 0 and s >= 0:
                for x in want:
                    x[:, t, :, :k] = x[:, s, :, :k]
        have = [x.clone() for x in pool + scale]
        args = have if layers > 1 else [x[0] for x in have]
        st = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        tv.copy_pages(i32(copies), *args, status=st, count=None if count is None else i32([count]))
        same(st, np.where(np.arange(n) < done, status, -7))
        for x, y in zip(have, want):
            assert torch.equal(x.cpu(), y)


def test_copy_past_32_bits():
    """Pages whose bytes lie past 2^32 of the pool's start."""
    ensure_built()
    pages = (1 << 32) // (8 * 16 * 128 * 2) + 40
    k = torch.zeros(1, pages, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, pages - 1], v[0, 3] = 2.0, 3.0
    tv.copy_pages(i32([[pages - 1, 0, 5], [3, pages - 2, 16]]), k, v)
    assert (k[0, 0, :, :5] == 2).all() and (k[0, 0, :, 5:] == 0).all() and (v[0, pages - 2] == 3).all()
    assert (k[0, pages - 2] == 0).all() and (v[0, 0] == 0).all()


def test_streams_and_graphs():
    """A beam step captured and replayed; two graphs with workspaces of their own."""
    ensure_built()
    table, refs, lens, g = sequences(12, 9, 400, 11)
    parents = [0, 0, 0, 3, 3, 5, 6, 6, 8, 9, 9, 9]
    t, r, ln, pa = i32(table), i32(refs), i32(lens), i32(parents)
    k = torch.randn(400, 2, 16, 64, device="cuda").to(torch.bfloat16)
    v = k.clone()
    out, ends, copies, st = torch.zeros_like(t), torch.zeros_like(ln), torch.zeros(12, 3, dtype=torch.int32, device="cuda"), torch.zeros_like(ln)
    ws = [torch.full((tv.page_workspace_size(t, r, new_rows=12),), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    start = r.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, w in zip(graphs, ws):
        with torch.cuda.graph(graph):
            tv.fork_pages(t, ln, pa, r, block_table_out=out, seq_lens_out=ends, copies=copies, status=st, workspace=w)
            tv.copy_pages(copies, k, v, status=st)
            tv.free_pages(out, r, keep_end=ends, status=st)
    want = oracle.fork_pages(table, lens, parents, list(refs))
    for graph in graphs + graphs:
        r.copy_(start)
        out.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        same(copies, want[2])
        same(ends, want[1])
        consistent(out, r)
        for s, d, n in want[2]:
            if s >= 0:
                assert torch.equal(k[d, :, :n], k[s, :, :n]) and torch.equal(v[d, :, :n], v[s, :, :n])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.copy_(start)
    got = tv.compact_pages(t, r, stream=s)
    st2 = tv.alloc_pages(got["block_table"], got["ref_counts"], ln, stream=s)
    s.synchronize()
    assert (st2 == 0).all()
    same(got["block_table"], oracle.compact_pages(table, refs)[0])


@pytest.mark.parametrize("held, full", [(90000, False), (180000, True)])
def test_a_large_pool_call_behind_call_in_graphs(held, full):
    """Allocations and releases of a pool that the whole GPU surveys, captured and
    replayed: malformed rows, and a pool that runs out."""
    ensure_built()
    pages, rows, width = 200003, 90, 1300
    table, refs, lens, g = sequences(rows, width, pages, 21, 0.4)
    for p in g.permutation(pages)[:held].tolist():  # the caller's own references
        refs[p] += 1
    table[7][2] = pages                             # names nothing
    ends = [[int(x) for x in g.integers(0, 16 * width + 1, rows)] for _ in range(2)]
    ends[0][5], ends[1][11] = -1, 16 * width + 1
    keep = [int(x) for x in g.integers(0, 16 * width + 1, rows)]
    t0, r0 = i32(table), i32(refs)
    t, r, e, kp = t0.clone(), r0.clone(), [i32(x) for x in ends], i32(keep)
    st = [torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(3)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    ws = [torch.full((tv.page_workspace_size(t, r),), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for graph, w in zip(graphs, ws):
        with torch.cuda.graph(graph):
            tv.alloc_pages(t, r, e[0], status=st[0], workspace=w)
            tv.free_pages(t, r, keep_end=kp, status=st[1])
            tv.alloc_pages(t, r, e[1], status=st[2], workspace=w)
    want = [oracle.alloc_pages(table, refs, [0] * rows, ends[0]), oracle.free_pages(table, refs, [0] * rows, keep),
            oracle.alloc_pages(table, refs, [0] * rows, ends[1])]
    assert 0 in want[0] and 5 in want[0] and (7 in want[0]) == full
    for graph in graphs + graphs:
        t.copy_(t0)
        r.copy_(r0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(st, want):
            same(x, y)
        same(t, table)
        same(r, refs)


def test_a_large_pool_of_many_rows_and_of_long_ones():
    ensure_built()
    rows = 65536
    t = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    r = torch.zeros(2 * rows, dtype=torch.int32, device="cuda")
    n = torch.full((rows,), 17, dtype=torch.int32, device="cuda")
    assert (tv.alloc_pages(t, r, n) == 0).all() and (r == 1).all()
    assert torch.equal(t.view(-1), torch.arange(2 * rows, dtype=torch.int32, device="cuda"))
    t = torch.full((2, 70000), -1, dtype=torch.int32, device="cuda")
    t[0, ::3] = 140000
    r = torch.zeros(140001, dtype=torch.int32, device="cuda")
    r[140000] = 1
    st = tv.alloc_pages(t, r, i32([16 * 70000, 16 * 70000]))
    assert (st == 0).all() and (r[:116666] == 1).all() and (r[116666:140000] == 0).all()
    mine = torch.ones(70000, dtype=torch.bool, device="cuda")
    mine[::3] = False
    assert torch.equal(torch.cat([t[0][mine], t[1]]), torch.arange(116666, dtype=torch.int32, device="cuda"))


def test_limits():
    ensure_built()
    for call in (lambda t, r, w: tv.alloc_pages(t, r, i32([5]), workspace=w),
                 lambda t, r, w: tv.fork_pages(t, i32([5]), i32([0]), r, workspace=w)):
        t, r = i32([[-1, -1]]), i32([0] * 100)
        with pytest.raises(tv.TVError):
            call(t, r, torch.empty(256, dtype=torch.uint8, device="cuda"))
    t, r = i32([[0, 1]]), i32([1, 1])
    with pytest.raises(tv.TVError):  # a fork needs other rows than its own
        tv.fork_pages(t, i32([5]), i32([0]), r, block_table_out=t)
    rows = 65536
    t, r = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows - 5, dtype=torch.int32, device="cuda")
    st = tv.alloc_pages(t, r, torch.full((rows,), 7, dtype=torch.int32, device="cuda"))
    assert (st[:-5] == 0).all() and (st[-5:] == 7).all() and (r == 1).all()
    assert torch.equal(t[:-5, 0], torch.arange(rows - 5, dtype=torch.int32, device="cuda")) and (t[-5:] == -1).all()
    out, ends, copies, st = tv.fork_pages(t, torch.full((rows,), 16, dtype=torch.int32, device="cuda"),
                                          torch.arange(rows, dtype=torch.int32, device="cuda").flip(0), r)
    assert torch.equal(out, t.flip(0)) and (r == 1).all() and (copies[:, :2] == -1).all() and (st == 0).all()
    with pytest.raises(tv.TVError):
        tv.alloc_pages(torch.cat([t, t]), r, torch.zeros(2 * rows, dtype=torch.int32, device="cuda"))
