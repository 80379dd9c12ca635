"""What the chunk attention, the cache calls and the logit penalties make of
malformed batches: which sequences fail, which rows are written and which stay."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from test_gpu_chunk import U_BF16, U_FP8, call, call_fp8, check, make, quantised
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

BAD_TREE = 5
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("total", [3, 40, 40000])
@pytest.mark.parametrize("at, value", [(0, LOW), (0, LOW + 5), (1, LOW), (2, LOW), (2, HIGH), (1, HIGH), (0, HIGH)])
def test_cache_offsets_at_the_ends_of_32_bits(total, at, value):
    """Every sequence fails, nothing is written, whichever CTA meets the offset
    (a CTA's tile starts at 0, 1 or up to 32 tokens on)."""
    ensure_built()
    off = np.array([0, total // 2, total], np.int64)
    off[at] = value
    blocks = 2 * (-(-total // 16)) + 1
    table = i32(np.arange(blocks - 1).reshape(2, -1))
    x = torch.randn(total, 1, 64, device="cuda").to(torch.bfloat16)
    wide = torch.full((blocks, 1, 16, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((blocks, 1, 16, 64), 7, dtype=torch.uint8, device="cuda")
    scale = torch.full((blocks, 1, 16), 3.0, device="cuda")
    at_ = (table, i32([total // 2, total - total // 2]), i32(off))
    out = torch.full((total, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    for st in (tv.append_kv(x, x, *at_, wide, wide), tv.append_kv_fp8(x, x, *at_, codes, scale, codes, scale),
               tv.read_kv_fp8(codes, scale, codes, scale, *at_, k_out=out, v_out=out)[2]):
        assert st.tolist() == [BAD_TREE, BAD_TREE]
    assert (wide == 2.0).all() and (codes == 7).all() and (scale == 3.0).all() and (out == 5.0).all()


@pytest.mark.parametrize("length", [LOW, -1, HIGH])
def test_cache_lengths_at_the_ends_of_32_bits(length):
    """A length below the chunk is malformed, one past the table has no page;
    the other sequence is served."""
    ensure_built()
    x = torch.randn(40, 1, 64, device="cuda").to(torch.bfloat16)
    pool = torch.zeros(9, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    st = tv.append_kv(x, x, i32(np.arange(8).reshape(2, 4)), i32([length, 20]), i32([0, 20, 40]), pool, pool.clone())
    assert st.tolist() == [7 if length == HIGH else BAD_TREE, 0]
    assert (pool[:4] == 0).all() and torch.equal(pool[4, 0], x[20:36, 0])


# ------------------------------------------------------------------ penalties
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_penalties_behind_decreasing_offsets(in_place, dtype):
    """Trees behind a negative one are malformed; rows that they share with a
    sound tree are penalised once, by that tree, and the others stay."""
    if in_place and dtype is torch.bfloat16:
        return
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(20, 5000, device="cuda", generator=g) * 3).to(dtype)
    history = torch.randint(0, 5000, (400,), device="cuda", generator=g, dtype=torch.int32)
    tokens = torch.randint(0, 5000, (20,), device="cuda", generator=g, dtype=torch.int32)
    parent = i32([-1] + list(range(9)) + [-1] + list(range(9)))
    kw = dict(max_nodes=20, history=history, repetition=torch.tensor([1.5, 1.2, 3.0, 0.5, 2.0], device="cuda"))
    # rows of (first sound trees, then the decrease): 0..9 | 10..4 | 5..14, 15..17, 18..19
    for off, first in (([0, 10, 5, 15, 18, 20], 10), ([0, 10, LOW, 3, 12, 20], 10), ([0, 10, 9, 10, 15, 15], 10)):
        kw["history_offsets"] = i32([0, 80, 160, 240, 320, 400])
        par = parent.clone()
        one, st = tv.penalize_logits(x, tokens, par, i32([0, 10]), max_nodes=20, history=history,
                                     history_offsets=i32([0, 80]), repetition=kw["repetition"][:1])
        assert st.tolist() == [0]
        buf = x.clone()
        out = buf if in_place else torch.full((20, 5000), 7.0, device="cuda")
        got, st = tv.penalize_logits(buf, tokens, par, i32(off), out=out, **kw)
        assert st.tolist() == [0] + [BAD_TREE] * 4, off
        assert torch.equal(got[:first], one[:first])
        kept = x.float()[first:]
        # rows of a malformed tree hold their logits, rows of none what they held
        last = max(off[2:])
        assert torch.equal(got[first:last], kept[:last - first])
        assert in_place or (got[last:] == 7.0).all()
        if off[-1] == 20 and off[1] == 10 and off[2] == 5:
            assert last == 20


def test_penalties_of_many_trees():
    """More trees than a block has threads, and a decrease far down the batch."""
    ensure_built()
    B = 1500
    x = torch.randn(B, 40, device="cuda")
    tokens, parent = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    kw = dict(max_nodes=1, history=torch.arange(B, dtype=torch.int32, device="cuda") % 40,
              history_offsets=i32(np.arange(B + 1)), presence=torch.ones(B, device="cuda"))
    want, st = tv.penalize_logits(x, tokens, parent, i32(np.arange(B + 1)), **kw)
    hit = torch.zeros(B, 40, device="cuda")
    hit[torch.arange(B), torch.arange(B) % 40] = 1.0
    assert (st == 0).all() and torch.equal(want, x - hit)
    off = np.arange(B + 1)
    off[1301:] -= 2  # tree 1300 has -1 nodes; the trees behind it share rows 1299 and on
    got, st = tv.penalize_logits(x, tokens, parent, i32(off), out=torch.full_like(x, 9.0), **kw)
    assert (st[:1300] == 0).all() and (st[1300:] == BAD_TREE).all()
    assert torch.equal(got[:1300], want[:1300]) and torch.equal(got[1300:B - 2], x[1300:B - 2]) and (got[B - 2:] == 9.0).all()


@pytest.mark.parametrize("off, bad", [([0, 0, 0], []), ([0, 5, 5], [0, 1]), ([0, 0, 1], [1]), ([-1, 0, 0], [0]),
                                      ([2, 1, 1], [0, 1]), ([1, 1, 1], [0, 1])])
@pytest.mark.parametrize("what", ["history", "bias"])
def test_penalty_extents_of_an_empty_list(off, bad, what):
    """A list without entries has extents too: one outside [0, 0] is malformed."""
    ensure_built()
    x = torch.randn(4, 100, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    kw = dict(history=none, history_offsets=i32(off)) if what == "history" else \
        dict(bias_ids=none, bias_values=none.float(), bias_offsets=i32(off))
    got, st = tv.penalize_logits(x, i32([3, 7, 3, 9]), i32([-1, 0, -1, 0]), i32([0, 2, 4]), max_nodes=2,
                                 presence=torch.ones(2, device="cuda"), **kw)
    assert st.tolist() == [BAD_TREE if b in bad else 0 for b in range(2)]
    want = x.clone()
    for b, (row, token) in enumerate(((1, 7), (3, 9))):
        if b not in bad:
            want[row, token] -= 1.0
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [64, 5001])
@pytest.mark.parametrize("off, bad, kept", [
    ([0, 10, 15, 30], [2], (15, 20)),       # rows past the last: those that are there
    ([0, 10, 15, HIGH], [2], (15, 20)),
    ([-4, 10, 15, 20], [0], (0, 10)),       # rows before the first
    ([LOW, 10, 15, 20], [0], (0, 10)),
    ([0, 10, 25, 30], [1, 2], (10, 20)),    # one past the last row, one wholly behind it
    ([0, 10, 10, 20], [1], (0, 0)),         # a tree without nodes
    ([HIGH, HIGH, HIGH, HIGH], [0, 1, 2], (0, 0)),
    ([0, 10, 30, 20], [1, 2], (10, 20)),    # past the last row, and a decrease behind it
])
def test_penalties_of_rows_outside_the_logits(off, bad, kept, vocab, dtype):
    """Of a malformed tree the rows that are there keep their logits; rows of no
    tree keep what the output held."""
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(20, vocab, device="cuda", generator=g).to(dtype)
    tokens = torch.randint(0, vocab, (20,), device="cuda", generator=g, dtype=torch.int32)
    parent = torch.full((20,), -1, dtype=torch.int32, device="cuda")
    for b in range(3):
        if b not in bad:
            n = off[b + 1] - off[b]
            parent[off[b]:off[b + 1]] = i32([-1] + list(range(n - 1)))
    out, st = tv.penalize_logits(x, tokens, parent, i32(off), max_nodes=20, presence=torch.ones(3, device="cuda"),
                                 out=torch.full((20, vocab), 7.0, device="cuda"))
    assert st.tolist() == [BAD_TREE if b in bad else 0 for b in range(3)]
    want = torch.full((20, vocab), 7.0, device="cuda")
    want[kept[0]:kept[1]] = x.float()[kept[0]:kept[1]]
    for b in set(range(3)) - set(bad):
        want[off[b]:off[b + 1]] = x.float()[off[b]:off[b + 1]]
        for r in range(off[b], off[b + 1]):
            seen = tokens[off[b] + 1:r + 1].long().unique()
            want[r, seen] -= 1.0
    assert torch.equal(out, want)


# ------------------------------------------------------------------ chunk attention
def check_all_but(got, good, c, zero, fp8, window, sinks):
    """The rows of sequences `zero` are zeros.  The others are theirs: within the
    tolerance, not bit for bit, because they are split otherwise where the work of
    a sequence goes."""
    got = got.copy()
    for b in zero:
        rows = slice(int(c["off"][b]), int(c["off"][b + 1]))
        assert (got[rows] == 0).all(), b
        got[rows] = good[rows]
    check(got, c, U_FP8 if fp8 else U_BF16, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [0, 3, 1000, -1])
def test_chunk_bad_page_of_a_split_unit(fp8, page):
    """A decode token's cache is shared out over many CTAs; one of them meets the
    bad page and all of the sequence's rows are zeros, each time."""
    c = make([16411, 700, 5], [1, 1, 1], 8, 2, 128, seed=4)
    run = call_fp8 if fp8 else call
    c = quantised(c) if fp8 else c
    good, st = run(c)
    assert (st == 0).all()
    bad = dict(c, table=c["table"].copy())
    bad["table"][0, page if page >= 0 else (16411 - 1) // 16] = c["k"].shape[0]
    for _ in range(10):
        got, st = run(bad)
        assert st.tolist() == [BAD_TREE, 0, 0]
        check_all_but(got, good, c, [0], fp8, 0, 0)


@pytest.mark.parametrize("off, want", [([0, 0, 0, 0], [0, 0, 0]), ([0, 5, 5, 5], [5, 0, 0]), ([0, 0, 1, 2], [0, 5, 5]),
                                       ([0, 0, -1, -1], [0, 5, 5]), ([3, 3, 3, 3], [0, 0, 0]), ([LOW, HIGH, HIGH, 0], [5, 0, 5])])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_offsets_without_rows(off, want, fp8):
    """Without rows every sequence that has some, or lies behind a decrease, is malformed."""
    ensure_built()
    lens, table = i32([30, 40, 50]), i32(np.arange(12).reshape(3, 4))
    elem = torch.uint8 if fp8 else torch.bfloat16
    pool = torch.zeros(12, 2, 16, 128, dtype=elem, device="cuda")
    q = torch.empty(0, 4, 128, dtype=elem, device="cuda")
    if fp8:
        scale = torch.ones(12, 2, 16, device="cuda")
        out, st = tv.chunk_attention_fp8(q, torch.empty(0, 4, device="cuda"), pool, scale, pool, scale, table, lens,
                                         i32(off), max_len=50)
    else:
        out, st = tv.chunk_attention(q, pool, pool, table, lens, i32(off), max_len=50)
    assert st.tolist() == want and out.shape == (0, 4, 128)


@pytest.mark.parametrize("out_dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("off, bad, zero", [
    ([0, 8, 58, 59, 62, 200], [4], (62, 82)),         # rows past the end: those that are there
    ([0, 8, 58, 59, 62, HIGH], [4], (62, 82)),
    ([-5, 8, 58, 59, 62, 82], [0], (0, 8)),           # rows before the first
    ([LOW, 8, 58, 59, 62, 82], [0], (0, 8)),
    ([0, 8, 58, 59, 90, 95], [3, 4], (59, 82)),       # one past the end, one wholly behind it
    ([0, 90, 58, 59, 62, 82], [0, 1, 2, 3, 4], (0, 82)),  # past the end, and a decrease behind it
    ([0, 8, 58, LOW, 62, 80], [2, 3, 4], (58, 80)),   # a decrease: only rows that no sound sequence has
])
def test_chunk_rows_outside_the_output(off, bad, zero, out_dtype):
    """Of a malformed sequence every row that is there and is no sound
    sequence's reads as zeros, and no other row changes."""
    c = make([40, 50, 60, 33, 20], [8, 50, 1, 3, 20], 8, 2, 128, seed=1)
    good, _ = call(c, out_dtype=out_dtype)
    got, st = call(dict(c, off=np.asarray(off, np.int32)), max_len=60, fill=5.0, out_dtype=out_dtype)
    assert st.tolist() == [BAD_TREE if b in bad else 0 for b in range(5)]
    want = np.full_like(good, 5.0)
    for b in set(range(5)) - set(bad):
        want[off[b]:off[b + 1]] = good[off[b]:off[b + 1]]
    want[zero[0]:zero[1]] = 0.0
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window, sinks", [(0, 0), (200, 20)])
@pytest.mark.parametrize("page", ["first", "middle", "last", "evicted"])
def test_chunk_bad_page_zeroes_the_whole_sequence(fp8, window, sinks, page):
    """A prompt of many units, of which some do not see the bad page: every row
    of the sequence is zeros.  A page that no row sees may be anything."""
    lens, chunks = [1203, 901, 40, 611], [1, 700, 40, 611]
    c = make(lens, chunks, 8, 2, 128, seed=11)
    run = call_fp8 if fp8 else call
    c = quantised(c) if fp8 else c
    kw = dict(window=window, sinks=sinks)
    good, st = run(c, **kw)
    assert (st == 0).all()
    first = 901 - 700
    at = {"first": 0, "middle": 500 // 16, "last": 900 // 16, "evicted": sinks // 16 + 1}[page]
    if page == "evicted" and not window:
        return
    for value in (-1, c["k"].shape[0], LOW, HIGH):
        bad = dict(c, table=c["table"].copy())
        bad["table"][1, at] = value
        got, st = run(bad, **kw)
        seen = not window or at * 16 < sinks or at * 16 + 15 > first - window
        assert st.tolist() == [0, BAD_TREE if seen else 0, 0, 0]
        check_all_but(got, good, c, [1] if seen else [], fp8, window, sinks)
        again, _ = run(bad, **kw)
        np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_every_page_is_looked_at(fp8):
    """Windows, sinks and chunks of many sizes: the status and the rows follow
    from the pages that some row of the sequence sees."""
    g = np.random.default_rng(3)
    run = call_fp8 if fp8 else call
    for rep in range(12):
        chunks = [int(x) for x in g.integers(1, 400, 4)]
        lens = [x + int(g.integers(0, 600)) for x in chunks]
        window, sinks = int(g.choice([0, 1, 16, 100, 500])), int(g.choice([0, 1, 16, 40]))
        c = make(lens, chunks, 4, 2, 128, seed=100 + rep)
        c = quantised(c) if fp8 else c
        good, _ = run(c, window=window, sinks=sinks)
        bad, status = dict(c, table=c["table"].copy()), []
        for b in range(4):
            at = int(g.integers(0, -(-lens[b] // 16)))
            bad["table"][b, at] = int(g.choice([-1, c["k"].shape[0], HIGH, LOW]))
            keys = np.arange(lens[b])
            seen = keys > lens[b] - chunks[b] - window if window else keys >= 0
            seen |= keys < sinks
            status.append(BAD_TREE if seen[at * 16:at * 16 + 16].any() else 0)
        got, st = run(bad, window=window, sinks=sinks)
        assert st.tolist() == status
        check_all_but(got, good, c, [b for b in range(4) if status[b]], fp8, window, sinks)


def test_chunk_pages_of_many_sequences():
    """More sequences than a launch of the check has CTAs, long tables, and a bad
    page here and there."""
    g = np.random.default_rng(8)
    B = 700
    lens = [int(x) for x in g.integers(1, 40, B)]
    lens[5], lens[650] = 5003, 9001
    c = make(lens, [1] * B, 2, 1, 64, seed=1)
    good, st = call(c)
    assert (st == 0).all()
    hit = [0, 5, 151, 152, 304, 650, 699]
    bad = dict(c, table=c["table"].copy())
    for b in hit:
        bad["table"][b, (lens[b] - 1) // 16] = -1
    got, st = call(bad)
    assert np.flatnonzero(st).tolist() == hit and (st[hit] == BAD_TREE).all()
    check_all_but(got, good, c, hit, False, 0, 0)


def test_chunk_workspace_that_is_no_tensor():
    c = make([20], [3], 4, 2, 64, seed=0)
    for bad in ([0] * 1024, 4096, torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(2, 1 << 20, device="cuda").t()):
        with pytest.raises(ValueError):
            call(c, workspace=bad)
