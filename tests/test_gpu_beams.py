"""GPU parity of tv_beam_select with fp64: tokens, parents, lengths and ends match
exactly, scores within the bound below.

Scores: one rounding to fp32, 2^-24 |score|, and LSE's error: every exp is off by
2^-22 (ex2.approx), the rounding of x - m and of its product with log2 e (relative
to d = m - x <= 32 where it counts: 3 d 2^-24 < 2^-17 for the smallest of them, whose
weight is e^-d; d e^-d <= 1/e), and 32 + 5 + 8 sums in fp32, 45 2^-24, and the join
of at most 33 parts, 5 more: below 2^-17 in all.  The cases' candidates that decide
an order between rows are further apart than 2^-15."""
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu
LSE = 2.0 ** -17
INF = float("inf")


def i32(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def run(logits, scores, beams, select, lengths=None, finished=None, end_token=-1, length_penalty=0.0, **kw):
    r = tv.beam_select(logits, torch.from_numpy(np.asarray(scores, np.float32)).cuda(), beams=beams, select=select,
                       lengths=i32(lengths), finished=i32(finished), end_token=end_token, length_penalty=length_penalty, **kw)
    return {k: None if v is None else v.cpu().numpy() for k, v in r.items()}


def compare(got, ref, lengths, gap=2.0 ** -15):
    for b, want in enumerate(ref):
        if want is None:
            assert got["status"][b] == tv.TV_ERR_BAD_TREE
            assert (got["tokens"][b] == -1).all() and (got["parents"][b] == -1).all()
            assert (got["scores"][b] == -INF).all() and (got["finished"][b] == 0).all()
            continue
        assert got["status"][b] == 0
        keys = [c[5] for c in want]
        for x, y, c, d in zip(keys, keys[1:], want, want[1:]):  # the case's own property
            assert c[1] == d[1] or not x - y < gap or x == y, "the case has a near tie"
        assert got["tokens"][b].tolist() == [c[0] for c in want]
        assert got["parents"][b].tolist() == [c[1] for c in want]
        if lengths is not None:
            assert got["lengths"][b].tolist() == [c[3] for c in want]
        assert got["finished"][b].tolist() == [c[4] for c in want]
        for x, c in zip(got["scores"][b].tolist(), want):
            assert x == c[2] or abs(x - c[2]) <= LSE + 2.0 ** -24 * abs(c[2])


CASES = [  # batch, beams, select, V, type, penalty, seed
    (1, 1, 1, 1, torch.float32, 0.0, 1),
    (2, 1, 3, 2, torch.bfloat16, 0.0, 2),
    (1, 4, 4, 1000, torch.float32, 0.0, 3),
    (3, 5, 10, 1001, torch.bfloat16, 0.7, 4),     # rows that are not 16-byte aligned
    (2, 3, 6, 8193, torch.float32, 1.0, 5),       # a part of one entry
    (2, 2, 64, 8184, torch.bfloat16, -0.5, 6),
    (2, 8, 16, 32000, torch.bfloat16, 0.6, 7),
    (1, 64, 64, 4099, torch.float32, 0.0, 8),
    (1, 40, 64, 70001, torch.bfloat16, 0.0, 9),   # more lists than a CTA has threads
    (1, 64, 64, 262143, torch.bfloat16, 0.0, 12), # more lists than a CTA holds
    (1, 64, 1, 262143, torch.float32, 0.0, 13),
    (1, 4, 8, 262143, torch.float32, 0.0, 10),    # the largest vocabulary
    (1, 1, 64, 151936, torch.bfloat16, 0.0, 11),  # one row, many of it
]


def make(batch, beams, vocab, dtype, seed, quantum=None):
    g = np.random.default_rng(seed)
    x = g.standard_normal((batch * beams, vocab)) * 2.5
    if quantum:  # many equal logits
        x = np.round(x / quantum) * quantum
    logits = torch.from_numpy(x).to(dtype)
    scores = (-30 * g.random((batch, 1)) - 4 * g.random((batch, beams))).reshape(-1).astype(np.float32)
    lengths = g.integers(1, 100, (batch, 1)).repeat(beams, 1).reshape(-1)
    return logits, scores, lengths, g


@pytest.mark.parametrize("case", CASES)
def test_parity(case):
    ensure_built()
    batch, beams, select, vocab, dtype, penalty, seed = case
    logits, scores, lengths, _ = make(batch, beams, vocab, dtype, seed)
    ref = oracle.beam_select(logits.double().numpy(), scores, beams, select, lengths, None, vocab // 2, penalty)
    got = run(logits.cuda(), scores, beams, select, lengths, None, vocab // 2, penalty)
    compare(got, ref, lengths, gap=2.0 ** -15 / max(1.0, float(lengths.max() + 1) ** penalty))


@pytest.mark.parametrize("quantum, vocab, select", [(0.5, 5000, 16), (2.0, 3001, 64), (100.0, 9000, 7), (100.0, 40000, 64)])
def test_equal_logits_come_by_token(quantum, vocab, select):
    """Thousands of equal logits in a row: the lower token first, also where they do
    not fit the list that is ranked."""
    ensure_built()
    for dtype in (torch.float32, torch.bfloat16):
        logits, scores, lengths, _ = make(2, 3, vocab, dtype, 5, quantum)
        scores = np.array([-1, -9.5, -20, -3, -18.25, -40], np.float32)
        if quantum == 100.0:
            logits[:] = 0.0
            logits[1, ::2] = -0.0  # the same value
        ref = oracle.beam_select(logits.double().numpy(), scores, 3, select, lengths)
        compare(run(logits.cuda(), scores, 3, select, lengths), ref, lengths)


def test_equal_rows_come_by_row():
    """Beams that are alike in everything: equal keys to the last bit."""
    ensure_built()
    logits, _, _, _ = make(1, 1, 20000, torch.float32, 3)
    logits = logits.repeat(6, 1)
    scores = np.full(6, -2.5, np.float32)
    got = run(logits.cuda(), scores, 6, 15)
    best = np.lexsort((np.arange(20000), -logits[0].numpy()))[:3]
    assert got["tokens"][0].tolist() == [int(v) for v in best.repeat(6)[:15]]
    assert got["parents"][0].tolist() == (list(range(6)) * 3)[:15]


def test_many_alike_rows_fall_back():
    """Constant logits in 40 alike rows: more candidates than are ranked."""
    ensure_built()
    logits = torch.zeros(40, 3000)
    finished = np.zeros(40, np.int32)
    finished[7] = finished[39] = 1
    scores = np.full(40, -2.0, np.float32)
    scores[7] = -2.0 - math.log(3000) - 1.0   # behind all candidates but the next row's
    scores[39] = -1.0                         # ahead of all
    ref = oracle.beam_select(logits.double().numpy(), scores, 40, 64, np.full(40, 3), finished, 11)
    got = run(logits.cuda(), scores, 40, 64, np.full(40, 3), finished, 11)
    # (all rows' scores are the same to the last bit: rows in order, tokens in order)
    assert got["parents"][0].tolist() == [39] + [0] * 63 and [c[1] for c in ref[0]] == got["parents"][0].tolist()
    assert got["tokens"][0].tolist() == [11] + list(range(63)) and got["status"][0] == 0
    scores[7] = -1.5                          # the second
    got = run(logits.cuda(), scores, 40, 64, np.full(40, 3), finished, 11)
    assert got["parents"][0].tolist() == [39, 7] + [0] * 62 and got["tokens"][0].tolist() == [11, 11] + list(range(62))
    assert got["finished"][0].tolist() == [1, 1] + [int(v == 11) for v in range(62)]
    # few tokens each: the ended beam between them is found too
    got = run(torch.zeros(40, 1, device="cuda"), np.where(finished, -2.5, -2.0), 40, 64, np.full(40, 3), finished, 0)
    assert got["parents"][0].tolist()[:38] == [r for r in range(40) if r not in (7, 39)]
    assert got["parents"][0].tolist()[38:] == [7, 39] + [-1] * 24


def test_ended_and_dead_beams():
    ensure_built()
    for seed, penalty in ((0, 0.0), (1, 0.8), (2, -0.3)):
        logits, scores, lengths, g = make(6, 5, 3000, torch.float32, seed)
        finished = (g.random(30) < 0.4).astype(np.int32)
        finished[5:10] = 1                    # a request whose beams have all ended
        lengths = np.where(finished, g.integers(0, 20, 30), lengths)
        scores[10:14] = -INF                  # the first step: one beam is live
        scores[15:20] = -INF                  # nothing is left
        logits[finished != 0] = float("nan")  # not read
        ref = oracle.beam_select(logits.double().numpy(), scores, 5, 7, lengths, finished, 17, penalty)
        got = run(logits.cuda(), scores, 5, 7, lengths, finished, 17, penalty)
        compare(got, ref, lengths, gap=2.0 ** -15 / 101.0 ** max(penalty, 0))
        assert (got["parents"][3] == -1).all() and got["status"][3] == 0
        assert (got["tokens"][1][:5] == 17).all() and (got["tokens"][1][5:] == -1).all()


def test_masked_logits():
    """-inf and NaN offer nothing; a row that offers nothing is as a dead one."""
    ensure_built()
    logits, scores, lengths, g = make(4, 3, 9000, torch.float32, 8)
    logits[torch.from_numpy(g.random((12, 9000)) < 0.9995)] = -INF
    logits[2] = -INF
    logits[3:6] = -INF
    logits[3, 8999], logits[4, 0] = 1.5, -3e38     # one token each
    logits[6, 100:200] = float("nan")
    logits[7] = float("nan")
    ref = oracle.beam_select(logits.double().numpy(), scores, 3, 8, lengths)
    got = run(logits.cuda(), scores, 3, 8, lengths)
    compare(got, ref, lengths)
    assert (got["parents"][1] >= 0).sum() == 2


def test_refused_requests_leave_the_others():
    ensure_built()
    logits, scores, lengths, _ = make(6, 2, 500, torch.bfloat16, 9)
    scores[2], scores[5] = float("nan"), INF
    logits[7, 3] = INF
    lengths = lengths.copy()
    lengths[8], lengths[11] = -1, (1 << 24) + 1
    ref = oracle.beam_select(logits.double().numpy(), scores, 2, 4, lengths)
    assert [x is None for x in ref] == [False, True, True, True, True, True]
    compare(run(logits.cuda(), scores, 2, 4, lengths), ref, lengths)
    finished = np.zeros(12, np.int32)
    finished[7] = 1  # its logits are not read
    assert run(logits.cuda(), scores, 2, 4, None, finished)["status"].tolist() == [0, 5, 5, 0, 0, 0]


def test_extremes():
    """The smallest and largest finite logits and scores."""
    ensure_built()
    logits = torch.full((2, 300), -3.3e38)
    logits[0, 7], logits[1, 9] = 3.3e38, -3.2e38
    got = run(logits.cuda(), [-1e30, -1e-30], 2, 3)
    assert got["tokens"][0].tolist() == [9, 7, 0] and got["parents"][0].tolist() == [1, 0, 1] and got["status"][0] == 0
    np.testing.assert_allclose(got["scores"][0], [-1e-30, -1e30, -1e37], rtol=1e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_of_the_lowest_value(dtype):
    """Masks that are finite: rows of which some, few, and no entries are above them."""
    ensure_built()
    low = torch.finfo(dtype).min
    logits, scores, lengths, g = make(3, 4, 20000, dtype, 21)
    logits[torch.from_numpy(g.random((12, 20000)) < 0.5)] = low
    logits[4:8][torch.from_numpy(g.random((4, 20000)) < 0.9999)] = low
    logits[8] = low             # nothing but masks: all tokens alike
    logits[9, :19000] = low     # whole parts of masks
    logits[10] = low
    logits[10, 5] = 1e30        # and next to the largest
    ref = oracle.beam_select(logits.double().numpy(), scores, 4, 8, lengths)
    got = run(logits.cuda(), scores, 4, 8, lengths)
    compare(got, ref, lengths)
    row = run(logits[8:9].cuda(), scores[8:9], 1, 3)
    assert row["tokens"][0].tolist() == [0, 1, 2]
    np.testing.assert_allclose(row["scores"][0], scores[8] - math.log(20000), rtol=0, atol=LSE + 2.0 ** -24 * 64)


def test_strided_rows_streams_graphs_and_workspaces():
    ensure_built()
    logits, scores, lengths, _ = make(3, 4, 32000, torch.bfloat16, 12)
    wide = torch.full((12, 32771), INF, dtype=torch.bfloat16, device="cuda")
    wide[:, :32000] = logits.cuda()
    want = run(logits.cuda(), scores, 4, 8, lengths)
    got = run(wide[:, :32000], scores, 4, 8, lengths)
    for k in want:
        np.testing.assert_array_equal(want[k], got[k])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, sc, ln = wide[:, :32000], torch.from_numpy(scores).cuda(), i32(lengths)
    s.wait_stream(torch.cuda.current_stream())
    r = tv.beam_select(x, sc, beams=4, select=8, lengths=ln, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(r["tokens"].cpu().numpy(), want["tokens"])
    ws = torch.full((tv.beam_workspace_size(x, beams=4, select=8),), 0xFF, dtype=torch.uint8, device="cuda")
    keep = {k: r[k].clone() for k in ("tokens", "parents")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.beam_select(x, sc, beams=4, select=8, lengths=ln, workspace=ws, scores_out=r["scores"],
                       lengths_out=r["lengths"], finished_out=r["finished"], status=r["status"], **keep)
    for _ in range(3):
        keep["tokens"].fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(keep["tokens"].cpu().numpy(), want["tokens"])
    with pytest.raises(tv.TVError):
        tv.beam_select(x, sc, beams=4, select=8, workspace=ws[:-16])


def test_many_requests_of_a_small_vocabulary():
    ensure_built()
    logits, scores, lengths, g = make(2000, 3, 37, torch.float32, 31, quantum=2.0 ** -6)
    finished = (g.random(6000) < 0.1).astype(np.int32)
    scores = np.round(scores * 8) / 8  # (rows' scores may be equal, their LSEs are not)
    ref = oracle.beam_select(logits.double().numpy(), scores, 3, 5, lengths, finished, 36, 1.0)
    got = run(logits.cuda(), scores, 3, 5, lengths, finished, 36, 1.0)
    # requests whose order between rows is decided by less than the bound are left out
    sure = [b for b, want in enumerate(ref)
            if all(c[1] == d[1] or c[5] - d[5] > 2.0 ** -15 or c[5] == d[5] for c, d in zip(want, want[1:]))]
    assert len(sure) > 1900
    pick = {k: None if v is None else v[sure] for k, v in got.items()}
    compare(pick, [ref[b] for b in sure], lengths)


def test_repeated_calls_agree_bit_for_bit():
    ensure_built()
    logits, scores, lengths, _ = make(8, 8, 60000, torch.float32, 13)
    x = logits.cuda()
    a = run(x, scores, 8, 16, lengths)
    for _ in range(5):
        b = run(x, scores, 8, 16, lengths)
        for k in a:
            np.testing.assert_array_equal(a[k], b[k])


def test_many_long_rows():
    """Rows of one CTA each and of the largest vocabulary: 65 turns of a warp, whose sums
    are 16 of a turn, 65 of turns, 5 of lanes and 8 of parts: 94 2^-24, below 2^-17 with
    the rest."""
    ensure_built()
    batch, beams, select, vocab = 170, 4, 8, 262143
    g = torch.Generator(device="cuda").manual_seed(41)
    logits = torch.randn(batch * beams, vocab, device="cuda", generator=g) * 3
    scores = -20 * torch.rand(batch * beams, device="cuda", generator=g)
    got = tv.beam_select(logits, scores, beams=beams, select=select)
    sure = 0
    some = range(0, batch, 7)
    for b in some:
        rows = slice(b * beams, (b + 1) * beams)
        x = logits[rows].double()
        best, at = (scores[rows].double()[:, None] + x - x.logsumexp(-1, keepdim=True)).flatten().topk(select + 1)
        assert (got["scores"][b].double() - best[:select]).abs().max() <= LSE + 2.0 ** -24 * 40
        if (best[:-1] - best[1:]).min() > 2.0 ** -15:
            sure += 1
            assert torch.equal(got["tokens"][b].long(), at[:select] % vocab)
            assert torch.equal(got["parents"][b].long(), b * beams + at[:select] // vocab)
    assert sure > len(some) // 2 and (got["status"] == 0).all()


def unlike(kind, dtype, vocab, seed):
    """Two requests of three beams whose best are all in some parts of a row."""
    logits, scores, lengths, g = make(2, 3, vocab, dtype, seed)
    if kind == "upper half":
        logits[:, vocab // 2:] = -INF
    elif kind == "lowest value":
        logits[:, vocab // 3:] = torch.finfo(dtype).min
    elif kind == "few":
        keep = logits[:, 1000:1300].clone()
        logits[:] = -INF
        logits[:, 1000:1300] = keep
    elif kind == "rising":
        logits[:] = (torch.arange(vocab) * 2.0 ** -10).to(dtype)
    elif kind == "falling":
        logits[:] = (torch.arange(vocab, 0, -1) * 2.0 ** -10).to(dtype)
    elif kind == "last":
        logits[:, -5:] += 20
    return logits, scores, lengths


KINDS = ["upper half", "lowest value", "few", "rising", "falling", "last"]


@pytest.mark.parametrize("select", [5, 16, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_parts_that_are_not_alike(kind, select):
    ensure_built()
    for dtype in (torch.float32, torch.bfloat16):
        for vocab in (40000, 9001):
            logits, scores, lengths = unlike(kind, dtype, vocab, 51)
            ref = oracle.beam_select(logits.double().numpy(), scores, 3, select, lengths)
            compare(run(logits.cuda(), scores, 3, select, lengths), ref, lengths)
