"""GPU parity of tv_penalize_logits against fp64.

Tolerance: at most five fp32 roundings (division or product, freq x c, two
differences, the bias), each of half an ulp of a value of at most A = the
largest of |logit| max(r, 1/r), |freq| c, |pres|, |bias| summed:
5 x 2^-24 x A per entry."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def make(nodes, vocab, hist, seed, biases=0, masked=False, chain=False):
    g = np.random.default_rng(seed)
    B = len(nodes)
    par = []
    for n in nodes:
        par += [-1] + [i - 1 if chain else int(g.integers(0, i)) for i in range(1, n)]
    off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    total = int(off[-1])
    ids = max(2, min(vocab, 40))
    c = dict(logits=(g.standard_normal((total, vocab)) * 3).astype(np.float32),
             draft_tokens=g.integers(0, ids, total).astype(np.int32), parent=np.asarray(par, np.int32),
             node_offsets=off, history=g.integers(0, ids, max(1, sum(hist))).astype(np.int32),
             history_offsets=np.concatenate([[0], np.cumsum(hist)]).astype(np.int32),
             prompt_lens=np.asarray([h // 2 for h in hist], np.int32),
             repetition=(0.7 + g.random(B)).astype(np.float32), presence=g.standard_normal(B).astype(np.float32),
             frequency=g.standard_normal(B).astype(np.float32))
    if biases:
        c.update(bias_ids=g.integers(0, vocab, biases * B).astype(np.int32),
                 bias_values=g.standard_normal(biases * B).astype(np.float32),
                 bias_offsets=np.arange(0, biases * B + 1, biases, dtype=np.int32))
    if masked:
        c["allowed"] = g.random((total, vocab)) < 0.5
        c["allowed"][0] = False  # a row that allows nothing
        c["allowed"][-1] = True
    return c


def words(allowed):
    v = allowed.shape[1]
    bits = np.zeros((allowed.shape[0], -(-v // 32) * 32), np.uint8)
    bits[:, :v] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view("<u4").view(np.int32)


def call(c, max_nodes=None, in_place=False, **kw):
    ensure_built()
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in c.items() if k != "allowed"}
    if "allowed" in c:
        t["allowed_mask"] = torch.from_numpy(words(c["allowed"])).cuda()
    if c["logits"].dtype == np.int16:
        t["logits"] = t["logits"].view(torch.bfloat16)
    first = [t.pop(k) for k in ("logits", "draft_tokens", "parent", "node_offsets")]
    if in_place:
        kw["out"] = first[0]
    n = int(np.diff(c["node_offsets"]).max())
    out, st = tv.penalize_logits(*first, max_nodes=max_nodes or n, **t, **kw)
    torch.cuda.synchronize()
    return out.cpu().numpy(), st.cpu().numpy()


def check(got, c):
    ref = oracle.penalize_logits(**c)
    rep = max(np.max(c["repetition"]), 1 / np.min(c["repetition"]))
    count = float(np.max(np.diff(c["history_offsets"]), initial=0) + np.diff(c["node_offsets"]).max())
    big = np.abs(np.where(np.isfinite(c["logits"]), c["logits"], 0)).max() * rep + np.abs(c["presence"]).max() + \
        np.abs(c["frequency"]).max() * count + np.abs(c.get("bias_values", np.zeros(1))).max()
    inf = ~np.isfinite(ref)
    np.testing.assert_array_equal(got[inf], ref[inf].astype(np.float32))
    assert np.abs(got[~inf] - ref[~inf]).max(initial=0) <= 5 * 2.0 ** -24 * big


CASES = [([1], 1, [0]), ([1], 7, [3]), ([5, 1], 33, [0, 9]), ([15], 1000, [40]), ([40, 3, 64], 4096, [100, 0, 7]),
         ([9], 4097, [60]), ([30, 20], 9001, [300, 50])]


@pytest.mark.parametrize("nodes, vocab, hist", CASES)
@pytest.mark.parametrize("biases, masked", [(0, False), (5, True)])
def test_against_fp64(nodes, vocab, hist, biases, masked):
    c = make(nodes, vocab, hist, vocab, biases, masked)
    got, st = call(c)
    assert (st == 0).all()
    check(got, c)


@pytest.mark.parametrize("vocab", [2047, 2049, 8192, 9001, 32000])
@pytest.mark.parametrize("in_place", [False, True])
def test_ids_all_over_the_vocabulary(vocab, in_place):
    """Histories, paths and biases meet every part of a row, its ends included,
    and one another."""
    c = make([64, 1, 17], vocab, [500, 0, 90], vocab, biases=30, masked=True)
    g = np.random.default_rng(vocab)
    pool = np.concatenate([[0, 1, vocab - 1, vocab // 2, 511, 512, 1023, 1024, 2046], g.integers(0, vocab, 40)])
    for k in ("draft_tokens", "history", "bias_ids"):
        c[k] = g.choice(pool, c[k].shape).astype(np.int32)
    got, st = call(c, in_place=in_place)
    assert (st == 0).all()
    check(got, c)


@pytest.mark.parametrize("vocab", [1000, 1001])
def test_bf16_logits_and_in_place(vocab):
    c = make([12, 30], vocab, [20, 50], 1, 4, True)
    c["logits"] = torch.from_numpy(c["logits"]).to(torch.bfloat16).float().numpy()
    want, _ = call(c)
    check(want, c)
    half = dict(c, logits=torch.from_numpy(c["logits"]).to(torch.bfloat16).view(torch.int16).numpy())
    got, _ = call(half)
    np.testing.assert_array_equal(got, want)
    got, _ = call(c, in_place=True)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("chain", [False, True])
def test_long_paths_with_repeats(chain):
    """512 nodes: paths of more than 32 drafted tokens, most of them repeated."""
    c = make([512, 100], 5000, [10, 0], 3, 0, False, chain)
    for in_place in (False, True):
        got, st = call(c, in_place=in_place)
        assert (st == 0).all()
        check(got, c)


def test_nothing_to_do_copies():
    ensure_built()
    x = torch.randn(3, 100, device="cuda")
    x[0, 5], x[1, 6], x[2, 7] = float("nan"), float("inf"), -0.0
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out, st = tv.penalize_logits(x, i([0, 1, 2]), i([-1, 0, 1]), i([0, 3]), max_nodes=3)
    assert st.item() == 0
    np.testing.assert_array_equal(out.cpu().numpy().view(np.int32), x.cpu().numpy().view(np.int32))


def test_special_logits():
    """-inf and inf stay what the formulas make of them; NaN stays NaN unless masked."""
    c = make([4], 64, [0], 2)
    c["logits"][:, :4] = [np.inf, -np.inf, np.nan, 0.0]
    c["history"], c["history_offsets"] = np.array([0, 1, 2, 3], np.int32), np.array([0, 4], np.int32)
    c["prompt_lens"][:] = 0
    c["draft_tokens"][:] = 9
    got, _ = call(c)
    ref = oracle.penalize_logits(**c)
    np.testing.assert_array_equal(got[:, :3], ref[:, :3].astype(np.float32))
    c["allowed"] = np.zeros((4, 64), bool)
    got, _ = call(c)
    assert (got == -np.inf).all()


def test_ids_outside_the_vocabulary_and_repeated_bias_ids():
    c = make([6], 500, [30], 5, 6)
    c["history"][::3] = [-1, 500, 10 ** 9, -2 ** 31, 501, 499, 0, -5, 7, 600]
    c["draft_tokens"][2:4] = [-1, 500]
    c["bias_ids"][:] = [7, 7, -1, 500, 499, 7]
    got, st = call(c)
    assert st[0] == 0
    check(got, c)


def test_malformed_sequences_keep_their_rows():
    good = make([5, 6, 7, 4], 300, [20, 20, 20, 20], 8, 3, True)

    def broken(**kw):
        c = {k: v.copy() for k, v in good.items()}
        for k, (at, x) in kw.items():
            c[k][at] = x
        return c

    for c, bad in ((broken(parent=(6, 3)), 1), (broken(parent=(0, 0)), 0), (broken(repetition=(2, 0.0)), 2),
                   (broken(repetition=(2, np.nan)), 2), (broken(presence=(3, np.inf)), 3),
                   (broken(frequency=(0, np.nan)), 0), (broken(history_offsets=(4, 81)), 3),
                   (broken(bias_offsets=(0, -1)), 0)):
        got, st = call(c, max_nodes=7)
        assert st.tolist() == [5 if b == bad else 0 for b in range(4)]
        n0, n1 = c["node_offsets"][bad:bad + 2]
        np.testing.assert_array_equal(got[n0:n1], c["logits"][n0:n1])
        keep = [r for r in range(22) if not n0 <= r < n1]
        ref = oracle.penalize_logits(**good)
        np.testing.assert_allclose(got[keep], ref[keep], rtol=0, atol=5 * 2.0 ** -24 * 200)
    got, st = call(good, max_nodes=6)  # a tree larger than max_nodes
    assert st.tolist() == [0, 0, 5, 0]
    np.testing.assert_array_equal(got[11:18], good["logits"][11:18])


def test_graph_side_stream_and_refusals():
    c = make([20, 9], 3000, [50, 0], 4, 3, True)
    want, _ = call(c)
    side = torch.cuda.Stream()
    got, _ = call(c, stream=side)
    np.testing.assert_array_equal(got, want)
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in c.items() if k != "allowed"}
    mask = torch.from_numpy(words(c["allowed"])).cuda()
    first = [t.pop(k) for k in ("logits", "draft_tokens", "parent", "node_offsets")]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, st = tv.penalize_logits(*first, max_nodes=20, allowed_mask=mask.view(torch.uint32), **t)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.cpu().numpy(), want)
    for kw in (dict(t, history=None), dict(t, bias_offsets=None), dict(t, repetition=t["repetition"].double()),
               dict(t, allowed_mask=mask[:, :-1].contiguous()), dict(t, out=out[:5]), dict(t, presence=t["presence"][:1]),
               dict(t, out=out.t()), dict(t, allowed_mask=mask.float())):
        with pytest.raises(ValueError):
            tv.penalize_logits(*first, max_nodes=20, **kw)
    with pytest.raises(ValueError):
        tv.penalize_logits(first[0].half(), *first[1:], max_nodes=20)
    with pytest.raises(tv.TVError):
        tv.penalize_logits(first[0].bfloat16(), *first[1:], max_nodes=600)


def test_large_rows_at_odd_widths():
    for vocab in (151936, 128255):
        c = make([70], vocab, [500], vocab, 20, True)
        got, st = call(c)
        assert (st == 0).all()
        check(got, c)
