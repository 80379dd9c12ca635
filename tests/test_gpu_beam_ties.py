"""tv_beam_select where the keys of a row's candidates round to one value: scores or
logits so large that what tells two tokens apart is below the last bit of their sum.
Within a row the order stays that of the logits, and of equal ones the lower token
comes first.  The references take the candidates of a row by logit, in fp64."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(logits, scores, beams, select, lengths=None, finished=None, end_token=-1, length_penalty=0.0):
    ensure_built()
    scores = np.asarray(scores, np.float32)
    ref = oracle.beam_select(logits.double().numpy(), scores, beams, select, lengths, finished, end_token, length_penalty)

    def i32(x):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()

    got = tv.beam_select(logits.cuda(), torch.from_numpy(scores).cuda(), beams=beams, select=select, lengths=i32(lengths),
                         finished=i32(finished), end_token=end_token, length_penalty=length_penalty)
    assert (got["status"] == 0).all()
    for b, want in enumerate(ref):
        assert got["parents"][b].tolist() == [c[1] for c in want]
        assert got["tokens"][b].tolist() == [c[0] for c in want]
        for x, c in zip(got["scores"][b].tolist(), want):
            # the sums' bound of 2^-15 and one rounding, half a step of fp32
            assert x == c[2] or abs(x - c[2]) <= 2.0 ** -15 + 2.0 ** -24 * abs(c[2])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [-1e10, -1e20, -1e30, float(np.finfo(np.float32).min), 1e15])
@pytest.mark.parametrize("vocab, select", [(300, 8), (5000, 16), (40000, 64), (128256, 33)])
def test_scores_of_large_magnitude(score, vocab, select, dtype):
    """Two beams, one of them with three tokens left by a mask; the other one's score is
    large, so that its tokens have (nearly) one key."""
    g = torch.Generator().manual_seed(vocab)
    logits = (torch.randn(2, vocab, generator=g) * 2.5).to(dtype)
    masked = 1 if score > 0 else 0
    keep = logits[masked, [1, vocab // 2, vocab - 2]].clone()
    logits[masked] = -INF
    logits[masked, [1, vocab // 2, vocab - 2]] = keep
    check(logits, [0.0, score], 2, select)
    check(logits, [0.0, score], 2, select, [7, 7], length_penalty=0.6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_forced_token(dtype):
    """One logit far above the others: those come by their logits behind it."""
    logits = torch.full((1, 4000), -50.0)
    logits[0, 0], logits[0, 3], logits[0, 5], logits[0, 3999] = 1e20, 1.0, 2.0, 1.5
    got = check(logits.to(dtype), [-2.0], 1, 4)
    assert got["tokens"][0].tolist() == [0, 5, 3999, 3]
    logits[0, 0] = 3.0e38
    check(logits.to(dtype), [-2.0], 1, 40)


@pytest.mark.parametrize("vocab", [20, 30, 3000])
@pytest.mark.parametrize("quantum", [0.0, 1.0])
def test_many_rows_of_one_key(vocab, quantum):
    """40 beams of one score whose candidates all have its key: by beam, then by logit,
    then by token (with 20 tokens a beam they are ranked by counting, with more they are
    merged one by one), ended beams at their place."""
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(40, vocab, generator=g) * 2.5
    if quantum:
        logits = torch.round(logits / quantum) * quantum
    finished = np.zeros(40, np.int32)
    check(logits, [-1e30] * 40, 40, 64)
    finished[1] = finished[3] = 1
    check(logits, [-1e30] * 40, 40, 64, np.full(40, 5), finished, 2)
    finished[0] = 1  # (its length without, the others' with one more: another key)
    check(logits, [-1e30] * 40, 40, 64, np.full(40, 5) + finished, finished, 2, 1.0)


def test_scores_of_a_step_with_beams_that_do_not_count_yet():
    """The first step of a search whose other beams carry -1e9: the first beam's tokens,
    then, where a mask leaves too few, the others' in order of their logits."""
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(8, 32000, generator=g) * 2.5
    logits[0, 5:] = -INF
    logits[4, 9:] = -INF
    check(logits, [0.0, -1e9, -2e9, -3e9] * 2, 4, 12)
