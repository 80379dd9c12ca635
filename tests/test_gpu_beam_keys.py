"""tv_beam_select: keys that are equal by their definition, score / length^penalty, of rows
of different lengths.  Ended beams' scores are given, so the quotients are known exactly:
equal ones come by row."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams, select", [(8, 8), (64, 64), (64, 7)])
@pytest.mark.parametrize("mean", [-1.0, -0.75, 3.0, -1024.0])
def test_equal_means_of_ended_beams_come_by_row(mean, beams, select):
    """Scores of one mean a token (a whole number of quarters, exact in fp32)."""
    ensure_built()
    g = np.random.default_rng(beams)
    requests = 40
    lengths = g.integers(1, 2000, requests * beams)
    lengths[:8] = [1, 49, 98, 103, 107, 161, 187, 197]  # (1 / n, n times, is not 1 of these)
    scores = (lengths * mean).astype(np.float32)
    assert (scores.astype(np.float64) / lengths == mean).all()
    finished = np.ones(requests * beams, np.int32)
    logits = torch.zeros(requests * beams, 40)
    ref = oracle.beam_select(logits.numpy(), scores, beams, select, lengths, finished, 3, 1.0)
    got = tv.beam_select(logits.cuda(), torch.from_numpy(scores).cuda(), beams=beams, select=select,
                         lengths=torch.from_numpy(lengths.astype(np.int32)).cuda(),
                         finished=torch.from_numpy(finished).cuda(), end_token=3, length_penalty=1.0)
    for b, want in enumerate(ref):
        assert got["parents"][b].tolist() == [c[1] for c in want] == list(range(b * beams, b * beams + select))
        assert got["scores"][b].tolist() == [c[2] for c in want]
        assert got["lengths"][b].tolist() == [c[3] for c in want]


def test_the_better_mean_first():
    """Next to equal means: a score that is one step of fp32 above or below."""
    ensure_built()
    lengths = np.array([49, 49, 49, 1, 98, 98], np.int32)
    scores = np.array([-49, np.nextafter(np.float32(-49), np.float32(0)), np.nextafter(np.float32(-49), np.float32(-50)),
                       -1, np.nextafter(np.float32(-98), np.float32(0)), -98], np.float32)
    got = tv.beam_select(torch.zeros(6, 9, device="cuda"), torch.from_numpy(scores).cuda(), beams=6,
                         lengths=torch.from_numpy(lengths).cuda(), finished=torch.ones(6, dtype=torch.int32, device="cuda"),
                         end_token=1, length_penalty=1.0)
    assert got["parents"][0].tolist() == [1, 4, 0, 3, 5, 2]
