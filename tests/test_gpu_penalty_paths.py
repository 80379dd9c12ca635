"""Penalties of drafted tokens alone: in a part of the vocabulary that neither
a history nor a bias touches, a path's tokens are rewritten right behind the
copy of their row."""
import numpy as np
import pytest
import torch

from test_gpu_penalty import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [2048, 8192, 8197])
@pytest.mark.parametrize("dtype", ["fp32", "in place", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
def test_paths_where_nothing_else_is_touched(vocab, dtype, masked):
    c = make([200, 64, 3], vocab, [0, 0, 0], vocab, masked=masked, chain=True)
    g = np.random.default_rng(vocab)
    # repeated, at the ends of the copy's blocks, and all over the vocabulary
    pool = np.concatenate([[0, 127, 128, 511, 512, 1023, 1024, vocab - 1], g.integers(0, vocab, 60)])
    c["draft_tokens"] = g.choice(pool, c["draft_tokens"].shape).astype(np.int32)
    c["logits"] = torch.from_numpy(c["logits"]).to(torch.bfloat16).float().numpy()
    want = None
    for _ in range(5):  # (an order between lanes that only mostly holds would not repeat itself)
        x = dict(c)
        if dtype == "bf16":
            x["logits"] = torch.from_numpy(c["logits"]).to(torch.bfloat16).view(torch.int16).numpy()
        got, st = call(x, in_place=dtype == "in place")
        assert (st == 0).all()
        want = got if want is None else want
        np.testing.assert_array_equal(got, want)
    check(want, c)


def test_the_history_touches_one_chunk_and_the_path_another():
    """A chunk of 2048 entries with touched entries beside one without, in place."""
    c = make([300], 6000, [50], 1, chain=True)
    c["history"] = np.random.default_rng(0).integers(2048, 4096, c["history"].shape).astype(np.int32)
    c["draft_tokens"] = np.random.default_rng(1).integers(0, 6000, c["draft_tokens"].shape).astype(np.int32)
    for in_place in (False, True):
        got, st = call(c, in_place=in_place)
        assert st.tolist() == [0]
        check(got, c)
