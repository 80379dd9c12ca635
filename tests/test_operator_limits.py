"""The largest calls that the chunk attention takes and the smallest that it
refuses, by the host's count of its work (no GPU needed)."""
import pytest

import speculative_decoding_tree_attention_gb300 as tv
from speculative_decoding_tree_attention_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return tv.load()


@pytest.mark.parametrize("tokens, ok", [(2 ** 19, True), (2 ** 20, False)])
def test_a_whole_prompt(tokens, ok):
    p = tv.ChunkParams(1, 64, 8, 128, 16, tokens // 16, tokens // 16, tokens, tokens, 0, 0, 0, 0.0, 0)
    assert (tv.chunk_workspace_size(p) > 0) == ok


@pytest.mark.parametrize("batch, length", [(4096, 2 ** 17), (16, 2 ** 20), (1, 2 ** 24)])
def test_decode_of_long_sequences(batch, length):
    p = tv.ChunkParams(batch, 64, 8, 128, 16, length // 16, 2 ** 20, batch, length, 0, 0, 0, 0.0, 0)
    assert tv.chunk_workspace_size(p) > 0


def test_a_window_shortens_the_work():
    p = tv.ChunkParams(1, 64, 8, 128, 16, 2 ** 16, 2 ** 16, 2 ** 20, 2 ** 20, 4096, 4, 0, 0.0, 0)
    assert tv.chunk_workspace_size(p) > 0
