"""What the chunk attention, the cache calls and the logit penalties make of
malformed batches: which sequences fail, which rows are written and which stay."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
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
