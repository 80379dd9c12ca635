"""The precision of chunk attention over an E4M3 cache.

V is fp16: the fp32 product of code and scale, rounded once (2^-11 of the
value).  P is fp16 (2^-11 of itself, or 2^-25 of the largest weight, once it is
subnormal) and the row sum adds the rounded weights.  So an fp32 output moves by
at most (3 x 2^-11 + 2 x keys x 2^-25) max|v|; S, the softmax and O are fp32,
below 1e-5 of max|v|."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from test_gpu_chunk import call_fp8, dev, make, quantised
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

ROUNDINGS = 3 * 2.0 ** -11


def bound(c):
    return ROUNDINGS + 2.0 * int(c["lens"].max()) * 2.0 ** -25 + 1e-5


def check(got, c, window=0, sinks=0, scale=None):
    ref = oracle.chunk_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["off"], window, sinks, scale)
    assert np.isfinite(got).all()
    for b in range(len(c["lens"])):
        r = slice(int(c["off"][b]), int(c["off"][b + 1]))
        pages = c["table"][b, : -(-int(c["lens"][b]) // 16)]
        big = np.abs(c["v"][pages]).max(initial=0)
        assert np.abs(got[r] - ref[r]).max(initial=0) <= bound(c) * big, b


def test_v_is_rounded_once():
    """One key a sequence: its V comes back, code x scale in fp32 rounded to
    fp16, as the tree attention takes it; scales of 2^-30 to 2^7."""
    n = 600
    c = quantised(make([1] * n, [1] * n, 4, 2, 128, seed=3))
    g = np.random.default_rng(0)
    c["v_codes"] = g.integers(0, 127, c["v_codes"].shape).astype(np.uint8) | (g.integers(0, 2, c["v_codes"].shape) << 7).astype(np.uint8)
    c["v_scale"] = ((1 + g.random(c["v_scale"].shape)) * 2.0 ** g.integers(-30, 7, c["v_scale"].shape)).astype(np.float32)
    got, st = call_fp8(c)
    assert (st == 0).all()
    for b in range(n):
        blk = c["table"][b, 0]
        codes = oracle.e4m3_table()[c["v_codes"][blk, :, 0]].astype(np.float32)
        v = (codes * c["v_scale"][blk, :, 0, None]).astype(np.float16).astype(np.float32)
        np.testing.assert_array_equal(got[b], np.repeat(v, 2, 0))


@pytest.mark.parametrize("lens, tokens, hq, hkv", [([20011, 4097, 9000], [1, 1, 65], 8, 1), ([33000], [1], 16, 2),
                                                   ([8192, 8193, 12001, 2], [1, 1, 1, 1], 32, 4), ([16400], [300], 4, 1)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (4099, 5)])
def test_long_caches_are_split_and_merged(lens, tokens, hq, hkv, window, sinks):
    c = quantised(make(lens, tokens, hq, hkv, 128, seed=len(lens)))
    got, st = call_fp8(c, window=window, sinks=sinks)
    assert (st == 0).all()
    check(got, c, window, sinks)
    again, _ = call_fp8(c, window=window, sinks=sinks)
    np.testing.assert_array_equal(got, again)


def test_one_value_in_verification_and_in_decode():
    """A cached token's V weighs the same in a plain decode step and as the
    prefix of a tree of one node, bit for bit where one key has all the weight."""
    c = quantised(make([17], [1], 4, 2, 128, seed=5))
    c["q_codes"][:] = 0x38                      # 1.0
    c["q_scale"][:] = 1.0
    c["k_codes"][:] = 0xB8                      # -1.0: a score of -128
    c["k_scale"][:] = 8.0
    blk = c["table"][0, 0]
    c["k_codes"][blk, :, 3] = 0x38              # 128 x 8 at key 3
    codes, scale = dev(c["q_codes"]), dev(c["q_scale"])
    pools = [dev(c[k]) for k in ("k_codes", "k_scale", "v_codes", "v_scale")]
    out, st = tv.chunk_attention_fp8(codes, scale, *pools, dev(c["table"]), dev(c["lens"]), dev(c["off"]), max_len=17,
                                     out_dtype="fp32")
    v = oracle.e4m3_table()[c["v_codes"][blk, :, 3]].astype(np.float32) * c["v_scale"][blk, :, 3, None]
    np.testing.assert_array_equal(out.cpu().numpy()[0], np.repeat(v.astype(np.float16).astype(np.float32), 2, 0))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    node = torch.full((1, 2, 128), 0xB8, dtype=torch.uint8, device="cuda")
    eight = torch.full((1, 2), 8.0, device="cuda")
    tree, st2 = tv.tree_attention_fp8(codes, scale, *pools, dev(c["table"]), node, eight, node, eight, i32([-1]), i32([16]),
                                      i32([0, 1]), max_nodes=1, max_prefix_len=16, out_dtype="fp32")
    assert st.tolist() == [0] and st2.tolist() == [0]
    torch.testing.assert_close(tree, out, rtol=0, atol=0)
