"""The precision of chunk attention over an E4M3 cache.

V is fp16: the fp32 product of code and scale, rounded once (2^-11 of the
value).  P is fp16, its largest entries between 2^7 and 2^15: a weight is off by
2^-11 of itself, or, once it is subnormal there, by 2^-25 of 2^7, which is 2^-32
of the largest weight.  The row sum adds the rounded weights.  So an fp32 output
moves by at most (3 x 2^-11 + 2 x keys x 2^-32) max|v|; S, the softmax and O are
fp32, below 1e-5 of max|v|."""
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
    return ROUNDINGS + 2.0 * int(c["lens"].max()) * 2.0 ** -32 + 1e-5


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


@pytest.mark.parametrize("hq", [8, 160])
@pytest.mark.parametrize("at", [0, 65000, 131072])
def test_one_key_outweighs_many(hq, at):
    """A key whose weight is e^17.5 times that of each of 131072 others: what
    they add up to, 3.3e-3 of the whole, is not lost.  So many sequences (over the
    same pages) that a CTA takes whole units, against one running maximum."""
    ensure_built()
    n, B = 131073, 304
    c = make([n], [1], hq, 1, 128, seed=1)
    c["q"][:] = 0.0
    c["q"][:, :, 0] = 1.0
    c["k"][:] = 0.0
    c["k"][c["table"][0, at // 16], 0, at % 16, 0] = 17.5
    c["v"][:] = 1.0
    c["v"][c["table"][0, at // 16], 0, at % 16] = 0.0
    c = quantised(c)
    c = dict(c, table=np.repeat(c["table"], B, 0), lens=np.repeat(c["lens"], B), off=np.arange(B + 1, dtype=np.int32),
             q_codes=np.repeat(c["q_codes"], B, 0), q_scale=np.repeat(c["q_scale"], B, 0))
    got, st = call_fp8(c, softmax_scale=1.0)
    assert (st == 0).all()
    w = 131072 * np.exp(-17.5)
    assert np.abs(got - w / (1.0 + w)).max() <= bound(c)


@pytest.mark.parametrize("std, scale", [(2.0, None), (1.0, 1.0), (4.0, 0.3)])
@pytest.mark.parametrize("tokens", [1, 70])
def test_peaked_rows(std, scale, tokens):
    c = quantised(make([3000, 401], [tokens, tokens], 8, 2, 128, seed=7, std=std))
    got, st = call_fp8(c, **({} if scale is None else dict(softmax_scale=scale)))
    assert (st == 0).all()
    check(got, c, scale=scale)


@pytest.mark.parametrize("log2", [20, 24, 25, 26])
def test_scores_of_large_magnitude(log2):
    """Scores near 2^log2 that differ by a few units, larger and larger ones: the
    rows stay weighted means of V, though fp32 scores no longer say which."""
    n = 1000
    c = quantised(make([n, 400], [3, 200], 4, 2, 128, seed=2))
    g = np.random.default_rng(log2)
    c["q_codes"][:], c["k_codes"][:] = 0, 0
    c["q_codes"][:, :, 0], c["q_codes"][:, :, 1] = 0x7E, 0x01   # 448 and 2^-9
    c["k_codes"][:, :, :, 0] = 0x7E
    for b, m in enumerate((n, 400)):
        for p in range(m):  # S = 448^2 + 2^-9 x (8 .. 448), in fp32 in steps of 2^-6
            c["k_codes"][c["table"][b, p // 16], :, p % 16, 1] = 0x50 + min(0x2E, p // 20 + int(g.integers(0, 4)))
    c["q_scale"][:] = 1.0
    c["k_scale"][:] = 2.0 ** log2 / 448.0 ** 2
    got, st = call_fp8(c, softmax_scale=float(np.log(2.0)))
    assert (st == 0).all() and np.isfinite(got).all()
    big = np.abs(c["v"]).max()
    assert np.abs(got).max() <= big * (1 + 2.0 ** -10) and (np.abs(got).max(-1) > 0).all()


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
