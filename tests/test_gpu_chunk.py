"""GPU parity of tv_chunk_attention and tv_chunk_attention_fp8 against fp64.

Tolerances.  bf16 inputs are exact; S, the softmax and O are fp32 (their
error is below 1e-5 of the row's largest |v| at these lengths).  Each weight
P is rounded to 16 bits once, by at most u = eps/2 of itself (bf16 2^-8, fp16
2^-11), and the row sum adds the rounded weights, so an fp32 output moves by
at most 2 u max|v| over the keys of the row (u from the numerator, u from the
sum).  An E4M3 cache adds two fp16 roundings of each v (its scale, the
product; 2^-11 each) to the two of P in fp16: 4 x 2^-11 max|v|.  The bf16 output is the fp32 one rounded once (checked bit
for bit)."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from speculative_decoding_tree_attention_gb300 import workloads as wl
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

SLACK = 1e-5


def make(lens, chunks, hq, hkv, d, seed=0, extra_rows=0, std=1.0):
    """A ragged batch over shuffled pages: real values (exact in bf16)."""
    g = np.random.default_rng(seed)
    nblk = [-(-n // 16) for n in lens]
    total = max(1, sum(nblk))
    perm = g.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, max(nblk))), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n

    def bf16(*shape):
        return wl.bf16_bits_to_f32(wl.to_bf16_bits(g.standard_normal(shape) * std))

    off = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    return dict(q=bf16(int(off[-1]) + extra_rows, hq, d), k=bf16(total, hkv, 16, d), v=bf16(total, hkv, 16, d),
                table=table, lens=np.asarray(lens, np.int32), off=off, hq=hq, hkv=hkv, d=d)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def call(c, out_dtype="fp32", fill=None, **kw):
    ensure_built()
    args = [dev(c[k], torch.bfloat16) for k in ("q", "k", "v")] + [dev(c[k]) for k in ("table", "lens", "off")]
    kw.setdefault("max_len", max(1, int(c["lens"].max())))
    if fill is not None:
        kw["out"] = torch.full(c["q"].shape, fill, device="cuda",
                               dtype=torch.float32 if out_dtype == "fp32" else torch.bfloat16)
    out, st = tv.chunk_attention(*args, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), st.cpu().numpy()


def quantised(c):
    out = dict(c)
    for k in ("q", "k", "v"):
        codes, scale = wl.quantize_e4m3_rows(c[k])
        out[k + "_codes"], out[k + "_scale"] = codes, scale
        out[k] = oracle.e4m3_table()[codes] * scale.astype(np.float64)[..., None]
    return out


def call_fp8(c, out_dtype="fp32", **kw):
    ensure_built()
    args = []
    for k in ("q", "k", "v"):
        args += [dev(c[k + "_codes"]), dev(c[k + "_scale"])]
    args += [dev(c[k]) for k in ("table", "lens", "off")]
    kw.setdefault("max_len", max(1, int(c["lens"].max())))
    out, st = tv.chunk_attention_fp8(*args, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), st.cpu().numpy()


def check(got, c, u, window=0, sinks=0, scale=None):
    """Every row within u x max|v| (over the sequence) of fp64."""
    ref = oracle.chunk_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["off"], window, sinks, scale)
    assert np.isfinite(got).all()
    for b in range(len(c["lens"])):
        r = slice(int(c["off"][b]), int(c["off"][b + 1]))
        if r.start == r.stop:
            continue
        pages = c["table"][b, : -(-int(c["lens"][b]) // 16)]
        big = np.nanmax(np.abs(np.where(np.isfinite(c["v"][pages]), c["v"][pages], 0)))
        err = np.abs(got[r] - ref[r]).max()
        assert err <= u * big + SLACK * big, f"sequence {b}: {err:.3e} > {u * big:.3e}"


U_BF16 = 2 * 2.0 ** -8
U_FP8 = 4 * 2.0 ** -11

SHAPES = [
    # lens, chunks, hq, hkv, d
    ([1], [1], 1, 1, 64),                                   # one token, one key
    ([1, 2, 15, 16, 17], [1, 1, 1, 1, 1], 4, 4, 64),        # page borders
    ([127, 128, 129, 255, 257], [1, 1, 1, 1, 1], 8, 1, 128),  # tile borders
    ([200], [200], 4, 4, 128),                              # a whole prompt, two m-tiles
    ([300, 40, 0, 513], [300, 7, 0, 256], 7, 1, 128),       # g = 7: units of 36 tokens
    ([130, 131, 700], [129, 1, 3], 6, 2, 64),
    ([900], [1], 32, 8, 128),                               # a decode token split over many CTAs
    ([2500, 1, 33], [37, 1, 33], 16, 2, 128),
]


@pytest.mark.parametrize("lens, chunks, hq, hkv, d", SHAPES)
def test_causal(lens, chunks, hq, hkv, d):
    c = make(lens, chunks, hq, hkv, d, seed=len(lens) + hq)
    got, st = call(c)
    assert (st == 0).all()
    check(got, c, U_BF16)
    g16, _ = call(c, out_dtype="bf16")
    np.testing.assert_array_equal(wl.to_bf16_bits(got), wl.to_bf16_bits(g16))


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (127, 17), (128, 130),
                                           (129, 1), (300, 4), (1000, 300), (100000, 4), (7, 100000)])
def test_window_and_sinks(window, sinks):
    c = make([700, 60, 901, 1], [150, 60, 1, 1], 6, 2, 64, seed=window)
    got, st = call(c, window=window, sinks=sinks)
    assert (st == 0).all()
    check(got, c, U_BF16, window, sinks)


@pytest.mark.parametrize("lens, chunks, hq, hkv", [
    ([1], [1], 1, 1), ([17, 128, 129, 300], [1, 128, 5, 1], 4, 2), ([600, 0, 77], [290, 0, 3], 7, 1),
    ([1500], [1], 32, 8)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (33, 4)])
def test_fp8(lens, chunks, hq, hkv, window, sinks):
    c = quantised(make(lens, chunks, hq, hkv, 128, seed=hq))
    got, st = call_fp8(c, window=window, sinks=sinks)
    assert (st == 0).all()
    check(got, c, U_FP8, window, sinks)


def mixed_batch(B, hq, hkv, d, seed, longest=700):
    """Many sequences: decode tokens, short chunks and prompts in random order,
    so that a CTA gets whole and split units of one and of two m-tiles in turn."""
    g = np.random.default_rng(seed)
    chunks = [int(g.choice([0, 1, 1, 1, g.integers(2, 40), g.integers(40, 300)])) for _ in range(B)]
    lens = [c + int(g.integers(0, longest)) for c in chunks]
    return make(lens, chunks, hq, hkv, d, seed)


@pytest.mark.parametrize("B, hq, hkv, d", [(300, 8, 4, 64), (200, 8, 8, 128), (400, 16, 2, 128), (40, 28, 4, 128)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (130, 4)])
def test_many_units_per_cta(B, hq, hkv, d, window, sinks):
    c = mixed_batch(B, hq, hkv, d, B + window)
    got, st = call(c, window=window, sinks=sinks)
    assert (st == 0).all()
    check(got, c, U_BF16, window, sinks)
    for _ in range(3):  # a race would not repeat itself
        again, _ = call(c, window=window, sinks=sinks)
        np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("window, sinks", [(0, 0), (130, 4)])
def test_many_units_per_cta_fp8(window, sinks):
    c = quantised(mixed_batch(250, 16, 4, 128, 5))
    got, st = call_fp8(c, window=window, sinks=sinks)
    assert (st == 0).all()
    check(got, c, U_FP8, window, sinks)
    for _ in range(3):
        again, _ = call_fp8(c, window=window, sinks=sinks)
        np.testing.assert_array_equal(got, again)


def test_long_decode_is_split_and_merged():
    c = make([20011, 4097, 9000], [1, 1, 65], 8, 1, 128, seed=3)
    got, st = call(c)
    assert (st == 0).all()
    check(got, c, U_BF16)
