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


# ------------------------------------------------------------------ what a caller may hand over
def test_malformed_sequences_are_zeroed_and_reported():
    c = make([40, 50, 60, 33, 20], [8, 50, 1, 3, 20], 8, 2, 128, seed=1)
    good, st = call(c)
    assert (st == 0).all()

    def rows(b):
        return slice(int(c["off"][b]), int(c["off"][b + 1]))

    for kind, b in (("len", 0), ("max", 2), ("block", 3), ("page", 1)):
        bad = dict(c, lens=c["lens"].copy(), table=c["table"].copy())
        if kind == "len":
            bad["lens"][b] = 7          # shorter than its chunk
        if kind == "max":
            bad["lens"][b] = 61         # above max_len
        if kind == "block":
            bad["table"][b, 1] = -7
        if kind == "page":
            bad["table"][b, 3] = bad["k"].shape[0]
        got, st = call(bad, max_len=60, fill=5.0)
        assert st.tolist() == [5 if i == b else 0 for i in range(5)], kind
        assert (got[rows(b)] == 0).all()
        for i in range(5):
            if i != b:
                np.testing.assert_array_equal(got[rows(i)], good[rows(i)])
    # offsets: a chunk of negative length, and rows past the end
    for off in ([0, 8, 4, 5, 8, 28], [0, 8, 58, 59, 62, 200]):
        got, st = call(dict(c, off=np.asarray(off, np.int32)), max_len=60)
        assert (st == 5).any() and np.isfinite(got).all()


def test_decreasing_offsets_end_the_batch():
    """What comes after a chunk of negative length is malformed too: its rows
    would be counted twice.  The second batch, so counted, has a line of work of
    more than 2^31."""
    c = make([40, 50, 60, 33, 20], [8, 50, 1, 3, 20], 8, 2, 128, seed=1)
    good, _ = call(c)
    got, st = call(dict(c, off=np.asarray([0, 8, 58, 50, 53, 73], np.int32)), max_len=60, fill=5.0)
    assert st.tolist() == [0, 0, 5, 5, 5]
    np.testing.assert_array_equal(got[:58], good[:58])  # (some of these are rows of sequences 3 and 4 too)
    assert (got[58:73] == 0).all() and (got[73:] == 5.0).all()
    for B in (128, 600):
        n, top = 8192, 1 << 20
        pool = torch.zeros(1, 64, 16, 64, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(n, 64, 64, dtype=torch.bfloat16, device="cuda")
        table = torch.zeros(B, top // 16, dtype=torch.int32, device="cuda")
        off = torch.tensor([n * (b % 2) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        lens[2:] = top  # (the first sequence is sound: 8192 tokens over themselves)
        _, st = tv.chunk_attention(q, pool, pool, table, lens, off, max_len=top)
        assert st.tolist() == [0] + [5] * (B - 1)


def test_rows_behind_the_last_sequence_stay():
    c = make([30, 9], [5, 9], 4, 2, 64, seed=2, extra_rows=7)
    for dt in ("fp32", "bf16"):
        got, st = call(c, out_dtype=dt, fill=-3.0)
        assert (st == 0).all() and (got[14:] == -3.0).all() and (got[:14] != -3.0).any()
    c = make([30, 9], [0, 0], 4, 2, 64, seed=2, extra_rows=3)
    got, st = call(c, fill=-3.0)
    assert (st == 0).all() and (got == -3.0).all()


def test_no_rows_at_all():
    c = make([30, 9], [0, 0], 4, 2, 64, seed=2)
    got, st = call(c)
    assert got.shape == (0, 4, 64) and (st == 0).all()


def poisoned(c, window, sinks):
    """The cache with NaN in every place that no row of its sequence's chunk
    sees, and no page where a whole page is unseen."""
    out = dict(c, k=np.full_like(c["k"], np.nan), v=np.full_like(c["v"], np.nan),
               table=np.full_like(c["table"], -1))
    for b, n in enumerate(c["lens"]):
        first = int(n) - int(c["off"][b + 1] - c["off"][b])
        if first == n:
            continue
        for p in range(int(n)):
            if not window or p > first - window or p < sinks:
                blk = out["table"][b, p // 16] = c["table"][b, p // 16]
                out["k"][blk, :, p % 16] = c["k"][blk, :, p % 16]
                out["v"][blk, :, p % 16] = c["v"][blk, :, p % 16]
    return out


@pytest.mark.parametrize("window, sinks", [(0, 0), (1, 0), (50, 0), (50, 4), (130, 20), (300, 129)])
@pytest.mark.parametrize("d, group", [(64, 1), (128, 4)])
def test_unseen_places_do_not_matter(window, sinks, d, group):
    """Freed pages, stale page tails and evicted positions may hold NaN.  A
    chunk of one unit: a place that some row sees, others may not."""
    c = make([900, 33, 400, 131], [1, 5, 30, 1], 2 * group, 2, d, seed=window + sinks)
    bad = poisoned(c, window, sinks)
    a, st = call(c, window=window, sinks=sinks)
    b, st2 = call(bad, window=window, sinks=sinks)
    assert (st == 0).all() and (st2 == 0).all()
    np.testing.assert_array_equal(a, b)


def test_unseen_places_do_not_matter_fp8():
    c = quantised(make([900, 33, 400], [1, 5, 30], 4, 2, 128, seed=9))
    for window, sinks in ((0, 0), (50, 4)):
        a, _ = call_fp8(c, window=window, sinks=sinks)
        bad = dict(c, table=np.full_like(c["table"], -1))
        for k in ("k", "v"):
            bad[k + "_codes"] = np.full_like(c[k + "_codes"], 0x7F)
            bad[k + "_scale"] = np.full_like(c[k + "_scale"], np.nan)
        for b, n in enumerate(c["lens"]):
            first = int(n) - int(c["off"][b + 1] - c["off"][b])
            for p in range(int(n)):
                if not window or p > first - window or p < sinks:
                    blk = bad["table"][b, p // 16] = c["table"][b, p // 16]
                    for k in ("k_codes", "v_codes", "k_scale", "v_scale"):
                        bad[k][blk, :, p % 16] = c[k][blk, :, p % 16]
        got, st = call_fp8(bad, window=window, sinks=sinks)
        assert (st == 0).all()
        np.testing.assert_array_equal(a, got)


def test_a_query_scale_that_is_nan_shows():
    """The rows of that query are NaN, not weighted by something else; the rows
    of the others do not change."""
    c = quantised(make([200, 40], [70, 3], 4, 2, 128, seed=13))
    want, _ = call_fp8(c)
    bad = dict(c, q_scale=c["q_scale"].copy())
    hit = [(0, 1), (69, 3), (71, 0)]
    for t, h in hit:
        bad["q_scale"][t, h] = np.nan
    got, st = call_fp8(bad)
    assert (st == 0).all()
    for t, h in hit:
        assert np.isnan(got[t, h]).all()
        got[t, h] = want[t, h]
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("hq, hkv, d", [(256, 1, 64), (100, 1, 128), (129, 1, 64), (48, 16, 128)])
def test_groups_of_every_size(hq, hkv, d):
    """g = 256: one token per unit; 129: one token, two m-tiles; 3: 85 tokens."""
    c = make([150, 20], [90, 3], hq, hkv, d, seed=hq)
    got, st = call(c)
    assert (st == 0).all()
    check(got, c, U_BF16)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_softmax_scale(scale):
    """Flat and peaked rows; scores of large magnitude rescale the accumulators."""
    c = make([300, 60], [40, 60], 4, 2, 64, seed=4, std=2.0)
    got, st = call(c, softmax_scale=scale)
    assert (st == 0).all()
    check(got, c, U_BF16, scale=scale)


def test_growing_scores_rescale():
    """Keys that grow with their position: the running maximum moves by more
    than 2^8 many times."""
    c = make([1000], [70], 2, 1, 64, seed=5)
    ramp = np.linspace(0.1, 12, 1000)
    for p in range(1000):
        blk = c["table"][0, p // 16]
        row = np.full(64, ramp[p])
        c["k"][blk, :, p % 16] = wl.bf16_bits_to_f32(wl.to_bf16_bits(row))
    c["q"][:] = wl.bf16_bits_to_f32(wl.to_bf16_bits(np.abs(c["q"]) + 0.5))
    got, st = call(c)
    assert (st == 0).all()
    check(got, c, U_BF16)


def test_strided_queries_and_given_buffers():
    ensure_built()
    c = make([64, 200], [64, 9], 8, 2, 128, seed=6)
    qkv = torch.randn(73, 12, 128, device="cuda").to(torch.bfloat16)
    qkv[:, :8] = dev(c["q"], torch.bfloat16)
    rest = [dev(c[k], torch.bfloat16) for k in ("k", "v")] + [dev(c[k]) for k in ("table", "lens", "off")]
    want, _ = tv.chunk_attention(qkv[:, :8].contiguous(), *rest, max_len=200)
    out = torch.empty(73, 8, 128, dtype=torch.bfloat16, device="cuda")
    st = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    prm = tv.chunk_params(qkv[:, :8], rest[0], rest[2], rest[3], max_len=200)
    assert prm.q_stride == 12 * 128
    ws = torch.full((tv.chunk_workspace_size(prm),), 0xFF, dtype=torch.uint8, device="cuda")
    got, st2 = tv.chunk_attention(qkv[:, :8], *rest, max_len=200, out=out, status=st, workspace=ws)
    assert got is out and st2 is st and torch.equal(got, want) and (st == 0).all()
    with pytest.raises(tv.TVError):
        tv.chunk_attention(qkv[:, :8], *rest, max_len=200, workspace=ws[:-256])
    for bad in (qkv[:, 1:9, :64], qkv[:, :8].transpose(0, 1), qkv[:, :8].float(), qkv[:, ::2][:, :4]):
        with pytest.raises((ValueError, tv.TVError)):
            tv.chunk_attention(bad, *rest, max_len=200)
    with pytest.raises(ValueError):
        tv.chunk_attention(qkv[:, :8], rest[0], rest[1].float(), *rest[2:], max_len=200)
    with pytest.raises(ValueError):
        tv.chunk_attention(qkv[:, :8], *rest[:3], rest[3].long(), rest[4], max_len=200)
    with pytest.raises(tv.TVError):
        tv.chunk_attention(qkv[:, :8], *rest, max_len=400)  # more pages than a table row has


def test_side_stream_and_graphs():
    """A call on another stream, and two captured graphs with workspaces of
    their own replayed at once and again on new inputs."""
    ensure_built()
    a, b = make([700, 30], [1, 30], 8, 2, 128, seed=7), make([90, 2000], [40, 1], 8, 2, 128, seed=8)
    graphs, outs, args, want = [], [], [], []
    for c in (a, b):
        t = [dev(c[k], torch.bfloat16) for k in ("q", "k", "v")] + [dev(c[k]) for k in ("table", "lens", "off")]
        want.append(tv.chunk_attention(*t, max_len=2000 if c is b else 700)[0].clone())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got, _ = tv.chunk_attention(*t, max_len=2000 if c is b else 700, stream=side)
        side.synchronize()
        assert torch.equal(got, want[-1])
        prm = tv.chunk_params(t[0], t[1], t[3], t[4], max_len=2000 if c is b else 700)
        ws = torch.empty(tv.chunk_workspace_size(prm), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = tv.chunk_attention(*t, max_len=2000 if c is b else 700, workspace=ws)
        graphs.append(g), outs.append(out), args.append((t, ws))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        for s, g in ((s1, graphs[0]), (s2, graphs[1])):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()
    args[0][0][0].mul_(0.5)  # the graph reads its inputs anew
    graphs[0].replay()
    fresh, _ = tv.chunk_attention(*args[0][0], max_len=700)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fresh) and not torch.equal(fresh, want[0])


def test_blocks_past_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^31 (and 2^32)."""
    ensure_built()
    hkv, d, blocks = 1, 128, 1_200_000  # 2.46e9 elements, 4.9 GB a pool
    small = make([50, 700], [3, 1], 4, hkv, d, seed=11)
    n = small["k"].shape[0]
    ids = (blocks - 1 - 3 * np.arange(n)).astype(np.int32)
    pools = [torch.empty(blocks, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for pool, x in zip(pools, (small["k"], small["v"])):
        pool[torch.from_numpy(ids).long().cuda()] = dev(x, torch.bfloat16)
    table = np.where(small["table"] >= 0, ids[np.maximum(small["table"], 0)], -1)
    out, st = tv.chunk_attention(dev(small["q"], torch.bfloat16), *pools, dev(table), dev(small["lens"]),
                                 dev(small["off"]), max_len=700, out_dtype="fp32")
    assert (st == 0).all()
    want, _ = call(small)
    np.testing.assert_array_equal(out.cpu().numpy(), want)
