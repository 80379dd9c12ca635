"""GPU parity of the cache writes and reads (tv_append_kv, tv_append_kv_fp8,
tv_read_kv_fp8, tv_quantize_rows, tv_commit_kv_fp8) against the oracle: codes,
scales, copies and statuses match bit for bit; a read is one fp32 product
rounded to bf16, computed here in numpy the same way."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from speculative_decoding_tree_attention_gb300 import workloads as wl
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def bf16(x):
    """Real values -> (bf16 tensor on the GPU, the same values in fp64)."""
    bits = wl.to_bf16_bits(x)
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    return t, wl.bf16_bits_to_f32(bits).astype(np.float64)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def rows_of_every_kind(n, heads, d, seed):
    """Rows of many magnitudes, with ties at code borders, zeros, tiny and huge ones."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, heads, d)) * 2.0 ** g.integers(-20, 20, (n, heads, 1))
    flat = x.reshape(-1, d)
    for r in range(0, len(flat), 5):
        # eighths of the largest over 7: quotients on and next to the middles
        flat[r] = g.integers(-448, 449, d) / 64.0 * 2.0 ** g.integers(-8, 8)
    if len(flat) > 4:
        flat[1] = 0.0
        flat[2] *= 1e-38 / np.abs(flat[2]).max()
        flat[3] *= 3e38 / np.abs(flat[3]).max()
        flat[4, ::3] = -0.0
    return x


@pytest.mark.parametrize("n, heads, d", [(1, 1, 64), (1, 1, 128), (37, 3, 64), (301, 8, 128)])
def test_quantize_rows(n, heads, d):
    ensure_built()
    t, x = bf16(rows_of_every_kind(n, heads, d, n + d))
    codes, scale = tv.quantize_rows(t)
    want, want_scale = oracle.quantize_rows(x)
    np.testing.assert_array_equal(scale.cpu().numpy(), want_scale)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)


def test_quantize_all_bf16_mantissas_against_every_largest():
    """Every 8-bit mantissa in units of every row maximum (all ties that bf16
    inputs can make), at normal and subnormal codes."""
    ensure_built()
    m = np.arange(128, 256).astype(np.float64)
    rows = []
    for amax in m:
        for e in (0, -3, -7, -9):
            rows.append(np.concatenate([[amax], (m * 2.0 ** e)[:127]]))
            rows.append(np.concatenate([[amax * 2.0 ** 9], m[1:]]))
    t, x = bf16(np.array(rows)[:, None, :])
    codes, scale = tv.quantize_rows(t)
    want, want_scale = oracle.quantize_rows(x)
    np.testing.assert_array_equal(scale.cpu().numpy(), want_scale)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)


def test_quantize_special_values():
    ensure_built()
    x = np.random.default_rng(0).standard_normal((4, 1, 128))
    x[0, 0, 5], x[1, 0, 7], x[1, 0, 9] = np.nan, np.inf, -np.inf
    x[2] = np.nan
    x[3] = np.inf
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    codes, scale = tv.quantize_rows(t)
    codes, scale = codes.cpu().numpy(), scale.cpu().numpy()
    want, want_scale = oracle.quantize_rows(t.double().cpu().numpy())
    np.testing.assert_array_equal(scale, want_scale)
    np.testing.assert_array_equal(codes, want)
    assert codes[0, 0, 5] == 0x7F and codes[1, 0, 7] == 0x7E and codes[1, 0, 9] == 0xFE
    assert (codes[2] == 0x7F).all() and scale[2] == 1 and (codes[3] == 0x7E).all()


def batch(lens, chunks, seed, width=None, extra=2):
    g = np.random.default_rng(seed)
    nblk = [-(-max(n, 1) // 16) for n in lens]
    total = sum(nblk) + extra
    perm = g.permutation(total).astype(np.int32)
    table = np.full((len(lens), width or max(nblk)), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, np.asarray(lens, np.int32), np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32), total


BATCHES = [([1], [1]), ([16, 17, 40], [1, 1, 3]), ([33, 0, 700, 5], [33, 0, 259, 5]),
           (list(range(1, 41)), [1] * 40), ([1000], [999])]


@pytest.mark.parametrize("lens, chunks", BATCHES)
@pytest.mark.parametrize("hkv, d, fp8", [(2, 128, True), (3, 64, True), (8, 128, False), (1, 64, False)])
def test_append(lens, chunks, hkv, d, fp8):
    ensure_built()
    table, seq, off, blocks = batch(lens, chunks, len(lens) + hkv)
    total = int(off[-1]) + 3  # rows of no sequence
    kt, k = bf16(rows_of_every_kind(total, hkv, d, 1))
    vt, v = bf16(rows_of_every_kind(total, hkv, d, 2))
    args = (kt, vt, i32(table), i32(seq), i32(off))
    status, places, _ = oracle.cache_places(table, seq, off, blocks, total)
    shape = (blocks, hkv, 16, d)
    if fp8:
        pools = [torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.full(shape[:3], 9.0, device="cuda") for _ in range(2)]
        st = tv.append_kv_fp8(*args, pools[0], scales[0], pools[1], scales[1])
        for x, pool, sc in ((k, pools[0], scales[0]), (v, pools[1], scales[1])):
            codes, scale = oracle.quantize_rows(x)
            want, want_s = np.full(shape, 0xA5, np.uint8), np.full(shape[:3], 9.0, np.float32)
            for r, (blk, at) in places.items():
                want[blk, :, at], want_s[blk, :, at] = codes[r], scale[r]
            np.testing.assert_array_equal(pool.cpu().numpy(), want)
            np.testing.assert_array_equal(sc.cpu().numpy(), want_s)
    else:
        pools = [torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        st = tv.append_kv(*args, *pools)
        for x, pool in ((k, pools[0]), (v, pools[1])):
            want = np.full(shape, 3.0)
            for r, (blk, at) in places.items():
                want[blk, :, at] = x[r]
            np.testing.assert_array_equal(pool.double().cpu().numpy(), want)
    np.testing.assert_array_equal(st.cpu().numpy(), status)


def test_append_strided_rows():
    """K and V as slices of a fused projection [token][(Hq + 2 Hkv) D]."""
    ensure_built()
    table, seq, off, blocks = batch([40, 19], [40, 3], 4)
    hq, hkv, d = 4, 2, 128
    qkv = torch.randn(int(off[-1]), hq + 2 * hkv, d, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    got = [torch.zeros(blocks, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    tv.append_kv(k, v, i32(table), i32(seq), i32(off), *got[:2])
    tv.append_kv(k.contiguous(), v.contiguous(), i32(table), i32(seq), i32(off), *got[2:])
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3]) and got[0].abs().sum() > 0
    c1 = tv.quantize_rows(qkv[:, :hq])
    c2 = tv.quantize_rows(qkv[:, :hq].contiguous())
    assert torch.equal(c1[0], c2[0]) and torch.equal(c1[1], c2[1])


@pytest.mark.parametrize("lens, chunks", BATCHES)
@pytest.mark.parametrize("hkv, d", [(2, 128), (3, 64)])
def test_read(lens, chunks, hkv, d):
    ensure_built()
    g = np.random.default_rng(7)
    table, seq, off, blocks = batch(lens, chunks, len(lens))
    total = int(off[-1]) + 2
    shape = (blocks, hkv, 16, d)
    codes = [g.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
    scale = [(2.0 ** g.integers(-30, 30, shape[:3]) * g.random(shape[:3])).astype(np.float32) for _ in range(2)]
    outs = [torch.full((total, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    args = [torch.from_numpy(x).cuda() for pair in zip(codes, scale) for x in pair]
    k, v, st = tv.read_kv_fp8(*args, i32(table), i32(seq), i32(off), k_out=outs[0], v_out=outs[1])
    status, places, _ = oracle.cache_places(table, seq, off, blocks, total)
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    for got, c, s in ((k, codes[0], scale[0]), (v, codes[1], scale[1])):
        want = np.full((total, hkv, d), 5.0, np.float32)
        with np.errstate(invalid="ignore"):
            values = oracle.e4m3_table().astype(np.float32)[c] * s[..., None]
        for r, (blk, at) in places.items():
            want[r] = values[blk, :, at]
        want = torch.from_numpy(want).to(torch.bfloat16)
        np.testing.assert_array_equal(got.float().cpu().numpy(), want.float().numpy())


def test_missing_pages_and_malformed_extents():
    """A failed sequence writes nothing and reads as zeros; the others are served."""
    ensure_built()
    lens, chunks = [40, 50, 10, 64, 30], [20, 30, 11, 64, 30]
    table, seq, off, blocks = batch(lens, chunks, 3, width=4)
    table[0, 1] = -1            # a page of the chunk is missing
    table[1, 0] = blocks        # before the chunk: not looked at (positions 20 .. 49)
    table[3, 3] = blocks + 5    # out of range
    total, hkv, d = int(off[-1]), 2, 128
    kt, k = bf16(np.random.default_rng(1).standard_normal((total, hkv, d)))
    shape = (blocks, hkv, 16, d)
    pools = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(shape[:3], device="cuda") for _ in range(2)]
    status, places, failed = oracle.cache_places(table, seq, off, blocks, total)
    assert status.tolist() == [7, 0, 5, 7, 0]
    cache = (pools[0], scales[0], pools[1], scales[1])
    st = tv.append_kv_fp8(kt, kt, i32(table), i32(seq), i32(off), *cache)
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    codes, scale = oracle.quantize_rows(k)
    want = np.zeros(shape, np.uint8)
    for r, (blk, at) in places.items():
        want[blk, :, at] = codes[r]
    np.testing.assert_array_equal(pools[0].cpu().numpy(), want)
    got, _, st = tv.read_kv_fp8(*cache, i32(table), i32(seq), i32(off), total_tokens=total)
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    assert (got[failed] == 0).all() and (got[sorted(places)].float().abs().sum((1, 2)) > 0).all()
    # offsets that are not non-decreasing: every sequence fails, nothing is touched
    for bad in ([0, 20, 10, 61, 125, 155], [-1, 20, 50, 61, 125, 155], [0, 20, 50, 61, 125, total + 1]):
        before = pools[0].clone()
        st = tv.append_kv_fp8(kt, kt, i32(table), i32(seq), i32(bad), *cache)
        assert (st.cpu().numpy() == 5).all() and torch.equal(before, pools[0])


def test_empty_call():
    ensure_built()
    table, seq, off, blocks = batch([5, 9], [0, 0], 1)
    pools = [torch.full((blocks, 2, 16, 64), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = tv.append_kv(none, none, i32(table), i32(seq), i32(off), *pools)
    assert (st == 0).all() and (pools[0] == 2).all()
    codes, scale = tv.quantize_rows(none)
    assert codes.shape == (0, 2, 64) and scale.shape == (0, 2)


@pytest.mark.parametrize("num", [2, 3])
def test_commit_fp8(num):
    """The E4M3 commit copies the codes and scales that the bf16 commit's rows
    would have: checked against the oracle's commit of the codes."""
    ensure_built()
    case = wl.make_case(wl.config(num, hkv=4, hq=4, prefix=(37, 90), batch=3), parts=("attn",))
    kp, vp, table = wl.extend_pool(case, 8)
    B, maxn = case["batch"], case["max_nodes"]
    off, par = case["node_offsets"], case["parent"]
    path, acc = np.full((B, maxn), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        cur = 0
        while acc[b] < 5 - b:
            kids = [v for v in range(1, off[b + 1] - off[b]) if par[off[b] + v] == cur]
            if not kids:
                break
            cur = path[b, acc[b]] = kids[-1]
            acc[b] += 1
    nodes = [tv.quantize_rows(torch.from_numpy(case[k].view(np.int16)).view(torch.bfloat16).cuda()) for k in ("k_nodes", "v_nodes")]
    shape = kp.shape
    g = np.random.default_rng(0)
    pools = [g.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
    scales = [g.random(shape[:3]).astype(np.float32) for _ in range(2)]
    dev = [torch.from_numpy(x).cuda() for pair in zip(pools, scales) for x in pair]
    new, st = tv.commit_kv_fp8(*nodes[0], *nodes[1], i32(par), i32(off), i32(acc), i32(path), i32(table),
                               i32(case["prefix_lens"]), *dev, max_nodes=maxn)
    assert (st == 0).all()
    np.testing.assert_array_equal(new.cpu().numpy(), case["prefix_lens"] + acc + 1)
    for (codes, scale), pool, sc, got, got_s in zip(nodes, pools, scales, dev[::2], dev[1::2]):
        want, want_s = pool.copy(), sc.copy()
        for b in range(B):
            for t, node in enumerate([0] + path[b, :acc[b]].tolist()):
                pos = case["prefix_lens"][b] + t
                want[table[b, pos // 16], :, pos % 16] = codes[off[b] + node].cpu().numpy()
                want_s[table[b, pos // 16], :, pos % 16] = scale[off[b] + node].cpu().numpy()
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        np.testing.assert_array_equal(got_s.cpu().numpy(), want_s)


def test_blocks_past_32_bit_offsets():
    """Writing to and reading from pages whose offsets pass 2^31 and 2^32."""
    ensure_built()
    hkv, d, blocks = 2, 128, 1_060_000  # 4.3e9 codes a pool
    k_pool, v_pool = (torch.empty(blocks, hkv, 16, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.empty(blocks, hkv, 16, device="cuda") for _ in range(2))
    table = i32([[blocks - 1, 3, blocks - 7]])
    lens, off = i32([45]), i32([0, 45])
    kt, k = bf16(np.random.default_rng(0).standard_normal((45, hkv, d)))
    vt, v = bf16(np.random.default_rng(1).standard_normal((45, hkv, d)))
    st = tv.append_kv_fp8(kt, vt, table, lens, off, k_pool, k_scale, v_pool, v_scale)
    back_k, back_v, st2 = tv.read_kv_fp8(k_pool, k_scale, v_pool, v_scale, table, lens, off, total_tokens=45)
    assert st.item() == 0 and st2.item() == 0
    for x, got in ((k, back_k), (v, back_v)):
        codes, scale = oracle.quantize_rows(x)
        want = torch.from_numpy((oracle.e4m3_table()[codes].astype(np.float32) * scale[..., None])).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    wide = torch.empty(blocks, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    st = tv.append_kv(kt, vt, table, lens, off, wide, wide.clone())
    assert st.item() == 0
    assert torch.equal(wide[blocks - 1].transpose(0, 1), kt[:16]) and torch.equal(wide[blocks - 7].transpose(0, 1)[:13], kt[32:])


def test_side_stream_and_graph():
    ensure_built()
    table, seq, off, blocks = batch([40, 19], [40, 3], 4)
    x = torch.randn(43, 2, 128, device="cuda").to(torch.bfloat16)
    pools = [torch.zeros(blocks, 2, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    scales = [torch.zeros(blocks, 2, 16, device="cuda") for _ in range(4)]
    args = (x, x, i32(table), i32(seq), i32(off))
    tv.append_kv_fp8(*args, pools[0], scales[0], pools[1], scales[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tv.append_kv_fp8(*args, pools[2], scales[2], pools[3], scales[3], stream=side)
    side.synchronize()
    assert torch.equal(pools[0], pools[2]) and torch.equal(scales[1], scales[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tv.append_kv_fp8(*args, pools[2], scales[2], pools[3], scales[3])
        k, _, _ = tv.read_kv_fp8(pools[2], scales[2], pools[3], scales[3], *args[2:], total_tokens=43)
    x.mul_(3.0)
    g.replay()
    tv.append_kv_fp8(*args, pools[0], scales[0], pools[1], scales[1])
    want, _, _ = tv.read_kv_fp8(pools[0], scales[0], pools[1], scales[1], *args[2:], total_tokens=43)
    assert torch.equal(k, want)


def test_binding_refuses_bad_tensors():
    ensure_built()
    table, seq, off, blocks = batch([40], [40], 4)
    k = torch.zeros(40, 2, 128, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(blocks, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    at = (i32(table), i32(seq), i32(off))
    for args in ((k.float(), k, *at, pool, pool), (k, k[:39], *at, pool, pool), (k[:, :1], k[:, :1], *at, pool, pool),
                 (k, k, i32(table).long(), *at[1:], pool, pool), (k, k, *at, pool, pool[:, :1]),
                 (k, k, at[0], at[1], i32([0]), pool, pool), (k, k, *at, pool, pool.cpu()),
                 (k.transpose(0, 1), k, *at, pool, pool), (k, torch.zeros(40, 4, 128, dtype=torch.bfloat16, device="cuda")[:, :2], *at, pool, pool),
                 (k, k, *at, pool.float(), pool.float())):
        with pytest.raises(ValueError):
            tv.append_kv(*args)
    with pytest.raises(ValueError):
        tv.read_kv_fp8(pool.to(torch.uint8), pool[..., 0].float(), pool.to(torch.uint8), pool[..., 0].float(), *at)
    with pytest.raises(ValueError):
        tv.append_kv(k, k, *at, pool, pool, stream=7)
