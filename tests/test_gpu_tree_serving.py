"""Verification of draft trees over a cache whose pages are given and taken back, as a
serving loop runs it: pages for the longest path (alloc_pages), the nodes' queries and keys
normed and turned by prefix length + depth (rotate_qk), tree_attention, accept, commit_kv,
and the pages that the accepted path left unused taken back (free_pages), for a bf16 and an
E4M3 cache; on the way a sequence ends and another takes its place, and the pool is
compacted.  Rotated rows and attention are compared with fp64, the cache with the rows
that were committed, the counts with the tables, after every step."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, V, N = 3, 8, 2, 128, 211, 24
WIDTH, PAGES, STEPS = 9, 30, 12


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def real(t, scale=None):
    if scale is None:
        return t.double().cpu().numpy()
    return oracle.e4m3_table()[t.cpu().numpy()] * scale.double().cpu().numpy()[..., None]


@pytest.mark.parametrize("fp8", [False, True])
def test_verify_and_commit(fp8):
    ensure_built()
    g = np.random.default_rng(7 + fp8)
    gen = torch.Generator(device="cuda").manual_seed(7 + int(fp8))
    weight = 1 + 0.1 * torch.randn(2, D, device="cuda", generator=gen)
    freq = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    f = torch.from_numpy(freq).cuda()
    shape = (PAGES, HKV, 16, D)
    if fp8:
        cache = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda"), torch.full(shape[:3], float("nan"), device="cuda"),
                 torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda"), torch.full(shape[:3], float("nan"), device="cuda")]
    else:
        cache = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    lens = np.zeros(B, np.int32)
    held = [[] for _ in range(B)]  # each sequence's committed rows, (k, v) in fp64
    tol = (4 * 2.0 ** -11 if fp8 else 2 * 2.0 ** -8) + 1e-5  # P is rounded to fp16 or bf16
    accepted = 0

    def check():
        t = table.cpu().numpy()
        np.testing.assert_array_equal(refs.cpu().numpy(), np.bincount(t[t >= 0], minlength=PAGES))
        np.testing.assert_array_equal((t >= 0).sum(1), -(-lens // 16))
        kk, vv = (real(cache[0], cache[1]), real(cache[2], cache[3])) if fp8 else (real(cache[0]), real(cache[1]))
        for b in range(B):
            at = np.arange(lens[b])
            for x, i in ((kk, 0), (vv, 1)):
                if lens[b]:
                    np.testing.assert_array_equal(x[t[b, at // 16], :, at % 16], np.stack([r[i] for r in held[b]]))

    for step in range(STEPS):
        sizes = g.integers(1, N + 1, B)
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        parent = np.concatenate([[-1] + [int(g.integers(max(0, i - 4), i)) for i in range(1, n)] for n in sizes]).astype(np.int32)
        depth = np.zeros(off[-1], np.int32)
        for b in range(B):
            for i in range(1, sizes[b]):
                depth[off[b] + i] = depth[off[b] + parent[off[b] + i]] + 1
        longest = np.array([depth[off[b]:off[b + 1]].max() + 1 for b in range(B)], np.int32)
        assert (tv.alloc_pages(table, refs, i32(lens + longest), begin=i32(lens)) == 0).all()
        total = int(off[-1])
        qkv = torch.randn(total, HQ + 2 * HKV, D, device="cuda", generator=gen).to(torch.bfloat16)
        pos = np.concatenate([lens[b] + depth[off[b]:off[b + 1]] for b in range(B)]).astype(np.int32)
        q, k = tv.rotate_qk(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], i32(pos), f, q_weight=weight[0], k_weight=weight[1])
        v = qkv[:, HQ + HKV:].contiguous()
        for x, heads, w in ((q, slice(0, HQ), 0), (k, slice(HQ, HQ + HKV), 1)):
            want = oracle.rotate(real(qkv[:, heads]), pos[None], freq, real(weight[w]))
            assert (np.abs(real(x) - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * np.abs(want).max()).all()
        kw = dict(max_nodes=N, max_prefix_len=max(1, int(lens.max())), out_dtype="fp32")
        index = (i32(parent), i32(lens), i32(off))
        if fp8:
            nodes = [*tv.quantize_rows(k), *tv.quantize_rows(v)]
            codes, qs = tv.quantize_rows(q)
            out, st = tv.tree_attention_fp8(codes, qs, *cache, table, *nodes, *index, **kw)
            qq, kn, vn = real(codes, qs), real(*nodes[:2]), real(*nodes[2:])
        else:
            nodes = [k, v]
            out, st = tv.tree_attention(q, *cache, table, *nodes, *index, **kw)
            qq, kn, vn = real(q), real(k), real(v)
        assert (st == 0).all()
        out = out.cpu().numpy()
        for b in range(B):
            for i in (0, int(sizes[b]) - 1):
                path, j = [], i
                while j >= 0:
                    path.append(off[b] + j)
                    j = parent[off[b] + j]
                rows = held[b] + [(kn[p], vn[p]) for p in path]
                for h in range(HQ):
                    keys, vals = (np.stack([r[c][h * HKV // HQ] for r in rows]) for c in (0, 1))
                    s = keys @ qq[off[b] + i, h] * D ** -0.5
                    w = np.exp(s - s.max())
                    assert np.abs(out[off[b] + i, h] - w @ vals / w.sum()).max() <= tol * np.abs(vals).max()
        tokens = g.integers(0, V, total)
        draft = torch.softmax(torch.randn(total, V, device="cuda", generator=gen), -1)
        target = torch.log(draft) + 0.3 * torch.randn(total, V, device="cuda", generator=gen)
        got = tv.accept(target, draft, i32(tokens), i32(parent), i32(off), torch.rand(total, device="cuda", generator=gen),
                        max_nodes=N, kind="logits")
        assert (got["status"] == 0).all()
        commit = tv.commit_kv_fp8 if fp8 else tv.commit_kv
        new, st = commit(*nodes, i32(parent), i32(off), got["accepted_len"], got["path"], table, i32(lens), *cache, max_nodes=N)
        assert (st == 0).all()
        paths, n = got["path"].cpu().numpy(), got["accepted_len"].cpu().numpy()
        for b in range(B):
            held[b] += [(kn[off[b] + i], vn[off[b] + i]) for i in [0] + paths[b, :n[b]].tolist()]
        lens = new.cpu().numpy()
        accepted += int(n.sum())
        assert (tv.free_pages(table, refs, keep_end=new) == 0).all()  # what the path did not reach
        check()
        longest_row = int(lens.argmax())
        if step % 4 == 3:  # a sequence ends
            lens[longest_row], held[longest_row] = 0, []
            assert (tv.free_pages(table, refs, keep_end=i32(lens)) == 0).all()
            check()
        if step == STEPS // 2:
            moved = tv.compact_pages(table, refs, block_table_out=table, ref_counts_out=refs)
            pools = [x[None] for x in cache]
            tv.copy_pages(moved["moves"], *(pools[::2] + pools[1::2] if fp8 else pools), count=moved["count"][1:])
            assert (moved["status"] == 0).all() and (refs[:int(moved["count"][0])] > 0).all()
            check()
    assert accepted > STEPS  # (paths of more than the root)
    assert (tv.free_pages(table, refs, keep_end=torch.zeros(B, dtype=torch.int32, device="cuda")) == 0).all()
    assert (refs == 0).all() and (table == -1).all()
