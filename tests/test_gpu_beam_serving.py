"""Beam search over the paged cache, as a serving loop runs it: pages are given
(alloc_pages), queries and keys normed and turned (rotate_qk), keys and values
appended, attention over the cache, penalties, the next beams (beam_select), new
tables with copies of half-filled pages (fork_pages, copy_pages), a compaction on
the way and everything freed at the end; two layers in one pool, once with a bf16
cache and once with an E4M3 cache.  Each beam's cache is compared with the rows of
its own tokens after every step, the attention and the choice with fp64."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

B, K, HQ, HKV, V, LAYERS, END = 2, 3, 4, 2, 97, 2, 5
PROMPTS = [13, 32]
STEPS = 40


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("fp8", [False, True])
def test_beam_search(fp8):
    ensure_built()
    d = 128 if fp8 else 64
    g = torch.Generator().manual_seed(int(fp8))
    embed = torch.randn(LAYERS, V, HQ + 2 * HKV, d, generator=g).to(torch.bfloat16).cuda()
    head = (torch.randn(LAYERS * HQ * d, V, generator=g) * 0.7 / np.sqrt(d)).cuda()
    weight = (1 + 0.1 * torch.randn(2, d, generator=g)).cuda()
    freq = torch.from_numpy(10000.0 ** (-np.arange(d // 2) / (d // 2))).cuda()
    pages, width = 60, 8
    shape = (LAYERS, pages, HKV, 16, d)
    if fp8:
        pool = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scale = [torch.full(shape[:4], float("nan"), device="cuda") for _ in range(2)]
    else:
        pool, scale = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)], []
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    # what each row's cache should hold: [layer][position] of (k row, v row)
    held = [[[] for _ in range(LAYERS)] for _ in range(B)]
    tokens = [np.random.default_rng(b).integers(0, V, n).tolist() for b, n in enumerate(PROMPTS)]
    history = [list(t) for t in tokens]

    def cached(row, layer):
        """K and V rows of a sequence, through its table."""
        n, t = int(lens[row]), table[row].long()
        at = torch.arange(n, device="cuda")
        parts = pool + scale
        return [x[layer][t[at // 16], :, at % 16] for x in parts]

    def check_cache():
        t, r = table.cpu().numpy(), refs.cpu().numpy()
        np.testing.assert_array_equal(r, np.bincount(t[t >= 0], minlength=pages))
        for row in range(table.shape[0]):
            for layer in range(LAYERS):
                have = cached(row, layer)
                for i, x in enumerate(have):
                    want = torch.stack([e[i] for e in held[row][layer]])
                    assert torch.equal(x.cpu(), want), (row, layer, i)

    def step(new):
        """Appends and attends new[row] tokens of every row; logits after the last of each."""
        nonlocal lens
        n = np.array([len(x) for x in new], np.int32)
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        old = lens
        lens = old + i32(n)
        assert (tv.alloc_pages(table, refs, lens, begin=old) == 0).all()
        at = (table, lens, i32(off))
        pos = i32(np.concatenate([np.arange(l, l + c) for l, c in zip(old.tolist(), n)]))
        ids = torch.tensor(sum(new, []), device="cuda")
        outs = []
        for layer in range(LAYERS):
            qkv = embed[layer][ids]
            q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
            q, k = tv.rotate_qk(q, k, pos, freq, q_weight=weight[0], k_weight=weight[1], q_out=q, k_out=k)
            if fp8:
                (kc, ks), (vc, vs) = tv.quantize_rows(k), tv.quantize_rows(v)
                rows = [kc, vc, ks, vs]
                cache = (pool[0][layer], scale[0][layer], pool[1][layer], scale[1][layer])
                assert (tv.append_kv_fp8(k, v, *at, *cache) == 0).all()
                codes, qs = tv.quantize_rows(q)
                out, st = tv.chunk_attention_fp8(codes, qs, *cache, *at, max_len=width * 16, out_dtype="fp32")
            else:
                rows = [k, v]
                cache = (pool[0][layer], pool[1][layer])
                assert (tv.append_kv(k, v, *at, *cache) == 0).all()
                out, st = tv.chunk_attention(q, *cache, *at, max_len=width * 16, out_dtype="fp32")
            assert (st == 0).all()
            rows = [x.cpu() for x in rows]
            for b in range(len(n)):
                for i in range(off[b], off[b + 1]):
                    held[b][layer].append([x[i] for x in rows])
            outs.append(out)
        last = torch.from_numpy(np.maximum(off[1:] - 1, 0)).long().cuda()
        x = torch.cat([o[last].reshape(len(n), -1) for o in outs], 1)
        # attention of each row's last token against fp64 on the rows that it should see
        values = oracle.e4m3_table() if fp8 else None
        for b in range(len(n)):
            if not n[b]:
                continue
            kk, vv = ([values[torch.stack([e[i] for e in held[b][layer]]).numpy()] *
                       torch.stack([e[i + 2] for e in held[b][layer]]).double().numpy()[..., None] for i in (0, 1)] if fp8
                      else [torch.stack([e[i] for e in held[b][layer]]).double().numpy() for i in (0, 1)])
            qq = (values[codes[off[b + 1] - 1].cpu().numpy()] * qs[off[b + 1] - 1].double().cpu().numpy()[..., None] if fp8
                  else q[off[b + 1] - 1].double().cpu().numpy())
            for h in range(HQ):
                s = kk[:, h * HKV // HQ] @ qq[h] * d ** -0.5
                w = np.exp(s - s.max())
                ref = w @ vv[:, h * HKV // HQ] / w.sum()
                tol = (4 * 2.0 ** -11 if fp8 else 2 * 2.0 ** -8) + 1e-5  # P is rounded to fp16 or bf16
                assert np.abs(out[off[b + 1] - 1, h].cpu().numpy() - ref).max() <= tol * np.abs(vv).max()
        # penalties over each sequence's tokens; a tree of its root alone per row
        hoff = np.concatenate([[0], np.cumsum([len(h) for h in history])]).astype(np.int32)
        rows = len(n)
        logits, st = tv.penalize_logits(
            x @ head, i32(np.zeros(rows)), i32(np.full(rows, -1)), i32(np.arange(rows + 1)), max_nodes=1,
            history=i32(sum(history, [])), history_offsets=i32(hoff),
            repetition=torch.full((rows,), 1.2, device="cuda"))
        assert (st == 0).all()
        return logits

    logits = step(tokens)
    check_cache()
    scores, finished = torch.zeros(B, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    lengths = torch.ones(B, dtype=torch.int32, device="cuda")
    beams, ended_once, copied = 1, False, 0
    for i in range(STEPS):
        r = tv.beam_select(logits, scores, beams=beams, select=K, lengths=lengths, finished=finished, end_token=END,
                           length_penalty=0.6)
        assert (r["status"] == 0).all()
        want = oracle.beam_select(logits.double().cpu().numpy(), scores.cpu().numpy(), beams, K, lengths.cpu().numpy(),
                                  finished.cpu().numpy(), END, 0.6)
        picked, parents = r["tokens"].reshape(-1).tolist(), r["parents"].reshape(-1).tolist()
        assert picked == [c[0] for b in want for c in b] and parents == [c[1] for b in want for c in b]
        done = finished.tolist()
        new = [[] if done[p] else [t] for p, t in zip(parents, picked)]
        scores, lengths, finished = (r[k].reshape(-1) for k in ("scores", "lengths", "finished"))
        table, lens, copies, st = tv.fork_pages(table, lens, r["parents"].reshape(-1), refs)
        assert (st == 0).all()
        copied += int((copies[:, 0] >= 0).sum())
        tv.copy_pages(copies, *pool, *scale)
        held = [[list(x) for x in held[p]] for p in parents]
        history = [list(history[p]) + t for p, t in zip(parents, new)]
        beams = K
        check_cache()
        if i == STEPS // 2:
            got = tv.compact_pages(table, refs)
            assert (got["status"] == 0).all()
            tv.copy_pages(got["moves"], *pool, *scale, count=got["count"][1:])
            table, refs = got["block_table"], got["ref_counts"]
            n = int(got["count"][0])
            assert (refs[:n] > 0).all() and (refs[n:] == 0).all()
            check_cache()
        if finished.all():
            break
        ended_once |= bool(finished.any())
        logits = step(new)
        check_cache()
    assert copied > 0
    # one sequence of each request stays, then none
    keep = i32([int(n) if row % K == 0 else 0 for row, n in enumerate(lens.tolist())])
    assert (tv.free_pages(table, refs, keep_end=keep) == 0).all()
    t, r = table.cpu().numpy(), refs.cpu().numpy()
    np.testing.assert_array_equal(r, np.bincount(t[t >= 0], minlength=pages))
    assert (t[1] == -1).all() and (t[0] >= 0).sum() == -(-int(lens[0]) // 16)
    assert (tv.free_pages(table, refs, keep_end=torch.zeros_like(lens)) == 0).all()
    assert (refs == 0).all() and (table == -1).all()
