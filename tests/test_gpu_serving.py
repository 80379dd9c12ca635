"""The operators together, as a serving loop calls them: a prompt in chunks is
appended and attended, tree nodes are verified against the same cache, their
penalised logits accepted, the accepted path committed, and a decode token
follows; once with a bf16 cache and once with an E4M3 cache.  Each attention is
compared with fp64 on what the cache should hold by then."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, V = 3, 8, 2, 128, 1000
PARENT = [-1, 0, 0, 1, 1, 3]          # one tree shape for every sequence
PROMPTS = [[100, 37, 5], [16, 1, 260], [3, 3, 3]]  # chunks of each sequence's prompt


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def real(t, scale=None):
    if scale is None:
        return t.double().cpu().numpy()
    return oracle.e4m3_table()[t.cpu().numpy()] * scale.double().cpu().numpy()[..., None]


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_verify_accept_commit_decode(fp8):
    ensure_built()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(fp8))
    g = np.random.default_rng(int(fp8))

    def rows(n, heads):
        return torch.randn(n, heads, D, device="cuda", generator=gen).to(torch.bfloat16)

    pages_per_seq = 24
    blocks = B * pages_per_seq + 5
    perm = g.permutation(blocks).astype(np.int32)
    table = perm[:B * pages_per_seq].reshape(B, pages_per_seq)
    t_table = i32(table)
    shape = (blocks, HKV, 16, D)
    if fp8:
        pool = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scale = [torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
        cache = (pool[0], scale[0], pool[1], scale[1])
    else:
        pool = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache = tuple(pool)
    lens = np.zeros(B, np.int32)
    tol = (4 * 2.0 ** -11 if fp8 else 2 * 2.0 ** -8) + 1e-5

    def values():
        return [real(cache[0], cache[1]), real(cache[2], cache[3])] if fp8 else [real(x) for x in cache]

    def step(chunks):
        """Appends and attends one chunk per sequence; checks it against fp64."""
        nonlocal lens
        lens = (lens + chunks).astype(np.int32)
        off = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        n = int(off[-1])
        qkv = rows(n, HQ + 2 * HKV)  # a fused projection: its slices are used as they are
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        at = (t_table, i32(lens), i32(off))
        if fp8:
            st = tv.append_kv_fp8(k, v, *at, *cache)
            codes, qs = tv.quantize_rows(q)
            out, st2 = tv.chunk_attention_fp8(codes, qs, *cache, *at, max_len=int(lens.max()), out_dtype="fp32")
            q = real(codes, qs)
        else:
            st = tv.append_kv(k, v, *at, *cache)
            out, st2 = tv.chunk_attention(q, *cache, *at, max_len=int(lens.max()), out_dtype="fp32")
            q = real(q)
        assert (st == 0).all() and (st2 == 0).all()
        kk, vv = values()
        ref = oracle.chunk_attention(q, kk, vv, table, lens, off)
        assert np.abs(out.cpu().numpy() - ref).max() <= tol * np.nanmax(np.abs(vv))
        if fp8:  # what was written reads back within half an E4M3 step (at least its smallest)
            back, _, st = tv.read_kv_fp8(*cache, *at, total_tokens=n)
            a, b = k.double(), back.double()
            top = a.abs().amax(-1, keepdim=True)
            assert ((a - b).abs() <= a.abs() * (2.0 ** -4 + 2.0 ** -7) + top / 448 * 2.0 ** -9).all()

    for chunk in range(3):
        step(np.array([PROMPTS[b][chunk] for b in range(B)], np.int32))

    # verification of a tree per sequence over the same cache
    N = len(PARENT)
    off = np.arange(B + 1, dtype=np.int32) * N
    parent = np.tile(PARENT, B).astype(np.int32)
    q, k, v = rows(B * N, HQ), rows(B * N, HKV), rows(B * N, HKV)
    kw = dict(max_nodes=N, max_prefix_len=int(lens.max()), out_dtype="fp32")
    if fp8:
        (qc, qs), (kc, ks), (vc, vs) = (tv.quantize_rows(x) for x in (q, k, v))
        out, st = tv.tree_attention_fp8(qc, qs, *cache, t_table, kc, ks, vc, vs, i32(parent), i32(lens), i32(off), **kw)
        q, kn, vn = real(qc, qs), real(kc, ks), real(vc, vs)
    else:
        out, st = tv.tree_attention(q, *cache, t_table, k, v, i32(parent), i32(lens), i32(off), **kw)
        q, kn, vn = real(q), real(k), real(v)
    assert (st == 0).all()
    kk, vv = values()
    for b in range(B):
        pos = np.arange(lens[b])
        for i in range(N):
            path, j = [], i
            while j >= 0:
                path.append(b * N + j)
                j = PARENT[j]
            for h in range(HQ):
                keys = np.concatenate([kk[table[b, pos // 16], h // 4, pos % 16], kn[path, h // 4]])
                vals = np.concatenate([vv[table[b, pos // 16], h // 4, pos % 16], vn[path, h // 4]])
                s = keys @ q[b * N + i, h] * D ** -0.5
                w = np.exp(s - s.max())
                assert np.abs(out[b * N + i, h].cpu().numpy() - w @ vals / w.sum()).max() <= tol * np.abs(vals).max()

    # penalised logits, with a grammar that forbids the draft of node 4, accepted
    tokens = g.integers(0, V, B * N).astype(np.int32)
    logits = torch.randn(B * N, V, device="cuda", generator=gen).to(torch.bfloat16)
    history = g.integers(0, V, 60).astype(np.int32)
    hoff, prompt = np.array([0, 20, 40, 60], np.int32), np.array([10, 20, 0], np.int32)
    rep, pres = np.array([1.3, 1.0, 0.9], np.float32), np.array([0.5, 0.0, 0.2], np.float32)
    allowed = np.ones((B * N, V), bool)
    for b in range(B):
        allowed[b * N + 1, tokens[b * N + 4]] = False
    bits = np.zeros((B * N, -(-V // 32) * 32), np.uint8)
    bits[:, :V] = allowed
    mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view("<u4").view(np.int32)).cuda()
    target, st = tv.penalize_logits(logits, i32(tokens), i32(parent), i32(off), max_nodes=N, history=i32(history),
                                    history_offsets=i32(hoff), prompt_lens=i32(prompt),
                                    repetition=torch.from_numpy(rep).cuda(), presence=torch.from_numpy(pres).cuda(),
                                    allowed_mask=mask)
    assert (st == 0).all()
    ref = oracle.penalize_logits(real(logits), tokens, parent, off, history, hoff, prompt, rep, pres, allowed=allowed)
    fine = np.isfinite(ref)
    np.testing.assert_allclose(target.cpu().numpy()[fine], ref[fine], rtol=0, atol=5 * 2.0 ** -24 * 20)
    draft = torch.softmax(torch.randn(B * N, V, device="cuda", generator=gen), -1)
    # a uniform that accepts and one that rejects: u q < p
    uniforms = torch.rand(B * N, device="cuda", generator=gen) * 0.5
    acc = tv.accept(target, draft, i32(tokens), i32(parent), i32(off), uniforms, max_nodes=N, kind="logits")
    assert (acc["status"] == 0).all()
    paths = acc["path"].cpu().numpy()
    for b in range(B):  # the forbidden draft is never on a path
        assert 4 not in paths[b]

    # the accepted path joins the cache; the next token sees it
    args = (i32(parent), i32(off), acc["accepted_len"], acc["path"], t_table, i32(lens))
    if fp8:
        new, st = tv.commit_kv_fp8(kc, ks, vc, vs, *args, *cache, max_nodes=N)
    else:
        new, st = tv.commit_kv(k, v, *args, *cache, max_nodes=N)
    assert (st == 0).all()
    np.testing.assert_array_equal(new.cpu().numpy(), lens + acc["accepted_len"].cpu().numpy() + 1)
    kk, _ = values()
    for b in range(B):
        for t, node in enumerate([0] + paths[b, :int(acc["accepted_len"][b])].tolist()):
            p = lens[b] + t
            np.testing.assert_array_equal(kk[table[b, p // 16], :, p % 16], kn[b * N + node])
    lens = new.cpu().numpy()
    step(np.ones(B, np.int32))
