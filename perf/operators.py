"""The operators of a serving step around tree verification, as they are measured.

Five operators: attention of a chunk of new tokens over the paged cache (bf16
and E4M3 caches, optionally with a sliding window and first tokens that stay
visible), the write of new K/V rows into the cache (bf16 copy, or quantised to
E4M3 codes with one fp32 scale per row), the read of an E4M3 cache back to
bf16, and the penalties, biases and grammar masks on the target logits of the
tree nodes.  ``run`` computes each in plain torch operations, or with
``own = True`` through the package.

Shapes are those of the repository's workloads: 32/8 heads of 128 with 512 to
4096 cached tokens (serving), 28/4 heads with 1600-token multimodal prompts,
64/8 heads over 32768 tokens (long context), 4/4 heads of 64 (tiny), and
vocabularies of 1000, 32000, 128256 and 151936.
"""
import math
import random

import torch

own = False

PAGE = 16
NEG_INF = float("-inf")


def _case(name, op, **kw):
    c = {"name": name, "op": op}
    c.update(kw)
    return c


def _attend(name, op, batch, hq, hkv, d, ctx, chunk, window=0, sinks=0, shape=1):
    """ctx, chunk: (lowest, highest) cached tokens before the chunk and chunk lengths."""
    return _case(name, op, batch=batch, hq=hq, hkv=hkv, d=d, ctx_lo=ctx[0], ctx_hi=ctx[1],
                 chunk_lo=chunk[0], chunk_hi=chunk[1], window=window, sinks=sinks, shape=shape)


def _move(name, op, form, batch, hkv, d, ctx, chunk, shape=1):
    return _case(name, op, form=form, batch=batch, hkv=hkv, d=d, ctx_lo=ctx[0], ctx_hi=ctx[1],
                 chunk_lo=chunk[0], chunk_hi=chunk[1], shape=shape)


def _penalize(name, batch, nodes, depth, vocab, history, biases, masked, dtype, shape=1):
    return _case(name, "penalize", batch=batch, nodes_lo=nodes[0], nodes_hi=nodes[1], depth=depth,
                 vocab=vocab, hist_lo=history[0], hist_hi=history[1], biases=biases, masked=masked,
                 dtype=dtype, shape=shape)


def listed():
    return [
        # one new token for each of 16 serving sequences: a plain decode step,
        # bound by one read of the cache
        _attend("decode, 16 x 512-4096", "attend", 16, 32, 8, 128, (511, 4095), (1, 1)),
        # four multimodal prompts prefilled from an empty cache, 28/4 heads
        _attend("prompt, 4 x 1600", "attend", 4, 28, 4, 128, (0, 0), (1600, 1600)),
        # a 2048-token chunk of a long prompt with 32768 tokens already cached
        _attend("long, 2048 over 32768", "attend", 1, 64, 8, 128, (32768, 32768), (2048, 2048)),
        # prompts, chunks and single tokens in one batch, of odd lengths, under
        # a 1024-token window with 4 first tokens kept
        _attend("mixed, window 1024", "attend", 12, 32, 8, 128, (0, 5003), (1, 701), 1024, 4),
        # decode over long E4M3 caches: half the bytes of bf16
        _attend("fp8 decode, 4 x 32768", "attend_fp8", 4, 64, 8, 128, (32000, 32767), (1, 1)),
        # chunks of prompts over E4M3 caches of odd lengths
        _attend("fp8 chunks, 8 x 513", "attend_fp8", 8, 32, 8, 128, (512, 3999), (65, 513)),
        # the K/V of one decode step written into the E4M3 cache: latency
        _move("append 16 tokens", "append", "e4m3", 16, 8, 128, (511, 4095), (1, 1)),
        # the K/V of whole prompts written into the E4M3 cache: bandwidth
        _move("append 4 x 8192", "append", "e4m3", 4, 8, 128, (0, 0), (8190, 8193)),
        # the cache of one short sequence handed to code that wants bf16
        _move("read 1001 tokens", "read", "e4m3", 1, 8, 128, (0, 0), (1001, 1001)),
        # the caches of four long sequences read back
        _move("read 4 x 32768", "read", "e4m3", 4, 8, 128, (0, 0), (32768, 32768)),
        # the target rows of one serving verification step, bf16 from the head
        _penalize("16 trees, V 32000", 16, (26, 64), 5, 32000, (512, 4096), 16, True, "bf16"),
        # the multimodal step's rows, fp32, with a grammar mask for every node
        _penalize("4 trees, V 151936", 4, (128, 128), 8, 151936, (1600, 1600), 300, True, "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend_fp8", "append", "read", "penalize"])
    shape = rng.randrange(1 << 20)
    if op.startswith("attend"):
        hq, hkv, d = rng.choice([(4, 4, 64), (32, 32, 128), (32, 8, 128), (28, 4, 128), (64, 8, 128), (8, 1, 64)])
        if op == "attend_fp8":
            d = 128
        while True:
            batch, ctx, chunk = _log(rng, 1, 48), _log(rng, 1, 40000), _log(rng, 1, 4000)
            if rng.random() < 0.3:
                chunk = 1
            cost = batch * hq * chunk * (ctx + chunk)
            if cost <= 2.2e9 and batch * (ctx + chunk) * hkv * d <= 3e8:
                break
        window, sinks = 0, 0
        if rng.random() < 0.4:
            window, sinks = _log(rng, 1, 5000), rng.choice([0, 1, 4, 17, 130])
        return {"op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
                "ctx_lo": rng.randrange(ctx + 1), "ctx_hi": ctx, "chunk_lo": rng.randint(min(chunk, 1), chunk),
                "chunk_hi": chunk, "window": window, "sinks": sinks, "shape": shape}
    if op in ("append", "read"):
        form = "e4m3" if op == "read" else rng.choice(["e4m3", "e4m3", "bf16", "rows"])
        while True:
            batch, chunk = _log(rng, 1, 64), _log(rng, 1, 33000)
            hkv, d = rng.choice([1, 4, 8, 32]), rng.choice([64, 128])
            ctx = rng.choice([0, _log(rng, 1, 4000)])
            if batch * (ctx + chunk) * hkv * d <= (1.3e8 if op == "read" else 6e7):
                break
        return {"op": op, "form": form, "batch": batch, "hkv": hkv, "d": d, "ctx_lo": 0, "ctx_hi": ctx,
                "chunk_lo": rng.randint(1, chunk), "chunk_hi": chunk, "shape": shape}
    while True:
        batch, nodes, vocab = _log(rng, 1, 32), _log(rng, 1, 256), _log(rng, 900, 200000)
        if batch * nodes * vocab <= 7e7:
            break
    hist = _log(rng, 1, 40000)
    return {"op": op, "batch": batch, "nodes_lo": rng.randint(1, nodes), "nodes_hi": nodes,
            "depth": rng.randint(1, 12), "vocab": vocab, "hist_lo": rng.randrange(hist + 1), "hist_hi": hist,
            "biases": rng.choice([0, 1, 16, 300]), "masked": rng.random() < 0.5,
            "dtype": rng.choice(["fp32", "bf16"]), "shape": shape}


# ------------------------------------------------------------------ shapes
def _lens(case):
    """(cached tokens before the chunk, chunk lengths), a pure function of the case."""
    r = random.Random(case["shape"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    chunk = [r.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(case["batch"])]
    return ctx, chunk


def _trees(case):
    """Parents (local, -1 at a root) of the trees, history lengths and prompt lengths."""
    r = random.Random(case["shape"])
    parents, hist, prompt = [], [], []
    for _ in range(case["batch"]):
        par, depth = [-1], [0]
        for i in range(1, r.randint(case["nodes_lo"], case["nodes_hi"])):
            p = r.choice([j for j in range(max(0, i - 24), i) if depth[j] < case["depth"]] or [0])
            par.append(p)
            depth.append(depth[p] + 1)
        parents.append(par)
        hist.append(r.randint(case["hist_lo"], case["hist_hi"]))
        prompt.append(r.randint(0, hist[-1]))
    return parents, hist, prompt


def _visible(ctx, chunk, window, sinks):
    """Keys that the rows of a chunk see, and the distinct ones among them."""
    pairs = 0
    for i in range(chunk):
        p = ctx + i
        low = max(0, p - window + 1) if window else 0
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, ctx - window + 1) if window else 0
    return pairs, ctx + chunk - low + min(sinks, low)


def work(case):
    op = case["op"]
    if op.startswith("attend"):
        ctx, chunk = _lens(case)
        pairs = keys = 0
        for x, c in zip(ctx, chunk):
            p, k = _visible(x, c, case["window"], case["sinks"])
            pairs, keys = pairs + p, keys + k
        d, rows = case["d"], sum(chunk) * case["hq"]
        el, sc = (1, 4) if op == "attend_fp8" else (2, 0)
        return {"bytes": keys * case["hkv"] * 2 * (d * el + sc) + rows * (d * el + sc) + rows * d * 2,
                "flops": 4 * pairs * case["hq"] * d}
    if op in ("append", "read"):
        rows = sum(_lens(case)[1]) * case["hkv"] * (1 if case["form"] == "rows" else 2)
        out = case["d"] * 2 if case["form"] == "bf16" else case["d"] + 4
        return {"bytes": rows * (case["d"] * 2 + out), "flops": 2 * rows * case["d"]}
    parents, hist, _ = _trees(case)
    rows, v = sum(map(len, parents)), case["vocab"]
    each = (2 if case["dtype"] == "bf16" else 4) + 4 + (1 / 8 if case["masked"] else 0)
    return {"bytes": int(rows * v * each) + 4 * sum(hist) + 8 * case["batch"] * case["biases"] + 8 * rows,
            "flops": 4 * rows * v}


# ------------------------------------------------------------------ inputs
def _paged(case, g, dev):
    """Sequence ends, cumulative chunk lengths and a shuffled block table."""
    ctx, chunk = _lens(case)
    ends = [x + c for x, c in zip(ctx, chunk)]
    pages = [-(-e // PAGE) for e in ends]
    total = sum(pages)
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    width = max(pages)
    start = torch.tensor([sum(pages[:i]) for i in range(len(pages))], device=dev)
    at = start[:, None] + torch.arange(width, device=dev)[None, :]
    have = torch.arange(width, device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
    table = torch.where(have, perm[at.clamp(max=total - 1)], torch.full((), -1, dtype=torch.int32, device=dev))
    offsets = torch.tensor([sum(chunk[:i]) for i in range(len(chunk) + 1)], dtype=torch.int32, device=dev)
    return {"lens": torch.tensor(ends, dtype=torch.int32, device=dev), "offsets": offsets,
            "table": table.contiguous(), "pages": total, "max_len": max(ends), "max_chunk": max(chunk),
            "total": sum(chunk)}


def _codes(shape, g, dev):
    """E4M3 codes of normal values in units of their row's largest / 448, and the row scales."""
    x = torch.randn(shape, generator=g, device=dev)
    scale = x.abs().amax(-1) / 448.0
    return (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    if op == "penalize":
        parents, hist, prompt = _trees(case)
        rows, v, batch = sum(map(len, parents)), case["vocab"], case["batch"]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        s = {"logits": torch.randn(rows, v, generator=g, device=dev) * 2.0,
             "tokens": torch.randint(0, v, (rows,), generator=g, device=dev, dtype=torch.int32),
             "parent": i32(sum(parents, [])),
             "offsets": i32([sum(map(len, parents[:i])) for i in range(batch + 1)]),
             # text repeats itself: half of the history from 200 tokens
             "history": torch.where(torch.rand(max(1, sum(hist)), generator=g, device=dev) < 0.5,
                                    torch.randint(0, min(200, v), (max(1, sum(hist)),), generator=g, device=dev),
                                    torch.randint(0, v, (max(1, sum(hist)),), generator=g, device=dev)).to(torch.int32),
             "history_offsets": i32([sum(hist[:i]) for i in range(batch + 1)]),
             "prompt_lens": i32(prompt),
             "repetition": 1.0 + torch.rand(batch, generator=g, device=dev) * 0.3,
             "presence": torch.rand(batch, generator=g, device=dev) - 0.2,
             "frequency": torch.rand(batch, generator=g, device=dev) - 0.2,
             "bias_ids": None, "bias_values": None, "bias_offsets": None, "allowed": None,
             "batch": batch, "rows": rows, "max_nodes": max(map(len, parents))}
        if case["dtype"] == "bf16":
            s["logits"] = s["logits"].to(torch.bfloat16)
        n = min(case["biases"], v)
        if n:
            s["bias_ids"] = torch.rand(batch, v, generator=g, device=dev).topk(n, 1).indices.to(torch.int32).reshape(-1)
            s["bias_values"] = torch.randn(batch * n, generator=g, device=dev) * 3.0
            s["bias_offsets"] = i32([n * i for i in range(batch + 1)])
        if case["masked"]:
            s["allowed"] = torch.randint(-(1 << 31), 1 << 31, (rows, -(-v // 32)), generator=g, device=dev).to(torch.int32)
        return s
    s = _paged(case, g, dev)
    hkv, d = case["hkv"], case["d"]
    pool = (s["pages"], hkv, PAGE, d)
    if op.startswith("attend"):
        s["window"], s["sinks"] = case["window"], case["sinks"]
        if op == "attend":
            s["q"] = normal(s["total"], case["hq"], d)
            s["k"], s["v"] = normal(*pool), normal(*pool)
        else:
            s["q"], s["q_scale"] = _codes((s["total"], case["hq"], d), g, dev)
            s["k"], s["k_scale"] = _codes(pool, g, dev)
            s["v"], s["v_scale"] = _codes(pool, g, dev)
        return s
    s["form"] = case["form"]
    if op == "read":
        s["k"], s["k_scale"] = _codes(pool, g, dev)
        s["v"], s["v_scale"] = _codes(pool, g, dev)
        return s
    s["k_new"] = normal(s["total"], hkv, d)
    if case["form"] == "rows":
        return s
    s["v_new"] = normal(s["total"], hkv, d)
    if case["form"] == "bf16":
        s["k"], s["v"] = torch.zeros(pool, device=dev, dtype=torch.bfloat16), torch.zeros(pool, device=dev, dtype=torch.bfloat16)
    else:
        s["k"], s["v"] = torch.zeros(pool, device=dev, dtype=torch.uint8), torch.zeros(pool, device=dev, dtype=torch.uint8)
        s["k_scale"], s["v_scale"] = torch.zeros(pool[:3], device=dev), torch.zeros(pool[:3], device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _token_places(s):
    """For each chunk token: its sequence, its index in the chunk and its position."""
    dev = s["offsets"].device
    t = torch.arange(s["total"], device=dev)
    offsets = s["offsets"].long()
    b = torch.searchsorted(offsets, t, right=True) - 1
    i = t - offsets[b]
    return b, i, s["lens"].long()[b] - (offsets[b + 1] - offsets[b]) + i


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None]


def _plain_attend(s):
    f8 = "q_scale" in s
    dev = s["q"].device
    lens, offsets = s["lens"].long(), s["offsets"].long()
    hkv, d = s["k"].shape[1], s["k"].shape[3]
    pos = torch.arange(s["max_len"], device=dev)
    page = s["table"].long()[:, pos // PAGE].clamp(min=0)
    k, v = s["k"][page, :, pos % PAGE], s["v"][page, :, pos % PAGE]  # [B, L, Hkv, D]
    q = s["q"]
    if f8:
        k = _values(k, s["k_scale"][page, :, pos % PAGE])
        v = _values(v, s["v_scale"][page, :, pos % PAGE])
        q = _values(q, s["q_scale"])
    chunk = offsets[1:] - offsets[:-1]
    c = torch.arange(s["max_chunk"], device=dev)
    row = (offsets[:-1, None] + c).clamp(max=s["total"] - 1)
    qp = (q[row].float() / math.sqrt(d)).view(row.shape[0], row.shape[1], hkv, -1, d)
    x = torch.einsum("bchgd,blhd->bhgcl", qp, k.float())
    at = (lens - chunk)[:, None] + c
    seen = pos <= at[:, :, None]
    if s["window"]:
        seen &= (pos > at[:, :, None] - s["window"]) | (pos < s["sinks"])
    x.masked_fill_(~seen[:, None, None], NEG_INF)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.einsum("bhgcl,blhd->bhgcd", x, v.float()) / total
    b, i, _ = _token_places(s)
    y = y.permute(0, 3, 1, 2, 4)[b, i].reshape(s["q"].shape)
    return {"out": y.to(torch.bfloat16)}


def _plain_quantise(x):
    """(codes, scale): scale = max|row| / 448 in fp32, codes of row / scale to nearest even."""
    x = x.float()
    scale = x.abs().amax(-1) / torch.full((), 448.0, device=x.device)  # (a division, not a product with 1 / 448)
    scale = torch.where(scale > 0, scale.clamp(min=2.0 ** -126), torch.ones((), device=x.device))
    y = x.double() / scale.double()[..., None]  # in 64 bits: quotients lie next to rounding borders
    f, e = torch.frexp(y.abs())  # f 2^e with f in [0.5, 1): 8 to 16 steps of 2^(e - 4), at least 2^-9
    m = torch.round(torch.where(e < -5, y.abs() * 512, f * 16)).to(torch.int32)
    code = (e.clamp(min=-5) + 5) * 8 + m
    return (code + 128 * torch.signbit(y)).to(torch.uint8), scale


def _plain_append(s):
    if s["form"] == "rows":
        codes, scale = _plain_quantise(s["k_new"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}
    b, _, pos = _token_places(s)
    page, row = s["table"].long()[b, pos // PAGE], pos % PAGE
    if s["form"] == "bf16":
        s["k"][page, :, row] = s["k_new"]
        s["v"][page, :, row] = s["v_new"]
        return {"k": s["k"], "v": s["v"]}
    for x, pool, scales in (("k_new", "k", "k_scale"), ("v_new", "v", "v_scale")):
        codes, scale = _plain_quantise(s[x])
        s[pool][page, :, row] = codes
        s[scales][page, :, row] = scale
    return _pools(s)


def _pools(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v": s["v"].view(torch.float8_e4m3fn), "v_scale": s["v_scale"]}


def _plain_read(s):
    b, _, pos = _token_places(s)
    page, row = s["table"].long()[b, pos // PAGE], pos % PAGE
    return {"k": _values(s["k"][page, :, row], s["k_scale"][page, :, row]).to(torch.bfloat16),
            "v": _values(s["v"][page, :, row], s["v_scale"][page, :, row]).to(torch.bfloat16)}


def _plain_penalize(s):
    x = s["logits"].float()
    rows, v = x.shape
    dev, batch = x.device, s["batch"]
    offsets, tokens = s["offsets"].long(), s["tokens"].long()
    node = torch.arange(rows, device=dev)
    seq = torch.searchsorted(offsets, node, right=True) - 1
    # history: counts of the generated tokens, presence of all of them
    h = s["history_offsets"].long()
    at = torch.arange(s["history"].shape[0], device=dev)
    hb = (torch.searchsorted(h, at, right=True) - 1).clamp(max=batch - 1)
    inside = (at < h[-1]).float()
    generated = inside * (at - h[hb] >= s["prompt_lens"].long()[hb])
    place = hb * v + s["history"].long()
    seen = torch.zeros(batch * v, device=dev).scatter_add_(0, place, inside).view(batch, v)
    count = torch.zeros(batch * v, device=dev).scatter_add_(0, place, generated).view(batch, v)
    # the drafted tokens on the path of each node: (1 + A)(1 + A^2)(1 + A^4)(1 + A^8)
    parent = s["parent"].long()
    root = parent < 0
    one = torch.eye(rows, device=dev)
    a = one[torch.where(root, node, offsets[seq] + parent)] * (~root)[:, None]
    a2 = a @ a
    a4 = a2 @ a2
    path = (one + a) @ (one + a2) @ (one + a4) @ (one + a4 @ a4)
    path = path * (~root)[None, :]
    drafted = torch.zeros(rows, v, device=dev).scatter_add_(1, tokens[None, :].expand(rows, rows), path)
    count = count[seq] + drafted
    seen = (seen[seq] + drafted) > 0
    rep = s["repetition"][seq][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][seq][:, None] * count
    x = x - s["presence"][seq][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        n = s["bias_ids"].shape[0] // batch
        bias = torch.zeros(batch, v, device=dev).scatter_(1, s["bias_ids"].long().view(batch, n), s["bias_values"].view(batch, n))
        x = x + bias[seq]
    if s["allowed"] is not None:
        bit = torch.arange(v, device=dev)
        ok = (s["allowed"][:, bit // 32] >> (bit % 32).to(torch.int32)) & 1
        x = x.masked_fill(ok == 0, NEG_INF)
    return {"out": x}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import speculative_decoding_tree_attention_gb300 as tv
    if "logits" in s:
        # the output and the status a serving loop keeps from step to step
        keep = s.setdefault("keep", {"out": torch.empty(s["logits"].shape, device=s["logits"].device),
                                     "status": torch.empty(s["batch"], dtype=torch.int32, device=s["logits"].device)})
        out, _ = tv.penalize_logits(
            s["logits"], s["tokens"], s["parent"], s["offsets"], max_nodes=s["max_nodes"],
            history=s["history"], history_offsets=s["history_offsets"], prompt_lens=s["prompt_lens"],
            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
            bias_ids=s["bias_ids"], bias_values=s["bias_values"], bias_offsets=s["bias_offsets"],
            allowed_mask=s["allowed"], **keep)
        return {"out": out}
    if "q" in s:
        kw = {"max_len": s["max_len"], "window": s["window"], "sinks": s["sinks"]}
        if "keep" not in s:  # the buffers a serving loop keeps from step to step
            prm = tv.chunk_params(s["q"], s["k"], s["table"], s["lens"], **kw)
            s["keep"] = {
                "out": torch.empty(s["q"].shape, device=s["q"].device, dtype=torch.bfloat16),
                "status": torch.empty(s["lens"].shape, device=s["q"].device, dtype=torch.int32),
                "workspace": torch.empty(tv.chunk_workspace_size(prm), device=s["q"].device, dtype=torch.uint8)}
        if "q_scale" in s:
            out, _ = tv.chunk_attention_fp8(s["q"], s["q_scale"], s["k"], s["k_scale"], s["v"], s["v_scale"],
                                            s["table"], s["lens"], s["offsets"], **kw, **s["keep"])
        else:
            out, _ = tv.chunk_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["offsets"], **kw, **s["keep"])
        return {"out": out}
    if "k_new" not in s:
        k, v, _ = tv.read_kv_fp8(s["k"], s["k_scale"], s["v"], s["v_scale"], s["table"], s["lens"], s["offsets"],
                                 total_tokens=s["total"])
        return {"k": k, "v": v}
    if s["form"] == "rows":
        codes, scale = tv.quantize_rows(s["k_new"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}
    if s["form"] == "bf16":
        tv.append_kv(s["k_new"], s["v_new"], s["table"], s["lens"], s["offsets"], s["k"], s["v"])
        return {"k": s["k"], "v": s["v"]}
    tv.append_kv_fp8(s["k_new"], s["v_new"], s["table"], s["lens"], s["offsets"], s["k"], s["k_scale"], s["v"], s["v_scale"])
    return _pools(s)


def run(state):
    if own:
        return _own(state)
    if "logits" in state:
        return _plain_penalize(state)
    if "q" in state:
        return _plain_attend(state)
    return _plain_append(state) if "k_new" in state else _plain_read(state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _e4m3_values(dev):
    """The value of each of the 256 E4M3 codes."""
    out = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(math.nan if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(out, dtype=torch.float64, device=dev)


def _exact_attend(case, s):
    ctx, chunk = _lens(case)
    group, d = case["hq"] // case["hkv"], case["d"]
    value = _e4m3_values("cuda")
    out = torch.empty(s["total"], case["hq"], d, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["batch"]):
        end, c = ctx[b] + chunk[b], chunk[b]
        pages = s["table"][b, : -(-end // PAGE)].long()
        at = torch.arange(ctx[b], end, device="cuda")[:, None]
        key = torch.arange(end, device="cuda")[None, :]
        hidden = key > at
        if case["window"]:
            hidden |= (key <= at - case["window"]) & (key >= case["sinks"])
        for h in range(case["hkv"]):
            k, v = s["k"][pages, h].reshape(-1, d)[:end], s["v"][pages, h].reshape(-1, d)[:end]
            q = s["q"][t0:t0 + c, h * group:(h + 1) * group]
            if case["op"] == "attend_fp8":
                k = value[k.long()] * s["k_scale"][pages, h].reshape(-1)[:end, None]
                v = value[v.long()] * s["v_scale"][pages, h].reshape(-1)[:end, None]
                q = value[q.long()] * s["q_scale"][t0:t0 + c, h * group:(h + 1) * group, None]
            k, v, q = k.double(), v.double(), q.double()
            for j in range(group):
                w = q[:, j] @ k.T * d ** -0.5
                w = torch.softmax(w.masked_fill(hidden, NEG_INF), 1)
                out[t0:t0 + c, h * group + j] = w @ v
        t0 += c
    return {"out": out}


def _exact_quantise(x):
    """The nearest E4M3 values (ties to the even code) of x in units of its row's scale."""
    x = x.double()
    scale = (x.abs().amax(-1) / 448.0).float()  # one fp32 division of a bf16 value
    y = x / scale.double()[..., None]
    grid = _e4m3_values(x.device)[:127]
    hi = torch.searchsorted(grid, y.abs().clamp(max=448.0)).clamp(1, 126)
    lo = hi - 1
    below, above = y.abs() - grid[lo], grid[hi] - y.abs()
    code = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[code], y), scale


def _exact_append(case, s):
    if case["form"] == "rows":
        value, scale = _exact_quantise(s["k_new"])
        return {"codes": value, "scale": scale.double()}
    ctx, chunk = _lens(case)
    out = {k: s[k].double() if s[k].dtype != torch.uint8 else torch.zeros(s[k].shape, dtype=torch.float64, device="cuda")
           for k in (("k", "v") if case["form"] == "bf16" else ("k", "k_scale", "v", "v_scale"))}
    t0 = 0
    for b in range(case["batch"]):
        pos = torch.arange(ctx[b], ctx[b] + chunk[b], device="cuda")
        page = s["table"][b].long()[pos // PAGE]
        for name in ("k", "v"):
            x = s[name + "_new"][t0:t0 + chunk[b]]
            if case["form"] == "bf16":
                out[name][page, :, pos % PAGE] = x.double()
                continue
            value, scale = _exact_quantise(x)
            out[name][page, :, pos % PAGE] = value
            out[name + "_scale"][page, :, pos % PAGE] = scale.double()
        t0 += chunk[b]
    return out


def _exact_read(case, s):
    ctx, chunk = _lens(case)
    value = _e4m3_values("cuda")
    got = {"k": [], "v": []}
    for b in range(case["batch"]):
        pages = s["table"][b, : -(-(ctx[b] + chunk[b]) // PAGE)].long()
        for name in got:
            x = value[s[name][pages].int()] * s[name + "_scale"][pages].double()[..., None]
            x = x.transpose(1, 2).reshape(-1, case["hkv"], case["d"])
            got[name].append(x[ctx[b]:ctx[b] + chunk[b]])
    return {k: torch.cat(x) for k, x in got.items()}


def _exact_penalize(case, s):
    parents, hist, prompt = _trees(case)
    v = case["vocab"]
    out = s["logits"].double()
    tokens, history = s["tokens"].tolist(), s["history"].tolist()
    h0 = r0 = 0
    for b, par in enumerate(parents):
        rep, pres, freq = (float(s[k][b]) for k in ("repetition", "presence", "frequency"))
        base = {}
        for i, t in enumerate(history[h0:h0 + hist[b]]):
            base[t] = base.get(t, 0) + (i >= prompt[b])
        paths = []
        for i, p in enumerate(par):
            paths.append([] if p < 0 else paths[p] + [tokens[r0 + i]])
            count = dict(base)
            for t in paths[i]:
                count[t] = count.get(t, 0) + 1
            if not count:
                continue
            ids = torch.tensor(list(count), device="cuda")
            n = torch.tensor(list(count.values()), dtype=torch.float64, device="cuda")
            x = out[r0 + i, ids]
            x = torch.where(x > 0, x / rep, x * rep) - freq * n - pres * (n > 0)
            out[r0 + i, ids] = x
        if s["bias_ids"] is not None:
            a, z = int(s["bias_offsets"][b]), int(s["bias_offsets"][b + 1])
            out[r0:r0 + len(par), s["bias_ids"][a:z].long()] += s["bias_values"][a:z].double()
        h0, r0 = h0 + hist[b], r0 + len(par)
    if s["allowed"] is not None:
        bits = torch.arange(32, dtype=torch.int32, device="cuda")
        ok = (s["allowed"][:, :, None] >> bits & 1).bool().reshape(out.shape[0], -1)[:, :v]
        out[~ok] = NEG_INF
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("attend"):
        return _exact_attend(case, s)
    if op == "append":
        return _exact_append(case, s)
    return _exact_read(case, s) if op == "read" else _exact_penalize(case, s)
