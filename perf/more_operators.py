"""The operators on the states of a decode step, as they are measured.

Three groups of calls next to the attention over the paged cache: the norm of
every query and key head with the position rotation (one position a token, or
several axes for images and video), the choice of the next beams over beams and
vocabulary, and the pages of the cache: given to sequences and taken back, passed
on to the children of a beam step with the copies that they need, and compacted.
``run`` computes each in plain torch operations, or with ``own = True`` through
the package.

Shapes are those of the repository's workloads: 32/8 heads of 128 with 512 to
4096 cached tokens (serving), 28/4 heads with 1600-token multimodal prompts (576
of them an image), 64/8 heads over 32768 tokens (long context), 4/4 heads of 64
(tiny), and vocabularies of 1000, 32000, 128256 and 151936.
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


def _rotate(name, tokens, hq, hkv, d, rot, axes, norm, interleaved=False, weights="bf16", far=4096, shape=1):
    """rot: the turned values of a head; axes: 1 or 3 (time, height, width); far: the largest position."""
    return _case(name, "rotate", tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, axes=axes, norm=norm,
                 interleaved=interleaved, weights=weights, far=far, shape=shape)


def _beams(name, batch, beams, select, vocab, dtype, ended=0.0, penalty=0.0, shape=1):
    return _case(name, "beams", batch=batch, beams=beams, select=select, vocab=vocab, dtype=dtype, ended=ended,
                 penalty=penalty, shape=shape)


def _fork(name, groups, beams, lens, tail, layers, hkv, d, form="bf16", shape=1):
    """lens: (shortest, longest) prompts, whose pages a group's beams share; tail: tokens that each beam has added."""
    return _case(name, "fork", groups=groups, beams=beams, len_lo=lens[0], len_hi=lens[1], tail=tail, layers=layers,
                 hkv=hkv, d=d, form=form, shape=shape)


def _turnover(name, rows, lens, gone, shape=1):
    return _case(name, "turnover", rows=rows, len_lo=lens[0], len_hi=lens[1], gone=gone, shape=shape)


def _compact(name, rows, lens, live, layers, hkv, d, form="bf16", shape=1):
    """live: the share of the pool's pages that is in use."""
    return _case(name, "compact", rows=rows, len_lo=lens[0], len_hi=lens[1], live=live, layers=layers, hkv=hkv, d=d,
                 form=form, shape=shape)


def listed():
    return [
        # one decode step of 16 serving sequences, head norms and rotation: latency
        _rotate("rotate 16 tokens, norms", 16, 32, 8, 128, 128, 1, True),
        # four 2048-token pieces of long prompts, 64/8 heads, far positions: bandwidth
        _rotate("rotate 8192 tokens, norms", 8192, 64, 8, 128, 128, 1, True, far=32768),
        # the nodes of four multimodal trees of 128 nodes, three axes, no norms
        _rotate("rotate 512 nodes, 3 axes", 512, 28, 4, 128, 128, 3, False),
        # four multimodal prompts of 1600 tokens, three axes and norms, fp32 weights
        _rotate("rotate 4 x 1600, 3 axes", 6400, 28, 4, 128, 128, 3, True, weights="fp32"),
        # one request with 4 beams, the 7B-like vocabulary: latency
        _beams("beams 1 x 4, V 32000", 1, 4, 4, 32000, "fp32"),
        # 64 requests of 8 beams over a large vocabulary, twice as many candidates
        # as beams (to go on with 8 when some of them end), a few beams ended
        _beams("beams 64 x 8, V 128256", 64, 8, 16, 128256, "bf16", 0.05, 0.6),
        # one beam step of 8 requests: new tables, counts, copies of half-filled pages
        _fork("fork 8 x 4 beams", 8, 4, (512, 4096), 40, 1, 8, 128),
        # 64 requests of 8 beams, two layers' pools in one allocation
        _fork("fork 64 x 8 beams", 64, 8, (512, 4096), 200, 2, 8, 128),
        # 4 of 16 serving sequences end, others take their place
        _turnover("turnover 16 rows", 16, (512, 4096), 0.25),
        # 512 long sequences, a sixteenth of them replaced: half a million pages
        _turnover("turnover 512 rows", 512, (1000, 32768), 0.0625),
        # the pool of a small server, a third of it holes
        _compact("compact 16 rows", 16, (512, 1600), 0.67, 1, 4, 128),
        # half of a larger pool in use, a quarter of its pages moves
        _compact("compact 64 rows", 64, (512, 1600), 0.5, 1, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "beams", "beams", "fork", "turnover", "compact"])
    shape = rng.randrange(1 << 20)
    if op == "rotate":
        while True:
            tokens = _log(rng, 1, 20000)
            hq, hkv, d = rng.choice([(4, 4, 64), (32, 32, 128), (32, 8, 128), (28, 4, 128), (64, 8, 128), (8, 1, 64), (5, 0, 64)])
            if tokens * (hq + hkv) * d <= 7.5e7:
                break
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4, d - 4]),
                "axes": rng.choice([1, 3]), "norm": rng.random() < 0.6, "interleaved": rng.random() < 0.3,
                "weights": rng.choice(["bf16", "fp32"]), "far": _log(rng, 100, 2000000), "shape": shape}
    if op == "beams":
        while True:
            batch, beams, vocab = _log(rng, 1, 96), _log(rng, 1, 32), _log(rng, 900, 200000)
            if batch * beams * vocab <= 6.5e7:
                break
        return {"op": op, "batch": batch, "beams": beams, "select": rng.choice([beams, beams, 2 * beams, rng.randint(1, 64)]),
                "vocab": vocab, "dtype": rng.choice(["fp32", "bf16"]), "ended": rng.choice([0.0, 0.1, 0.5]),
                "penalty": rng.choice([0.0, 0.6, 1.0]), "shape": shape}
    if op == "turnover":
        hi = _log(rng, 20, 32768)
        return {"op": op, "rows": _log(rng, 4, 512), "len_lo": rng.randint(1, hi), "len_hi": hi,
                "gone": rng.choice([0.02, 0.1, 0.3, 0.5]), "shape": shape}
    while True:
        c = {"op": op, "len_hi": _log(rng, 20, 8000), "layers": rng.choice([1, 1, 2, 4]), "hkv": rng.choice([1, 4, 8]),
             "d": rng.choice([64, 128]), "form": rng.choice(["bf16", "e4m3"]), "shape": shape}
        c["len_lo"] = rng.randint(1, c["len_hi"])
        if op == "fork":
            c["groups"], c["beams"], c["tail"] = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 1, 300)
            pages = c["groups"] * (c["len_hi"] // PAGE + 1 + c["beams"] * (c["tail"] // PAGE + 3))
        else:
            c["rows"], c["live"] = _log(rng, 1, 200), rng.uniform(0.2, 0.95)
            pages = c["rows"] * (c["len_hi"] // PAGE + 1) / c["live"]
        if pages * c["layers"] * c["hkv"] * c["d"] <= 3.5e7:
            return c


# ------------------------------------------------------------------ shapes
def _lens(case):
    """Lengths of the sequences (of a fork: of the groups' prompts), a pure function of the case."""
    r = random.Random(case["shape"])
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case.get("rows") or case["groups"])]


def _pages(n):
    return -(-n // PAGE)


def _page_bytes(case):
    return 2 * case["layers"] * case["hkv"] * PAGE * (case["d"] * 2 if case["form"] == "bf16" else case["d"] + 4)


def _parents(case):
    """The parent rows of a beam step: every child of a group from one of the group's beams."""
    r = random.Random(case["shape"] + 1)
    return [g * case["beams"] + r.randrange(case["beams"]) for g in range(case["groups"]) for _ in range(case["beams"])]


def _replaced(case):
    """Which rows of a turnover end, and the lengths of those that take their place."""
    r = random.Random(case["shape"] + 1)
    n = case["rows"]
    gone = set(r.sample(range(n), max(1, int(n * case["gone"]))))
    return [i in gone for i in range(n)], [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]


def _pool_size(case):
    """Pages of a turnover's pool: old and new sequences, and a fifth."""
    used = sum(map(_pages, _lens(case)))
    gone, new = _replaced(case)
    return used + sum(_pages(n) for n, g in zip(new, gone) if g) + used // 5 + 3


def work(case):
    op = case["op"]
    if op == "rotate":
        rows, d = case["tokens"] * (case["hq"] + case["hkv"]), case["d"]
        return {"bytes": rows * d * 4 + 4 * case["axes"] * case["tokens"],
                "flops": rows * (4 * d * case["norm"] + 3 * case["rot"])}
    if op == "beams":
        entries = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": int(entries * (2 if case["dtype"] == "bf16" else 4) * (1 - case["ended"])), "flops": 4 * entries}
    lens = _lens(case)
    if op == "turnover":
        gone, new = _replaced(case)
        touched = sum(_pages(a) + _pages(b) for a, b, g in zip(lens, new, gone) if g)
        return {"bytes": 4 * _pool_size(case) + 16 * touched, "flops": touched}
    if op == "compact":
        used = sum(map(_pages, lens))
        n = int(used / case["live"]) + 1
        moved = int(used * (1 - used / n))
        return {"bytes": 8 * used + 12 * n + 2 * moved * _page_bytes(case), "flops": n}
    ends = [n + case["tail"] for n in lens for _ in range(case["beams"])]
    seen, tokens, extra = set(), 0, 0
    for p in _parents(case):
        if p in seen:
            tokens += ends[p] % PAGE
            extra += _pages(ends[p])
        seen.add(p)
    lost = sum(_pages(ends[p]) for p in range(len(ends)) if p not in seen)
    return {"bytes": 8 * sum(_pages(ends[p]) for p in _parents(case)) + 8 * (extra + lost)
            + 2 * tokens * _page_bytes(case) // PAGE, "flops": extra + lost}


# ------------------------------------------------------------------ inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pools(case, pages, g):
    shape = (case["layers"], pages, case["hkv"], PAGE, case["d"])
    s = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if case["form"] == "bf16":
            s[name] = x
        else:
            s[name] = (x * 64.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = torch.rand(shape[:4], generator=g, device="cuda") * 0.02 + 0.001
    return s


def _table(pages, width, ids):
    """Block-table rows of the given numbers of pages, out of the ids in turn, -1 behind them."""
    n = torch.tensor(pages, device="cuda")
    start = torch.cumsum(n, 0) - n
    cols = torch.arange(width, device="cuda")
    have = cols < n[:, None]
    at = (start[:, None] + cols).clamp(max=ids.numel() - 1)
    return torch.where(have, ids[at].to(torch.int32), torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def _counts(table, pages):
    used = table[table >= 0].long()
    return torch.zeros(pages, dtype=torch.int32, device="cuda").index_add_(0, used, torch.ones_like(used, dtype=torch.int32))


def _axis_of_pair(case):
    """The position axis of each pair: a quarter time, the rest height and width in equal parts."""
    n = case["rot"] // 2
    if case["axes"] == 1:
        return [0] * n
    t = n // 4
    h = (n - t) // 2
    return [0] * t + [1] * h + [2] * (n - t - h)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "rotate":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        # q, k and v side by side, as a fused projection leaves them
        row = torch.randn(t, (hq + 2 * hkv) * d, generator=g, device="cuda", dtype=torch.bfloat16)
        start = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        if case["axes"] == 1:
            pos = ((start + at) % case["far"])[None]
        else:  # text, then an image of 24 columns, then text again, over and over
            in_image = at % 1600 < 576
            pos = torch.stack([torch.where(in_image, start + at // 1600, start + at),
                               torch.where(in_image, start + at % 1600 // 24, start + at),
                               torch.where(in_image, start + at % 24, start + at)])
        s = {"op": op, "q": row[:, : hq * d].view(t, hq, d), "d": d, "rot": case["rot"],
             "k": row[:, hq * d: (hq + hkv) * d].view(t, hkv, d) if hkv else None,
             "positions": pos.to(torch.int32).contiguous(), "interleaved": case["interleaved"], "eps": 1e-6,
             "frequencies": 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"]),
             "axes": _axis_of_pair(case), "q_weight": None, "k_weight": None}
        if case["norm"]:
            dt = torch.bfloat16 if case["weights"] == "bf16" else torch.float32
            s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if hkv else None
        s["axis_index"] = torch.tensor(s["axes"], device="cuda", dtype=torch.long)
        return s
    if op == "beams":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        logits = torch.randn(b * k, v, generator=g, device="cuda") * 2.5
        s = {"op": op, "logits": logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits,
             "scores": -30.0 * torch.rand(b, 1, generator=g, device="cuda").expand(b, k).reshape(-1)
             - 3.0 * torch.rand(b * k, generator=g, device="cuda"),
             "beams": k, "select": case["select"], "end_token": 2 % v, "penalty": case["penalty"],
             "finished": (torch.rand(b * k, generator=g, device="cuda") < case["ended"]).to(torch.int32)}
        length = torch.randint(2, 200, (b, 1), generator=g, device="cuda").expand(b, k).reshape(-1)
        early = (length * torch.rand(b * k, generator=g, device="cuda")).long() + 1
        s["lengths"] = torch.where(s["finished"] != 0, torch.minimum(early, length), length).to(torch.int32)
        return s
    lens = _lens(case)
    if op == "turnover":
        gone, new = _replaced(case)
        pages = _pool_size(case)
        width = max(map(_pages, lens + new))
        table = _table(list(map(_pages, lens)), width, torch.randperm(pages, generator=g, device="cuda"))
        return {"op": op, "table": table, "refs": _counts(table, pages),
                "keep_end": _i32([0 if x else n for n, x in zip(lens, gone)]),
                "begin": _i32([0 if x else n for n, x in zip(lens, gone)]),
                "lens": _i32([m if x else n for n, m, x in zip(lens, new, gone)])}
    if op == "compact":
        used = sum(map(_pages, lens))
        pages = int(used / case["live"]) + 1
        table = _table(list(map(_pages, lens)), max(map(_pages, lens)) + 2, torch.randperm(pages, generator=g, device="cuda"))
        return {"op": op, "table": table, "refs": _counts(table, pages), **_pools(case, pages, g)}
    # a fork: the prompts' full pages shared by a group's beams, what follows their own
    beams, tail = case["beams"], case["tail"]
    shared = [n // PAGE for n in lens for _ in range(beams)]
    ends = [n + tail for n in lens for _ in range(beams)]
    private = [_pages(e) - c for e, c in zip(ends, shared)]
    prompt = [n // PAGE for n in lens]
    # room for the copies of a step and for the pages that they replace
    pages = sum(prompt) + sum(private) + 3 * len(ends)
    ids = torch.randperm(pages, generator=g, device="cuda")
    width = max(map(_pages, ends)) + 1
    common = _table(prompt, width, ids).repeat_interleave(beams, 0)
    own_pages = _table(private, width, ids[sum(prompt):])
    at = torch.arange(width, device="cuda") - torch.tensor(shared, device="cuda")[:, None]
    table = torch.where(at < 0, common, own_pages.gather(1, at.clamp(min=0)))
    return {"op": op, "table": table.contiguous(), "spare": torch.full_like(table, -1), "refs": _counts(table, pages),
            "lens": _i32(ends), "spare_lens": _i32(ends), "parents": _i32(_parents(case)), **_pools(case, pages, g)}


# ------------------------------------------------------------------ plain forms
def _turn(x, weight, eps, cos, sin, rot, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_rotate(s):
    angle = s["positions"].double()[s["axis_index"]] * s["frequencies"][:, None]
    cos, sin = torch.cos(angle).float().T[:, None], torch.sin(angle).float().T[:, None]
    out = {"q": _turn(s["q"], s["q_weight"], s["eps"], cos, sin, s["rot"], s["interleaved"])}
    if s["k"] is not None:
        out["k"] = _turn(s["k"], s["k_weight"], s["eps"], cos, sin, s["rot"], s["interleaved"])
    return out


def _plain_beams(s):
    k, n = s["beams"], s["select"]
    x = s["logits"].float()
    rows, v = x.shape
    live = s["finished"] == 0
    top = x.amax(1, keepdim=True)
    lse = top[:, 0].double() + torch.log(torch.exp((x - top).double()).sum(1))
    # whole numbers that order a row: by logit, then the lower token first
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 18) + ((1 << 18) - 1 - torch.arange(v, device=x.device))
    each = min(n, v)
    token = (1 << 18) - 1 - (torch.topk(order, each, 1).values & ((1 << 18) - 1))
    score = s["scores"].double()[:, None] + (x.gather(1, token).double() - lse[:, None])
    first = torch.arange(each, device=x.device) == 0  # an ended beam has one candidate: itself
    score = torch.where(live[:, None], score, torch.where(first, s["scores"].double()[:, None], NEG_INF))
    token = torch.where(live[:, None], token, s["end_token"])
    length = s["lengths"][:, None] + live[:, None].int()
    key = score / length.clamp(min=1).double() ** s["penalty"]
    best = torch.sort(key.view(-1, k * each), dim=1, descending=True, stable=True).indices[:, :n]
    pad = torch.nn.functional.pad
    lack = n - best.shape[1]

    def take(a, fill):
        return pad(a.expand(rows, each).reshape(-1, k * each).gather(1, best), (0, lack), value=fill)

    row = torch.arange(rows, device=x.device)[:, None]
    none = pad(torch.isinf(key.view(-1, k * each).gather(1, best)), (0, lack), value=True)
    token, score = take(token, -1), take(score, NEG_INF)
    return {"tokens": torch.where(none, -1, token).int(), "parents": torch.where(none, -1, take(row, -1)).int(),
            "scores": torch.where(none, NEG_INF, score).float(), "lengths": torch.where(none, 0, take(length, 0)).int(),
            "finished": torch.where(none, 0, (~take(live[:, None], False) | (token == s["end_token"])).int()).int()}


def _entries(table):
    """Pages that a table's entries name (0 for none) and how often each entry counts (1, 0 for none)."""
    return table.clamp(min=0).flatten().long(), (table >= 0).flatten().int()


def _free_in_order(refs):
    return torch.sort((refs != 0).to(torch.int8), stable=True).indices


def _values(s):
    if "k_scale" not in s:
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _copy_rows(pool, src, dst, tokens):
    inside = (torch.arange(PAGE, device=pool.device) < tokens[:, None])[None, :, None]
    inside = inside if pool.dim() == 4 else inside[..., None]
    pool[:, dst] = torch.where(inside, pool[:, src], pool[:, dst])


def _copy_pools(s, src, dst, tokens):
    _copy_rows(s["k"], src, dst, tokens)
    _copy_rows(s["v"], src, dst, tokens)
    if "k_scale" in s:
        _copy_rows(s["k_scale"], src, dst, tokens)
        _copy_rows(s["v_scale"], src, dst, tokens)


def _plain_fork(s):
    table, refs, parent = s["table"], s["refs"], s["parents"].long()
    rows, width = table.shape
    at, cols = torch.arange(rows, device=table.device), torch.arange(width, device=table.device)
    first = torch.full((rows,), rows, device=table.device).scatter_reduce(0, parent, at, "amin")[parent] == at
    lens = s["lens"][parent]
    full, part = lens.long() // PAGE, lens % PAGE
    old = table[parent]
    src = old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0].long()
    need = (part > 0) & (~first | (refs[src.clamp(min=0)] > 1))
    dst = _free_in_order(refs)[: rows][(torch.cumsum(need, 0) - 1).clamp(min=0)]
    new = torch.where((cols < full[:, None]) | first[:, None], old, -1)
    here = (cols == full[:, None]) & (part > 0)[:, None]
    new = torch.where(here, torch.where(need, dst, src)[:, None], new).int()
    page, once = _entries(table)
    refs.index_add_(0, page, -once)
    page, once = _entries(new)
    refs.index_add_(0, page, once)
    _copy_pools(s, src[need], dst[need], part[need])
    s["table"], s["spare"] = new, table
    s["lens"] = lens
    return {"table": new, "lens": lens, "refs": refs, **_values(s)}


def _plain_turnover(s):
    table, refs = s["table"], s["refs"]
    cols = torch.arange(table.shape[1], device=table.device)
    out = cols >= (s["keep_end"][:, None] + PAGE - 1) // PAGE
    page, once = _entries(table)
    refs.index_add_(0, page, -once * out.flatten())
    table.masked_fill_(out, -1)
    need = (cols >= s["begin"][:, None] // PAGE) & (cols < (s["lens"][:, None] + PAGE - 1) // PAGE) & (table < 0)
    rank = (torch.cumsum(need.flatten(), 0) - 1).clamp(min=0)
    table.copy_(torch.where(need, _free_in_order(refs)[rank].view(table.shape).int(), table))
    refs.index_add_(0, table.clamp(min=0).flatten().long(), need.flatten().int())
    return {"table": table, "refs": refs}


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    live, at = refs != 0, torch.arange(refs.shape[0], device=refs.device)
    n = live.sum()
    moves = live & (at >= n)
    holes = _free_in_order(refs)  # those below n come first
    to = torch.where(moves, holes[(torch.cumsum(moves, 0) - 1).clamp(min=0)], torch.where(live, at, -1))
    new = torch.where(table >= 0, to[table.clamp(min=0).long()], -1).int()
    counts = torch.where(at < n, refs, 0).index_add_(0, to.clamp(min=0), refs * moves)
    src = moves.nonzero()[:, 0]
    dst, all_of_it = to[src], torch.full_like(src, PAGE)
    _copy_pools(s, src, dst, all_of_it)
    return {"table": new, "refs": counts, "page_map": to.int(), "count": n.int().view(1), **_values(s)}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import speculative_decoding_tree_attention_gb300 as tv
    op = s["op"]
    empty = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    if op == "rotate":
        if "keep" not in s:  # the buffers a serving loop keeps from step to step
            s["keep"] = {"q_out": empty(s["q"].shape, torch.bfloat16),
                         "k_out": None if s["k"] is None else empty(s["k"].shape, torch.bfloat16)}
        q, k = tv.rotate_qk(s["q"], s["k"], s["positions"], s["frequencies"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                            eps=s["eps"], axes=s["axes"], interleaved=s["interleaved"], **s["keep"])
        return {"q": q} if k is None else {"q": q, "k": k}
    if op == "beams":
        if "keep" not in s:
            shape = (s["logits"].shape[0] // s["beams"], s["select"])
            s["keep"] = {"tokens": empty(shape, i32), "parents": empty(shape, i32), "scores_out": empty(shape, torch.float32),
                         "lengths_out": empty(shape, i32), "finished_out": empty(shape, i32), "status": empty(shape[:1], i32),
                         "workspace": empty(tv.beam_workspace_size(s["logits"], beams=s["beams"], select=s["select"]), torch.uint8)}
        r = tv.beam_select(s["logits"], s["scores"], beams=s["beams"], select=s["select"], lengths=s["lengths"],
                           finished=s["finished"], end_token=s["end_token"], length_penalty=s["penalty"], **s["keep"])
        return {n: r[n] for n in ("tokens", "parents", "scores", "lengths", "finished")}
    rows = s["table"].shape[0]
    if "status" not in s:
        s["status"] = empty(rows, i32)
        s["workspace"] = empty(tv.page_workspace_size(s["table"], s["refs"], new_rows=rows), torch.uint8)
    if op == "turnover":
        tv.free_pages(s["table"], s["refs"], keep_end=s["keep_end"], status=s["status"])
        tv.alloc_pages(s["table"], s["refs"], s["lens"], begin=s["begin"], status=s["status"], workspace=s["workspace"])
        return {"table": s["table"], "refs": s["refs"]}
    scales = {"k_scale": s.get("k_scale"), "v_scale": s.get("v_scale")}
    if op == "compact":
        if "keep" not in s:
            s["keep"] = {"block_table_out": torch.empty_like(s["table"]), "ref_counts_out": torch.empty_like(s["refs"]),
                         "page_map": torch.empty_like(s["refs"]), "count": empty(2, i32),
                         "moves": empty((max(1, s["refs"].shape[0] // 2), 3), i32)}
        r = tv.compact_pages(s["table"], s["refs"], status=s["status"], **s["keep"])
        tv.copy_pages(r["moves"], s["k"], s["v"], count=r["count"][1:], **scales)
        return {"table": r["block_table"], "refs": r["ref_counts"], "page_map": r["page_map"], "count": r["count"][:1], **_values(s)}
    if "copies" not in s:
        s["copies"] = empty((rows, 3), i32)
    tv.fork_pages(s["table"], s["lens"], s["parents"], s["refs"], block_table_out=s["spare"], seq_lens_out=s["spare_lens"],
                  copies=s["copies"], status=s["status"], workspace=s["workspace"])
    tv.copy_pages(s["copies"], s["k"], s["v"], **scales)
    s["table"], s["spare"] = s["spare"], s["table"]
    s["lens"], s["spare_lens"] = s["spare_lens"], s["lens"]
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], **_values(s)}


def run(state):
    if own:
        return _own(state)
    plain = {"rotate": _plain_rotate, "beams": _plain_beams, "fork": _plain_fork, "turnover": _plain_turnover,
             "compact": _plain_compact}
    return plain[state["op"]](state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_rotate(case, s):
    rot, d = case["rot"], case["d"]
    pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2) for i in range(rot // 2)]
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x = s[name].double()
        if s[name + "_weight"] is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * s[name + "_weight"].double()
        y = x.clone()
        for i, (a, b) in enumerate(pairs):
            theta = s["positions"][_axis_of_pair(case)[i]].double() * 10000.0 ** (-2 * i / rot)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(theta), theta)[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        out[name] = y
    return out


def _exact_beams(case, s):
    k, n, v = case["beams"], case["select"], case["vocab"]
    out = {"tokens": [], "parents": [], "scores": [], "lengths": [], "finished": []}
    scores, lengths, finished = s["scores"].double().tolist(), s["lengths"].tolist(), s["finished"].tolist()
    for b in range(case["batch"]):
        found = []  # (key, row, token, score, length, ended): the best of every beam
        for r in range(b * k, b * k + k):
            if finished[r]:
                found.append((scores[r] / lengths[r] ** case["penalty"], r, s["end_token"], scores[r], lengths[r], 1))
                continue
            p = torch.log_softmax(s["logits"][r].double(), 0)
            best = torch.sort(p, descending=True, stable=True)
            for x, t in zip(best.values[:n].tolist(), best.indices[:n].tolist()):
                found.append(((scores[r] + x) / (lengths[r] + 1) ** case["penalty"], r, t, scores[r] + x, lengths[r] + 1,
                              int(t == s["end_token"])))
        found.sort(key=lambda c: (-c[0], c[1], c[2]))
        found = (found + [(0, -1, -1, NEG_INF, 0, 0)] * n)[:n]
        for name, i in (("parents", 1), ("tokens", 2), ("scores", 3), ("lengths", 4), ("finished", 5)):
            out[name].append([c[i] for c in found])
    return {name: torch.tensor(x, dtype=torch.float64 if name == "scores" else torch.int32) for name, x in out.items()}


def _recount(table, pages):
    refs = [0] * pages
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return refs


def _exact_fork(case, s):
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    free = iter([p for p, n in enumerate(refs) if n == 0])
    new, ends, seen = [], [], set()
    for p in s["parents"].tolist():
        row, last, tokens = list(table[p]), lens[p] // PAGE, lens[p] % PAGE
        if p in seen:
            row[lens[p] // PAGE + (tokens > 0):] = [-1] * (len(row) - lens[p] // PAGE - (tokens > 0))
        if tokens and (p in seen or refs[row[last]] > 1):
            src, row[last] = row[last], next(free)
            for name in ("k", "v", "k_scale", "v_scale"):
                if name in s:
                    s[name][:, row[last], :, :tokens] = s[name][:, src, :, :tokens]
        seen.add(p)
        new.append(row)
        ends.append(lens[p])
    return {"table": _i32(new), "lens": _i32(ends), "refs": _i32(_recount(new, len(refs))), **_values(s)}


def _exact_turnover(case, s):
    table, pages = s["table"].tolist(), s["refs"].shape[0]
    for row, keep in zip(table, s["keep_end"].tolist()):
        row[_pages(keep):] = [-1] * (len(row) - _pages(keep))
    free = iter([p for p, n in enumerate(_recount(table, pages)) if n == 0])
    for row, lo, hi in zip(table, s["begin"].tolist(), s["lens"].tolist()):
        for t in range(lo // PAGE, _pages(hi)):
            if row[t] < 0:
                row[t] = next(free)
    return {"table": _i32(table), "refs": _i32(_recount(table, pages))}


def _exact_compact(case, s):
    table, refs = s["table"].tolist(), s["refs"].tolist()
    n = sum(r != 0 for r in refs)
    to = [p if r else -1 for p, r in enumerate(refs)]
    src = [p for p in range(n, len(refs)) if refs[p]]
    dst = [p for p in range(n) if not refs[p]]
    for a, b in zip(src, dst):
        to[a] = b
    for name in ("k", "v", "k_scale", "v_scale"):
        if name in s:
            s[name][:, dst] = s[name][:, src]
    new = [[to[e] if e >= 0 else -1 for e in row] for row in table]
    return {"table": _i32(new), "refs": _i32(_recount(new, len(refs))), "page_map": _i32(to), "count": _i32([n]), **_values(s)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "beams": _exact_beams, "fork": _exact_fork, "turnover": _exact_turnover,
            "compact": _exact_compact}[case["op"]](case, s)
