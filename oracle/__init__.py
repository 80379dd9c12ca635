"""fp64 CPU oracle for tree verification -- TEST INFRASTRUCTURE ONLY.

Only the test suite, the package smoke check and the benchmark's CPU-baseline
leg import this module.  The product path (the C-ABI library and its binding)
never imports, links or calls it, and shares no code with it.

The arithmetic lives in ``oracle.c`` (plain C, fp64, pthreads); this file
compiles it with gcc and marshals numpy arrays through ctypes.  See the header
of ``oracle.c`` for what is computed and which passage of the pages each step
follows.  The one step without arithmetic, the commit of the accepted path
(a copy by definition), is written out here with numpy: ``commit_kv``.
"""
from __future__ import annotations

import ctypes as C
import math
import os
import subprocess
import threading
from fractions import Fraction

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "oracle.c")
_LIB = os.path.join(_HERE, "liboracle.so")
_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile oracle.c into liboracle.so (no fast math, no fp contraction)."""
    with _lock:
        if force or not os.path.exists(_LIB) or os.path.getmtime(_LIB) < os.path.getmtime(_SRC):
            tmp = _LIB + f".tmp{os.getpid()}"
            subprocess.check_call(
                ["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-fPIC",
                 "-shared", "-pthread", _SRC, "-o", tmp, "-lm"])
            os.replace(tmp, _LIB)
    return _LIB


class _AttnArgs(C.Structure):
    _fields_ = [
        ("batch", C.c_int), ("num_q_heads", C.c_int), ("num_kv_heads", C.c_int),
        ("head_dim", C.c_int), ("block_size", C.c_int), ("max_blocks_per_seq", C.c_int),
        ("scale", C.c_double),
        ("q", C.c_void_p), ("k_prefix", C.c_void_p), ("v_prefix", C.c_void_p),
        ("block_table", C.c_void_p), ("k_nodes", C.c_void_p), ("v_nodes", C.c_void_p),
        ("parent", C.c_void_p), ("prefix_lens", C.c_void_p), ("node_offsets", C.c_void_p),
        ("dtype", C.c_int),
        ("q_scale", C.c_void_p), ("k_prefix_scale", C.c_void_p), ("v_prefix_scale", C.c_void_p),
        ("k_nodes_scale", C.c_void_p), ("v_nodes_scale", C.c_void_p),
    ]


class _AcceptArgs(C.Structure):
    _fields_ = [
        ("batch", C.c_int), ("vocab", C.c_int), ("kind", C.c_int), ("max_nodes", C.c_int),
        ("target", C.c_void_p), ("draft_probs", C.c_void_p), ("draft_tokens", C.c_void_p),
        ("parent", C.c_void_p), ("node_offsets", C.c_void_p), ("uniforms", C.c_void_p),
        ("retained_mask", C.c_void_p),
        ("accepted_len", C.c_void_p), ("path", C.c_void_p), ("bonus_token", C.c_void_p),
        ("status", C.c_void_p), ("pq_out", C.c_void_p),
        ("test", C.c_int), ("log_clamp", C.c_float), ("gamma", C.c_void_p),
    ]


def _load():
    global _lib
    if _lib is None:
        lib = C.CDLL(build())
        lib.oracle_tree_attention_rows.argtypes = [C.POINTER(_AttnArgs), C.c_int, C.c_void_p,
                                                   C.c_void_p, C.c_int]
        lib.oracle_tree_attention_rows.restype = C.c_int
        lib.oracle_accept.argtypes = [C.POINTER(_AcceptArgs), C.c_int]
        lib.oracle_accept.restype = C.c_int
        lib.oracle_quantise.argtypes = [C.c_float]
        lib.oracle_quantise.restype = C.c_uint64
        lib.oracle_scaled_draw.argtypes = [C.c_float, C.c_uint64]
        lib.oracle_scaled_draw.restype = C.c_uint64
        lib.oracle_retained_mass_row.argtypes = [C.c_void_p, C.c_void_p, C.c_int]
        lib.oracle_retained_mass_row.restype = C.c_float
        lib.oracle_retained_set_row.argtypes = [C.c_void_p, C.c_int, C.c_uint64, C.c_void_p,
                                                C.POINTER(C.c_uint64), C.POINTER(C.c_float),
                                                C.POINTER(C.c_int)]
        lib.oracle_retained_set_row.restype = C.c_int
        _lib = lib
    return _lib


def _ptr(a):
    return None if a is None else a.ctypes.data


def _c(a, dtype):
    return None if a is None else np.ascontiguousarray(a, dtype=dtype)


def default_threads() -> int:
    return max(1, os.cpu_count() or 1)


def tree_attention_rows(case: dict, rows, nthreads: int | None = None) -> np.ndarray:
    """fp64 outputs for the listed (b, local node, q head) rows -> [len(rows), D].
    Inputs are bf16 bit patterns, or, when case["dtype"] == "e4m3", E4M3 codes
    (uint8) with fp32 row scales case["<name>_scale"] (one per row of D)."""
    lib = _load()
    e4m3 = case.get("dtype", "bf16") == "e4m3"
    names = ("q", "k_prefix", "v_prefix", "k_nodes", "v_nodes")
    keep = {k: _c(case[k], np.uint8 if e4m3 else np.uint16) for k in names}
    scales = {k: (_c(case[k + "_scale"], np.float32) if e4m3 else None) for k in names}
    for k in ("block_table", "parent", "prefix_lens", "node_offsets"):
        keep[k] = _c(case[k], np.int32)
    rows = np.ascontiguousarray(np.asarray(rows, dtype=np.int32).reshape(-1, 3))
    hq, hkv, d = case["num_q_heads"], case["num_kv_heads"], case["head_dim"]
    scale = case.get("softmax_scale") or 1.0 / np.sqrt(d)
    args = _AttnArgs(int(case["batch"]), int(hq), int(hkv), int(d), int(case["block_size"]),
                     int(keep["block_table"].shape[1]), float(scale),
                     *[_ptr(keep[k]) for k in ("q", "k_prefix", "v_prefix", "block_table",
                                               "k_nodes", "v_nodes", "parent", "prefix_lens",
                                               "node_offsets")],
                     1 if e4m3 else 0, *[_ptr(scales[k]) for k in names])
    out = np.zeros((rows.shape[0], d), dtype=np.float64)
    rc = lib.oracle_tree_attention_rows(C.byref(args), rows.shape[0], _ptr(rows), _ptr(out),
                                        int(nthreads or default_threads()))
    if rc != 0:
        raise ValueError("oracle_tree_attention_rows: unsupported arguments")
    return out


def all_rows(case: dict) -> np.ndarray:
    """Every (b, i, h) row in output order ([total_nodes][Hq])."""
    off = np.asarray(case["node_offsets"])
    hq = case["num_q_heads"]
    rows = []
    for b in range(case["batch"]):
        for i in range(off[b + 1] - off[b]):
            for h in range(hq):
                rows.append((b, i, h))
    return np.asarray(rows, dtype=np.int32).reshape(-1, 3)


def tree_attention(case: dict, nthreads: int | None = None) -> np.ndarray:
    """Full fp64 output [total_nodes][Hq][D]."""
    rows = all_rows(case)
    out = tree_attention_rows(case, rows, nthreads)
    tot = int(np.asarray(case["node_offsets"])[-1])
    return out.reshape(tot, case["num_q_heads"], case["head_dim"])


def accept(case: dict, nthreads: int | None = None, want_pq: bool = True, test: int = 0,
           log_clamp: float = 20.0, gamma=None) -> dict:
    """Oracle accept pass.  Returns accepted_len, path, bonus_token, status, pq.
    test 0: ratio test with calibration factors `gamma` ([batch] fp32, None = 1);
    test 1: the log-space clamped test with bound `log_clamp`;
    test 2: the multi-candidate walk (siblings in order, residual updates)."""
    lib = _load()
    off = _c(case["node_offsets"], np.int32)
    batch = off.shape[0] - 1
    tot = int(off[-1])
    max_nodes = int(case["max_nodes"])
    keep = {
        "target": _c(case["target"], np.float32),
        "draft_probs": _c(case["draft_probs"], np.float32),
        "draft_tokens": _c(case["draft_tokens"], np.int32),
        "parent": _c(case["parent"], np.int32),
        "uniforms": _c(case["uniforms"], np.float32),
        "retained_mask": _c(case.get("retained_mask"), np.uint32),
        "gamma": None if gamma is None else _c(gamma, np.float32),
    }
    out = {
        "accepted_len": np.zeros(batch, np.int32),
        "path": np.zeros((batch, max_nodes), np.int32),
        "bonus_token": np.zeros(batch, np.int32),
        "status": np.zeros(batch, np.int32),
        "pq": np.zeros((max(tot, 1), 2), np.float32) if want_pq else None,
    }
    kind = 1 if case.get("kind", "probs") == "logits" else 0
    args = _AcceptArgs(batch, int(case["vocab"]), kind, max_nodes,
                       _ptr(keep["target"]), _ptr(keep["draft_probs"]), _ptr(keep["draft_tokens"]),
                       _ptr(keep["parent"]), _ptr(off), _ptr(keep["uniforms"]),
                       _ptr(keep["retained_mask"]),
                       _ptr(out["accepted_len"]), _ptr(out["path"]), _ptr(out["bonus_token"]),
                       _ptr(out["status"]), _ptr(out["pq"]), int(test), float(log_clamp),
                       _ptr(keep["gamma"]))
    rc = lib.oracle_accept(C.byref(args), int(nthreads or default_threads()))
    if rc != 0:
        raise ValueError("oracle_accept: unsupported arguments")
    return out


def e4m3_value(code: int) -> float:
    """The oracle's decoding of one E4M3 code."""
    lib = _load()
    lib.oracle_e4m3_to_f64.restype = C.c_double
    lib.oracle_e4m3_to_f64.argtypes = [C.c_uint8]
    return float(lib.oracle_e4m3_to_f64(code))


def quantise(r: float) -> int:
    return int(_load().oracle_quantise(C.c_float(r)))


def scaled_draw(u: float, S: int) -> int:
    return int(_load().oracle_scaled_draw(C.c_float(u), C.c_uint64(S)))


def retained_mass(q_row, mask_row) -> float:
    q = _c(q_row, np.float32)
    m = None if mask_row is None else _c(mask_row, np.uint32)
    return float(_load().oracle_retained_mass_row(_ptr(q), _ptr(m), int(q.shape[0])))


def commit_kv(k_nodes, v_nodes, parent, node_offsets, accepted_len, path, block_table,
              prefix_lens, k_pool, v_pool, max_nodes):
    """Commit of the accepted path, by definition (multimodal page §9.1 item 2:
    tree-node KV scattered into the preallocated target KV cache; on-device
    LLM page §2.3.2: slots only for the unique accepted path; edge-cloud page
    §5.2: the prefix cache grows by the accepted path).

    For each sequence b with a = accepted_len[b] and L = prefix_lens[b]: the
    root (local node 0) and path[b][0..a-1] become positions L .. L+a; the K
    and V rows of those nodes (every KV head) go to row pos % 16 of page
    block_table[b][pos // 16].  Status 5 (malformed: a < 0, a >= N, a bad
    extent, or a path step that is not a child of the previous node) or 7 (a
    position without a page) leaves the sequence untouched.  Arrays are numpy
    (bf16 as uint16 bit patterns).  Returns (k_pool, v_pool, new_prefix_lens,
    status) as new arrays."""
    k_pool = np.array(k_pool, copy=True)
    v_pool = np.array(v_pool, copy=True)
    off = np.asarray(node_offsets, np.int64)
    B = off.shape[0] - 1
    total = int(np.asarray(k_nodes).shape[0])
    num_blocks = k_pool.shape[0]
    table = np.asarray(block_table)
    new_lens = np.array(prefix_lens, np.int32, copy=True)
    status = np.zeros(B, np.int32)
    for b in range(B):
        n0, N = int(off[b]), int(off[b + 1] - off[b])
        a, L = int(accepted_len[b]), int(prefix_lens[b])
        ok = 1 <= N <= max_nodes and n0 >= 0 and n0 + N <= total and 0 <= a < N and L >= 0
        nodes = [0]
        if ok:
            for d in range(a):
                v = int(path[b][d])
                if not (1 <= v < N and int(parent[n0 + v]) == nodes[-1]):
                    ok = False
                    break
                nodes.append(v)
        if not ok:
            status[b] = 5
            continue
        pages = []
        for t in range(a + 1):
            pg = (L + t) // 16
            blk = int(table[b][pg]) if pg < table.shape[1] else -1
            if not 0 <= blk < num_blocks:
                break
            pages.append(blk)
        if len(pages) < a + 1:
            status[b] = 7
            continue
        for t, (v, blk) in enumerate(zip(nodes, pages)):
            k_pool[blk, :, (L + t) % 16, :] = k_nodes[n0 + v]
            v_pool[blk, :, (L + t) % 16, :] = v_nodes[n0 + v]
        new_lens[b] = L + a + 1
    return k_pool, v_pool, new_lens, status


def retained_threshold(mass: float) -> int:
    """T = floor(mass * 2^40) for an fp32 mass (exact in fp64)."""
    return int(np.floor(float(np.float32(mass)) * 2.0 ** 40))


def retained_set(q_rows, mass: float):
    """Retained set of every row of q_rows [R][V] fp32 (see oracle.c,
    oracle_retained_set_row).  Returns (mask [R][ceil(V/32)] uint32,
    z_fixed [R] uint64, z [R] fp32 = z_fixed * 2^-40 rounded once, kept [R])."""
    q = _c(np.atleast_2d(q_rows), np.float32)
    R, V = q.shape
    T = retained_threshold(mass)
    masks = np.zeros((R, (V + 31) // 32), np.uint32)
    zf = np.zeros(R, np.uint64)
    z32 = np.zeros(R, np.float32)
    kept = np.zeros(R, np.int32)
    lib = _load()
    for r in range(R):
        z = C.c_uint64(0)
        zs = C.c_float(0.0)
        k = C.c_int(0)
        row = np.ascontiguousarray(q[r])
        mrow = np.zeros((V + 31) // 32, np.uint32)
        if lib.oracle_retained_set_row(_ptr(row), int(V), C.c_uint64(T), _ptr(mrow), C.byref(z),
                                       C.byref(zs), C.byref(k)) != 0:
            raise ValueError("oracle_retained_set_row: bad arguments")
        masks[r] = mrow
        zf[r] = z.value
        z32[r] = zs.value
        kept[r] = k.value
    return masks, zf, z32, kept


# ------------------------------------------------------------------ chunk attention
def e4m3_table() -> np.ndarray:
    """The value of each of the 256 E4M3 codes."""
    return np.array([e4m3_value(c) for c in range(256)])


def chunk_attention(q, k_pool, v_pool, block_table, seq_lens, token_offsets, window: int = 0,
                    sinks: int = 0, scale: float | None = None, out=None) -> np.ndarray:
    """fp64 attention of every sequence's last C_b tokens over its pages, on
    real values: q [total, Hq, D], pools [blocks, Hkv, 16, D].  Row i of
    sequence b sits at p = seq_lens[b] - C_b + i and sees key k iff k <= p and
    (window == 0 or k > p - window or k < sinks).  Rows of no sequence keep
    what `out` holds (zeros by default)."""
    q, k_pool, v_pool = (np.asarray(x, np.float64) for x in (q, k_pool, v_pool))
    hq, d = q.shape[1:]
    g = hq // k_pool.shape[1]
    out = np.zeros(q.shape) if out is None else out
    for b, n in enumerate(np.asarray(seq_lens).tolist()):
        r0, r1 = int(token_offsets[b]), int(token_offsets[b + 1])
        if r1 <= r0:
            continue
        p = np.arange(n - (r1 - r0), n)[:, None]
        k = np.arange(n)
        seen = (k <= p) & ((k > p - window) | (k < sinks) if window else True)
        blk = np.asarray(block_table)[b, k // 16]
        used = seen.any(0)  # (pages that no row sees may be anything)
        for h in range(hq):
            keys = np.where(used[:, None], k_pool[np.where(used, blk, 0), h // g, k % 16], 0.0)
            vals = np.where(used[:, None], v_pool[np.where(used, blk, 0), h // g, k % 16], 0.0)
            s = np.where(seen, q[r0:r1, h] @ keys.T * (scale or d ** -0.5), -np.inf)
            w = np.exp(s - s.max(1, keepdims=True))
            out[r0:r1, h] = w @ vals / w.sum(1, keepdims=True)
    return out


# ------------------------------------------------------------------ cache writes and reads
def quantize_rows(x):
    """(codes, scale) of real rows [..., D], from the definition: scale =
    fl32(max|finite x| / 448), at least 2^-126, 1 for a row of zeros; the code
    of the E4M3 value nearest to x / scale (ties to the even code), saturating,
    NaN as 0x7F.  x / scale is compared with the middle of two values as x with
    scale times it: exact, a product of 24 by 5 bits."""
    x = np.asarray(x, np.float64)
    mag = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    with np.errstate(over="ignore"):
        scale = np.where(mag > 0, np.maximum((mag.astype(np.float32) / np.float32(448)), np.float32(2.0 ** -126)),
                         np.float32(1)).astype(np.float32)
    value = e4m3_table()[:127]
    codes = np.empty(x.shape, np.uint8)
    for i in np.ndindex(x.shape[:-1]):
        s = float(scale[i])
        middle = (value[:-1] + value[1:]) / 2 * s
        a = np.abs(x[i])
        lo = np.searchsorted(middle, a, side="left")    # ties down
        hi = np.searchsorted(middle, a, side="right")   # ties up
        c = np.where(lo % 2 == 0, lo, hi)
        c = np.where(np.signbit(x[i]), c | 0x80, c)
        codes[i] = np.where(np.isnan(x[i]), 0x7F, c)
    return codes, scale


def cache_places(block_table, seq_lens, token_offsets, num_blocks, total):
    """(status per sequence, {row: (block, position % 16)}, rows of failed
    sequences) of the chunks' tokens."""
    off = [int(o) for o in token_offsets]
    B = len(off) - 1
    if off[0] < 0 or any(b < a for a, b in zip(off, off[1:])) or off[-1] > total:
        return np.full(B, 5, np.int32), {}, []
    status, places, failed = np.zeros(B, np.int32), {}, []
    for b in range(B):
        c, n = off[b + 1] - off[b], int(seq_lens[b])
        if c == 0:
            continue
        pos = range(n - c, n)
        blocks = [int(block_table[b][p // 16]) if 0 <= p // 16 < len(block_table[b]) else -1 for p in pos] if n >= c else []
        if n < c:
            status[b] = 5
        elif any(k < 0 or k >= num_blocks for k in blocks):
            status[b] = 7
        rows = range(off[b], off[b + 1])
        if status[b]:
            failed += list(rows)
        else:
            places.update({r: (k, p % 16) for r, k, p in zip(rows, blocks, pos)})
    return status, places, failed


# ------------------------------------------------------------------ penalties
def penalize_logits(logits, draft_tokens, parent, node_offsets, history=(), history_offsets=None,
                    prompt_lens=None, repetition=None, presence=None, frequency=None, bias_ids=(),
                    bias_values=(), bias_offsets=None, allowed=None):
    """fp64 penalised rows from the definition; allowed: bool [total, V] or None."""
    out = np.asarray(logits, np.float64).copy()
    V = out.shape[1]
    for b in range(len(node_offsets) - 1):
        n0, n1 = int(node_offsets[b]), int(node_offsets[b + 1])
        h = list(history[int(history_offsets[b]):int(history_offsets[b + 1])]) if history_offsets is not None else []
        prompt = int(prompt_lens[b]) if prompt_lens is not None else 0
        bias = {}
        if bias_offsets is not None:
            for k in range(int(bias_offsets[b]), int(bias_offsets[b + 1])):
                bias[int(bias_ids[k])] = float(bias_values[k])
        rep = float(repetition[b]) if repetition is not None else 1.0
        pres = float(presence[b]) if presence is not None else 0.0
        freq = float(frequency[b]) if frequency is not None else 0.0
        for i in range(n1 - n0):
            c, j = {}, i
            for k, t in enumerate(h):
                c[int(t)] = c.get(int(t), 0) + (1 if k >= prompt else 0)
            while j > 0:
                t = int(draft_tokens[n0 + j])
                c[t] = c.get(t, 0) + 1
                j = int(parent[n0 + j])
            row = out[n0 + i]
            for t, n in c.items():
                if 0 <= t < V:
                    x = row[t]
                    x = x / rep if x > 0 else x * rep
                    row[t] = x - freq * n - (pres if n > 0 else 0.0)
            for t, x in bias.items():
                if 0 <= t < V:
                    row[t] += x
    return out if allowed is None else np.where(allowed, out, -np.inf)


# ------------------------------------------------------------------ head norms and positions
_TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136,
                   10 ** 99)


def rotate(x, positions, frequencies, weight=None, eps=1e-6, axes=None, interleaved=False, scale=1.0):
    """Rows x [T, H, D] normed and turned, in fp64; positions [axes, T]."""
    x = np.asarray(x, np.float64).copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    n = len(frequencies)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        f = float(frequencies[i])
        pos = np.asarray(positions[axes[i] if axes is not None else 0], np.int64)
        turn = pos * f
        if np.abs(turn).max(initial=0) >= 2.0 ** 20:  # whole turns taken off the exact product
            turn = np.array([float(Fraction(int(p)) * Fraction(f) % _TWO_PI) for p in pos])
        c, s = scale * np.cos(turn)[:, None], scale * np.sin(turn)[:, None]
        x[..., a], x[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return x


# ------------------------------------------------------------------ beams
def beam_select(logits, scores, beams, select, lengths=None, finished=None, end_token=-1, length_penalty=0.0):
    """(token, parent row, score, length, finished, key) lists of every request, from
    the definition in fp64; None for a request that is refused."""
    out = []
    for b in range(len(scores) // beams):
        found, bad = [], False
        for r in range(b * beams, (b + 1) * beams):
            s = float(scores[r])
            n = int(lengths[r]) if lengths is not None else 0
            ended = finished is not None and int(finished[r]) != 0
            bad |= math.isnan(s) or s == math.inf or n < 0 or n > 1 << 24
            if bad or s == -math.inf:
                continue
            if ended:
                found.append((s / max(n, 1) ** length_penalty, r, end_token, s, n, 1))
                continue
            x = np.asarray(logits[r], np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            if x.max() == np.inf:
                bad = True
            if bad or x.max() == -np.inf:
                continue
            total = math.log(np.exp(x - x.max()).sum())
            for v in np.lexsort((np.arange(len(x)), -x))[:select]:
                if x[v] > -np.inf:
                    d = s + (float(x[v] - x.max()) - total)  # (the maximum off first: it may be 1e38)
                    found.append((d / max(n + 1, 1) ** length_penalty, r, int(v), d, n + 1, int(v == end_token)))
        if bad:
            out.append(None)
            continue
        # (within a row by logit: the order that they are in)
        found = [c + (i,) for i, c in enumerate(found)]
        found.sort(key=lambda c: (-c[0], c[1], c[6]))
        found = found[:select] + [(-math.inf, -1, -1, -math.inf, 0, 0, 0)] * (select - len(found))
        out.append([(t, r, d, n, e, k) for k, r, t, d, n, e, _ in found])
    return out


# ------------------------------------------------------------------ pages
def _page_count(tokens):
    return -(-tokens // 16)


def alloc_pages(table, refs, begin, end):
    """Status per row; table (lists) and refs change in place."""
    free = [p for p, n in enumerate(refs) if n == 0]
    at, status = 0, []
    for row, lo, hi in zip(table, begin, end):
        if lo < 0 or hi < 0 or hi > 16 * len(row) or any(e >= len(refs) for e in row[lo // 16:_page_count(hi)]):
            status.append(5)
            continue
        lack = [t for t in range(lo // 16, _page_count(hi)) if row[t] < 0]
        fits = not lack or at + len(lack) <= len(free)
        status.append(0 if fits else 7)
        if fits:
            for i, t in enumerate(lack):
                row[t] = free[at + i]
                refs[row[t]] = 1
        at += len(lack)
    return status


def free_pages(table, refs, keep_begin, keep_end, sinks=0):
    status = []
    for row, lo, hi in zip(table, keep_begin, keep_end):
        bad = lo < 0 or hi < 0
        for t in range(len(row) if not bad else 0):
            if (t < lo // 16 and t >= _page_count(sinks)) or t >= _page_count(hi):
                if row[t] >= len(refs):
                    bad = True
                elif row[t] >= 0:
                    refs[row[t]] -= 1
                if row[t] >= 0:
                    row[t] = -1
        status.append(5 if bad else 0)
    return status


def fork_pages(table, lens, parents, refs):
    """(new table, new lengths, copies, status); refs change in place."""
    free = [p for p, n in enumerate(refs) if n == 0]
    before, width, pages = list(refs), len(table[0]), len(refs)
    new, ends, copies, status, at, seen = [], [], [], [], 0, set()
    for p in parents:
        row, copy, code, end = [-1] * width, (-1, -1, 0), 0, 0
        if p < -1 or p >= len(table) or (p >= 0 and not 0 <= lens[p] <= 16 * width):
            code = 5
        elif p >= 0:
            first, full, part = p not in seen, lens[p] // 16, lens[p] % 16
            seen.add(p)
            e = table[p][full] if part else None
            if part and (e < 0 or e >= pages or before[e] < 1):
                code = 5
            else:
                row = [x if t < full + (part > 0) or first else -1 for t, x in enumerate(table[p])]
                if part and (not first or before[e] > 1):
                    if at < len(free):
                        copy = (e, free[at], part)
                        row[full] = free[at]
                    else:
                        row, code = [-1] * width, 7
                    at += 1
                if code == 0:
                    end = lens[p]
                    if any(x >= pages for x in row):
                        code = 5
                    row = [-1 if x < 0 or x >= pages else x for x in row]
        new.append(row)
        ends.append(end)
        copies.append(copy)
        status.append(code)
    for rows, by in ((table, -1), (new, 1)):
        for row in rows:
            for e in row:
                if 0 <= e < pages:
                    refs[e] += by
    return new, ends, copies, status


def compact_pages(table, refs):
    """(new table, new refs, page map, moves, pages in use, status)."""
    n = sum(r != 0 for r in refs)
    to = [p if r else -1 for p, r in enumerate(refs)]
    moves = list(zip([p for p in range(n, len(refs)) if refs[p]], [p for p in range(n) if not refs[p]]))
    for src, dst in moves:
        to[src] = dst
    counts = [0] * len(refs)
    for p, r in enumerate(refs):
        if r:
            counts[to[p]] = r
    new = [[to[e] if 0 <= e < len(refs) else -1 for e in row] for row in table]
    status = [5 if any(e >= 0 and x < 0 for e, x in zip(row, out)) else 0 for row, out in zip(table, new)]
    return new, counts, to, [(s, d, 16) for s, d in moves], n, status
