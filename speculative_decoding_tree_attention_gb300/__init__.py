"""Tree verification for speculative decoding on GB300 (sm_103a).

Thin Python binding over the C-ABI library ``libtv.so`` (declared in
``include/tv.h``): argument marshalling only.  Every step of the computation
runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
the functions raise if the library cannot be loaded.

PyTorch is used for device memory and the current CUDA stream only.

    tree_attention(...)  -> out, status      (tv_tree_attention)
    tree_attention_fp8(...) -> out, status   (tv_tree_attention_fp8, E4M3 inputs)
    accept(...)          -> dict of outputs  (tv_accept)
    commit_kv(...)       -> new_prefix_lens, status (tv_commit_kv)
    retained_set(...)    -> mask, z_fixed, z, kept (tv_retained_set)
    chunk_attention(...) -> out, status      (tv_chunk_attention: prompts and decode tokens)
    chunk_attention_fp8(...) -> out, status  (tv_chunk_attention_fp8, E4M3 cache)
    append_kv(...), append_kv_fp8(...) -> status (tv_append_kv, tv_append_kv_fp8)
    read_kv_fp8(...)     -> k, v, status     (tv_read_kv_fp8)
    quantize_rows(...)   -> codes, scale     (tv_quantize_rows)
    commit_kv_fp8(...)   -> new_prefix_lens, status (tv_commit_kv_fp8)
    penalize_logits(...) -> out, status      (tv_penalize_logits)
"""
from __future__ import annotations

import ctypes as C
import os

__all__ = ["TVError", "load", "tree_attention", "tree_attention_fp8", "accept", "commit_kv", "retained_set",
           "chunk_attention", "chunk_attention_fp8", "chunk_params", "chunk_workspace_size",
           "append_kv", "append_kv_fp8", "read_kv_fp8", "quantize_rows", "commit_kv_fp8",
           "penalize_logits",
           "attention_workspace_size", "attention_plan", "attention_params",
           "TV_MAX_NODES", "TV_OK", "TV_ERR_BAD_TREE", "TV_ERR_DEVICE_TIMEOUT", "TV_ERR_NO_PAGE",
           "status_string"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libtv.so")

TV_OK = 0
TV_ERR_INVALID_ARG = 1
TV_ERR_UNSUPPORTED = 2
TV_ERR_WORKSPACE = 3
TV_ERR_CUDA = 4
TV_ERR_BAD_TREE = 5
TV_ERR_DEVICE_TIMEOUT = 6
TV_ERR_NO_PAGE = 7
TV_MAX_NODES = 512
TV_BLOCK_SIZE = 16
EXPORTS = ("tv_status_string", "tv_version", "tv_tree_attention_workspace_size",
           "tv_tree_attention", "tv_accept_workspace_size", "tv_accept", "tv_accept_ex",
           "tv_commit_kv",
           "tv_retained_set", "tv_selftest_wait_timeout", "tv_tree_attention_plan",
           "tv_tree_attention_no_alloc", "tv_tree_attention_fp8",
           "tv_chunk_attention_workspace_size", "tv_chunk_attention", "tv_chunk_attention_fp8",
           "tv_append_kv", "tv_append_kv_fp8", "tv_read_kv_fp8", "tv_quantize_rows",
           "tv_commit_kv_fp8", "tv_penalize_logits")


class TVError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class AttnParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("block_size", C.c_int32),
                ("max_blocks_per_seq", C.c_int32), ("num_blocks", C.c_int32),
                ("max_nodes", C.c_int32), ("total_nodes", C.c_int32),
                ("max_prefix_len", C.c_int32), ("softmax_scale", C.c_float),
                ("out_dtype", C.c_int32)]


class AttnPlan(C.Structure):
    _fields_ = [("ctas", C.c_int32), ("lanes", C.c_int32), ("virtual_ctas", C.c_int32),
                ("min_tiles", C.c_int32), ("workspace_bytes", C.c_size_t)]


class AcceptParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("vocab", C.c_int32), ("max_nodes", C.c_int32),
                ("total_nodes", C.c_int32), ("kind", C.c_int32)]


class AcceptOptions(C.Structure):
    _fields_ = [("test", C.c_int32), ("log_clamp", C.c_float), ("gamma", C.c_void_p)]


class RetainParams(C.Structure):
    _fields_ = [("rows", C.c_int32), ("vocab", C.c_int32), ("mass", C.c_float)]


class CommitParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("num_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("block_size", C.c_int32), ("max_blocks_per_seq", C.c_int32),
                ("num_blocks", C.c_int32), ("max_nodes", C.c_int32), ("total_nodes", C.c_int32)]


class ChunkParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("block_size", C.c_int32),
                ("max_blocks_per_seq", C.c_int32), ("num_blocks", C.c_int32),
                ("total_tokens", C.c_int32), ("max_len", C.c_int32), ("window", C.c_int32),
                ("sinks", C.c_int32), ("out_dtype", C.c_int32), ("softmax_scale", C.c_float),
                ("q_stride", C.c_int64)]


class CacheParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("num_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("block_size", C.c_int32), ("max_blocks_per_seq", C.c_int32),
                ("num_blocks", C.c_int32), ("total_tokens", C.c_int32), ("kv_stride", C.c_int64)]


class QuantParams(C.Structure):
    _fields_ = [("tokens", C.c_int32), ("heads", C.c_int32), ("head_dim", C.c_int32),
                ("stride", C.c_int64)]


class PenaltyParams(C.Structure):
    _fields_ = [("batch", C.c_int32), ("vocab", C.c_int32), ("max_nodes", C.c_int32),
                ("total_nodes", C.c_int32), ("total_history", C.c_int32), ("total_bias", C.c_int32),
                ("logits_dtype", C.c_int32)]


_lib = None


def load(path: str | None = None) -> C.CDLL:
    """Loads libtv.so (built in-tree by ``_build.build()``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise OSError(f"libtv.so not found at {p}: build it with "
                      "speculative_decoding_tree_attention_gb300._build.build()")
    lib = C.CDLL(p)
    vp, sz = C.c_void_p, C.c_size_t
    lib.tv_status_string.argtypes = [C.c_int]
    lib.tv_status_string.restype = C.c_char_p
    lib.tv_version.restype = C.c_int
    lib.tv_tree_attention_workspace_size.argtypes = [C.POINTER(AttnParams)]
    lib.tv_tree_attention_workspace_size.restype = sz
    lib.tv_tree_attention.argtypes = [C.POINTER(AttnParams)] + [vp] * 11 + [vp, sz, vp]
    lib.tv_tree_attention.restype = C.c_int
    lib.tv_tree_attention_fp8.argtypes = [C.POINTER(AttnParams)] + [vp] * 16 + [vp, sz, vp]
    lib.tv_tree_attention_fp8.restype = C.c_int
    lib.tv_accept_workspace_size.argtypes = [C.POINTER(AcceptParams)]
    lib.tv_accept_workspace_size.restype = sz
    lib.tv_accept.argtypes = [C.POINTER(AcceptParams)] + [vp] * 12 + [vp, sz, vp]
    lib.tv_accept.restype = C.c_int
    lib.tv_accept_ex.argtypes = [C.POINTER(AcceptParams), C.c_void_p] + [vp] * 12 + [vp, sz, vp]
    lib.tv_accept_ex.restype = C.c_int
    lib.tv_tree_attention_no_alloc.argtypes = [C.POINTER(AttnParams)] + [vp] * 11 + [vp]
    lib.tv_tree_attention_no_alloc.restype = C.c_int
    lib.tv_selftest_wait_timeout.argtypes = [vp, vp, C.c_ulonglong, vp]
    lib.tv_selftest_wait_timeout.restype = C.c_int
    lib.tv_tree_attention_plan.argtypes = [C.POINTER(AttnParams), C.c_int32, C.POINTER(AttnPlan)]
    lib.tv_tree_attention_plan.restype = C.c_int
    lib.tv_commit_kv.argtypes = [C.POINTER(CommitParams)] + [vp] * 12 + [vp]
    lib.tv_commit_kv.restype = C.c_int
    lib.tv_retained_set.argtypes = [C.POINTER(RetainParams)] + [vp] * 5 + [vp]
    lib.tv_retained_set.restype = C.c_int
    lib.tv_chunk_attention_workspace_size.argtypes = [C.POINTER(ChunkParams)]
    lib.tv_chunk_attention_workspace_size.restype = sz
    lib.tv_chunk_attention.argtypes = [C.POINTER(ChunkParams)] + [vp] * 9 + [sz, vp]
    lib.tv_chunk_attention.restype = C.c_int
    lib.tv_chunk_attention_fp8.argtypes = [C.POINTER(ChunkParams)] + [vp] * 12 + [sz, vp]
    lib.tv_chunk_attention_fp8.restype = C.c_int
    lib.tv_append_kv.argtypes = [C.POINTER(CacheParams)] + [vp] * 8 + [vp]
    lib.tv_append_kv.restype = C.c_int
    lib.tv_append_kv_fp8.argtypes = [C.POINTER(CacheParams)] + [vp] * 10 + [vp]
    lib.tv_append_kv_fp8.restype = C.c_int
    lib.tv_read_kv_fp8.argtypes = [C.POINTER(CacheParams)] + [vp] * 10 + [vp]
    lib.tv_read_kv_fp8.restype = C.c_int
    lib.tv_quantize_rows.argtypes = [C.POINTER(QuantParams)] + [vp] * 3 + [vp]
    lib.tv_quantize_rows.restype = C.c_int
    lib.tv_commit_kv_fp8.argtypes = [C.POINTER(CommitParams)] + [vp] * 16 + [vp]
    lib.tv_commit_kv_fp8.restype = C.c_int
    lib.tv_penalize_logits.argtypes = [C.POINTER(PenaltyParams)] + [vp] * 16 + [vp]
    lib.tv_penalize_logits.restype = C.c_int
    if path is None:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().tv_status_string(int(code)).decode()
    except OSError:
        return {0: "TV_OK", 1: "TV_ERR_INVALID_ARG", 2: "TV_ERR_UNSUPPORTED",
                3: "TV_ERR_WORKSPACE", 4: "TV_ERR_CUDA", 5: "TV_ERR_BAD_TREE",
                6: "TV_ERR_DEVICE_TIMEOUT", 7: "TV_ERR_NO_PAGE"}.get(int(code), "TV_ERR_UNKNOWN")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _check_dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


OUT_DTYPES = {"bf16": 0, "fp32": 1}


def attention_params(q_nodes, k_prefix_blocks, block_table, prefix_lens, *, num_kv_heads,
                     max_nodes, max_prefix_len, softmax_scale=0.0, out_dtype="bf16") -> AttnParams:
    total, hq, d = q_nodes.shape
    nb = k_prefix_blocks.shape[0]
    return AttnParams(int(prefix_lens.shape[0]), int(hq), int(num_kv_heads), int(d),
                      int(k_prefix_blocks.shape[2]), int(block_table.shape[1]), int(nb),
                      int(max_nodes), int(total), int(max_prefix_len), float(softmax_scale),
                      OUT_DTYPES[out_dtype])


def attention_workspace_size(params: AttnParams) -> int:
    return int(load().tv_tree_attention_workspace_size(C.byref(params)))


def attention_plan(params: AttnParams, sms: int = 0) -> dict:
    """tv_tree_attention_plan: the launch plan for `sms` SMs (0: the current
    device).  Raises TVError for invalid parameters."""
    plan = AttnPlan()
    rc = load().tv_tree_attention_plan(C.byref(params), int(sms), C.byref(plan))
    if rc != TV_OK:
        raise TVError(rc, "tv_tree_attention_plan")
    return {k: int(getattr(plan, k)) for k, _ in AttnPlan._fields_}


def tree_attention(q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes, v_nodes,
                   parent, prefix_lens, node_offsets, *, max_nodes: int, max_prefix_len: int,
                   softmax_scale: float = 0.0, out=None, status=None, workspace=None,
                   stream=None, out_dtype: str = "bf16"):
    """tv_tree_attention on the current stream.  Shapes as in include/tv.h:
    q_nodes [total, Hq, D] bf16; k/v_prefix_blocks [num_blocks, Hkv, 16, D] bf16;
    block_table [B, max_blocks] int32; k/v_nodes [total, Hkv, D] bf16;
    parent [total] int32; prefix_lens [B] int32; node_offsets [B+1] int32.
    out_dtype "bf16" or "fp32" (the output tensor's type).
    Returns (out, status); nothing is synchronised."""
    import torch
    lib = load()
    _check_dev(q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes, v_nodes,
               parent, prefix_lens, node_offsets)
    prm = attention_params(q_nodes, k_prefix_blocks, block_table, prefix_lens,
                           num_kv_heads=k_prefix_blocks.shape[1], max_nodes=max_nodes,
                           max_prefix_len=max_prefix_len, softmax_scale=softmax_scale,
                           out_dtype=out_dtype)
    if out is None:
        out = torch.empty(q_nodes.shape, device=q_nodes.device,
                          dtype=torch.float32 if out_dtype == "fp32" else torch.bfloat16)
    if status is None:
        status = torch.empty(prm.batch, dtype=torch.int32, device=q_nodes.device)
    need = int(lib.tv_tree_attention_workspace_size(C.byref(prm)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_nodes.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.tv_tree_attention(C.byref(prm), _ptr(q_nodes), _ptr(k_prefix_blocks),
                               _ptr(v_prefix_blocks), _ptr(block_table), _ptr(k_nodes),
                               _ptr(v_nodes), _ptr(parent), _ptr(prefix_lens),
                               _ptr(node_offsets), _ptr(out), _ptr(status), _ptr(workspace),
                               C.c_size_t(ws_bytes), _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_tree_attention")
    return out, status


def tree_attention_fp8(q_codes, q_scale, k_prefix_blocks, k_prefix_scale, v_prefix_blocks,
                       v_prefix_scale, block_table, k_nodes, k_nodes_scale, v_nodes,
                       v_nodes_scale, parent, prefix_lens, node_offsets, *, max_nodes: int,
                       max_prefix_len: int, softmax_scale: float = 0.0, out=None, status=None,
                       workspace=None, stream=None, out_dtype: str = "bf16"):
    """tv_tree_attention_fp8 on the current stream: E4M3 codes (uint8) with one
    fp32 scale per row of D = 128 codes.  q_codes [total, Hq, 128],
    q_scale [total, Hq]; k/v_prefix_blocks [num_blocks, Hkv, 16, 128],
    k/v_prefix_scale [num_blocks, Hkv, 16]; k/v_nodes [total, Hkv, 128],
    k/v_nodes_scale [total, Hkv]; the index arrays as for tree_attention.
    Returns (out, status); nothing is synchronised."""
    import torch
    lib = load()
    _check_dev(q_codes, q_scale, k_prefix_blocks, k_prefix_scale, v_prefix_blocks,
               v_prefix_scale, block_table, k_nodes, k_nodes_scale, v_nodes, v_nodes_scale,
               parent, prefix_lens, node_offsets)
    prm = attention_params(q_codes, k_prefix_blocks, block_table, prefix_lens,
                           num_kv_heads=k_prefix_blocks.shape[1], max_nodes=max_nodes,
                           max_prefix_len=max_prefix_len, softmax_scale=softmax_scale,
                           out_dtype=out_dtype)
    if out is None:
        out = torch.empty(q_codes.shape, device=q_codes.device,
                          dtype=torch.float32 if out_dtype == "fp32" else torch.bfloat16)
    if status is None:
        status = torch.empty(prm.batch, dtype=torch.int32, device=q_codes.device)
    need = int(lib.tv_tree_attention_workspace_size(C.byref(prm)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_codes.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.tv_tree_attention_fp8(C.byref(prm), _ptr(q_codes), _ptr(q_scale),
                                   _ptr(k_prefix_blocks), _ptr(k_prefix_scale),
                                   _ptr(v_prefix_blocks), _ptr(v_prefix_scale), _ptr(block_table),
                                   _ptr(k_nodes), _ptr(k_nodes_scale), _ptr(v_nodes),
                                   _ptr(v_nodes_scale), _ptr(parent), _ptr(prefix_lens),
                                   _ptr(node_offsets), _ptr(out), _ptr(status), _ptr(workspace),
                                   C.c_size_t(ws_bytes), _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_tree_attention_fp8")
    return out, status


def tree_attention_no_alloc(q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes,
                            v_nodes, parent, prefix_lens, node_offsets, *, max_nodes: int,
                            max_prefix_len: int, softmax_scale: float = 0.0, out=None,
                            status=None, stream=None):
    """tv_tree_attention_no_alloc: as tree_attention, for callers that cannot
    allocate device memory; any device scratch the launch plan needs comes
    from a fixed device array owned by the library (see include/tv.h).  Output
    tensors must be supplied by a caller that cannot allocate; they are
    created here only for convenience."""
    import torch
    lib = load()
    _check_dev(q_nodes, k_prefix_blocks, v_prefix_blocks, block_table, k_nodes, v_nodes,
               parent, prefix_lens, node_offsets)
    prm = attention_params(q_nodes, k_prefix_blocks, block_table, prefix_lens,
                           num_kv_heads=k_prefix_blocks.shape[1], max_nodes=max_nodes,
                           max_prefix_len=max_prefix_len, softmax_scale=softmax_scale)
    if out is None:
        out = torch.empty_like(q_nodes)
    if status is None:
        status = torch.empty(prm.batch, dtype=torch.int32, device=q_nodes.device)
    rc = lib.tv_tree_attention_no_alloc(C.byref(prm), _ptr(q_nodes), _ptr(k_prefix_blocks),
                                        _ptr(v_prefix_blocks), _ptr(block_table), _ptr(k_nodes),
                                        _ptr(v_nodes), _ptr(parent), _ptr(prefix_lens),
                                        _ptr(node_offsets), _ptr(out), _ptr(status),
                                        _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_tree_attention_no_alloc")
    return out, status


def accept(target, draft_probs, draft_tokens, parent, node_offsets, uniforms,
           retained_mask=None, *, max_nodes: int, kind: str = "probs", debug_pq: bool = False,
           outputs: dict | None = None, stream=None, test: str = "ratio", log_clamp: float = 0.0,
           gamma=None) -> dict:
    """tv_accept_ex on the current stream.  target/draft_probs [total, V] fp32,
    draft_tokens/parent [total] int32, node_offsets [B+1] int32, uniforms
    [total] fp32, retained_mask [total, ceil(V/32)] int32/uint32 or None.
    test: "ratio" (fl32(u q~) < fl32(gamma p~)), "log_clamp" (the clamped
    log-space test, bound log_clamp, 0 => 20) or "multi" (siblings tried in
    order with residual updates); gamma: [B] fp32 CUDA tensor of calibration
    factors or None (1).
    Returns dict(accepted_len, path, bonus_token, status, debug_pq)."""
    import torch
    lib = load()
    _check_dev(target, draft_probs, draft_tokens, parent, node_offsets, uniforms, retained_mask)
    total, V = target.shape
    B = node_offsets.shape[0] - 1
    dev = target.device
    prm = AcceptParams(int(B), int(V), int(max_nodes), int(total),
                       1 if kind == "logits" else 0)
    o = outputs or {}
    acc = o.get("accepted_len")
    if acc is None:
        acc = torch.empty(B, dtype=torch.int32, device=dev)
    path = o.get("path")
    if path is None:
        path = torch.empty(B, max_nodes, dtype=torch.int32, device=dev)
    bonus = o.get("bonus_token")
    if bonus is None:
        bonus = torch.empty(B, dtype=torch.int32, device=dev)
    status = o.get("status")
    if status is None:
        status = torch.empty(B, dtype=torch.int32, device=dev)
    dpq = o.get("debug_pq")
    if dpq is None and debug_pq:
        dpq = torch.empty(total, 2, dtype=torch.float32, device=dev)
    ws = o.get("workspace")
    if ws is None and (kind == "logits" or retained_mask is not None):
        need = int(lib.tv_accept_workspace_size(C.byref(prm)))
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check_dev(gamma)
    tests = {"ratio": 0, "log_clamp": 1, "multi": 2}
    if test not in tests:
        raise ValueError("test must be 'ratio', 'log_clamp' or 'multi'")
    opts = AcceptOptions(tests[test], float(log_clamp), None if gamma is None else gamma.data_ptr())
    rc = lib.tv_accept_ex(C.byref(prm), C.byref(opts), _ptr(target), _ptr(draft_probs), _ptr(draft_tokens),
                       _ptr(parent), _ptr(node_offsets), _ptr(uniforms), _ptr(retained_mask),
                       _ptr(acc), _ptr(path), _ptr(bonus), _ptr(status), _ptr(dpq), _ptr(ws),
                       C.c_size_t(ws_bytes), _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_accept")
    return dict(accepted_len=acc, path=path, bonus_token=bonus, status=status, debug_pq=dpq)


def selftest_wait_timeout(limit_ms: float = 10.0, stream=None):
    """tv_selftest_wait_timeout: a device wait that nothing ends, bounded by
    limit_ms.  Returns (status, waited_ns) after synchronising."""
    import torch
    lib = load()
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    waited = torch.zeros(1, dtype=torch.int64, device="cuda")
    rc = lib.tv_selftest_wait_timeout(_ptr(status), _ptr(waited), C.c_ulonglong(int(limit_ms * 1e6)),
                                      _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_selftest_wait_timeout")
    torch.cuda.synchronize()
    return int(status.item()), int(waited.item())


def commit_kv(k_nodes, v_nodes, parent, node_offsets, accepted_len, path, block_table,
              prefix_lens, k_prefix_blocks, v_prefix_blocks, *, max_nodes: int,
              new_prefix_lens=None, status=None, stream=None):
    """tv_commit_kv on the current stream: writes the root and the accepted
    path of every sequence into the paged pool (k/v_prefix_blocks, in place).
    Shapes as in include/tv.h; path [B, max_nodes] from accept().
    Returns (new_prefix_lens, status); nothing is synchronised."""
    import torch
    lib = load()
    _check_dev(k_nodes, v_nodes, parent, node_offsets, accepted_len, path, block_table,
               prefix_lens, k_prefix_blocks, v_prefix_blocks)
    total, hkv, d = k_nodes.shape
    B = int(node_offsets.shape[0] - 1)
    prm = CommitParams(B, int(hkv), int(d), int(k_prefix_blocks.shape[2]),
                       int(block_table.shape[1]), int(k_prefix_blocks.shape[0]), int(max_nodes),
                       int(total))
    dev = k_nodes.device
    if new_prefix_lens is None:
        new_prefix_lens = torch.empty(B, dtype=torch.int32, device=dev)
    if status is None:
        status = torch.empty(B, dtype=torch.int32, device=dev)
    rc = lib.tv_commit_kv(C.byref(prm), _ptr(k_nodes), _ptr(v_nodes), _ptr(parent),
                          _ptr(node_offsets), _ptr(accepted_len), _ptr(path), _ptr(block_table),
                          _ptr(prefix_lens), _ptr(k_prefix_blocks), _ptr(v_prefix_blocks),
                          _ptr(new_prefix_lens), _ptr(status), _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_commit_kv")
    return new_prefix_lens, status


def retained_set(draft_probs, mass: float, *, mask=None, z_fixed=None, z=None, kept=None,
                 stream=None):
    """tv_retained_set on the current stream: draft_probs [R, V] fp32.
    Returns (mask [R, ceil(V/32)] int32 bit patterns, z_fixed [R] int64
    (uint64 bits), z [R] fp32, kept [R] int32); nothing is synchronised."""
    import torch
    lib = load()
    _check_dev(draft_probs)
    R, V = draft_probs.shape
    dev = draft_probs.device
    if mask is None:
        mask = torch.empty(R, (V + 31) // 32, dtype=torch.int32, device=dev)
    if z_fixed is None:
        z_fixed = torch.empty(R, dtype=torch.int64, device=dev)
    if z is None:
        z = torch.empty(R, dtype=torch.float32, device=dev)
    if kept is None:
        kept = torch.empty(R, dtype=torch.int32, device=dev)
    prm = RetainParams(int(R), int(V), float(mass))
    rc = lib.tv_retained_set(C.byref(prm), _ptr(draft_probs), _ptr(mask), _ptr(z_fixed), _ptr(z),
                             _ptr(kept), _stream(stream))
    if rc != TV_OK:
        raise TVError(rc, "tv_retained_set")
    return mask, z_fixed, z, kept


# ---------------------------------------------------------------- chunks of new tokens
# The calls below take tensors of one CUDA device, which need not be the
# current one, and run on `stream` or on that device's current stream; buffers
# that they create belong to that stream.  A call costs the host a few
# microseconds per argument, more than the smallest of them take on the device,
# so the checks are written for the passing case.

def _torch():
    global _t
    if _t is None:
        import torch
        _t = torch
    return _t


_t = None


def _bad(name, what):
    raise ValueError(f"{name} must be {what}")


def _device(name, t):
    """The device index of the tensor that the others of a call go by."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        _bad(name, "a CUDA tensor")
    return t.get_device()


def _arg(name, t, dtype, shape, dev):
    """Checks one argument: a contiguous tensor of device `dev`, of dtype and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or t.get_device() != dev:
        _bad(name, f"a tensor on CUDA device {dev}")
    if t.dtype is not dtype:
        _bad(name, f"of type {dtype}, not {t.dtype}")
    if t.shape != shape:
        _bad(name, f"of shape {tuple(shape)}, not {tuple(t.shape)}")
    _bad(name, "contiguous")


def _rows(name, t, dtype, shape, dev):
    """_arg for rows that may lie a stride apart; returns that stride (0: packed)."""
    try:
        if t.is_contiguous() or t.shape[0] < 2:
            stride = 0
        else:
            stride = t.stride(0)
            if not t[0].is_contiguous() or stride < t[0].numel():
                _bad(name, "contiguous but for the stride between its rows")
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if stride == 0 and not t.is_contiguous() and not t[0].is_contiguous():
                _bad(name, "contiguous but for the stride between its rows")
            return stride
    except (AttributeError, IndexError):
        pass
    _arg(name, t, dtype, shape, dev)
    return 0


def _dims(name, t, n):
    """The shape of a tensor of n dimensions."""
    if not isinstance(t, _torch().Tensor) or t.dim() != n:
        _bad(name, f"a tensor of {n} dimensions")
    return t.shape


def _run(dev, stream, call):
    """call(stream handle) with `dev` and the stream current, so that what the
    call allocates belongs to that stream."""
    torch = _torch()
    if stream is None and torch.cuda.current_device() == dev:
        return call(_raw_stream(dev))  # (the handle alone: 3 us less than a Stream object)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif not isinstance(stream, torch.cuda.Stream) or stream.device.index != dev:
        _bad("stream", f"a stream of CUDA device {dev}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _raw_stream(dev):
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(dev).cuda_stream if get is None else get(dev)


def _empty(t, shape, dtype, dev):
    return _torch().empty(shape, dtype=dtype, device=f"cuda:{dev}") if t is None else t


def _int32(**counts):
    """Refuses what ctypes would cut to its low 32 bits."""
    for name, n in counts.items():
        if not -2 ** 31 <= n < 2 ** 31:
            _bad(name, "a 32-bit count")


def chunk_params(q, k_pool, block_table, seq_lens, *, max_len: int, window: int = 0, sinks: int = 0,
                 softmax_scale: float = 0.0, out_dtype: str = "bf16") -> ChunkParams:
    """The parameters of a chunk_attention or chunk_attention_fp8 call."""
    if out_dtype not in OUT_DTYPES:
        _bad("out_dtype", "'bf16' or 'fp32'")
    _int32(max_len=max_len, window=window, sinks=sinks)
    total, hq, d = q.shape
    return ChunkParams(seq_lens.shape[0], hq, k_pool.shape[1], d, k_pool.shape[2],
                       block_table.shape[1], k_pool.shape[0], total, max_len, window, sinks,
                       OUT_DTYPES[out_dtype], softmax_scale,
                       0 if q.is_contiguous() or total < 2 else q.stride(0))


def chunk_workspace_size(params: ChunkParams) -> int:
    return int(load().tv_chunk_attention_workspace_size(C.byref(params)))


def _chunk(q, q_scale, k_pool, k_scale, v_pool, v_scale, block_table, seq_lens, token_offsets, out,
           status, workspace, stream, max_len, window, sinks, softmax_scale, out_dtype):
    torch = _torch()
    lib = load()
    fp8 = q_scale is not None
    dev = _device("q", q)
    i32, f32, elem = torch.int32, torch.float32, torch.uint8 if fp8 else torch.bfloat16
    qs, ps = _dims("q", q, 3), _dims("k_pool", k_pool, 4)
    _rows("q", q, elem, qs, dev)
    _arg("k_pool", k_pool, elem, (ps[0], ps[1], TV_BLOCK_SIZE, qs[2]), dev)
    _arg("v_pool", v_pool, elem, ps, dev)
    if fp8:
        _arg("q_scale", q_scale, f32, qs[:2], dev)
        _arg("k_scale", k_scale, f32, ps[:3], dev)
        _arg("v_scale", v_scale, f32, ps[:3], dev)
    (batch,) = _dims("seq_lens", seq_lens, 1)
    _arg("seq_lens", seq_lens, i32, (batch,), dev)
    _arg("block_table", block_table, i32, (batch, _dims("block_table", block_table, 2)[1]), dev)
    _arg("token_offsets", token_offsets, i32, (batch + 1,), dev)
    prm = chunk_params(q, k_pool, block_table, seq_lens, max_len=max_len, window=window, sinks=sinks,
                       softmax_scale=softmax_scale, out_dtype=out_dtype)
    odt = f32 if prm.out_dtype else torch.bfloat16
    if out is not None:
        _arg("out", out, odt, qs, dev)
    if status is not None:
        _arg("status", status, i32, (batch,), dev)
    if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.get_device() == dev
                                      and workspace.is_contiguous()):
        _bad("workspace", f"a contiguous tensor on CUDA device {dev}")

    def call(handle):
        o, st = _empty(out, qs, odt, dev), _empty(status, batch, i32, dev)
        ws = workspace
        if ws is None:
            ws = _empty(None, int(lib.tv_chunk_attention_workspace_size(C.byref(prm))), torch.uint8, dev)
        tail = (block_table.data_ptr(), seq_lens.data_ptr(), token_offsets.data_ptr(), o.data_ptr(),
                st.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), handle)
        if fp8:
            rc = lib.tv_chunk_attention_fp8(C.byref(prm), q.data_ptr(), q_scale.data_ptr(), k_pool.data_ptr(),
                                            k_scale.data_ptr(), v_pool.data_ptr(), v_scale.data_ptr(), *tail)
        else:
            rc = lib.tv_chunk_attention(C.byref(prm), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), *tail)
        if rc != TV_OK:
            raise TVError(rc, "tv_chunk_attention_fp8" if fp8 else "tv_chunk_attention")
        return o, st

    return _run(dev, stream, call)


def chunk_attention(q, k_pool, v_pool, block_table, seq_lens, token_offsets, *, max_len: int,
                    window: int = 0, sinks: int = 0, softmax_scale: float = 0.0, out=None,
                    status=None, workspace=None, stream=None, out_dtype: str = "bf16"):
    """tv_chunk_attention: causal attention of the last token_offsets[b+1] -
    token_offsets[b] of the seq_lens[b] cached tokens of every sequence over
    that sequence's pages, optionally with a sliding window next to which the
    first `sinks` tokens stay visible.  q [total, Hq, D] bf16 (rows may be
    strided: a slice of a fused projection); k/v_pool [num_blocks, Hkv, 16, D]
    bf16; block_table [B, max_blocks], seq_lens [B], token_offsets [B+1] int32;
    max_len an upper bound of seq_lens.  Returns (out, status); nothing is
    synchronised."""
    return _chunk(q, None, k_pool, None, v_pool, None, block_table, seq_lens, token_offsets, out,
                  status, workspace, stream, max_len, window, sinks, softmax_scale, out_dtype)


def chunk_attention_fp8(q_codes, q_scale, k_pool, k_scale, v_pool, v_scale, block_table, seq_lens,
                        token_offsets, *, max_len: int, window: int = 0, sinks: int = 0,
                        softmax_scale: float = 0.0, out=None, status=None, workspace=None,
                        stream=None, out_dtype: str = "bf16"):
    """tv_chunk_attention_fp8: chunk_attention over an E4M3 cache: codes
    (uint8) with one fp32 scale per row of 128; q_codes and q_scale come from
    quantize_rows, the pools from append_kv_fp8.  Returns (out, status);
    nothing is synchronised."""
    if q_scale is None:
        _bad("q_scale", "a tensor")
    return _chunk(q_codes, q_scale, k_pool, k_scale, v_pool, v_scale, block_table, seq_lens,
                  token_offsets, out, status, workspace, stream, max_len, window, sinks,
                  softmax_scale, out_dtype)


# ---------------------------------------------------------------- the cache
def _cache_args(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, token_offsets, fp8):
    torch = _torch()
    dev = _device("k_pool", k_pool)
    i32, elem = torch.int32, torch.uint8 if fp8 else torch.bfloat16
    ps = _dims("k_pool", k_pool, 4)
    _arg("k_pool", k_pool, elem, (ps[0], ps[1], TV_BLOCK_SIZE, ps[3]), dev)
    _arg("v_pool", v_pool, elem, ps, dev)
    if fp8:
        _arg("k_scale", k_scale, torch.float32, ps[:3], dev)
        _arg("v_scale", v_scale, torch.float32, ps[:3], dev)
    (batch,) = _dims("seq_lens", seq_lens, 1)
    _arg("seq_lens", seq_lens, i32, (batch,), dev)
    width = _dims("block_table", block_table, 2)[1]
    _arg("block_table", block_table, i32, (batch, width), dev)
    _arg("token_offsets", token_offsets, i32, (batch + 1,), dev)
    return dev, batch, width, ps


def _row_pair(names, k, v, hkv, d, dev):
    """Checks K and V rows (bf16, strided by tokens alike); (rows, their stride)."""
    bf16 = _torch().bfloat16
    shape = (_dims(names[0], k, 3)[0], hkv, d)
    stride = _rows(names[0], k, bf16, shape, dev)
    if _rows(names[1], v, bf16, shape, dev) != stride:
        _bad(names[1], f"strided as {names[0]}")
    return shape[0], stride


def _append(k_new, v_new, block_table, seq_lens, token_offsets, k_pool, k_scale, v_pool, v_scale,
            status, stream, fp8):
    i32 = _torch().int32
    lib = load()
    dev, batch, width, ps = _cache_args(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                                        token_offsets, fp8)
    total, stride = _row_pair(("k_new", "v_new"), k_new, v_new, ps[1], ps[3], dev)
    if status is not None:
        _arg("status", status, i32, (batch,), dev)
    prm = CacheParams(batch, ps[1], ps[3], TV_BLOCK_SIZE, width, ps[0], total, stride)

    def call(handle):
        st = _empty(status, batch, i32, dev)
        rows = (k_new.data_ptr(), v_new.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                token_offsets.data_ptr())
        if fp8:
            rc = lib.tv_append_kv_fp8(C.byref(prm), *rows, k_pool.data_ptr(), k_scale.data_ptr(),
                                      v_pool.data_ptr(), v_scale.data_ptr(), st.data_ptr(), handle)
        else:
            rc = lib.tv_append_kv(C.byref(prm), *rows, k_pool.data_ptr(), v_pool.data_ptr(),
                                  st.data_ptr(), handle)
        if rc != TV_OK:
            raise TVError(rc, "tv_append_kv_fp8" if fp8 else "tv_append_kv")
        return st

    return _run(dev, stream, call)


def append_kv(k_new, v_new, block_table, seq_lens, token_offsets, k_pool, v_pool, *, status=None,
              stream=None):
    """tv_append_kv: writes the K/V rows of every sequence's chunk (rows
    token_offsets[b] .. token_offsets[b+1]-1 of k_new, v_new [total, Hkv, D]
    bf16, which may be strided by tokens) into the last positions of its
    seq_lens[b] cached tokens, in place in the pools [num_blocks, Hkv, 16, D].
    Returns status; nothing is synchronised."""
    return _append(k_new, v_new, block_table, seq_lens, token_offsets, k_pool, None, v_pool, None,
                   status, stream, False)


def append_kv_fp8(k_new, v_new, block_table, seq_lens, token_offsets, k_pool, k_scale, v_pool,
                  v_scale, *, status=None, stream=None):
    """tv_append_kv_fp8: append_kv into an E4M3 cache: every row becomes codes
    (uint8 pools) and one fp32 scale ([num_blocks, Hkv, 16]).  Returns status;
    nothing is synchronised."""
    return _append(k_new, v_new, block_table, seq_lens, token_offsets, k_pool, k_scale, v_pool,
                   v_scale, status, stream, True)


def read_kv_fp8(k_pool, k_scale, v_pool, v_scale, block_table, seq_lens, token_offsets, *,
                total_tokens: int | None = None, k_out=None, v_out=None, status=None, stream=None):
    """tv_read_kv_fp8: the last token_offsets[b+1] - token_offsets[b] of the
    seq_lens[b] cached tokens of every sequence, from an E4M3 cache back to bf16
    rows [total_tokens, Hkv, D] (total_tokens >= token_offsets[-1]; taken from
    k_out where that is given).  Returns (k, v, status); nothing is
    synchronised."""
    torch = _torch()
    lib = load()
    dev, batch, width, ps = _cache_args(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                                        token_offsets, True)
    hkv, d = ps[1], ps[3]
    if (k_out is None) != (v_out is None) or (k_out is None and total_tokens is None):
        raise ValueError("read_kv_fp8 needs total_tokens, or both k_out and v_out")
    total, stride = total_tokens, 0
    if k_out is not None:
        total, stride = _row_pair(("k_out", "v_out"), k_out, v_out, hkv, d, dev)
        if total_tokens not in (None, total):
            _bad("total_tokens", "the rows of k_out")
    if status is not None:
        _arg("status", status, torch.int32, (batch,), dev)
    prm = CacheParams(batch, hkv, d, TV_BLOCK_SIZE, width, ps[0], total, stride)

    def call(handle):
        k, v = _empty(k_out, (total, hkv, d), torch.bfloat16, dev), _empty(v_out, (total, hkv, d), torch.bfloat16, dev)
        st = _empty(status, batch, torch.int32, dev)
        rc = lib.tv_read_kv_fp8(C.byref(prm), k_pool.data_ptr(), k_scale.data_ptr(), v_pool.data_ptr(),
                                v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                token_offsets.data_ptr(), k.data_ptr(), v.data_ptr(), st.data_ptr(), handle)
        if rc != TV_OK:
            raise TVError(rc, "tv_read_kv_fp8")
        return k, v, st

    return _run(dev, stream, call)


def quantize_rows(x, *, codes=None, scale=None, stream=None):
    """tv_quantize_rows: bf16 rows [tokens, heads, D] (which may be strided by
    tokens) to E4M3 codes [tokens, heads, D] uint8 and scales [tokens, heads]
    fp32.  Returns (codes, scale); nothing is synchronised."""
    torch = _torch()
    lib = load()
    dev = _device("x", x)
    xs = _dims("x", x, 3)
    stride = _rows("x", x, torch.bfloat16, xs, dev)
    if codes is not None:
        _arg("codes", codes, torch.uint8, xs, dev)
    if scale is not None:
        _arg("scale", scale, torch.float32, xs[:2], dev)
    prm = QuantParams(xs[0], xs[1], xs[2], stride)

    def call(handle):
        c, s = _empty(codes, xs, torch.uint8, dev), _empty(scale, xs[:2], torch.float32, dev)
        rc = lib.tv_quantize_rows(C.byref(prm), x.data_ptr(), c.data_ptr(), s.data_ptr(), handle)
        if rc != TV_OK:
            raise TVError(rc, "tv_quantize_rows")
        return c, s

    return _run(dev, stream, call)


def commit_kv_fp8(k_nodes, k_nodes_scale, v_nodes, v_nodes_scale, parent, node_offsets,
                  accepted_len, path, block_table, prefix_lens, k_prefix_blocks, k_prefix_scale,
                  v_prefix_blocks, v_prefix_scale, *, max_nodes: int, new_prefix_lens=None,
                  status=None, stream=None):
    """tv_commit_kv_fp8: commit_kv of an E4M3 cache (codes and scales of the
    tree nodes, as tree_attention_fp8 takes them, copied to the pools in place).
    Returns (new_prefix_lens, status); nothing is synchronised."""
    torch = _torch()
    lib = load()
    dev = _device("k_nodes", k_nodes)
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    total, hkv, d = _dims("k_nodes", k_nodes, 3)
    ps = _dims("k_prefix_blocks", k_prefix_blocks, 4)
    (batch,) = _dims("prefix_lens", prefix_lens, 1)
    width = _dims("block_table", block_table, 2)[1]
    for name, t, dtype, shape in (
            ("k_nodes", k_nodes, u8, (total, hkv, d)), ("v_nodes", v_nodes, u8, (total, hkv, d)),
            ("k_nodes_scale", k_nodes_scale, f32, (total, hkv)),
            ("v_nodes_scale", v_nodes_scale, f32, (total, hkv)), ("parent", parent, i32, (total,)),
            ("node_offsets", node_offsets, i32, (batch + 1,)), ("accepted_len", accepted_len, i32, (batch,)),
            ("path", path, i32, (batch, max_nodes)), ("block_table", block_table, i32, (batch, width)),
            ("prefix_lens", prefix_lens, i32, (batch,)),
            ("k_prefix_blocks", k_prefix_blocks, u8, (ps[0], hkv, TV_BLOCK_SIZE, d)),
            ("v_prefix_blocks", v_prefix_blocks, u8, ps), ("k_prefix_scale", k_prefix_scale, f32, ps[:3]),
            ("v_prefix_scale", v_prefix_scale, f32, ps[:3]),
            ("new_prefix_lens", new_prefix_lens, i32, (batch,)), ("status", status, i32, (batch,))):
        if t is not None or name not in ("new_prefix_lens", "status"):
            _arg(name, t, dtype, shape, dev)
    _int32(max_nodes=max_nodes)
    prm = CommitParams(batch, hkv, d, TV_BLOCK_SIZE, width, ps[0], max_nodes, total)

    def call(handle):
        new, st = _empty(new_prefix_lens, batch, i32, dev), _empty(status, batch, i32, dev)
        rc = lib.tv_commit_kv_fp8(
            C.byref(prm), k_nodes.data_ptr(), k_nodes_scale.data_ptr(), v_nodes.data_ptr(),
            v_nodes_scale.data_ptr(), parent.data_ptr(), node_offsets.data_ptr(), accepted_len.data_ptr(),
            path.data_ptr(), block_table.data_ptr(), prefix_lens.data_ptr(), k_prefix_blocks.data_ptr(),
            k_prefix_scale.data_ptr(), v_prefix_blocks.data_ptr(), v_prefix_scale.data_ptr(),
            new.data_ptr(), st.data_ptr(), handle)
        if rc != TV_OK:
            raise TVError(rc, "tv_commit_kv_fp8")
        return new, st

    return _run(dev, stream, call)


# ---------------------------------------------------------------- logits
def _ptr_or_null(t):
    return None if t is None else t.data_ptr() or None


def penalize_logits(logits, draft_tokens, parent, node_offsets, *, max_nodes: int, history=None,
                    history_offsets=None, prompt_lens=None, repetition=None, presence=None,
                    frequency=None, bias_ids=None, bias_values=None, bias_offsets=None,
                    allowed_mask=None, out=None, status=None, stream=None):
    """tv_penalize_logits: repetition, frequency and presence penalties (counted
    over each sequence's history and each node's drafted path), biases and
    grammar masks on the target logits [total, V] (fp32 or bf16) of tree nodes,
    into out [total, V] fp32 (which may be fp32 logits themselves).  history
    [H], bias_ids [E] int32 and bias_values [E] fp32 are ragged by
    history_offsets and bias_offsets [B+1]; prompt_lens [B] int32; repetition,
    presence, frequency [B] fp32; allowed_mask [total, ceil(V/32)] int32 or
    uint32 bits.  Returns (out, status); nothing is synchronised."""
    torch = _torch()
    lib = load()
    i32, f32 = torch.int32, torch.float32
    dev = _device("logits", logits)
    total, vocab = _dims("logits", logits, 2)
    if logits.dtype is not f32 and logits.dtype is not torch.bfloat16:
        _bad("logits", f"of type float32 or bfloat16, not {logits.dtype}")
    _arg("logits", logits, logits.dtype, (total, vocab), dev)
    batch = _dims("node_offsets", node_offsets, 1)[0] - 1
    _arg("node_offsets", node_offsets, i32, (batch + 1,), dev)
    _arg("draft_tokens", draft_tokens, i32, (total,), dev)
    _arg("parent", parent, i32, (total,), dev)
    n_hist = n_bias = 0
    if (history is None) != (history_offsets is None):
        raise ValueError("history and history_offsets go together")
    if history is not None:
        (n_hist,) = _dims("history", history, 1)
        _arg("history", history, i32, (n_hist,), dev)
        _arg("history_offsets", history_offsets, i32, (batch + 1,), dev)
    if (bias_ids is None) != (bias_values is None) or (bias_ids is None) != (bias_offsets is None):
        raise ValueError("bias_ids, bias_values and bias_offsets go together")
    if bias_ids is not None:
        (n_bias,) = _dims("bias_ids", bias_ids, 1)
        _arg("bias_ids", bias_ids, i32, (n_bias,), dev)
        _arg("bias_values", bias_values, f32, (n_bias,), dev)
        _arg("bias_offsets", bias_offsets, i32, (batch + 1,), dev)
    if prompt_lens is not None:
        _arg("prompt_lens", prompt_lens, i32, (batch,), dev)
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        if t is not None:
            _arg(name, t, f32, (batch,), dev)
    if allowed_mask is not None:
        bits = torch.uint32 if getattr(allowed_mask, "dtype", None) is torch.uint32 else i32
        _arg("allowed_mask", allowed_mask, bits, (total, (vocab + 31) // 32), dev)
    if out is not None:
        _arg("out", out, f32, (total, vocab), dev)
    if status is not None:
        _arg("status", status, i32, (batch,), dev)
    _int32(max_nodes=max_nodes, history=n_hist, bias_ids=n_bias)
    prm = PenaltyParams(batch, vocab, max_nodes, total, n_hist, n_bias, 1 if logits.dtype is f32 else 0)

    def call(handle):
        o, st = _empty(out, (total, vocab), f32, dev), _empty(status, batch, i32, dev)
        p = _ptr_or_null
        rc = lib.tv_penalize_logits(
            C.byref(prm), p(logits), p(draft_tokens), p(parent), p(node_offsets),
            p(history), p(history_offsets),  # (an empty list has no address)
            p(prompt_lens), p(repetition), p(presence), p(frequency),
            p(bias_ids), p(bias_values), p(bias_offsets),
            p(allowed_mask), p(o), p(st), handle)
        if rc != TV_OK:
            raise TVError(rc, "tv_penalize_logits")
        return o, st

    return _run(dev, stream, call)
