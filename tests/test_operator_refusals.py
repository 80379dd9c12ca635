"""What the chunk attention, the cache writes and reads and the logit penalties
refuse before anything is enqueued (no GPU needed): bad sizes, missing and
misaligned pointers, short workspaces, and, in the binding, tensors that are
not CUDA tensors."""
import ctypes as C

import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from speculative_decoding_tree_attention_gb300 import _build

P = C.c_void_p(4096)    # never dereferenced: the calls fail on the host
ODD = C.c_void_p(4104)  # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tv.load()


def chunk(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=8,
                num_blocks=16, total_tokens=20, max_len=100, window=0, sinks=0, out_dtype=0,
                softmax_scale=0.0, q_stride=0)
    return tv.ChunkParams(**dict(base, **kw))


BAD_CHUNK = [dict(batch=0), dict(num_q_heads=0), dict(num_q_heads=9), dict(num_kv_heads=0), dict(block_size=32),
             dict(max_blocks_per_seq=0), dict(num_blocks=0), dict(total_tokens=-1), dict(max_len=-1),
             dict(max_len=129), dict(max_len=2 ** 31 - 1, max_blocks_per_seq=2 ** 30), dict(window=-1),
             dict(sinks=-1), dict(out_dtype=2), dict(num_blocks=2 ** 27, num_kv_heads=2),
             dict(total_tokens=2 ** 29), dict(q_stride=1023), dict(q_stride=8 * 128 + 4), dict(q_stride=-1024),
             dict(q_stride=2 ** 40), dict(softmax_scale=-0.1), dict(softmax_scale=float("nan")),
             dict(softmax_scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_CHUNK)
def test_chunk_arguments(lib, bad):
    p = chunk(**bad)
    ok = C.c_size_t(1 << 40)
    assert lib.tv_chunk_attention(C.byref(p), *[P] * 9, ok, None) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_chunk_attention_fp8(C.byref(p), *[P] * 12, ok, None) == tv.TV_ERR_INVALID_ARG
    if "q_stride" not in bad:
        assert tv.chunk_workspace_size(p) == 0


def test_chunk_unsupported(lib):
    ok = C.c_size_t(1 << 40)
    for p in (chunk(head_dim=96), chunk(num_q_heads=514)):
        assert lib.tv_chunk_attention(C.byref(p), *[P] * 9, ok, None) == tv.TV_ERR_UNSUPPORTED
    p = chunk(head_dim=64)
    assert lib.tv_chunk_attention_fp8(C.byref(p), *[P] * 12, ok, None) == tv.TV_ERR_UNSUPPORTED


def test_chunk_pointers_and_workspace(lib):
    p = chunk()
    need = tv.chunk_workspace_size(p)
    # a counter per CTA, rounded to 256 bytes, and two slots of 256 rows x D
    # fp32, 256 (m, l) and a 256-byte flag area
    slot = 256 * 128 * 4 + 256 * 8 + 256
    assert need > 0 and (need - 256) % (2 * slot) == 0
    for i in range(8):
        for x in (None, ODD):
            args = [P] * 9
            args[i] = x
            assert lib.tv_chunk_attention(C.byref(p), *args, C.c_size_t(need), None) == tv.TV_ERR_INVALID_ARG
    for i in range(11):
        args = [P] * 12
        args[i] = None
        assert lib.tv_chunk_attention_fp8(C.byref(p), *args, C.c_size_t(need), None) == tv.TV_ERR_INVALID_ARG
    for ws, size in ((None, need), (P, need - 1), (ODD, need)):
        assert lib.tv_chunk_attention(C.byref(p), *[P] * 8, ws, C.c_size_t(size), None) == tv.TV_ERR_WORKSPACE
    assert lib.tv_chunk_attention(None, *[P] * 9, C.c_size_t(need), None) == tv.TV_ERR_INVALID_ARG


def test_chunk_workspace_does_not_grow_past_the_sms(lib):
    slot = 256 * 128 * 4 + 256 * 8 + 256
    p = chunk(batch=500, total_tokens=100000, max_len=100000, max_blocks_per_seq=6250)
    assert tv.chunk_workspace_size(p) <= 160 * 2 * slot + 1024


def cache(**kw):
    base = dict(batch=2, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=8, num_blocks=16,
                total_tokens=20, kv_stride=0)
    return tv.CacheParams(**dict(base, **kw))


def cache_calls(lib, p, args=lambda n: [P] * n):
    yield lib.tv_append_kv(C.byref(p), *args(8), None)
    yield lib.tv_append_kv_fp8(C.byref(p), *args(10), None)
    yield lib.tv_read_kv_fp8(C.byref(p), *args(10), None)


@pytest.mark.parametrize("bad", [dict(batch=0), dict(num_kv_heads=0), dict(block_size=8), dict(max_blocks_per_seq=0),
                                 dict(num_blocks=0), dict(total_tokens=-1), dict(num_blocks=2 ** 26, num_kv_heads=2),
                                 dict(total_tokens=2 ** 30), dict(kv_stride=255), dict(kv_stride=260),
                                 dict(kv_stride=2 ** 39)])
def test_cache_arguments(lib, bad):
    for rc in cache_calls(lib, cache(**bad)):
        assert rc == tv.TV_ERR_INVALID_ARG


def test_cache_pointers(lib):
    for rc in cache_calls(lib, cache(head_dim=32)):
        assert rc == tv.TV_ERR_UNSUPPORTED
    for i in range(10):
        for x in (None, ODD):
            def args(n):
                out = [P] * n
                out[min(i, n - 1)] = x
                return out
            for rc in cache_calls(lib, cache(), args):
                assert rc == tv.TV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(heads=0), dict(stride=100), dict(stride=1028)])
def test_quantize_arguments(lib, bad):
    p = tv.QuantParams(**dict(dict(tokens=4, heads=8, head_dim=128, stride=0), **bad))
    assert lib.tv_quantize_rows(C.byref(p), P, P, P, None) == tv.TV_ERR_INVALID_ARG
    p = tv.QuantParams(4, 8, 96, 0)
    assert lib.tv_quantize_rows(C.byref(p), P, P, P, None) == tv.TV_ERR_UNSUPPORTED
    p = tv.QuantParams(4, 8, 128, 0)
    for i in range(3):
        args = [P] * 3
        args[i] = None
        assert lib.tv_quantize_rows(C.byref(p), *args, None) == tv.TV_ERR_INVALID_ARG


def test_commit_fp8_arguments(lib):
    base = dict(batch=2, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=8, num_blocks=16,
                max_nodes=16, total_nodes=20)
    for bad in (dict(batch=0), dict(block_size=8), dict(max_nodes=600), dict(total_nodes=1)):
        p = tv.CommitParams(**dict(base, **bad))
        assert lib.tv_commit_kv_fp8(C.byref(p), *[P] * 16, None) == tv.TV_ERR_INVALID_ARG
    p = tv.CommitParams(**base)
    for i in (0, 1, 3, 10, 11, 13, 15):
        args = [P] * 16
        args[9] = C.c_void_p(8192)
        args[i] = None
        assert lib.tv_commit_kv_fp8(C.byref(p), *args, None) == tv.TV_ERR_INVALID_ARG


def penalty(**kw):
    base = dict(batch=2, vocab=100, max_nodes=8, total_nodes=10, total_history=5, total_bias=5, logits_dtype=1)
    return tv.PenaltyParams(**dict(base, **kw))


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=65536, total_nodes=70000), dict(vocab=0),
                                 dict(vocab=1 << 18), dict(max_nodes=0), dict(max_nodes=513), dict(total_nodes=1),
                                 dict(total_history=-1), dict(total_bias=-1), dict(logits_dtype=2),
                                 dict(total_history=2 ** 30 + 1), dict(total_bias=2 ** 31 - 1)])
def test_penalty_arguments(lib, bad):
    assert lib.tv_penalize_logits(C.byref(penalty(**bad)), *[P] * 16, None) == tv.TV_ERR_INVALID_ARG


def test_penalty_pointers(lib):
    # logits, tokens, parent, offsets, history, its offsets, prompts, rates x 3,
    # bias ids, values, offsets, mask, out, status
    for i in (0, 1, 2, 3, 5, 11, 12, 14, 15):
        args = [P] * 16
        args[i] = None
        assert lib.tv_penalize_logits(C.byref(penalty()), *args, None) == tv.TV_ERR_INVALID_ARG
    for i in range(16):
        args = [P] * 16
        args[i] = C.c_void_p(4100)
        assert lib.tv_penalize_logits(C.byref(penalty()), *args, None) == tv.TV_ERR_INVALID_ARG
    args = [P] * 16  # bf16 logits cannot be their own output
    assert lib.tv_penalize_logits(C.byref(penalty(logits_dtype=0)), *args, None) == tv.TV_ERR_INVALID_ARG


def test_penalty_outputs_over_other_logits(lib):
    """out may be fp32 logits themselves; any other overlap is refused.  10 rows
    of 100: 4000 bytes of fp32, 2000 of bf16."""
    def at(logits, out, dtype):
        args = [P] * 16
        args[0], args[14] = C.c_void_p(logits), C.c_void_p(out)
        return lib.tv_penalize_logits(C.byref(penalty(logits_dtype=dtype)), *args, None)
    for dtype, size in ((1, 4000), (0, 2000)):
        for logits, out in ((1 << 20, (1 << 20) + 16), ((1 << 20) + 400, 1 << 20), (1 << 20, (1 << 20) + size - 16),
                            ((1 << 20) + 4000 - 16, 1 << 20)):
            assert at(logits, out, dtype) == tv.TV_ERR_INVALID_ARG


def test_binding_counts_of_64_bits():
    q, pool, table = torch.zeros(2, 2, 128), torch.zeros(2, 2, 16, 128), torch.zeros(1, 4, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    for kw in (dict(max_len=2 ** 32 + 5), dict(max_len=5, window=2 ** 31), dict(max_len=5, sinks=2 ** 32)):
        with pytest.raises(ValueError):
            tv.chunk_params(q, pool, table, lens, **kw)


def test_binding_wants_cuda_tensors():
    f, i = torch.zeros(2, 2, 128), torch.zeros(3, dtype=torch.int32)
    pool = torch.zeros(2, 2, 16, 128)
    for call in (lambda: tv.chunk_attention(f, pool, pool, i, i, i, max_len=1),
                 lambda: tv.chunk_attention_fp8(f, f, pool, pool, pool, pool, i, i, i, max_len=1),
                 lambda: tv.chunk_attention_fp8(f, None, pool, pool, pool, pool, i, i, i, max_len=1),
                 lambda: tv.append_kv(f, f, i, i, i, pool, pool),
                 lambda: tv.append_kv_fp8(f, f, i, i, i, pool, pool, pool, pool),
                 lambda: tv.read_kv_fp8(pool, pool, pool, pool, i, i, i, total_tokens=1),
                 lambda: tv.quantize_rows(f), lambda: tv.penalize_logits(f, i, i, i, max_nodes=1),
                 lambda: tv.commit_kv_fp8(f, f, f, f, i, i, i, i, i, i, pool, pool, pool, pool, max_nodes=1),
                 lambda: tv.quantize_rows(None), lambda: tv.chunk_attention(None, pool, pool, i, i, i, max_len=1)):
        with pytest.raises(ValueError):
            call()
