"""What the head norms with rotation, the beam selection and the page calls refuse
before anything is enqueued (no GPU needed): bad sizes, missing and misaligned
pointers, overlapping arrays, short workspaces, and, in the binding, tensors that
are not CUDA tensors."""
import ctypes as C

import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from speculative_decoding_tree_attention_gb300 import _build

ODD = C.c_void_p(8 + (1 << 20))  # 8-byte aligned only


def at(i):
    """Addresses far apart, never dereferenced: the calls fail on the host."""
    return C.c_void_p((i + 1) << 40)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tv.load()


def each_pointer(n, required, call):
    """Every required pointer missing, every pointer misaligned."""
    for i in range(n):
        for x in (None, ODD):
            if x is None and i not in required:
                continue
            args = [at(j) for j in range(n)]
            args[i] = x
            assert call(args) == tv.TV_ERR_INVALID_ARG, (i, x)


# ------------------------------------------------------------------ rotation
def rotate(axes=(0,) * 64, **kw):
    base = dict(tokens=5, num_q_heads=4, num_kv_heads=2, head_dim=128, rotary_dim=128, interleaved=0, num_axes=1,
                weight_dtype=0, eps=1e-6, scale=0.0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0,
                axis_of_pair=(C.c_uint8 * 64)(*axes))
    return tv.RotateParams(**dict(base, **kw))


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(num_q_heads=0), dict(num_kv_heads=-1), dict(rotary_dim=130),
                                 dict(rotary_dim=-2), dict(rotary_dim=63), dict(head_dim=64), dict(interleaved=2),
                                 dict(num_axes=0), dict(num_axes=5), dict(weight_dtype=2), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=-1.0),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=511),
                                 dict(q_stride=516), dict(k_stride=248), dict(k_out_stride=-256),
                                 dict(q_out_stride=2 ** 39), dict(num_q_heads=2 ** 20 + 1),
                                 dict(tokens=2 ** 30, num_q_heads=2 ** 20), dict(tokens=2 ** 30 + 1),
                                 dict(axes=(0,) * 63 + (1,)), dict(axes=(3,) + (0,) * 63, num_axes=3)])
def test_rotate_arguments(lib, bad):
    assert lib.tv_rotate_qk(C.byref(rotate(**bad)), *[at(i) for i in range(8)], None) == tv.TV_ERR_INVALID_ARG


def test_rotate_pointers(lib):
    each_pointer(8, {0, 1, 4, 5, 6, 7}, lambda args: lib.tv_rotate_qk(C.byref(rotate()), *args, None))
    assert lib.tv_rotate_qk(None, *[at(i) for i in range(8)], None) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_rotate_qk(C.byref(rotate(head_dim=96)), *[at(i) for i in range(8)], None) == tv.TV_ERR_UNSUPPORTED
    # no tokens: nothing is enqueued, whatever the pointers
    assert lib.tv_rotate_qk(C.byref(rotate(tokens=0)), *[None] * 8, None) == tv.TV_OK


def test_rotate_overlaps(lib):
    """q is 5 rows of 512 values, k of 256; the slices of a projection of 1024."""
    def call(q, k, qo, ko, **strides):
        args = [at(i) for i in range(8)]
        args[0], args[1], args[6], args[7] = (C.c_void_p((1 << 30) + 2 * x) for x in (q, k, qo, ko))
        return lib.tv_rotate_qk(C.byref(rotate(**strides)), *args, None)
    far = 1 << 20
    wide = dict(q_stride=1024, k_stride=1024)
    wide_out = dict(q_out_stride=1024, k_out_stride=1024)
    for q, k, qo, ko, strides in ((0, far, 8, 2 * far, {}), (0, far, 4 * 512 + 504, 2 * far, {}),
                                  (0, far, far, 2 * far, {}), (0, far, 2 * far, 2 * far + 5 * 512 - 8, {}),
                                  (0, far, 2 * far, 0, {}), (0, far, 0, far + 8, {}),
                                  (0, 512, 8, 512, dict(wide, **wide_out)),          # within the rows
                                  (0, 512, 0, 512, dict(wide, q_out_stride=1024)),   # keys of another stride
                                  (0, 512, 256, 3 * far, dict(wide, **wide_out)),
                                  (0, 512, 768, 3 * far, dict(wide, **wide_out)),    # the end reaches the next row
                                  (0, 512, 2 * far, 2 * far + 256, wide_out)):
        assert call(q, k, qo, ko, **strides) == tv.TV_ERR_INVALID_ARG


def test_rotate_outputs_over_small_inputs(lib):
    """The weights (256 bytes), positions (20) and frequencies (512) of 5 tokens, at or
    next to the ends of q_out (5120 bytes) and k_out (2560)."""
    for o, rows in ((6, 5120), (7, 2560)):
        for i, size in ((2, 256), (3, 256), (4, 20), (5, 512)):
            for shift in (0, -((rows - 1) // 16 * 16), (size - 1) // 16 * 16):
                args = [at(j) for j in range(8)]
                args[o] = C.c_void_p(args[i].value + shift)
                assert lib.tv_rotate_qk(C.byref(rotate()), *args, None) == tv.TV_ERR_INVALID_ARG


# ------------------------------------------------------------------ beams
def beams(**kw):
    base = dict(batch=2, beams=3, select=6, vocab=1000, logits_dtype=1, end_token=2, length_penalty=0.5, logits_stride=0)
    return tv.BeamParams(**dict(base, **kw))


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=65536), dict(beams=0), dict(beams=65), dict(select=0),
                                 dict(select=65), dict(vocab=0), dict(vocab=1 << 18), dict(logits_dtype=2),
                                 dict(end_token=-2), dict(end_token=1000), dict(length_penalty=4.1),
                                 dict(length_penalty=-5.0), dict(length_penalty=float("nan")),
                                 dict(logits_stride=999), dict(logits_stride=-1000), dict(logits_stride=2 ** 38)])
def test_beam_arguments(lib, bad):
    p = beams(**bad)
    ok = C.c_size_t(1 << 40)
    assert lib.tv_beam_select(C.byref(p), *[at(i) for i in range(11)], ok, None) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_beam_select_workspace_size(C.byref(p)) == 0


def test_beam_pointers_and_workspace(lib):
    p = beams()
    need = lib.tv_beam_select_workspace_size(C.byref(p))
    # two parts a row (of whole 512 entries): a maximum and a sum each, a factor a
    # row (rounded to 256 bytes in all), and 6 entries a part
    assert need == 2 * 256 + 12 * 6 * 8
    big = beams(batch=64, beams=8, select=16, vocab=128256)
    # a CTA of 8 warps a row: four for every SM
    assert lib.tv_beam_select_workspace_size(C.byref(big)) == 512 * 8 + 512 * 8 * 8 * (1 + 16)

    def call(args):
        return lib.tv_beam_select(C.byref(p), *args, at(20), C.c_size_t(need), None)
    # logits, scores, lengths, finished, tokens, parents, scores_out, lengths_out, finished_out, status
    each_pointer(10, {0, 1, 2, 4, 5, 6, 9}, call)
    args = [at(i) for i in range(10)]
    for ws, size in ((None, need), (at(20), need - 1), (ODD, need)):
        assert lib.tv_beam_select(C.byref(p), *args, ws, C.c_size_t(size), None) == tv.TV_ERR_WORKSPACE
    # lengths are needed for their outputs and for a penalty
    args[2] = None
    assert lib.tv_beam_select(C.byref(beams(length_penalty=0.0)), *args, at(20), C.c_size_t(need), None) == tv.TV_ERR_INVALID_ARG
    # outputs over inputs (6 values each in, 12 out)
    for o in (4, 5, 6, 7, 8):
        for i in (1, 2, 3):
            for shift in (0, -32, 16):
                args = [at(j) for j in range(10)]
                args[o] = C.c_void_p(args[i].value + shift)
                assert call(args) == tv.TV_ERR_INVALID_ARG


def test_beam_overlaps_of_logits_and_workspace(lib):
    p = beams()
    need = lib.tv_beam_select_workspace_size(C.byref(p))

    def call(args, ws=at(20)):
        return lib.tv_beam_select(C.byref(p), *args, ws, C.c_size_t(need), None)
    for o in (4, 5, 6, 7, 8, 9):  # logits: 6 rows of 1000 fp32
        args = [at(j) for j in range(10)]
        args[o] = C.c_void_p(args[0].value + 6 * 4000 - 16)
        assert call(args) == tv.TV_ERR_INVALID_ARG
    for i in range(10):
        args = [at(j) for j in range(10)]
        assert call(args, args[i]) == tv.TV_ERR_INVALID_ARG
        assert call(args, C.c_void_p(args[i].value - need // 16 * 16 + 16)) == tv.TV_ERR_INVALID_ARG


# ------------------------------------------------------------------ pages
def pages(**kw):
    base = dict(rows=4, new_rows=6, block_size=16, max_blocks_per_seq=8, num_blocks=100, sinks=0)
    return tv.PageParams(**dict(base, **kw))


def page_calls(lib, p, args=lambda n: [at(i) for i in range(n)]):
    ok = C.c_size_t(1 << 30)
    yield lib.tv_alloc_pages(C.byref(p), *args(6), ok, None)
    yield lib.tv_free_pages(C.byref(p), *args(5), None)
    yield lib.tv_fork_pages(C.byref(p), *args(9), ok, None)
    yield lib.tv_compact_pages(C.byref(p), *args(8), None)


@pytest.mark.parametrize("bad", [dict(rows=0), dict(rows=65537), dict(block_size=32), dict(max_blocks_per_seq=0),
                                 dict(max_blocks_per_seq=2 ** 27 + 1), dict(num_blocks=0), dict(num_blocks=2 ** 30 + 1)])
def test_page_arguments(lib, bad):
    p = pages(**bad)
    for rc in page_calls(lib, p):
        assert rc == tv.TV_ERR_INVALID_ARG
    assert lib.tv_pages_workspace_size(C.byref(p)) == 0


def test_tables_whose_needs_pass_32_bits(lib):
    """Rows that lack 2^31 pages in all would wrap the sums of what they need."""
    p = pages(rows=65536, max_blocks_per_seq=32768)
    for rc in page_calls(lib, p):
        assert rc == tv.TV_ERR_INVALID_ARG
    assert lib.tv_pages_workspace_size(C.byref(p)) == 0
    p = pages(rows=65536, max_blocks_per_seq=32767)
    assert lib.tv_pages_workspace_size(C.byref(p)) > 0


def test_page_arguments_of_one_call(lib):
    ok = C.c_size_t(1 << 30)
    assert lib.tv_free_pages(C.byref(pages(sinks=-1)), *[at(i) for i in range(5)], None) == tv.TV_ERR_INVALID_ARG
    for n in (0, -1, 65537):
        assert lib.tv_fork_pages(C.byref(pages(new_rows=n)), *[at(i) for i in range(9)], ok, None) == tv.TV_ERR_INVALID_ARG


def test_page_pointers_and_workspace(lib):
    p = pages()
    need = lib.tv_pages_workspace_size(C.byref(p))
    # a list of all pages, a word a row (256 bytes at least each), 4096 words
    assert need == 512 + 256 + 4096 * 4
    size = C.c_size_t(need)
    each_pointer(5, {0, 1, 3, 4}, lambda a: lib.tv_alloc_pages(C.byref(p), *a, at(9), size, None))
    each_pointer(5, {0, 1, 4}, lambda a: lib.tv_free_pages(C.byref(p), *a, None))
    each_pointer(8, set(range(8)), lambda a: lib.tv_fork_pages(C.byref(p), *a, at(9), size, None))
    each_pointer(8, set(range(8)), lambda a: lib.tv_compact_pages(C.byref(p), *a, None))
    for ws, n in ((None, need), (at(9), need - 1), (ODD, need)):
        assert lib.tv_alloc_pages(C.byref(p), *[at(i) for i in range(5)], ws, C.c_size_t(n), None) == tv.TV_ERR_WORKSPACE
        assert lib.tv_fork_pages(C.byref(p), *[at(i) for i in range(8)], ws, C.c_size_t(n), None) == tv.TV_ERR_WORKSPACE


def test_page_overlaps(lib):
    p = pages()
    size = C.c_size_t(1 << 20)

    def fork(i, o, shift):
        args = [at(j) for j in range(8)]
        args[o] = C.c_void_p(args[i].value + shift)
        return lib.tv_fork_pages(C.byref(p), *args, at(9), size, None)
    # table (128 bytes), lens (16), parents (24) and counts (400) in; table (192),
    # lens (24), copies (72), status (24) out
    for i, n in ((0, 128), (1, 16), (2, 24), (3, 400)):
        for o, m in ((4, 192), (5, 24), (6, 72), (7, 24)):
            assert fork(i, o, 0) == tv.TV_ERR_INVALID_ARG
            assert fork(i, o, -((m - 1) // 16 * 16)) == tv.TV_ERR_INVALID_ARG
            assert fork(i, o, (n - 1) // 16 * 16) == tv.TV_ERR_INVALID_ARG

    def compact(i, o, shift):
        args = [at(j) for j in range(8)]
        args[o] = C.c_void_p(args[i].value + shift)
        return lib.tv_compact_pages(C.byref(p), *args, None)
    for i, o in ((0, 2), (1, 3)):  # in place as a whole or not at all
        assert compact(i, o, 16) == compact(i, o, -16) == tv.TV_ERR_INVALID_ARG
    for i, o in ((0, 3), (0, 4), (0, 5), (0, 6), (0, 7), (1, 2), (1, 4), (1, 5), (1, 6), (1, 7), (2, 3), (2, 4), (3, 4),
                 (4, 5), (3, 5), (2, 7)):
        assert compact(i, o, 0) == tv.TV_ERR_INVALID_ARG
    args = [at(j) for j in range(5)]
    for i, o in ((0, 1), (0, 4), (1, 4), (1, 2), (3, 0), (4, 3), (2, 4)):
        a = list(args)
        a[o] = a[i]
        assert lib.tv_alloc_pages(C.byref(p), *a, at(9), size, None) == tv.TV_ERR_INVALID_ARG
        assert lib.tv_free_pages(C.byref(p), *a, None) == tv.TV_ERR_INVALID_ARG


def copy(**kw):
    base = dict(entries=4, layers=1, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=100)
    return tv.CopyParams(**dict(base, **kw))


@pytest.mark.parametrize("bad", [dict(entries=-1), dict(layers=0), dict(num_kv_heads=0), dict(block_size=8),
                                 dict(num_blocks=0), dict(num_blocks=2 ** 26, num_kv_heads=2), dict(layers=2 ** 17)])
def test_copy_arguments(lib, bad):
    p = copy(**bad)
    assert lib.tv_copy_pages(C.byref(p), *[at(i) for i in range(5)], None) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_copy_pages_fp8(C.byref(p), *[at(i) for i in range(7)], None) == tv.TV_ERR_INVALID_ARG


def test_copy_pointers(lib):
    p = copy()
    # (count: 4-byte aligned)
    for n, call in ((5, lambda a: lib.tv_copy_pages(C.byref(p), *a, None)),
                    (7, lambda a: lib.tv_copy_pages_fp8(C.byref(p), *a, None))):
        for i in range(n):
            for x in (None, C.c_void_p((1 << 20) + 2) if i == 1 else ODD):
                if x is None and i in (1, n - 1):  # (count and status are optional)
                    continue
                args = [at(j) for j in range(n)]
                args[i] = x
                assert call(args) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_copy_pages(C.byref(copy(head_dim=96)), *[at(i) for i in range(5)], None) == tv.TV_ERR_UNSUPPORTED
    assert lib.tv_copy_pages(C.byref(copy(entries=0)), *[None] * 5, None) == tv.TV_OK


def test_page_workspace_and_copy_overlaps(lib):
    p = pages()
    need = lib.tv_pages_workspace_size(C.byref(p))
    size = C.c_size_t(need)
    for n, call in ((5, lib.tv_alloc_pages), (8, lib.tv_fork_pages)):
        for i in range(n):
            for shift in (0, -((need - 1) // 16 * 16)):
                args = [at(j) for j in range(n)]
                assert call(C.byref(p), *args, C.c_void_p(args[i].value + shift), size, None) == tv.TV_ERR_INVALID_ARG
    q = copy()
    # copies (48 bytes), count (4), pools of 100 pages of 2 heads
    for n, call, outs in ((5, lib.tv_copy_pages, {2: 819200, 3: 819200, 4: 16}),
                          (7, lib.tv_copy_pages_fp8, {2: 409600, 3: 12800, 4: 409600, 5: 12800, 6: 16})):
        for o, size in outs.items():
            for i in set(range(n)) - {o}:
                for shift in (0, -((size - 1) // 16 * 16)):
                    args = [at(j) for j in range(n)]
                    args[o] = C.c_void_p(args[i].value + shift)
                    assert call(C.byref(q), *args, None) == tv.TV_ERR_INVALID_ARG, (n, o, i)


# ------------------------------------------------------------------ the binding
def test_binding_wants_cuda_tensors():
    x, i, f = torch.zeros(2, 2, 128), torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.float64)
    t, pool = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(4, 2, 16, 128)
    for call in (lambda: tv.rotate_qk(x, None, i, f), lambda: tv.rotate_qk(None, None, None, None),
                 lambda: tv.beam_select(x[0], torch.zeros(2), beams=2), lambda: tv.beam_select(None, None, beams=1),
                 lambda: tv.alloc_pages(t, i, i), lambda: tv.free_pages(t, i), lambda: tv.fork_pages(t, i, i, i),
                 lambda: tv.compact_pages(t, i), lambda: tv.copy_pages(t[:, :3], pool, pool),
                 lambda: tv.copy_pages(None, pool, pool)):
        with pytest.raises(ValueError):
            call()


def test_rotary_axes():
    assert tv.rotary_axes([2, 3, 1]) == (0, 0, 1, 1, 1, 2)
    # axes in turn as long as they last; axis 0 takes the rest
    assert tv.rotary_axes([4, 2, 2], interleaved=True) == (0, 1, 2, 0, 1, 2, 0, 0)
    a = tv.rotary_axes([24, 20, 20], interleaved=True)
    assert [a.count(x) for x in range(3)] == [24, 20, 20] and a[58:] == (1, 2, 0, 0, 0, 0)
    for bad in ([], [3, -1]):
        with pytest.raises(ValueError):
            tv.rotary_axes(bad)
