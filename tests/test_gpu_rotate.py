"""GPU parity of tv_rotate_qk (head norms and rotation by positions on one or
several axes) with fp64: both pairings, partial rotations, head sizes, strides, far
and negative positions, in place.

Tolerance of a value y of a pair of length r = scale hypot(a, b) (of a value that is
not turned: r = |y|): half a bf16 step, 2^-8 |y|, and 2^-19 r for the fp32
arithmetic: of the norm, the sum of 128 squares (4 lanes-deep shuffles and 8
products in turn: 13 roundings, halved by the root), the root (2 ulp) and two
products; of the angle, a rounding to 24 bits of a half-turn (pi 2^-25), sincospif (2
ulp), the factor; two products and a sum: less than 24 roundings of 2^-24 in all."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu


def rows(n, heads, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g) * 2.0 ** torch.randint(-6, 7, (n, heads, 1), generator=g)
    return x.to(torch.bfloat16)


def frequencies(pairs, base=10000.0):
    return torch.from_numpy(base ** (-np.arange(pairs) / max(pairs, 1)))


def check(got, x, positions, freq, weight, eps, axes, interleaved, scale):
    x = x.double().numpy()
    w = None if weight is None else weight.double().numpy()
    f = freq.numpy()
    ref = oracle.rotate(x, positions, f, w, eps, axes, interleaved, scale)
    plain = oracle.rotate(x, positions, [], w, eps)
    n = len(f)
    r = np.abs(plain)
    a, b = (np.s_[..., 0:2 * n:2], np.s_[..., 1:2 * n:2]) if interleaved else (np.s_[..., :n], np.s_[..., n:2 * n])
    r[a] = r[b] = scale * np.hypot(plain[a], plain[b])
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * r + 1e-40).all(), float((err - 2.0 ** -8 * np.abs(ref)).max())


CASES = [  # tokens, Hq, Hkv, D, pairs, axes, interleaved, norms, weights' type
    (1, 1, 1, 128, 64, 1, False, True, torch.bfloat16),
    (1, 32, 8, 128, 64, 1, False, True, torch.bfloat16),
    (7, 28, 4, 128, 64, 3, False, False, None),
    (33, 28, 4, 128, 64, 4, True, True, torch.float32),
    (5, 4, 4, 64, 32, 1, True, True, torch.bfloat16),
    (300, 5, 3, 64, 32, 3, False, True, torch.float32),
    (3, 3, 0, 128, 64, 1, False, True, torch.bfloat16),
    (17, 7, 1, 128, 16, 1, False, True, torch.bfloat16),   # a quarter is turned
    (17, 7, 1, 128, 62, 3, False, True, torch.bfloat16),   # halves that are not 8-byte aligned
    (17, 7, 1, 128, 61, 2, False, False, None),
    (17, 7, 1, 128, 61, 2, True, True, torch.float32),
    (9, 2, 2, 64, 3, 1, False, True, torch.bfloat16),
    (9, 2, 2, 64, 1, 1, True, False, None),
    (9, 2, 2, 64, 0, 1, False, True, torch.float32),       # norms alone
    (2500, 8, 2, 128, 64, 1, False, True, torch.bfloat16),
    (20000, 1, 0, 64, 32, 1, False, False, None),
]


@pytest.mark.parametrize("case", CASES)
def test_parity(case):
    ensure_built()
    t, hq, hkv, d, pairs, n_axes, interleaved, norms, wt = case
    q, k = rows(t, hq, d, t + d), rows(t, max(hkv, 1), d, t + d + 1)
    g = np.random.default_rng(t)
    pos = g.integers(0, 40000, (n_axes, t)).astype(np.int32)
    axes = tuple(int(x) for x in g.integers(0, n_axes, pairs)) if n_axes > 1 else None
    qw = (1 + 0.3 * torch.randn(d)).to(wt) if norms else None
    kw = (1 + 0.3 * torch.randn(d)).to(wt) if norms and hkv else None
    freq = frequencies(pairs)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    p, f = (torch.from_numpy(pos).cuda(), freq.cuda()) if pairs else (None, None)
    if n_axes == 1 and pairs:
        p = p[0]
    qo, ko = tv.rotate_qk(dev(q), dev(k) if hkv else None, p, f, q_weight=dev(qw), k_weight=dev(kw), eps=1e-5,
                          axes=axes, interleaved=interleaved, scale=1.25)
    check(qo, q, pos, freq, qw, 1e-5, axes, interleaved, 1.25)
    if hkv:
        check(ko, k, pos, freq, kw, 1e-5, axes, interleaved, 1.25)
    else:
        assert ko is None


def test_far_and_negative_positions():
    """Angles of up to 2^31 radians, exactly reduced; the other sign turns back."""
    ensure_built()
    pos = np.array([[0, 1, -1, 2 ** 20, -2 ** 24, 2 ** 31 - 1, -2 ** 31, 123456789]], np.int32)
    q = rows(8, 2, 128, 0)
    freq = frequencies(64)
    freq[1] = 3.0 * np.pi   # more than a turn each
    freq[2] = -0.7
    p, f = torch.from_numpy(pos).cuda(), freq.cuda()
    qo, _ = tv.rotate_qk(q.cuda(), None, p, f)
    check(qo, q, pos, freq, None, 0.0, None, False, 1.0)
    back, _ = tv.rotate_qk(qo, None, p, -f)
    err = (back.double().cpu() - q.double()).abs()
    length = torch.hypot(q[..., :64].double(), q[..., 64:].double()).repeat(1, 1, 2)
    # two roundings to bf16 of values up to the pair's length, turned
    assert (err <= length * (2.0 ** -8 * 2.5 + 2.0 ** -17)).all()


def test_a_frequency_that_is_not_finite_makes_its_pair_nan():
    ensure_built()
    q = rows(4, 2, 64, 0).cuda()
    f = frequencies(32).cuda()
    f[5], f[9] = float("inf"), float("nan")
    out, _ = tv.rotate_qk(q, None, torch.arange(4, dtype=torch.int32, device="cuda"), f)
    nan = torch.isnan(out).all(0).all(0).cpu()
    assert nan.nonzero()[:, 0].tolist() == [5, 9, 37, 41] and not torch.isnan(out[..., :5]).any()


def test_values_that_are_not_finite_stay_in_their_pairs():
    ensure_built()
    q = torch.ones(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 3], q[0, 1, 100] = float("nan"), float("inf")
    p, f = torch.ones(1, dtype=torch.int32, device="cuda"), frequencies(32).cuda()  # of 64 values
    out, _ = tv.rotate_qk(q, None, p, f)
    bad = ~torch.isfinite(out[0].float())
    assert bad[0].nonzero()[:, 0].tolist() == [3, 35] and bad[1].nonzero()[:, 0].tolist() == [100]
    assert (out[0, 1, 64:100] == 1).all() and out[0, 1, 100] == float("inf")


@pytest.mark.parametrize("case", [(40, 8, 2, 128, 64, False), (40, 8, 2, 128, 61, False), (5, 3, 1, 64, 32, True)])
def test_slices_of_a_fused_projection_in_place(case):
    ensure_built()
    t, hq, hkv, d, pairs, interleaved = case
    heads = hq + 2 * hkv
    qkv = rows(t, heads, d, 3).cuda()
    before = qkv.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    p = torch.arange(100, 100 + t, dtype=torch.int32, device="cuda")
    f = frequencies(pairs).cuda()
    w = (1 + 0.1 * torch.randn(d)).cuda()
    kw = dict(q_weight=w, k_weight=w, interleaved=interleaved)
    want = tv.rotate_qk(q, k, p, f, **kw)
    assert torch.equal(qkv, before)
    # strided outputs, of which what lies between stays
    wide = torch.full((t, heads + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    tv.rotate_qk(q, k, p, f, q_out=wide[:, 1:1 + hq], k_out=wide[:, 2 + hq:2 + hq + hkv], **kw)
    assert torch.equal(wide[:, 1:1 + hq], want[0]) and torch.equal(wide[:, 2 + hq:2 + hq + hkv], want[1])
    assert (wide[:, 0] == 7).all() and (wide[:, 1 + hq] == 7).all() and (wide[:, 2 + hq + hkv:] == 7).all()
    qo, ko = tv.rotate_qk(q, k, p, f, q_out=q, k_out=k, **kw)
    assert qo is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before[:, hq + hkv:])


def test_overlapping_outputs_are_refused():
    ensure_built()
    x = torch.zeros(8, 6, 64, dtype=torch.bfloat16, device="cuda")
    p, f = torch.zeros(8, dtype=torch.int32, device="cuda"), frequencies(32).cuda()
    for q, k, qo, ko in ((x[:, :2], x[:, 2:4], x[:, 1:3], None), (x[:, :2], x[:, 2:4], x[:, 2:4], None),
                         (x[:, :2], x[:, 2:4], x[:, 4:6], x[:, 3:5]), (x[:, :2], x[:, 2:4], None, x[:, :2]),
                         (x[:, :2], x[:, 2:4], x.view(-1)[:8 * 128].view(8, 2, 64), None)):
        with pytest.raises(tv.TVError):
            tv.rotate_qk(q, k, p, f, q_out=qo, k_out=ko)


def test_no_tokens_and_streams_and_graphs():
    ensure_built()
    f = frequencies(64).cuda()
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    q, k = tv.rotate_qk(e, e[:, :2], torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)
    x = rows(65, 4, 128, 1).cuda()
    p = torch.arange(65, dtype=torch.int32, device="cuda")
    want, _ = tv.rotate_qk(x, None, p, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = tv.rotate_qk(x, None, p, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.rotate_qk(x, None, p, f, q_out=out)
    x2 = rows(65, 4, 128, 2).cuda()
    want2, _ = tv.rotate_qk(x2, None, p, f)
    x.copy_(x2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


MANY = [  # as CASES, of so many rows that warps take stretches of them
    (3500, 28, 4, 128, 64, 3, False, True, torch.float32),
    (15001, 4, 3, 128, 61, 2, False, True, torch.bfloat16),
    (9001, 9, 2, 64, 32, 1, True, False, None),
    (31000, 1, 0, 128, 16, 1, False, True, torch.bfloat16),
    (60001, 5, 1, 128, 64, 1, False, True, torch.bfloat16),    # more rows than L2 holds
    (3601, 100, 3, 128, 64, 1, False, True, torch.bfloat16),
    (2, 59000, 1, 64, 32, 1, False, True, torch.bfloat16),
    (1, 400001, 3, 128, 64, 1, True, True, torch.bfloat16),
]


@pytest.mark.parametrize("case", MANY)
def test_many_rows(case):
    """Some tokens' heads against fp64; all of them, strided and in place, against calls
    of few rows each, which another kernel takes: each within a rounding to bf16 and the
    arithmetic of the same value, of a row of at most `most`."""
    ensure_built()
    t, hq, hkv, d, pairs, n_axes, interleaved, norms, wt = case
    torch.manual_seed(t)
    wide = torch.randn(t, hq + hkv + 1, d, device="cuda").to(torch.bfloat16)
    before = wide.clone()
    q, k = wide[:, :hq], wide[:, hq:hq + hkv] if hkv else None
    g = np.random.default_rng(t)
    pos = g.integers(-40000, 40000, (n_axes, t)).astype(np.int32)
    axes = tuple(int(x) for x in g.integers(0, n_axes, pairs)) if n_axes > 1 else None
    w = (1 + 0.3 * torch.randn(d)).to(wt) if norms else None
    freq = frequencies(pairs)
    p, f, dw = torch.from_numpy(pos).cuda(), freq.cuda(), None if w is None else w.cuda()
    kw = dict(eps=1e-5, axes=axes, interleaved=interleaved, scale=1.25)
    assert tv.rotate_qk(q, k, p, f, q_weight=dw, k_weight=dw if hkv else None, q_out=q, k_out=k, **kw)[0] is q
    assert torch.equal(wide[:, hq + hkv:], before[:, hq + hkv:])
    some = sorted({0, t - 1, *g.integers(0, t, 40).tolist()})
    heads = sorted({0, hq - 1, *g.integers(0, hq, 40).tolist()})
    pick = lambda x, h: x[some][:, h].cpu()  # noqa: E731
    check(pick(q, heads).cuda(), pick(before, heads), pos[:, some], freq, w, 1e-5, axes, interleaved, 1.25)
    if hkv:
        last = list(range(hq, hq + hkv))
        check(pick(wide, last).cuda(), pick(before, last), pos[:, some], freq, w, 1e-5, axes, interleaved, 1.25)
    # few tokens at a time, and of one token's many heads few at a time
    step, part = max(1, 10000 // (hq + hkv)), 10000
    for t0 in range(0, t, step):
        for h0 in range(0, hq + hkv, part):
            x = before[t0:t0 + step, h0:min(h0 + part, hq + hkv)].contiguous()
            want, _ = tv.rotate_qk(x, None, p[:, t0:t0 + step].clone(), f, q_weight=dw, **kw)
            got = wide[t0:t0 + step, h0:h0 + part][:, :x.shape[1]]
            most = want.float().abs().amax(-1, keepdim=True)
            assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -17 * most).all(), (t0, h0)
