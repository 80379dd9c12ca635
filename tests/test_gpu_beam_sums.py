"""LSE in tv_beam_select on rows that are hard for sums in fp32: against fp64, within the
bound that include/tv.h states.

The bound, in u = 2^-24 of the sum (whose logarithm is off by as much): a power 4 (2^-22,
ex2.approx), the rounding of its argument 11 (half a step of [16, 32) times ln 2; of smaller
ones nothing is left), the constant for log2 e 3; 15 sums of a turn and 64 of turns (fp32:
7 and 64, bf16: 15 and 32, so 71); where the maximum rises, the factor by a power, its
argument and a product, 5 for each of 64 turns; the lane's last factor 2; lanes 6 and a power
with its factors 8; parts 5 and expf with its factors 4; logf 1; of rows that are passed over twice the
difference from the maximum 8.  Together 443 u, below 2^-15 = 512 u; without rises 123 u,
below 2^-17 = 128 u.  The score is that of the best token, near 0 (so
that its own rounding is far below), from a score that is rounded to fp32 before."""
import pytest
import torch

import speculative_decoding_tree_attention_gb300 as tv
from tv_testlib import ensure_built

pytestmark = pytest.mark.gpu
ROWS = 320  # (a row is then a CTA's: eight parts of most entries)


def rows_of(kind, vocab, dtype):
    entry = torch.arange(vocab)
    chunk = ((vocab + 7) // 8 + 511) // 512 * 512
    turn = 32 * 4 * (4 if dtype is torch.float32 else 8)  # entries that a warp takes at a time
    depth = torch.linspace(0.1, 14, ROWS)[:, None]
    step = 2.0 ** torch.linspace(-14, 1, ROWS)[:, None]
    if kind == "a peak of every lane, then equal ones":
        peak = (entry % chunk < turn) & (entry % (turn // 32) == 0)
        return torch.where(peak, 0.0, -depth)
    if kind == "one peak":
        return torch.where(entry == 0, 0.0, -depth)
    if kind == "equal":
        return depth.expand(ROWS, vocab)
    if kind == "parts that rise":
        return (entry % chunk // turn) * step
    if kind == "a row that rises":
        return (entry // turn) * step
    g = torch.Generator().manual_seed(5)
    return (entry % chunk // turn) * step + torch.rand(ROWS, vocab, generator=g) * 0.01


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [262143, 32000, 517])
@pytest.mark.parametrize("kind", ["a peak of every lane, then equal ones", "one peak", "equal", "parts that rise",
                                  "a row that rises", "rough parts that rise"])
def test_log_sums(kind, vocab, dtype):
    ensure_built()
    logits = rows_of(kind, vocab, dtype).to(dtype).cuda().contiguous()
    best = logits.amax(1).double()
    lse = torch.cat([torch.logsumexp(x.double(), 1) for x in logits.split(32)])
    scores = (lse - best).float()
    got = tv.beam_select(logits, scores, beams=1, select=1)
    assert (got["status"] == 0).all()
    off = (got["scores"][:, 0].double() - (scores.double() + (best - lse))).abs()
    assert off.max() <= (2.0 ** -15 if "rise" in kind else 2.0 ** -17), float(off.max())
