"""Verification of drafted tokens at the ends of its range: totals past f32, and random numbers next to the
borders between tokens."""

from fractions import Fraction

import pytest
import torch

from tests.test_gpu_accept import plain

pytestmark = pytest.mark.gpu


def _into_sentinels(target, tokens, u, r, draft):
    """keep and tokens of a call whose output buffers held -7 throughout."""
    from gated_delta_rule_scan_gb300 import mixer
    N, T = target.shape[:2]
    keep = torch.full((N,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((N, T), -7, dtype=torch.int32, device="cuda")
    mixer.kda_draft_accept(target=target.cuda(), tokens=tokens.cuda(), u=u.cuda(), r=r.cuda(),
                           draft=None if draft is None else draft.cuda(), keep=keep, out_tokens=out)
    return keep.cpu(), out.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 50, 5000, 70001])
@pytest.mark.parametrize("kind", ["sample", "rest", "lookup", "nothing left"])
def test_totals_past_f32(dtype, V, kind):
    """Finite weights whose sum is not: each draws what 64 bits draw."""
    N, T = 6, 1 if kind == "sample" else 2
    g = torch.Generator().manual_seed(V)
    target = (1e38 + 2e38 * torch.rand(N, T, V, generator=g)).to(dtype)
    target[:, :, V // 3] = 3e38
    target[1] *= 1e-30                             # one sequence of ordinary size, one with few large weights
    target[2, :, 2:] = 1e-3
    assert torch.isfinite(target).all()
    r = torch.rand(N, generator=g)
    r[3], r[4] = 0.0, 1 - 2.0 ** -24
    u = torch.full((N, T - 1), 1 - 2.0 ** -24)
    # (an id outside the vocabulary is refused, whatever its probabilities)
    tokens = torch.full((N, T - 1), V if kind == "nothing left" else V // 2, dtype=torch.int32)
    draft = None
    if kind == "rest":
        draft = (target[:, :1].float() * 0.25).to(dtype)
        draft[:, 0, V // 2] = 3.2e38               # refused there
    elif kind == "lookup":
        u[:] = 1.0
        target[:, 0, V // 2] = 0.5
    elif kind == "nothing left":
        draft = target[:, :1].clone()
    want = plain(target, tokens, u, r, draft, None)
    got = _into_sentinels(target, tokens, u, r, draft)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("V", [40001, 99991, 131072])
def test_random_numbers_at_the_borders(V):
    """Rows of equal weights and, for 256 tokens j, the two f32 numbers around j / V: the token is floor(r V) in
    exact arithmetic.  r V is a multiple of 2^-27 for r above an eighth, so that a sum off by 2^-45 of the total
    (4e-9 weights) names every token, and one off by 2^-27 of it (f32 sums) does not."""
    rows = []
    for j in range(V // 8 + 1, V, V // 292)[:256]:
        r = torch.tensor(j / V, dtype=torch.float32)           # within half a step of j / V
        if Fraction(float(r)) > Fraction(j, V):
            rows += [torch.nextafter(r, torch.tensor(0.0)), r]
        else:
            rows += [r, torch.nextafter(r, torch.tensor(1.0))]
    r = torch.stack(rows)
    want = torch.tensor([int(Fraction(float(x)) * V) for x in r], dtype=torch.int32)
    N = len(r)
    target = torch.full((1, 1, V), 1.0 / V).expand(N, 1, V).contiguous()
    empty = torch.zeros(N, 0)
    keep, out = _into_sentinels(target, empty.int(), empty, r, None)
    assert bool((keep == 1).all()) and torch.equal(out[:, 0], want)
