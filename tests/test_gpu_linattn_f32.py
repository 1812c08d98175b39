"""f32 prompts in chunks carry all of f32: errors relative to a head's norm, and elements of any size beside each other.

Tolerances, in steps of 2^-23.  The tensor cores truncate their sums, by half a step on average: o 12 of its largest
term and 8 of the scores' (10 steps), the state 4 (2).  The factors e^(g n) come from g n rounded, n up to 33 away from
0, and tokens at least one apart see it: 33 |g| e^-|g| 2^-24 / sqrt(3), 3.5 steps at most; expf, v' and the state's own
roundings and factors 2.5 (3 for the state).  Three parts of everything leave 2^-24 a product: below that.  16 for o,
8.5 for the state; the recurrence's sums are smaller than either.  (Two parts of everything: 55 and 40.)
Each element: 64 truncated sums of 2^-23 of the sums of magnitudes."""

import math

import pytest
import torch

from tests.test_gpu_linattn_decays import _check, _closed

pytestmark = pytest.mark.gpu

D = 128
STEP = 2.0 ** -23


def _run(q, k, v, g, S, lengths, Hk):
    from gated_delta_rule_scan_gb300 import kda, mixer
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    H = len(g)
    out = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g.cuda(), H=H, Hk=Hk, state_in=S, cu_seqlens=cu.cuda(),
                                    cu_seqlens_host=cu)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    for n in range(len(lengths)):
        at = slice(int(cu[n]), int(cu[n + 1]))
        for h in range(H):
            head = lambda x, i: x[at, i * D:(i + 1) * D].double()
            a = (head(q, h % Hk), head(k, h % Hk), head(v, h))
            S0, gh = S[n, h].double(), float(g[h])
            yield (n, h, (head(out["o"], h), out["state_out"][n, h]), _closed(*a, gh, S0, D ** -0.5),
                   _closed(*(x.abs() for x in a), gh, S0.abs(), D ** -0.5))


@pytest.mark.parametrize("lengths", [[32], [64], [65, 31, 200], [129, 0, 63, 333], [1500], [700, 1333]])
@pytest.mark.parametrize("Hk,fused", [(5, False), (2, True)])
def test_norms(lengths, Hk, fused):
    g = torch.tensor([-0.002, -0.05, -0.4, -0.93, -1.2])
    gen = torch.Generator(device="cuda").manual_seed(sum(lengths))
    widths = (Hk * D, Hk * D, len(g) * D)
    x = torch.randn(sum(lengths), sum(widths), generator=gen, device="cuda")
    q, k, v = x.split(widths, 1) if fused else (t.contiguous() for t in x.split(widths, 1))
    S = torch.randn(len(lengths), len(g), D, D, generator=gen, device="cuda")
    for n, h, got, want, mag in _run(q, k, v, g, S, lengths, Hk):
        _check(got[0].float(), want[0], mag[0], 16 * STEP, 64 * STEP, ("o", n, h))
        _check(got[1], want[1], mag[1], 8.5 * STEP, 64 * STEP, ("state", n, h))


@pytest.mark.parametrize("lengths", [[200], [1400]])
def test_sizes_side_by_side(lengths):
    """Tokens from 1e-6 to 1e6 in k and in v, keys and values from 1e-3 to 1e3, states too: each element is as good as
    its own sums, whatever lies beside it."""
    g = torch.tensor([-0.01, -0.3, -0.99, -2.0])
    T, H = sum(lengths), len(g)
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    power = lambda e, *s: 10.0 ** (e * (2 * torch.rand(*s, generator=gen, device="cuda") - 1))
    q, k, v = (r(T, H * D) * power(3, 1, H * D) for _ in range(3))
    k, v = k * power(6, T, 1), v * power(6, T, 1)
    S = r(1, H, D, D) * power(3, 1, H, 1, D) * power(3, 1, H, D, 1)
    for n, h, got, want, mag in _run(q, k, v, g, S, lengths, H):
        _check(got[0].float(), want[0], mag[0], math.inf, 64 * STEP, ("o", n, h))
        _check(got[1], want[1], mag[1], math.inf, 64 * STEP, ("state", n, h))
