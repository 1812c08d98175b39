"""The chunked form of linear attention over the range of decays, head by head: on both sides of e^-1 a token, where
its scaled sums end and the separate ones begin, whole and cut into segments, with states from 1e-20 to 1e20.

Tolerances, relative to a head's norm, in steps of 2^-23.  The tensor cores truncate their sums, by half a step on
average: o 12 sums of its largest term (6 steps), the state 4 (2).  The factors e^(g n) come from g n rounded, n up to
33 away from 0: 33 |g| 2^-24 / sqrt(3), which tokens at least one apart see, |g| e^-|g| <= 0.37: 3.5 steps.  expf, the
state's own roundings and its factors on the way in and out: 2.5, 3 for the state.  12 and 8.5 in all (two bf16 parts
in place of three alone would cost o 17 to 20, the state 7 to 20).  f32: each of five operands is off by 2^-18 at most, two products leave out
lo * lo of 2^-18, independent of each other: sqrt(7) * 2^-18 more.
Each element: 64 truncated sums of 2^-23 of the sums of magnitudes, for f32 9 * 2^-17 more."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
DECAYS = [-0.3, -0.97, -0.9999, -1.0, -1.0001, -1.5, -3.0, -8.0]


def _closed(q, k, v, g, S, scale):
    """One head of one sequence in 64 bits: o [T, Dv] and the last state [Dv, 128]."""
    T = q.shape[0]
    t = torch.arange(T, device=q.device, dtype=torch.float64)
    gap = t[:, None] - t
    seen = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
    o = scale * (((q @ k.T) * seen) @ v + torch.exp(g * (t + 1))[:, None] * (q @ S.T))
    return o, math.exp(g * T) * S + (v * torch.exp(g * (T - 1 - t))[:, None]).T @ k


def _check(got, want, mag, norm_tol, tol, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert bool((err <= tol * mag).all()), (what, "element", float((err / mag).max()))
    if float(want.norm()) > 0:
        assert float(err.norm() / want.norm()) <= norm_tol, (what, "norm", float(err.norm() / want.norm()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,cut", [([200, 64, 65, 33, 257] * 8, False), ([1500], True), ([700, 1333], True)])
@pytest.mark.parametrize("size", [1e-10, 1.0, 1e10])
@pytest.mark.parametrize("Hk", [8, 3])
def test_decays(lengths, cut, size, Hk, dtype):
    """k and v are of `size`, states of its square."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    if cut is False and size != 1.0:
        lengths = lengths[:5]
    rows, N, H, g = sum(lengths), len(lengths), len(DECAYS), torch.tensor(DECAYS)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    q, k, v = (torch.randn(rows, h * D, generator=gen, device="cuda") for h in (Hk, Hk, H))
    q, k, v = q.to(dtype), (k * size).to(dtype), (v * size).to(dtype)
    S = torch.randn(N, H, D, D, generator=gen, device="cuda") * (4.0 * size * size)
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    if dtype == torch.bfloat16:                # (cut prompts keep their segments' states there)
        assert (kda.kda_linattn_workspace_bytes(N, rows, H, Hk) > 0) == (cut or N < 38)
    out = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g.cuda(), H=H, Hk=Hk, state_in=S, cu_seqlens=cu.cuda(),
                                    cu_seqlens_host=cu)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    f32 = dtype == torch.float32
    more, tol = math.sqrt(7) * 2.0 ** -18 if f32 else 0.0, 64 * 2.0 ** -23 + (9 * 2.0 ** -17 if f32 else 0.0)
    for n in sorted(set(list(range(min(N, 5))) + [N - 1])):
        at = slice(int(cu[n]), int(cu[n + 1]))
        for h in range(H):
            head = lambda x, i: x[at, i * D:(i + 1) * D].double()
            a = (head(q, h % Hk), head(k, h % Hk), head(v, h))
            gh = float(g[h])
            o, last = _closed(*a, gh, S[n, h].double(), D ** -0.5)
            om, lm = _closed(*(x.abs() for x in a), gh, S[n, h].double().abs(), D ** -0.5)
            _check(head(out["o"], h), o, om, 12 * 2.0 ** -23 + more, tol, ("o", n, DECAYS[h]))
            _check(out["state_out"][n, h], last, lm, 8.5 * 2.0 ** -23 + more, tol, ("state", n, DECAYS[h]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [5, 64, 100, 1500])
def test_minus_infinity_forgets_everything(T, dtype):
    """A log-decay of -infinity beside an ordinary one: each token sees itself alone, the state is the last token's."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(T, 2 * D, generator=gen, device="cuda").to(dtype) for _ in range(3))
    S = torch.randn(1, 2, D, D, generator=gen, device="cuda")
    g = torch.tensor([-float("inf"), -0.1], device="cuda")
    out = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g, H=2, N=1, T=T, state_in=S)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0 and torch.isfinite(out["o"]).all()
    a = [x[:, :D].double() for x in (q, k, v)]
    o = D ** -0.5 * (a[0] * a[1]).sum(1, keepdim=True) * a[2]
    # (q k summed over 128 keys, its 8 largest truncated sums of 2^-23, and v's product)
    mag = D ** -0.5 * (a[0] * a[1]).abs().sum(1, keepdim=True) * a[2].abs()
    assert bool(((out["o"][:, :D].double() - o).abs() <= 64 * 2.0 ** -23 * mag).all())
    last = a[2][-1][:, None] * a[1][-1][None]
    assert bool(((out["state_out"][0, 0].double() - last).abs() <= 8 * 2.0 ** -23 * last.abs()).all())
