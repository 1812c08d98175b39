"""The recurrent form of linear attention, chosen for prompts of any length.

Tolerance of the recurrence.  Relative to the same sums of magnitudes: a state element carries at most 3
roundings a token still remembered, the readout's sum 19 (four terms a lane and pair of accumulators, the
lane's own four sums, 8 lanes), scale and decay 5: (24 + 3 * min(T, 1 / (1 - e^g))) * 2^-24 for each head."""

import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

D = 128


def _inputs(rows, H, Hk, Dv, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, w, generator=gen).to(dtype) for w in (Hk * D, Hk * D, H * Dv)]


def _prefill(q, k, v, g, H, Hk, Dv, S, lengths, algo):
    from gated_delta_rule_scan_gb300 import mixer
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    return mixer.kda_linattn_prefill(q=q.cuda(), k=k.cuda(), v=v.cuda(), log_decay=g.cuda(), H=H, Hk=Hk, Dv=Dv,
                                     state_in=S.cuda(), cu_seqlens=cu.cuda(), cu_seqlens_host=cu, algo=algo), cu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths,H,Hk,Dv,decays", [
    ([1, 31, 32, 0, 100], 3, 1, 128, [-0.4, -0.01, 0.0]), ([700], 2, 2, 256, [-0.05, -2.0]),
    ([33, 257], 4, 2, 128, [-1.0, -60.0, -0.2, -0.003])])
def test_recurrence_at_any_length(lengths, H, Hk, Dv, decays, dtype):
    from gated_delta_rule_scan_gb300 import kda
    rows, N, g = sum(lengths), len(lengths), torch.tensor(decays)
    q, k, v = _inputs(rows, H, Hk, Dv, dtype, rows)
    S = torch.randn(N, H, Dv, D, generator=torch.Generator().manual_seed(rows))
    assert kda.linattn_workspace(N, rows, H, "cuda", Hk=Hk, Dv=Dv, dtype=dtype, algo=kda.ALGO_SEQ) is None
    out, cu = _prefill(q, k, v, g, H, Hk, Dv, S, lengths, kda.ALGO_SEQ)
    for n, L in enumerate(lengths):
        at = slice(int(cu[n]), int(cu[n + 1]))
        (o, last), (om, lm) = ref.both(q[at], k[at], v[at], g, S[n], H, Hk, Dv, D ** -0.5)
        horizon = torch.minimum(torch.tensor(float(max(L, 1)), dtype=torch.float64),
                                1 / (1 - torch.exp(g.double())).clamp(min=1e-9))
        tol = (24 + 3 * horizon) * 2.0 ** -24
        err = (out["o"][at].double().cpu() - o).abs().view(L, H, Dv)
        assert bool((err <= tol[:, None] * om.view(L, H, Dv) + 1e-37).all())
        err = (out["state_out"][n].double().cpu() - last).abs()
        assert bool((err <= tol[:, None, None] * lm + 1e-37).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bits_do_not_depend_on_the_batch(dtype):
    """By the recurrence a sequence has the same bits alone, packed with long ones and in another place."""
    from gated_delta_rule_scan_gb300 import kda
    H, g, lengths = 2, torch.tensor([-0.2, -0.01]), [10, 700, 45, 1]
    q, k, v = _inputs(sum(lengths), H, H, D, dtype, 3)
    S = torch.randn(len(lengths), H, D, D, generator=torch.Generator().manual_seed(4))
    out, cu = _prefill(q, k, v, g, H, H, D, S, lengths, kda.ALGO_SEQ)
    for n, L in enumerate(lengths):
        at = slice(int(cu[n]), int(cu[n + 1]))
        alone, _ = _prefill(q[at], k[at], v[at], g, H, H, D, S[n:n + 1], [L], kda.ALGO_SEQ)
        assert torch.equal(alone["o"], out["o"][at]) and torch.equal(alone["state_out"][0], out["state_out"][n])


def test_unknown_forms_are_refused():
    from gated_delta_rule_scan_gb300 import kda, mixer
    x, g = torch.zeros(4, D, device="cuda"), torch.zeros(1, device="cuda")
    for algo in (kda.ALGO_CHUNK, 3, -1):
        with pytest.raises(kda.KdaError) as e:
            mixer.kda_linattn_prefill(q=x, k=x, v=x, log_decay=g, H=1, N=1, T=4, algo=algo)
        assert e.value.status == 40007
