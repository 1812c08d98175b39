"""The recurrence of linear attention over many calls: prompts against chained decode calls, bit for bit, and
decays next to 1 over 20000 tokens."""

import pytest
import torch

from tests.test_gpu_linattn_forms import D, _inputs, _prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,algo,T", [
    (torch.bfloat16, 0, 1), (torch.bfloat16, 0, 17), (torch.bfloat16, 0, 19), (torch.float32, 0, 1),
    (torch.float32, 0, 17), (torch.float32, 0, 31), (torch.bfloat16, 1, 133), (torch.float32, 1, 64)])
@pytest.mark.parametrize("step", [1, 5, 16])
def test_prompts_equal_chained_decode_calls(dtype, algo, T, step):
    """A prompt by the recurrence, short or asked for, against calls of `step` tokens, bit for bit."""
    from gated_delta_rule_scan_gb300 import mixer
    N, H, Hk, Dv, g = 3, 3, 1, 256, torch.tensor([-0.3, -0.002, -4.0])
    q, k, v = (x.cuda() for x in _inputs(N * T, H, Hk, Dv, dtype, T))
    S = torch.randn(N, H, Dv, D, generator=torch.Generator().manual_seed(T)).cuda()
    out, _ = _prefill(q, k, v, g, H, Hk, Dv, S, [T] * N, algo)
    pool = S.clone()
    for t in range(0, T, step):
        n = min(step, T - t)
        rows = (torch.arange(N, device="cuda")[:, None] * T + torch.arange(t, t + n, device="cuda")).reshape(-1)
        o = mixer.kda_linattn_decode(q=q[rows], k=k[rows], v=v[rows], log_decay=g.cuda(), pool=pool, N=N, T=n, H=H,
                                     Hk=Hk, Dv=Dv)
        assert torch.equal(o, out["o"][rows])
    assert torch.equal(pool, out["state_out"])


# e^g is farther than most from an f32 number, and so is e^(64 g): rounded to f32 they would be off, in one
# direction at each step, by 2.8e-8 (20000 tokens: 5.6e-4) and by 3.0e-8 (313 chunks: 9.3e-6).
NEXT_TO_ONE = -2.6854000680032186e-05


def _mean_error(state, before):
    want = before.double() * torch.exp(torch.tensor(NEXT_TO_ONE, dtype=torch.float64) * 20000).item()
    return float(((state.double() - want) / want).mean())


def _rounded_steps(before, tokens):
    """The state after decays of `tokens` tokens each, every step S + (e^g - 1) S with the product and the sum
    rounded to f32.  (These roundings do not average out: a step's depends on where the one before left S.)"""
    S = before.clone()
    for n in tokens:
        f = torch.expm1(torch.tensor(NEXT_TO_ONE, dtype=torch.float64) * n).float().double().item()
        S = (S.double() + (S.double() * f).float().double()).float()
    return S


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step", [1, 16])
def test_many_decode_steps_next_to_one(dtype, step):
    """20000 tokens by the decode kernel.  The mean error over the state's elements is that of the same steps
    rounded to f32 one by one, but for e^g - 1 itself, off by 2^-22 of 2.7e-5 a step (1.3e-7 in all) at most."""
    from gated_delta_rule_scan_gb300 import mixer
    H, T = 2, 20000
    g = torch.full((H,), NEXT_TO_ONE, device="cuda")
    before = 0.5 + torch.rand(1, H, D, D, generator=torch.Generator().manual_seed(1)).cuda()
    pool, x = before.clone(), torch.zeros(step, H * D, dtype=dtype, device="cuda")
    o = torch.zeros(step, H * D, device="cuda")
    for _ in range(T // step):
        mixer.kda_linattn_decode(q=x, k=x, v=x, log_decay=g, pool=pool, N=1, T=step, H=H, o=o)
    want = _mean_error(_rounded_steps(before, [1] * T), before)
    assert abs(_mean_error(pool, before) - want) < 1.3e-7


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_prompts_next_to_one(dtype):
    """313 chunks of prompts too many to be cut, likewise; e^(64 g) - 1 is off by 2^-22 of 1.7e-3 a step (1.3e-7
    in all), the state's factor on its way in and out by 4 * 2^-24 (2.4e-7)."""
    from gated_delta_rule_scan_gb300 import mixer
    N, T = 304, 20000
    g = torch.tensor([NEXT_TO_ONE], device="cuda")
    x = torch.zeros(N * T, D, dtype=dtype, device="cuda")
    before = 0.5 + torch.rand(N, 1, D, D, generator=torch.Generator().manual_seed(1)).cuda()
    out = mixer.kda_linattn_prefill(q=x, k=x, v=x, log_decay=g, H=1, N=N, T=T, state_in=before)
    want = _mean_error(_rounded_steps(before, [64] * (T // 64) + [T % 64]), before)
    assert abs(_mean_error(out["state_out"], before) - want) < 3.7e-7
