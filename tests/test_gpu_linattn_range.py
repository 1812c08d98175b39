"""Offsets past 32 bits: each call's last rows, beyond 2^31 elements, against the same rows in a small call or in
64 bits."""

import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt(dtype):
    """After 200 tokens of e^-0.5 each nothing of 1e-40 is left of what came before."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    H, T, tail = 64, 2 ** 31 // (64 * D) + 333, 200
    g = torch.full((H,), -0.5)
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.empty(T, H * D, dtype=dtype, device="cuda").normal_(generator=gen) for _ in range(3))
    assert q.numel() > 2 ** 31
    out = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g.cuda(), H=H, N=1, T=T)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    pick = lambda x: x[-tail:].reshape(tail, H, D)[:, [0, H - 1]].reshape(tail, -1).cpu()
    (o, last), (om, lm) = ref.both(pick(q), pick(k), pick(v), g[:2], torch.zeros(2, D, D), 2, 2, D, D ** -0.5)
    # 64 truncated sums of 2^-23, for f32 three operands and two products of 17 bits (9 * 2^-17); the first of the
    # tail's tokens still see what was before it: half of them are looked at
    tol = 64 * 2.0 ** -23 + (9 * 2.0 ** -17 if dtype == torch.float32 else 0)
    half = tail // 2
    assert bool(((pick(out["o"]).double() - o).abs()[half:] <= tol * om[half:] + 1e-20).all())
    assert bool(((out["state_out"][0, [0, H - 1]].double().cpu() - last).abs() <= tol * lm + 1e-20).all())


def test_pool():
    from gated_delta_rule_scan_gb300 import kda, mixer
    H, P = 2, 2 ** 31 // (2 * D * D) + 3
    pool = torch.zeros(P, H, D, D, device="cuda")
    assert pool.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool[P - 1].normal_(generator=gen)
    small = pool[P - 1:].clone()
    q, k, v = (torch.randn(2, H * D, generator=gen, device="cuda") for _ in range(3))
    g = torch.tensor([-0.1, -0.01], device="cuda")
    i = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    o = mixer.kda_linattn_decode(q=q, k=k, v=v, log_decay=g, pool=pool, N=1, T=2, H=H, slots=i(P - 1),
                                 slots_out=i(P - 2))
    want = mixer.kda_linattn_decode(q=q, k=k, v=v, log_decay=g, pool=small, N=1, T=2, H=H)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    assert torch.equal(o, want) and torch.equal(pool[P - 2], small[0])


def test_probabilities():
    from gated_delta_rule_scan_gb300 import mixer
    N, T, V = 1040, 16, 131072
    target = torch.empty(N, T, V, dtype=torch.bfloat16, device="cuda").uniform_()
    assert target.numel() > 2 ** 31
    tokens = torch.randint(0, V, (N, T - 1), dtype=torch.int32, device="cuda")
    u, r = torch.rand(N, T - 1, device="cuda"), torch.rand(N, device="cuda")
    keep, out = mixer.kda_draft_accept(target=target, tokens=tokens, u=u, r=r)
    want = mixer.kda_draft_accept(target=target[-5:].clone(), tokens=tokens[-5:].clone(), u=u[-5:].clone(),
                                  r=r[-5:].clone())
    assert torch.equal(keep[-5:], want[0]) and torch.equal(out[-5:], want[1])


def test_norms():
    from gated_delta_rule_scan_gb300 import mixer
    F = 16384
    rows = 2 ** 31 // F + 5
    x = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda").normal_()
    y, w = torch.empty_like(x).normal_(), torch.rand(F, device="cuda")
    h, z = mixer.kda_residual_rmsnorm(residual=x, block=y, block_w=w, norm_w=w)
    want = mixer.kda_residual_rmsnorm(residual=x[-7:].clone(), block=y[-7:].clone(), block_w=w, norm_w=w)
    assert torch.equal(h[-7:], want[0]) and torch.equal(z[-7:], want[1])
