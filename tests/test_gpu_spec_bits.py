"""Rounds of a verify on a pool of linear attention states, the verification of its drafts and the rollback by its
keep: after each, the states are those of one-token calls over the rows that stand, bit for bit, at every size."""

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-15, 1.0])
@pytest.mark.parametrize("T", [2, 4, 16])
def test_rounds(T, size, dtype):
    from gated_delta_rule_scan_gb300 import kda, mixer
    N, H, Hk, V = 5, 3, 1, 40
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")
    g = torch.tensor([-0.7, -0.01, -3.0], device="cuda")
    kw = dict(log_decay=g, H=H, Hk=Hk, Dv=256)
    pool = r(2 * N + 1, H, 256, D) * size
    slots = torch.tensor([7, 0, 3, 9, 10], dtype=torch.int32, device="cuda")
    spare = torch.tensor([1, 2, 4, 5, 6], dtype=torch.int32, device="cuda")
    single, kept = pool[slots.long()].clone(), []
    for _ in range(4):
        q, k, v = (r(N * T, w).to(dtype) for w in (Hk * D, Hk * D, H * 256))
        v = (v.float() * size).to(dtype)
        step = dict(q=q, k=k, v=v, pool=pool, N=N, T=T, slots=slots, slots_out=spare, **kw)
        before = pool.clone()
        o = mixer.kda_linattn_decode(**step)
        draft = torch.softmax(r(N, T - 1, V), -1)
        target = torch.softmax(torch.cat([draft.log(), r(N, 1, V)], 1) + 0.2 * r(N, T, V), -1)
        tokens = torch.multinomial(draft.reshape(-1, V), 1, generator=gen).reshape(N, T - 1).int()
        keep, _ = mixer.kda_draft_accept(target=target, draft=draft, tokens=tokens, u=rand(N, T - 1), r=rand(N))
        assert torch.equal(mixer.kda_linattn_decode(keep=keep, **step).reshape(N, T, -1)[:, 0],
                           o.reshape(N, T, -1)[:, 0])
        for n in range(N):
            own = single[n:n + 1].clone()
            for t in range(int(keep[n])):
                row = n * T + t
                ot = mixer.kda_linattn_decode(q=q[row:row + 1], k=k[row:row + 1], v=v[row:row + 1], pool=own, N=1, T=1,
                                              **kw)
                assert torch.equal(ot[0], o[row])
            assert torch.equal(pool[int(spare[n])], own[0])
            single[n] = own[0]
        untouched = torch.ones(2 * N + 1, dtype=torch.bool, device="cuda")
        untouched[spare.long()] = False
        assert torch.equal(pool[untouched], before[untouched])
        kept += keep.tolist()
        slots, spare = spare, slots
    assert len(set(kept)) > 1 and kda.kda_device_status() == 0
