"""The operators of a speculative round together, as a serving loop calls them: prompts into a pool of
linear attention states, then rounds of norm, projections, verify beside the states of before, logits,
draft verification and rollback by its keep; and the same calls on other streams and in CUDA graphs."""

import pytest
import torch

from tests.test_gpu_accept import plain

pytestmark = pytest.mark.gpu

D, H, F, V, T = 128, 2, 256, 512, 4
BUSY = 200_000_000            # clock cycles: about a tenth of a second


class Layer:
    """One linear attention layer over random embeddings, and a readout of V tokens."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.gen, self.embed = g, r(V, F)
        self.w_in, self.w_out = r(3 * H * D, F) / F ** 0.5, r(F, H * D) / (H * D) ** 0.5
        self.readout = r(V, F) * 2.0 / F ** 0.5
        self.norms = [1 + 0.1 * r(F) for _ in range(3)]
        self.log_decay = torch.tensor([-0.5, -0.02], device="cuda")

    def qkv(self, tokens):
        from gated_delta_rule_scan_gb300 import mixer
        x = self.embed[tokens.long().reshape(-1)]
        _, z = mixer.kda_residual_rmsnorm(residual=x, norm_w=self.norms[0])
        return x, (z @ self.w_in.T).split(H * D, 1)

    def probs(self, x, o):
        from gated_delta_rule_scan_gb300 import mixer
        _, z = mixer.kda_residual_rmsnorm(residual=x, block=o @ self.w_out.T, block_w=self.norms[1],
                                          norm_w=self.norms[2], block_scale=0.7)
        return torch.softmax(z @ self.readout.T, -1)

    def step(self, tokens, pool, slots, slots_out=None, keep=None):
        from gated_delta_rule_scan_gb300 import mixer
        N, t = tokens.shape
        x, (q, k, v) = self.qkv(tokens)
        o = mixer.kda_linattn_decode(q=q, k=k, v=v, log_decay=self.log_decay, pool=pool, N=N, T=t, H=H,
                                     slots=slots, slots_out=slots_out, keep=keep)
        return self.probs(x, o).reshape(N, t, V)


def _prompts(layer, lengths, pool, slots):
    from gated_delta_rule_scan_gb300 import mixer
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    tokens = torch.randint(0, V, (sum(lengths),), generator=layer.gen, device="cuda")
    _, (q, k, v) = layer.qkv(tokens)
    out = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=layer.log_decay, H=H, cu_seqlens=cu.cuda(),
                                    cu_seqlens_host=cu)
    pool[slots.long()] = out["state_out"]
    return tokens[cu[1:].long() - 1].to(torch.int32), tokens, cu


def test_rounds():
    """Rounds of one to four tokens a sequence: what stands after each is what one-token steps over the
    accepted tokens leave, bit for bit, and the tokens follow from the probabilities as defined."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    layer, N = Layer(1), 5
    pool = torch.zeros(2 * N + 1, H, D, D, device="cuda")
    slots = torch.tensor([7, 0, 3, 9, 10], dtype=torch.int32, device="cuda")
    spare = torch.tensor([1, 2, 4, 5, 6], dtype=torch.int32, device="cuda")
    last, _, _ = _prompts(layer, [40, 3, 150, 1, 64], pool, slots)
    single = pool[slots.long()].clone()
    g = torch.Generator(device="cuda").manual_seed(2)
    for i in range(4):
        drafts = torch.randint(0, V, (N, T - 1), generator=g, device="cuda", dtype=torch.int32)
        guess = torch.softmax(torch.randn(N, T - 1, V, generator=g, device="cuda"), -1)
        if i % 2:                                # a drafter that knows the target's favourite
            tokens = torch.cat([last[:, None], drafts], 1)
            for t in range(T - 1):
                p = layer.step(tokens[:, :t + 1].contiguous(), pool, slots, spare)
                tokens[:, t + 1] = p[:, t].argmax(-1)
            drafts = tokens[:, 1:].contiguous()
            guess = None
        batch = torch.cat([last[:, None], drafts], 1)
        before = pool.clone()
        target = layer.step(batch, pool, slots, spare)
        u, r = torch.rand(N, T - 1, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        keep, out = mixer.kda_draft_accept(target=target, tokens=drafts, u=u, r=r, draft=guess)
        want = plain(target.cpu(), drafts.cpu(), u.cpu(), r.cpu(), None if guess is None else guess.cpu(), None)
        assert torch.equal(keep.cpu(), want[0]) and torch.equal(out.cpu(), want[1])
        layer.step(batch, pool, slots, spare, keep=keep)
        for n in range(N):
            k = int(keep[n])
            own = single[n:n + 1].clone()
            for t in range(k):
                layer.step(batch[n:n + 1, t:t + 1].contiguous(), own, None)
            assert torch.allclose(pool[int(spare[n])], own[0], rtol=0, atol=1e-3)
            single[n] = own[0]
            # (the projections are torch's, whose rounding hangs on the batch: the recurrence alone is exact)
            assert torch.equal(pool[int(slots[n])], before[int(slots[n])])
        last = out.gather(1, (keep - 1).long()[:, None])[:, 0].contiguous()
        single = pool[spare.long()].clone()
        slots, spare = spare, slots
    assert kda.kda_device_status() == 0


def test_a_captured_round_replays():
    """Verify, draft verification, rollback and norms captured once: a replay on new inputs equals the calls
    made one by one.  Prompts too, with a workspace of their own each."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    N = 3
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    decay = torch.tensor([-0.1, -0.01], device="cuda")
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    static = dict(q=r(N * T, H * D), k=r(N * T, H * D), v=r(N * T, H * D), target=torch.softmax(r(N, T, V), -1),
                  draft=torch.softmax(r(N, T - 1, V), -1), u=torch.rand(N, T - 1, device="cuda"),
                  r=torch.rand(N, device="cuda"), x=r(N, F), y=r(N, F), w=r(F), pool=r(2 * N, H, D, D),
                  long_q=r(2000, H * D), long_k=r(2000, H * D), long_v=r(2000, H * D))
    tokens = torch.randint(0, V, (N, T - 1), device="cuda", dtype=torch.int32)
    ws = [kda.linattn_workspace(1, 2000, H, "cuda", dtype=t) for t in (torch.float32, torch.bfloat16)]

    def call(s):
        o = torch.zeros(N * T, H * D, device="cuda")
        kw = dict(N=N, T=T, H=H, slots=slots, slots_out=slots + N)
        kda.kda_linattn_decode(s["q"], s["k"], s["v"], decay, s["pool"], o, **kw)
        keep, out = mixer.kda_draft_accept(target=s["target"], tokens=tokens, u=s["u"], r=s["r"], draft=s["draft"])
        kda.kda_linattn_decode(s["q"], s["k"], s["v"], decay, s["pool"], o, keep=keep, **kw)
        h, z = mixer.kda_residual_rmsnorm(residual=s["x"], block=s["y"], norm_w=s["w"], block_w=s["w"])
        p32 = mixer.kda_linattn_prefill(q=s["long_q"], k=s["long_k"], v=s["long_v"], log_decay=decay, H=H, N=1, T=2000,
                                        workspace=ws[0])
        b = [s[k].bfloat16() for k in ("long_q", "long_k", "long_v")]
        p16 = mixer.kda_linattn_prefill(q=b[0], k=b[1], v=b[2], log_decay=decay, H=H, N=1, T=2000, workspace=ws[1])
        return [o, keep, out, h, z, p32["o"], p32["state_out"], p16["o"], p16["state_out"]]
    call({k: v.clone() for k, v in static.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(static)
    for i in range(3):
        fresh = {k: torch.softmax(r(*v.shape), -1) if k in ("target", "draft") else torch.rand_like(v)
                 if k in ("u", "r") else r(*v.shape) for k, v in static.items()}
        for k, v in fresh.items():
            static[k].copy_(v)
        graph.replay()
        want = call(fresh)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(static["pool"], fresh["pool"])
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("as_int", [False, True])
def test_calls_beside_a_busy_stream(as_int):
    """Calls on a side stream, with buffers and workspaces of their own, while the current one is busy."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    decay = torch.tensor([-0.1, -0.01], device="cuda")
    q, k, v, pool = r(1500, H * D), r(1500, H * D), r(1500, H * D), r(4, H, D, D)
    target, u, rr = torch.softmax(r(4, 1, V), -1), torch.zeros(4, 0, device="cuda"), torch.rand(4, device="cuda")
    none = torch.zeros(4, 0, dtype=torch.int32, device="cuda")
    x, w = r(40, F), r(F)
    calls = [lambda st: list(mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=decay, H=H, N=1, T=1500,
                                                       stream=st).values()),
             lambda st: [mixer.kda_linattn_decode(q=q[:4], k=k[:4], v=v[:4], log_decay=decay, pool=pool.clone(), N=4,
                                                  T=1, H=H, stream=st)],
             lambda st: list(mixer.kda_draft_accept(target=target, tokens=none, u=u, r=rr, stream=st)),
             lambda st: list(mixer.kda_residual_rmsnorm(residual=x, block=x, norm_w=w, stream=st))]
    side = torch.cuda.Stream()
    for n, call in enumerate(calls):
        want = call(None)
        torch.cuda.synchronize()
        if n == 1:
            continue                             # (its pool's copy is made on the current stream: below)
        torch.cuda._sleep(BUSY)
        got = [call(side.cuda_stream if as_int else side) for _ in range(4)]
        torch.cuda.synchronize()
        for out in got:
            for a, b in zip(out, want):
                assert torch.equal(a, b)
    want_pool = pool.clone()
    want = mixer.kda_linattn_decode(q=q[:4], k=k[:4], v=v[:4], log_decay=decay, pool=want_pool, N=4, T=1, H=H)
    mine = pool.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = mixer.kda_linattn_decode(q=q[:4], k=k[:4], v=v[:4], log_decay=decay, pool=mine, N=4, T=1, H=H,
                                   stream=side.cuda_stream if as_int else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(mine, want_pool)
    assert kda.kda_device_status() == 0


def test_two_prompts_at_once():
    """Two streams, two workspaces: neither call disturbs the other, and a second run of either gives the
    same bits."""
    from gated_delta_rule_scan_gb300 import mixer
    g = torch.Generator(device="cuda").manual_seed(8)
    decay = torch.tensor([-0.1, -0.01], device="cuda")
    jobs = []
    for dtype, n in ((torch.bfloat16, 3000), (torch.float32, 1111)):
        q, k, v = (torch.randn(n, H * D, generator=g, device="cuda").to(dtype) for _ in range(3))
        jobs.append(dict(q=q, k=k, v=v, log_decay=decay, H=H, N=1, T=n))
    want = [mixer.kda_linattn_prefill(**j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [mixer.kda_linattn_prefill(stream=streams[i % 2], **jobs[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for key in ("o", "state_out"):
            assert torch.equal(out[key], want[i % 2][key])
