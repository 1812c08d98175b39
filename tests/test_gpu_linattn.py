"""Linear attention with one log-decay a head: prompts (both forms) and the decode / verify step on a
pool of states, against the recurrence in 64 bits.

Tolerance.  Relative to the same sums of magnitudes, an output of the recurrent form carries at most 3
roundings a token still remembered, 16 + 8 in the readout's sum and a few for the scale; the chunked
form of bf16 60 or so accumulation steps, which the tensor cores may truncate (2^-23 each), and splits to
24 bits.  64 * 2^-23 + 3 * min(T, 1 / (1 - lambda)) * 2^-24 covers both;
log_decay enters e^(g n) with n g rounded, an error of x 2^-24 e^-x <= 2^-25 more.
The chunked form of f32 (32 tokens and more) splits q, k and v themselves: on the way through the state k,
its decayed form, v, the state and q are each off by 2^-17, and the two products leave out lo * lo, at most
2^-8 * 2^-8 = 2 * 2^-17 each: 9 * 2^-17 in all (within a chunk q, k, v, P and two products: 8)."""

import pytest
import torch

from tests import linattn_ref as ref

pytestmark = pytest.mark.gpu

D = 128


def _decays(H, kind="mixed"):
    if kind == "none":
        return torch.zeros(H)
    if kind == "strong":
        return torch.full((H,), -60.0)
    h = torch.arange(1, H + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / H)).float()


def _tol(T, g, dtype=torch.bfloat16, longest=None):
    if dtype == torch.float32 and (T if longest is None else longest) >= 32:
        return _tol(T, g) + 9 * 2.0 ** -17
    lam = torch.exp(g.double())
    horizon = torch.minimum(torch.tensor(float(max(T, 1)), dtype=torch.float64), 1 / (1 - lam).clamp(min=1e-9))
    return 64 * 2.0 ** -23 + 3 * float(horizon.max()) * 2.0 ** -24


def _close(got, want, mag, tol, what):
    err = (got.double().cpu() - want).abs()
    bound = tol * mag + 1e-37
    assert torch.isfinite(got).all(), what
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


def _inputs(rows, H, Hk, Dv, dtype, seed, fused=False):
    gen = torch.Generator().manual_seed(seed)
    w = (Hk * D, Hk * D, H * Dv)
    x = torch.randn(rows, sum(w), generator=gen).to(dtype)
    parts = x.split(w, 1)
    dev = x.cuda().split(w, 1) if fused else [p.contiguous().cuda() for p in parts]
    return parts, dev


CASES = [
    # lengths, H, Hk, Dv, decays
    ([1], 1, 1, 128, "mixed"),
    ([63], 2, 2, 128, "mixed"),
    ([64], 3, 1, 128, "none"),
    ([65], 2, 1, 256, "mixed"),
    ([128, 0, 1, 129, 64], 4, 2, 128, "mixed"),
    ([200, 77], 3, 2, 384, "strong"),
    ([0, 0], 2, 2, 128, "mixed"),
    ([333, 5, 640, 31], 5, 3, 128, "mixed"),
    ([1500], 2, 2, 128, "mixed"),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths,H,Hk,Dv,kind", CASES)
@pytest.mark.parametrize("state,fused", [(True, False), (False, True)])
def test_prefill(lengths, H, Hk, Dv, kind, dtype, state, fused):
    from gated_delta_rule_scan_gb300 import kda, mixer
    rows, N = sum(lengths), len(lengths)
    (q, k, v), (dq, dk, dv) = _inputs(rows, H, Hk, Dv, dtype, 5 + rows, fused)
    g = _decays(H, kind)
    S = (torch.randn(N, H, Dv, D, generator=torch.Generator().manual_seed(rows)) if state
         else torch.zeros(N, H, Dv, D))
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    out = mixer.kda_linattn_prefill(q=dq, k=dk, v=dv, log_decay=g.cuda(), H=H, Hk=Hk, Dv=Dv,
                                    state_in=S.cuda() if state else None, cu_seqlens=cu.cuda(),
                                    cu_seqlens_host=cu)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    for n, L in enumerate(lengths):
        b, e = int(cu[n]), int(cu[n + 1])
        (o, last), (om, lm) = ref.both(q[b:e], k[b:e], v[b:e], g, S[n], H, Hk, Dv, D ** -0.5)
        _close(out["o"][b:e], o, om, _tol(L, g, dtype, max(lengths)), ("o", n))
        _close(out["state_out"][n], last, lm, _tol(L, g, dtype, max(lengths)), ("state", n))


@pytest.mark.parametrize("N,T", [(1, 64), (2, 100), (3, 1)])
def test_prefill_uniform_equals_packed(N, T):
    """The same sequences given by (N, T) and by cu_seqlens."""
    from gated_delta_rule_scan_gb300 import mixer
    H = 3
    for dtype in (torch.float32, torch.bfloat16):
        _, (q, k, v) = _inputs(N * T, H, H, D, dtype, 3)
        g = _decays(H).cuda()
        cu = torch.arange(0, N * T + 1, T, dtype=torch.int32)
        a = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g, H=H, N=N, T=T)
        b = mixer.kda_linattn_prefill(q=q, k=k, v=v, log_decay=g, H=H, cu_seqlens=cu.cuda(),
                                      cu_seqlens_host=cu)
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["state_out"], b["state_out"])


def _decode_inputs(N, T, H, Hk, Dv, dtype, P, seed=1):
    gen = torch.Generator().manual_seed(seed)
    (q, k, v), dev = _inputs(N * T, H, Hk, Dv, dtype, seed, True)
    pool = torch.randn(P, H, Dv, D, generator=gen)
    perm = torch.randperm(P, generator=gen).to(torch.int32)
    return (q, k, v), dev, pool, perm[:N].contiguous(), perm[N:2 * N].contiguous()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,T,H,Hk,Dv,kind", [(1, 1, 1, 1, 128, "mixed"), (5, 3, 4, 2, 256, "mixed"),
                                              (3, 16, 3, 3, 128, "mixed"), (2, 4, 2, 1, 128, "strong"),
                                              (40, 2, 2, 2, 128, "none")])
@pytest.mark.parametrize("keep", [False, True])
def test_decode(N, T, H, Hk, Dv, kind, dtype, keep):
    from gated_delta_rule_scan_gb300 import kda, mixer
    P = 2 * N + 2
    (q, k, v), (dq, dk, dv), pool, slots, outs = _decode_inputs(N, T, H, Hk, Dv, dtype, P)
    g = _decays(H, kind)
    if N > 2:
        slots[N - 1] = -1
    kept = torch.randint(-1, T + 2, (N,), generator=torch.Generator().manual_seed(9),
                         dtype=torch.int32) if keep else None
    dpool = pool.cuda()
    o0 = torch.full((N * T, H * Dv), 7.0, device="cuda")
    o = mixer.kda_linattn_decode(q=dq, k=dk, v=dv, log_decay=g.cuda(), pool=dpool, N=N, T=T, H=H, Hk=Hk,
                                 Dv=Dv, slots=slots.cuda(), slots_out=outs.cuda(), o=o0,
                                 keep=kept.cuda() if keep else None)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    untouched = set(range(P))
    for n in range(N):
        t = T if kept is None else max(0, min(T, int(kept[n])))
        at = slice(n * T, n * T + t)
        if int(slots[n]) < 0:
            assert bool((o[n * T:(n + 1) * T] == 7.0).all())
            continue
        (want, last), (om, lm) = ref.both(q[at], k[at], v[at], g, pool[int(slots[n])], H, Hk, Dv, D ** -0.5)
        _close(o[at], want, om, _tol(T, g), ("o", n))
        assert bool((o[n * T + t:(n + 1) * T] == 7.0).all())
        got = dpool[int(outs[n])]
        if t == 0:
            assert torch.equal(got.cpu(), pool[int(slots[n])])
        _close(got, last, lm, _tol(T, g), ("state", n))
        untouched.discard(int(outs[n]))
    for s in untouched:
        assert torch.equal(dpool[s].cpu(), pool[s]), s


def test_verify_equals_single_tokens_and_rollback():
    """A T-token call is T one-token calls bit for bit, and so is a rollback to a kept prefix; a prompt
    in the recurrent form (f32) is the same recurrence again."""
    from gated_delta_rule_scan_gb300 import mixer
    N, T, H, Hk, Dv = 4, 5, 3, 1, 256
    for dtype in (torch.float32, torch.bfloat16):
        _, (q, k, v), pool, _, _ = _decode_inputs(N, T, H, Hk, Dv, dtype, 2 * N)
        g = _decays(H).cuda()
        kw = dict(log_decay=g, H=H, Hk=Hk, Dv=Dv, N=N)
        a, b = pool.cuda(), pool.cuda()
        outs = torch.arange(N, 2 * N, dtype=torch.int32, device="cuda")
        slots = torch.arange(N, dtype=torch.int32, device="cuda")
        o = mixer.kda_linattn_decode(q=q, k=k, v=v, pool=a, T=T, slots=slots, slots_out=outs, **kw)
        assert torch.equal(a[:N], b[:N])
        states = [b[:N].clone()]
        for t in range(T):
            rows = torch.arange(N, device="cuda") * T + t
            ot = mixer.kda_linattn_decode(q=q[rows], k=k[rows], v=v[rows], pool=b, T=1, **kw)
            assert torch.equal(ot, o[rows])
            states.append(b[:N].clone())
        assert torch.equal(a[N:], states[T])
        keep = torch.tensor([0, 2, 5, 1], dtype=torch.int32, device="cuda")
        mixer.kda_linattn_decode(q=q, k=k, v=v, pool=a, T=T, slots=slots, slots_out=outs, keep=keep, **kw)
        for n in range(N):
            assert torch.equal(a[N + n], states[int(keep[n])][n])


def test_slots_left_out():
    """Slots past the pool, an output slot named twice and one that another row reads are left out and
    reported; nothing is written for them."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    N, H = 5, 2
    _, (q, k, v), pool, _, _ = _decode_inputs(N, 1, H, H, D, torch.float32, 8)
    g = _decays(H).cuda()
    slots = torch.tensor([0, 1, 2, 8, 4], dtype=torch.int32, device="cuda")
    outs = torch.tensor([5, 5, 0, 6, 4], dtype=torch.int32, device="cuda")
    d = pool.cuda()
    o = torch.zeros(N, H * D, device="cuda")
    mixer.kda_linattn_decode(q=q, k=k, v=v, log_decay=g, pool=d, N=N, T=1, H=H, slots=slots,
                             slots_out=outs, o=o)
    assert kda.kda_device_status() == 40013
    assert kda.kda_device_status() == 0
    for n in (1, 2, 3):                       # second writer of 5, writer of slot 0 that row 0 reads, past the pool
        assert bool((o[n] == 0).all())
    assert bool((o[0] != 0).any()) and bool((o[4] != 0).any())
    for s in (0, 1, 2, 3, 6, 7):
        assert torch.equal(d[s].cpu(), pool[s])
    assert not torch.equal(d[5].cpu(), pool[5]) and not torch.equal(d[4].cpu(), pool[4])


def test_long_memory_keeps_a_decay_next_to_one():
    """20000 one-token steps with e^g next to 1: the state's decay is not off by the rounding of e^g,
    which would be 20000 * 2^-25."""
    from gated_delta_rule_scan_gb300 import mixer
    H, T = 1, 20000
    g = torch.tensor([-1.0e-5])
    z = torch.zeros(T, D)
    S = torch.ones(1, H, D, D)
    for dtype in (torch.float32, torch.bfloat16):
        x = z.to(dtype).cuda()
        out = mixer.kda_linattn_prefill(q=x, k=x, v=x, log_decay=g.cuda(), H=H, N=1, T=T, state_in=S.cuda())
        want = torch.exp(g.double() * T)
        # a step rounds the state once: at most T / 2 half-ulps would be 3e-4, in practice they average out;
        # the systematic part alone is bounded by 2^-24 of g T
        err = (out["state_out"].double().cpu() / want - 1).abs().max()
        assert float(err) < 20000 * 2.0 ** -26


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths,H,kind", [([5000], 1, "mixed"), ([3000, 1, 900, 2100], 2, "mixed"),
                                            ([2500], 3, "strong"), ([4097], 2, "none"),
                                            ([64 * 40], 5, "mixed")])
def test_few_long_prompts(lengths, H, kind, dtype):
    """Long prompts of few heads are cut into segments: outputs and states as of the whole."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    rows, N = sum(lengths), len(lengths)
    (q, k, v), (dq, dk, dv) = _inputs(rows, H, H, D, dtype, rows)
    g = _decays(H, kind) if kind != "mixed" else _decays(H, kind) * 0.02
    S = torch.randn(N, H, D, D, generator=torch.Generator().manual_seed(rows))
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    assert kda.kda_linattn_workspace_bytes(N, rows, H, dtype=dtype) > 0
    out = mixer.kda_linattn_prefill(q=dq, k=dk, v=dv, log_decay=g.cuda(), H=H, state_in=S.cuda(),
                                    cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    for n, L in enumerate(lengths):
        b, e = int(cu[n]), int(cu[n + 1])
        (o, last), (om, lm) = ref.both(q[b:e], k[b:e], v[b:e], g, S[n], H, H, D, D ** -0.5)
        _close(out["o"][b:e], o, om, _tol(L, g, dtype, max(lengths)), ("o", n))
        _close(out["state_out"][n], last, lm, _tol(L, g, dtype, max(lengths)), ("state", n))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths,H,kind", [([1700], 52, "mixed"), ([1300, 1700, 0], 26, "none"),
                                            ([2111], 60, "strong")])
def test_many_heads_long_prompts(lengths, H, kind, dtype):
    """Heads enough for few segments, whose states are then formed in pieces; of the heads, which are
    independent, some are looked at."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    rows, N = sum(lengths), len(lengths)
    (q, k, v), (dq, dk, dv) = _inputs(rows, H, H, D, dtype, 31)
    g = _decays(H, kind)
    S = torch.randn(N, H, D, D, generator=torch.Generator().manual_seed(6))
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    out = mixer.kda_linattn_prefill(q=dq, k=dk, v=dv, log_decay=g.cuda(), H=H, state_in=S.cuda(),
                                    cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    some = [0, H // 2, H - 1]
    pick = lambda x: x.reshape(rows, H, D)[:, some].reshape(rows, -1)
    for n in range(N):
        b, e = int(cu[n]), int(cu[n + 1])
        (o, last), (om, lm) = ref.both(pick(q)[b:e], pick(k)[b:e], pick(v)[b:e], g[some], S[n, some], 3, 3,
                                       D, D ** -0.5)
        tol = _tol(e - b, g[some], dtype, max(lengths))
        _close(pick(out["o"].cpu())[b:e], o, om, tol, ("o", n))
        _close(out["state_out"][n, some], last, lm, tol, ("state", n))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,decay", [(10, -0.1), (200, -0.1), (200, -5.0), (3000, -0.01)])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_no_number_reaches_earlier_tokens(what, T, decay, dtype):
    """A NaN or an infinity in one token's row leaves the tokens before it, the other sequences and (in v) the
    other value columns as they are, bit for bit, and is seen where it counts."""
    from gated_delta_rule_scan_gb300 import mixer
    H, at, col = 2, 2 * T // 3, 17
    _, dev = _inputs(3 * T, H, H, D, dtype, T)
    x = dict(zip("qkv", (d.clone() for d in dev)))
    g = torch.full((H,), decay, device="cuda")

    def run():
        return mixer.kda_linattn_prefill(**x, log_decay=g, H=H, N=3, T=T)
    clean = run()
    for value in (float("nan"), float("inf"), float("-inf")):
        x[what][T + at, D + col] = value                   # sequence 1, head 1
        out = run()
        x[what][T + at, D + col] = dev["qkv".index(what)][T + at, D + col]
        o, o0 = (r["o"].view(3, T, H, D) for r in (out, clean))
        s, s0 = (r["state_out"] for r in (out, clean))
        same = torch.ones(3, T, H, D, dtype=torch.bool, device="cuda")
        if what == "q":
            same[1, at, 1] = False
        else:
            same[1, at:, 1, col if what == "v" else slice(None)] = False
        assert torch.equal(o[same], o0[same])
        assert not bool(torch.isfinite(o[1, at, 1, col]))
        live = torch.ones(3, H, D, D, dtype=torch.bool, device="cuda")
        if what == "v":
            live[1, 1, col] = False
        elif what == "k":
            live[1, 1, :, col] = False
        assert torch.equal(s[live], s0[live])
        if what != "q":
            assert not bool(torch.isfinite(s[1, 1, col, col]))


def test_neighbours_that_are_no_numbers():
    """Packed sequences of odd lengths: one of NaN throughout leaves the others as they are."""
    from gated_delta_rule_scan_gb300 import mixer
    H, lengths = 2, [70, 33, 90, 1, 64]
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    for dtype in (torch.float32, torch.bfloat16):
        _, (q, k, v) = _inputs(sum(lengths), H, H, D, dtype, 1)
        g = _decays(H).cuda()
        kw = dict(log_decay=g, H=H, cu_seqlens=cu.cuda(), cu_seqlens_host=cu)
        clean = mixer.kda_linattn_prefill(q=q, k=k, v=v, **kw)
        for x in (q, k, v):
            x[int(cu[1]):int(cu[2])] = float("nan")
        out = mixer.kda_linattn_prefill(q=q, k=k, v=v, **kw)
        for n in (0, 2, 3, 4):
            at = slice(int(cu[n]), int(cu[n + 1]))
            assert torch.equal(out["o"][at], clean["o"][at])
            assert torch.equal(out["state_out"][n], clean["state_out"][n])
        assert bool(torch.isnan(out["o"][int(cu[1]):int(cu[2])]).all())
