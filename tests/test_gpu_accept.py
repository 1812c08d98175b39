"""Verification of drafted tokens against the target's probabilities: keep and tokens against a plain
64-bit form, which they have to equal."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def plain(target, tokens, u, r, draft, n_draft):
    N, T, V = target.shape
    keep, out = [], []
    for n in range(N):
        count = T - 1 if n_draft is None else min(int(n_draft[n]), T - 1)
        if count < 0:
            keep.append(0)
            out.append([-1] * T)
            continue
        line, w = [], None
        for i in range(count):
            x = int(tokens[n, i])
            if 0 <= x < V:
                p = float(target[n, i, x])
                q = 1.0 if draft is None else float(draft[n, i, x])
                if float(u[n, i]) * q < p:
                    line.append(x)
                    continue
            w = target[n, i].double().clone()
            if draft is not None:
                q = draft[n, i].double()
                w -= torch.where(q > 0, q, torch.zeros_like(q))
            elif 0 <= x < V:
                w[x] = 0.0
            w[~((w > 0) & torch.isfinite(w))] = 0.0
            if not bool((w > 0).any()):
                w = None
            break
        if w is None:
            w = target[n, len(line)].double().clone()
            w[~((w > 0) & torch.isfinite(w))] = 0.0
        cum = w.cumsum(0)
        new = -1
        if float(cum[-1]) > 0:
            new = int(torch.searchsorted(cum, float(r[n]) * float(cum[-1]), right=True))
        keep.append(len(line) + 1)
        out.append(line + [new] + [-1] * (T - 1 - len(line)))
    return torch.tensor(keep, dtype=torch.int32), torch.tensor(out, dtype=torch.int32).reshape(N, T)


def _case(N, T, V, dtype, seed, sharp=3.0, noise=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(N, T, V, generator=g) * sharp
    target = torch.softmax(logits, -1).to(dtype)
    draft = torch.softmax(logits[:, :T - 1] + noise * torch.randn(N, T - 1, V, generator=g), -1).to(dtype)
    tokens = (torch.multinomial(draft.float().reshape(-1, V), 1, generator=g).reshape(N, T - 1).to(torch.int32)
              if T > 1 else torch.zeros(N, 0, dtype=torch.int32))
    return target, draft, tokens, torch.rand(N, T - 1, generator=g), torch.rand(N, generator=g), g


def _run(target, tokens, u, r, draft, n_draft=None):
    from gated_delta_rule_scan_gb300 import mixer
    c = lambda t: None if t is None else t.cuda()
    keep, out = mixer.kda_draft_accept(target=c(target), tokens=c(tokens), u=c(u), r=c(r), draft=c(draft),
                                       n_draft=c(n_draft))
    return keep.cpu(), out.cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,T,V", [(1, 1, 1), (3, 4, 7), (5, 2, 1024), (4, 16, 1025), (2, 3, 4099),
                                   (1, 4, 65536), (3, 4, 50021), (300, 3, 640), (2, 2, 1200007)])
@pytest.mark.parametrize("lookup", [False, True])
def test_against_plain(N, T, V, dtype, lookup):
    target, draft, tokens, u, r, g = _case(N, T, V, dtype, N + T + V)
    if lookup:
        draft = None
    if T == 1:
        draft = None
    n_draft = torch.randint(-1, T, (N,), generator=g, dtype=torch.int32) if N > 2 else None
    want = plain(target, tokens, u, r, draft, n_draft)
    got = _run(target, tokens, u, r, draft, n_draft)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("V", [777, 40000])
def test_flat_rows_and_every_border(V):
    """Rows of equal weights, r on a fine grid: a sum off by one weight's 2^-20 would name another index."""
    N = 64
    target = torch.full((N, 1, V), 1.0 / V)
    r = torch.arange(N).float() / N + 2.0 ** -12
    empty = torch.zeros(N, 0)
    got = _run(target, empty.int(), empty, r, None)
    w = torch.full((V,), 1.0, dtype=torch.float64) * float(target[0, 0, 0])
    cum = w.cumsum(0)
    want = torch.searchsorted(cum, r.double() * cum[-1], right=True).to(torch.int32)
    assert torch.equal(got[1][:, 0], want)


def test_edges():
    V, T = 64, 3
    t = torch.zeros(8, T, V)
    t[:, :, 5] = 1.0
    d = t[:, :T - 1].clone()
    tokens = torch.full((8, T - 1), 5, dtype=torch.int32)
    u, r = torch.zeros(8, T - 1), torch.full((8,), 0.999)
    u[0] = 1.0 - 2.0 ** -24                        # 0: equal probabilities hold for any u below 1
    tokens[1, 0] = 7                               # 1: p = q = 0: refused, nothing left of p - q: p itself
    tokens[2, 0] = V                               # 2: ids outside the vocabulary are refused
    tokens[3, 0] = -3
    t[4, 0] = 0.0                                  # 4: a row without weights
    t[5, 0, 9] = float("nan")                      # 5: NaN and infinities weigh nothing
    t[5, 0, 10] = float("inf")
    tokens[5, 0] = 9
    r[6] = 1.0                                     # 6: r past its range is clamped
    r[7] = float("nan")
    want = plain(t, tokens, u, torch.where(torch.isfinite(r), r.clamp(max=1 - 2.0 ** -24), 0), d, None)
    got = _run(t, tokens, u, r, d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert got[1][4, 0] == -1 and got[0][4] == 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lookup", [False, True])
def test_no_numbers_in_long_rows(dtype, lookup):
    """NaN, infinities and negative entries in rows of many whole tiles, in either side."""
    N, T, V = 12, 2, 5120
    target, draft, tokens, u, r, g = _case(N, T, V, dtype, 77)
    u[:] = 1 - 2.0 ** -24
    for i, bad in enumerate([float("nan"), float("inf"), -float("inf"), -0.5]):
        target[:, :, 500 + 700 * i] = bad
        draft[:, :, 600 + 700 * i] = bad
        target[1::2, :, 900 + 700 * i] = bad         # in both
        draft[1::2, :, 900 + 700 * i] = bad
    tokens[:] = torch.randint(0, V, (N, 1), generator=g, dtype=torch.int32)
    draft = None if lookup else draft
    want = plain(target, tokens, u, r, draft, None)
    got = _run(target, tokens, u, r, draft)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_denormal_probabilities():
    """Weights of a few times 2^-149: r times their sum may round to the sum, u q to p."""
    tiny = 2.0 ** -149
    V, cases = 9, [[1], [1, 1], [0, 3, 2], [5, 0, 0, 1], [0, 0, 0, 0, 0, 0, 0, 0, 1]]
    N = 4 * len(cases)
    target = torch.zeros(N, 2, V)
    for i in range(N):
        row = cases[i // 4]
        target[i, :, :len(row)] = torch.tensor(row, dtype=torch.float64).mul(tiny).float()
    r = torch.tensor([1 - 2.0 ** -24, 0.6, 0.4, 0.0]).repeat(len(cases))
    empty = torch.zeros(N, 0)
    want = plain(target[:, :1], empty.int(), empty, r, None, None)
    got = _run(target[:, :1].contiguous(), empty.int(), empty, r, None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    draft = target[:, :1].clone()
    tokens = torch.tensor([row.index(max(row)) for row in cases], dtype=torch.int32).repeat_interleave(4)[:, None]
    u = torch.tensor([1 - 2.0 ** -24, 0.9, 0.5, 0.0]).repeat(len(cases))[:, None]
    want = plain(target, tokens, u, r, draft, None)
    got = _run(target, tokens, u, r, draft)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_of_a_padded_vocabulary():
    """target and draft as slices of wider rows."""
    N, T, V, W = 3, 4, 1500, 1537
    target, draft, tokens, u, r, _ = _case(N, T, V, torch.float32, 4)
    from gated_delta_rule_scan_gb300 import mixer
    wide = torch.full((N, T, W), 9.0, device="cuda")
    wide_d = torch.full((N, T - 1, W), 9.0, device="cuda")
    wide[:, :, :V] = target.cuda()
    wide_d[:, :, :V] = draft.cuda()
    keep, out = mixer.kda_draft_accept(target=wide[:, :, :V], tokens=tokens.cuda(), u=u.cuda(), r=r.cuda(),
                                       draft=wide_d[:, :, :V])
    want = plain(target, tokens, u, r, draft, None)
    assert torch.equal(keep.cpu(), want[0]) and torch.equal(out.cpu(), want[1])


def test_distribution():
    """Over many draws the accepted-or-redrawn first token follows the target (chi-square, 15 cells:
    mean 15, deviation 5.5; 60 is 8 deviations out)."""
    N, V = 20000, 16
    target, draft, _, _, _, g = _case(1, 2, V, torch.float32, 3, sharp=1.0)
    p, q = target.expand(N, 2, V).contiguous(), draft.expand(N, 1, V).contiguous()
    tokens = torch.multinomial(q.reshape(N, V), 1, generator=g).to(torch.int32)
    _, out = _run(p, tokens, torch.rand(N, 1, generator=g), torch.rand(N, generator=g), q)
    seen = torch.bincount(out[:, 0].long(), minlength=V).double()
    want = N * target[0, 0].double()
    assert float(((seen - want) ** 2 / want).sum()) < 60
