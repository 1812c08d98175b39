"""Cases for timing what a speculative serving step needs around and beside the delta-rule mixer:
linear attention with one decay a head (`kda.kda_linattn_prefill[_varlen]` for prompts,
`kda.kda_linattn_decode` for single tokens and verify batches), the verification of drafted tokens
(`kda.kda_draft_accept`), and the norms around a block fused with its gate and residual
(`kda.kda_residual_rmsnorm`).

Each case exists twice: `run` computes it in elementary torch operations in 32 bits (64 for sums
next to a border), or, with `own` set, by the library's calls.  `exact` computes the same from the
definitions in 64 bits.
"""

import math
import random

import torch

own = False

D = 128                      # key width: the state of a value head is [Dv, D]
EPS = 1e-6
CHUNK = 128                  # tokens the plain prefill takes at a time


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _lengths(N, lo, hi, seed):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(N)]


def _prefill(name, N, lo, hi, H, Hk=None, m=1, x="bf16", ragged=True, fused=False):
    """N sequences of lo .. hi tokens; fused: q, k and v are slices of one projection's rows."""
    return dict(name=name, kind="prefill", N=N, lo=lo, hi=hi, H=H, Hk=Hk or H, m=m, x=x,
                ragged=ragged, fused=fused)


def _decode(name, N, T, H, Hk=None, m=1, x="bf16", pad=0, keep=False):
    return dict(name=name, kind="decode", N=N, T=T, H=H, Hk=Hk or H, m=m, x=x, pad=pad, keep=keep)


def _accept(name, N, T, V, x="f32", draft=True, ragged=False):
    return dict(name=name, kind="accept", N=N, T=T, V=V, x=x, draft=draft, ragged=ragged)


def _norms(name, rows, F, x="bf16", stream="bf16", z="bf16", post=True, gate="none"):
    """x, stream, z: types of the block's output, the residual stream and the normed output."""
    return dict(name=name, kind="norms", rows=rows, F=F, x=x, stream=stream, z=z, post=post,
                gate=gate)


def listed():
    return [
        # the benchmark's single prompt
        _prefill("prefill 1x4096 H64", 1, 4096, 4096, 64, ragged=False),
        # the benchmark's packed prompts: 16 sequences of 256 to 8192 tokens
        _prefill("prefill 16 ragged H64", 16, 256, 8192, 64),
        # one long prompt of a narrower layer, prepared planes in f32
        _prefill("prefill 1x16384 H32 f32", 1, 16384, 16384, 32, x="f32", ragged=False),
        # short prompts of a small odd layer: grouped queries, wide value heads, a fused projection
        _prefill("prefill 5 short H6 Hk2 Dv256", 5, 1, 700, 6, 2, 2, fused=True),
        # one user's decode step: latency
        _decode("decode 1x1 H64", 1, 1, 64),
        # the benchmark's decode batch
        _decode("decode 64x1 H64", 64, 1, 64),
        # a padded verify batch with accepted prefixes, grouped queries, wide value heads
        _decode("decode 37x3 H16 Hk4 Dv256 f32", 37, 3, 16, 4, 2, "f32", 5, True),
        # one user's round of three drafted tokens over a large vocabulary
        _accept("accept 1x4 V131072", 1, 4, 131072),
        # the same for the benchmark's batch
        _accept("accept 64x4 V131072", 64, 4, 131072),
        # drafts from a lookup (no probabilities), ragged, an odd vocabulary, bf16
        _accept("accept 37x7 V50021 bf16 lookup", 37, 7, 50021, "bf16", False, True),
        # one token through a layer at the benchmark's width
        _norms("norms 1x6144", 1, 6144, stream="f32", z="f32"),
        # the benchmark's prompt through it, with a gate computed from the input
        _norms("norms 4096x6144 gated", 4096, 6144, gate="sigmoid"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "accept", "accept",
                       "norms", "norms"])
    types = ["f32", "bf16"]
    if kind == "prefill":
        m = rng.choice([1, 1, 2, 3])
        H = max(1, _log_int(rng, 1, 64) // m)
        N = _log_int(rng, 1, 24)
        hi = _log_int(rng, 1, 16384 // N)
        lo = rng.randint(0, hi)
        c = _prefill("", N, lo, hi, H, rng.choice([H, H, rng.randint(1, H)]), m, rng.choice(types),
                     rng.random() < 0.7, rng.random() < 0.4)
    elif kind == "decode":
        m = rng.choice([1, 1, 2])
        H = max(1, _log_int(rng, 1, 64) // m)
        N = _log_int(rng, 1, 64)
        c = _decode("", N, rng.choice([1, 1, 2, 3, 4, 7, 16]), H,
                    rng.choice([H, H, rng.randint(1, H)]), m, rng.choice(types),
                    rng.randrange(0, (N + 3) // 4), rng.random() < 0.4)
    elif kind == "accept":
        c = _accept("", _log_int(rng, 1, 64), rng.randint(1, 8), _log_int(rng, 200, 131072),
                    rng.choice(types), rng.random() < 0.7, rng.random() < 0.5)
    else:
        c = _norms("", _log_int(rng, 1, 4096), 8 * _log_int(rng, 8, 768), rng.choice(types),
                   rng.choice(types), rng.choice(types), rng.random() < 0.7,
                   rng.choice(["none", "channel", "sigmoid", "silu"]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _case_lengths(c):
    if not c["ragged"]:
        return [c["hi"]] * c["N"]
    return _lengths(c["N"], c["lo"], c["hi"], 7 * c["N"] + c["hi"])


def _slopes(H, dev):
    """Log-decays of the heads, a geometric series from e^-0.9 or so to nearly none."""
    h = torch.arange(1, H + 1, device=dev, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / H)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c = case
    s = dict(case=c)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    if c["kind"] in ("prefill", "decode"):
        H, Hk, Dv, N = c["H"], c["Hk"], D * c["m"], c["N"]
        lengths = _case_lengths(c) if c["kind"] == "prefill" else [c["T"]] * N
        rows = sum(lengths)
        x = _dtype(c["x"])
        widths = (Hk * D, Hk * D, H * Dv)
        if c.get("fused"):
            s["q"], s["k"], s["v"] = randn(rows, sum(widths)).to(x).split(widths, 1)
        else:
            s["q"], s["k"], s["v"] = (randn(rows, w).to(x) for w in widths)
        s["log_decay"] = _slopes(H, dev)
        s["o"] = torch.zeros(rows, H * Dv, device=dev)
        if c["kind"] == "prefill":
            s["lengths"] = lengths
            cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
            s["cu_host"], s["cu"] = cu, cu.to(dev)
            s["state_in"] = randn(N, H, Dv, D)
            s["state_out"] = torch.empty_like(s["state_in"])
            if own:
                from gated_delta_rule_scan_gb300 import kda
                s["workspace"] = kda.linattn_workspace(N, rows, H, dev, Hk=Hk, Dv=Dv, dtype=x)
        else:
            # a pool in use: the step reads some slots and writes others, as a verify does
            P = 2 * N + 3
            s["pool"] = randn(P, H, Dv, D)
            perm = torch.randperm(P, generator=g, device=dev).to(torch.int32)
            s["slots"], s["slots_out"] = perm[:N].contiguous(), perm[N:2 * N].contiguous()
            s["slots"][N - c["pad"]:] = -1      # a padded batch: the last rows carry no sequence
            s["keep"] = (torch.randint(0, c["T"] + 1, (N,), generator=g, device=dev,
                                       dtype=torch.int32) if c["keep"] else None)
    elif c["kind"] == "accept":
        N, T, V, x = c["N"], c["T"], c["V"], _dtype(c["x"])
        logits = randn(N, T, V).mul_(3.0)
        s["target"] = torch.softmax(logits, -1).to(x)
        # a smaller model's guess at the same distribution; its tokens are drawn from it
        logits = logits[:, :T - 1].add_(randn(N, T - 1, V).mul_(1.0))
        guess = torch.softmax(logits, -1).to(x)
        s["tokens"] = (torch.multinomial(guess.float().reshape(-1, V), 1, generator=g)
                       .reshape(N, T - 1).to(torch.int32) if T > 1
                       else torch.zeros(N, 0, dtype=torch.int32, device=dev))
        s["draft"] = guess if c["draft"] else None
        s["n_draft"] = (torch.randint(0, T, (N,), generator=g, device=dev, dtype=torch.int32)
                        if c["ragged"] else None)
        s["u"], s["r"] = rand(N, T - 1), rand(N)
        s["keep"] = torch.zeros(N, dtype=torch.int32, device=dev)
        s["out_tokens"] = torch.zeros(N, T, dtype=torch.int32, device=dev)
    else:
        rows, F = c["rows"], c["F"]
        # a residual stream with a few outlier channels
        res = randn(rows, F).mul_(2.0)
        res[:, ::97] *= 20.0
        s["residual"] = res.to(_dtype(c["stream"]))
        s["block"] = randn(rows, F).mul_(0.7).to(_dtype(c["x"]))
        s["w_post"] = randn(F).mul_(0.1).add_(1.0) if c["post"] else None
        s["w_pre"] = randn(F).mul_(0.1).add_(1.0)
        s["gate"] = (None if c["gate"] == "none" else randn(F).mul_(0.2).add_(1.0)
                     if c["gate"] == "channel" else randn(rows, F).to(_dtype(c["x"])))
        s["h"] = torch.empty_like(s["residual"])
        s["z"] = torch.empty(rows, F, device=dev, dtype=_dtype(c["z"]))
    return s


RES_SCALE, BLOCK_SCALE = 0.9, 0.35


# ------------------------------------------------------------------------------------------
# the plain forms and the library's calls
# ------------------------------------------------------------------------------------------

def _plain_prefill(s):
    c = s["case"]
    H, Hk, Dv = c["H"], c["Hk"], D * c["m"]
    g = s["log_decay"]
    head = torch.arange(H, device=g.device) % Hk
    row = 0
    for n, L in enumerate(s["lengths"]):
        S = s["state_in"][n]                                    # [H, Dv, D]
        for c0 in range(0, L, CHUNK):
            C = min(CHUNK, L - c0)
            at = slice(row + c0, row + c0 + C)
            q = s["q"][at].float().reshape(C, Hk, D)[:, head].transpose(0, 1)
            k = s["k"][at].float().reshape(C, Hk, D)[:, head].transpose(0, 1)
            v = s["v"][at].float().reshape(C, H, Dv).transpose(0, 1)
            t = torch.arange(C, device=g.device)
            gap = t[:, None] - t[None, :]
            w = torch.exp(g[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
            o = ((q @ k.transpose(1, 2)) * w) @ v
            o = o + torch.exp(g[:, None] * (t + 1))[:, :, None] * (q @ S.transpose(1, 2))
            s["o"][at] = (o * D ** -0.5).transpose(0, 1).reshape(C, H * Dv)
            k = k * torch.exp(g[:, None] * (C - 1 - t))[:, :, None]
            S = torch.exp(g * C)[:, None, None] * S + v.transpose(1, 2) @ k
        s["state_out"][n] = S
        row += L
    return s["o"], s["state_out"]


def _plain_decode(s):
    c = s["case"]
    N, T, H, Hk, Dv = c["N"], c["T"], c["H"], c["Hk"], D * c["m"]
    live = N - c["pad"]
    src, dst = s["slots"][:live].long(), s["slots_out"][:live].long()
    keep = s["keep"][:live].long() if s["keep"] is not None else torch.full_like(src, T)
    head = torch.arange(H, device=src.device) % Hk
    q = s["q"].float().reshape(N, T, Hk, D)[:live, :, head]
    k = s["k"].float().reshape(N, T, Hk, D)[:live, :, head]
    v = s["v"].float().reshape(N, T, H, Dv)[:live]
    decay = torch.exp(s["log_decay"])[:, None, None]
    S = s["pool"][src]
    out = s["o"].reshape(N, T, H, Dv)
    for t in range(T):
        on = t < keep
        new = S * decay + v[:, t, :, :, None] * k[:, t, :, None, :]
        S = torch.where(on[:, None, None, None], new, S)
        o = (S * q[:, t, :, None, :]).sum(-1) * D ** -0.5
        out[:live, t] = torch.where(on[:, None, None], o, out[:live, t])
    s["pool"][dst] = S
    return s["o"], s["pool"]


def _plain_accept(s):
    c = s["case"]
    N, T, V = c["N"], c["T"], c["V"]
    dev = s["r"].device
    rows = torch.arange(N, device=dev)
    count = (s["n_draft"].long() if s["n_draft"] is not None
             else torch.full((N,), T - 1, device=dev))
    step = torch.arange(T - 1, device=dev)
    tok = s["tokens"].long()
    p = s["target"][:, :T - 1].gather(2, tok[:, :, None])[..., 0].double()
    q = (s["draft"].gather(2, tok[:, :, None])[..., 0].double() if s["draft"] is not None
         else torch.ones_like(p))
    good = (s["u"].double() * q < p) & (step < count[:, None])
    taken = good.long().cumprod(1).sum(1)                       # drafts accepted in a row
    refused = taken < count
    w = s["target"][rows, taken].double()
    if T > 1:
        at = taken.clamp(max=T - 2)
        if s["draft"] is not None:
            rest = (w - s["draft"][rows, at].double()).clamp(min=0.0)
        else:
            rest = w.scatter(1, tok[rows, at][:, None], 0.0)
        # where nothing is left over, p itself stands in
        use = refused & (rest.sum(1) > 0)
        w = torch.where(use[:, None], rest, w)
    cum = w.cumsum(1)
    aim = s["r"].double() * cum[:, -1]
    new = (cum <= aim[:, None]).sum(1)
    s["keep"].copy_(taken + 1)
    place = torch.arange(T, device=dev)
    padded = torch.cat([tok, torch.full((N, 1), -1, device=dev)], 1)
    out = torch.where(place < taken[:, None], padded, torch.full_like(padded, -1))
    out[rows, taken] = new
    s["out_tokens"].copy_(out)
    return s["keep"], s["out_tokens"]


def _plain_norms(s):
    c = s["case"]
    y = s["block"].float()
    if s["w_post"] is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * {"channel": lambda: z, "sigmoid": lambda: torch.sigmoid(z),
                 "silu": lambda: z * torch.sigmoid(z)}[c["gate"]]()
    h = RES_SCALE * s["residual"].float() + BLOCK_SCALE * y
    z = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w_pre"]
    s["h"].copy_(h)
    s["z"].copy_(z)
    return s["h"], s["z"]


def _own(s):
    from gated_delta_rule_scan_gb300 import kda
    c = s["case"]
    if c["kind"] == "prefill":
        args = (s["q"], s["k"], s["v"], s["log_decay"], s["state_in"], s["state_out"], s["o"],
                s["workspace"])
        heads = dict(H=c["H"], Hk=c["Hk"], Dv=D * c["m"])
        if c["ragged"]:
            kda.kda_linattn_prefill_varlen(*args, s["cu"], s["cu_host"], **heads)
        else:
            kda.kda_linattn_prefill(*args, N=c["N"], T=c["hi"], **heads)
        return s["o"], s["state_out"]
    if c["kind"] == "decode":
        kda.kda_linattn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], s["o"],
                               N=c["N"], T=c["T"], H=c["H"], Hk=c["Hk"], Dv=D * c["m"],
                               slots=s["slots"], slots_out=s["slots_out"], keep=s["keep"])
        return s["o"], s["pool"]
    if c["kind"] == "accept":
        kda.kda_draft_accept(s["target"], s["tokens"], s["u"], s["r"], s["keep"], s["out_tokens"],
                             draft=s["draft"], n_draft=s["n_draft"])
        return s["keep"], s["out_tokens"]
    act = c["gate"] if c["gate"] in ("sigmoid", "silu") else "none"
    kda.kda_residual_rmsnorm(s["residual"], s["block"], s["h"], s["z"], s["w_pre"],
                             block_w=s["w_post"], gate=s["gate"], gate_act=act,
                             res_scale=RES_SCALE, block_scale=BLOCK_SCALE, eps=EPS)
    return s["h"], s["z"]


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "accept": _plain_accept,
            "norms": _plain_norms}[state["case"]["kind"]](state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without, and its exact outputs
# ------------------------------------------------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    c = case
    if c["kind"] in ("prefill", "decode"):
        H, Hk, Dv, N = c["H"], c["Hk"], D * c["m"], c["N"]
        if c["kind"] == "prefill":
            tokens, live = sum(_case_lengths(c)), N
        else:
            live = N - c["pad"]
            tokens = live * c["T"]
        moved = tokens * ((2 * Hk * D + H * Dv) * _size(c["x"]) + H * Dv * 4)
        # a token's products with the state: one to update it, one to read it out
        return {"bytes": moved + 2 * live * H * Dv * D * 4 + H * 4,
                "flops": tokens * H * Dv * D * 4}
    if c["kind"] == "accept":
        N, T, V = c["N"], c["T"], c["V"]
        # the row the new token is drawn from; the draft's beside it where one was refused, which
        # about three sequences in four see
        row = V * _size(c["x"]) * (1.75 if c["draft"] and T > 1 else 1.0)
        return {"bytes": int(N * (row + (T - 1) * (8 + 2 * _size(c["x"])) + 4 * (T + 2))),
                "flops": 2 * N * V}
    rows, F = c["rows"], c["F"]
    per = _size(c["x"]) + 2 * _size(c["stream"]) + _size(c["z"])
    if c["gate"] in ("sigmoid", "silu"):
        per += _size(c["x"])
    return {"bytes": rows * F * per + F * 4 * (1 + c["post"] + (c["gate"] == "channel")),
            "flops": rows * F * 10}


def _exact_prefill(s):
    """The recurrence token by token, the sequences side by side, longest first."""
    c = s["case"]
    N, H, Hk, Dv = c["N"], c["H"], c["Hk"], D * c["m"]
    dev = s["o"].device
    lengths, cu = s["lengths"], s["cu_host"].tolist()
    order = sorted(range(N), key=lambda n: -lengths[n])
    starts = torch.tensor([cu[n] for n in order], device=dev)
    decay = s["log_decay"].double().exp()
    S = s["state_in"].double()[order].mT.reshape(N * H, D, Dv).contiguous()   # [key, value]
    lam = decay.repeat(N)[:, None, None]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=dev)
    group = [h % Hk for h in range(H)]
    live = N
    for t in range(max(lengths, default=0)):
        while live and lengths[order[live - 1]] <= t:
            live -= 1
        at = starts[:live] + t
        q = s["q"][at].double().view(live, Hk, D)[:, group].reshape(live * H, D, 1)
        k = s["k"][at].double().view(live, Hk, D)[:, group].reshape(live * H, D, 1)
        v = s["v"][at].double().view(live * H, 1, Dv)
        part = S[:live * H]
        part.mul_(lam[:live * H]).add_(k * v)
        o[at] = (part.mT @ q).view(live, H * Dv) / math.sqrt(D)
    out = torch.empty(N, H, Dv, D, dtype=torch.float64, device=dev)
    out[order] = S.view(N, H, D, Dv).mT
    return o, out


def _exact_decode(s):
    """In closed form: token t's readout sees the tokens up to it and the state decayed t + 1 times."""
    c = s["case"]
    N, T, H, Hk, Dv = c["N"], c["T"], c["H"], c["Hk"], D * c["m"]
    pool, o = s["pool"].double(), s["o"].double().view(N, T, H, Dv)
    keep = [T] * N if s["keep"] is None else s["keep"].tolist()
    g = s["log_decay"].double()
    group = [h % Hk for h in range(H)]
    slots, outs = s["slots"].tolist(), s["slots_out"].tolist()
    written = {}
    for n in range(N - c["pad"]):
        t = torch.arange(keep[n], device=g.device, dtype=torch.float64)
        q, k = (s[x].double().view(N, T, Hk, D)[n, :keep[n]][:, group] for x in ("q", "k"))
        v = s["v"].double().view(N, T, H, Dv)[n, :keep[n]]
        S0 = pool[slots[n]]
        gap = (t[:, None] - t)[None]
        w = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0)
        near = torch.einsum("thi,shi->hts", q, k) * w
        far = torch.einsum("hji,thi->thj", S0, q) * torch.exp((t[:, None] + 1) * g)[:, :, None]
        o[n, :keep[n]] = (torch.einsum("hts,shj->thj", near, v) + far) / math.sqrt(D)
        left = torch.exp((keep[n] - 1 - t)[:, None] * g)[:, :, None]
        written[outs[n]] = (S0 * torch.exp(keep[n] * g)[:, None, None]
                            + torch.einsum("shj,shi->hji", v * left, k))
    for slot, S in written.items():
        pool[slot] = S
    return o.view(N * T, H * Dv), pool


def _exact_accept(s):
    c = s["case"]
    N, T, V = c["N"], c["T"], c["V"]
    keep, out = [], []
    tokens, u, r = s["tokens"].tolist(), s["u"].tolist(), s["r"].tolist()
    count = [T - 1] * N if s["n_draft"] is None else s["n_draft"].tolist()
    for n in range(N):
        line = []
        weights = None
        for i in range(count[n]):
            x = tokens[n][i]
            p = float(s["target"][n, i, x])
            q = 1.0 if s["draft"] is None else float(s["draft"][n, i, x])
            if u[n][i] * q < p:
                line.append(x)
                continue
            weights = s["target"][n, i].double().clone()
            if s["draft"] is None:
                weights[x] = 0.0
            else:
                weights = torch.relu(weights - s["draft"][n, i].double())
            if not bool((weights > 0).any()):
                weights = None
            break
        if weights is None:
            weights = s["target"][n, len(line)].double()
        cum = weights.cumsum(0)
        # the first index whose running sum passes r of the whole
        new = int(torch.searchsorted(cum, r[n] * cum[-1], right=True))
        keep.append(len(line) + 1)
        out.append(line + [new] + [-1] * (T - 1 - len(line)))
    dev = s["keep"].device
    return (torch.tensor(keep, dtype=torch.int32, device=dev),
            torch.tensor(out, dtype=torch.int32, device=dev).view(N, T))


def _exact_norms(s):
    c = s["case"]
    y = s["block"].double()
    if s["w_post"] is not None:
        y = y * torch.rsqrt(y.pow(2).mean(1, True) + EPS) * s["w_post"].double()
    if s["gate"] is not None:
        z = s["gate"].double()
        if c["gate"] == "sigmoid":
            z = 1.0 / (1.0 + torch.exp(-z))
        elif c["gate"] == "silu":
            z = z / (1.0 + torch.exp(-z))
        y = y * z
    h = RES_SCALE * s["residual"].double() + BLOCK_SCALE * y
    return h, h * torch.rsqrt(h.pow(2).mean(1, True) + EPS) * s["w_pre"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_prefill, "decode": _exact_decode, "accept": _exact_accept,
            "norms": _exact_norms}[case["kind"]](s)
