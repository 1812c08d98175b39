"""Cases for timing the mixer's low-bit serving operators: projections by 4-bit weights with group
scales (`mixer.kda_proj_w4`), the 8-bit pool of recurrent states written and read back
(`kda.kda_state_store_q8`, `kda.kda_state_load_q8`), and the decode / verify step on that pool
(`kda.kda_decode_fused_q8`).

Each case exists twice: `run` computes it in elementary torch operations in 32 bits, or, with `own`
set, by the library's calls.  `exact` computes the same from the definitions in 64 bits.
"""

import math

import torch

own = False

D = 128                      # head width: the state of a value head is [Dv, D]
L2_EPS = RMS_EPS = 1e-6
GATE_LB = -5.0
E4M3_MAX, INT8_MAX = 448.0, 127.0
TINY = 2.0 ** -100           # a state row whose largest magnitude is below this is stored as zero


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _proj(name, t, H, in_f, group, x="f32", scale="bf16", zeros=False):
    return dict(name=name, kind="proj", t=t, H=H, in_f=in_f, group=group, x=x, scale=scale,
                zeros=zeros)


def _store(name, N, H, m=1, pool=None):
    return dict(name=name, kind="store", N=N, H=H, m=m, pool=pool or 2 * N + 3)


def _load(name, N, H, m=1, pool=None):
    return dict(name=name, kind="load", N=N, H=H, m=m, pool=pool or 2 * N + 3)


def _decode(name, N, T, H, Hk=None, m=1, gdn=False, raw="bf16", pad=0, K=4, keep=False):
    return dict(name=name, kind="decode", N=N, T=T, H=H, Hk=Hk or H, m=m, gdn=gdn, raw=raw,
                pad=pad, K=K, keep=keep)


def listed():
    return [
        # one token through a small layer: the launch and the first bytes' latency
        _proj("proj t1 H4 512 g32 zeros", 1, 4, 512, 32, scale="f32", zeros=True),
        # one user's decode step at the benchmark's layer width: the weights' bytes bound it
        _proj("proj t1 H64 6144 g128", 1, 64, 6144, 128),
        # an odd batch of bf16 activations, zero points, a width that is not a power of two
        _proj("proj t13 H16 2176 g64 zeros", 13, 16, 2176, 64, x="bf16", zeros=True),
        # the benchmark's decode batch of 64 rows
        _proj("proj t64 H64 6144 g128", 64, 64, 6144, 128),
        # 64 users by a 4-token verify: the most rows of one call
        _proj("proj t256 H64 6144 g128", 256, 64, 6144, 128),
        # the whole decode batch's states put away (preempted, or kept as prefixes)
        _store("store 64 x H64", 64, 64),
        # a few sequences of an odd layer with wide value heads
        _store("store 3 x H5 Dv256", 3, 5, 2),
        # cached prefixes brought back for the benchmark's batch
        _load("load 64 x H64", 64, 64),
        # one user: latency
        _decode("decode 1x1 H64", 1, 1, 64),
        # the benchmark's decode batch
        _decode("decode 64x1 H64", 64, 1, 64),
        # its 4-token verify, written beside the states from before the round
        _decode("decode 64x4 H64", 64, 4, 64),
        # grouped queries, wide value heads, per-head gate, a padded batch with accepted prefixes
        _decode("decode 37x3 H16 Hk4 Dv256 gdn", 37, 3, 16, 4, 2, True, "f32", 5, 4, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["proj", "proj", "proj", "store", "load", "decode", "decode", "decode"])
    if kind == "proj":
        c = _proj("", _log_int(rng, 1, 256), _log_int(rng, 1, 64), 128 * _log_int(rng, 1, 48),
                  rng.choice([32, 64, 128]), rng.choice(["f32", "bf16"]),
                  rng.choice(["f32", "bf16"]), rng.random() < 0.5)
    elif kind in ("store", "load"):
        N, m = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 3])
        c = (_store if kind == "store" else _load)("", N, max(1, _log_int(rng, 1, 64) // m), m,
                                                   N + rng.randrange(1, N + 4))
    else:
        m = rng.choice([1, 1, 2])
        H = max(1, _log_int(rng, 1, 64) // m)
        N = _log_int(rng, 1, 64)
        c = _decode("", N, rng.choice([1, 1, 2, 3, 4]), H,
                    rng.choice([H, H, rng.randrange(1, H + 1)]), m, rng.random() < 0.4,
                    rng.choice(["f32", "bf16"]), rng.randrange(0, (N + 3) // 4),
                    rng.choice([4, 4, 2, 3, 6]), rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _dims(H):
    return (H * D, H * D, H * D, D, D, H)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _perm(g, n, dev):
    return torch.randperm(n, generator=g, device=dev).to(torch.int32)


def _channels(c):
    return 2 * c["Hk"] * D + c["H"] * c["m"] * D


def _random_pool(g, dev, P, H, Dv, fmt):
    """Codes and row scales of a pool that has been in use: states ~ N(0, 0.02) in 8 bits."""
    x = torch.randn(P, H, Dv, D, generator=g, device=dev).mul_(0.02)
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "e4m3":
        codes = (x * (E4M3_MAX / amax)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return codes, (amax / E4M3_MAX).squeeze(-1).contiguous()
    codes = (x * (INT8_MAX / amax)).round_().clamp_(-INT8_MAX, INT8_MAX).to(torch.int8)
    return codes, (amax / INT8_MAX).squeeze(-1).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c = case
    s = dict(case=c)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["kind"] == "proj":
        in_f, group, t = c["in_f"], c["group"], c["t"]
        # activations with a few outlier channels, as the layer norm before a mixer leaves them
        x = randn(t, in_f)
        x[:, ::97] *= 20.0
        s["x"] = x.to(_dtype(c["x"]))
        s["w"], s["scales"], s["zeros"], s["outs"] = [], [], [], []
        for rows in _dims(c["H"]):
            q = randn(rows, in_f).mul_(2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
            s["w"].append(q[:, 0::2] | (q[:, 1::2] << 4))
            ng = in_f // group
            s["scales"].append(((0.8 + 0.4 * torch.rand(rows, ng, generator=g, device=dev))
                                * 0.38 / math.sqrt(in_f)).to(_dtype(c["scale"])))
            s["zeros"].append((8.0 + randn(rows, ng)).round_().clamp_(0, 15)
                              .to(_dtype(c["scale"])))
            s["outs"].append(torch.empty(t, rows, device=dev))
        if not c["zeros"]:
            s["zeros"] = None
        return s

    Dv = D * c["m"]
    N, H = c["N"], c["H"]
    if c["kind"] in ("store", "load"):
        P = c["pool"]
        R = 3 * (2 * H * D + H * Dv)
        s["slots"] = _perm(g, P, dev)[:N].contiguous()
        s["rows"] = _perm(g, N, dev)
        if c["kind"] == "store":
            s["state"] = randn(N, H, Dv, D).mul_(0.02)
            s["ring"] = randn(N, R)
            s["codes"] = torch.zeros(P, H, Dv, D, device=dev).to(torch.float8_e4m3fn)
            s["scales"] = torch.zeros(P, H, Dv, device=dev)
            s["ring_pool"] = torch.zeros(P, R, device=dev)
        else:
            s["codes"], s["scales"] = _random_pool(g, dev, P, H, Dv, "int8")
            s["ring_pool"] = randn(P, R)
            s["state"] = torch.zeros(N, H, Dv, D, device=dev)
            s["ring"] = torch.zeros(N, R, device=dev)
        return s

    T, Hk, K = c["T"], c["Hk"], c["K"]
    rows, live = N * T, N - c["pad"]
    P = 2 * N + 3
    ch = _channels(c)
    raw = _dtype(c["raw"])
    s["q"], s["k"] = (randn(rows, Hk * D).to(raw) for _ in range(2))
    s["v"] = randn(rows, H * Dv).to(raw)
    s["conv_w"] = randn(ch, K).mul_(0.5)
    s["ring_pool"] = randn(P, ch, K - 1)
    s["f"] = randn(rows, H if c["gdn"] else H * D)
    s["dt_bias"] = randn(H if c["gdn"] else H * D).mul_(0.5)
    s["a_log"] = torch.rand(H, generator=g, device=dev).mul_(15.0).add_(1.0).log_()
    s["beta"] = randn(rows, H)
    s["norm_w"] = randn(Dv).mul_(0.1).add_(1.0)
    s["z"] = randn(rows, H * Dv)
    s["codes"], s["scales"] = _random_pool(g, dev, P, H, Dv, "e4m3")
    perm = _perm(g, P, dev)
    s["slots"], s["slots_out"] = perm[:N].contiguous(), perm[N:2 * N].contiguous()
    s["slots"][live:] = -1                     # a padded batch: the last rows carry no sequence
    s["keep"] = (torch.randint(0, T + 1, (N,), generator=g, device=dev, dtype=torch.int32)
                 if c["keep"] else None)
    s["y"] = torch.zeros(rows, H * Dv, device=dev)
    return s


# ------------------------------------------------------------------------------------------
# the plain forms and the library's calls
# ------------------------------------------------------------------------------------------

def _unpack(w):
    return torch.stack((w & 15, w >> 4), dim=-1).reshape(w.shape[0], -1)


def _plain_proj(s):
    group = s["case"]["group"]
    x = s["x"].float()
    out = []
    for i, w in enumerate(s["w"]):
        q = _unpack(w).float().reshape(w.shape[0], -1, group)
        z = 8.0 if s["zeros"] is None else s["zeros"][i].float()[:, :, None]
        wf = (q - z) * s["scales"][i].float()[:, :, None]
        out.append(x @ wf.reshape(w.shape[0], -1).T)
    return out


def _plain_quantise(x):
    """e4m3 codes and f32 scales of rows of 128 (IEEE divisions: tensor by tensor)."""
    amax = x.abs().amax(-1)
    top = torch.full_like(amax, E4M3_MAX)
    live = amax >= TINY
    inv = torch.where(live, top / amax, torch.zeros_like(amax))
    scale = torch.where(live, amax / top, torch.zeros_like(amax))
    return (x * inv[..., None]).to(torch.float8_e4m3fn), scale


def _bytes(t):
    return t.view(torch.uint8)


def _plain_store(s):
    codes, scales = _plain_quantise(s["state"][s["rows"].long()])
    dst = s["slots"].long()
    _bytes(s["codes"])[dst] = _bytes(codes)
    s["scales"][dst] = scales
    s["ring_pool"][dst] = s["ring"][s["rows"].long()]
    return s["codes"], s["scales"], s["ring_pool"]


def _plain_load(s):
    src, dst = s["slots"].long(), s["rows"].long()
    s["state"][dst] = s["codes"][src].float() * s["scales"][src][..., None]
    s["ring"][dst] = s["ring_pool"][src]
    return s["state"], s["ring"]


def _plain_decode(s):
    c = s["case"]
    N, T, H, Hk, m, K = c["N"], c["T"], c["H"], c["Hk"], c["m"], c["K"]
    live, Dv, R = N - c["pad"], D * m, K - 1
    src, dst = s["slots"][:live].long(), s["slots_out"][:live].long()
    keep = s["keep"][:live].long() if s["keep"] is not None else torch.full_like(src, T)

    def by_seq(x):
        return x.reshape(N, T, -1)[:live].float()

    # conv + SiLU over the carried ring and the new rows, and the ring after `keep` rows
    raw = torch.cat([by_seq(s["q"]), by_seq(s["k"]), by_seq(s["v"])], -1).transpose(1, 2)
    window = torch.cat([s["ring_pool"][src], raw], -1)             # [live, channels, R + T]
    conv = (window.unfold(2, K, 1) * s["conv_w"][:, None, :]).sum(-1)
    x = (conv * torch.sigmoid(conv)).transpose(1, 2)               # [live, T, channels]
    at = keep[:, None] + torch.arange(R, device=keep.device)
    new_ring = torch.gather(window, 2, at[:, None, :].expand(-1, window.shape[1], -1))
    q = x[..., :Hk * D].reshape(live, T, Hk, D)
    k = x[..., Hk * D:2 * Hk * D].reshape(live, T, Hk, D)
    v = x[..., 2 * Hk * D:].reshape(live, T, H, Dv)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    head = torch.arange(H, device=q.device) % Hk
    q, k = q[:, :, head], k[:, :, head]
    rate = torch.exp(s["a_log"])
    if c["gdn"]:
        u = by_seq(s["f"]) + s["dt_bias"]
        g = -rate * (torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs())))
        decay = torch.exp(g)[..., None]                            # [live, T, H, 1]
    else:
        u = (by_seq(s["f"]) + s["dt_bias"]).reshape(live, T, H, D) * rate[:, None]
        decay = torch.exp(GATE_LB * torch.sigmoid(u))
    beta = torch.sigmoid(by_seq(s["beta"]))

    S = s["codes"][src].float() * s["scales"][src][..., None]      # [live, H, Dv, D]
    o = []
    for t in range(T):
        P = S * decay[:, t, :, None, :]
        u = v[:, t] - (P * k[:, t, :, None, :]).sum(-1)
        P = P + (beta[:, t, :, None] * u)[..., None] * k[:, t, :, None, :]
        S = torch.where((t < keep)[:, None, None, None], P, S)
        o.append((S * q[:, t, :, None, :]).sum(-1) * D ** -0.5)
    o = torch.stack(o, 1)                                          # [live, T, H, Dv]
    z = by_seq(s["z"]).reshape(live, T, H, Dv)
    gate = torch.sigmoid(z) * z if c["gdn"] else torch.sigmoid(z)
    y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + RMS_EPS) * s["norm_w"] * gate
    taken = (torch.arange(T, device=keep.device) < keep[:, None])[:, :, None]
    out = s["y"].reshape(N, T, -1)
    out[:live] = torch.where(taken, y.reshape(live, T, -1), out[:live])

    codes, scales = _plain_quantise(S)
    _bytes(s["codes"])[dst] = _bytes(codes)
    s["scales"][dst] = scales
    s["ring_pool"][dst] = new_ring
    return s["y"], s["codes"], s["scales"], s["ring_pool"]


def _own(s):
    from gated_delta_rule_scan_gb300 import kda, mixer
    c = s["case"]
    if c["kind"] == "proj":
        return mixer.kda_proj_w4(x=s["x"], weights=s["w"], scales=s["scales"], zeros=s["zeros"],
                                 group=c["group"], outs=s["outs"])
    if c["kind"] == "store":
        kda.kda_state_store_q8(s["state"], s["codes"], s["scales"], src=s["rows"],
                               dst=s["slots"], N=c["N"], H=c["H"], Dv=D * c["m"],
                               ring=s["ring"], ring_pool=s["ring_pool"])
        return s["codes"], s["scales"], s["ring_pool"]
    if c["kind"] == "load":
        kda.kda_state_load_q8(s["codes"], s["scales"], s["state"], src=s["slots"], dst=s["rows"],
                              N=c["N"], H=c["H"], Dv=D * c["m"], ring_pool=s["ring_pool"],
                              ring=s["ring"])
        return s["state"], s["ring"]
    mode = kda.GATE_PER_HEAD | kda.NORM_SILU if c["gdn"] else kda.GATE_PER_CHANNEL
    kda.kda_decode_fused_q8(s["q"], s["k"], s["v"], s["conv_w"], s["ring_pool"], s["f"],
                            s["dt_bias"], s["a_log"], s["beta"], s["codes"], s["scales"],
                            s["norm_w"], s["z"], s["y"], slots=s["slots"],
                            slots_out=s["slots_out"], keep=s["keep"], N=c["N"], T=c["T"],
                            H=c["H"], Hk=c["Hk"], Dv=D * c["m"], K=c["K"], gate_mode=mode,
                            gate_lb=GATE_LB, l2_eps=L2_EPS, rms_eps=RMS_EPS)
    return s["y"], s["codes"], s["scales"], s["ring_pool"]


def run(state):
    if own:
        return _own(state)
    return {"proj": _plain_proj, "store": _plain_store, "load": _plain_load,
            "decode": _plain_decode}[state["case"]["kind"]](state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without, and its exact outputs
# ------------------------------------------------------------------------------------------

def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    c = case
    if c["kind"] == "proj":
        rows, in_f = sum(_dims(c["H"])), c["in_f"]
        params = rows * (in_f // c["group"]) * _size(c["scale"]) * (2 if c["zeros"] else 1)
        return {"bytes": rows * in_f // 2 + params + c["t"] * (in_f * _size(c["x"]) + rows * 4),
                "flops": 2 * c["t"] * rows * in_f}
    N, H, Dv = c["N"], c["H"], D * c["m"]
    if c["kind"] in ("store", "load"):
        elems, ring = N * H * Dv * D, N * 3 * (2 * H * D + H * Dv)
        # the float and its code, a scale for each row of 128, the conv ring there and back
        return {"bytes": elems * 5 + elems // D * 4 + ring * 8 + N * 8,
                "flops": elems * (2 if c["kind"] == "store" else 1)}
    T, K, ch = c["T"], c["K"], _channels(c)
    live = N - c["pad"]
    elems, tokens = live * H * Dv * D, live * T
    return {"bytes": 2 * (elems + elems // D * 4 + live * ch * (K - 1) * 4)      # state and ring
            + tokens * (ch * _size(c["raw"]) + (H if c["gdn"] else H * D) * 4 + H * 4
                        + 2 * H * Dv * 4)                                         # rows in, y out
            + ch * K * 4 + (H if c["gdn"] else H * D) * 4 + (H + Dv + 3 * N) * 4,
            "flops": elems * T * 7}


def _exact_proj(s):
    group, x = s["case"]["group"], s["x"].double()
    out = []
    for i, w in enumerate(s["w"]):
        rows = w.shape[0]
        codes = torch.empty(rows, 2 * w.shape[1], dtype=torch.float64, device=w.device)
        codes[:, 0::2] = (w % 16).double()
        codes[:, 1::2] = torch.div(w, 16, rounding_mode="floor").double()
        codes -= (8.0 if s["zeros"] is None
                  else s["zeros"][i].double().repeat_interleave(group, dim=1))
        codes *= s["scales"][i].double().repeat_interleave(group, dim=1)
        out.append(torch.einsum("tk,rk->tr", x, codes))
    return out


def _exact_decode(s):
    """The recurrence with the state as [key, value] matrices; the codes stand for the state
    before its last rounding, over the row's scale."""
    c = s["case"]
    N, T, H, Hk, K, Dv = c["N"], c["T"], c["H"], c["Hk"], c["K"], D * c["m"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)
         and v.dtype not in (torch.int32, torch.int8)}
    live = N - c["pad"]
    slots, outs = s["slots"].tolist()[:live], s["slots_out"].tolist()[:live]
    keep = [T] * live if s["keep"] is None else s["keep"].tolist()[:live]
    most = max(keep, default=0)
    raw = torch.cat((d["q"], d["k"], d["v"]), 1).view(N, T, -1)[:live]
    ring = d["ring_pool"][slots]                                   # [live, channels, K - 1]
    S = (d["codes"][slots] * d["scales"][slots].unsqueeze(-1)).mT  # [live, H, D, Dv]
    kept = torch.tensor(keep, device=S.device)
    row = {k: d[k].view(N, T, -1)[:live] for k in ("f", "beta", "z")}
    group = [h % Hk for h in range(H)]
    for t in range(most):
        on = t < kept
        seen = torch.cat((ring, raw[:, t].unsqueeze(-1)), 2)
        x = torch.einsum("nck,ck->nc", seen, d["conv_w"])
        x = x / (1.0 + torch.exp(-x))
        qk, v = x[:, :2 * Hk * D].view(live, 2, Hk, D), x[:, 2 * Hk * D:].view(live, H, Dv)
        qk = qk * torch.rsqrt(qk.pow(2).sum(3, True) + L2_EPS)
        q, k = qk[:, 0, group], qk[:, 1, group]
        a = d["a_log"].exp()
        if c["gdn"]:
            decay = torch.exp(-a * torch.nn.functional.softplus(row["f"][:, t] + d["dt_bias"],
                                                                threshold=50.0))
            A = S * decay[:, :, None, None]
        else:
            pre = (row["f"][:, t] + d["dt_bias"]).view(live, H, D) * a.view(H, 1)
            A = S * torch.exp(GATE_LB / (1.0 + torch.exp(-pre))).unsqueeze(-1)
        u = v - torch.einsum("nhij,nhi->nhj", A, k)
        b = 1.0 / (1.0 + torch.exp(-row["beta"][:, t]))
        A = A + torch.einsum("nhi,nhj,nh->nhij", k, u, b)
        o = torch.einsum("nhij,nhi->nhj", A, q) / math.sqrt(D)
        z = row["z"][:, t].view(live, H, Dv)
        gate = 1.0 / (1.0 + torch.exp(-z)) * (z if c["gdn"] else 1.0)
        y = (o * torch.rsqrt(o.pow(2).mean(2, True) + RMS_EPS) * d["norm_w"] * gate)
        at = torch.arange(live, device=S.device)[on] * T + t
        d["y"][at] = y.reshape(live, -1)[on]
        S = torch.where(on.view(-1, 1, 1, 1), A, S)
        ring = torch.where(on.view(-1, 1, 1), seen[:, :, 1:], ring)
    scale = S.abs().amax(2) / E4M3_MAX                              # [live, H, Dv]
    d["codes"][outs] = (S / scale.unsqueeze(2)).mT
    d["scales"][outs] = scale
    d["ring_pool"][outs] = ring
    return d["y"], d["codes"], d["scales"], d["ring_pool"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "proj":
        return _exact_proj(s)
    slots, rows = s["slots"].tolist(), s["rows"].tolist() if "rows" in s else None
    if case["kind"] == "store":
        x = s["state"].double()[rows]
        scale = x.abs().amax(-1) / E4M3_MAX
        codes, scales, ring = (s[k].double() for k in ("codes", "scales", "ring_pool"))
        codes[slots], scales[slots] = x / scale.unsqueeze(-1), scale
        ring[slots] = s["ring"].double()[rows]
        return codes, scales, ring
    if case["kind"] == "load":
        state, ring = s["state"].double(), s["ring"].double()
        state[rows] = s["codes"].double()[slots] * s["scales"].double()[slots].unsqueeze(-1)
        ring[rows] = s["ring_pool"].double()[slots]
        return state, ring
    return _exact_decode(s)
