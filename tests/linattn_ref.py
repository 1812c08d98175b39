"""Plain 64-bit forms of linear attention with one log-decay a head, on the CPU: the outputs, and the
sums of magnitudes that error bounds are relative to."""

import numpy as np
import torch

D = 128


def recurrence(q, k, v, g, S, H, Hk, Dv, scale):
    """One sequence: q, k [T, Hk*128], v [T, H*Dv], g [H], S [H, Dv, 128].  Returns o [T, H*Dv] and
    the last state, in f64."""
    T = q.shape[0]
    head = torch.arange(H) % Hk
    q, k = (x.double().reshape(T, Hk, D)[:, head] for x in (q, k))
    v = v.double().reshape(T, H, Dv)
    lam = torch.exp(g.double())[:, None, None]
    S = S.double().clone()
    o = torch.empty(T, H, Dv, dtype=torch.float64)
    for t in range(T):
        S = lam * S + v[t, :, :, None] * k[t, :, None, :]
        o[t] = scale * torch.einsum("hji,hi->hj", S, q[t])
    return o.reshape(T, H * Dv), S


def both(q, k, v, g, S, H, Hk, Dv, scale):
    """(o, state) and the same recurrence of the inputs' magnitudes."""
    with np.errstate(all="ignore"):
        ref = recurrence(q, k, v, g, S, H, Hk, Dv, scale)
        mag = recurrence(q.abs(), k.abs(), v.abs(), g, S.abs(), H, Hk, Dv, abs(scale))
    return ref, mag
