"""GPU tests of kda_decode_fused_q8 on calls of 5 to 16 tokens, whose state stays in registers from
token to token, in all their forms, and of the readout's accuracy on ordinary inputs at any length.

Accuracy.  With M_j a bound of |S_j| that lets nothing cancel (M_j <- a M_j + beta (|v_j| + a M_j),
a the largest decay, from |S_j| on; k and q have length 1 at most), a readout o_j is formed from terms
of magnitude B_j = scale (a M_j + beta (|v_j| + a M_j)) in all, and is off by
  - the decays: their exponent, at most 5 in magnitude where it matters, is known to 2^-19 (hardware
    exponential and reciprocal, rate * (f + dt) in f32): 2^-19 B_j a token;
  - k, q and v: conv, SiLU and l2 norm, a few 2^-22 of each element: 2^-20 B_j;
  - sums of 128 terms, whose roundings are independent and at most 2^-24 of the sum of magnitudes'
    root of squares: 8 sqrt(128) 2^-24 B_j = 5.4e-6 B_j.
Together 2e-5 B_j up to 4 tokens and 5e-5 B_j up to 16.  (Not of |o_j|: a head whose state has decayed
by 1e-10 reads w_j (k . q), and where k . q is 3e-5 the rounding of k and q to f32 alone moves it by
6e-5 of itself.)  The RMSNorm takes an error d of o to at most |w g| inv (d_j + |o_j| inv rms(d)), and
the norm and its gate add 2^-20 of |y|.  The new state and y's contract: see test_gpu_decode_q8.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_decode_q8 import SHAPES, Work, _idx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def _free(w):
    return [s for s in range(w.P) if s not in w.slots][:w.N]


LONG = [
    dict(N=2, H=2, P=5), dict(N=3, H=3, P=7, fmt="e4m3", raw="f32", K=2),
    dict(N=2, H=4, P=6, Hk=2, fmt="e4m3"), dict(N=2, H=5, P=5, Hk=3, raw="f32", K=6),
    dict(N=2, H=2, P=5, Dv=256, gdn=True, norm_gate="silu"),
    dict(N=2, H=3, P=5, Hk=1, Dv=384, gdn=True, fmt="e4m3", raw="f32", K=8),
    dict(N=1, H=1, P=2, Dv=1024, K=3), dict(N=3, H=2, P=8, gdn=True, K=8),
    dict(N=2, H=2, P=4, Dv=256, Hk=1, fmt="e4m3"), dict(N=2, H=3, P=4, gdn=True, raw="f32", fmt="e4m3"),
    dict(N=2, H=2, P=4, Dv=256, gdn=True, fmt="e4m3"), dict(N=2, H=2, P=4, Dv=256, K=5),
]


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("T", [5, 9, 16])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_against_oracle(i, T, inplace):
    w = Work(700 + i, T=T, **LONG[i])
    out = w.slots if inplace else _free(w)
    if len(out) < w.N:
        pytest.skip("no free slots in this pool")
    y = w.decode(slots_out=None if inplace else _idx(out))
    w.check(y, out)
    w.others_untouched(out)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_prefixes(i, inplace):
    """keep takes 1 .. T rows, beyond T is clamped, and 0 or less passes the slot on."""
    T = 9
    w = Work(800 + i, T=T, **{**LONG[i], "N": 5, "P": 11})
    out = w.slots if inplace else _free(w)
    keep = [T - 1, T + 3, 1, 3, 6]
    took = [min(k, T) for k in keep]
    y = w.decode(slots_out=None if inplace else _idx(out), keep=_idx(keep))
    w.check(y, out, took)
    w.others_untouched(out)
    w.reset()
    y = w.decode(slots_out=None if inplace else _idx(out), keep=_idx([0, -2, T, 0, -2147483648]))
    assert (y[:2 * T] == 77.0).all() and (y[3 * T:] == 77.0).all() and (y[2 * T:3 * T] != 77.0).any()
    for n in (0, 1, 3, 4):
        for t, b in zip((w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring), w.before):
            assert torch.equal(t[out[n]], b[w.slots[n]])


@pytest.mark.parametrize("i", [0, 3, 5, 10])
def test_a_prefix_is_a_shorter_long_call(i):
    """Of calls of more than 4 tokens, bit for bit, and whatever else is in the batch."""
    w = Work(900 + i, T=12, **{**LONG[i], "N": 3, "P": 7})
    out = _free(w)
    y = w.decode(slots_out=_idx(out), keep=_idx([5, 12, 8]))
    got = [t[out].clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    for n, t in enumerate([5, 12, 8]):
        w.reset()
        yn = w.decode(slots=[w.slots[n]], rows=[n], T=t)
        assert torch.equal(y[12 * n:12 * n + t], yn)
        for g, x in zip(got, (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)):
            assert torch.equal(g[n], x[w.slots[n]])


@pytest.mark.parametrize("T", [7, 16])
def test_non_finite_samples_and_states_stay_in_their_heads(T):
    w = Work(13, N=3, T=T, H=3, P=3, raw="f32", Hk=3)
    clean = w.decode()
    after = w.pool.scales.clone()
    w.reset()
    w.inp.k_raw[T, 128 + 7] = float("nan")                # sequence 1, head 1
    w.pool.scales[w.slots[2], 2, 5] = float("inf")
    y = w.decode()
    for n in range(3):
        for h in range(3):
            a = y[n * T:(n + 1) * T, h * 128:(h + 1) * 128]
            b = clean[n * T:(n + 1) * T, h * 128:(h + 1) * 128]
            if (n, h) in ((1, 1), (2, 2)):
                assert not torch.isfinite(a[0]).all()
            else:
                assert torch.equal(a, b)
                assert torch.equal(w.pool.scales[w.slots[n], h], after[w.slots[n], h])


def _bounds(w, ref, tol):
    """What each element of y may be off by, [rows, H, Dv]."""
    i, N, T, H = w.inp, w.N, w.T, w.H
    Hk = i.Hk or H
    rows = N * T
    v = np.abs(ref["v_hat"]).reshape(rows, H, -1)
    Dv = v.shape[-1]
    a = np.exp(ref["g"]).reshape(rows, H, -1).max(-1)
    beta = np.asarray(ref["beta"]).reshape(rows, H)
    codes = w.before[0].view(w.pool.codes.dtype)
    S = (codes[w.slots].float() * w.before[1][w.slots][..., None]).double().cpu().numpy()
    M = np.sqrt((S ** 2).sum(-1)).reshape(N, H, Dv)
    assert Hk <= H and (np.asarray(ref["k_hat"]).reshape(rows, Hk, 128) ** 2).sum(-1).max() <= 1 + 1e-9
    z = i.gate_raw.double().numpy().reshape(rows, H, Dv)
    gate = 1 / (1 + np.exp(-z)) * (z if w.norm_gate == "silu" else 1.0)
    gate = np.abs(gate * i.norm_w.double().numpy())
    o = np.abs(np.asarray(ref["o"])).reshape(rows, H, Dv)
    inv = 1 / np.sqrt((o ** 2).mean(-1, keepdims=True) + 1e-6)
    out = np.empty((rows, H, Dv))
    for n in range(N):
        m = M[n]
        for t in range(T):
            r = n * T + t
            old = a[r][:, None] * m
            m = old + beta[r][:, None] * (v[r] + old)
            d = tol * 128 ** -0.5 * m
            rms = np.sqrt((d ** 2).mean(-1, keepdims=True))
            out[r] = gate[r] * inv[r] * (d + o[r] * inv[r] * rms) + 2.0 ** -20 * gate[r] * inv[r] * o[r]
    return out


@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 16])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_accuracy_on_ordinary_inputs(i, T):
    w = Work(1000 + i, **{**SHAPES[i], "T": T})
    y = w.decode()
    at, ref = w.oracle()
    got = y[at].double().cpu().numpy().reshape(len(at), w.H, -1)
    want = np.asarray(ref["y"]).reshape(got.shape)
    over = np.abs(got - want) / _bounds(w, ref, 2e-5 if T <= 4 else 5e-5)
    assert over.max() <= 1, over.max()
