"""GPU tests of kda_decode_fused_q8 where little is left of the state: strong decays with a closed
beta (the old state is then all there is to read), and q rows far below unit length.

Tolerance: the repository's parity contract (1e-3), taken of the largest |y| of each token row and
head on its own, since a head's rows may be many orders apart.  The decays of a row multiply up to
e^-60 here, whose exponent, at most 60, is known to 2^-20 of itself in f32 by any route: 6e-5.
"""

import numpy as np
import pytest
import torch

from tests.gpu_util import TOL
from tests.test_gpu_decode_q8 import D, Work, _idx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def _faded(seed, T, gdn, f, q=1.0, **kw):
    """Work whose tokens have a closed beta, the gate input `f` (a number or (from, to)) and q rows
    of scale `q`.  Per head, a_log = 0 makes the log-decay -softplus(f); per channel, -5 sigmoid(f)."""
    w = Work(seed, N=3, T=T, H=2, P=7, gdn=gdn, raw="f32", slots=[5, 0, 2], **kw)
    i = w.inp
    i.a_log.zero_()
    i.dt_bias.zero_()
    i.beta_raw.fill_(-60.0)
    if isinstance(f, tuple):
        g = torch.Generator().manual_seed(seed)
        i.f_raw.copy_(f[0] + (f[1] - f[0]) * torch.rand(i.f_raw.shape, generator=g))
    else:
        i.f_raw.fill_(f)
    i.q_raw.mul_(q)
    if q != 1.0:
        w.pool.ring[:, :i.q_raw.shape[1]] *= q
        i.ring_in[:, :i.q_raw.shape[1]] *= q
        w.before[2].copy_(w.pool.ring)
    return w


def _check(w, y):
    at, ref = w.oracle()
    got = y[at].double().cpu().numpy().reshape(len(at), w.H, -1)
    want = np.asarray(ref["y"]).reshape(got.shape)
    top = np.abs(want).max(-1)
    assert (top > 1e-34).all()                          # (f32 holds what is compared)
    err = np.abs(got - want).max(-1) / top
    assert err.max() <= TOL, err


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T,f", [(1, 5.0), (1, 11.0), (1, 16.0), (1, 20.0), (1, 25.0), (1, 30.0),
                                 (2, 15.0), (3, 12.0), (4, 8.0), (4, 15.0), (6, 10.0)])
def test_strong_decay_per_head(T, f, fmt):
    w = _faded(int(f) + T, T, True, f, fmt=fmt)
    y = w.decode()
    _check(w, y)
    w.check(y, w.slots)


@pytest.mark.parametrize("f", [30.0, (0.0, 8.0), (-8.0, 8.0)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7])
def test_strong_decay_per_channel(T, f):
    w = _faded(40 + T, T, False, f)
    y = w.decode()
    _check(w, y)
    w.check(y, w.slots)


@pytest.mark.parametrize("gdn", [True, False])
def test_strong_decay_of_wide_heads(gdn):
    w = _faded(50 + gdn, 4, gdn, 14.0, Dv=256, fmt="e4m3")
    _check(w, w.decode())


@pytest.mark.parametrize("gdn", [True, False])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("q", [1e-6, 1e-9, 1e-12])
def test_short_queries(q, T, gdn):
    w = _faded(60 + T, T, gdn, (-2.0, 0.0), q=q)
    _check(w, w.decode())


def test_prefixes_of_a_faded_row_are_the_shorter_calls():
    """keep still equals a call of that many tokens bit for bit."""
    w = _faded(70, 4, False, (2.0, 9.0))
    out = [1, 3, 4]
    y = w.decode(slots_out=_idx(out), keep=_idx([1, 2, 3]))
    state = w.pool.codes.view(torch.uint8)[out].clone()
    for n, t in enumerate([1, 2, 3]):
        w.reset()
        yn = w.decode(slots=[w.slots[n]], rows=[n], T=t)
        assert torch.equal(y[4 * n:4 * n + t], yn) and yn.shape[1] == 2 * D
        assert torch.equal(w.pool.codes.view(torch.uint8)[w.slots[n]], state[n])
