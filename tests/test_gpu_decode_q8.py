"""GPU tests of kda_decode_fused_q8: decode, verify and rollback on the 8-bit state pool, against
the f64 oracle run from the pool's own values.

Tolerances.  A column's state S_j, its dot products with the unit vectors k and q and its update are
f32: 128-term sums carry at most 130 * 2^-24 |S_j| |k| each, with |S_j| <= sqrt(128) amax, so a token
adds at most three of those, 2.7e-4 of the row's amax, to a state element and (relative to typical
readouts, |S_j| / sqrt(128)) to the readout.  y: the repository's parity contract, 1e-3 of the
largest |y|, covers the four tokens run here.  The state out: the same times T, plus the rounding to
8 bits: half a step, amax / 254 (int8), or 2^-4 of the element and amax 2^-10 / 448 (e4m3).
"""

import numpy as np
import pytest
import torch

from gated_delta_rule_scan_gb300 import inputs
from tests.gpu_util import TOL, rel_linf

pytestmark = pytest.mark.gpu

D = 128
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def _idx(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(codes, scales, slots):
    """The pool's state rows as f32, on the CPU."""
    c = codes.view(torch.uint8)[slots].view(codes.dtype).float()
    return (c * scales[slots][..., None]).cpu()


class Work:
    """A seeded batch and a pool whose slots hold its states (stored by the library)."""

    def __init__(self, seed, N, T, H, P, *, Hk=None, Dv=None, gdn=False, raw="bf16", K=4,
                 fmt="int8", norm_gate="sigmoid", slots=None):
        from gated_delta_rule_scan_gb300 import mixer
        self.N, self.T, self.H, self.P, self.gdn = N, T, H, P, gdn
        self.norm_gate = norm_gate
        self.inp = inputs.make_inputs(seed, H=H, N=N, T=T, K=K, raw_dtype=raw, ring="randn",
                                      gate_mode=int(gdn), state="randn", Hk=Hk, Dv=Dv)
        self.pool = mixer.StatePoolQ8(P, H, "cuda", Hk=Hk, Dv=Dv, K=K, fmt=fmt)
        self.pool.codes.view(torch.uint8).fill_(0x2a)
        self.pool.scales.fill_(0.5)
        self.pool.ring.fill_(4.0)
        rng = np.random.default_rng(seed)
        self.slots = rng.permutation(P)[:N].tolist() if slots is None else slots
        self.pool.store(self.inp.state_in.cuda(), self.inp.ring_in.cuda(), _idx(self.slots))
        self.before = [t.clone() for t in (self.pool.codes.view(torch.uint8), self.pool.scales,
                                           self.pool.ring)]

    def reset(self):
        for t, b in zip((self.pool.codes.view(torch.uint8), self.pool.scales, self.pool.ring),
                        self.before):
            t.copy_(b)

    def rows(self, rows=None, T=None):
        """The batch's device arrays (of the listed sequences, of their first T tokens)."""
        rows = range(self.N) if rows is None else rows
        T = self.T if T is None else T
        at = torch.tensor([n * self.T + t for n in rows for t in range(T)], dtype=torch.long)
        d = {k: getattr(self.inp, k).cuda() for k in ("conv_w", "dt_bias", "a_log", "norm_w")}
        for k in ("q_raw", "k_raw", "v_raw", "f_raw", "beta_raw", "gate_raw"):
            d[k] = getattr(self.inp, k)[at].cuda().contiguous()
        return d

    def decode(self, slots=None, rows=None, T=None, **kw):
        n = len(range(self.N) if rows is None else rows)
        T = self.T if T is None else T
        y = torch.full((n * T, self.inp.C), 77.0, device="cuda")
        slots = self.slots if slots is None else slots
        self.pool.decode(slots=_idx(slots), T=T, y=y, gate_mode=int(self.gdn),
                         norm_gate=self.norm_gate, **self.rows(rows, T), **kw)
        torch.cuda.synchronize()
        return y

    def oracle(self, keep=None):
        """y rows taken (in order), state and ring in f64, from the pool's values before the call."""
        from oracle import oracle as orc
        keep = [self.T] * self.N if keep is None else keep
        at = [n * self.T + t for n in range(self.N) for t in range(keep[n])]
        i = self.inp
        codes = self.before[0].view(self.pool.codes.dtype)
        ref = orc.forward(
            q_raw=i.q_raw[at], k_raw=i.k_raw[at], v_raw=i.v_raw[at], f_raw=i.f_raw[at],
            dt_bias=i.dt_bias, a_log=i.a_log, beta_raw=i.beta_raw[at],
            state_in=_values(codes, self.before[1], self.slots), H=self.H, D=D, conv_w=i.conv_w,
            ring_in=i.ring_in, cu_seqlens=np.concatenate(([0], np.cumsum(keep))).astype(np.int64),
            gate_mode=int(self.gdn), norm_w=i.norm_w, gate_raw=i.gate_raw[at],
            norm_gate=self.norm_gate, Hk=i.Hk, Dv=i.Dv)
        return at, ref

    def check(self, y, slots_out, keep=None):
        at, ref = self.oracle(keep)
        assert rel_linf(y[at], ref["y"]) <= TOL
        rest = sorted(set(range(self.N * self.T)) - set(at))
        assert (y[rest] == 77.0).all()
        got = _values(self.pool.codes, self.pool.scales, slots_out).double().numpy()
        want = ref["state_out"].reshape(got.shape)
        amax = np.abs(want).max(-1, keepdims=True)
        tol = 2.7e-4 * self.T * amax
        if self.pool.codes.dtype == torch.int8:
            tol = tol + amax / 254
        else:
            tol = tol + np.maximum(np.abs(want) / 16, amax * 2.0 ** -10 / 448)
        assert (np.abs(got - want) <= tol * 1.001).all()
        assert np.array_equal(self.pool.ring[slots_out].cpu().numpy(),
                              ref["ring_out"].astype(np.float32))

    def others_untouched(self, written):
        rest = [s for s in range(self.P) if s not in set(written)]
        for t, b in zip((self.pool.codes.view(torch.uint8), self.pool.scales, self.pool.ring),
                        self.before):
            assert torch.equal(t[rest], b[rest])


SHAPES = [
    dict(N=3, T=1, H=2, P=3), dict(N=5, T=4, H=3, P=11, fmt="e4m3"),
    dict(N=2, T=3, H=4, P=6, Hk=2, raw="f32"), dict(N=3, T=2, H=5, P=7, Hk=3, fmt="e4m3", K=2),
    dict(N=2, T=2, H=2, P=5, Dv=256, gdn=True, norm_gate="silu"),
    dict(N=2, T=4, H=3, P=4, Hk=1, Dv=384, gdn=True, fmt="e4m3", raw="f32", K=6),
    dict(N=1, T=1, H=1, P=2, Dv=1024, K=8), dict(N=4, T=2, H=2, P=9, gdn=True, K=3),
]


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_against_oracle(i, inplace):
    w = Work(100 + i, **SHAPES[i])
    if inplace:
        y = w.decode()
        w.check(y, w.slots)
        w.others_untouched(w.slots)
    else:
        free = [s for s in range(w.P) if s not in w.slots][:w.N]
        if len(free) < w.N:
            pytest.skip("no free slots in this pool")
        y = w.decode(slots_out=_idx(free))
        w.check(y, free)
        w.others_untouched(free)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_longest_verify(fmt):
    """T = 16, the longest call: y against the oracle to the contract's bound."""
    w = Work(7, N=2, T=16, H=2, P=4, fmt=fmt)
    at, ref = w.oracle()
    assert rel_linf(w.decode(), ref["y"]) <= TOL


@pytest.mark.parametrize("i", [1, 3, 4, 5])
def test_keep_equals_a_shorter_call(i):
    """keep[n] rows give, bit for bit, what a call with only those rows gives; 0 copies the slot;
    values outside 0 .. T are clamped."""
    w = Work(200 + i, **{**SHAPES[i], "N": 4, "P": 9})
    T = w.T
    keep = [0, T + 3, -2, max(1, T - 1)]
    took = [min(max(k, 0), T) for k in keep]
    out = [s for s in range(w.P) if s not in w.slots][:4]
    y = w.decode(slots_out=_idx(out), keep=_idx(keep))
    w.check(y, out, took) if all(took) else None
    got = [t[out].clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    w.others_untouched(out)
    for n in range(4):
        w.reset()
        if took[n] == 0:
            want = [b[w.slots[n]] for b in w.before]
        else:
            yn = w.decode(slots=[w.slots[n]], rows=[n], T=took[n])
            want = [t[w.slots[n]] for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
            assert torch.equal(y[n * T:n * T + took[n]], yn)
        assert (y[n * T + took[n]:(n + 1) * T] == 77.0).all()
        assert all(torch.equal(g[n], x) for g, x in zip(got, want))
    # in place, nothing kept: untouched
    w.reset()
    w.decode(keep=_idx([0] * 4))
    w.others_untouched([])


@pytest.mark.parametrize("i", [0, 2, 4])
def test_rows_do_not_depend_on_the_batch(i):
    w = Work(300 + i, **{**SHAPES[i], "N": 3, "P": 8})
    y = w.decode()
    full = [t[w.slots].clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    for n in range(3):
        w.reset()
        yn = w.decode(slots=[w.slots[n]], rows=[n])
        assert torch.equal(yn, y[n * w.T:(n + 1) * w.T])
        for t, f in zip((w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring), full):
            assert torch.equal(t[w.slots[n]], f[n])


def test_padding_conflicts_and_bad_slots():
    from gated_delta_rule_scan_gb300 import kda
    w = Work(8, N=6, T=2, H=2, P=12, slots=[0, 1, 2, 3, 4, 5])
    good = w.decode(slots_out=_idx([6, 7, 8, 9, 10, 11]))
    want = [t.clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    assert kda.kda_device_status() == 0
    T = w.T

    def run(slots, out, live):
        """live: {row: slot written}; every other row and slot stays as it was."""
        w.reset()
        y = w.decode(slots=slots, slots_out=_idx(out))
        for n in range(6):
            rows = y[n * T:(n + 1) * T]
            assert torch.equal(rows, good[n * T:(n + 1) * T]) if n in live else (rows == 77.0).all()
        for n, s in live.items():
            for t, f in zip((w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring), want):
                assert torch.equal(t[s], f[6 + n])
        w.others_untouched(list(live.values()))
        return kda.kda_device_status()
    # padding in either array
    assert run([0, -1, 2, 3, -5, 5], [6, 7, -1, 9, 10, 11], {0: 6, 3: 9, 5: 11}) == 0
    # outside the pool
    assert run([0, 12, 2, 3, 4, 5], [6, 7, 8, 2147483647, 10, 11], {0: 6, 2: 8, 4: 10, 5: 11}) == 40013
    # rows 1 and 4 write slot 7: the first has it
    assert run([0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 7, 11], {0: 6, 1: 7, 2: 8, 3: 9, 5: 11}) == 40013
    # row 2 would write slot 3, which row 3 reads
    assert run([0, 1, 2, 3, 4, 5], [6, 7, 3, 9, 10, 11], {0: 6, 1: 7, 3: 9, 4: 10, 5: 11}) == 40013
    # one slot twice in place: both left out
    w.reset()
    y = w.decode(slots=[0, 1, 2, 1, 4, 5])
    assert (y[2:4] == 77.0).all() and (y[6:8] == 77.0).all() and kda.kda_device_status() == 40013
    w.others_untouched([0, 2, 4, 5])
    # a shared prefix: two rows read slot 0 and write their own
    w.reset()
    w.decode(slots=[0, 0, 2, 3, 4, 5], slots_out=_idx([6, 7, 8, 9, 10, 11]))
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("T", [1, 6])
def test_conflicts_among_many_rows(T):
    """More rows than a block has threads: conflicts with rows far behind are found all the same."""
    from gated_delta_rule_scan_gb300 import kda
    N = 300
    w = Work(12, N=N, T=T, H=1, P=2 * N + 1, slots=list(range(N)))
    out = list(range(N, 2 * N))
    good = w.decode(slots_out=_idx(out))
    want = [t.clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    w.reset()
    out[290] = out[5]                          # row 5 has it
    out[131] = 299                             # row 299 reads it
    out[260] = 2 * N + 1                       # past the pool
    slots = list(range(N))
    slots[200] = -3                            # padding
    y = w.decode(slots=slots, slots_out=_idx(out))
    gone = {290, 131, 260, 200}
    for n in range(N):
        rows = y[n * T:(n + 1) * T]
        assert (rows == 77.0).all() if n in gone else torch.equal(rows, good[n * T:(n + 1) * T])
    left = [out[n] for n in range(N) if n not in gone]
    for t, f in zip((w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring), want):
        assert torch.equal(t[left], f[left])
    w.others_untouched(left)
    assert kda.kda_device_status() == 40013


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("raw", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
def test_every_short_length(T, raw, fmt):
    w = Work(400 + T, N=3, T=T, H=3, P=4, raw=raw, fmt=fmt)
    y = w.decode()
    w.check(y, w.slots)
    w.others_untouched(w.slots)


@pytest.mark.parametrize("T", [1, 4])
def test_decays_beyond_one(T):
    """A positive gate bound (decays up to e^2 a token): against kda_decode_fused from the pool's
    values."""
    from gated_delta_rule_scan_gb300 import mixer
    w = Work(500 + T, N=2, T=T, H=2, P=3)
    state, ring = w.pool.load(_idx(w.slots))
    ref = mixer.kda_decode(state_in=state, ring_in=ring, N=2, T=T, H=2, gate_lb=2.0, **w.rows())
    y = w.decode(gate_lb=2.0)
    assert rel_linf(y, ref["y"].double().cpu().numpy()) <= TOL
    got, _ = w.pool.load(_idx(w.slots))
    want = ref["state_out"].reshape(got.shape)
    amax = want.abs().amax(-1, keepdim=True)
    assert ((got - want).abs() <= amax * (1 / 254 + 2.7e-4 * T) * 1.001).all()


def test_non_finite_state_stays_in_its_head():
    w = Work(9, N=2, T=1, H=2, P=2)
    clean = w.decode()
    w.reset()
    w.pool.scales[w.slots[0], 1, 5] = float("nan")
    y = w.decode()
    assert torch.isnan(y[0, 128:]).all()                  # that head's RMSNorm row
    assert torch.equal(y[0, :128], clean[0, :128]) and torch.equal(y[1], clean[1])
    assert torch.isnan(w.pool.scales[w.slots[0], 1, 5])
    assert int(torch.isnan(w.pool.scales).sum()) == 1


def test_graph_replay_and_other_stream():
    """A step captured on a side stream and replayed equals the same steps launched eagerly."""
    w = Work(10, N=3, T=1, H=4, P=5, Hk=2)
    d, slots = w.rows(), _idx(w.slots)
    y = torch.zeros(3, w.inp.C, device="cuda")
    eager = []
    for _ in range(3):
        w.pool.decode(slots=slots, y=y, **d)
        eager.append(y.clone())
    after = w.pool.codes.view(torch.uint8).clone()
    w.reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w.pool.decode(slots=slots, y=y, **d)
    w.reset()
    for e in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, e)
    assert torch.equal(w.pool.codes.view(torch.uint8), after)
    w.reset()
    side.wait_stream(torch.cuda.current_stream())
    w.pool.decode(slots=slots, y=y, stream=side, **d)
    side.synchronize()
    assert torch.equal(y, eager[0])


@pytest.mark.parametrize("T", [1, 3, 4])
def test_non_finite_samples_stay_in_their_heads(T):
    """A NaN in a token's k and an infinity in another row's v reach their own heads' rows only."""
    w = Work(13, N=3, T=T, H=3, P=3, raw="f32")
    clean = w.decode()
    after = w.pool.scales.clone()
    w.reset()
    w.inp.k_raw[0 * T, 128 + 7] = float("nan")            # row 0, head 1
    w.inp.v_raw[2 * T, 256 + 9] = float("inf")            # row 2, head 2
    y = w.decode()
    hit = torch.zeros(3, 3, dtype=torch.bool)
    hit[0, 1] = hit[2, 2] = True
    for n in range(3):
        for h in range(3):
            a = y[n * T:(n + 1) * T, h * D:(h + 1) * D]
            b = clean[n * T:(n + 1) * T, h * D:(h + 1) * D]
            if hit[n, h]:
                assert not torch.isfinite(a[0]).all()
            else:
                assert torch.equal(a, b)
                assert torch.equal(w.pool.scales[w.slots[n], h], after[w.slots[n], h])
    assert torch.isnan(w.pool.scales[w.slots[0], 1]).all()
    assert torch.isnan(w.pool.scales[w.slots[2], 2, 9])


def test_calls_at_once_on_two_streams():
    """Decode steps of two pools and projections of two sizes, on two streams at the same time."""
    from gated_delta_rule_scan_gb300 import kda, mixer
    jobs = []
    for i, (T, t) in enumerate([(1, 3), (3, 24)]):
        w = Work(600 + i, N=8, T=T, H=16, P=8, Hk=4, gdn=bool(i))
        g = torch.Generator().manual_seed(i)
        w4 = torch.randint(0, 256, (700, 1024), generator=g, dtype=torch.uint8).cuda()
        sc = torch.rand(700, 2048 // 64, generator=g).cuda()
        x = torch.randn(t, 2048, generator=g).cuda()
        jobs.append(dict(w=w, d=w.rows(), slots=_idx(w.slots), w4=w4, sc=sc, x=x,
                         y=torch.zeros(8 * T, w.inp.C, device="cuda"),
                         out=torch.zeros(t, 700, device="cuda"),
                         ws=kda.proj_w4_workspace(t, 2048, "cuda"), s=torch.cuda.Stream()))

    def step(j, stream):
        w = j["w"]
        w.pool.decode(slots=j["slots"], T=w.T, y=j["y"], gate_mode=int(w.gdn), stream=stream, **j["d"])
        kda.kda_proj_w4(j["x"], [j["w4"]], [j["sc"]], [j["out"]], group=64, workspace=j["ws"],
                        stream=stream)
    want = []
    for j in jobs:
        for _ in range(6):
            step(j, None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (j["y"], j["out"], j["w"].pool.codes.view(torch.uint8),
                                         j["w"].pool.ring)])
        j["w"].reset()
    torch.cuda.synchronize()
    for _ in range(6):
        for j in jobs:
            step(j, j["s"])
    torch.cuda.synchronize()
    for j, f in zip(jobs, want):
        for a, b in zip((j["y"], j["out"], j["w"].pool.codes.view(torch.uint8), j["w"].pool.ring), f):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A slot whose code offset passes 2^32."""
    H, P = 64, 4100
    w = Work(11, N=1, T=1, H=H, P=P, slots=[4098])
    y = w.decode(slots_out=_idx([4099]))
    w.check(y, [4099])


def test_a_sequence_through_the_operators():
    """Prefill in f32, its state and ring into the pool, decode steps whose q, k, v and beta come
    from 4-bit projections, a verify rolled back to its accepted prefix, and the state back to f32:
    each step against the oracle from the pool's values before it."""
    from gated_delta_rule_scan_gb300 import mixer
    from oracle import oracle as orc
    H, N, in_f, G = 2, 3, 256, 64
    C = H * D
    pre = inputs.make_inputs(20, H=H, N=N, T=24, raw_dtype="f32", ring="randn", state="randn")
    d = {k: getattr(pre, k).cuda() for k in ("q_raw", "k_raw", "v_raw", "conv_w", "ring_in", "f_raw",
                                             "dt_bias", "a_log", "beta_raw", "state_in", "norm_w",
                                             "gate_raw")}
    out = mixer.kda_prefill(H=H, N=N, T=24, **d)
    pool = mixer.StatePoolQ8(8, H, "cuda", fmt="int8")
    slots = _idx([6, 1, 3])
    pool.store(out["state_out"], out["ring_out"], slots)
    g = torch.Generator().manual_seed(21)
    dims = (C, C, C, D, D, H)
    w4 = [torch.randint(0, 256, (r, in_f // 2), generator=g, dtype=torch.uint8) for r in dims]
    sc = [(0.2 + torch.rand(r, in_f // G, generator=g)) / in_f ** 0.5 for r in dims]
    wf = [(torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1).double() - 8)
          * s.double().repeat_interleave(G, 1) for w, s in zip(w4, sc)]
    weights = dict(conv_w=d["conv_w"], dt_bias=d["dt_bias"], a_log=d["a_log"], norm_w=d["norm_w"])

    def step(T, at_in, at_out, keep=None):
        x = torch.randn(N * T, in_f, generator=g)
        f, z = torch.randn(N * T, C, generator=g), torch.randn(N * T, C, generator=g)
        q, k, v, _, _, b = mixer.kda_proj_w4(x=x.cuda(), weights=[w.cuda() for w in w4],
                                             scales=[s.cuda() for s in sc], group=G)
        S = _values(pool.codes, pool.scales, at_in.long())
        ring = pool.ring[at_in.long()].cpu()
        kd = None if keep is None else _idx(keep)
        y = pool.decode(q_raw=q, k_raw=k, v_raw=v, beta_raw=b, f_raw=f.cuda(), gate_raw=z.cuda(),
                        slots=at_in, slots_out=at_out, T=T, keep=kd, **weights)
        keep = [T] * N if keep is None else keep
        at = [n * T + t for n in range(N) for t in range(keep[n])]
        rq, rk, rv, rb = (x.double() @ wf[i].T for i in (0, 1, 2, 5))
        ref = orc.forward(q_raw=rq[at], k_raw=rk[at], v_raw=rv[at], beta_raw=rb[at], f_raw=f[at],
                          dt_bias=pre.dt_bias, a_log=pre.a_log, state_in=S, H=H, D=D,
                          conv_w=pre.conv_w, ring_in=ring, norm_w=pre.norm_w, gate_raw=z[at],
                          cu_seqlens=np.concatenate(([0], np.cumsum(keep))).astype(np.int64))
        assert rel_linf(y[at], ref["y"]) <= TOL
        to = (at_in if at_out is None else at_out).long()
        got = _values(pool.codes, pool.scales, to).double().numpy()
        want = ref["state_out"].reshape(got.shape)
        amax = np.abs(want).max(-1, keepdims=True)
        assert (np.abs(got - want) <= amax * (1 / 254 + 2.7e-4 * T + 1e-3)).all()
        return ref
    for _ in range(2):
        step(1, slots, None)                               # decode in place
    other = _idx([0, 2, 4])
    step(4, slots, other)                                  # verify, beside the states before it
    ref = step(4, slots, other, keep=[2, 4, 1])            # a round rolled back to its prefixes
    state, ring = pool.load(other)
    amax = np.abs(ref["state_out"]).max(-1, keepdims=True)
    err = np.abs(state.cpu().double().numpy() - ref["state_out"].reshape(state.shape))
    assert (err <= amax.reshape(N, H, D, 1) * (1 / 254 + 2.1e-3)).all()
    assert torch.equal(ring, pool.ring[other.long()])


def test_refusals_on_device():
    from gated_delta_rule_scan_gb300 import kda
    w = Work(12, N=2, T=1, H=2, P=3)
    d, p = w.rows(), w.pool
    y = torch.full((2, 256), 77.0, device="cuda")

    def call(**bad):
        a = dict(d, codes=p.codes, scales=p.scales, ring=p.ring, y=y, slots=_idx(w.slots), N=2, T=1,
                 H=2, K=4, Hk=None, slots_out=None, keep=None)
        a.update(bad)
        kda.kda_decode_fused_q8(a["q_raw"], a["k_raw"], a["v_raw"], a["conv_w"], a["ring"], a["f_raw"],
                                a["dt_bias"], a["a_log"], a["beta_raw"], a["codes"], a["scales"],
                                a["norm_w"], a["gate_raw"], a["y"], slots=a["slots"],
                                slots_out=a["slots_out"], keep=a["keep"], N=a["N"], T=a["T"],
                                H=a["H"], K=a["K"], Hk=a["Hk"])
    for bad in (dict(N=3), dict(T=2), dict(H=4), dict(Hk=1), dict(K=5), dict(y=y[:1]),
                dict(q_raw=d["q_raw"].float()), dict(q_raw=d["q_raw"].half()),
                dict(slots=w.slots), dict(slots=torch.tensor(w.slots, device="cuda")),
                dict(keep=torch.ones(2, device="cuda")), dict(codes=p.codes.float()),
                dict(codes=p.codes[:2]), dict(gate_raw=d["gate_raw"].cpu()),
                dict(f_raw=torch.zeros(512, 2, device="cuda").t()[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(kda.KdaError) as e:                 # Hk > H
        call(Hk=3, q_raw=torch.zeros(2, 384, device="cuda"), k_raw=torch.zeros(2, 384, device="cuda"),
             v_raw=torch.zeros(2, 256, device="cuda"), conv_w=torch.zeros(1024, 4, device="cuda"),
             ring=torch.zeros(3, 1024, 3, device="cuda"))
    assert e.value.status == 40005
    assert (y == 77.0).all()
    w.others_untouched([])


@pytest.mark.parametrize("T", [2, 6])
def test_a_row_left_out_claims_no_slot(T):
    """Rows with a slot past the pool, or of padding, read and write nothing: others may write the
    slots that they name."""
    from gated_delta_rule_scan_gb300 import kda
    w = Work(14, N=6, T=T, H=2, P=12, slots=[0, 1, 2, 3, 4, 5])
    good = w.decode(slots_out=_idx([6, 7, 8, 9, 10, 11]))
    want = [t.clone() for t in (w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring)]
    w.reset()
    # row 0's source and row 2's target are outside; rows 1 and 3 write what those name
    y = w.decode(slots=[12, 1, 8, 3, -1, 5], slots_out=_idx([7, 7, 12, 8, 11, 11]))
    assert kda.kda_device_status() == 40013
    for n in range(6):
        rows = y[n * T:(n + 1) * T]
        assert torch.equal(rows, good[n * T:(n + 1) * T]) if n in (1, 3, 5) else (rows == 77.0).all()
    for slot, n in ((7, 1), (8, 3), (11, 5)):
        for t, f in zip((w.pool.codes.view(torch.uint8), w.pool.scales, w.pool.ring), want):
            assert torch.equal(t[slot], f[6 + n])
    w.others_untouched([7, 8, 11])
