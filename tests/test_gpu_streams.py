"""GPU tests of calls on streams: calls that run on another stream than the current one and make
their own buffers (the current stream is kept busy meanwhile, so that work put on it would land after
the results), and launches that wait for a full queue."""

import threading
import time

import pytest
import torch

from gated_delta_rule_scan_gb300 import inputs

pytestmark = pytest.mark.gpu

BUSY = 200_000_000            # clock cycles: about a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def _batch(seed, N, T, H):
    i = inputs.make_inputs(seed, H=H, N=N, T=T, raw_dtype="f32", ring="randn", state="randn")
    d = {k: getattr(i, k).cuda() for k in ("q_raw", "k_raw", "v_raw", "conv_w", "ring_in", "f_raw",
                                           "dt_bias", "a_log", "beta_raw", "state_in", "norm_w",
                                           "gate_raw")}
    return d


def _handle(stream, as_int):
    return stream.cuda_stream if as_int else stream


@pytest.mark.parametrize("as_int", [False, True])
def test_pool_calls_beside_a_busy_stream(as_int):
    from gated_delta_rule_scan_gb300 import mixer
    N, H = 6, 4
    d = _batch(1, N, 1, H)
    pool = mixer.StatePoolQ8(2 * N, H, "cuda")
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    pool.store(d["state_in"], d["ring_in"], slots)
    rows = {k: v for k, v in d.items() if k not in ("state_in", "ring_in")}
    want = pool.decode(slots=slots, slots_out=slots + N, **rows)
    want_state, want_ring = pool.load(slots)
    out = slots + N
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    y = pool.decode(slots=slots, slots_out=out, stream=_handle(side, as_int), **rows)
    state, ring = pool.load(slots, stream=_handle(side, as_int))
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(state, want_state) and torch.equal(ring, want_ring)


def test_projections_on_two_streams_with_their_own_workspaces():
    """Each call drops its workspace on return, while its kernels still run."""
    from gated_delta_rule_scan_gb300 import mixer
    g = torch.Generator().manual_seed(3)
    jobs = []
    for t in (24, 40):
        jobs.append(dict(
            x=torch.randn(t, 2048, generator=g).cuda(),
            weights=[torch.randint(0, 256, (900, 1024), generator=g, dtype=torch.uint8).cuda()],
            scales=[torch.rand(900, 16, generator=g).cuda()], group=128))
    want = [mixer.kda_proj_w4(**j)[0] for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for j, s in zip(jobs, streams):
            got.append(mixer.kda_proj_w4(stream=s, **j)[0])
    torch.cuda.synchronize()
    for n, o in enumerate(got):
        assert torch.equal(o, want[n % 2])


def test_results_outlive_the_callers_work():
    """A result dropped while the current stream still reads it is not handed out to the next call
    on the side stream."""
    from gated_delta_rule_scan_gb300 import mixer
    N, H = 4, 4
    d = _batch(2, N, 1, H)
    pool = mixer.StatePoolQ8(N, H, "cuda")
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    pool.store(d["state_in"], d["ring_in"], slots)
    want, _ = pool.load(slots)
    side = torch.cuda.Stream()
    # (a kernel's first use loads its module, which may wait for the device)
    assert torch.full_like(want * 1.0, 9.0).all()
    torch.cuda.synchronize()
    state, ring = pool.load(slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = state * 1.0                         # reads it after the pause
    at = state.data_ptr()
    del state, ring
    others = []
    for _ in range(3):
        with torch.cuda.stream(side):
            others.append(torch.full_like(kept, 9.0))
    assert all(o.data_ptr() != at for o in others)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_f32_calls_beside_a_busy_stream():
    """Prefill, the staged mixer, decode and a rollback (whose untaken rows are zeros), each with
    buffers of its own."""
    from gated_delta_rule_scan_gb300 import mixer
    N, T, H = 2, 3, 2
    d = _batch(4, N, T, H)
    keep = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for call, extra in ((mixer.kda_prefill, {}), (mixer.kda_forward, {}), (mixer.kda_decode, {}),
                        (mixer.kda_verify_rollback, dict(keep=keep))):
        want = call(N=N, T=T, H=H, **d, **extra)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        got = [call(N=N, T=T, H=H, stream=side, **d, **extra) for _ in range(4)]
        torch.cuda.synchronize()
        for g in got:
            for k in ("y", "state_out", "ring_out"):
                assert torch.equal(g[k], want[k]), (call, k)


def test_a_full_queue_holds_up_no_other_thread():
    """More launches than a stream's queue takes behind a pause: the launching thread waits there,
    without the interpreter's lock."""
    from gated_delta_rule_scan_gb300 import mixer
    pool = mixer.StatePoolQ8(1, 1, "cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    state, ring = pool.load(slots)
    torch.cuda.synchronize()
    gap, stop = [0.0], threading.Event()

    def ticks():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0], last = max(gap[0], now - last), now
    t = threading.Thread(target=ticks)
    t.start()
    try:
        start = time.perf_counter()
        torch.cuda._sleep(8 * BUSY)            # 0.8 s
        for _ in range(6000):
            pool.load(slots, state=state, ring=ring)
        took = time.perf_counter() - start
        torch.cuda.synchronize()
    finally:
        stop.set()
        t.join()
    assert took > 0.5, took                    # (the queue was full)
    assert gap[0] < 0.25, (gap, took)
