"""GPU tests of kda_proj_w4 (projections by 4-bit weights with group scales) against the product in
64 bits.

Tolerance, element by element, for M = sum_k c (|q - 8| + |8 - z|) |x|, the sum of the magnitudes
that enter an output: x is held to 2^-22 of each element (f16 hi + lo; half a step of each is 2^-11);
a group's sum of G products is at most G additions of relative error 2^-23 each (a tensor core may
truncate); scale and power-of-two factor, zero-point term and their additions are 4 roundings of
2^-24 a group; the in_f / G groups, 8 warps and 8 blocks add in_f / G + 16 more of 2^-24:
    |error| <= M (2^-22 + G 2^-23 + (in_f / G + 20) 2^-24).
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def _case(seed, t, in_f, rows, group, x="f32", scale="bf16", zeros=False):
    g = torch.Generator().manual_seed(seed)
    dt = dict(f32=torch.float32, bf16=torch.bfloat16)
    xs = torch.randn(t, in_f, generator=g)
    xs[:, ::97] *= 30.0                       # outlier channels
    c = dict(x=xs.to(dt[x]), w=[], s=[], z=[] if zeros else None, group=group)
    for r in rows:
        c["w"].append(torch.randint(0, 256, (r, in_f // 2), generator=g, dtype=torch.uint8))
        c["s"].append(((0.1 + torch.rand(r, in_f // group, generator=g))
                       / in_f ** 0.5).to(dt[scale]))
        if zeros:
            c["z"].append((8 + 3 * torch.randn(r, in_f // group, generator=g)).to(dt[scale]))
    return c


def _reference(c):
    """(outputs, tolerances) in 64 bits."""
    x, G = c["x"].double(), c["group"]
    outs, tols = [], []
    for i, w in enumerate(c["w"]):
        q = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], 2 * w.shape[1]).double()
        s = c["s"][i].double().repeat_interleave(G, 1)
        z = 8.0 if c["z"] is None else c["z"][i].double().repeat_interleave(G, 1)
        outs.append(x @ ((q - z) * s).T)
        mag = x.abs() @ (((q - 8).abs() + abs(8 - z)) * s).T
        n = q.shape[1] // G
        tols.append(mag * (2.0 ** -22 + G * 2.0 ** -23 + (n + 20) * 2.0 ** -24))
    return outs, tols


def _gpu(c, dev="cuda", **kw):
    from gated_delta_rule_scan_gb300 import kda
    t, in_f = c["x"].shape
    outs = [torch.full((t, w.shape[0]), float("nan"), device=dev) for w in c["w"]]
    d = {k: None if c[k] is None else [v.to(dev) for v in c[k]] for k in ("w", "s", "z")}
    kda.kda_proj_w4(c["x"].to(dev), d["w"], d["s"], outs, group=c["group"], zeros=d["z"],
                    workspace=kda.proj_w4_workspace(t, in_f, dev), **kw)
    torch.cuda.synchronize()
    return outs


def _check(c, outs):
    refs, tols = _reference(c)
    for o, r, tol in zip(outs, refs, tols):
        bad = (o.cpu().double() - r).abs() > tol
        assert not bad.any(), (int(bad.sum()), float(((o.cpu().double() - r).abs() / tol).max()))


SIX = (256, 256, 256, 128, 128, 2)            # the layer's six projections at H = 2


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x,scale,zeros", [("f32", "bf16", False), ("f32", "f32", True),
                                           ("bf16", "bf16", True), ("bf16", "f32", False)])
@pytest.mark.parametrize("t", [1, 3, 4, 5, 8])
def test_small_batches(t, x, scale, zeros, group):
    c = _case(t * 31 + group, t, 384, SIX, group, x, scale, zeros)
    _check(c, _gpu(c))


@pytest.mark.parametrize("t,in_f,rows,group,x,zeros", [
    (9, 128, (1,), 128, "f32", False), (13, 640, (17, 300), 64, "bf16", True),
    (16, 256, SIX, 32, "f32", True), (17, 512, SIX, 128, "bf16", False),
    (33, 896, (130, 1, 63), 64, "f32", False), (64, 384, SIX, 128, "f32", False),
    (100, 256, (129,), 32, "bf16", True), (200, 1152, (33,), 128, "f32", True),
    (256, 256, SIX, 64, "f32", False), (256, 128, (5,), 32, "bf16", False)])
def test_large_batches(t, in_f, rows, group, x, zeros):
    c = _case(t + in_f, t, in_f, rows, group, x, "bf16", zeros)
    _check(c, _gpu(c))


@pytest.mark.parametrize("t,in_f,x", [(1, 32768, "f32"), (8, 16384, "f32"), (8, 20480, "bf16"),
                                      (5, 9984, "f32"), (20, 16384, "f32"), (16, 8192, "f32"),
                                      (11, 3968, "f32"), (16, 32768, "bf16"), (9, 32768, "f32")])
def test_wide_inputs(t, in_f, x):
    """x wider than one block's shared memory holds, with uneven shares of K."""
    c = _case(in_f + t, t, in_f, (40, 3), 128, x, "bf16", True)
    _check(c, _gpu(c))


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("t", [6, 9, 12, 15, 16])
def test_up_to_sixteen_rows(t, x, group, zeros):
    c = _case(t * 7 + group, t, 640, (200, 1, 16, 33), group, x, "f32" if group == 64 else "bf16", zeros)
    _check(c, _gpu(c))


@pytest.mark.parametrize("t,rows,x", [(13, 4096, "f32"), (9, 4112, "f32"), (16, 8192, "bf16")])
def test_few_rows_of_large_weights(t, rows, x):
    """Rows past which the form for batches is taken at this size."""
    c = _case(70 + t, t, 5120, (rows,), 128, x)
    _check(c, _gpu(c))


@pytest.mark.slow
@pytest.mark.parametrize("t", [1, 64])
def test_full_size(t):
    """The layer's projections at 64 heads, hidden 6144, one token and a decode batch."""
    c = _case(t, t, 6144, (8192, 8192, 8192, 128, 128, 64), 128)
    _check(c, _gpu(c))


def test_eight_weights_and_empty_ones():
    c = _case(3, 4, 256, (16, 0, 5, 128, 1, 0, 33, 7), 64)
    _check(c, _gpu(c))
    c = _case(4, 0, 256, (16,), 64)
    assert _gpu(c)[0].shape == (0, 16)


@pytest.mark.parametrize("t", [1, 6, 24])
def test_extreme_magnitudes(t):
    """Rows of x far from 1, zero chunks, and a wide range inside one chunk."""
    c = _case(40 + t, t, 512, (70,), 32, zeros=True)
    c["x"][:, :128] *= 1e30
    c["x"][:, 128:256] = 0.0
    c["x"][:, 256:384] *= 1e-20
    c["x"][0, 300] = 1e4
    _check(c, _gpu(c))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("t", [1, 4, 7, 20])
def test_groups_of_the_zero_point_are_zero(t, x):
    """Codes of 8 (and any codes at a scale of 0) add nothing, however large x is there."""
    c = _case(80 + t, t, 512, (70,), 64, x)
    c["w"][0][:, 64:192] = 0x88               # k = 128 .. 383
    c["x"][:, 128:384] *= 1000.0
    if t <= 4:                                # x is scaled by 128 k (beyond: by rows)
        with_them = _gpu(c)[0]
        c["x"][:, 128:384] = 0.0
        assert torch.equal(_gpu(c)[0], with_them)
    c["w"][0][:] = 0x88
    assert not _gpu(c)[0].any()


@pytest.mark.parametrize("outlier", [1e2, 1e4, 1e6])
@pytest.mark.parametrize("t", [2, 4])
def test_small_elements_beside_a_large_one(t, outlier):
    """A large element whose codes are 8 costs the others no more than 2^-25 of it each, and the
    f32 sums nothing: they are differences of exact sums."""
    c = _case(90 + t, t, 256, (48,), 128)
    c["x"][:, 17] = outlier
    c["w"][0][:, 8] = (c["w"][0][:, 8] & 15) | 0x80
    refs, tols = _reference(c)
    # |code - 8| <= 8, 128 k to a largest element; then lo's sums, below 2^-11 of the largest
    # element, in 10 steps of f32 each: 2^-11 * 15 * 128 * 10 * 2^-24
    s = c["s"][0].double()[:, 0]
    more = outlier * s * (128 * 8 * 2.0 ** -25 + 15 * 128 * 10 * 2.0 ** -35)
    out = _gpu(c)[0].cpu().double()
    own = _reference(dict(c, x=torch.where(c["x"].abs() >= outlier, 0.0, c["x"])))[1][0]
    assert ((out - refs[0]).abs() <= own + more).all()


@pytest.mark.parametrize("t", [3, 7, 40])
def test_non_finite_rows_stay_apart(t):
    c = _case(60 + t, t, 384, (50, 130), 64)
    clean = _gpu(c)
    c["x"][0, 5] = float("nan")
    c["x"][t - 1, 200] = float("inf")
    for o, k in zip(_gpu(c), clean):
        assert not torch.isfinite(o[0]).any() and not torch.isfinite(o[t - 1]).any()
        assert torch.equal(o[1:t - 1], k[1:t - 1])


@pytest.mark.parametrize("t", [1, 8, 64])
def test_repeatable(t):
    c = _case(70 + t, t, 1024, SIX, 128)
    a, b = _gpu(c), _gpu(c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [2, 48])
def test_graph_replay_on_another_stream(t):
    """Captured on a side stream and replayed with new x: outputs follow the inputs in place."""
    from gated_delta_rule_scan_gb300 import mixer
    c = _case(80, t, 512, SIX, 64)
    dev = torch.device("cuda")
    x = c["x"].to(dev)
    w, s = [v.to(dev) for v in c["w"]], [v.to(dev) for v in c["s"]]
    outs = mixer.kda_proj_w4(x=x, weights=w, scales=s, group=64)     # first call: attributes set
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mixer.kda_proj_w4(x=x, weights=w, scales=s, group=64, outs=outs)
    for seed in (81, 82):
        c["x"] = _case(seed, t, 512, (1,), 64)["x"]
        x.copy_(c["x"])
        graph.replay()
        torch.cuda.synchronize()
        _check(c, outs)


def test_refusals_on_device():
    from gated_delta_rule_scan_gb300 import kda
    c = _case(90, 2, 256, (16, 8), 64)
    dev = torch.device("cuda")
    x, w, s = c["x"].to(dev), [v.to(dev) for v in c["w"]], [v.to(dev) for v in c["s"]]
    outs = [torch.empty(2, 16, device=dev), torch.empty(2, 8, device=dev)]
    for bad in (dict(x=x.t().contiguous().t()), dict(w=[w[0][:, ::2], w[1]]), dict(w=[w[0]]),
                dict(s=[s[0].cpu(), s[1]]), dict(s=[s[0].float(), s[1]]), dict(outs=[outs[1], outs[0]]),
                dict(s=[s[0][:, :3].contiguous(), s[1]]), dict(x=x[0])):
        a = dict(x=x, w=w, s=s, outs=outs)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_proj_w4(a["x"], a["w"], a["s"], a["outs"], group=64)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_proj_w4(x, w, [v[:, :1].contiguous() for v in s], outs, group=256)
    assert e.value.status == 40007
    _check(c, _gpu(c))


def test_first_calls_of_many_threads():
    """Host threads whose calls want different amounts of shared memory of the same kernels, at once;
    the largest still launch afterwards."""
    import threading
    cases = [_case(500 + n, t, in_f, (130,), 128, x) for n, (t, in_f, x) in enumerate(
        [(1, 512, "f32"), (4, 9728, "f32"), (2, 19456, "f32"), (3, 128, "f32"), (5, 4864, "f32"),
         (7, 512, "f32"), (24, 512, "f32"), (64, 512, "f32"), (80, 256, "f32"), (128, 256, "f32")])]
    start, got, errors = threading.Barrier(len(cases)), [None] * len(cases), []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                got[n] = _gpu(cases[n])
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, o in zip(cases, got):
        _check(c, o)
    for c, o in zip(cases, got):
        assert all(torch.equal(a, b) for a, b in zip(_gpu(c), o))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x,zeros", [("f32", False), ("f32", True), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("t", [17, 24, 64, 65, 200])
def test_batches_by_f32_scales(t, x, zeros, group):
    c = _case(t * 13 + group, t, 384, (130, 1, 77), group, x, "f32", zeros)
    _check(c, _gpu(c))
