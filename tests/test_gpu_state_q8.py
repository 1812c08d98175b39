"""GPU tests of the 8-bit state pool's store and load: the codes and scales are one exact function
of the f32 state (three f32 roundings a row and one a code), so they are compared bit for bit with
the same arithmetic in numpy, and the values read back with code * scale in f32."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    from gated_delta_rule_scan_gb300 import kda
    assert kda.kda_device_status() == 0


def quantise(x, fmt):
    """(codes as bytes, scales) of rows of 128 f32, in numpy f32 (IEEE); codes through torch's CPU
    e4m3 rounding."""
    x = x.numpy().astype(np.float32)
    top = np.float32(448.0 if fmt == "e4m3" else 127.0)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        bad = ~np.isfinite(x).all(-1)
        tiny = amax < np.float32(2.0 ** -100)
        scale = (amax / top).astype(np.float32)
        mul = (top / amax).astype(np.float32)
        y = (x * mul[..., None]).astype(np.float32)
    y[tiny | bad] = 0.0
    scale[tiny] = 0.0
    scale[bad] = np.nan
    if fmt == "e4m3":
        codes = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[torch.from_numpy(tiny | bad)] = 0
    else:
        codes = torch.from_numpy(np.rint(y).astype(np.int8)).view(torch.uint8)
    return codes, torch.from_numpy(scale)


def _state(seed, S, H, Dv):
    g = torch.Generator().manual_seed(seed)
    x = 0.02 * torch.randn(S, H, Dv, 128, generator=g)
    x *= torch.exp(3 * torch.randn(S, H, Dv, 1, generator=g))
    return x


def _pool(P, H, Dv, fmt, ring=0):
    codes = torch.full((P, H, Dv, 128), 0x55, dtype=torch.uint8, device="cuda").view(FORMATS[fmt])
    scales = torch.full((P, H, Dv), 7.0, device="cuda")
    return codes, scales, torch.full((P, ring), 9.0, device="cuda") if ring else None


def _idx(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("S,P,N,H,Dv,ring", [(1, 1, 1, 1, 128, 0), (5, 9, 4, 3, 128, 1152),
                                             (3, 4, 3, 2, 256, 4), (2, 6, 2, 1, 1024, 5124),
                                             (20, 33, 17, 5, 384, 132)])
def test_store_and_load(S, P, N, H, Dv, ring, fmt):
    from gated_delta_rule_scan_gb300 import kda
    state = _state(S * 7 + H, S, H, Dv)
    rng = np.random.default_rng(N)
    src, dst = rng.integers(0, S, N), rng.permutation(P)[:N]      # sources may repeat
    codes, scales, pool = _pool(P, H, Dv, fmt, ring)
    rg = torch.randn(S, ring).cuda() if ring else None
    kda.kda_state_store_q8(state.cuda(), codes, scales, N=N, H=H, Dv=Dv, src=_idx(src.tolist()),
                           dst=_idx(dst.tolist()), ring=rg, ring_pool=pool)
    want_c, want_s = quantise(state[src], fmt)
    got_c = codes.view(torch.uint8).cpu()
    assert torch.equal(got_c[dst], want_c) and torch.equal(scales.cpu()[dst], want_s)
    rest = [i for i in range(P) if i not in set(dst.tolist())]
    assert (got_c[rest] == 0x55).all() and (scales.cpu()[rest] == 7.0).all()
    if ring:
        assert torch.equal(pool[dst.tolist()], rg[src.tolist()]) and (pool[rest] == 9.0).all()
    # back, into other rows
    back = torch.full((P + 2, H, Dv, 128), -3.0, device="cuda")
    rback = torch.full((P + 2, ring), -3.0, device="cuda") if ring else None
    to = rng.permutation(P + 2)[:N]
    kda.kda_state_load_q8(codes, scales, back, N=N, H=H, Dv=Dv, src=_idx(dst.tolist()),
                          dst=_idx(to.tolist()), ring_pool=pool, ring=rback)
    value = codes.cpu()[dst].float() if fmt == "int8" else \
        codes.cpu().view(torch.uint8)[dst].view(torch.float8_e4m3fn).float()
    assert torch.equal(back.cpu()[to], value * want_s[..., None])
    others = [i for i in range(P + 2) if i not in set(to.tolist())]
    assert (back.cpu()[others] == -3.0).all()
    if ring:
        assert torch.equal(rback[to.tolist()], pool[dst.tolist()]) and (rback[others] == -3.0).all()
    # the stated bounds: half a step of the row's grid (int8), 2^-4 of the element (e4m3), plus
    # three f32 roundings
    x = state[src].double()
    amax = x.abs().amax(-1, keepdim=True)
    err = (value.double() * want_s.double()[..., None] - x).abs()
    tol = amax / 254 if fmt == "int8" else torch.maximum(x.abs() / 16, amax * 2.0 ** -10 / 448)
    assert (err <= tol + 3 * 2.0 ** -24 * amax).all()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_identity_rows_and_empty_call(fmt):
    from gated_delta_rule_scan_gb300 import kda
    state = _state(1, 3, 2, 128)
    codes, scales, _ = _pool(4, 2, 128, fmt)
    kda.kda_state_store_q8(state.cuda(), codes, scales, N=0, H=2)
    assert (codes.view(torch.uint8) == 0x55).all()
    kda.kda_state_store_q8(state.cuda(), codes, scales, N=3, H=2)
    want_c, want_s = quantise(state, fmt)
    assert torch.equal(codes.view(torch.uint8).cpu()[:3], want_c)
    assert torch.equal(scales.cpu()[:3], want_s) and (scales.cpu()[3] == 7.0).all()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_special_rows(fmt):
    """Zero rows, tiny rows, the smallest that is kept, huge rows, ties, and rows that hold a NaN or
    an infinity (which read back as NaN throughout, and leave the others alone)."""
    from gated_delta_rule_scan_gb300 import kda
    x = _state(2, 1, 1, 128)
    x[0, 0, 0] = 0.0
    x[0, 0, 1] = 1e-38
    x[0, 0, 2] = 0.0
    x[0, 0, 2, 5] = 2.0 ** -100
    x[0, 0, 3] *= 1e30
    x[0, 0, 4, 17] = float("nan")
    x[0, 0, 5, 127] = float("-inf")
    x[0, 0, 6] = torch.arange(128).float() / 2 - 0.25     # halves of a step at amax 63.25
    x[0, 0, 7] = torch.arange(128).float() - 0.5
    x[0, 0, 7, 0] = 127.0                                 # scale 1: codes exactly at ties
    x[0, 0, 8] = 0.0
    x[0, 0, 8, 0] = -0.0
    x[0, 0, 9] = 3.0e38
    codes, scales, _ = _pool(1, 1, 128, fmt)
    kda.kda_state_store_q8(x.cuda(), codes, scales, N=1, H=1)
    want_c, want_s = quantise(x, fmt)
    got = codes.view(torch.uint8).cpu()
    assert torch.equal(got, want_c)
    assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(want_s))
    fine = ~torch.isnan(want_s)
    assert torch.equal(scales.cpu()[fine], want_s[fine])
    back = torch.empty(1, 1, 128, 128, device="cuda")
    kda.kda_state_load_q8(codes, scales, back, N=1, H=1)
    nan = torch.isnan(back.cpu()[0, 0])
    assert nan[4].all() and nan[5].all() and int(nan.sum()) == 256
    assert (back.cpu()[0, 0, :2] == 0).all()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_every_code_reads_back(fmt):
    from gated_delta_rule_scan_gb300 import kda
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(64).view(1, 1, 128, 128)
    if fmt == "e4m3":
        codes[(codes & 0x7f) == 0x7f] = 0                  # NaN codes are never written
    scales = torch.rand(1, 1, 128) + 0.5
    back = torch.empty(1, 1, 128, 128, device="cuda")
    kda.kda_state_load_q8(codes.cuda().view(FORMATS[fmt]), scales.cuda(), back, N=1, H=1)
    assert torch.equal(back.cpu(), codes.view(FORMATS[fmt]).float() * scales[..., None])


def test_padding_and_bad_slots():
    """Negative rows are padding; rows past an array and the second row of a destination are left
    out and reported, and nothing else is touched."""
    from gated_delta_rule_scan_gb300 import kda
    state = _state(3, 4, 2, 128)
    want_c, _ = quantise(state, "int8")
    st = state.cuda()
    codes, scales, pool = _pool(5, 2, 128, "int8", 8)
    ring = torch.randn(4, 8).cuda()

    def store(src, dst):
        kda.kda_state_store_q8(st, codes, scales, N=len(src), H=2, src=_idx(src), dst=_idx(dst),
                               ring=ring, ring_pool=pool)
    store([0, -1, 2], [3, 1, -7])                          # one live row
    assert kda.kda_device_status() == 0
    got = codes.view(torch.uint8).cpu()
    assert torch.equal(got[3], want_c[0]) and (got[[0, 1, 2, 4]] == 0x55).all()
    assert torch.equal(pool[3], ring[0]) and (pool[[0, 1, 2, 4]] == 9.0).all()
    store([1, 2, 4, 3], [5, 0, 1, 2147483647])             # slots 5 and 2^31 - 1, row 4: outside
    assert kda.kda_device_status() == 40013
    got = codes.view(torch.uint8).cpu()
    assert torch.equal(got[0], want_c[2]) and (got[[1, 2, 4]] == 0x55).all()
    store([1, -1, 3, 2], [2, 4, 2, 4])                     # slot 2 twice: the first row's; the
    assert kda.kda_device_status() == 40013                # padding does not name slot 4
    got = codes.view(torch.uint8).cpu()
    assert torch.equal(got[2], want_c[1]) and torch.equal(got[4], want_c[2])
    back = torch.full((3, 2, 128, 128), -3.0, device="cuda")
    kda.kda_state_load_q8(codes, scales, back, N=4, H=2, src=_idx([3, 5, 0, 2]),
                          dst=_idx([1, 0, 1, -1]))
    assert kda.kda_device_status() == 40013
    assert torch.equal(back[1].cpu(), codes[3].cpu().float() * scales[3].cpu()[..., None])
    assert (back[[0, 2]] == -3.0).all()
    assert kda.kda_device_status() == 0


def test_many_rows_with_one_duplicate():
    """More rows than a block has threads, the duplicate far behind its owner."""
    from gated_delta_rule_scan_gb300 import kda
    N = 600
    state = _state(4, N, 1, 128).cuda()
    codes, scales, _ = _pool(N, 1, 128, "int8")
    dst = list(range(N))
    dst[599] = 1
    kda.kda_state_store_q8(state, codes, scales, N=N, H=1, dst=_idx(dst))
    assert kda.kda_device_status() == 40013
    want, _ = quantise(state.cpu(), "int8")
    got = codes.view(torch.uint8).cpu()
    assert torch.equal(got[:599], want[:599]) and (got[599] == 0x55).all()


def test_offsets_past_32_bits():
    """Slots and state rows whose byte offsets pass 2^32."""
    from gated_delta_rule_scan_gb300 import kda
    H, P = 64, 4100                                        # 4.3 GB of codes
    codes = torch.zeros(P, H, 128, 128, dtype=torch.int8, device="cuda")
    scales = torch.zeros(P, H, 128, device="cuda")
    state = torch.zeros(1030, H, 128, 128, device="cuda")  # 4.3 GB of f32
    x = _state(5, 1, H, 128)
    state[1029] = x[0].cuda()
    kda.kda_state_store_q8(state, codes, scales, N=1, H=H, src=_idx([1029]), dst=_idx([4099]))
    want_c, want_s = quantise(x, "int8")
    assert torch.equal(codes[4099].view(torch.uint8).cpu(), want_c[0])
    assert not codes[:4099].any()
    kda.kda_state_load_q8(codes, scales, state, N=1, H=H, src=_idx([4099]), dst=_idx([1028]))
    assert torch.equal(state[1028].cpu(), codes[4099].cpu().float() * want_s[0][..., None])


def test_refusals_on_device():
    from gated_delta_rule_scan_gb300 import kda
    codes, scales, pool = _pool(4, 2, 128, "int8", 8)
    st, ring = torch.zeros(3, 2, 128, 128, device="cuda"), torch.zeros(3, 8, device="cuda")
    for bad in (dict(state=st.transpose(2, 3)), dict(scales=scales.double()), dict(src=_idx([0])),
                dict(dst=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(H=1),
                dict(ring=ring), dict(ring=ring[:2], ring_pool=pool),
                dict(ring=ring[:, :4].contiguous(), ring_pool=pool), dict(state=st.cpu())):
        a = dict(state=st, codes=codes, scales=scales, N=2, H=2)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.kda_state_store_q8(a.pop("state"), a.pop("codes"), a.pop("scales"), **a)
    with pytest.raises(kda.KdaError) as e:                 # more rows than states, no row indices
        kda.kda_state_store_q8(st, codes, scales, N=4, H=2)
    assert e.value.status == 40005
    assert (codes.view(torch.uint8) == 0x55).all()


def test_a_row_left_out_claims_no_destination():
    """An earlier row whose source lies past its array is left out; the next row that names its
    destination is the first of those that store, and is kept (in both directions)."""
    from gated_delta_rule_scan_gb300 import kda
    H, P, S = 2, 5, 4
    state = _state(70, S, H, 128).cuda()
    src = torch.tensor([S, 1, -1, 2, 2147483647, 3, 0], dtype=torch.int32, device="cuda")
    dst = torch.tensor([3, 3, 0, 0, 4, 4, 3], dtype=torch.int32, device="cuda")
    want = {3: 1, 0: 2, 4: 3}                  # slot: row; the last row finds slot 3 taken
    codes, scales = _pool(P, H, 128, "int8")[:2]
    before = codes.clone(), scales.clone()
    kda.kda_state_store_q8(state, codes, scales, src=src, dst=dst, N=7, H=H)
    assert kda.kda_device_status() == 40013
    ref_codes, ref_scales = quantise(state.cpu(), "int8")
    for p in range(P):
        c, s = codes[p].view(torch.uint8).cpu(), scales[p].cpu()
        if p in want:
            assert torch.equal(c, ref_codes[want[p]]) and torch.equal(s, ref_scales[want[p]])
        else:
            assert torch.equal(codes[p], before[0][p]) and torch.equal(scales[p], before[1][p])
    kda.kda_state_store_q8(state, codes, scales, N=4, H=H)
    out = torch.full((P, H, 128, 128), 9.0, device="cuda")
    src[0] = P
    kda.kda_state_load_q8(codes, scales, out, src=src, dst=dst, N=7, H=H)
    assert kda.kda_device_status() == 40013
    back = codes.float() * scales[..., None]
    for p in range(P):
        assert torch.equal(out[p], back[want[p]]) if p in want else (out[p] == 9.0).all()
