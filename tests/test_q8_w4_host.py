"""Host-side checks (no GPU) of the 8-bit state pool's and the 4-bit projections' entry points:
contract violations are refused before any CUDA call, through the C ABI with fake pointers and
through the Python binding with CPU tensors."""

import ctypes

import pytest
import torch

FAKE = 0x10000          # 16-byte aligned, never dereferenced
FAR = 1 << 44           # apart from FAKE by more than any size below


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_scan_gb300 import _build
    _build.build()
    from gated_delta_rule_scan_gb300 import kda as mod
    return mod


def _store(kda, **kw):
    a = dict(state=FAKE, codes=FAR, scales=2 * FAR, fmt=0, rows=FAKE, slots=FAKE, S=4, P=8, N=3,
             H=2, Dk=128, Dv=128, ring=None, ring_pool=None, ring_row=0)
    a.update(kw)
    return kda.library().kda_state_store_q8(
        a["state"], a["codes"], a["scales"], a["fmt"], a["rows"], a["slots"], a["S"], a["P"],
        a["N"], a["H"], a["Dk"], a["Dv"], a["ring"], a["ring_pool"], a["ring_row"], None)


def _load(kda, **kw):
    a = dict(state=FAKE, codes=FAR, scales=2 * FAR, fmt=0, rows=FAKE, slots=FAKE, S=4, P=8, N=3,
             H=2, Dk=128, Dv=128, ring=None, ring_pool=None, ring_row=0)
    a.update(kw)
    return kda.library().kda_state_load_q8(
        a["codes"], a["scales"], a["state"], a["fmt"], a["slots"], a["rows"], a["P"], a["S"],
        a["N"], a["H"], a["Dk"], a["Dv"], a["ring_pool"], a["ring"], a["ring_row"], None)


@pytest.mark.parametrize("move", [_store, _load])
@pytest.mark.parametrize("kw,status", [
    (dict(Dk=64), 40001), (dict(Dv=192), 40001), (dict(Dv=1152), 40001), (dict(Dv=0), 40001),
    (dict(N=-1), 40005), (dict(N=65536, rows=FAKE), 40005), (dict(S=-1), 40005),
    (dict(P=-1), 40005), (dict(H=0), 40005), (dict(H=65535, Dv=256), 40005),
    (dict(rows=None, S=2), 40005), (dict(slots=None, P=2), 40005), (dict(ring_row=6), 40005),
    (dict(ring_row=-4), 40005), (dict(fmt=2), 40007), (dict(state=None), 40004),
    (dict(codes=None), 40004), (dict(scales=None), 40004), (dict(ring_row=8), 40004),
    (dict(ring_row=8, ring=FAKE), 40004), (dict(state=FAKE + 4), 40010),
    (dict(codes=FAR + 8), 40010), (dict(scales=FAR * 2 + 4), 40010),
    (dict(ring_row=8, ring=FAKE + 4, ring_pool=FAR * 3), 40010),
    (dict(codes=FAKE), 40003), (dict(scales=FAR + 16), 40003),
    (dict(ring_row=8, ring=FAR * 3, ring_pool=FAR * 3 + 16), 40003), (dict(N=0), 0)])
def test_state_move_contract(kda, move, kw, status):
    assert move(kda, **kw) == status


def _decode(kda, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, raw=0, conv=FAKE, ring=FAKE, f=FAKE, dt=FAKE, al=FAKE, mode=0,
             beta=FAKE, codes=FAR, scales=2 * FAR, fmt=0, slots=FAKE, so=None, keep=None, nw=FAKE,
             z=FAKE, y=FAKE, P=8, N=3, T=1, H=2, Hk=2, Dk=128, Dv=128, K=4)
    a.update(kw)
    return kda.library().kda_decode_fused_q8(
        a["q"], a["k"], a["v"], a["raw"], a["conv"], a["ring"], a["f"], a["dt"], a["al"], a["mode"],
        -5.0, a["beta"], a["codes"], a["scales"], a["fmt"], a["slots"], a["so"], a["keep"],
        a["nw"], a["z"], a["y"], a["P"], a["N"], a["T"], a["H"], a["Hk"], a["Dk"], a["Dv"], a["K"],
        1e-6, 1.0, 1e-6, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Dk=64), 40001), (dict(Dv=64), 40001), (dict(Dv=2048), 40001), (dict(N=-1), 40005),
    (dict(N=65536), 40005), (dict(T=0), 40005), (dict(T=17), 40005), (dict(H=0), 40005),
    (dict(Hk=0), 40005), (dict(Hk=3), 40005), (dict(P=-1), 40005), (dict(slots=None, P=2), 40005),
    (dict(raw=2), 40007), (dict(fmt=-1), 40007), (dict(mode=2), 40007), (dict(mode=8), 40007),
    (dict(K=1), 40002), (dict(K=9), 40002), (dict(y=None), 40004), (dict(ring=None), 40004),
    (dict(codes=None), 40004), (dict(al=None), 40004), (dict(codes=FAR + 4), 40010),
    (dict(z=FAKE + 4), 40010), (dict(q=FAKE + 4), 40010), (dict(f=FAKE + 4), 40010),
    (dict(scales=FAR + 32), 40003), (dict(N=0), 0)])
def test_decode_q8_contract(kda, kw, status):
    assert _decode(kda, **kw) == status


def _proj(kda, **kw):
    a = dict(x=FAKE, xd=0, t=2, in_f=256, w=[FAKE, FAKE], s=[FAKE, FAKE], z=None, sd=0, group=64,
             rows=[3, 5], out=[FAKE, FAKE], n=None)
    a.update(kw)

    def arr(v):
        return None if v is None else (ctypes.c_void_p * max(len(v), 1))(*v)
    n = len(a["rows"]) if a["n"] is None else a["n"]
    return kda.library().kda_proj_w4(
        a["x"], a["xd"], a["t"], a["in_f"], n, arr(a["w"]), arr(a["s"]), arr(a["z"]), a["sd"],
        a["group"], (ctypes.c_int * max(len(a["rows"]), 1))(*a["rows"]), arr(a["out"]), None, 0,
        None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), 40005), (dict(t=257), 40005), (dict(in_f=0), 40005), (dict(in_f=192), 40005),
    (dict(in_f=32896), 40005), (dict(n=9), 40005), (dict(n=-1), 40005), (dict(rows=[3, -1]), 40005),
    (dict(rows=[2**31 - 1] * 2, w=[FAKE] * 2), 40005), (dict(xd=2), 40007), (dict(sd=3), 40007),
    (dict(group=16), 40007), (dict(group=256), 40007), (dict(w=None), 40004), (dict(s=None), 40004),
    (dict(out=None), 40004), (dict(x=None), 40004), (dict(w=[FAKE, None]), 40004),
    (dict(s=[None, FAKE]), 40004), (dict(out=[FAKE, None]), 40004), (dict(z=[FAKE, None]), 40004),
    (dict(x=FAKE + 8), 40010), (dict(w=[FAKE, FAKE + 8]), 40010), (dict(s=[FAKE + 2, FAKE]), 40010),
    (dict(sd=1, s=[FAKE + 1, FAKE]), 40010), (dict(out=[FAKE + 2, FAKE]), 40010),
    (dict(t=0), 0), (dict(rows=[0, 0], w=[None, None], s=[None] * 2, out=[None] * 2), 0),
    (dict(rows=[], w=[], s=[], out=[]), 0)])
def test_proj_w4_contract(kda, kw, status):
    assert _proj(kda, **kw) == status


def test_proj_w4_workspace_of_bad_sizes(kda):
    for t, in_f in ((0, 256), (257, 256), (1, 100), (1, 0), (1, 65536)):
        assert kda.kda_proj_w4_workspace_bytes(t, in_f) == 0


def test_status_string_and_formats(kda):
    assert kda.status_string(40013) != "unknown status"
    assert (kda.Q8_INT8, kda.Q8_E4M3) == (0, 1)


def test_python_refusals(kda):
    """Tensors of the CPU, of a wrong type or shape, and broken lists raise before the C call."""
    codes = torch.zeros(2, 1, 128, 128, dtype=torch.int8)
    scales, state = torch.zeros(2, 1, 128), torch.zeros(2, 1, 128, 128)
    with pytest.raises(ValueError):
        kda.kda_state_store_q8(state, codes, scales, N=2, H=1)
    with pytest.raises(TypeError):
        kda.kda_state_store_q8(state, codes.float(), scales, N=2, H=1)
    with pytest.raises(ValueError):
        kda.kda_state_load_q8(codes, scales, state, N=2, H=2)
    x, w = torch.zeros(1, 128), torch.zeros(4, 64, dtype=torch.uint8)
    s, o = torch.zeros(4, 4), torch.zeros(1, 4)
    with pytest.raises(ValueError):
        kda.kda_proj_w4(x, [w], [s], [o], group=32)
    with pytest.raises(TypeError):
        kda.kda_proj_w4(x.double(), [w], [s], [o], group=32)
    with pytest.raises(TypeError):
        kda.kda_proj_w4([1], [w], [s], [o], group=32)


def test_pool_format_names(kda):
    from gated_delta_rule_scan_gb300 import mixer
    with pytest.raises(ValueError):
        mixer.StatePoolQ8(2, 1, "cpu", fmt="int4")
    p = mixer.StatePoolQ8(3, 4, "cpu", Hk=2, Dv=256, K=3, fmt="e4m3")
    assert p.codes.shape == (3, 4, 256, 128) and p.codes.dtype == torch.float8_e4m3fn
    assert p.scales.shape == (3, 4, 256) and p.ring.shape == (3, 2 * 2 * 128 + 4 * 256, 2)


@pytest.mark.parametrize("move", [_store, _load])
@pytest.mark.parametrize("kw", [
    dict(ring=FAKE), dict(ring=FAKE + 4 * 2 * 128 * 128 * 4 - 16), dict(ring=FAR),
    dict(ring=FAR + 8 * 2 * 128 * 128 - 16), dict(ring=2 * FAR), dict(ring_pool=FAKE),
    dict(ring_pool=FAR + 64), dict(ring_pool=2 * FAR + 8 * 2 * 128 * 4 - 16)])
def test_rings_apart_from_states_and_codes(kda, move, kw):
    """The rings overlap no other array of the call: states of 4 rows, codes and scales of 8 slots."""
    assert move(kda, **{"ring_row": 8, "ring": FAR * 3, "ring_pool": FAR * 4, **kw}) == 40003


@pytest.mark.parametrize("kw", [dict(ring=FAR), dict(ring=FAR + 8 * 2 * 128 * 128 - 16),
                                dict(ring=2 * FAR), dict(ring=2 * FAR - 8 * 768 * 3 * 4 + 16)])
def test_decode_ring_pool_apart_from_codes_and_scales(kda, kw):
    assert _decode(kda, **kw) == 40003
