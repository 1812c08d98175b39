"""Host-side checks (no GPU) of linear attention, draft verification and the norms around a block: contract
violations are refused before any CUDA call, through the C ABI with fake pointers and through the Python
binding with CPU tensors."""

import ctypes

import pytest
import torch

FAKE = 0x10000          # 16-byte aligned, never dereferenced
FAR = 1 << 44           # apart by more than any size below


@pytest.fixture(scope="module")
def kda():
    from gated_delta_rule_scan_gb300 import _build
    _build.build()
    from gated_delta_rule_scan_gb300 import kda as mod
    return mod


def _prefill(kda, varlen, **kw):
    a = dict(q=FAR, qs=256, k=2 * FAR, ks=256, v=3 * FAR, vs=512, raw=1, g=FAKE, si=4 * FAR, so=5 * FAR, o=6 * FAR,
             N=2, T=64, H=2, Hk=2, Dk=128, Dv=256, ws=7 * FAR, wb=1 << 40, cu=FAKE, cu_host=[0, 60, 128])
    a.update(kw)
    head = (a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["raw"], a["g"], a["si"], a["so"], a["o"])
    tail = (a["H"], a["Hk"], a["Dk"], a["Dv"], 1.0, a["ws"], a["wb"], None)
    lib = kda.library()
    if not varlen:
        return lib.kda_linattn_prefill(*head, a["N"], a["T"], *tail)
    cu = a["cu_host"]
    arr = None if cu is None else (ctypes.c_int * len(cu))(*cu)
    return lib.kda_linattn_prefill_varlen(*head, a["cu"], arr, a["N"], a["N"] * a["T"], *tail)


@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(Dk=64), 40001), (dict(Dv=64), 40001), (dict(Dv=2048), 40001), (dict(N=-1), 40005),
    (dict(N=65536), 40005), (dict(T=-1), 40005), (dict(H=0), 40005), (dict(Hk=0), 40005),
    (dict(Hk=3), 40005), (dict(H=65535, Hk=1, vs=1 << 25), 40005), (dict(T=1 << 30), 40005),
    (dict(qs=248), 40005), (dict(qs=260), 40005), (dict(ks=255), 40005), (dict(vs=511), 40005),
    (dict(vs=516), 40005), (dict(raw=0, vs=514), 40005), (dict(qs=1 << 31), 40005), (dict(raw=2), 40007),
    (dict(g=None), 40004), (dict(q=None), 40004), (dict(k=None), 40004), (dict(v=None), 40004),
    (dict(o=None), 40004), (dict(so=None), 40004), (dict(q=FAR + 8), 40010), (dict(o=6 * FAR + 4), 40010),
    (dict(si=4 * FAR + 8), 40010), (dict(so=4 * FAR + 64), 40003), (dict(o=FAR), 40003),
    (dict(o=3 * FAR + 128 * 1024 - 16), 40003), (dict(v=6 * FAR + 2048), 40003), (dict(o=5 * FAR), 40003),
    (dict(si=6 * FAR + 16), 40003), (dict(raw=0, ws=None), 40009), (dict(raw=0, wb=16), 40009),
    (dict(raw=0, ws=7 * FAR + 8), 40010), (dict(k=5 * FAR + 64), 40003), (dict(raw=0, ws=FAR), 40003),
    (dict(raw=0, ws=6 * FAR - 4096), 40003), (dict(raw=0, ws=4 * FAR), 40003), (dict(N=0, cu_host=[0]), 0)])
def test_prefill_contract(kda, varlen, kw, status):
    if varlen and kw.get("N", 2) * kw.get("T", 64) != 128 and status == 40005:
        kw = dict(kw, cu_host=None)
    assert _prefill(kda, varlen, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), 40004), (dict(cu_host=None), 40004), (dict(cu_host=[1, 60, 128]), 40006),
    (dict(cu_host=[0, 130, 128]), 40006), (dict(cu_host=[0, 60, 127]), 40006)])
def test_prefill_lengths_contract(kda, kw, status):
    assert _prefill(kda, True, **kw) == status


def test_prefill_workspace_of_bad_sizes(kda):
    lib = kda.library()
    for a in ((-1, 8, 2, 2, 128, 128), (1, -8, 2, 2, 128, 128), (1, 8, 0, 2, 128, 128), (1, 8, 2, 3, 128, 128),
              (1, 8, 2, 2, 64, 128), (1, 8, 2, 2, 128, 100)):
        assert lib.kda_linattn_workspace_bytes(*a, 0) == 0
    assert lib.kda_linattn_workspace_bytes(2, 100, 4, 2, 128, 256, 0) >= 100 * (2 * 2 + 4 * 2) * 128 * 4


def _decode(kda, **kw):
    a = dict(q=FAR, qs=256, k=2 * FAR, ks=256, v=3 * FAR, vs=512, raw=0, g=FAKE, pool=4 * FAR, slots=FAKE, so=None,
             keep=None, o=6 * FAR, P=8, N=3, T=2, H=2, Hk=2, Dk=128, Dv=256)
    a.update(kw)
    return kda.library().kda_linattn_decode(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["raw"], a["g"], a["pool"], a["slots"], a["so"],
        a["keep"], a["o"], a["P"], a["N"], a["T"], a["H"], a["Hk"], a["Dk"], a["Dv"], 1.0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Dk=64), 40001), (dict(Dv=192), 40001), (dict(T=0), 40005), (dict(T=17), 40005), (dict(N=-1), 40005),
    (dict(N=65536), 40005), (dict(P=-1), 40005), (dict(slots=None, P=2), 40005), (dict(Hk=3), 40005),
    (dict(qs=128), 40005), (dict(ks=258), 40005), (dict(raw=5), 40007), (dict(g=None), 40004),
    (dict(pool=None), 40004), (dict(o=None), 40004), (dict(v=None), 40004), (dict(pool=4 * FAR + 4), 40010),
    (dict(k=2 * FAR + 4), 40010), (dict(o=4 * FAR + 8 * 2 * 256 * 512 - 16), 40003), (dict(o=FAR + 16), 40003),
    (dict(v=4 * FAR + 4096), 40003), (dict(N=0), 0)])
def test_decode_contract(kda, kw, status):
    assert _decode(kda, **kw) == status


def _accept(kda, **kw):
    a = dict(t=FAR, ts=1000, d=2 * FAR, ds=1000, dt=0, tok=FAKE, u=FAKE + 4096, r=FAKE + 8192, nd=None,
             keep=3 * FAR, out=4 * FAR, N=3, T=4, V=1000)
    a.update(kw)
    return kda.library().kda_draft_accept(a["t"], a["ts"], a["d"], a["ds"], a["dt"], a["tok"], a["u"], a["r"],
                                          a["nd"], a["keep"], a["out"], a["N"], a["T"], a["V"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 40005), (dict(N=65536), 40005), (dict(T=0), 40005), (dict(T=17), 40005), (dict(V=0), 40005),
    (dict(ts=999), 40005), (dict(ds=999), 40005), (dict(ts=1 << 40), 40005), (dict(dt=2), 40007),
    (dict(t=None), 40004), (dict(tok=None), 40004), (dict(u=None), 40004), (dict(r=None), 40004),
    (dict(keep=None), 40004), (dict(out=None), 40004), (dict(out=3 * FAR + 8), 40003), (dict(out=FAKE), 40003),
    (dict(keep=FAKE + 8192), 40003), (dict(nd=3 * FAR), 40003), (dict(out=FAR + 4000), 40003), (dict(keep=2 * FAR), 40003),
    (dict(t=FAR + 2), 40010), (dict(d=2 * FAR + 1, dt=1), 40010), (dict(N=0), 0)])
def test_accept_contract(kda, kw, status):
    assert _accept(kda, **kw) == status


def _norm(kda, **kw):
    a = dict(x=FAR, xd=0, y=2 * FAR, yd=0, bw=FAKE, g=None, per=0, act=0, nw=FAKE + 4096, h=3 * FAR, z=4 * FAR,
             zd=0, rows=4, F=256)
    a.update(kw)
    return kda.library().kda_residual_rmsnorm(a["x"], a["xd"], a["y"], a["yd"], a["bw"], a["g"], a["per"], a["act"],
                                              1.0, 1.0, a["nw"], a["h"], a["z"], a["zd"], a["rows"], a["F"], 1e-6,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(xd=2), 40007), (dict(yd=-1), 40007), (dict(zd=3), 40007), (dict(act=3), 40007), (dict(act=-1), 40007),
    (dict(per=2), 40007), (dict(rows=-1), 40005), (dict(rows=1 << 31), 40005), (dict(F=0), 40005),
    (dict(F=252), 40005), (dict(F=16392), 40005), (dict(x=None), 40004), (dict(nw=None), 40004),
    (dict(x=FAR + 8), 40010), (dict(bw=FAKE + 4), 40010), (dict(z=4 * FAR + 8), 40010),
    (dict(g=5 * FAR + 8), 40010), (dict(h=FAR + 16), 40003), (dict(h=2 * FAR), 40003), (dict(z=3 * FAR + 64), 40003),
    (dict(z=FAR), 40003), (dict(z=2 * FAR + 16), 40003), (dict(z=2 * FAR, zd=1), 40003),
    (dict(z=FAKE + 4096), 40003), (dict(g=4 * FAR, per=0), 40003), (dict(rows=0), 0), (dict(h=None, z=None), 0)])
def test_norm_contract(kda, kw, status):
    assert _norm(kda, **kw) == status


def test_python_refusals(kda):
    """Tensors of the CPU, of a wrong type or shape raise before the C call."""
    q, v, g = torch.zeros(4, 256), torch.zeros(4, 256), torch.zeros(2)
    s, o = torch.zeros(2, 2, 128, 128), torch.zeros(4, 256)
    kw = dict(N=2, T=2, H=2)
    with pytest.raises(ValueError, match="q"):
        kda.kda_linattn_prefill(q, q, v, g, s, s, o, None, **kw)
    with pytest.raises(TypeError, match="q"):
        kda.kda_linattn_prefill(q.double(), q, v, g, s, s, o, None, **kw)
    cu = torch.tensor([0, 3, 2], dtype=torch.int32)
    with pytest.raises(kda.KdaError) as e:
        kda.kda_linattn_prefill_varlen(q, q, v, g, s, s, o, None, cu, cu, H=2)
    assert e.value.status == 40006
    with pytest.raises(ValueError, match="cu_seqlens_host"):
        kda.kda_linattn_prefill_varlen(q, q, v, g, s, s, o, None, cu, cu.long(), H=2)
    with pytest.raises(ValueError):
        kda.kda_linattn_decode(q, q, v, g, s, o, N=2, T=2, H=2)
    p, t = torch.zeros(2, 3, 10), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="target"):
        kda.kda_draft_accept(p, t, p, p, t, t)
    with pytest.raises(TypeError, match="target"):
        kda.kda_draft_accept(p.double(), t, p, p, t, t)
    with pytest.raises(ValueError, match="target"):
        kda.kda_draft_accept(p[0], t, p, p, t, t)
    with pytest.raises(ValueError):
        kda.kda_residual_rmsnorm(q, q, q, q, g)
    with pytest.raises(ValueError):
        kda.kda_residual_rmsnorm(q, q, q, q, g, gate_act="tanh")


def test_buffers_are_made_on_the_calls_stream(kda, monkeypatch):
    """The mixer's calls make their buffers while the call's own stream is the current one."""
    import contextlib
    from gated_delta_rule_scan_gb300 import mixer
    current, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def noted(make):
        def wrapper(*args, **kw):
            seen.append(current[-1])
            return make(*args, **kw)
        return wrapper
    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    for name in ("kda_linattn_prefill", "kda_linattn_decode", "kda_draft_accept", "kda_residual_rmsnorm"):
        monkeypatch.setattr(kda, name, lambda *args, **kw: None)
    q = torch.ones(4, 256)
    for stream in (None, "side"):
        seen.clear()
        mixer.kda_linattn_prefill(q=q, k=q, v=q, log_decay=None, H=2, N=2, T=2, stream=stream)
        assert seen == [stream] * 3                        # o, state_out, the workspace
        seen.clear()
        o = mixer.kda_linattn_decode(q=q, k=q, v=q, log_decay=None, pool=q, N=2, T=2, H=2, stream=stream)
        assert seen == [stream] and o.shape == (4, 256)
        seen.clear()
        keep, out = mixer.kda_draft_accept(target=q.reshape(2, 2, 256), tokens=None, u=None, r=None, stream=stream)
        assert seen == [stream] * 2 and keep.shape == (2,) and out.shape == (2, 2)
        seen.clear()
        h, z = mixer.kda_residual_rmsnorm(residual=q, norm_w=q[0], stream=stream)
        assert seen == [stream] * 2 and h.shape == z.shape == q.shape
