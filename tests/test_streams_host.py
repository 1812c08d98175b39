"""Buffers that the mixer's calls make for themselves, without a GPU: each is made while the call's
own stream is the current one.  The library's entries and torch's streams are stand-ins here."""

import contextlib

import pytest
import torch


@pytest.fixture
def made(monkeypatch):
    """Switches the entries to stand-ins; the list collects, for every buffer made, the stream that
    was current."""
    from gated_delta_rule_scan_gb300 import _build
    _build.build()
    from gated_delta_rule_scan_gb300 import kda
    current, seen = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def noted(make):
        def wrapper(*args, **kw):
            seen.append(current[-1])
            return make(*args, **{**kw, "device": "cpu"} if "device" in kw else kw)
        return wrapper
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("handle", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, noted(getattr(torch, name)))
    for name in ("kda_proj_w4", "kda_state_load_q8", "kda_decode_fused_q8", "kda_decode_fused",
                 "kda_verify_rollback", "kda_prefill_fused", "kda_conv_l2norm_prep", "kda_scan",
                 "kda_gated_rmsnorm_out"):
        monkeypatch.setattr(kda, name, lambda *args, **kw: None)
    return seen


STREAMS = [(None, None), ("side", "side"), (0, "default"), (77, ("handle", 77))]


@pytest.mark.parametrize("stream,want", STREAMS)
def test_low_bit_buffers_are_made_on_the_calls_stream(made, stream, want):
    from gated_delta_rule_scan_gb300 import mixer
    pool = mixer.StatePoolQ8(4, 2, "cpu")
    slots = torch.tensor([1, 2], dtype=torch.int32)
    any_ = dict.fromkeys(("q_raw", "k_raw", "v_raw", "conv_w", "f_raw", "dt_bias", "a_log",
                          "beta_raw", "norm_w", "gate_raw"))
    made.clear()
    state, ring = pool.load(slots, stream=stream)
    assert made == [want] * 2 and not state.any() and not ring.any()
    made.clear()
    pool.load(slots, state=state, stream=stream)
    assert made == [want]
    made.clear()
    assert not pool.decode(slots=slots, stream=stream, **any_).any()
    assert made == [want]
    made.clear()
    x, w = torch.ones(5, 256), torch.ones(3, 128, dtype=torch.uint8)
    mixer.kda_proj_w4(x=x, weights=[w, w], scales=[x, x], group=128, stream=stream)
    assert made == [want] * 3                  # two outputs and the workspace


@pytest.mark.parametrize("stream,want", STREAMS)
def test_f32_buffers_are_made_on_the_calls_stream(made, stream, want):
    from gated_delta_rule_scan_gb300 import mixer
    x, state, ring = torch.ones(6, 256), torch.ones(2, 2, 128, 128), torch.ones(2, 768, 3)
    args = dict(q_raw=x, k_raw=x, v_raw=x, conv_w=x, ring_in=ring, f_raw=x, dt_bias=x, a_log=x,
                beta_raw=x, state_in=state, norm_w=x, gate_raw=x, N=2, T=3, H=2, stream=stream)
    for call, buffers, extra in ((mixer.kda_decode, 3, {}), (mixer.kda_verify_rollback, 3, dict(keep=x)),
                                 (mixer.kda_prefill, 4, {}), (mixer.kda_forward, 10, {})):
        made.clear()
        out = call(**args, **extra)
        assert made == [want] * buffers, call
        assert out["y"].shape == (6, 256) and out["state_out"].shape == state.shape
