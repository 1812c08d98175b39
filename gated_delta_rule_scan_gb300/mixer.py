"""Whole-mixer convenience calls over the C ABI: allocate the intermediate and output buffers
with torch on the inputs' device and run the entry points in the mixer's stage order
(prep -> scan -> gated RMSNorm, or the single fused decode/verify launch).  Plumbing only: every
value is computed by the library's kernels.
"""

from __future__ import annotations

import contextlib

import torch

from . import kda


def _norm_flag(norm_gate):
    if norm_gate not in ("sigmoid", "silu"):
        raise ValueError(norm_gate)
    return kda.NORM_SILU if norm_gate == "silu" else 0


def _empty(shape, like):
    return torch.empty(shape, dtype=torch.float32, device=like.device)


def _made(made, t):
    made.append(t)
    return t


_CURRENT = contextlib.nullcontext()


def _on(stream, device):
    """Where a call makes its own buffers: on the stream that it runs on (None: the current one).
    Made elsewhere, a fill could land after the kernels' results, and a workspace dropped on return
    be handed out again while they still run."""
    if stream is None:
        return _CURRENT
    if isinstance(stream, int):
        # (ExternalStream takes a handle of 0 for none given and opens a stream of its own)
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def _hand_over(stream, *tensors):
    """Results made on `stream` go to the caller, whose work on the current stream their memory
    outlives: it is not handed out again before that work is done."""
    if stream is not None:
        for t in tensors:
            if t.is_cuda:
                t.record_stream(torch.cuda.current_stream(t.device))


def kda_forward(*, q_raw, k_raw, v_raw, f_raw, dt_bias, a_log, beta_raw, state_in, H,
                conv_w=None, ring_in=None, norm_w=None, gate_raw=None, cu_seqlens=None,
                cu_seqlens_host=None, N=None, T=None, K=4, gate_mode=0, gate_lb=-5.0,
                l2_eps=1e-6, rms_eps=1e-6, scale=None, algo=kda.ALGO_AUTO, state_out=None,
                ring_out=None, out=None, gate_exp=None, workspace=None, stream=None,
                norm_gate="sigmoid", Hk=None, Dv=None):
    """Run the mixer on device tensors.  Either (N, T) for N sequences of T tokens, or
    cu_seqlens (int32 device) + cu_seqlens_host (int32 CPU) for packed sequences.
    gate_exp: hand the gate from the prep to the scan as decay factors exp(log-decay) (the
    prep takes the exp once per element instead of every sequential-scan CTA taking it); the
    returned g then holds decay factors.  Default: on for the sequential form, off otherwise (the
    chunked form consumes log-decays).
    workspace: scratch for the chunked form; allocated here when algo is AUTO or CHUNK and none
    is given.
    norm_gate: the RMSNorm's gate, "sigmoid" (KDA) or "silu" (GDN's gated_rmsnorm).
    Hk: grouped queries (q_raw / k_raw of Hk heads, value head h reads q/k head h % Hk).
    Dv: value heads Dv wide (a multiple of 128; q/k heads stay 128 wide; state [N, H, Dv, 128]).
    Returns a dict with q_hat, k_hat, v_hat, g, beta, o, y (None without an epilogue),
    state_out and ring_out."""
    D = kda.HEAD_DIM
    wide = Dv is not None
    Dv = D if Dv is None else Dv
    C = H * Dv
    Cg = H * D                      # per-channel gate rows: the key dim of every value head
    Cq = (H if Hk is None else Hk) * D
    rows = q_raw.shape[0]
    varlen = cu_seqlens is not None
    if not varlen:
        assert N is not None and T is not None and N * T == rows
    n_seq = (cu_seqlens_host.numel() - 1) if varlen else N
    buf, made = out if out is not None else {}, []

    def take(name, shape):
        t = buf.get(name)
        return t if t is not None else _made(made, _empty(shape, q_raw))
    with _on(stream, q_raw.device):
        q_hat = take("q_hat", (rows, Cq))
        k_hat = take("k_hat", (rows, Cq))
        v_hat = take("v_hat", (rows, C))
        g = take("g", (rows, Cg) if gate_mode == 0 else (rows, H))
        beta = take("beta", (rows, H))
        o = take("o", (rows, C))
        y = take("y", (rows, C)) if norm_w is not None else None
        if state_out is None:
            state_out = _made(made, torch.empty_like(state_in))
        if conv_w is not None and ring_out is None:
            ring_out = _made(made, torch.empty_like(ring_in))
        if workspace is None and algo != kda.ALGO_SEQ:
            workspace = kda.scan_workspace(n_seq, rows, H * Dv // D, q_raw.device, algo)
    if gate_exp is None:
        gate_exp = algo == kda.ALGO_SEQ
    gm = gate_mode | (kda.GATE_EXP if gate_exp else 0)
    common = dict(H=H, K=K, gate_mode=gm, gate_lb=gate_lb, l2_eps=l2_eps, stream=stream, Hk=Hk)
    scan_kw = dict(H=H, gate_mode=gm, scale=scale, algo=algo, workspace=workspace, stream=stream)
    if wide:
        common.update(Dv=Dv)
        scan_kw.update(Hk=Hk, Dv=Dv)
        if varlen:
            kda.kda_conv_l2norm_prep_varlen_dv(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out,
                                               f_raw, dt_bias, a_log, beta_raw, q_hat, k_hat,
                                               v_hat, g, beta, cu_seqlens, cu_seqlens_host,
                                               **common)
            kda.kda_scan_varlen_dv(q_hat, k_hat, v_hat, g, beta, state_in, state_out, o,
                                   cu_seqlens, cu_seqlens_host, **scan_kw)
        else:
            kda.kda_conv_l2norm_prep_dv(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw,
                                        dt_bias, a_log, beta_raw, q_hat, k_hat, v_hat, g, beta,
                                        N=N, T=T, **common)
            kda.kda_scan_dv(q_hat, k_hat, v_hat, g, beta, state_in, state_out, o, N=N, T=T,
                            **scan_kw)
    elif varlen:
        kda.kda_conv_l2norm_prep_varlen(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw,
                                        dt_bias, a_log, beta_raw, q_hat, k_hat, v_hat, g, beta,
                                        cu_seqlens, cu_seqlens_host, **common)
        scan_args = (q_hat, k_hat, v_hat, g, beta, state_in, state_out, o, cu_seqlens,
                     cu_seqlens_host)
        if Hk is None:
            kda.kda_scan_varlen(*scan_args, **scan_kw)
        else:
            kda.kda_scan_varlen_gqa(*scan_args, Hk=Hk, **scan_kw)
    else:
        kda.kda_conv_l2norm_prep(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw, dt_bias,
                                 a_log, beta_raw, q_hat, k_hat, v_hat, g, beta, N=N, T=T,
                                 **common)
        scan_args = (q_hat, k_hat, v_hat, g, beta, state_in, state_out, o)
        if Hk is None:
            kda.kda_scan(*scan_args, N=N, T=T, **scan_kw)
        else:
            kda.kda_scan_gqa(*scan_args, N=N, T=T, Hk=Hk, **scan_kw)
    if norm_w is not None:
        _norm_flag(norm_gate)
        norm = kda.kda_gated_rmsnorm_silu_out if norm_gate == "silu" else kda.kda_gated_rmsnorm_out
        norm(o, norm_w, gate_raw, y, rows=rows * H, eps=rms_eps, D=Dv, stream=stream)
    _hand_over(stream, *made)
    return dict(q_hat=q_hat, k_hat=k_hat, v_hat=v_hat, g=g, beta=beta, o=o, y=y,
                state_out=state_out, ring_out=ring_out, n_seq=n_seq)


def kda_prefill(*, q_raw, k_raw, v_raw, f_raw, dt_bias, a_log, beta_raw, state_in, H, conv_w,
                ring_in, norm_w, gate_raw, cu_seqlens=None, cu_seqlens_host=None, N=None, T=None,
                K=4, gate_mode=0, gate_lb=-5.0, l2_eps=1e-6, rms_eps=1e-6, scale=None,
                state_out=None, ring_out=None, y=None, workspace=None, stream=None,
                norm_gate="sigmoid", Hk=None, Dv=None):
    """The whole mixer for a prefill in one library call (kda_prefill_fused[_varlen]): conv +
    SiLU, l2 norm, gates, the chunked scan and the gated RMSNorm, the intermediates kept in the
    workspace.  Either (N, T) or cu_seqlens (int32 device) + cu_seqlens_host (int32
    CPU).  workspace: from kda.prefill_workspace (allocated here when None).
    norm_gate: the RMSNorm's gate, "sigmoid" (KDA) or "silu" (GDN's gated_rmsnorm).
    Dv: value heads Dv wide (the _dv entries; the workspace counts H * Dv / 128 units).
    Returns a dict with y, state_out and ring_out."""
    units = H if Dv is None else H * Dv // kda.HEAD_DIM
    C = units * kda.HEAD_DIM
    rows = q_raw.shape[0]
    varlen = cu_seqlens is not None
    if not varlen:
        assert N is not None and T is not None and N * T == rows
    n_seq = (cu_seqlens_host.numel() - 1) if varlen else N
    made = []
    with _on(stream, q_raw.device):
        if y is None:
            y = _made(made, _empty((rows, C), q_raw))
        if state_out is None:
            state_out = _made(made, torch.empty_like(state_in))
        if ring_out is None and conv_w is not None:
            ring_out = _made(made, torch.empty_like(ring_in))
        if workspace is None:
            workspace = kda.prefill_workspace(n_seq, rows, units, q_raw.device, gate_mode)
    args = (q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw, dt_bias, a_log, beta_raw,
            state_in, state_out, norm_w, gate_raw, y, workspace)
    common = dict(H=H, K=K, gate_mode=gate_mode | _norm_flag(norm_gate), gate_lb=gate_lb,
                  l2_eps=l2_eps, scale=scale, rms_eps=rms_eps, stream=stream, Hk=Hk, Dv=Dv)
    if varlen:
        kda.kda_prefill_fused_varlen(*args, cu_seqlens, cu_seqlens_host, **common)
    else:
        kda.kda_prefill_fused(*args, N=N, T=T, **common)
    _hand_over(stream, *made)
    return dict(y=y, state_out=state_out, ring_out=ring_out, n_seq=n_seq)


def kda_decode(*, q_raw, k_raw, v_raw, conv_w, ring_in, f_raw, dt_bias, a_log, beta_raw,
               state_in, norm_w, gate_raw, N, T, H, K=4, gate_mode=0, gate_lb=-5.0,
               l2_eps=1e-6, rms_eps=1e-6, scale=None, state_out=None, ring_out=None, y=None,
               stream=None, norm_gate="sigmoid", Hk=None, Dv=None):
    """One fused decode (T=1) or T-token verify launch.  ring_out may be ring_in and state_out
    state_in (in place).  norm_gate: "sigmoid" (KDA) or "silu" (GDN's gated_rmsnorm).
    Dv: value heads Dv wide (kda_decode_fused_dv)."""
    made = []
    with _on(stream, q_raw.device):
        if state_out is None:
            state_out = _made(made, torch.empty_like(state_in))
        if ring_out is None:
            ring_out = _made(made, torch.empty_like(ring_in))
        if y is None:
            y = _made(made, _empty((q_raw.shape[0], H * (kda.HEAD_DIM if Dv is None else Dv)), q_raw))
    kda.kda_decode_fused(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw, dt_bias, a_log,
                         beta_raw, state_in, state_out, norm_w, gate_raw, y, N=N, T=T, H=H, K=K,
                         gate_mode=gate_mode | _norm_flag(norm_gate), gate_lb=gate_lb,
                         l2_eps=l2_eps, scale=scale,
                         rms_eps=rms_eps, stream=stream, Hk=Hk, Dv=Dv)
    _hand_over(stream, *made)
    return dict(y=y, state_out=state_out, ring_out=ring_out)


def kda_verify_rollback(*, q_raw, k_raw, v_raw, conv_w, ring_in, f_raw, dt_bias, a_log,
                        beta_raw, state_in, norm_w, gate_raw, keep, N, T, H, K=4, gate_mode=0,
                        gate_lb=-5.0, l2_eps=1e-6, rms_eps=1e-6, scale=None, state_out=None,
                        ring_out=None, y=None, stream=None, norm_gate="sigmoid", Hk=None,
                        Dv=None):
    """Roll a T-token verify round back to the accepted prefixes: keep (int32 device [N]) tokens
    of each sequence, from the pre-round state_in and ring_in.  ring_out may be ring_in."""
    made = []
    with _on(stream, q_raw.device):
        if state_out is None:
            state_out = _made(made, torch.empty_like(state_in))
        if ring_out is None:
            ring_out = _made(made, torch.empty_like(ring_in))
        if y is None:
            y = _made(made, torch.zeros((q_raw.shape[0], H * (kda.HEAD_DIM if Dv is None else Dv)),
                                        dtype=torch.float32, device=q_raw.device))
    kda.kda_verify_rollback(q_raw, k_raw, v_raw, conv_w, ring_in, ring_out, f_raw, dt_bias,
                            a_log, beta_raw, state_in, state_out, norm_w, gate_raw, y, keep,
                            N=N, T=T, H=H, K=K, gate_mode=gate_mode | _norm_flag(norm_gate),
                            gate_lb=gate_lb, l2_eps=l2_eps, scale=scale, rms_eps=rms_eps,
                            stream=stream, Hk=Hk, Dv=Dv)
    _hand_over(stream, *made)
    return dict(y=y, state_out=state_out, ring_out=ring_out)


def kda_proj_w4(*, x, weights, scales, group, zeros=None, outs=None, workspace=None, stream=None):
    """Projections of x [t, in_f] by 4-bit weights with group scales (lists, one entry a weight; the
    layer's six in kda_proj6's order, or any others that read x).  Returns the list of outputs."""
    t, in_f = x.shape
    made = outs is None
    with _on(stream, x.device):
        if made:
            outs = [_empty((t, w.shape[0]), x) for w in weights]
        if workspace is None:
            workspace = kda.proj_w4_workspace(t, in_f, x.device)
    kda.kda_proj_w4(x, weights, scales, outs, group=group, zeros=zeros, workspace=workspace,
                    stream=stream)
    if made:
        _hand_over(stream, *outs)
    return outs


def kda_linattn_prefill(*, q, k, v, log_decay, H, state_in=None, cu_seqlens=None,
                        cu_seqlens_host=None, N=None, T=None, Hk=None, Dv=None, scale=None,
                        algo=kda.ALGO_AUTO, state_out=None, o=None, workspace=None, stream=None):
    """Linear attention with one log-decay a head over (N, T) or packed sequences (cu_seqlens int32
    device + cu_seqlens_host int32 CPU), from state_in (None: zero).  algo: kda.ALGO_AUTO (long
    prompts in chunks on the tensor cores) or kda.ALGO_SEQ (the recurrence in f32).  workspace: from
    kda.linattn_workspace (allocated here when None).  Returns a dict with o and state_out."""
    Dv = kda.HEAD_DIM if Dv is None else Dv
    rows, made = q.shape[0], []
    varlen = cu_seqlens is not None
    if not varlen:
        assert N is not None and T is not None and N * T == rows
    n_seq = (cu_seqlens_host.numel() - 1) if varlen else N
    with _on(stream, q.device):
        if o is None:
            o = _made(made, _empty((rows, H * Dv), q))
        if state_out is None:
            state_out = _made(made, _empty((n_seq, H, Dv, kda.HEAD_DIM), q))
        if workspace is None:
            workspace = kda.linattn_workspace(n_seq, rows, H, q.device, Hk=Hk, Dv=Dv, dtype=q.dtype, algo=algo)
    args = (q, k, v, log_decay, state_in, state_out, o, workspace)
    common = dict(H=H, Hk=Hk, Dv=Dv, scale=scale, algo=algo, stream=stream)
    if varlen:
        kda.kda_linattn_prefill_varlen(*args, cu_seqlens, cu_seqlens_host, **common)
    else:
        kda.kda_linattn_prefill(*args, N=N, T=T, **common)
    _hand_over(stream, *made)
    return dict(o=o, state_out=state_out)


def kda_linattn_decode(*, q, k, v, log_decay, pool, N, T, H, slots=None, slots_out=None, keep=None,
                       Hk=None, Dv=None, scale=None, o=None, stream=None):
    """One decode step or T-token verify of linear attention on a pool of f32 states [slots, H, Dv,
    128]; with keep the rollback of a verify that ran into other slots.  Returns o (zero in rows not
    computed when it is allocated here)."""
    Dv, made = kda.HEAD_DIM if Dv is None else Dv, o is None
    if made:
        with _on(stream, pool.device):
            o = torch.zeros(N * T, H * Dv, device=pool.device)
    kda.kda_linattn_decode(q, k, v, log_decay, pool, o, N=N, T=T, H=H, slots=slots,
                           slots_out=slots_out, keep=keep, Hk=Hk, Dv=Dv, scale=scale, stream=stream)
    if made:
        _hand_over(stream, o)
    return o


def kda_draft_accept(*, target, tokens, u, r, draft=None, n_draft=None, keep=None, out_tokens=None,
                     stream=None):
    """Verify drafted tokens against the target's probabilities.  Returns keep [N], the rows of the
    verify that stand (what kda_verify_rollback, StatePoolQ8.decode and kda_linattn_decode take), and
    out_tokens [N, T]: the accepted drafts, the new token, then -1."""
    made = []
    with _on(stream, target.device):
        if keep is None:
            keep = _made(made, torch.empty(target.shape[0], dtype=torch.int32, device=target.device))
        if out_tokens is None:
            out_tokens = _made(made, torch.empty(target.shape[:2], dtype=torch.int32,
                                                 device=target.device))
    kda.kda_draft_accept(target, tokens, u, r, keep, out_tokens, draft=draft, n_draft=n_draft,
                         stream=stream)
    _hand_over(stream, *made)
    return keep, out_tokens


def kda_residual_rmsnorm(*, residual, block=None, norm_w=None, block_w=None, gate=None, gate_act=None,
                         res_scale=1.0, block_scale=1.0, eps=1e-6, h=None, z=None, z_dtype=None,
                         stream=None):
    """The norms after and before a block with its gate, scale and residual.  Returns (h, z), both
    allocated when not given (z in z_dtype, residual's by default; no z without norm_w)."""
    made = []
    with _on(stream, residual.device):
        if h is None:
            h = _made(made, torch.empty_like(residual))
        if z is None and norm_w is not None:
            z = _made(made, torch.empty_like(residual, dtype=z_dtype))
    kda.kda_residual_rmsnorm(residual, block, h, z, norm_w, block_w=block_w, gate=gate,
                             gate_act=gate_act, res_scale=res_scale, block_scale=block_scale, eps=eps,
                             stream=stream)
    _hand_over(stream, *made)
    return h, z


class StatePoolQ8:
    """States and conv rings of up to `slots` sequences, the states in 8 bits (include/kda.h, "The
    8-bit state pool"): codes [slots, H, Dv, 128], scales [slots, H, Dv], rings [slots, channels,
    K-1].  `fmt`: "int8" or "e4m3".  Slots are handed out by the caller; index tensors are int32 on
    the pool's device, negative entries are padding."""

    FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}

    def __init__(self, slots, H, device, *, Hk=None, Dv=None, K=4, fmt="int8"):
        if fmt not in self.FORMATS:
            raise ValueError(fmt)
        self.H, self.K = H, K
        self.Hk = H if Hk is None else Hk
        self.Dv = kda.HEAD_DIM if Dv is None else Dv
        channels = 2 * self.Hk * kda.HEAD_DIM + H * self.Dv
        self.codes = torch.zeros(slots, H, self.Dv, kda.HEAD_DIM, dtype=torch.uint8,
                                 device=device).view(self.FORMATS[fmt])
        self.scales = torch.zeros(slots, H, self.Dv, device=device)
        self.ring = torch.zeros(slots, channels, K - 1, device=device)

    def store(self, state, ring, slots, rows=None, stream=None):
        """Rows `rows` (None: n) of state and ring, as a prefill returns them, into slots[n]."""
        kda.kda_state_store_q8(state, self.codes, self.scales, src=rows, dst=slots,
                               N=slots.numel(), H=self.H, Dv=self.Dv, ring=ring,
                               ring_pool=self.ring, stream=stream)

    def load(self, slots, state=None, ring=None, rows=None, stream=None):
        """slots[n] into rows `rows` (None: n) of state and ring; returns both."""
        n, made = slots.numel(), []
        with _on(stream, self.codes.device):
            if state is None:
                state = _made(made, torch.zeros(n, self.H, self.Dv, kda.HEAD_DIM,
                                                device=self.codes.device))
            if ring is None:
                ring = _made(made, torch.zeros(state.shape[0], *self.ring.shape[1:],
                                               device=self.codes.device))
        kda.kda_state_load_q8(self.codes, self.scales, state, src=slots, dst=rows, N=n, H=self.H,
                              Dv=self.Dv, ring_pool=self.ring, ring=ring, stream=stream)
        _hand_over(stream, *made)
        return state, ring

    def decode(self, *, q_raw, k_raw, v_raw, conv_w, f_raw, dt_bias, a_log, beta_raw, norm_w,
               gate_raw, slots, T=1, slots_out=None, keep=None, gate_mode=0, gate_lb=-5.0,
               l2_eps=1e-6, rms_eps=1e-6, scale=None, y=None, norm_gate="sigmoid", stream=None):
        """One decode step or T-token verify of the sequences in slots[n], written to slots_out[n]
        (None: in place).  With keep (int32 [N]) only the first keep[n] tokens are taken: the
        rollback of a verify that ran into other slots.  Returns y (zero in rows not computed when
        it is allocated here)."""
        N, made = slots.numel(), y is None
        if made:
            with _on(stream, self.codes.device):
                y = torch.zeros(N * T, self.H * self.Dv, device=self.codes.device)
        kda.kda_decode_fused_q8(q_raw, k_raw, v_raw, conv_w, self.ring, f_raw, dt_bias, a_log,
                                beta_raw, self.codes, self.scales, norm_w, gate_raw, y, N=N, T=T,
                                H=self.H, slots=slots, slots_out=slots_out, keep=keep, K=self.K,
                                gate_mode=gate_mode | _norm_flag(norm_gate), gate_lb=gate_lb,
                                l2_eps=l2_eps, scale=scale, rms_eps=rms_eps, stream=stream,
                                Hk=self.Hk, Dv=self.Dv)
        if made:
            _hand_over(stream, y)
        return y


class HostPrefillStream:
    """Prefill over batches that live in pinned host memory, pipelined over three CUDA streams:
    while batch i runs kda_prefill on the device, batch i+1 is copied in and the results of
    batch i-1 are copied out (the host<->device link is full duplex, so the two copies overlap
    each other as well as the kernels).  Every batch moves its own inputs and results; nothing is
    cached between batches.

    Layout: `slots` (default 2) device copies of the per-batch inputs and outputs, used in turn;
    one prefill workspace, since the prefills run in order on one stream.  The weights (conv_w,
    dt_bias, a_log, norm_w) are model parameters and stay resident on the device.
    Fixed-length batches only: every batch has the N, T, H given here.

    submit(host_in, host_out) queues one batch and returns at once.  host_in maps BATCH_KEYS to
    pinned CPU tensors (ring_in only when the mixer has a conv); host_out maps y, state_out and
    (with a conv) ring_out to pinned CPU tensors that receive the results.  Neither may be
    touched by the host until synchronize() returns.  Ordering: a slot's inputs are overwritten
    only after the prefill that read them finished, and its outputs only after they were copied
    out (CUDA events on the streams; the host never blocks in submit)."""

    BATCH_KEYS = ("q_raw", "k_raw", "v_raw", "f_raw", "beta_raw", "gate_raw", "state_in",
                  "ring_in")

    def __init__(self, *, like, conv_w, dt_bias, a_log, norm_w, H, N, T, K=4, gate_mode=0,
                 gate_lb=-5.0, l2_eps=1e-6, rms_eps=1e-6, scale=None, slots=2):
        dev = dt_bias.device
        if dev.type != "cuda":
            raise ValueError("HostPrefillStream: the weights must be CUDA tensors")
        self.keys = tuple(k for k in self.BATCH_KEYS
                          if not (k == "ring_in" and conv_w is None))
        self.weights = dict(conv_w=conv_w, dt_bias=dt_bias, a_log=a_log, norm_w=norm_w)
        self.params = dict(H=H, N=N, T=T, K=K, gate_mode=gate_mode, gate_lb=gate_lb,
                           l2_eps=l2_eps, rms_eps=rms_eps, scale=scale)
        rows, C = N * T, H * kda.HEAD_DIM
        self.slots = []
        for _ in range(slots):
            din = {k: torch.empty(like[k].shape, dtype=like[k].dtype, device=dev)
                   for k in self.keys}
            dout = dict(y=torch.empty(rows, C, dtype=torch.float32, device=dev),
                        state_out=torch.empty_like(din["state_in"]))
            if conv_w is not None:
                dout["ring_out"] = torch.empty_like(din["ring_in"])
            self.slots.append((din, dout, dict(copied=torch.cuda.Event(),
                                               ran=torch.cuda.Event(),
                                               drained=torch.cuda.Event())))
        self.workspace = kda.prefill_workspace(N, rows, H, dev, gate_mode)
        self.copy_in = torch.cuda.Stream(dev)
        self.run = torch.cuda.Stream(dev)
        self.copy_out = torch.cuda.Stream(dev)
        self.submitted = 0
        # the buffers live on the default stream's pool but are used on the three streams: the
        # allocator keeps their memory until work queued there has finished, even if this
        # object is dropped early
        for din, dout, _ in self.slots:
            for t in (*din.values(), *dout.values()):
                for st in (self.copy_in, self.run, self.copy_out):
                    t.record_stream(st)
        self.workspace.record_stream(self.run)

    @property
    def h2d_bytes_per_batch(self) -> int:
        din = self.slots[0][0]
        return sum(t.numel() * t.element_size() for t in din.values())

    @property
    def d2h_bytes_per_batch(self) -> int:
        dout = self.slots[0][1]
        return sum(t.numel() * t.element_size() for t in dout.values())

    def submit(self, host_in, host_out):
        din, dout, ev = self.slots[self.submitted % len(self.slots)]
        reused = self.submitted >= len(self.slots)
        if reused:                          # the slot's previous prefill has read its inputs
            self.copy_in.wait_event(ev["ran"])
        with torch.cuda.stream(self.copy_in):
            for k in self.keys:
                din[k].copy_(host_in[k], non_blocking=True)
        ev["copied"].record(self.copy_in)
        self.run.wait_event(ev["copied"])
        if reused:                          # the slot's previous results have been copied out
            self.run.wait_event(ev["drained"])
        kda_prefill(**{"ring_in": None, **din}, **self.weights, **self.params, y=dout["y"],
                    state_out=dout["state_out"], ring_out=dout.get("ring_out"),
                    workspace=self.workspace, stream=self.run)
        ev["ran"].record(self.run)
        self.copy_out.wait_event(ev["ran"])
        with torch.cuda.stream(self.copy_out):
            for k, t in dout.items():
                host_out[k].copy_(t, non_blocking=True)
        ev["drained"].record(self.copy_out)
        self.submitted += 1

    def record_done(self, event):
        """Record `event` on the copy-out stream: it completes once every batch submitted so far
        has been copied in, run and copied out."""
        event.record(self.copy_out)

    def synchronize(self):
        self.copy_out.synchronize()
        self.run.synchronize()
        self.copy_in.synchronize()

    def close(self):
        """Wait for every submitted batch; the host buffers given to submit() are then free."""
        self.synchronize()
