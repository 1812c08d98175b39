"""The norms around a block fused with its gate, scale and residual, against the formula in 64 bits.

Tolerance: a row sum of up to 16384 squares by pieces of at most 32 a thread and a tree (40 roundings
in all, halved by the square root), the square root and division (2 ulp), exp and division of the gate
(3 ulp), a few products: 2^-24 * 40 relative to each term's magnitude, plus half a step of the output's
type."""

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-6


def plain(x, y, bw, gate, act, rs, bs, w):
    h = rs * x.double()
    mag = h.abs()
    if y is not None:
        b = y.double()
        if bw is not None:
            b = b * torch.rsqrt(b.pow(2).mean(1, True) + EPS) * bw.double()
        if gate is not None:
            z = gate.double()
            s = torch.sigmoid(z)
            b = b * (z if act is None else s if act == "sigmoid" else z * s)
        h = h + bs * b
        mag = mag + (bs * b).abs()
    inv = torch.rsqrt(h.pow(2).mean(1, True) + EPS)
    return h, mag, h * inv * w.double(), mag * inv * w.double().abs()


def _close(got, want, mag):
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    bound = 40 * 2.0 ** -24 * mag + step * (want.abs() + 40 * 2.0 ** -24 * mag)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp(min=1e-300)).max())


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("rows,F", [(1, 8), (3, 64), (5, 264), (130, 512), (2, 520), (7, 2056), (3, 4104),
                                    (2, 6144), (2, 8192), (1, 8200), (1, 16384), (700, 96)])
@pytest.mark.parametrize("xt,st,zt", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (F32, BF16, F32)])
@pytest.mark.parametrize("post,gate", [(True, "none"), (False, "channel"), (True, "sigmoid"), (True, "silu")])
def test_against_formula(rows, F, xt, st, zt, post, gate):
    from gated_delta_rule_scan_gb300 import mixer
    g = torch.Generator(device="cuda").manual_seed(rows + F)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, y = (3 * r(rows, F)).to(st), r(rows, F).to(xt)
    bw, w = 1 + 0.1 * r(F) if post else None, 1 + 0.1 * r(F)
    gt = None if gate == "none" else r(F) if gate == "channel" else (3 * r(rows, F)).to(xt)
    act = gate if gate in ("sigmoid", "silu") else None
    h, z = mixer.kda_residual_rmsnorm(residual=x, block=y, block_w=bw, gate=gt, gate_act=act, res_scale=0.9,
                                      block_scale=-0.4, norm_w=w, eps=EPS, z_dtype=zt)
    hw, hm, zw, zm = plain(x, y, bw, gt, act, 0.9, -0.4, w)
    assert h.dtype == st and z.dtype == zt
    _close(h, hw, hm)
    _close(z, zw, zm)


def test_parts_and_in_place():
    from gated_delta_rule_scan_gb300 import kda, mixer
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y, w = (torch.randn(9, 1024, generator=g, device="cuda") for _ in range(3))
    w = w[0].contiguous()
    # the norm before a first block: no block
    h, z = mixer.kda_residual_rmsnorm(residual=x, norm_w=w)
    hw, hm, zw, zm = plain(x, None, None, None, None, 1.0, 1.0, w)
    assert torch.equal(h, x)
    _close(z, zw, zm)
    # the last residual: no norm after it
    h, z = mixer.kda_residual_rmsnorm(residual=x, block=y)
    assert z is None
    _close(h, (x.double() + y.double()), x.double().abs() + y.double().abs())
    # h over the residual, z over the block
    want = mixer.kda_residual_rmsnorm(residual=x, block=y, norm_w=w, block_w=w)
    x2, y2 = x.clone(), y.clone()
    kda.kda_residual_rmsnorm(x2, y2, x2, y2, w, block_w=w)
    assert torch.equal(x2, want[0]) and torch.equal(y2, want[1])
    # no rows
    h, z = mixer.kda_residual_rmsnorm(residual=x[:0], block=y[:0], norm_w=w)
    assert h.shape == z.shape == (0, 1024)


def test_rows_do_not_mix():
    """A row of zeros gives zeros, a row with a NaN or an infinity stays its own."""
    from gated_delta_rule_scan_gb300 import mixer
    for F in (96, 6144):
        x, y = torch.randn(6, F, device="cuda"), torch.randn(6, F, device="cuda")
        w = torch.ones(F, device="cuda")
        clean = mixer.kda_residual_rmsnorm(residual=x, block=y, norm_w=w, block_w=w)
        x[1], y[1] = 0.0, 0.0
        y[2, 5] = float("nan")
        x[4, 7] = float("inf")
        h, z = mixer.kda_residual_rmsnorm(residual=x, block=y, norm_w=w, block_w=w)
        assert bool((h[1] == 0).all()) and bool((z[1] == 0).all())
        assert bool(torch.isnan(z[2]).all()) and not bool(torch.isfinite(z[4, 7]))
        for n in (0, 3, 5):
            assert torch.equal(h[n], clean[0][n]) and torch.equal(z[n], clean[1][n])
