"""Resets: a decay of 0 drops the state before its token whatever entered it, also in its own 64-token chunk.

Inputs that are infinite or NaN may reach all outputs of their own chunk (tokens 64 to 127 here), so those are left out; where
the definition itself is NaN nothing is compared; everything else has to be finite and right, by the tolerances of
test_gpu_linear_attn.py.
"""

import numpy as np
import pytest

from oracle import mixer
from test_gpu_linear_attn import HALF, U, _close, _dt, _inputs, _np

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
RESET = 70


def _spoil(x, side, d_o=None):
    """Bad rows on one side of the reset, the chunk's first among them (which rows behind a sequence's end repeat)."""
    import torch
    x["log_alpha"][:, RESET] = -INF
    if side == "before":
        x["k"][:, 64], x["v"][:, 66, :, 5], x["k"][:, 67, :, 3], x["q"][:, 68] = NAN, INF, -INF, NAN
        x["log_alpha"][:, 68] = NAN
    else:
        x["q"][:, 72, :, 7], x["log_alpha"][:, 75] = INF, NAN
        if d_o is not None:
            d_o[:, 73], d_o[:, 80, :, 2] = NAN, -INF
    torch.cuda.synchronize()


def _outside(x):
    """NaN in the spoilt chunk: not compared."""
    x = x.copy()
    x[:, 64:128] = np.nan
    return x


SIZES = [(2, 100, 2, 64, 64), (1, 128, 1, 128, 128), (1, 300, 2, 64, 128), (1, 2000, 1, 128, 64)]


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,dk,dv", SIZES)
def test_reset_drops_what_entered_in_its_chunk(gpu_lib, B, T, H, dk, dv, dtype):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    x = _inputs(B, T, H, H, H, H, dk, dv, dtype, seed=21, mild=8.0)
    x["S0"][:, 0] = NAN
    _spoil(x, "before")
    S = torch.empty_like(x["S0"])
    o = ccq_linear_attn(**x, S_out=S)
    want, last, os, ss = mixer.linear_attn(*(_np(x[m]) for m in "qkv"), _np(x["log_alpha"]), x["scale"], _np(x["S0"]))
    assert np.isfinite(last).all() and np.isfinite(want[:, 128:]).all()
    tol = (T + dk + 16) * U
    _close(_np(S), last, ss, tol, U, "S")
    _close(_np(o), _outside(want), os, tol + (1.01 * 2.0 ** -8 if dtype == "bf16" else 0), HALF[dtype], "o")


@pytest.mark.filterwarnings("ignore:invalid value")
@pytest.mark.parametrize("side", ["before", "behind"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,dk,dv", SIZES)
def test_reset_in_the_gradient(gpu_lib, B, T, H, dk, dv, dtype, side):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    x = _inputs(B, T, H, H, H, H, dk, dv, dtype, seed=22, mild=8.0)
    g = torch.Generator().manual_seed(1)
    d_o, dS = torch.randn(B, T, H, dv, generator=g).to(_dt(dtype)).cuda(), torch.randn(B, H, dv, dk, generator=g).cuda()
    if side == "behind":
        dS[:, 0] = NAN
    else:
        x["S0"][:, 0] = NAN
    _spoil(x, side, d_o)
    got = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS, want_dS0=True)
    want, size = mixer.linear_attn_backward(*(_np(x[m]) for m in "qkv"), _np(d_o), _np(x["log_alpha"]), x["scale"], _np(x["S0"]),
                                            _np(dS))
    tol = (T + dk + dv + 16) * U
    for m in ("dq", "dk", "dv"):
        _close(_np(got[m]), _outside(want[m]), size[m], tol + (2.1 * 2.0 ** -16 if dtype == "bf16" else 0) + U, HALF[dtype], m)
    clean = "dq" if side == "before" else "dk"
    assert np.isfinite(want[clean][:, 128:] if side == "before" else want[clean][:, :64]).all()
    if side == "behind":
        assert np.isfinite(want["dS0"]).all()
        _close(_np(got["dS0"]), want["dS0"], size["dS0"], tol, U, "dS0")


@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("gate,above,below", [("f32", -87.33, -87.34), ("bf16", -87.0, -87.5)])
def test_where_a_decay_counts_as_zero(gpu_lib, T, gate, above, below):
    """A decay below fp32's least normal number, 2^-126, is a reset; one above it is not, and keeps a state that is NaN."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    x = _inputs(1, T, 2, 2, 2, 2, 64, 64, "f32", gate=gate, seed=23)
    x["S0"].fill_(NAN)
    x["log_alpha"].fill_(-0.5)
    x["log_alpha"][:, 1, 0], x["log_alpha"][:, 1, 1] = below, above
    S = torch.empty_like(x["S0"])
    o = ccq_linear_attn(**x, S_out=S)
    assert o[0, 1:, 0].isfinite().all() and S[0, 0].isfinite().all()
    assert o[0, :, 1].isnan().all() and S[0, 1].isnan().all() and o[0, 0].isnan().all()
    x["S0"].fill_(1e30)
    d_g = ccq_linear_attn_backward(**x, d_o=torch.ones_like(o))["dlog_alpha"]
    assert (d_g[0, 1, 0] == 0).all() and (d_g[0, 1, 1] != 0).all()


@pytest.mark.parametrize("T", [8, 100, 2000])
def test_an_infinite_state_lasts_without_a_reset(gpu_lib, T):
    """Decays whose product leaves fp32's range drop a finite state, and an infinite one stays infinite or NaN, as it would token
    by token."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    x = _inputs(1, T, 1, 1, 1, 1, 64, 64, "f32", gate="f32", seed=24)
    x["log_alpha"].fill_(-30.0)
    S = torch.empty_like(x["S0"])
    for value in (1e30, INF):
        x["S0"].fill_(value)
        o = ccq_linear_attn(**x, S_out=S)
        if value == INF:
            assert not o.isfinite().any() and not S.isfinite().any()
        else:
            assert o[0, 7:].isfinite().all() and S.isfinite().all()


@pytest.mark.filterwarnings("ignore:invalid value", "ignore:overflow")
@pytest.mark.parametrize("T,resets,bad", [
    (100, [70], False), (300, [1, 2, 63, 64, 65, 131], False), (300, [1, 2, 63, 64, 65, 131], True), (600, list(range(3, 600, 7)), False),
    (5000, [903, 904, 950, 4700], False), (5000, [903, 904, 950, 4700], True), (5000, [10, 1000], False), (5000, [10, 1000], True)])
def test_gradient_of_decays_before_a_reset(gpu_lib, T, resets, bad):
    """The decays of a sequence take nothing from the sequence behind a reset: not the roundings of its large rows, and not its
    NaN (in another chunk)."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    H, d = 2, 64
    x = _inputs(1, T, H, H, H, H, d, d, "f32", gate="f32", seed=25, mild=8.0)
    g = torch.Generator().manual_seed(2)
    d_o, dS = torch.randn(1, T, H, d, generator=g).cuda(), torch.randn(1, H, d, d, generator=g).cuda()
    x["log_alpha"][:, resets] = -INF
    last = resets[-1]
    for t in (x["q"], x["v"], d_o):
        t[:, last:] *= 1e4
    if bad:
        d_o[:, T - 1, :, 1] = NAN
    got = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS)["dlog_alpha"]
    want, size = mixer.linear_attn_backward(*(_np(x[m]) for m in "qkv"), _np(d_o), _np(x["log_alpha"]), x["scale"], _np(x["S0"]),
                                            _np(dS))
    want, size = want["dlog_alpha"], size["dlog_alpha"]
    assert np.isfinite(want[:, :last]).all()
    _close(_np(got), want, size, (T + 2 * d + 16) * U, U, "dlog_alpha")
    assert (got[:, resets] == 0).all()


@pytest.mark.parametrize("zero", [-88.0, -100.0, -INF])
@pytest.mark.parametrize("T", [7, 60, 130])
def test_growth_behind_a_reset_brings_nothing_back(gpu_lib, T, zero):
    """A decay just below the limit is 0, also where the decays behind it are above 1: large rows before it leave no trace."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    H, d, at = 1, 64, 3
    x = _inputs(1, T, H, H, H, H, d, d, "f32", gate="f32", seed=26)
    x["log_alpha"].fill_(0.6)
    x["log_alpha"][:, at] = zero
    x["v"][:, :at] *= 1e35
    x["S0"].mul_(1e35)
    d_o = torch.randn(1, T, H, d, generator=torch.Generator().manual_seed(3)).cuda()
    S = torch.empty_like(x["S0"])
    o = ccq_linear_attn(**x, S_out=S)
    dq = ccq_linear_attn_backward(**x, d_o=d_o)["dq"]
    want, last, os, ss = mixer.linear_attn(*(_np(x[m]) for m in "qkv"), _np(x["log_alpha"]), x["scale"], _np(x["S0"]))
    back, size = mixer.linear_attn_backward(*(_np(x[m]) for m in "qkv"), _np(d_o), _np(x["log_alpha"]), x["scale"], _np(x["S0"]))
    # a product of growing gates is a power of two of the sum of its logs: an error of a unit of a sum of up to 0.6 T log2 e, and ln 2 of that
    tol = (2 * T + d + 16) * U
    for got, w, sz in ((o, want, os), (S, last, ss), (dq, back["dq"], size["dq"])):
        _close(_np(got), w, sz, tol, U, "behind")
