"""ccq_group_norm and its gradient against the fp64 definitions (oracle/mixer.py).

Tolerances.  u = 2^-24.  A row's sums go over eight channels a lane and then six steps between lanes: below 24 u of
themselves with the squares.  Taking the mean off rounds at the size of x, so the normalised row is right to
24 u (1 + max|x| r) of (|n| + |x| r): C = 32 covers that with the few operations behind it.  The activation's exponential is
off by 2 u of its argument and itself.  The result is rounded once.
"""

import numpy as np
import pytest

from oracle import mixer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _dt(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(B, T, G, d, dtype, affine="full", gate=True, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = _dt(dtype)
    x = dict(x=(rn(B, T, G, d) + 0.5).to(dt).cuda(), gate=(2 * rn(B, T, G, d)).to(dt).cuda() if gate else None)
    shape = {"full": (G, d), "shared": (d,), "none": None}[affine]
    x["weight"] = None if shape is None else (1 + 0.3 * rn(*shape)).cuda()
    x["bias"] = None if shape is None else (0.3 * rn(*shape)).cuda()
    return x, rn(B, T, G, d).to(dt).cuda()


def _bounds(x, center, eps, activation):
    """y, and how far fp32 may leave it."""
    a = {m: _np(t) for m, t in x.items()}
    y, n, r, z = mixer.group_norm(**a, center=center, eps=eps, activation=activation)
    w = 1.0 if a["weight"] is None else np.abs(a["weight"])
    b = 0.0 if a["bias"] is None else np.abs(a["bias"])
    far = 32 * U * (1 + np.abs(a["x"]).max(-1, keepdims=True) * r)
    dz = far * (np.abs(n) + np.abs(a["x"]) * r) * w + 4 * U * (np.abs(z) + b)
    if a["gate"] is None:
        return y, 1.2 * dz + 8 * U * np.abs(y) * (1 + np.abs(z)), far, n, r, z, w
    f = np.abs(mixer._act(a["gate"], activation)[0])
    return y, dz * f + 8 * U * np.abs(y) * (1 + np.abs(a["gate"])), far, n, r, z, w


def _close(got, want, bound, tag):
    err = np.abs(got - want)
    assert np.isfinite(got).all(), tag
    assert (err <= bound + 1e-30).all(), f"{tag}: {np.max(err / (bound + 1e-30)):.2f} of the bound"


CASES = [  # B, T, G, d, affine, gate, center, activation
    (1, 1, 1, 8, "none", False, False, "none"), (2, 3, 5, 16, "full", True, True, "silu"), (1, 33, 3, 24, "shared", False, True, "silu"),
    (3, 17, 4, 64, "full", True, False, "silu"), (2, 70, 16, 128, "full", True, False, "silu"), (1, 9, 7, 80, "full", False, True, "sigmoid"),
    (64, 1, 2, 136, "shared", True, True, "sigmoid"), (2, 5, 3, 256, "none", True, False, "none"), (1, 40, 2, 504, "full", False, False, "silu"),
    (1, 6, 3, 512, "full", True, True, "silu"), (2, 3, 2, 520, "shared", True, True, "silu"), (1, 5, 1, 1024, "full", False, True, "none")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(gpu_lib, case, dtype):
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    B, T, G, d, affine, gate, center, activation = case
    x, dy = _inputs(B, T, G, d, dtype, affine, gate, seed=d)
    how = dict(center=center, eps=1e-5, activation=activation)
    y, bound, far, n, r, z, w = _bounds(x, **how)
    _close(_np(ccq_group_norm(**x, **how)), y, bound + HALF[dtype] * np.abs(y), "y")
    got = ccq_group_norm_backward(**x, dy=dy, **how)
    a = {m: _np(t) for m, t in x.items()}
    dx, dgate, dw, db = mixer.group_norm_backward(**a, dy=_np(dy), **how)
    g = np.abs(_np(dy))
    arg = z if a["gate"] is None else a["gate"]
    f, slope = (np.abs(s) for s in mixer._act(arg, activation))
    # the slope's own slope is below 0.5, and it is formed from the sigmoid and the argument
    dz = g * (slope if a["gate"] is None else f)
    off = g * ((0.5 * (bound / np.maximum(slope, 1.0)) if a["gate"] is None else 0.0) + 16 * U * (1 + np.abs(arg)))
    dn, dn_off = dz * w, off * w
    rows = lambda s: s.mean(-1, keepdims=True)  # noqa: E731
    size = r * (dn + rows(dn) + np.abs(n) * rows(dn * np.abs(n)))
    loose = r * (dn_off + rows(dn_off) + np.abs(n) * rows(dn_off * np.abs(n)))
    # n enters twice, each time off by `far` of (|n| + |x| r)
    wide = np.abs(n) + np.abs(a["x"]) * r
    loose = loose + 3 * far * (size + r * wide * rows(dn * (np.abs(n) + wide)))
    _close(_np(got["dx"]), dx, loose + HALF[dtype] * np.abs(dx), "dx")
    if gate:
        bd = g * slope * (far * wide * w + 8 * U * np.abs(z) + 4 * U) + 16 * U * g * np.abs(z) * (1 + np.abs(arg))
        _close(_np(got["dgate"]), dgate, bd + HALF[dtype] * np.abs(dgate), "dgate")
    else:
        assert got["dgate"] is None
    total = lambda s: s.sum((0, 1)) if affine == "full" else s.sum((0, 1, 2))  # noqa: E731
    if affine == "none":
        assert got["dweight"] is None and got["dbias"] is None
        return
    _close(_np(got["dbias"]), db, total(off) + 64 * U * total(dz), "dbias")
    _close(_np(got["dweight"]), dw, total(off * np.abs(n) + dz * far * wide) + 64 * U * total(dz * np.abs(n)), "dweight")
    again = ccq_group_norm_backward(**x, dy=dy, **how)
    assert all(got[m] is None or torch.equal(got[m], again[m]) for m in got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_in_place(gpu_lib, dtype):
    """Head-major rows to token-major ones, parts of a packed projection, y in x or in gate, dx in dy and dgate in gate."""
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    B, T, G, d = 2, 37, 3, 64
    x, dy = _inputs(B, T, G, d, dtype, seed=1)
    how = dict(weight=x["weight"], bias=x["bias"], activation="silu", center=True)
    want = ccq_group_norm(x["x"], gate=x["gate"], **how)
    back = ccq_group_norm_backward(x["x"], dy, gate=x["gate"], **how)
    packed = torch.full((B, T, 2, G, d), 9.0, dtype=_dt(dtype), device="cuda")
    packed[:, :, 1] = x["gate"]
    major = x["x"].transpose(1, 2).contiguous().transpose(1, 2)
    y = torch.empty(B, G, T, d, dtype=_dt(dtype), device="cuda").transpose(1, 2)
    assert torch.equal(ccq_group_norm(major, gate=packed[:, :, 1], y=y, **how), want)
    dx = torch.empty_like(y)
    got = ccq_group_norm_backward(major, dy.transpose(1, 2).contiguous().transpose(1, 2), gate=packed[:, :, 1], dx=dx, dgate=packed[:, :, 1], **how)
    assert torch.equal(got["dx"], back["dx"]) and torch.equal(packed[:, :, 1], back["dgate"]) and (packed[:, :, 0] == 9.0).all()
    assert torch.equal(got["dweight"], back["dweight"]) and torch.equal(got["dbias"], back["dbias"])
    for place in ("x", "gate"):
        a = {m: x[m].clone() for m in ("x", "gate")}
        assert torch.equal(ccq_group_norm(**a, y=a[place], **how), want)
    g = dy.clone()
    assert torch.equal(ccq_group_norm_backward(x["x"], g, gate=x["gate"], dx=g, **how)["dx"], back["dx"])


def test_rows_alone(gpu_lib):
    """A NaN or an infinity stays in its row; a row of zeros is zeros (eps above 0); other rows do not see it."""
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    x, dy = _inputs(1, 20, 3, 24, "f32", "full", False, seed=2)
    want = ccq_group_norm(x["x"], weight=x["weight"])
    bad = x["x"].clone()
    bad[0, 3, 1, 5], bad[0, 7, 2, 0], bad[0, 9, 0] = float("nan"), float("inf"), 0.0
    y = ccq_group_norm(bad, weight=x["weight"])
    touched = torch.zeros(20, 3, dtype=torch.bool, device="cuda")
    touched[3, 1] = touched[7, 2] = touched[9, 0] = True
    assert torch.equal(y[0][~touched], want[0][~touched]) and torch.isnan(y[0, 3, 1]).all() and (y[0, 9, 0] == 0).all()
    got = ccq_group_norm_backward(bad, dy, weight=x["weight"])
    back = ccq_group_norm_backward(x["x"], dy, weight=x["weight"])
    assert torch.equal(got["dx"][0][~touched], back["dx"][0][~touched]) and torch.isfinite(got["dx"][0, 9, 0]).all()


def test_streams_and_graphs(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    x, dy = _inputs(3, 700, 4, 128, "bf16", seed=3)
    want, back = ccq_group_norm(**x, activation="silu"), ccq_group_norm_backward(**x, dy=dy, activation="silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ccq_group_norm(**x, activation="silu", stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = ccq_group_norm(**x, activation="silu"), ccq_group_norm_backward(**x, dy=dy, activation="silu")
    for _ in range(3):
        r[0].zero_()
        for t in r[1].values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r[0], want) and all(torch.equal(r[1][m], back[m]) for m in back)
        assert torch.equal(ccq_group_norm(**x, activation="silu"), want)


def test_gradient_by_differences(gpu_lib):
    """Central differences of the fp32 forward: the roundings over the step, and step^2 times a third derivative, which the
    smooth inputs here keep below 1e-3 of the gradient's size."""
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    x, dy = _inputs(1, 6, 2, 64, "f32", seed=4)
    how = dict(center=True, eps=1e-3, activation="silu")
    got = ccq_group_norm_backward(**x, dy=dy, **how)
    gen = torch.Generator().manual_seed(5)
    step = 2.0 ** -6
    for m, name in (("x", "dx"), ("gate", "dgate"), ("weight", "dweight"), ("bias", "dbias")):
        u = torch.randn(x[m].shape, generator=gen).cuda()
        f = [float((ccq_group_norm(**{**x, m: x[m] + s * u}, **how).double() * dy.double()).sum()) for s in (step, -step)]
        mine = float((got[name].double() * u.double()).sum())
        size = float((got[name].double().abs() * u.double().abs()).sum())
        assert abs((f[0] - f[1]) / (2 * step) - mine) <= 1e-3 * size, name


def test_binding_refusals_on_device(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import CcqError, ccq_group_norm, ccq_group_norm_backward
    x, dy = _inputs(1, 4, 2, 64, "bf16")
    for kw in (dict(x=x["x"][0]), dict(x=x["x"].half()), dict(gate=x["gate"][:, :2]), dict(gate=x["gate"].float()), dict(weight=x["weight"][:1]),
               dict(bias=x["bias"].double()), dict(activation="relu"), dict(y=dy.float()), dict(x=x["x"][..., ::2])):
        with pytest.raises((ValueError, TypeError)):
            ccq_group_norm(**{**x, **kw})
    with pytest.raises(CcqError):
        ccq_group_norm(x["x"][..., :12].contiguous())
    with pytest.raises(CcqError):
        ccq_group_norm(**x, eps=-1.0)
    with pytest.raises((ValueError, TypeError)):
        ccq_group_norm_backward(x["x"], dy, dgate=dy)
    with pytest.raises(CcqError):
        ccq_group_norm_backward(**x, dy=dy, dx=x["x"])
