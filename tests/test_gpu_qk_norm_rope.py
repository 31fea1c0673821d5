"""ccq_qk_norm_rope and its gradient on the GPU against their fp64 definitions.

Tolerances.  u = 2^-24.  A forward entry goes through: the sum of squares (eight terms in a row, then
at most four levels: 13 roundings of like-signed terms), of which the root takes half; root, division,
product by r, by w (4); cosine and sine, within 2 units each, of an angle rounded to fp32 turns below
1/2 (2^-26 turns, 1.6 u radians); two products and a sum (2): in all 6.5 + 4 + 3.6 + 2 < 20 u of
hypot(entry, partner).  The gradient adds the dot product (eight terms in a row of three factors each,
four levels: 16) to both: 40 u of the sizes that the oracle gives.  Storing as bf16 adds half a step,
2^-8 of the value.
"""

import numpy as np
import pytest

from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": 0.0}


def _torch():
    import torch
    return torch, {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _make(dtype, B, T, Hq, Hk, d, rot, weights, seed, far=0):
    torch, dts = _torch()
    g = torch.Generator().manual_seed(seed)
    packed = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=g).to(dts[dtype]).cuda()
    q = packed[..., : Hq * d].view(B, T, Hq, d) if Hq else None
    k = packed[..., Hq * d : (Hq + Hk) * d].view(B, T, Hk, d) if Hk else None
    pos = (torch.randint(0, 1000 + far, (B, 1), generator=g) + torch.arange(T)).cuda()
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda() if rot else None
    w = [(1 + 0.1 * torch.randn(d, generator=g)).cuda() if weights else None for _ in range(2)]
    return q, k, pos, f, w[0], w[1]


def _check(got, want, size, dtype, units, tag):
    err = np.abs(_np(got) - want)
    tol = units * U * size + STEP[dtype] * (np.abs(want) + units * U * size) + 1e-37
    bad = err > tol
    assert not bad.any(), f"{tag}: {bad.sum()} of {bad.size} off, worst {np.max(err / tol):.2f} of the tolerance"


CASES = [
    # dtype, B, T, Hq, Hk, d, rot, interleaved, expand, q_norm, k_norm, weights, far
    ("bf16", 2, 5, 4, 4, 128, 128, False, False, "rms", "l2", True, 0),
    ("bf16", 64, 1, 3, 1, 128, 128, True, True, "rms", "l2", False, 100_000),
    ("f32", 1, 33, 6, 2, 64, 32, True, True, "l2", "rms", True, 10_000_000),
    ("f32", 2, 17, 1, 1, 64, 64, False, False, "none", "l2", False, 0),
    ("f32", 1, 1, 2, 2, 128, 16, False, False, "rms", "none", True, 0),
    ("bf16", 1, 67, 8, 2, 64, 0, False, True, "l2", "l2", True, 0),
    ("f32", 3, 129, 5, 5, 128, 48, False, False, "rms", "l2", True, 1000),
    ("bf16", 1, 300, 16, 4, 128, 96, True, False, "rms", "l2", True, 1000),
]


@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(gpu_lib, case):
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, dts = _torch()
    dtype, B, T, Hq, Hk, d, rot, inter, expand, qn, kn, weights, far = case
    q, k, pos, f, wq, wk = _make(dtype, B, T, Hq, Hk, d, rot, weights, 11, far)
    how = dict(positions=pos, inv_freq=f, q_weight=wq, k_weight=wk, q_norm=qn, k_norm=kn, eps=1e-5, interleaved=inter)
    qo, ko = ccq_qk_norm_rope(q, k, expand_keys=expand, **how)
    copies = Hq // Hk if expand else 1
    for got, x, w, norm, c, tag in ((qo, q, wq, qn, 1, "q"), (ko, k, wk, kn, copies, "k")):
        want, size = layer.norm_rope(_np(x), _np(w), norm, 1e-5, _np(pos), _np(f), inter, c)
        assert got.dtype == x.dtype and tuple(got.shape) == want.shape
        _check(got, want, size, dtype, 20, tag)

    gen = torch.Generator().manual_seed(12)
    dqo = torch.randn(B, Hq, T, d, generator=gen).cuda()
    dko = torch.randn(B, Hk * copies, T, d, generator=gen).cuda()
    out = ccq_qk_norm_rope_backward(q, k, dqo, dko, **how)
    again = ccq_qk_norm_rope_backward(q, k, dqo, dko, **how)
    for x, w, norm, g, c, s in ((q, wq, qn, dqo, 1, "q"), (k, wk, kn, dko, copies, "k")):
        dx, dw, dxs, dws = layer.norm_rope_backward(_np(x), _np(w), norm, 1e-5, _np(pos), _np(f), inter, _np(g), c)
        assert torch.equal(out["d" + s], again["d" + s])
        _check(out["d" + s], dx, dxs, dtype, 40, "d" + s)
        if weights:
            # a sum over B T H rows: no path is longer than all rows in a row
            _check(out[f"d{s}_weight"], dw, dws, "f32", 40 + B * T * x.shape[2], f"d{s}_weight")
            assert torch.equal(out[f"d{s}_weight"], again[f"d{s}_weight"])
        else:
            assert out[f"d{s}_weight"] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_orders_and_absent_sides(gpu_lib, dtype):
    """A transposed view, heads that share one row of memory (stride 0), one side alone, and gradients
    written into the parts of a packed buffer, whose other part stays as it was."""
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, dts = _torch()
    B, T, H, d = 2, 21, 3, 64
    g = torch.Generator().manual_seed(3)
    base = torch.randn(H, B, T, d, generator=g).to(dts[dtype]).cuda()
    q = base.permute(1, 2, 0, 3)
    k = torch.randn(B, T, 1, d, generator=g).to(dts[dtype]).cuda().expand(B, T, H, d)
    f = torch.linspace(1.0, 0.01, d // 2).cuda()
    qo, ko = ccq_qk_norm_rope(q, k, inv_freq=f, position_offset=100)
    q1, none = ccq_qk_norm_rope(q.contiguous(), None, inv_freq=f, position_offset=100)
    none2, k1 = ccq_qk_norm_rope(None, k.contiguous(), inv_freq=f, position_offset=100)
    assert none is None and none2 is None and torch.equal(qo, q1) and torch.equal(ko, k1)
    pos = np.arange(T)[None].repeat(B, 0) + 100
    want, size = layer.norm_rope(_np(q), None, "rms", 1e-6, pos, _np(f), False)
    _check(qo, want, size, dtype, 20, "q")

    dqo, dko = torch.randn(2, B, H, T, d, generator=g).cuda()
    packed = torch.full((B, T, 3 * H * d), 7.0, dtype=dts[dtype], device="cuda")
    dq, dk = packed[..., : H * d].view(B, T, H, d), packed[..., H * d : 2 * H * d].view(B, T, H, d)
    out = ccq_qk_norm_rope_backward(q, k, dqo, dko, inv_freq=f, position_offset=100, dq=dq, dk=dk)
    plain = ccq_qk_norm_rope_backward(q, k, dqo, dko, inv_freq=f, position_offset=100)
    assert out["dq"] is dq and torch.equal(dq, plain["dq"]) and torch.equal(dk, plain["dk"])
    assert (packed[..., 2 * H * d :] == 7.0).all()


def test_values_are_laid_out_as_they_are(gpu_lib):
    from curvature_conditioned_query_amd import ccq_qk_norm_rope
    torch, _ = _torch()
    v = torch.randn(2, 37, 3, 128).to(torch.bfloat16).cuda()
    _, out = ccq_qk_norm_rope(None, v, k_norm="none")
    assert torch.equal(out, v.transpose(1, 2))


def test_zero_rows_floors_and_bad_rows_stay_apart(gpu_lib):
    """A zero row gives zeros and, under L2, its floor's gradient; NaN and inf stay in their own row."""
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, _ = _torch()
    B, T, H, d = 1, 9, 2, 64
    g = torch.Generator().manual_seed(5)
    q, k = torch.randn(2, B, T, H, d, generator=g).cuda()
    clean = ccq_qk_norm_rope(q, k)
    q[0, 2], k[0, 2] = 0.0, 0.0
    q[0, 3, 1, 5], k[0, 4, 0, 0] = float("nan"), float("inf")
    qo, ko = ccq_qk_norm_rope(q, k)
    assert (qo[0, :, 2] == 0).all() and (ko[0, :, 2] == 0).all()
    assert qo[0, 1, 3].isnan().all() and ko[0, 0, 4, 0].isnan()
    rows = torch.ones(B, H, T, dtype=torch.bool, device="cuda")
    rows[0, :, 2] = False
    qr, kr = rows.clone(), rows.clone()
    qr[0, 1, 3], kr[0, 0, 4] = False, False
    assert torch.equal(qo[qr], clean[0][qr]) and torch.equal(ko[kr], clean[1][kr])
    go = torch.ones(B, H, T, d, device="cuda")
    out = ccq_qk_norm_rope_backward(q, k, go, go, eps=1e-6)
    assert torch.allclose(out["dk"][0, 2], torch.full((H, d), 1e12, device="cuda"))
    assert torch.allclose(out["dq"][0, 2], torch.full((H, d), 1e3, device="cuda"))


def test_other_stream_and_replayed_capture(gpu_lib):
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, dts = _torch()
    q, k, pos, f, wq, wk = _make("bf16", 2, 40, 4, 2, 128, 128, True, 21)
    how = dict(positions=pos, inv_freq=f, q_weight=wq, k_weight=wk)
    dqo, dko = torch.randn(2, 2, 4, 40, 128, device="cuda")
    want = ccq_qk_norm_rope(q, k, expand_keys=True, **how)
    back = ccq_qk_norm_rope_backward(q, k, dqo, dko, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ccq_qk_norm_rope(q, k, expand_keys=True, stream=side, **how)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ccq_qk_norm_rope(q, k, expand_keys=True, **how)
        gback = ccq_qk_norm_rope_backward(q, k, dqo, dko, **how)
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        want = ccq_qk_norm_rope(q, k, expand_keys=True, **how)
        back = ccq_qk_norm_rope_backward(q, k, dqo, dko, **how)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(torch.equal(back[n], gback[n]) for n in back)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_entries_that_are_not_rotated_pass_as_they_are(gpu_lib, dtype, interleaved):
    """Behind the rotated part an infinity stays one, and neither it nor a NaN reaches the entry beside it;
    inside, only the two of a pair."""
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, dts = _torch()
    inf, nan = float("inf"), float("nan")
    q = torch.randn(1, 9, 2, 128, generator=torch.Generator().manual_seed(4)).to(dts[dtype]).cuda()
    f = torch.linspace(1.0, 0.1, 16).cuda()
    how = dict(inv_freq=f, q_norm="none", position_offset=3, interleaved=interleaved)
    clean, _ = ccq_qk_norm_rope(q, None, **how)
    assert torch.equal(clean[..., 32:], q.transpose(1, 2)[..., 32:])
    q[0, 4, 1, 40], q[0, 5, 0, 101], q[0, 6, 1, 2] = inf, nan, nan
    out, _ = ccq_qk_norm_rope(q, None, **how)
    touched = torch.zeros_like(out, dtype=torch.bool)
    touched[0, 1, 4, 40] = touched[0, 0, 5, 101] = touched[0, 1, 6, 2] = touched[0, 1, 6, 3 if interleaved else 18] = True
    assert out[0, 1, 4, 40] == inf and out[0, 0, 5, 101].isnan() and torch.equal(out[~touched], clean[~touched])
    grad = torch.zeros(1, 2, 9, 128, device="cuda")
    grad[0, 1, 4, 40], grad[0, 0, 5, 101] = -inf, nan
    dq = ccq_qk_norm_rope_backward(torch.ones_like(q), None, grad, None, **how)["dq"]
    assert dq[0, 4, 1, 40] == -inf and dq[0, 5, 0, 101].isnan()
    dq[0, 4, 1, 40], dq[0, 5, 0, 101] = 0, 0
    assert (dq == 0).all()


def test_a_nan_fills_its_row_under_both_norms(gpu_lib):
    """A row's norm is NaN with one of its entries, and so are the row and its gradient; its neighbours' are not."""
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    torch, dts = _torch()
    for dt in dts.values():
        for norm in ("rms", "l2"):
            q = torch.randn(1, 9, 2, 64, generator=torch.Generator().manual_seed(6)).to(dt).cuda()
            grad = torch.randn(1, 2, 9, 64, generator=torch.Generator().manual_seed(7)).cuda()
            clean = ccq_qk_norm_rope(q, None, q_norm=norm)[0], ccq_qk_norm_rope_backward(q, None, grad, None, q_norm=norm)["dq"]
            q[0, 4, 1, 7] = float("nan")
            out = ccq_qk_norm_rope(q, None, q_norm=norm)[0], ccq_qk_norm_rope_backward(q, None, grad, None, q_norm=norm)["dq"]
            assert out[0][0, 1, 4].isnan().all() and out[1][0, 4, 1].isnan().all(), norm
            out[0][0, 1, 4], out[1][0, 4, 1] = clean[0][0, 1, 4], clean[1][0, 4, 1]
            assert torch.equal(out[0], clean[0]) and torch.equal(out[1], clean[1]), norm


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_a_norm_the_gradient_does_not_see_the_row(gpu_lib, dtype):
    """Rows of infinities and NaN, as in a padded batch: dq is the gradient turned back, whatever the row holds."""
    from curvature_conditioned_query_amd import ccq_qk_norm_rope_backward
    torch, dts = _torch()
    f = torch.linspace(1.0, 0.1, 16).cuda()
    grad = torch.randn(1, 2, 9, 64, generator=torch.Generator().manual_seed(8)).cuda()
    q = torch.randn(1, 9, 2, 64, generator=torch.Generator().manual_seed(9)).to(dts[dtype]).cuda()
    want = ccq_qk_norm_rope_backward(q, None, grad, None, inv_freq=f, q_norm="none")["dq"]
    q[0, 3], q[0, 4, 1, 7], q[0, 5] = float("inf"), -float("inf"), float("nan")
    assert torch.equal(ccq_qk_norm_rope_backward(q, None, grad, None, inv_freq=f, q_norm="none")["dq"], want)
