"""ccq_logits_adjust against the fp64 definition (oracle/mixer.py).

Tolerance: each value passes a division or product, two differences and its biases in fp32, then one rounding:
(6 + biases) 2^-24 of the size of the terms, and half a step of the result.
"""

import numpy as np
import pytest

from oracle import mixer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(R, V, L, n, dtype, mask=True, lengths=True, prompts=True, rows=True, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    c = dict(logits=(3 * torch.randn(R, V, generator=g)).to(dt).cuda())
    if L:
        c["history"] = (V * torch.rand(R, L, generator=g) ** 3).int()
        c["history"][:, ::7] = torch.randint(-3, V + 3, c["history"][:, ::7].shape, generator=g, dtype=torch.int32)
        c["history"] = c["history"].cuda()
        if lengths:
            c["lengths"] = torch.randint(-1, L + 2, (R,), generator=g, dtype=torch.int32).cuda()
        if prompts:
            c["prompt_lengths"] = torch.randint(-1, L + 2, (R,), generator=g, dtype=torch.int32).cuda()
    for m, v in (("repetition", 1.3), ("presence", 0.4), ("frequency", 0.2)):
        c[m] = (v * (0.8 + 0.4 * torch.rand(R, generator=g))).cuda() if rows else v
    if n:
        c["bias_token"] = torch.randint(-2, V + 2, (R, n), generator=g, dtype=torch.int32)
        c["bias_token"][:, n // 2] = c["bias_token"][:, 0]  # twice in the list
        c["bias_token"] = c["bias_token"].cuda()
        c["bias_value"] = torch.randn(R, n, generator=g).cuda()
    if mask:
        c["allowed"] = torch.randint(-2**31, 2**31, (R, (V + 31) // 32), generator=g).int().cuda()
    return c


def _oracle(c):
    a = {m: (_np(t) if m in ("logits", "bias_value") else t.cpu().numpy()) if hasattr(t, "cpu") else t for m, t in c.items()}
    for m in ("repetition", "presence", "frequency"):
        if m in a:
            a[m] = np.asarray(a[m], np.float64) if np.ndim(a[m]) else float(np.float32(a[m]))
    return mixer.logits_adjust(**a)


def _check(got, c, dtype):
    want, size = _oracle(c)
    got = _np(got).reshape(want.shape)
    off = np.isinf(want) | np.isnan(want)
    assert np.array_equal(got[off], want[off], equal_nan=True)
    n = c["bias_token"].shape[1] if "bias_token" in c else 0
    err, bound = np.abs(got - want)[~off], ((6 + n) * U * size + HALF[dtype] * np.abs(want))[~off] + 1e-37
    assert (err <= bound).all(), np.max(err / bound)
    # what nothing touches stays as it is, to the bit
    untouched = want == _np(c["logits"])
    assert np.array_equal(got[untouched], want[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,L,n,kw", [
    (1, 1, 3, 1, {}), (3, 31, 10, 4, {}), (2, 33, 0, 0, {}), (2, 100, 40, 0, dict(mask=False)), (4, 1001, 300, 7, dict(prompts=False)),
    (2, 8191, 50, 33, dict(lengths=False)), (2, 8193, 1000, 1, dict(rows=False)), (1, 16400, 3, 0, dict(mask=False, lengths=False, prompts=False)),
    (3, 40003, 2000, 300, {}), (2, 20001, 0, 1024, dict(mask=False))])
def test_adjust(gpu_lib, R, V, L, n, kw, dtype):
    from curvature_conditioned_query_amd import ccq_logits_adjust
    c = _case(R, V, L, n, dtype, seed=V, **kw)
    _check(ccq_logits_adjust(**c), c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_views_and_beams(gpu_lib, dtype):
    import torch
    from curvature_conditioned_query_amd import ccq_logits_adjust
    c = _case(6, 1003, 50, 5, dtype, seed=1)
    want = ccq_logits_adjust(**c)
    wide = torch.full((6, 1100), 4.0, dtype=c["logits"].dtype, device="cuda")
    wide[:, :1003] = c["logits"]
    view = wide[:, :1003]
    assert torch.equal(ccq_logits_adjust(**{**c, "logits": view}), want) and torch.equal(view, c["logits"])
    out = torch.empty(2, 3, 1003, dtype=want.dtype, device="cuda")
    ccq_logits_adjust(**{**c, "logits": c["logits"].view(2, 3, 1003)}, out=out)
    assert torch.equal(out.view(6, 1003), want)
    r = ccq_logits_adjust(**{**c, "logits": view}, out=view)
    assert r.data_ptr() == wide.data_ptr() and torch.equal(view, want) and (wide[:, 1003:] == 4.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unusual_values(gpu_lib, dtype):
    """Infinities, NaN, zeros and the lowest finite value; a mask that leaves nothing; a mask over a NaN."""
    import torch
    from curvature_conditioned_query_amd import ccq_logits_adjust
    c = _case(4, 100, 0, 0, dtype, mask=False, rows=False)
    x = c["logits"]
    x[0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, torch.finfo(x.dtype).min], device="cuda").to(x.dtype)
    same = ccq_logits_adjust(x)
    assert torch.equal(same.view(torch.uint8), x.view(torch.uint8))
    c["history"] = torch.tensor([[1, 2, 3, 4, 0]] * 4, dtype=torch.int32, device="cuda")
    y = ccq_logits_adjust(x, history=c["history"], repetition=2.0)
    assert torch.isnan(y[0, 0]) and y[0, 1] == float("inf") and y[0, 2] == -float("inf") and (y[0, 3:5] == 0).all()
    none = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    assert (ccq_logits_adjust(x, allowed=none) == -float("inf")).all()
    y = ccq_logits_adjust(x, allowed=none, bias_token=torch.full((4, 1), 7, dtype=torch.int32, device="cuda"), bias_value=torch.ones(4, 1, device="cuda"))
    assert (y == -float("inf")).all()


def test_before_a_selection_in_a_graph(gpu_lib):
    """Adjusted in place, then selected from, captured and replayed."""
    import torch
    from curvature_conditioned_query_amd import ccq_beam_select, ccq_logits_adjust
    c = _case(8, 5001, 200, 9, "bf16", seed=2)
    scores = -torch.rand(2, 4, device="cuda")
    logits = c.pop("logits").view(2, 4, 5001)
    want = ccq_logits_adjust(logits, **c)
    pick = ccq_beam_select(want, scores, 4)
    buf = logits.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccq_logits_adjust(buf, **c, out=buf)
        got = ccq_beam_select(buf, scores, 4)
    for _ in range(3):
        buf.copy_(logits)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want) and all(torch.equal(got[m], pick[m]) for m in pick)
    bits = c["allowed"].cpu().numpy().astype(np.uint32).reshape(2, 4, -1)
    for n in range(2):
        for t, k in zip(pick["token"][n].tolist(), pick["parent"][n].tolist()):
            assert (int(bits[n, k, t // 32]) >> (t % 32)) & 1


def test_binding_refusals_on_device(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import CcqError, ccq_logits_adjust
    c = _case(4, 100, 10, 3, "bf16")
    for kw in (dict(logits=c["logits"].half()), dict(history=c["history"].long()), dict(history=c["history"][:3]), dict(history=None),
               dict(lengths=c["lengths"][:2]), dict(repetition=c["repetition"].double()), dict(bias_token=c["bias_token"][:, :2]),
               dict(bias_value=None), dict(allowed=c["allowed"][:, :3]), dict(out=torch.empty(4, 101, dtype=torch.bfloat16, device="cuda")),
               dict(out=torch.empty(4, 100, device="cuda"))):
        with pytest.raises((ValueError, TypeError, CcqError)):
            ccq_logits_adjust(**{**c, **kw})
    with pytest.raises(CcqError):
        ccq_logits_adjust(c["logits"], repetition=0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [32767, 32768])
def test_one_token_all_along_a_history(gpu_lib, L, dtype):
    """The largest counts of 16-bit entries and the first beyond them, beside neighbours that stand there once, with biases
    at a stretch's first and last tokens."""
    import torch
    from curvature_conditioned_query_amd import ccq_logits_adjust
    c = _case(4, 20001, L, 6, dtype, mask=False, lengths=False, prompts=False, seed=2)
    h = c["history"]
    h[:2], h[2:] = 16383, 8192
    h[1, 5], h[1, 6], h[3, 7], h[3, 8] = 16382, 16384, 8193, 8191
    c["prompt_lengths"] = torch.tensor([0, 1, L, L - 1], dtype=torch.int32, device="cuda")
    c["bias_token"][:, :4] = torch.tensor([16383, 16384, 8191, 0], dtype=torch.int32, device="cuda")
    c["frequency"] = 2.0 ** -10
    _check(ccq_logits_adjust(**c), c, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_a_larger_batch(gpu_lib, dtype):
    """Parts that begin anywhere: only the elements' alignment is asked for."""
    from curvature_conditioned_query_amd import ccq_logits_adjust
    c = _case(5, 1003, 51, 5, dtype, seed=3)
    part = ccq_logits_adjust(**{m: t[1:4] for m, t in c.items()})
    _check(part, {m: t[1:4] for m, t in c.items()}, dtype)
