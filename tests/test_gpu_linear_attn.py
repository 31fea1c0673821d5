"""ccq_linear_attn and its gradient against the token-by-token fp64 definitions (oracle/mixer.py).

Tolerances.  u = 2^-24.  A fp32 result is a sum over at most T tokens and d channels, each term a product of a few
factors with an error of a unit or two: (T + d + 16) u times the sum's size, the same sum with absolute terms.  With bf16
inputs o also rounds a chunk's scores and the state's copy to bf16 (2^-8 of their part of the size, together 2^-8 of it),
and the result (2^-8 of itself); the gradient keeps scores and states as two bf16 parts (2^-16 each); what enters a state
is three bf16 parts, 2^-24.
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
    return t.detach().double().cpu().numpy()


def _inputs(B, T, H, Hq, Hk, Hv, dk, dv, dtype, gate="bf16", seed=0, state=True, mild=4.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = _dt(dtype)
    x = dict(q=rn(B, T, Hq, dk), k=torch.nn.functional.normalize(rn(B, T, Hk, dk), dim=-1), v=rn(B, T, Hv, dv))
    x = {m: t.to(dt).cuda() for m, t in x.items()}
    x["log_alpha"] = None if gate is None else (torch.nn.functional.logsigmoid(rn(B, T, H) + 1) / mild).to(_dt(gate)).cuda()
    x["S0"] = rn(B, H, dv, dk).cuda() if state else None
    x["scale"] = 0.3
    return x


def _oracle(x, **kw):
    return mixer.linear_attn(*(_np(x[m]) for m in "qkv"), None if x["log_alpha"] is None else _np(x["log_alpha"]), x["scale"],
                             None if x["S0"] is None else _np(x["S0"]), **kw)


def _close(got, want, size, tol, half, tag):
    live = ~np.isnan(want)
    err, bound = np.abs(got - want)[live], (tol * size + half * np.abs(want))[live] + 1e-30
    assert np.isfinite(got[live]).all(), tag
    assert (err <= bound).all(), f"{tag}: {np.max(err / bound):.2f} of the bound"


def _check_forward(x, o, S, dtype, T, step=False, **kw):
    want, last, os, ss = _oracle(x, **kw)
    d = x["q"].shape[-1]
    tol = (T + d + 16) * U
    _close(_np(o), want, os, tol + (1.01 * 2.0 ** -8 if dtype == "bf16" and not step else 0), HALF[dtype], "o")
    if S is not None:
        _close(_np(S), last, ss, tol, U, "S")


SHAPES = [  # B, T, H, Hq, Hk, Hv, dk, dv
    (2, 1, 2, 2, 2, 2, 64, 64), (3, 2, 4, 2, 1, 4, 128, 64), (1, 8, 3, 1, 3, 3, 64, 128), (2, 9, 2, 2, 2, 2, 128, 128),
    (1, 63, 1, 1, 1, 1, 64, 64), (2, 64, 4, 1, 2, 4, 64, 128), (1, 65, 6, 6, 2, 3, 128, 64), (2, 130, 2, 2, 2, 1, 128, 128),
    (9, 200, 1, 1, 1, 1, 64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(gpu_lib, shape, dtype):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    B, T, H, _, _, _, dk, dv = shape
    x = _inputs(*shape, dtype, gate="f32" if T % 2 else dtype, seed=T, state=T != 63)
    S = torch.empty(B, H, dv, dk, device="cuda")
    o = ccq_linear_attn(**x, S_out=S)
    _check_forward(x, o, S, dtype, T, step=T <= 8)


@pytest.mark.parametrize("gate", [None, "bf16", "f32"])
def test_gates(gpu_lib, gate):
    """No decay, strong decay, a decay for each head, zeros (resets) and gates above 1."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    shape = (2, 150, 3, 3, 3, 3, 64, 64)
    for mild in (0.05, 20.0):
        x = _inputs(*shape, "f32", gate=gate, mild=mild, seed=2)
        if gate is not None:
            la = x["log_alpha"]
            la[0, 40], la[0, 64, 0], la[1, 0] = -float("inf"), -float("inf"), -float("inf")
            la[1, 100:104] = 0.5
            x["S0"][1] = float("nan")  # dropped by the first token's gate
        o = ccq_linear_attn(**x)
        _check_forward(x, o, None, "f32", 150)
    if gate is not None:
        x["log_alpha"] = x["log_alpha"][:1, 5:6].expand(2, 150, 3)
        x["S0"][1] = 1.0
        _check_forward(x, ccq_linear_attn(**x), None, "f32", 150)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 100])
def test_lengths(gpu_lib, T, dtype):
    """Rows of no token may hold anything, reach nothing, and are left as they were."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    B, H, d = 5, 2, 64
    n = [T, 0, T - 1, 1, T + 7]
    x = _inputs(B, T, H, H, H, H, d, d, dtype, seed=3)
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    for m in ("q", "k", "v", "log_alpha"):
        for b in range(B):
            x[m][b, n[b]:] = float("nan")
    o = torch.full((B, T, H, d), 7.0, dtype=_dt(dtype), device="cuda")
    S = torch.empty(B, H, d, d, device="cuda")
    ccq_linear_attn(**x, lengths=lengths, o=o, S_out=S)
    _check_forward(x, o, S, dtype, T, step=T <= 8, lengths=n)
    for b in range(B):
        assert (o[b, n[b]:] == 7.0).all()
    assert torch.equal(S[1], x["S0"][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("most", [200, 70])
def test_packed(gpu_lib, dtype, most):
    """Sequences one behind the other, an empty one, rows before the first and behind the last, and one longer than
    max_length, of which the first tokens count."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    at = [3, 3, 133, 134, 300]
    rows, B, H, d = 310, 4, 2, 64
    x = _inputs(1, rows, H, H, 1, H, d, 128, dtype, seed=4, state=False)
    S0 = torch.randn(B, H, 128, d, generator=torch.Generator().manual_seed(1)).cuda()
    o = torch.full((1, rows, H, 128), 5.0, dtype=_dt(dtype), device="cuda")
    S = torch.empty_like(S0)
    kw = dict(offsets=torch.tensor(at, dtype=torch.int32, device="cuda"), max_length=most)
    ccq_linear_attn(**{**x, "S0": S0}, o=o, S_out=S, **kw)
    touched = torch.zeros(rows, dtype=torch.bool)
    for b in range(B):
        n = min(at[b + 1] - at[b], most)
        sl = slice(at[b], at[b] + n)
        touched[sl] = True
        if n == 0:
            assert torch.equal(S[b], S0[b])
            continue
        part = {m: x[m][:, sl] for m in ("q", "k", "v", "log_alpha")}
        _check_forward({**part, "S0": S0[b:b + 1], "scale": x["scale"]}, o[:, sl], S[b:b + 1], dtype, n)
    assert (o[0, ~touched.cuda()] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views(gpu_lib, dtype):
    """Parts of a packed projection, head-major rows, a gate inside another tensor, o as part of a wider one."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    B, T, H, d = 2, 70, 2, 64
    x = _inputs(B, T, H, H, H, H, d, d, dtype, seed=5)
    packed = torch.empty(B, T, 3 * H * d, dtype=_dt(dtype), device="cuda")
    q, k = packed[..., : H * d].view(B, T, H, d), packed[..., H * d : 2 * H * d].view(B, T, H, d)
    v = torch.empty(B, H, T, d, dtype=_dt(dtype), device="cuda").transpose(1, 2)
    la = torch.empty(B, H, 3, T, dtype=_dt(dtype), device="cuda")[:, :, 1].transpose(1, 2)
    for dst, m in ((q, "q"), (k, "k"), (v, "v"), (la, "log_alpha")):
        dst.copy_(x[m])
    wide = torch.full((B, T, H, 2 * d), 3.0, dtype=_dt(dtype), device="cuda")
    o = ccq_linear_attn(q, k, v, la, x["scale"], x["S0"], o=wide[..., d:])
    want = ccq_linear_attn(**x)
    assert torch.equal(o, want) and (wide[..., :d] == 3.0).all() and o.data_ptr() == wide[..., d:].data_ptr()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1000, 2049])
def test_long_sequences_cut_and_joined(gpu_lib, T, dtype):
    """Few heads: the sequence is cut along its tokens; the state in place; lengths that leave pieces empty."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    B, H, dk, dv = 3, 1, 64, 64
    x = _inputs(B, T, H, H, H, H, dk, dv, dtype, seed=6, mild=30.0)
    n = [T, 5, 0]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    S = x["S0"].clone()
    o = torch.zeros(B, T, H, dv, dtype=_dt(dtype), device="cuda")
    ccq_linear_attn(**{**x, "S0": S}, S_out=S, o=o, lengths=lengths)
    _check_forward(x, o, S, dtype, T, lengths=n)
    again, S2 = torch.zeros_like(o), torch.empty_like(S)
    ccq_linear_attn(**x, S_out=S2, o=again, lengths=lengths)
    assert torch.equal(again, o) and torch.equal(S2, S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_single_tokens(gpu_lib, dtype):
    """A prompt's state goes on token by token, in place, as one longer prompt would."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    B, T, H, d, first = 2, 80, 2, 128, 72
    x = _inputs(B, T, H, H, H, H, d, d, dtype, seed=7, state=False)
    part = lambda a, b: {m: x[m][:, a:b] for m in ("q", "k", "v", "log_alpha")}  # noqa: E731
    S = torch.empty(B, H, d, d, device="cuda")
    outs = [ccq_linear_attn(**part(0, first), scale=x["scale"], S_out=S)]
    for t in range(first, T):
        outs.append(ccq_linear_attn(**part(t, t + 1), scale=x["scale"], S0=S, S_out=S))
    _check_forward(x, torch.cat(outs, 1), S, dtype, T)


BACK = [  # B, T, H, Hq, Hk, Hv, dk, dv
    (1, 1, 1, 1, 1, 1, 64, 64), (2, 5, 2, 2, 2, 2, 128, 64), (2, 64, 4, 2, 1, 4, 64, 128), (1, 65, 6, 6, 2, 3, 64, 64),
    (2, 130, 2, 2, 2, 1, 128, 128), (1, 600, 1, 1, 1, 1, 64, 64), (9, 70, 1, 1, 1, 1, 128, 64)]


def _check_back(x, got, d_o, dS, dtype, grad, T, **kw):
    d = x["q"].shape[-1] + x["v"].shape[-1]
    want, size = mixer.linear_attn_backward(*(_np(x[m]) for m in "qkv"), _np(d_o), None if x["log_alpha"] is None else _np(x["log_alpha"]),
                                            x["scale"], None if x["S0"] is None else _np(x["S0"]), None if dS is None else _np(dS), **kw)
    tol = (T + d + 16) * U
    split = 2.1 * 2.0 ** -16 if dtype == "bf16" else 0.0
    heads = x["log_alpha"].shape[2] if x["log_alpha"] is not None else d_o.shape[2]
    for m in ("dq", "dk", "dv"):
        _close(_np(got[m]), want[m], size[m], tol + split + heads * U, HALF[grad], m)
    if "dS0" in got:
        _close(_np(got["dS0"]), want["dS0"], size["dS0"], tol, U, "dS0")
    if "dlog_alpha" in got:
        half = HALF["bf16" if "bfloat16" in str(got["dlog_alpha"].dtype) else "f32"]
        _close(_np(got["dlog_alpha"]), want["dlog_alpha"], size["dlog_alpha"], tol + split, half, "dlog_alpha")


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("shape", BACK)
def test_backward(gpu_lib, shape, dtype, grad):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    B, T, H, _, _, _, dk, dv = shape
    x = _inputs(*shape, dtype, gate="f32" if T % 2 else dtype, seed=T, state=T != 64)
    g = torch.Generator().manual_seed(T)
    d_o = torch.randn(B, T, H, dv, generator=g).to(_dt(dtype)).cuda()
    dS = torch.randn(B, H, dv, dk, generator=g).cuda() if T != 5 else None
    got = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS, want_dS0=True, grad_dtype=_dt(grad))
    assert got["dq"].dtype == _dt(grad)
    _check_back(x, got, d_o, dS, dtype, grad, T)
    twice = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS, want_dS0=True, grad_dtype=_dt(grad))
    assert all(torch.equal(got[m], twice[m]) for m in got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [1, 2])
def test_backward_of_lengths_and_packed_sequences(gpu_lib, dtype, share):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    B, T, H, d = 4, 90, 2, 64
    n = [T, 0, 65, 1]
    x = _inputs(B, T, H, H // share, H, H // share, d, d, dtype, seed=8)
    d_o = torch.randn(B, T, H, d, generator=torch.Generator().manual_seed(2)).to(_dt(dtype)).cuda()
    dS = torch.randn(B, H, d, d, generator=torch.Generator().manual_seed(3)).cuda()
    x["log_alpha"][0, 70] = -float("inf")
    rows = {m: torch.cat([x[m][b, :n[b]] for b in range(B)])[None] for m in ("q", "k", "v", "log_alpha")}
    rows_o = torch.cat([d_o[b, :n[b]] for b in range(B)])[None]
    for m in ("q", "k", "v", "log_alpha"):
        for b in range(B):
            x[m][b, n[b]:] = float("nan")
    for b in range(B):
        d_o[b, n[b]:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    got = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS, want_dS0=True, lengths=lengths)
    _check_back(x, got, d_o, dS, dtype, dtype, T, lengths=n)
    for m in ("dq", "dk", "dv", "dlog_alpha"):
        assert all((got[m][b, n[b]:] == 0).all() for b in range(B)), m
    assert (got["dlog_alpha"][0, 70] == 0).all()
    offsets = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    packed = ccq_linear_attn_backward(**rows, scale=x["scale"], S0=x["S0"], d_o=rows_o, dS_out=dS, want_dS0=True, offsets=offsets,
                                      max_length=T)
    for m in ("dq", "dk", "dv", "dlog_alpha"):
        assert torch.equal(packed[m][0], torch.cat([got[m][b, :n[b]] for b in range(B)])), m
    assert torch.equal(packed["dS0"], got["dS0"])


def test_backward_into_one_packed_gradient(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    B, T, H, d = 2, 70, 2, 64
    x = _inputs(B, T, H, H, H, H, d, d, "bf16", seed=9)
    d_o = torch.randn(B, H, T, d, device="cuda").bfloat16().transpose(1, 2)
    packed = torch.empty(B, T, 3, H, d, dtype=torch.bfloat16, device="cuda")
    got = ccq_linear_attn_backward(**x, d_o=d_o, dq=packed[:, :, 0], dk=packed[:, :, 1], dv=packed[:, :, 2])
    want = ccq_linear_attn_backward(**x, d_o=d_o.contiguous())
    for i, m in enumerate(("dq", "dk", "dv")):
        assert torch.equal(packed[:, :, i], want[m]) and got[m].data_ptr() == packed[:, :, i].data_ptr()
    assert "dS0" not in got
    x["log_alpha"] = None
    got = ccq_linear_attn_backward(**x, d_o=d_o)
    assert "dlog_alpha" not in got
    _check_back(x, got, d_o, None, "bf16", "bf16", T)


def test_gradient_by_differences(gpu_lib):
    """q, k, v and the state enter linearly, so a central difference is exact; along one token's gate a term is A + B e^s,
    whose difference is B sinh(s) / s.  The outputs' roundings, over the step, are what is left."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    B, T, H, d, step = 1, 100, 2, 64, 0.25
    x = _inputs(B, T, H, 1, H, H, d, d, "f32", gate="f32", seed=10)
    g = torch.Generator().manual_seed(4)
    d_o, dS = torch.randn(B, T, H, d, generator=g).cuda(), torch.randn(B, H, d, d, generator=g).cuda()
    got = ccq_linear_attn_backward(**x, d_o=d_o, dS_out=dS, want_dS0=True)
    S = torch.empty_like(dS)

    def loss(**kw):
        o = ccq_linear_attn(**{**x, **kw}, S_out=S)
        return float((o.double() * d_o.double()).sum() + (S.double() * dS.double()).sum())
    for m, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0"), ("log_alpha", "dlog_alpha")):
        u = torch.zeros_like(x[m])
        if m == "log_alpha":
            u[0, 37, 1] = 1.0
        else:
            u.copy_((torch.randn(u.shape, generator=g) > 0).float() * 2 - 1)
        up, down = {**x, m: x[m] + step * u}, {**x, m: x[m] - step * u}
        size = sum((np.abs(_np(d_o)) * r[2]).sum() + (np.abs(_np(dS)) * r[3]).sum() for r in (_oracle(up), _oracle(down)))
        want = (loss(**{m: up[m]}) - loss(**{m: down[m]})) / (2 * step)
        mine = float((got[name].double() * u.double()).sum()) * (np.sinh(step) / step if m == "log_alpha" else 1.0)
        # each output is off by (T + d + 16) u of its size, and so is the gradient; random signs leave far less
        assert abs(want - mine) <= 2 * (T + d + 16) * U * size / (2 * step), (m, want, mine)


def test_streams_and_graphs(gpu_lib):
    """On another stream, and replayed from two graphs that run one after the other, with eager calls between."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    B, T, H, d = 1, 1500, 2, 64
    x = _inputs(B, T, H, H, H, H, d, d, "bf16", seed=11)
    d_o = torch.randn(B, T, H, d, device="cuda").bfloat16()
    want, back = ccq_linear_attn(**x), ccq_linear_attn_backward(**x, d_o=d_o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = ccq_linear_attn(**x, stream=side)
    side.synchronize()
    assert torch.equal(o, want)
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                r = (ccq_linear_attn(**x), ccq_linear_attn_backward(**x, d_o=d_o))
            graphs.append((g, r))
    for _ in range(3):
        for g, r in graphs:
            r[0].zero_()
            for t in r[1].values():
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(r[0], want) and all(torch.equal(r[1][m], back[m]) for m in back)
            assert torch.equal(ccq_linear_attn(**x), want)


def test_binding_refusals_on_device(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import CcqError, ccq_linear_attn, ccq_linear_attn_backward
    x = _inputs(1, 20, 2, 2, 2, 2, 64, 64, "bf16")
    bad = [dict(q=x["q"].half()), dict(k=x["k"][:, :10]), dict(v=x["v"].float()), dict(log_alpha=x["log_alpha"][:, :, :1]),
           dict(log_alpha=x["log_alpha"].half()), dict(S0=x["S0"][:, :1]), dict(S0=x["S0"].bfloat16()),
           dict(lengths=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(lengths=torch.zeros(1, dtype=torch.int64, device="cuda")),
           dict(offsets=torch.zeros(1, dtype=torch.int32, device="cuda")), dict(max_length=5), dict(q=x["q"][..., ::2]),
           dict(q=x["q"][:, :, :1].expand(1, 20, 3, 64)), dict(o=torch.empty(1, 20, 2, 64, device="cuda")), dict(S_out=x["S0"].cpu())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            ccq_linear_attn(**{**x, **kw})
    with pytest.raises(CcqError):
        ccq_linear_attn(**{**x, "scale": float("nan")})
    both = torch.zeros(2 * 64 * 64 + 4, device="cuda")
    with pytest.raises(CcqError):
        ccq_linear_attn(**{**x, "S0": both[:-4].view(1, 2, 64, 64)}, S_out=both[4:].view(1, 2, 64, 64))
    with pytest.raises(CcqError):
        ccq_linear_attn(**x, o=x["q"])
    with pytest.raises((ValueError, TypeError)):
        ccq_linear_attn_backward(**x, d_o=x["v"].float())
    with pytest.raises(TypeError):
        ccq_linear_attn_backward(**x, d_o=x["v"], grad_dtype=torch.float16)
