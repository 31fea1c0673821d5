"""ccq_scan and its gradient on the GPU against their token-by-token fp64 definitions.

Tolerances.  u = 2^-24.  A step of the recurrence rounds the gate (exp, within 4 u), the product, the
scaled input (at most 4 u) and the sum: under 10 u of alpha_t A_{t-1} + |s_t x_t|, A the recurrence of
the absolute values; an error made once is carried on by the gates, as the oracle's majorant E carries
it.  Pieces that are joined multiply their gates and then the state, which rounds each gate's product
once: the same bound a step.  So |error| <= 10 u E, and half a step of the stored type (2^-8 of the
value for bf16).  The gradient has the same bound with its own majorants, twice over where an adjoint
meets a state (20 u).
"""

import numpy as np
import pytest

from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": 0.0}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(got, want, size, dtype, units, tag):
    got = _np(got)
    live = ~np.isnan(want)
    err = np.abs(got - want)[live]
    tol = (units * U * size + STEP[dtype] * (np.abs(want) + units * U * size) + 1e-37)[live]
    assert not (err > tol).any(), f"{tag}: worst {np.max(err / tol):.2f} of the tolerance"


def _make(dtype, B, T, D, seed, decay=1 / 8, h0=True, lengths=None):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, D, generator=g).to(dt).cuda()
    la = (torch.nn.functional.logsigmoid(torch.randn(B, T, D, generator=g)) * decay).to(dt).cuda()
    h = torch.randn(B, D, generator=g).cuda() if h0 else None
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return x, la, h, n


def _both(dtype, x, la, h0, n, complement, keep=True, tag=""):
    """Forward with its chunk carries, and the gradient from them and without them."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward, scan_carry_shape
    B, T, D = x.shape
    y = torch.full((B, T, D), 7.0, dtype=x.dtype, device="cuda")
    h = torch.empty(B, D, device="cuda")
    carry = torch.empty(scan_carry_shape(x), device="cuda")
    assert ccq_scan(x, la, h0=h0, h_out=h, y=y, lengths=n, complement=complement, chunk_carry=carry) is y
    lens = None if n is None else n.tolist()
    hs, last, es, last_err = layer.scan(_np(x), _np(la), _np(h0), lens, complement)
    _check(y, hs, es, dtype, 10, tag + "y")
    assert (y[torch.from_numpy(np.isnan(hs)).cuda()] == 7.0).all(), "a row behind its length was written"
    _check(h, last, last_err, "f32", 10, tag + "h")
    for c in range(carry.shape[1]):
        for b in range(B):
            if 64 * c < (T if lens is None else lens[b]):
                want = hs[b, 64 * c - 1] if c else (np.zeros(D) if h0 is None else _np(h0)[b])
                size = es[b, 64 * c - 1] if c else np.zeros(D)
                _check(carry[b, c], want, size, "f32", 10, tag + "carry")
    g = torch.Generator().manual_seed(99)
    dy = torch.randn(B, T, D, generator=g).to(x.dtype).cuda()
    dh = torch.randn(B, D, generator=g).cuda()
    want = layer.scan_backward(_np(x), _np(la), _np(dy), _np(h0), _np(dh), lens, complement)
    for given in (carry, None):
        out = ccq_scan_backward(x, la, dy, h0=h0, dh_out=dh, lengths=n, complement=complement, chunk_carry=given, want_dh0=True)
        for i, name in enumerate(("dx", "dlog_alpha", "dh0")):
            _check(out[name], want[i], want[3 + i], "f32" if name == "dh0" else dtype, 20, f"{tag}{name} kept={given is not None} ")
    return y, h


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (3, 2, 24), (2, 63, 64), (1, 64, 72), (2, 65, 200), (1, 127, 128), (1, 257, 8),
                                   (2, 513, 136), (1, 1500, 64)])
def test_forward_and_backward(gpu_lib, dtype, complement, B, T, D):
    print(f"scan {dtype} complement={complement} B{B} T{T} D{D}", flush=True)
    x, la, h0, _ = _make(dtype, B, T, D, 1 + T)
    _both(dtype, x, la, h0, None, complement)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lengths", [(300, [0, 1, 300, 64, 65]), (1100, [1100, 255, 256, 257, 1024]), (70, [-5, 99, 70, 2, 0])])
def test_lengths(gpu_lib, dtype, T, lengths):
    """Empty sequences, single tokens, ends at and beside a piece's end, lengths outside 0 .. T."""
    print(f"scan lengths {dtype} T{T} {lengths}", flush=True)
    x, la, h0, n = _make(dtype, len(lengths), T, 40, 5, lengths=lengths)
    for b, k in enumerate(lengths):
        x[b, max(0, k):] = float("nan")
        la[b, max(0, k):] = float("inf")
    _both(dtype, x, la, h0, n, True)


@pytest.mark.parametrize("dtype,complement", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_short_sequences_among_long_ones(gpu_lib, dtype, complement):
    """Many tiles behind a sequence's end, beginning or ending a group of them, and not a multiple of a group."""
    T, lengths = 4700, [0, 1, 4700, 2048, 2049, 130, 4601]
    print(f"scan lengths {dtype} T{T} {lengths}", flush=True)
    x, la, h0, n = _make(dtype, len(lengths), T, 136, 6, lengths=lengths)
    for b, k in enumerate(lengths):
        x[b, k:] = float("nan")
        la[b, k:] = float("inf")
    _both(dtype, x, la, h0, n, complement)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9, 64, 65])
@pytest.mark.parametrize("state", [True, False])
def test_gradient_of_one_chunk(gpu_lib, dtype, T, state):
    """Up to 64 tokens the gradient needs no state but h0, which may be absent; beyond, it forms them."""
    print(f"scan one chunk {dtype} T{T} h0={state}", flush=True)
    x, la, h0, n = _make(dtype, 3, T, 136, 7, h0=state, lengths=[T, T // 2, 0])
    _both(dtype, x, la, h0, n, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,T,D", [(70, 9, 136), (33, 17, 8), (9, 33, 264), (40, 4, 128), (130, 1, 72), (5, 48, 640)])
def test_many_short_sequences(gpu_lib, dtype, complement, B, T, D):
    """Several sequences a workgroup: lengths from 0 to T beside each other, resets in some of them."""
    print(f"scan short {dtype} B{B} T{T} D{D}", flush=True)
    lengths = [(7 * b) % (T + 1) for b in range(B)]
    x, la, h0, n = _make(dtype, B, T, D, 8, lengths=lengths)
    la[1::3, T // 2, ::5] = -float("inf")
    for b, k in enumerate(lengths):
        x[b, k:] = float("nan")
        la[b, k:] = float("inf")
    _both(dtype, x, la, h0, n, complement)


@pytest.mark.parametrize("T", [1, 7, 20, 64])
def test_short_sequences_in_place(gpu_lib, T):
    """h_out over h0, which other threads of the sequence read."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan
    x, la, h0, _ = _make("bf16", 50, T, 256, 9)
    h, apart = h0.clone(), torch.empty_like(h0)
    y = ccq_scan(x, la, h0=h0, h_out=apart)
    assert torch.equal(ccq_scan(x, la, h0=h, h_out=h), y) and torch.equal(h, apart)


@pytest.mark.parametrize("decay", [1e-5, 20.0])
def test_slow_and_fast_gates(gpu_lib, decay):
    """Gates next to 1 (nothing is lost over the whole length) and gates that forget within a token."""
    x, la, h0, _ = _make("f32", 1, 900, 64, 6, decay=decay)
    _both("f32", x, la, h0, None, False)
    _both("f32", x, la, h0, None, True)


@pytest.mark.parametrize("where", [0, 1, 100, 255, 256, 700])
def test_reset_drops_what_came_before(gpu_lib, where):
    """log_alpha = -inf at one token: NaN and infinities before it do not pass, in no direction."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    x, la, h0, _ = _make("f32", 2, 800, 64, 7)
    la[:, where] = -float("inf")
    want = ccq_scan(x[:, where:], la[:, where:])
    dy, dh = torch.randn_like(x), torch.randn(2, 64, device="cuda")
    clean = ccq_scan_backward(x, la, dy, h0=h0, dh_out=dh, want_dh0=True)
    x[:, :where] = float("nan")
    h0[:] = float("inf")
    y = ccq_scan(x, la, h0=h0)
    assert torch.isfinite(y[:, where:]).all()
    hs, _, es, _ = layer.scan(_np(x[:, where:]), _np(la[:, where:]), None, None, False)
    _check(y[:, where:], hs, es, "f32", 10, "y")
    _check(want, hs, es, "f32", 10, "y alone")
    out = ccq_scan_backward(x, la, dy, h0=h0, dh_out=dh, want_dh0=True)
    for name in ("dx", "dlog_alpha"):
        assert torch.isfinite(out[name][:, where:]).all()
    assert (out["dlog_alpha"][:, where] == 0).all()
    assert torch.equal(out["dx"], clean["dx"])  # the adjoint does not see the states
    if where == 0:
        assert (out["dh0"] == 0).all()


def test_an_infinity_or_nan_stays_until_a_reset(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_scan
    x, la, h0, _ = _make("f32", 1, 1000, 64, 8, decay=2.0)
    x[0, 3, 0], x[0, 5, 1] = float("inf"), float("nan")
    y = ccq_scan(x, la, h0=h0)
    assert (y[0, 3:, 0] == float("inf")).all() and y[0, 5:, 1].isnan().all() and torch.isfinite(y[0, :, 2:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs(gpu_lib, dtype):
    """Parts of a packed projection, a time-major tensor, and inputs shared by all sequences (stride 0)."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    B, T, D = 2, 90, 48
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    packed = torch.randn(B, T, 3 * D).to(dt).cuda()
    x = packed[..., D : 2 * D]
    la = -torch.rand(T, B, D).to(dt).cuda().transpose(0, 1)
    assert torch.equal(ccq_scan(x, la), ccq_scan(x.contiguous(), la.contiguous()))
    one = -torch.rand(1, T, D).to(dt).cuda().expand(B, T, D)
    dy = packed[..., 2 * D :]
    a, b = ccq_scan_backward(x, one, dy), ccq_scan_backward(x.contiguous(), one.contiguous(), dy.contiguous())
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dlog_alpha"], b["dlog_alpha"])


def test_steps_continue_a_prefill_in_place(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_scan
    x, la, h0, _ = _make("f32", 3, 131, 64, 9)
    hs, _, es, _ = layer.scan(_np(x), _np(la), _np(h0), None, True)
    h = h0.clone()
    _check(ccq_scan(x[:, :100], la[:, :100], h0=h, h_out=h, complement=True), hs[:, :100], es[:, :100], "f32", 10, "prefill")
    for t in range(100, 131):
        y = ccq_scan(x[:, t : t + 1], la[:, t : t + 1], h0=h, h_out=h, complement=True)
        _check(y, hs[:, t : t + 1], es[:, t : t + 1], "f32", 10, f"step {t}")
        assert torch.equal(y[:, 0], h)


def test_many_sequences_and_channels_run_again_alike(gpu_lib):
    """A size that is cut along T and over many workgroups: bit for bit the same twice, forward and back,
    and right at sampled channels."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    x, la, h0, _ = _make("bf16", 2, 5000, 1032, 10)
    h = torch.empty_like(h0)
    y = ccq_scan(x, la, h0=h0, h_out=h)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).to(x.dtype).cuda()
    out = ccq_scan_backward(x, la, dy, h0=h0, want_dh0=True)
    for _ in range(2):
        assert torch.equal(y, ccq_scan(x, la, h0=h0))
        more = ccq_scan_backward(x, la, dy, h0=h0, want_dh0=True)
        assert all(torch.equal(out[n], more[n]) for n in out)
    at = [0, 7, 63, 64, 512, 1024, 1031]
    hs, last, es, le = layer.scan(_np(x[..., at]), _np(la[..., at]), _np(h0[:, at]), None, False)
    _check(y[..., at], hs, es, "bf16", 10, "y")
    _check(h[:, at], last, le, "f32", 10, "h")
    want = layer.scan_backward(_np(x[..., at]), _np(la[..., at]), _np(dy[..., at]), _np(h0[:, at]), None, None, False)
    _check(out["dx"][..., at], want[0], want[3], "bf16", 20, "dx")
    _check(out["dlog_alpha"][..., at], want[1], want[4], "bf16", 20, "dlog_alpha")
    _check(out["dh0"][:, at], want[2], want[5], "f32", 20, "dh0")


@pytest.mark.parametrize("T", [1, 700])
def test_other_stream_and_replayed_capture(gpu_lib, T):
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    x, la, h0, _ = _make("bf16", 2, T, 256, 11)
    dy = torch.randn_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = ccq_scan(x, la, h0=h0)
    got = ccq_scan(x, la, h0=h0, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ccq_scan(x, la, h0=h0)
        out = ccq_scan_backward(x, la, dy, h0=h0, want_dh0=True)
    for _ in range(4):
        x.copy_(torch.randn_like(x))
        want, back = ccq_scan(x, la, h0=h0), ccq_scan_backward(x, la, dy, h0=h0, want_dh0=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, y) and all(torch.equal(back[n], out[n]) for n in out)


def test_two_streams_at_once(gpu_lib):
    """Calls in flight together, each with its own workspace, do not see each other."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan
    sets = [_make("bf16", 2, 3000, 512, 20 + i) for i in range(4)]
    want = [ccq_scan(x, la, h0=h0) for x, la, h0, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got = [ccq_scan(x, la, h0=h0, stream=s) for s, (x, la, h0, _) in zip(streams, sets)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [1e-8, 1e-7, 1e-5, 1e-3, 0.05])
@pytest.mark.parametrize("T", [8, 9, 64, 65, 700])
def test_complement_of_gates_next_to_one(gpu_lib, dtype, decay, T):
    """From no state, a channel holds (1 - alpha) x, which keeps its own relative rounding however small 1 - alpha is;
    also where one token's input is far above the others',
    and the gradient at tokens without an input, which see that state alone."""
    x, la, _, _ = _make(dtype, 2, T, 64, 12, decay=decay, h0=False)
    x[0, 1::2] = 0
    x[1, T // 2] *= 512
    x[1, T // 2 + 1 :: 3] = 0
    _both(dtype, x, la, None, None, True, tag=f"decay {decay} ")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [8, 30, 64, 300])
@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), 200.0])
def test_reset_beside_a_gate_that_is_no_number(gpu_lib, dtype, T, bad):
    """A NaN or infinite gate just before a reset, or just behind it, at every place of a thread's run: the states
    behind the reset do not see the first, the adjoints before it do not see the second."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward

    def gradient(part, tag):
        out = ccq_scan_backward(x, la, dy, h0=h0, dh_out=dh, complement=complement, want_dh0=True)
        want = layer.scan_backward(_np(x), _np(la), _np(dy), _np(h0), _np(dh), None, complement)
        for i, name in enumerate(("dx", "dlog_alpha")):
            got = out[name][:, part]
            assert torch.isfinite(got).all() and np.isfinite(want[i][:, part]).all(), (tag, name)
            _check(got, want[i][:, part], want[3 + i][:, part], dtype, 20, f"{tag} {name} ")
        return out["dh0"], want[2], want[5]

    for where in range(max(1, T // 2 - 3), T // 2 + 2):
        for complement in (False, True):
            tag = f"reset at {where} complement={complement}"
            x, clean, h0, _ = _make(dtype, 1, T, 24, where)
            clean[:, where, ::2] = -float("inf")
            dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(x.dtype).cuda()
            dh = torch.randn(1, 24, generator=torch.Generator().manual_seed(3)).cuda()
            want_y = ccq_scan(x, clean, h0=h0, complement=complement)
            la = clean.clone()
            la[:, where - 1, ::2] = bad
            y = ccq_scan(x, la, h0=h0, complement=complement)
            assert torch.equal(y[:, where:], want_y[:, where:]), tag
            gradient(slice(where, T), tag + ", before it")
            if where + 1 < T:
                la = clean.clone()
                la[:, where + 1, ::2] = bad
                got, want, size = gradient(slice(0, where), tag + ", behind it")
                assert torch.isfinite(got).all(), tag
                _check(got, want, size, "f32", 20, tag + " dh0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("T", [8, 60, 64, 300, 2500])
def test_gates_above_one_leave_a_zero_state_alone(gpu_lib, dtype, complement, T):
    """The gates' product passes every number, but there is no state to grow: inputs and gradients only at a few tokens."""
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    x, la, _, _ = _make(dtype, 2, T, 72, 13, h0=False)
    la[:] = 1.5
    x[:, : T - 5] = 0
    y = ccq_scan(x, la, complement=complement)
    hs, _, es, _ = layer.scan(_np(x), _np(la), None, None, complement)
    _check(y, hs, es, dtype, 10, "y")
    assert (y[:, : T - 5] == 0).all()
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(x.dtype).cuda()
    dy[:, 5:] = 0
    out = ccq_scan_backward(x, la, dy, complement=complement, want_dh0=True)
    want = layer.scan_backward(_np(x), _np(la), _np(dy), None, None, None, complement)
    for i, name in enumerate(("dx", "dlog_alpha", "dh0")):
        assert torch.isfinite(out[name]).all(), name
        _check(out[name], want[i], want[3 + i], "f32" if name == "dh0" else dtype, 20, name)
    assert (out["dx"][:, 5:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 30, 64, 65, 300, 2500])
def test_gradient_of_the_state_in_place(gpu_lib, dtype, T):
    """dh0 over dh_out, through the C interface: the serving step's counterpart in training by pieces."""
    import ctypes
    import torch
    from curvature_conditioned_query_amd import ccq_scan_backward
    from curvature_conditioned_query_amd.binding import ScanBwdParams
    for complement in (0, 1):
        x, la, h0, n = _make(dtype, 3, T, 136, 14, lengths=[T, T // 2, 0])
        dy, dh = torch.randn_like(x), torch.randn_like(h0)
        want = ccq_scan_backward(x, la, dy, h0=h0, dh_out=dh, lengths=n, complement=bool(complement), want_dh0=True)
        dx, dg = torch.empty_like(x), torch.empty_like(x)
        p = ScanBwdParams(dtype=1 if dtype == "bf16" else 0, B=3, T=T, D=136, complement=complement, x=x.data_ptr(),
                          log_alpha=la.data_ptr(), dy=dy.data_ptr(), lengths=n.data_ptr(), h0=h0.data_ptr(), dh_out=dh.data_ptr(),
                          dx=dx.data_ptr(), dlog_alpha=dg.data_ptr(), dh0=dh.data_ptr())
        for name in ("x", "la", "dy"):
            setattr(p, name + "_stride_b", T * 136)
            setattr(p, name + "_stride_t", 136)
        need = gpu_lib.ccq_scan_backward_workspace_bytes(ctypes.byref(p))
        work = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
        p.workspace, p.workspace_bytes = work.data_ptr(), need
        assert gpu_lib.ccq_scan_backward(ctypes.byref(p), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(dx, want["dx"]) and torch.equal(dg, want["dlog_alpha"]) and torch.equal(dh, want["dh0"])
