"""Linear attention, group norm and adjusted logits as a model runs them, with the operators that stand before and behind
them: a prompt, beam search over the carried states and histories, the decode step as a graph, and a training step.

Every stage's inputs are the stage before's stored outputs, so each is compared with its own fp64 definition on the values
it was given: picks and moved rows exactly; attention to (T + d + 16) 2^-24 of a sum's size, and with bf16 inputs another
2^-8 of it for a prompt's rounded scores; normed rows to 2^-17 of their norm; adjusted logits to a few units of their
terms; and each to the half step of its own type, 2^-8 or 2^-24.  Gradients in fp32: 1e-4 normwise, as the read step's.
"""

import numpy as np
import pytest

from oracle import layer, mixer, normwise_error

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H, D, V, K = 2, 64, 1501, 4  # heads, head size, vocabulary, beams
WIDTH = H * D


def _np(t):
    return t.detach().double().cpu().numpy()


class _Model:
    """One layer of linear attention between torch products."""

    def __init__(self, dtype):
        import torch
        g = torch.Generator().manual_seed(21)
        w = lambda *s: (torch.randn(*s, generator=g) / s[0] ** 0.5).to(dtype).cuda()  # noqa: E731
        self.embed = torch.randn(V, WIDTH, generator=g).to(dtype).cuda()
        self.proj, self.decay, self.out = w(WIDTH, 4 * WIDTH), w(WIDTH, H), w(WIDTH, V)
        self.norm = (1 + 0.1 * torch.randn(H, D, generator=g)).cuda()
        self.inv_freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()

    def inputs(self, tokens, positions):
        import torch
        from curvature_conditioned_query_amd import ccq_qk_norm_rope
        e = self.embed[tokens.long()]
        B, T, _ = e.shape
        packed = (e @ self.proj).view(B, T, 4, H, D)
        q, k = ccq_qk_norm_rope(packed[:, :, 0], packed[:, :, 1], positions=positions, inv_freq=self.inv_freq)
        la = torch.nn.functional.logsigmoid((e @ self.decay).float()) / 4
        return dict(q=q.transpose(1, 2), k=k.transpose(1, 2), v=packed[:, :, 2], log_alpha=la), packed[:, :, 3]

    def mix(self, x, gate, S0, S_out, **kw):
        import curvature_conditioned_query_amd as ccq
        o = ccq.ccq_linear_attn(**x, scale=D ** -0.5, S0=S0, S_out=S_out, **kw)
        return o, ccq.ccq_group_norm(o, weight=self.norm, gate=gate, activation="silu")


def _check(m, x, gate, S0, o, y, S, prompt, lengths=None):
    want, last, os, ss = mixer.linear_attn(*(_np(x[n]) for n in "qkv"), _np(x["log_alpha"]), D ** -0.5, S0, lengths)
    live = ~np.isnan(want)
    tol = (want.shape[1] + D + 16) * U
    assert (np.abs(_np(o) - want) <= (tol + 1.01 * 2.0 ** -8 * prompt) * os + 2.0 ** -8 * np.abs(want) + 1e-30)[live].all()
    assert (np.abs(_np(S) - last) <= tol * ss + U * np.abs(last)).all()
    normed = mixer.group_norm(_np(o), _np(m.norm), gate=_np(gate), activation="silu")[0]
    err = np.where(live, np.abs(_np(y) - normed), 0.0)
    size = np.linalg.norm(np.where(live, normed, 0.0), axis=-1, keepdims=True)
    assert (err <= 2.0 ** -8 * np.abs(normed) + 2.0 ** -17 * size + 1e-30)[live].all()


def test_prompt_then_beam_search(gpu_lib):
    import torch
    import curvature_conditioned_query_amd as ccq
    m = _Model(torch.bfloat16)
    N, T, steps = 2, 100, 5
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, V, (N, T), generator=g).cuda()
    n = [T, 71]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    x, gate = m.inputs(prompt, torch.arange(T, device="cuda").expand(N, T).contiguous())
    S = torch.empty(N, H, D, D, device="cuda")
    o, y = m.mix(x, gate, None, S, lengths=lengths, o=torch.zeros(N, T, H, D, dtype=torch.bfloat16, device="cuda"))
    _check(m, x, gate, None, o, y, S, True, n)
    # every beam of a request goes on from its prompt's state and tokens; one beam is alive
    R = N * K
    S = S.repeat_interleave(K, 0).contiguous()
    history = torch.zeros(N, T + steps, dtype=torch.int32, device="cuda")
    history[:, :T] = prompt
    history = history.repeat_interleave(K, 0).contiguous()
    count, first = lengths.repeat_interleave(K), lengths.repeat_interleave(K)
    scores = torch.full((N, K), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    ends = y[torch.arange(N), (lengths - 1).long()]
    logits = (ends.reshape(N, WIDTH) @ m.out).repeat_interleave(K, 0).view(N, K, V).contiguous()
    bias = torch.randint(0, V, (R, 6), generator=g).int().cuda()
    value = torch.randn(R, 6, generator=g).cuda()
    for step in range(steps):
        allowed = torch.randint(-2 ** 31, 2 ** 31, (R, (V + 31) // 32), generator=g).int().cuda()
        how = dict(history=history, lengths=count, prompt_lengths=first, repetition=1.2, presence=0.3, frequency=0.1,
                   bias_token=bias, bias_value=value, allowed=allowed)
        want, size = mixer.logits_adjust(_np(logits).reshape(R, V), **{a: b.cpu().numpy() if hasattr(b, "cpu") else b
                                                                         for a, b in how.items()})
        adjusted = ccq.ccq_logits_adjust(logits, **how)
        got, off = _np(adjusted).reshape(R, V), np.isneginf(want)
        assert np.array_equal(np.isneginf(got), off)
        assert (np.abs(got[~off] - want[~off]) <= (12 * U * size + 2.0 ** -8 * np.abs(want))[~off] + 1e-37).all()
        pick = ccq.ccq_beam_select(adjusted, scores, K)
        t, p, _ = layer.beam_select(_np(adjusted), _np(scores), K, np.zeros((N, K), bool), 0)
        assert np.array_equal(_np(pick["token"]), t) and np.array_equal(_np(pick["parent"]), p)
        before = [S.clone(), history.clone()]
        ccq.ccq_beam_reorder([S, history], pick["parent"])
        for new, old in zip((S, history), before):
            assert np.array_equal(new.cpu().numpy(), layer.beam_reorder(old.cpu().numpy(), p))
        scores = pick["score"]
        tokens = pick["token"].view(R, 1)
        history.scatter_(1, count[:, None].long(), tokens)
        x, gate = m.inputs(tokens, count[:, None].long().contiguous())
        count = count + 1
        S0 = _np(S)
        o, y = m.mix(x, gate, S, S)
        _check(m, x, gate, S0, o, y, S, False)
        logits = (y.reshape(R, WIDTH) @ m.out).view(N, K, V)


def test_decode_step_as_a_graph(gpu_lib):
    """Attention, norm, adjustment, selection and the states' move on static buffers: replays between eager work give
    the eager steps' bits."""
    import torch
    import curvature_conditioned_query_amd as ccq
    N, L = 2, 40
    R = N * K
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    bf = lambda *s: rn(*s).bfloat16()  # noqa: E731
    x = dict(q=bf(R, 1, H, D), k=bf(R, 1, H, D), v=bf(R, 1, H, D), log_alpha=-rn(R, 1, H).abs())
    gate, weight, head = bf(R, 1, H, D), 1 + 0.1 * rn(H, D), (rn(WIDTH, V) / 11).bfloat16()
    history = torch.randint(0, V, (R, L), generator=g).int().cuda()
    scores, S = rn(N, K), rn(R, H, D, D)

    def step():
        o = ccq.ccq_linear_attn(**x, S0=S, S_out=S)
        y = ccq.ccq_group_norm(o, weight=weight, gate=gate, activation="silu")
        logits = ccq.ccq_logits_adjust((y.view(R, WIDTH) @ head).view(N, K, V), history=history, repetition=1.3, presence=0.1)
        pick = ccq.ccq_beam_select(logits, scores, K)
        ccq.ccq_beam_reorder([S, history], pick["parent"])
        scores.copy_(pick["score"])
        return pick["token"], y
    start = [t.clone() for t in (S, history, scores)]
    eager = [[t.clone() for t in (*step(), S, history, scores)] for _ in range(4)]

    def reset():
        for dst, src in zip((S, history, scores), start):
            dst.copy_(src)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    reset()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*out, S, history, scores), want))
        ccq.ccq_group_norm(bf(3, 5, H, D), weight=weight)  # eager work in between


def test_training_step_through_the_layer(gpu_lib):
    """loss = <dy, group norm of the attention of a prepared projection>, back to the packed projection and the decays,
    against the gradients in 64 bits of each stage."""
    import torch
    import curvature_conditioned_query_amd as ccq
    B, T = 2, 70
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(B, T, 4, H, D, generator=g).cuda()
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    la = (torch.nn.functional.logsigmoid(torch.randn(B, T, H, generator=g)) / 4).cuda()
    weight, bias = (1 + 0.1 * torch.randn(H, D, generator=g)).cuda(), (0.1 * torch.randn(H, D, generator=g)).cuda()
    dy = torch.randn(B, T, H, D, generator=g).cuda()
    raw_q, raw_k, v, gate = packed.unbind(2)
    q, k = ccq.ccq_qk_norm_rope(raw_q, raw_k, inv_freq=inv)
    x = dict(q=q.transpose(1, 2), k=k.transpose(1, 2), v=v, log_alpha=la, scale=D ** -0.5)
    norm = dict(weight=weight, bias=bias, gate=gate, center=True, activation="silu")
    o = ccq.ccq_linear_attn(**x)
    grad = torch.empty_like(packed)
    n = ccq.ccq_group_norm_backward(o, dy, dgate=grad[:, :, 3], **norm)
    # head-major gradients of q and k, as the preparation's gradient takes them
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    a = ccq.ccq_linear_attn_backward(**x, d_o=n["dx"], dq=dq.transpose(1, 2), dk=dk.transpose(1, 2), dv=grad[:, :, 2])
    ccq.ccq_qk_norm_rope_backward(raw_q, raw_k, dq, dk, inv_freq=inv, dq=grad[:, :, 0], dk=grad[:, :, 1])

    how = dict(weight=_np(weight), bias=_np(bias), gate=_np(gate), center=True, activation="silu")
    ref_o = mixer.linear_attn(*(_np(x[m]) for m in "qkv"), _np(la), D ** -0.5)[0]
    dx, dgate, dw, db = mixer.group_norm_backward(ref_o, _np(dy), **how)
    back, _ = mixer.linear_attn_backward(*(_np(x[m]) for m in "qkv"), dx, _np(la), D ** -0.5)
    pos = np.arange(T)[None]
    ref_q = layer.norm_rope_backward(_np(raw_q), None, "rms", 1e-6, pos, _np(inv), False, back["dq"].transpose(0, 2, 1, 3))[0]
    ref_k = layer.norm_rope_backward(_np(raw_k), None, "l2", 0, pos, _np(inv), False, back["dk"].transpose(0, 2, 1, 3))[0]
    for got, want, tag in ((grad[:, :, 0], ref_q, "dq"), (grad[:, :, 1], ref_k, "dk"), (grad[:, :, 2], back["dv"], "dv"),
                           (grad[:, :, 3], dgate, "dgate"), (a["dlog_alpha"], back["dlog_alpha"], "dlog_alpha"),
                           (n["dweight"], dw, "dweight"), (n["dbias"], db, "dbias")):
        e = normwise_error(_np(got).reshape(1, 1, -1), want.reshape(1, 1, -1))
        print(f"training step {tag} err {e:.2e}", flush=True)
        assert e <= 1e-4
