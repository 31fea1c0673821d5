"""The operators as a model runs them: a prompt through the query/key preparation, the read step and the
gated recurrence; beam search over the carried states of both; and a training step back through them.

Every stage's inputs are the stage before's stored outputs, so each is compared with its own fp64
definition on the values it was given: picks and moved states exactly, the rest to the bars of the
read step's own tests (2e-2 normwise with bf16 inputs, 1e-4 with fp32) or of the operators' own tests.
"""

import numpy as np
import pytest

import oracle
from oracle import layer, normwise_error

pytestmark = pytest.mark.gpu

H, D, V, K = 2, 128, 2003, 4  # heads, head size, vocabulary, beams


def _np(t):
    return t.double().cpu().numpy()


class _Model:
    """One read-step layer beside one gated recurrence, and an output projection (torch products)."""

    def __init__(self, dtype):
        import torch
        g = torch.Generator().manual_seed(42)
        w = lambda *s: (torch.randn(*s, generator=g) / s[0] ** 0.5).to(dtype).cuda()  # noqa: E731
        width = H * D
        self.embed = torch.randn(V, width, generator=g).to(dtype).cuda()
        self.qkv, self.gates, self.xg, self.out = w(width, 3 * width), w(width, width), w(width, 2 * width), w(width, V)
        self.inv_freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        self.w_lam, self.b_lam = (torch.randn(H, D, generator=g) / D ** 0.5).cuda(), torch.full((H,), -2.0).cuda()

    def inputs(self, tokens, positions):
        """q, k, v, log_alpha of the read step and x, log_alpha of the recurrence, for tokens [B, T]."""
        import torch
        from curvature_conditioned_query_amd import ccq_qk_norm_rope
        e = self.embed[tokens.long()]
        B, T, _ = e.shape
        packed = (e @ self.qkv).view(B, T, 3, H, D)
        q, k = ccq_qk_norm_rope(packed[:, :, 0], packed[:, :, 1], positions=positions, inv_freq=self.inv_freq)
        _, v = ccq_qk_norm_rope(None, packed[:, :, 2], k_norm="none")
        a = torch.nn.functional.logsigmoid((e @ self.gates).float()) / 16
        a = a.to(e.dtype).view(B, T, H, D).transpose(1, 2).contiguous()
        xg = e @ self.xg
        return packed, q, k, v, a, xg[..., : H * D], -torch.nn.functional.softplus(xg[..., H * D :]) / 4


def test_prompt_then_beam_search(gpu_lib):
    import torch
    import curvature_conditioned_query_amd as ccq
    m = _Model(torch.bfloat16)
    N, T = 2, 100
    prompt = torch.randint(0, V, (N, T), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.arange(T, device="cuda").expand(N, T).contiguous()
    packed, q, k, v, a, x, xa = m.inputs(prompt, pos)
    want, _ = layer.norm_rope(_np(packed[:, :, 1]), None, "l2", 0.0, _np(pos), _np(m.inv_freq), False)
    assert normwise_error(_np(k), want) <= 2e-2 and torch.equal(v, packed[:, :, 2].transpose(1, 2))
    S, C, ks = torch.empty(N, H, D, D).cuda(), torch.empty(N, H, D, D).cuda(), torch.empty(N, H, D).cuda()
    n = torch.empty(N, H, dtype=torch.int64).cuda()
    h = torch.empty(N, H * D).cuda()
    o = ccq.ccq_fwd_chunked("gla", q, k, v, a, None, m.w_lam, m.b_lam, carry_out=(S, C, ks, n))
    y = ccq.ccq_scan(x, xa, h_out=h)
    # every beam of a request starts from its prompt's states; one beam is alive
    states = [t.repeat_interleave(K, 0).contiguous() for t in (S, C, ks, n, h)]
    scores = torch.full((N, K), -float("inf")).cuda()
    scores[:, 0] = 0.0
    mixed = (o[:, :, -1].reshape(N, -1).float() + y[:, -1].float()).to(torch.bfloat16)
    logits = (mixed @ m.out).repeat_interleave(K, 0).view(N, K, V)
    done = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    for step in range(5):
        pick = ccq.ccq_beam_select(logits.contiguous(), scores, K, finished=done, pad_token=0)
        t, p, s = layer.beam_select(_np(logits), _np(scores), K, done.cpu().numpy(), 0)
        assert np.array_equal(_np(pick["token"]), t) and np.array_equal(_np(pick["parent"]), p)
        assert np.allclose(_np(pick["score"]), s, rtol=1e-6, atol=1e-5)
        before = [t.clone() for t in states]
        ccq.ccq_beam_reorder(states, pick["parent"])
        for new, old in zip(states, before):
            assert np.array_equal(_np(new), _np(torch.from_numpy(layer.beam_reorder(old.cpu().numpy(), p))))
        scores = pick["score"]
        done = done.gather(1, pick["parent"].long()) | (pick["token"] % 7 == 3)
        here = torch.full((N * K, 1), T + step, device="cuda")
        _, q, k, v, a, x, xa = m.inputs(pick["token"].view(N * K, 1), here)
        S, C, ks, n, h = states
        carry = oracle.Carry(*(_np(t) for t in (S, C, ks)), n.cpu().numpy())
        ref, after = oracle.ccq_decode_step(*(_np(t[:, :, 0]) for t in (q, k, v, a)), None, _np(m.w_lam), _np(m.b_lam),
                                            "gla", carry)
        hs, last, es, le = layer.scan(_np(x), _np(xa), _np(h), None, False)
        o = ccq.ccq_decode_step("gla", *(t[:, :, 0].contiguous() for t in (q, k, v, a)), None, m.w_lam, m.b_lam, S, C, ks, n)
        y = ccq.ccq_scan(x, xa, h0=h, h_out=h)
        assert normwise_error(_np(o), ref) <= 2e-2 and normwise_error(_np(S), after.S) <= 1e-4
        assert (np.abs(_np(h) - last) <= 10 * 2.0 ** -24 * le + 1e-37).all()
        logits = ((o.reshape(N * K, -1).float() + y[:, 0].float()).to(torch.bfloat16) @ m.out).view(N, K, V)
    assert n.eq(T + 5).all()


def test_training_step_through_the_layer(gpu_lib):
    """loss = <do, read step> + <dy, recurrence>: the gradient of the packed projection, through the
    chunked backward and the preparation's, against differentiation in 64 bits."""
    import torch
    import curvature_conditioned_query_amd as ccq
    B, T, d = 1, 70, 64
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(B, T, 3, H, d, generator=g).cuda()
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    wq = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    la = (torch.nn.functional.logsigmoid(torch.randn(B, H, T, d, generator=g)) / 16).cuda()
    w_lam, b_lam = (torch.randn(H, d, generator=g) / d ** 0.5).cuda(), torch.full((H,), -1.0).cuda()
    do = torch.randn(B, H, T, d, generator=g).cuda()
    how = dict(inv_freq=inv, q_weight=wq)
    q, k = ccq.ccq_qk_norm_rope(packed[:, :, 0], packed[:, :, 1], **how)
    _, v = ccq.ccq_qk_norm_rope(None, packed[:, :, 2], k_norm="none")
    back = ccq.ccq_bwd_chunked("gla", q, k, v, la, w_lam, b_lam, do)
    dpacked = torch.empty_like(packed)
    out = ccq.ccq_qk_norm_rope_backward(packed[:, :, 0], packed[:, :, 1], back["dq"], back["dk"], dq=dpacked[:, :, 0],
                                        dk=dpacked[:, :, 1], **how)
    ccq.ccq_qk_norm_rope_backward(None, packed[:, :, 2], None, back["dv"], k_norm="none", dk=dpacked[:, :, 2])

    ref = oracle.ccq_sequence_backward(_np(q), _np(k), _np(v), _np(la), None, _np(w_lam), _np(b_lam), "gla", _np(do))
    pos = np.arange(T)[None]
    dq, dw, _, _ = layer.norm_rope_backward(_np(packed[:, :, 0]), _np(wq), "rms", 1e-6, pos, _np(inv), False, ref["dq"])
    dk, _, _, _ = layer.norm_rope_backward(_np(packed[:, :, 1]), None, "l2", 0, pos, _np(inv), False, ref["dk"])
    for got, want, tag in ((dpacked[:, :, 0], dq, "dq"), (dpacked[:, :, 1], dk, "dk"), (out["dq_weight"], dw, "dw"),
                           (dpacked[:, :, 2], ref["dv"].transpose(0, 2, 1, 3), "dv")):
        e = normwise_error(_np(got).reshape(1, 1, -1), want.reshape(1, 1, -1))
        print(f"training step {tag} err {e:.2e}", flush=True)
        assert e <= 1e-4
