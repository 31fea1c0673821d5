"""Pins of the fp64 definitions in oracle/mixer.py: closed forms, other operators' definitions, finite differences."""

import numpy as np
import pytest

import oracle
from oracle import mixer


def _case(seed, B=2, T=5, H=4, Hq=2, Hk=1, Hv=4, dk=3, dv=2):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(B, T, Hq, dk)), k=r.normal(size=(B, T, Hk, dk)), v=r.normal(size=(B, T, Hv, dv)),
                log_alpha=-np.abs(r.normal(size=(B, T, H))), S0=r.normal(size=(B, H, dv, dk)), scale=0.7)


def test_attention_is_the_quadratic_form():
    c = _case(0)
    o, S, _, _ = mixer.linear_attn(**c)
    q, k, v = (np.repeat(c[m], 4 // c[m].shape[2], 2) for m in "qkv")
    run = np.cumsum(c["log_alpha"], 1)
    for b in range(2):
        for h in range(4):
            w = np.tril(np.exp(run[b, :, None, h] - run[b, None, :, h]))
            want = (w * (q[b, :, h] @ k[b, :, h].T)) @ v[b, :, h] + np.exp(run[b, :, h])[:, None] * (q[b, :, h] @ c["S0"][b, h].T)
            assert np.allclose(o[b, :, h], 0.7 * want, atol=1e-12)


def test_attention_is_the_read_step_without_cleaning():
    """One decay for all key channels, gate bias -inf: the read step's own recurrence."""
    r = np.random.default_rng(1)
    B, H, T, d = 1, 2, 7, 4
    q, k, v = (r.normal(size=(B, H, T, d)) for _ in range(3))
    g = -np.abs(r.normal(size=(B, H, T)))
    want, carry = oracle.ccq_recurrent(q, k, v, np.repeat(g[..., None], d, -1), None, np.zeros((H, d)), np.full(H, -np.inf), "gla")
    t = lambda x: np.swapaxes(x, 1, 2)  # noqa: E731
    o, S, _, _ = mixer.linear_attn(t(q), t(k), t(v), t(g))
    assert np.allclose(t(o), want, atol=1e-12) and np.allclose(S, carry.S, atol=1e-12)


def test_attention_resumes_and_stops():
    c = _case(2)
    o, S, _, _ = mixer.linear_attn(**c, lengths=[3, 0])
    assert np.isnan(o[0, 3:]).all() and np.isnan(o[1]).all() and np.array_equal(S[1], c["S0"][1])
    first = {m: c[m][:1, :3] for m in ("q", "k", "v", "log_alpha")}
    rest = {m: c[m][:1, 3:] for m in first}
    _, mid, _, _ = mixer.linear_attn(**first, S0=c["S0"][:1], scale=0.7)
    assert np.allclose(mid, S[:1])
    o2, end, _, _ = mixer.linear_attn(**rest, S0=mid, scale=0.7)
    whole, last, _, _ = mixer.linear_attn(**c)
    assert np.allclose(o2[0], whole[0, 3:]) and np.allclose(end[0], last[0])


def test_a_gate_of_zero_drops_the_state():
    c = _case(3, B=1)
    c["log_alpha"][0, 2] = -np.inf
    c["S0"][:] = np.inf
    o, S, _, _ = mixer.linear_attn(**c)
    fresh = {m: c[m][:, 2:] for m in ("q", "k", "v", "log_alpha")}
    o2, S2, _, _ = mixer.linear_attn(**fresh, scale=0.7)
    assert np.allclose(o[:, 2:], o2) and np.allclose(S, S2)


@pytest.mark.parametrize("lengths", [None, [4, 0]])
def test_attention_gradient_by_differences(lengths):
    c = _case(4)
    r = np.random.default_rng(5)
    d_o, dS = r.normal(size=(2, 5, 4, 2)), r.normal(size=c["S0"].shape)

    def loss(**kw):
        o, S, _, _ = mixer.linear_attn(**kw, lengths=lengths)
        return np.nansum(o * d_o) + (S * dS).sum()
    got, size = mixer.linear_attn_backward(c["q"], c["k"], c["v"], d_o, c["log_alpha"], 0.7, c["S0"], dS, lengths)
    for m, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_alpha", "dlog_alpha"), ("S0", "dS0")):
        flat = c[m].reshape(-1)
        for i in r.choice(flat.size, 12, replace=False):
            old = flat[i]
            up, down = (loss(**{**c, m: _with(c[m], i, old + s)}) for s in (1e-6, -1e-6))
            assert abs((up - down) / 2e-6 - got[name].reshape(-1)[i]) < 1e-6
        assert (np.abs(got[name]) <= size[name] * (1 + 1e-12) + 1e-12).all()


def _with(x, i, value):
    y = x.copy()
    y.reshape(-1)[i] = value
    return y


@pytest.mark.parametrize("activation", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_group_norm_against_torch_and_differences(activation, gated, center):
    import torch
    r = np.random.default_rng(6)
    x, dy = r.normal(size=(2, 3, 4, 8)), r.normal(size=(2, 3, 4, 8))
    w, b = r.normal(size=(4, 8)), r.normal(size=(4, 8))
    gate = r.normal(size=x.shape) if gated else None
    t = {n: torch.tensor(a, requires_grad=True) for n, a in (("x", x), ("w", w), ("b", b)) if a is not None}
    if center:  # torch's own group norm over [B T, G d]
        n = torch.nn.functional.group_norm(t["x"].reshape(6, 32), 4, eps=1e-3).reshape(x.shape)
    else:
        n = t["x"] * torch.rsqrt((t["x"] ** 2).mean(-1, keepdim=True) + 1e-3)
    z = n * t["w"] + t["b"]
    f = {"none": lambda s: s, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[activation]
    if gated:
        t["g"] = torch.tensor(gate, requires_grad=True)
    y = z * f(t["g"]) if gated else f(z)
    got = mixer.group_norm(x, w, b, gate, center, 1e-3, activation)[0]
    assert np.allclose(got, y.detach().numpy(), atol=1e-10)
    y.backward(torch.tensor(dy))
    dx, dgate, dw, db = mixer.group_norm_backward(x, dy, w, b, gate, center, 1e-3, activation)
    for a, n in ((dx, "x"), (dw, "w"), (db, "b")) + (((dgate, "g"),) if gated else ()):
        assert np.allclose(a, t[n].grad.numpy(), atol=1e-9)
    shared = mixer.group_norm_backward(x, dy, w[0], b[0], gate, center, 1e-3, activation)
    each = mixer.group_norm_backward(x, dy, np.tile(w[0], (4, 1)), np.tile(b[0], (4, 1)), gate, center, 1e-3, activation)
    assert np.allclose(shared[2], each[2].sum(0)) and np.allclose(shared[3], each[3].sum(0))


def test_adjusted_logits_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 0.5, np.nan, 3.0]])
    y, _ = mixer.logits_adjust(x, [[0, 1, 1, 3, 3, 9, -1, 2]], [7], [2], 2.0, 0.25, 0.5, [[5, 2, 5, 7]], [[1.0, -1.0, 2.0, 9.0]],
                               np.array([[0b101111]]))
    # 0: prompt alone; 1: in the prompt and once behind it; 3: twice behind it; 2: a bias; 4: not allowed; 5: two biases
    assert np.array_equal(y, [[1.0, -4.0 - 0.5 - 0.25, 0.0, 0.25 - 1.0 - 0.25, -np.inf, 6.0]])
