"""fp64 definitions of the operators of a linear-attention layer, in NumPy, token by token.

Linear attention with a decay for each head, the group norm behind it, and adjusted logits, with the
gradients of the first two.  Alongside each result of the attention comes its size: the same sum with
every term taken absolutely, which is what its roundings are relative to.
"""

import numpy as np


# ---------------------------------------------------------------- linear attention


def _shared(x, H):
    """[B, T, Hx, d] -> [B, T, H, d]."""
    return np.repeat(np.asarray(x, np.float64), H // x.shape[2], axis=2)


RESET = -126.0 * np.log(2.0)  # a log decay below this counts as a decay of 0: fp32's least normal number


def _gates(log_alpha, B, T, H):
    g = np.zeros((B, T, H)) if log_alpha is None else np.asarray(log_alpha, np.float64)
    return np.where(g < RESET, 0.0, np.exp(g))


def _decayed(S, a):
    """S a, and 0 where a is 0 whatever S holds."""
    a = a[..., None, None]
    with np.errstate(invalid="ignore"):
        return np.where(a == 0, 0.0, S * a)


def linear_attn(q, k, v, log_alpha=None, scale=1.0, S0=None, lengths=None):
    """o [B, T, H, d_v] (NaN behind a length), S [B, H, d_v, d_k], and the sizes of both."""
    H = max(q.shape[2], k.shape[2], v.shape[2], 0 if log_alpha is None else log_alpha.shape[2])
    q, k, v = (_shared(x, H) for x in (q, k, v))
    B, T, _, dk = q.shape
    dv = v.shape[-1]
    a = _gates(log_alpha, B, T, H)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    S = np.zeros((B, H, dv, dk)) if S0 is None else np.asarray(S0, np.float64).copy()
    size = np.abs(S)
    o, os = np.full((B, T, H, dv), np.nan), np.full((B, T, H, dv), np.nan)
    for b in range(B):
        for t in range(n[b]):
            new = v[b, t][:, :, None] * k[b, t][:, None, :]
            S[b] = _decayed(S[b], a[b, t]) + new
            size[b] = _decayed(size[b], a[b, t]) + np.abs(new)
            o[b, t] = scale * np.einsum("hij,hj->hi", S[b], q[b, t])
            os[b, t] = abs(scale) * np.einsum("hij,hj->hi", size[b], np.abs(q[b, t]))
    return o, S, os, size


def linear_attn_backward(q, k, v, d_o, log_alpha=None, scale=1.0, S0=None, dS_out=None, lengths=None):
    """A dict of the gradients dq, dk, dv, dlog_alpha, dS0 and one of their sizes."""
    H = max(q.shape[2], k.shape[2], v.shape[2], 0 if log_alpha is None else log_alpha.shape[2])
    shares = [H // x.shape[2] for x in (q, k, v)]
    q, k, v, d_o = _shared(q, H), _shared(k, H), _shared(v, H), np.asarray(d_o, np.float64)
    B, T, _, dk = q.shape
    dv = v.shape[-1]
    a = _gates(log_alpha, B, T, H)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    out = dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape), dlog_alpha=np.zeros((B, T, H)),
               dS0=np.zeros((B, H, dv, dk)))
    size = {m: np.zeros(x.shape) for m, x in out.items()}
    mv = lambda M, x: np.einsum("hij,hj->hi", M, x)  # noqa: E731
    tv = lambda M, x: np.einsum("hij,hi->hj", M, x)  # noqa: E731
    for b in range(B):
        S = np.zeros((H, dv, dk)) if S0 is None else np.asarray(S0[b], np.float64).copy()
        mag, states, mags = np.abs(S), [], []
        for t in range(n[b]):
            states.append(S)
            mags.append(mag)
            new = v[b, t][:, :, None] * k[b, t][:, None, :]
            S, mag = _decayed(S, a[b, t]) + new, _decayed(mag, a[b, t]) + np.abs(new)
            out["dq"][b, t], size["dq"][b, t] = scale * tv(S, d_o[b, t]), abs(scale) * tv(mag, np.abs(d_o[b, t]))
        A = np.zeros((H, dv, dk)) if dS_out is None else np.asarray(dS_out[b], np.float64).copy()
        # the sum that forms dlog_alpha rounds at the size of its terms
        As, gs = np.abs(A), (np.abs(A) * mag).sum((1, 2))
        for t in reversed(range(n[b])):
            new = scale * d_o[b, t][:, :, None] * q[b, t][:, None, :]
            A, As = A + new, As + np.abs(new)
            out["dk"][b, t], size["dk"][b, t] = tv(A, v[b, t]), tv(As, np.abs(v[b, t]))
            out["dv"][b, t], size["dv"][b, t] = mv(A, k[b, t]), mv(As, np.abs(k[b, t]))
            gs = gs + (np.abs(q[b, t]) * size["dq"][b, t]).sum(-1) + (np.abs(k[b, t]) * size["dk"][b, t]).sum(-1)
            with np.errstate(invalid="ignore"):
                dg = a[b, t] * (A * states[t]).sum((1, 2))
            out["dlog_alpha"][b, t] = np.where(a[b, t] == 0, 0.0, dg)
            size["dlog_alpha"][b, t] = np.where(a[b, t] == 0, 0.0, gs)
            A, As = _decayed(A, a[b, t]), _decayed(As, a[b, t])
            gs = np.where(a[b, t] == 0, 0.0, gs)
        out["dS0"][b], size["dS0"][b] = A, As
    for d in (out, size):
        for m, share in zip(("dq", "dk", "dv"), shares):
            x = d[m]
            d[m] = x.reshape(B, T, H // share, share, x.shape[-1]).sum(3)
    return out, size


# ---------------------------------------------------------------- group norm


def _act(x, kind):
    """Value and slope."""
    if kind == "none":
        return x, np.ones_like(x)
    s = 1.0 / (1.0 + np.exp(-x))
    return (x * s, s * (1 + x * (1 - s))) if kind == "silu" else (s, s * (1 - s))


def group_norm(x, weight=None, bias=None, gate=None, center=False, eps=1e-6, activation="none"):
    """y, and the normalised rows, their scale and z."""
    x = np.asarray(x, np.float64)
    u = x - x.mean(-1, keepdims=True) if center else x
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = u * r
    z = n * (1.0 if weight is None else np.asarray(weight, np.float64)) + (0.0 if bias is None else np.asarray(bias, np.float64))
    y = _act(z, activation)[0] if gate is None else z * _act(np.asarray(gate, np.float64), activation)[0]
    return y, n, r, z


def group_norm_backward(x, dy, weight=None, bias=None, gate=None, center=False, eps=1e-6, activation="none"):
    """dx, dgate, dweight, dbias ([G, d]; summed over groups for a weight [d])."""
    _, n, r, z = group_norm(x, weight, bias, gate, center, eps, activation)
    dy = np.asarray(dy, np.float64)
    dgate = None
    if gate is None:
        dz = dy * _act(z, activation)[1]
    else:
        f, slope = _act(np.asarray(gate, np.float64), activation)
        dz, dgate = dy * f, dy * z * slope
    dn = dz * (1.0 if weight is None else np.asarray(weight, np.float64))
    dx = r * (dn - (dn.mean(-1, keepdims=True) if center else 0.0) - n * (dn * n).mean(-1, keepdims=True))
    total = lambda d, w: d.sum((0, 1)) if np.ndim(w) == 2 else d.sum((0, 1, 2))  # noqa: E731
    return dx, dgate, None if weight is None else total(dz * n, weight), None if bias is None else total(dz, bias)


# ---------------------------------------------------------------- logits


def logits_adjust(logits, history=None, lengths=None, prompt_lengths=None, repetition=1.0, presence=0.0, frequency=0.0,
                  bias_token=None, bias_value=None, allowed=None):
    """logits [R, V] adjusted, one token at a time, and the size of the rounding."""
    x = np.asarray(logits, np.float64).copy()
    R, V = x.shape
    size = np.abs(x)
    row = lambda p, r: float(p[r]) if np.ndim(p) else float(p)  # noqa: E731
    for r in range(R):
        seen, count = set(), {}
        if history is not None:
            L = len(history[r])
            n = L if lengths is None else min(max(int(lengths[r]), 0), L)
            p = 0 if prompt_lengths is None else min(max(int(prompt_lengths[r]), 0), n)
            for i in range(n):
                t = int(history[r][i])
                if 0 <= t < V:
                    seen.add(t)
                    if i >= p:
                        count[t] = count.get(t, 0) + 1
        for t in seen:
            theta = row(repetition, r)
            x[r, t] = x[r, t] / theta if x[r, t] > 0 else x[r, t] * theta
            c = count.get(t, 0)
            off = row(frequency, r) * c + (row(presence, r) if c else 0.0)
            size[r, t] = abs(x[r, t]) + abs(row(frequency, r) * c) + abs(row(presence, r))
            x[r, t] -= off
        if bias_token is not None:
            for t, b in zip(bias_token[r], bias_value[r]):
                if 0 <= t < V:
                    x[r, t] += float(b)
                    size[r, t] += abs(float(b))
        if allowed is not None:
            bits = np.asarray(allowed[r]).astype(np.uint32)
            for t in range(V):
                if not (int(bits[t // 32]) >> (t % 32)) & 1:
                    x[r, t], size[r, t] = -np.inf, 0.0
    return x, size
