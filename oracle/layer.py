"""fp64 definitions of the operators around the read step, in NumPy, one row and one token at a time.

Queries and keys (norm, weight, rotation, layout), the gated linear recurrence, beam selection and
reordering, with the gradients of the first two.  Alongside each result comes a majorant of the
rounding of an fp32 evaluation, so that a test's tolerance is a multiple of 2^-24 times a number that
stands here and not a guess.
"""

import numpy as np

L2_FLOOR = 1e-12


# ---------------------------------------------------------------- queries and keys


def _angles(positions, inv_freq, rot, interleaved):
    """cos and signed sin of every rotated entry [.., rot], and the index of its partner [rot]."""
    a = np.asarray(positions, np.float64)[..., None] * np.asarray(inv_freq, np.float64)
    half = rot // 2
    i = np.arange(rot)
    pair = i // 2 if interleaved else i % half
    first = (i % 2 == 0) if interleaved else (i < half)
    partner = i ^ 1 if interleaved else np.where(first, i + half, i - half)
    return np.cos(a)[..., pair], np.where(first, -1.0, 1.0) * np.sin(a)[..., pair], partner


def rotate(x, positions, inv_freq, interleaved, back=False):
    """x [B, T, H, d] turned by positions [B, T]; and hypot(entry, partner), the size its rounding has."""
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    size = np.abs(x).copy()
    if rot == 0:
        return x, size
    c, s, partner = _angles(positions, inv_freq, rot, interleaved)
    c, s = c[:, :, None], (-s if back else s)[:, :, None]
    y = x.copy()
    y[..., :rot] = x[..., :rot] * c + x[..., partner] * s
    size[..., :rot] = np.hypot(x[..., :rot], x[..., partner])
    return y, size


def row_scale(x, norm, eps):
    if norm == "rms":
        return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if norm == "l2":
        return 1.0 / np.maximum(np.sqrt((x * x).sum(-1, keepdims=True)), L2_FLOOR)
    return np.ones(x.shape[:-1] + (1,))


def norm_rope(x, w, norm, eps, positions, inv_freq, interleaved, copies=1):
    """One side of ccq_qk_norm_rope: [B, T, H, d] -> [B, H copies, T, d], and the rounding's size."""
    x = np.asarray(x, np.float64)
    y = x * row_scale(x, norm, eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    y, size = rotate(y, positions, inv_freq, interleaved)
    lay = lambda a: np.repeat(a.transpose(0, 2, 1, 3), copies, axis=1)  # noqa: E731
    return lay(y), lay(size)


def norm_rope_backward(x, w, norm, eps, positions, inv_freq, interleaved, d_out, copies=1):
    """Gradients (dx [B, T, H, d], dw [d]) of one side, and the sizes of their rounding."""
    x = np.asarray(x, np.float64)
    B, T, H, d = x.shape
    g = np.asarray(d_out, np.float64).reshape(B, H, copies, T, d).transpose(0, 3, 1, 2, 4)
    z = np.zeros_like(x)
    zs = np.zeros_like(x)
    for c in range(copies):
        turned, size = rotate(g[:, :, :, c], positions, inv_freq, interleaved, back=True)
        z += turned
        zs += size
    w1 = np.ones(d) if w is None else np.asarray(w, np.float64)
    r = row_scale(x, norm, eps)
    over = d if norm == "rms" else 1
    has = norm != "none"
    if norm == "l2":
        has = np.sqrt((x * x).sum(-1, keepdims=True)) > L2_FLOOR
    pull = np.where(has, r ** 3 / over, 0.0)
    dx = w1 * z * r - x * pull * (w1 * z * x).sum(-1, keepdims=True)
    dx_size = np.abs(w1) * zs * r + np.abs(x) * pull * (np.abs(w1) * zs * np.abs(x)).sum(-1, keepdims=True)
    return dx, (z * x * r).sum((0, 1, 2)), dx_size, (zs * np.abs(x) * r).sum((0, 1, 2))


# ---------------------------------------------------------------- gated linear recurrence


def scan(x, log_alpha, h0, lengths, complement):
    """Returns h [B, T, D] (NaN behind a length), the last state [B, D], and the majorant of h's rounding:
    E_t = alpha_t E_{t-1} + A_t with A_t = alpha_t A_{t-1} + |s_t x_t|, for 2^-24 times a constant."""
    x, g = np.asarray(x, np.float64), np.asarray(log_alpha, np.float64)
    B, T, D = x.shape
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    size, err = np.abs(h), np.zeros((B, D))
    hs, es = np.full((B, T, D), np.nan), np.full((B, T, D), np.nan)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(B):
            n = T if lengths is None else min(max(int(lengths[b]), 0), T)
            for t in range(n):
                a = np.exp(g[b, t])
                u = x[b, t] * (-np.expm1(g[b, t]) if complement else 1.0)
                h[b] = np.where(a == 0, u, a * h[b] + u)
                size[b] = np.where(a == 0, np.abs(u), a * size[b] + np.abs(u))
                err[b] = np.where(a == 0, size[b], a * err[b] + size[b])
                hs[b, t], es[b, t] = h[b], err[b]
    return hs, h, es, err


def scan_backward(x, log_alpha, dy, h0, dh_out, lengths, complement):
    """Gradients dx, dlog_alpha [B, T, D], dh0 [B, D], and the sizes of their rounding."""
    x, g, dy = (np.asarray(v, np.float64) for v in (x, log_alpha, dy))
    B, T, D = x.shape
    hs, _, es, _ = scan(x, g, h0, lengths, complement)
    start = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64)
    d = np.zeros((B, D)) if dh_out is None else np.asarray(dh_out, np.float64).copy()
    size, err = np.abs(d), np.zeros((B, D))
    dx, dg, dxs, dgs = (np.zeros((B, T, D)) for _ in range(4))
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(B):
            n = T if lengths is None else min(max(int(lengths[b]), 0), T)
            for t in reversed(range(n)):
                a = np.exp(g[b, t])
                d[b] += dy[b, t]
                size[b] += np.abs(dy[b, t])
                err[b] += size[b]
                s = -np.expm1(g[b, t]) if complement else np.ones(D)
                before = hs[b, t - 1] if t else start[b]
                before_err = es[b, t - 1] if t else np.zeros(D)
                diff = before - x[b, t] if complement else before
                mag = np.abs(before) + (np.abs(x[b, t]) if complement else 0.0)
                dx[b, t], dxs[b, t] = s * d[b], np.abs(s) * err[b]
                dg[b, t] = np.where(a == 0, 0.0, a * d[b] * diff)
                dgs[b, t] = np.where(a == 0, 0.0, a * (err[b] * mag + np.abs(d[b]) * (before_err + mag)))
                d[b], size[b], err[b] = (np.where(a == 0, 0.0, a * v) for v in (d[b], size[b], err[b]))
    return dx, dg, d, dxs, dgs, err


# ---------------------------------------------------------------- beams


def beam_select(logits, scores, m, finished=None, pad=0):
    """token, parent [N, m] int and score [N, m]: the m best by (score falling, beam, token)."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    N, K, V = x.shape
    token, parent, score = np.zeros((N, m), int), np.zeros((N, m), int), np.zeros((N, m))
    for n in range(N):
        total = np.full((K, V), -np.inf)
        for k in range(K):
            s = float(scores[n][k])
            s = -np.inf if np.isnan(s) else s
            if finished is not None and finished[n][k]:
                total[k, pad] = s
                continue
            top = x[n, k].max()
            if s == -np.inf or top == -np.inf:
                continue
            total[k] = s + (x[n, k] - top) - np.log(np.exp(x[n, k] - top).sum())
        flat = total.reshape(-1)
        best = np.argsort(-flat, kind="stable")[:m]
        token[n], parent[n], score[n] = best % V, best // V, flat[best]
    return token, parent, score


def beam_reorder(state, parent):
    """Rows of state [N K, ...] moved to the beams that continue them."""
    N, K = parent.shape
    rows = [n * K + (parent[n, j] if 0 <= parent[n, j] < K else j) for n in range(N) for j in range(K)]
    return state[rows]
