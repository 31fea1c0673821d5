"""Cases of the operators around the CCQ read step, with their plain forms.

Three families, in the order a recurrent language model runs them:

  qk       queries and keys of a packed projection, normalised per head, rotated by their position and laid out for the
           read step; forward (one token a sequence, whole prompts) and backward
  scan     the elementwise gated linear recurrence h_t = alpha_t h_{t-1} + s_t x_t, alpha = exp(log_alpha); forward over
           one token, prompts and long sequences, and backward
  beam     beam search: the best continuations over beams and vocabulary, and the reordering of the carried states

``run`` computes them in elementary torch operations; with ``own`` set, by the library's entry points.  ``exact`` holds
the definitions in 64 bits.
"""

import math
import random

import torch

own = False

L2_FLOOR = 1e-12
RMS_EPS = 1e-6
ROPE_BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one new token for each of 64 sequences, 16 heads: what a decode step prepares, where latency counts
        _qk("qk_step_bf16", "fwd", "bf16", B=64, T=1, Hq=16, Hk=16, d=128, rot=128),
        # the headline prefill's queries and keys: 4 prompts of 4096 tokens, 16 heads of 128
        _qk("qk_prefill_bf16", "fwd", "bf16", B=4, T=4096, Hq=16, Hk=16, d=128, rot=128),
        # fp32, d = 64, an odd prompt length, two key heads shared by six query heads, half the head rotated, in pairs
        _qk("qk_prefill_f32_shared", "fwd", "f32", B=2, T=1021, Hq=6, Hk=2, d=64, rot=32, pairs=True, expand=True),
        # the training step's gradient at the headline prefill, key heads shared by four query heads
        _qk("qk_backward_bf16", "bwd", "bf16", B=4, T=4096, Hq=16, Hk=4, d=128, rot=128, expand=True),
        # one new token for each of 256 sequences through a 2048-channel recurrence
        _scan("scan_step_bf16", "fwd", "bf16", B=256, T=1, D=2048),
        # a prefill of 4 prompts of 4096 tokens through 16 x 128 channels
        _scan("scan_prefill_bf16", "fwd", "bf16", B=4, T=4096, D=2048),
        # the length-extrapolation shape: one sequence of 20480 tokens, fp32, with the complement input scale
        _scan("scan_long_f32", "fwd", "f32", B=1, T=20480, D=1024, complement=True),
        # a padded training batch of odd length: the gradient of a 4 x 4095 x 2048 recurrence
        _scan("scan_backward_bf16", "bwd", "bf16", B=4, T=4095, D=2048, complement=True, ragged=True),
        # one request with four beams
        _beam("beam_select_one_f32", "f32", N=1, K=4, V=32000, M=4),
        # 32 requests with eight beams over a large odd vocabulary, twice as many picks as beams
        _beam("beam_select_many_bf16", "bf16", N=32, K=8, V=131071, M=16),
        # the carries of one request's four beams (16 heads of 128)
        _reorder("beam_reorder_one", N=1, K=4, H=16, d=128),
        # the decode benchmark's 256 sequences as 64 requests of four beams: 0.5 GB of carries
        _reorder("beam_reorder_many", N=64, K=4, H=16, d=128),
    ]


def draw(rng: random.Random):
    kind = rng.choice(["qk_fwd", "qk_bwd", "scan_fwd", "scan_bwd", "select", "reorder"])
    dtype = rng.choice(["bf16", "f32"])
    if kind.startswith("qk"):
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        group = rng.choice([1, 1, 2, 4])
        tokens = _log(rng, 1, 16384 * 128 * 16 // (2 * d * Hk * max(1, group)) if dtype == "f32" else 16384 * 128 * 32 // (2 * d * Hk * group))
        T = min(tokens, _log(rng, 1, 20480))
        rot = rng.choice([0, 16, d // 2, d])
        c = _qk("", kind[3:], dtype, B=min(256, max(1, tokens // T)), T=T, Hq=Hk * group, Hk=Hk, d=d, rot=rot,
                pairs=rng.random() < 0.4, expand=group > 1 and rng.random() < 0.6)
        c["weights"] = rng.random() < 0.7
    elif kind.startswith("scan"):
        D = 8 * _log(rng, 4, 512)
        elements = _log(rng, D, (33_000_000 if dtype == "bf16" else 20_000_000))
        rows = max(1, elements // D)
        T = min(rows, _log(rng, 1, 20480))
        c = _scan("", kind[5:], dtype, B=min(256, max(1, rows // T)), T=T, D=D, complement=rng.random() < 0.5,
                  ragged=rng.random() < 0.4)
    elif kind == "select":
        K = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        V = _log(rng, 1000, 131072)
        N = _log(rng, 1, max(1, min(64, 33_000_000 // (K * V * (2 if dtype == "f32" else 1)))))
        c = _beam("", dtype, N=N, K=K, V=V, M=rng.choice([K, 2 * K]))
    else:
        K = rng.choice([2, 3, 4, 5, 8, 16])
        d = rng.choice([64, 128])
        H = rng.choice([1, 2, 5, 8, 16])
        N = _log(rng, 1, max(1, 250 * 16 * 128 * 128 // (K * H * d * d)))
        c = _reorder("", N=N, K=K, H=H, d=d)
        c["packed"] = rng.random() < 0.3
    del c["name"]
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def _qk(name, way, dtype, B, T, Hq, Hk, d, rot, pairs=False, expand=False):
    return dict(name=name, op="qk", way=way, dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, pairs=pairs,
                expand=expand, weights=True)


def _scan(name, way, dtype, B, T, D, complement=False, ragged=False):
    return dict(name=name, op="scan", way=way, dtype=dtype, B=B, T=T, D=D, complement=complement, ragged=ragged)


def _beam(name, dtype, N, K, V, M):
    return dict(name=name, op="select", dtype=dtype, N=N, K=K, V=V, M=M)


def _reorder(name, N, K, H, d):
    return dict(name=name, op="reorder", N=N, K=K, H=H, d=d, packed=False)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"qk": _prepare_qk, "scan": _prepare_scan, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _prepare_qk(c, g):
    dt = DTYPES[c["dtype"]]
    B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
    # what the projection leaves: queries, keys and values of a token side by side
    packed = _randn(g, B, T, (Hq + 2 * Hk) * d, dtype=dt)
    s = dict(case=c, q=packed[..., : Hq * d].view(B, T, Hq, d), k=packed[..., Hq * d : (Hq + Hk) * d].view(B, T, Hk, d))
    start = torch.randint(0, 200_000, (B, 1), generator=g, device="cuda", dtype=torch.int64)
    s["positions"] = start + torch.arange(T, device="cuda", dtype=torch.int64)
    s["inv_freq"] = (ROPE_BASE ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / max(1, c["rot"]))).float() if c["rot"] else None
    s["wq"] = 1.0 + 0.1 * _randn(g, d) if c["weights"] else None
    s["wk"] = 1.0 + 0.1 * _randn(g, d) if c["weights"] else None
    if c["way"] == "bwd":
        s["dq_out"] = _randn(g, B, Hq, T, d)
        s["dk_out"] = _randn(g, B, Hq if c["expand"] else Hk, T, d)
    return s


def _prepare_scan(c, g):
    dt = DTYPES[c["dtype"]]
    B, T, D = c["B"], c["T"], c["D"]
    s = dict(case=c, x=_randn(g, B, T, D, dtype=dt))
    s["log_alpha"] = (torch.nn.functional.logsigmoid(_randn(g, B, T, D)) / 8).to(dt)
    s["h0"] = _randn(g, B, D)
    s["lengths"] = torch.randint(T // 2, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else None
    s["y"] = torch.zeros(B, T, D, device="cuda", dtype=dt)
    if c["way"] == "fwd":
        s["h"] = torch.empty(B, D, device="cuda")
    else:
        s["dy"] = _randn(g, B, T, D, dtype=dt)
        s["dh"] = _randn(g, B, D)
        # the states that the forward pass of the same training step left behind
        s["carry"] = _chunk_states(s)
    return s


def _prepare_select(c, g):
    N, K, V = c["N"], c["K"], c["V"]
    # beams of a request see nearly the same distribution: shared logits, each beam's own part, a long tail
    logits = 2.5 * _randn(g, N, 1, V) + 1.0 * _randn(g, N, K, V)
    s = dict(case=c, logits=logits.to(DTYPES[c["dtype"]]), scores=-4.0 * _rand(g, N, K) - 10.0)
    s["finished"] = (_rand(g, N, K) < 0.1).to(torch.uint8)
    return s


def _prepare_reorder(c, g):
    N, K, H, d = c["N"], c["K"], c["H"], c["d"]
    S = _randn(g, N * K, H, d, d)
    C = _randn(g, N * K, H, d * (d + 1) // 2) if c["packed"] else _randn(g, N * K, H, d, d)
    n = torch.randint(1, 9000, (N * K, H), generator=g, device="cuda", dtype=torch.int64)
    parent = torch.randint(0, K, (N, K), generator=g, device="cuda", dtype=torch.int32)
    return dict(case=c, states=[S, C, _randn(g, N * K, H, d), n], parent=parent)


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"qk": _plain_qk, "scan": _plain_scan, "select": _plain_select, "reorder": _plain_reorder}[c["op"]](s, c)


def _run_own(s, c):
    import curvature_conditioned_query_amd as ccq

    if c["op"] == "qk":
        how = dict(positions=s["positions"], inv_freq=s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"], q_norm="rms",
                   k_norm="l2", eps=RMS_EPS, interleaved=c["pairs"])
        if c["way"] == "fwd":
            return ccq.ccq_qk_norm_rope(s["q"], s["k"], expand_keys=c["expand"], **how)
        return ccq.ccq_qk_norm_rope_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], **how)
    if c["op"] == "scan":
        how = dict(h0=s["h0"], lengths=s["lengths"], complement=c["complement"])
        if c["way"] == "fwd":
            y = ccq.ccq_scan(s["x"], s["log_alpha"], h_out=s["h"], y=s["y"], **how)
            return {"y": y, "h": s["h"]}
        return ccq.ccq_scan_backward(s["x"], s["log_alpha"], s["dy"], dh_out=s["dh"], chunk_carry=s["carry"],
                                     want_dh0=True, **how)
    if c["op"] == "select":
        return ccq.ccq_beam_select(s["logits"], s["scores"], c["M"], finished=s["finished"], pad_token=0)
    ccq.ccq_beam_reorder(s["states"], s["parent"])
    return s["states"]


# ---------------------------------------------------------------- plain forms


def _angles(s, c):
    a = s["positions"].double()[:, :, None, None] * s["inv_freq"].double()  # [B, T, 1, rot / 2]; far positions: 64 bits
    return torch.cos(a).float(), torch.sin(a).float()


def _halves(x, c):
    r = c["rot"]
    return (x[..., 0:r:2], x[..., 1:r:2]) if c["pairs"] else (x[..., : r // 2], x[..., r // 2 : r])


def _joined(a, b, x, c):
    r = c["rot"]
    turned = torch.stack((a, b), -1).flatten(-2) if c["pairs"] else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _rotate(x, s, c, sign):
    if not c["rot"]:
        return x
    cos, sin = _angles(s, c)
    a, b = _halves(x, c)
    return _joined(a * cos - sign * b * sin, b * cos + sign * a * sin, x, c)


def _scale(x, kind):
    """1 / norm of each row, [.., 1]."""
    if kind == "rms":
        return torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS)
    return 1.0 / (x * x).sum(-1, keepdim=True).sqrt().clamp_min(L2_FLOOR)


def _plain_qk(s, c):
    dt = DTYPES[c["dtype"]]
    outs = []
    for x, w, kind in ((s["q"], s["wq"], "rms"), (s["k"], s["wk"], "l2")):
        x = x.float()
        shared = c["Hq"] // c["Hk"] if kind == "l2" and c["expand"] else 1
        if c["way"] == "fwd":
            y = x * _scale(x, kind)
            y = y if w is None else y * w
            y = _rotate(y, s, c, 1.0).to(dt).permute(0, 2, 1, 3)
            outs.append(y.repeat_interleave(shared, 1) if shared > 1 else y.contiguous())
            continue
        dz = (s["dq_out"] if kind == "rms" else s["dk_out"]).permute(0, 2, 1, 3)
        dz = _rotate(dz, s, c, -1.0)
        if shared > 1:
            dz = dz.reshape(c["B"], c["T"], c["Hk"], shared, c["d"]).sum(3)
        r = _scale(x, kind)
        u = dz if w is None else dz * w
        dot = (u * x).sum(-1, keepdim=True)
        dx = u * r - x * (r * r * r) * dot / (c["d"] if kind == "rms" else 1)
        outs.append(dx.to(dt))
        outs.append((dz * x * r).sum((0, 1, 2)) if w is not None else None)
    if c["way"] == "fwd":
        return outs[0], outs[1]
    return {"dq": outs[0], "dq_weight": outs[1], "dk": outs[2], "dk_weight": outs[3]}


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling: after a step every place holds the sum over twice as many terms."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat((b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return b


def _inside(s, c):
    t = torch.arange(c["T"], device="cuda")[None, :, None]
    n = s["lengths"]
    return None if n is None else t < n[:, None, None]


def _gates(s, c):
    """alpha and the scaled input of every token; past a sequence's length the state stays as it is."""
    g, x, live = s["log_alpha"].float(), s["x"].float(), _inside(s, c)
    a = torch.exp(g)
    b = -torch.expm1(g) * x if c["complement"] else x
    if live is not None:
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    return a, b


def _states(s, c):
    a, b = _gates(s, c)
    b = torch.cat((b[:, :1] + a[:, :1] * s["h0"][:, None], b[:, 1:]), 1)
    return a, _linear_scan(a, b)


def _chunk_states(s):
    """The state before every 64-token chunk, [B, ceil(T / 64), D]."""
    _, h = _states(s, s["case"])
    return torch.cat((s["h0"][:, None], h[:, 63:-1:64]), 1).contiguous()


def _plain_scan(s, c):
    dt = DTYPES[c["dtype"]]
    live = _inside(s, c)
    a, h = _states(s, c)
    if c["way"] == "fwd":
        y = h.to(dt)
        return {"y": y if live is None else torch.where(live, y, s["y"]), "h": h[:, -1].clone()}
    dy = s["dy"].float() if live is None else torch.where(live, s["dy"].float(), 0.0)
    # adjoint of h_t: dy_t + alpha_{t+1} adjoint of h_{t+1}, the same recurrence from the end
    dy = torch.cat((dy[:, :-1], dy[:, -1:] + s["dh"][:, None]), 1)
    after = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    dh = _linear_scan(after.flip(1), dy.flip(1)).flip(1)
    before = torch.cat((s["h0"][:, None], h[:, :-1]), 1)
    dx, dg = dh, a * before * dh
    if c["complement"]:
        dx = dh * -torch.expm1(s["log_alpha"].float())
        dg = a * (before - s["x"].float()) * dh
    if live is not None:
        dx, dg = torch.where(live, dx, 0.0), torch.where(live, dg, 0.0)
    return {"dx": dx.to(dt), "dlog_alpha": dg.to(dt), "dh0": a[:, 0] * dh[:, 0]}


def _plain_select(s, c):
    # values next to a border decide which tokens are picked: 64 bits
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    total = s["scores"].double()[..., None] + x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    done = s["finished"].bool()[..., None]
    pad = torch.arange(c["V"], device="cuda") == 0
    total = torch.where(done, torch.where(pad, s["scores"].double()[..., None], -math.inf), total)
    best, at = torch.sort(total.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, : c["M"]], at[:, : c["M"]]
    return {"token": (at % c["V"]).int(), "parent": (at // c["V"]).int(), "score": best.float()}


def _plain_reorder(s, c):
    first = torch.arange(c["N"], device="cuda")[:, None] * c["K"]
    rows = (first + s["parent"]).flatten()
    for t in s["states"]:
        t.copy_(t[rows])
    return s["states"]


# ---------------------------------------------------------------- work


def work(c):
    if c["op"] == "qk":
        e = 2 if c["dtype"] == "bf16" else 4
        rows, d = c["B"] * c["T"], c["d"]
        out_k = c["Hq"] if c["expand"] else c["Hk"]
        if c["way"] == "fwd":
            return {"bytes": rows * (d * e * (c["Hq"] + c["Hk"] + c["Hq"] + out_k) + 8), "flops": 8 * rows * d * (c["Hq"] + c["Hk"])}
        return {"bytes": rows * (d * (2 * e * (c["Hq"] + c["Hk"]) + 4 * (c["Hq"] + out_k)) + 8), "flops": 18 * rows * d * (c["Hq"] + c["Hk"])}
    if c["op"] == "scan":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"] * c["D"] * (0.75 if c["ragged"] else 1.0)
        if c["way"] == "fwd":
            return {"bytes": 3 * e * n + 8 * c["B"] * c["D"], "flops": 5 * n}
        whole = c["B"] * c["T"] * c["D"]  # gradients are written for every row
        return {"bytes": 3 * e * n + 2 * e * whole + 4 * c["B"] * c["D"] * (3 + -(-c["T"] // 64)), "flops": 12 * n}
    if c["op"] == "select":
        n = c["N"] * c["K"] * c["V"] * 0.9  # a finished beam's logits need not be read
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + c["N"] * (5 * c["K"] + 12 * c["M"]), "flops": 4 * n}
    K, H, d = c["K"], c["H"], c["d"]
    row = H * (4 * (d * d + (d * (d + 1) // 2 if c["packed"] else d * d) + d) + 8)
    # parents are uniform: a beam stays where it is with 1 / K; a carry is read if some other beam wants it
    written = K - 1
    read = K * (1 - (1 - 1 / K) ** (K - 1))
    return {"bytes": c["N"] * (row * (written + read) + 4 * K), "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "scan": _exact_scan, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](s, case)


def _exact_qk(s, c):
    """The rotation as a product of complex numbers, the gradient by differentiation."""
    B, T, d, r = c["B"], c["T"], c["d"], c["rot"]
    outs = {}
    for name, x, w in (("q", s["q"], s["wq"]), ("k", s["k"], s["wk"])):
        back = c["way"] == "bwd"
        x = x.double().contiguous().requires_grad_(back)
        w = None if w is None else w.double().requires_grad_(back)
        with torch.enable_grad():
            size = x.pow(2).sum(-1, keepdim=True)
            y = x / torch.sqrt(size / d + RMS_EPS) if name == "q" else x / torch.sqrt(size)
            y = y if w is None else y * w
            if r:
                turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[..., None] * s["inv_freq"].double())
                z = y[..., :r].unflatten(-1, (r // 2, 2)) if c["pairs"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, :, None])
                z = z.flatten(-2) if c["pairs"] else z.transpose(-1, -2).flatten(-2)
                y = torch.cat((z, y[..., r:]), -1)
            y = y.transpose(1, 2)
            if name == "k" and c["expand"]:
                y = y[:, :, None].expand(B, c["Hk"], c["Hq"] // c["Hk"], T, d).reshape(B, c["Hq"], T, d)
        if not back:
            outs[name] = y.contiguous()
            continue
        got = torch.autograd.grad(y, [x] if w is None else [x, w], s["d%s_out" % name].double())
        outs["d" + name] = got[0]
        outs["d%s_weight" % name] = got[1] if w is not None else None
    return (outs["q"], outs["k"]) if c["way"] == "fwd" else outs


def _exact_scan(s, c):
    """Token by token."""
    T = c["T"]
    n = (torch.full((c["B"],), T, device="cuda") if s["lengths"] is None else s["lengths"].long())[:, None]
    g, x = s["log_alpha"].double(), s["x"].double()
    a = g.exp()
    scale = 1 - a if c["complement"] else torch.ones_like(a)
    h, before = s["h0"].double(), []
    y = s["y"].double()
    for t in range(T):
        before.append(h)
        h = torch.where(t < n, torch.addcmul(scale[:, t] * x[:, t], a[:, t], h), h)
        if c["way"] == "fwd":
            y[:, t] = torch.where(t < n, h, y[:, t])
    if c["way"] == "fwd":
        return {"y": y, "h": h}
    d = s["dh"].double()
    dx, dg = torch.zeros_like(x), torch.zeros_like(x)
    for t in reversed(range(T)):
        live = t < n
        d = torch.where(live, d + s["dy"][:, t].double(), d)
        dx[:, t] = torch.where(live, d * scale[:, t], 0.0)
        da = d * (before[t] - x[:, t]) if c["complement"] else d * before[t]
        dg[:, t] = torch.where(live, da * a[:, t], 0.0)
        d = torch.where(live, d * a[:, t], d)
    return {"dx": dx, "dlog_alpha": dg, "dh0": d}


def _exact_select(s, c):
    p = torch.log_softmax(s["logits"].double(), -1) + s["scores"].double()[..., None]
    best = p.topk(min(c["M"], c["V"]), -1).values
    done = s["finished"].bool()[..., None]
    alone = torch.full_like(best, -math.inf)
    alone[..., 0] = s["scores"].double()
    best = torch.where(done, alone, best).flatten(1).sort(-1, descending=True).values
    return {"token": None, "parent": None, "score": best[:, : c["M"]]}


def _exact_reorder(s, c):
    rows = [c["K"] * i + p for i, ps in enumerate(s["parent"].tolist()) for p in ps]
    return [t.double()[rows] if t.is_floating_point() else None for t in s["states"]]
