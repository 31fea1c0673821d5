"""Cases of the operators that stand around a layer of linear attention, with their plain forms.

Three families, in the order a recurrent language model runs them:

  attn     linear attention with one decay for each head, S_t = a_t S_{t-1} + v_t k_t^T, o_t = s S_t q_t: single tokens,
           whole prompts (padded or packed sequences), and the gradient
  norm     group norm of each token, channels last, with an activation or a gate: what the attention's heads go through on
           the way to the output projection; and the gradient
  adjust   penalties for tokens seen, biases and grammar masks on logits: what comes before a selection

``run`` computes them in elementary torch operations; with ``own`` set, by the library's entry points.  ``exact`` holds
the definitions in 64 bits.
"""

import math
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one new token for each of four sequences (one request's beams), 16 heads of 128: a decode step where latency counts
        _attn("attn_step_few_bf16", "step", "bf16", B=4, T=1, H=16, dk=128, dv=128, held=True),
        # one new token for each of 256 sequences: a decode step that moves half a gigabyte of states
        _attn("attn_step_many_bf16", "step", "bf16", B=256, T=1, H=16, dk=128, dv=128, held=True),
        # a prefill of 4 prompts of 4096 tokens, 16 heads of 128
        _attn("attn_prefill_bf16", "fwd", "bf16", B=4, T=4096, H=16, dk=128, dv=128),
        # one sequence of 20480 tokens that continues from a state, a fixed decay for each head
        _attn("attn_long_bf16", "fwd", "bf16", B=1, T=20480, H=16, dk=128, dv=128, fixed=True, held=True),
        # prompts of odd lengths one behind the other, fp32, narrow queries and keys shared by three heads
        _attn("attn_packed_f32", "fwd", "f32", B=7, T=777, H=6, dk=64, dv=128, share=3, rows="packed"),
        # the training step's gradient: 4 x 4096 tokens, 16 heads of 128
        _attn("attn_backward_bf16", "bwd", "bf16", B=4, T=4096, H=16, dk=128, dv=128, held=True),
        # a decode step's outputs, 64 tokens of 16 heads of 128, on their way to the projection
        _norm("norm_step_bf16", "fwd", "bf16", B=64, T=1, G=16, d=128, center=False, act="silu", gate=True),
        # the prefill's: head-major as the read step leaves them, gated
        _norm("norm_prefill_bf16", "fwd", "bf16", B=4, T=4096, G=16, d=128, center=False, act="silu", gate=True),
        # the training step's gradient, centred, the activation on the norm itself, fp32, odd sizes
        _norm("norm_backward_f32", "bwd", "f32", B=3, T=2047, G=12, d=80, center=True, act="silu", gate=False),
        # one request with four beams, a few hundred tokens seen
        _adjust("adjust_one_f32", "f32", N=1, K=4, V=32000, L=300, bias=8, mask=True),
        # 32 requests with eight beams over a large odd vocabulary, thousands of tokens seen
        _adjust("adjust_many_bf16", "bf16", N=32, K=8, V=131071, L=4096, bias=64, mask=True),
    ]


def draw(rng: random.Random):
    kind = rng.choice(["step", "fwd", "fwd", "bwd", "norm_fwd", "norm_bwd", "adjust"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("step", "fwd", "bwd"):
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        share = rng.choice([1, 1, 1, 2, 3, 4])
        H = share * rng.choice([1, 2, 3, 4, 5])
        if kind == "step":
            return _free(_attn("", "step", dtype, B=_log(rng, 1, 256 * 16 // H), T=1, H=H, dk=dk, dv=dv, share=share, held=True))
        most = 4 * 4096 * 16 // H  # rows that the largest listed case has for so many heads
        if dtype == "f32":
            most //= 6
        T = _log(rng, 2, min(most, 20480 if kind == "fwd" else 8192))
        rows = rng.choice(["all", "all", "padded", "packed"]) if T > 8 else "all"
        c = _attn("", kind, dtype, B=min(64, max(1, _log(rng, 1, most) // T)), T=T, H=H, dk=dk, dv=dv, share=share, rows=rows,
                  fixed=rng.random() < 0.3, held=rng.random() < 0.5)
        return _free(c)
    if kind.startswith("norm"):
        d = 8 * rng.choice([4, 8, 8, 10, 16, 16, 24, 32, 64])
        G = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        most = 4 * 4096 * 2048 // (2 if dtype == "f32" else 1) // (2 if kind == "norm_bwd" else 1)
        tokens = _log(rng, 1, max(1, most // (G * d)))
        T = min(tokens, _log(rng, 1, 8192))
        gate = rng.random() < 0.5
        return _free(_norm("", kind[5:], dtype, B=max(1, tokens // T), T=T, G=G, d=d, center=rng.random() < 0.5,
                           act=rng.choice(["none", "silu", "silu", "sigmoid"]), gate=gate))
    K = rng.choice([1, 2, 3, 4, 5, 8])
    V = _log(rng, 1000, 131072)
    N = _log(rng, 1, max(1, min(64, 33_000_000 // (K * V * (2 if dtype == "f32" else 1)))))
    return _free(_adjust("", dtype, N=N, K=K, V=V, L=_log(rng, 1, 8192), bias=rng.choice([0, 1, 7, 64, 300]), mask=rng.random() < 0.6))


def _free(c):
    del c["name"]
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def _attn(name, way, dtype, B, T, H, dk, dv, share=1, rows="all", fixed=False, held=False):
    """share: heads of a query and key; rows: "all" T of each sequence, "padded" to T, or "packed" one behind the other;
    fixed: a decay for each head, not for each token too; held: sequences go on from a state."""
    return dict(name=name, op="attn", way=way, dtype=dtype, B=B, T=T, H=H, dk=dk, dv=dv, share=share, rows=rows, fixed=fixed,
                held=held)


def _norm(name, way, dtype, B, T, G, d, center, act, gate):
    return dict(name=name, op="norm", way=way, dtype=dtype, B=B, T=T, G=G, d=d, center=center, act=act, gate=gate)


def _adjust(name, dtype, N, K, V, L, bias, mask):
    return dict(name=name, op="adjust", dtype=dtype, N=N, K=K, V=V, L=L, bias=bias, mask=mask)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"attn": _prepare_attn, "norm": _prepare_norm, "adjust": _prepare_adjust}[case["op"]](case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lengths(c):
    """Tokens of each sequence; the longest has T.  They make the packed tensors' shape, so they are the case's own."""
    r = random.Random(1000 * c["T"] + c["B"])
    return [c["T"]] + [r.randint(1, c["T"]) for _ in range(c["B"] - 1)]


def _prepare_attn(c, g):
    dt = DTYPES[c["dtype"]]
    B, T, H, dk, dv, Hq = c["B"], c["T"], c["H"], c["dk"], c["dv"], c["H"] // c["share"]
    s = dict(case=c, lengths=None, offsets=None)
    rows = (B, T)
    if c["rows"] != "all":
        n = _lengths(c)
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        if c["rows"] == "packed":
            s["offsets"] = torch.tensor([0] + n, device="cuda").cumsum(0).int()
            rows = (1, sum(n))
    # what the projection leaves: queries, keys, values side by side; keys are unit vectors
    packed = _randn(g, *rows, 2 * Hq * dk + H * dv, dtype=dt)
    s["q"] = packed[..., : Hq * dk].view(*rows, Hq, dk)
    s["k"] = packed[..., Hq * dk : 2 * Hq * dk].view(*rows, Hq, dk)
    s["k"].copy_(torch.nn.functional.normalize(s["k"].float(), dim=-1))
    s["v"] = packed[..., 2 * Hq * dk :].view(*rows, H, dv)
    if c["fixed"]:
        # heads that remember 32 tokens, 64, 128 and so on
        gate = torch.log1p(-torch.exp2(-5.0 - torch.arange(H, device="cuda", dtype=torch.float64) % 8))
        s["log_alpha"] = gate.to(dt).expand(*rows, H)
    else:
        s["log_alpha"] = (torch.nn.functional.logsigmoid(_randn(g, *rows, H) + 2.0) / 2).to(dt)
    s["scale"] = dk ** -0.5
    s["S0"] = _randn(g, B, H, dv, dk) if c["held"] else None
    if c["way"] == "bwd":
        s["do"] = _randn(g, *rows, H, dv, dtype=dt)
        s["dS"] = 0.1 * _randn(g, B, H, dv, dk)
    else:
        s["o"] = torch.zeros(*rows, H, dv, device="cuda", dtype=dt)
        s["S"] = torch.empty(B, H, dv, dk, device="cuda")
    return s


def _prepare_norm(c, g):
    dt = DTYPES[c["dtype"]]
    B, T, G, d = c["B"], c["T"], c["G"], c["d"]
    # the heads' outputs are head-major
    s = dict(case=c, x=(_randn(g, B, G, T, d) * torch.exp(_randn(g, B, G, T, 1)) + 0.3).to(dt).transpose(1, 2))
    s["gate"] = _randn(g, B, T, G, d, dtype=dt) if c["gate"] else None
    s["weight"] = 1.0 + 0.1 * _randn(g, G, d)
    s["bias"] = 0.1 * _randn(g, G, d) if c["center"] else None
    if c["way"] == "bwd":
        s["dy"] = _randn(g, B, T, G, d, dtype=dt)
    return s


def _prepare_adjust(c, g):
    N, K, V, L = c["N"], c["K"], c["V"], c["L"]
    R = N * K
    s = dict(case=c, logits=(2.5 * _randn(g, N, K, V)).to(DTYPES[c["dtype"]]))
    # text repeats itself: tokens of a history are drawn towards the front of the vocabulary
    s["history"] = (V * _rand(g, R, L) ** 3).int().clamp_max(V - 1)
    s["lengths"] = torch.randint(0, L + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    s["prompt"] = (s["lengths"] * _rand(g, R)).int()
    s["repetition"] = 1.0 + 0.3 * _rand(g, R)
    s["presence"], s["frequency"] = 0.5 * _rand(g, R), 0.2 * _rand(g, R)
    s["bias_token"] = torch.randint(0, V, (R, c["bias"]), generator=g, device="cuda", dtype=torch.int32) if c["bias"] else None
    s["bias_value"] = _randn(g, R, c["bias"]) if c["bias"] else None
    # a grammar lets some words of 32 tokens through whole, some not at all, some in part
    s["allowed"] = None
    if c["mask"]:
        words = (V + 31) // 32
        bits = torch.randint(-2**31, 2**31, (R, words), generator=g, device="cuda", dtype=torch.int64).int()
        which = _rand(g, R, words)
        s["allowed"] = torch.where(which < 0.3, torch.zeros_like(bits), torch.where(which < 0.5, torch.full_like(bits, -1), bits))
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"attn": _plain_attn, "norm": _plain_norm, "adjust": _plain_adjust}[c["op"]](s, c)


def _run_own(s, c):
    import curvature_conditioned_query_amd as ccq

    if c["op"] == "attn":
        how = dict(log_alpha=s["log_alpha"], scale=s["scale"], S0=s["S0"])
        if c["rows"] == "packed":
            how.update(offsets=s["offsets"], max_length=c["T"])
        elif c["rows"] == "padded":
            how.update(lengths=s["lengths"])
        if c["way"] == "bwd":
            return ccq.ccq_linear_attn_backward(s["q"], s["k"], s["v"], s["do"], dS_out=s["dS"], want_dS0=s["S0"] is not None, **how)
        o = ccq.ccq_linear_attn(s["q"], s["k"], s["v"], o=s["o"], S_out=s["S"], **how)
        return {"o": o, "S": s["S"]}
    if c["op"] == "norm":
        how = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], center=c["center"], eps=EPS, activation=c["act"])
        if c["way"] == "fwd":
            return ccq.ccq_group_norm(s["x"], **how)
        return ccq.ccq_group_norm_backward(s["x"], s["dy"], **how)
    return ccq.ccq_logits_adjust(s["logits"], history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompt"],
                                 repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                 bias_token=s["bias_token"], bias_value=s["bias_value"], allowed=s["allowed"])


# ---------------------------------------------------------------- plain forms


def _rows(s, c, x):
    """x [B, T, ..] or packed rows [1, total, ..] as [B, T, ..], zeros behind a sequence's end."""
    if s["lengths"] is None:
        return x
    t = torch.arange(c["T"], device="cuda")
    live = t < s["lengths"][:, None]
    live = live.view(*live.shape, *[1] * (x.dim() - 2))
    if s["offsets"] is not None:
        x = x[0][(s["offsets"][:-1, None] + t).clamp_max(x.shape[1] - 1)]
    return torch.where(live, x, 0.0)


def _unrows(s, c, x, old):
    """x [B, T, ..] where it belongs in `old`, which has the inputs' rows."""
    if s["lengths"] is None:
        return x
    live = torch.arange(c["T"], device="cuda") < s["lengths"][:, None]
    if s["offsets"] is not None:
        return x[live][None]
    return torch.where(live.view(*live.shape, *[1] * (x.dim() - 2)), x, old)


def _heads(x, share):
    """[B, T, Hx, d] -> [B, H, T, d] in 32 bits."""
    return x.float().repeat_interleave(share, 2).transpose(1, 2)


def _chunks(x, T):
    """[.., T, d] -> [.., chunks, 64, d], zeros behind T."""
    x = torch.nn.functional.pad(x, (0, 0, 0, -T % CHUNK))
    return x.unflatten(-2, (-1, CHUNK))


def _decayed(x, y, z, g, state):
    """out_i = e^{g_1 + .. + g_i} state x_i + sum_{j <= i} e^{g_{j+1} + .. + g_i} (x_i y_j) z_j, and the state behind the
    last token, [.., dx, dz].  Sums of gates are long: 64 bits."""
    T = x.shape[-2]
    x, y, z = _chunks(x, T), _chunks(y, T), _chunks(z, T)
    run = _chunks(g[..., None], T)[..., 0].cumsum(-1)
    whole = run[..., -1].cumsum(-1)
    tri = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    near = (run[..., :, None] - run[..., None, :]).masked_fill(~tri, -math.inf).exp().float()
    out = ((x @ y.transpose(-1, -2)) * near) @ z
    added = (y * (run[..., -1:] - run).exp().float()[..., None]).transpose(-1, -2) @ z
    # the state before every chunk, and behind the last: a sum over the chunks before it
    C = whole.shape[-1]
    before = torch.nn.functional.pad(whole, (1, 0))  # [.., C + 1]
    far = torch.ones(C + 1, C, device="cuda", dtype=torch.bool).tril(-1)
    far = (before[..., :, None] - whole[..., None, :]).masked_fill(~far, -math.inf).exp().float()
    states = (far @ added.flatten(-2)).unflatten(-1, added.shape[-2:])
    if state is not None:
        states = states + before.exp().float()[..., None, None] * state[..., None, :, :]
    out = out + run.exp().float()[..., None] * (x @ states[..., :-1, :, :])
    return out.flatten(-3, -2)[..., :T, :], states[..., -1, :, :]


def _plain_attn(s, c):
    dt = DTYPES[c["dtype"]]
    B, T, H, share = c["B"], c["T"], c["H"], c["share"]
    q, k, v = (_heads(_rows(s, c, s[n]), f) for n, f in (("q", share), ("k", share), ("v", 1)))
    g = _rows(s, c, s["log_alpha"]).double().transpose(1, 2)
    S0 = s["S0"]
    if c["way"] != "bwd":
        o, S = _decayed(q, k, v, g, None if S0 is None else S0.transpose(-1, -2))
        o = (s["scale"] * o).transpose(1, 2).to(dt)
        return {"o": _unrows(s, c, o, s["o"]), "S": S.transpose(-1, -2).contiguous()}
    do, dS = s["scale"] * _heads(_rows(s, c, s["do"]), 1), s["dS"]
    dq, S = _decayed(do, v, k, g, S0)
    # from the end: the gate that leads from a token to the next
    back = torch.cat((g[..., 1:], torch.zeros_like(g[..., :1])), -1).flip(-1)
    dk, A = _decayed(v.flip(-2), do.flip(-2), q.flip(-2), back, dS)
    dv, _ = _decayed(k.flip(-2), q.flip(-2), do.flip(-2), back, dS.transpose(-1, -2))
    dk, dv = dk.flip(-2), dv.flip(-2)
    r = ((q * dq).sum(-1) - (k * dk).sum(-1)).double()
    dg = (r.flip(-1).cumsum(-1).flip(-1) + (S * dS).double().sum((-1, -2))[..., None]).float()
    if s["lengths"] is not None:
        dg = torch.where(torch.arange(T, device="cuda") < s["lengths"][:, None, None], dg, 0.0)
    shared = lambda x: x.unflatten(1, (H // share, share)).sum(2)  # noqa: E731
    out = dict(dq=shared(dq), dk=shared(dk), dv=dv)
    out = {n: _unrows(s, c, x.transpose(1, 2).to(dt), torch.zeros((), device="cuda", dtype=dt)) for n, x in out.items()}
    out["dlog_alpha"] = _unrows(s, c, dg.transpose(1, 2).to(dt), torch.zeros((), device="cuda", dtype=dt))
    if S0 is not None:
        out["dS0"] = g[..., 0].exp().float()[..., None, None] * A
    return out


def _act(x, kind):
    if kind == "none":
        return x
    return x * torch.sigmoid(x) if kind == "silu" else torch.sigmoid(x)


def _act_slope(x, kind):
    if kind == "none":
        return torch.ones_like(x)
    p = torch.sigmoid(x)
    return p * (1 + x * (1 - p)) if kind == "silu" else p * (1 - p)


def _plain_norm(s, c):
    dt = DTYPES[c["dtype"]]
    x = s["x"].float()
    u = x - x.mean(-1, keepdim=True) if c["center"] else x
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    n = u * r
    z = n * s["weight"] if s["bias"] is None else n * s["weight"] + s["bias"]
    gate = None if s["gate"] is None else s["gate"].float()
    if c["way"] == "fwd":
        return (_act(z, c["act"]) if gate is None else z * _act(gate, c["act"])).to(dt).contiguous()
    dy = s["dy"].float()
    dz = dy * _act_slope(z, c["act"]) if gate is None else dy * _act(gate, c["act"])
    dn = dz * s["weight"]
    pull = dn.mean(-1, keepdim=True) if c["center"] else 0.0
    dx = r * (dn - pull - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": dx.to(dt), "dgate": None if gate is None else (dy * z * _act_slope(gate, c["act"])).to(dt),
            "dweight": (dz * n).sum((0, 1)), "dbias": None if s["bias"] is None else dz.sum((0, 1))}


def _plain_adjust(s, c):
    N, K, V, L = c["N"], c["K"], c["V"], c["L"]
    R = N * K
    x = s["logits"].float().view(R, V)
    t = torch.arange(L, device="cuda")
    at = s["history"].long()
    seen = t < s["lengths"][:, None]
    mine = seen & (t >= s["prompt"][:, None])
    seen = torch.zeros(R, V, device="cuda").scatter_add_(1, at, seen.float()) > 0
    count = torch.zeros(R, V, device="cuda").scatter_add_(1, at, mine.float())
    theta = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / theta, x * theta), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    if s["bias_token"] is not None:
        x = x + torch.zeros(R, V, device="cuda").scatter_add_(1, s["bias_token"].long(), s["bias_value"])
    if s["allowed"] is not None:
        token = torch.arange(V, device="cuda")
        bit = (s["allowed"][:, token // 32] >> (token % 32).int()) & 1
        x = torch.where(bit != 0, x, -math.inf)
    return x.to(DTYPES[c["dtype"]]).view(N, K, V)


# ---------------------------------------------------------------- work


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "attn":
        H, dk, dv, Hq = c["H"], c["dk"], c["dv"], c["H"] // c["share"]
        # lengths are uniform from 1 to T, the first is T
        n = c["B"] * c["T"] if c["rows"] == "all" else c["T"] * (c["B"] + 1) / 2
        state = 4 * c["B"] * H * dk * dv
        inputs = n * (e * (2 * Hq * dk + H * dv) + (0 if c["fixed"] else e * H))
        held = 1 if c["held"] else 0
        if c["way"] != "bwd":
            return {"bytes": inputs + n * e * H * dv + (1 + held) * state, "flops": 5 * n * H * dk * dv}
        whole = n if c["rows"] == "packed" else c["B"] * c["T"]  # gradients are written for every row
        outputs = whole * e * (2 * Hq * dk + H * dv + H)
        return {"bytes": inputs + n * e * H * dv + outputs + (1 + 2 * held) * state, "flops": 14 * n * H * dk * dv}
    if c["op"] == "norm":
        n = c["B"] * c["T"] * c["G"] * c["d"]
        gate = 1 if c["gate"] else 0
        if c["way"] == "fwd":
            return {"bytes": n * e * (2 + gate), "flops": 10 * n}
        return {"bytes": n * e * (3 + 2 * gate), "flops": 25 * n}
    R, V = c["N"] * c["K"], c["V"]
    return {"bytes": R * (2 * V * e + (V / 8 if c["mask"] else 0) + 2 * c["L"] + 8 * c["bias"] + 20), "flops": R * (2 * V + 8 * c["L"])}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "norm": _exact_norm, "adjust": _exact_adjust}[case["op"]](s, case)


def _exact_attn(s, c):
    """Every sequence and head by itself: all pairs of tokens at once, the gradient by differentiation."""
    B, T, H, share = c["B"], c["T"], c["H"], c["share"]
    back = c["way"] == "bwd"
    if B * H * T * T * (8 if back else 3) > 2.5e10:
        return None
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    first = [0] * B if s["offsets"] is None else s["offsets"].tolist()[:-1]
    row = (lambda b: 0) if s["offsets"] is not None else (lambda b: b)
    full = {m: s[m].double() for m in ("q", "k", "v", "log_alpha")}
    outs = {}
    if back:
        for m in ("q", "k", "v", "log_alpha"):
            outs["d" + m] = torch.zeros(full[m].shape, dtype=torch.float64, device="cuda")
        if s["S0"] is not None:
            outs["dS0"] = torch.zeros_like(s["S0"], dtype=torch.float64)
    else:
        outs["o"] = s["o"].double()
        outs["S"] = torch.zeros_like(s["S"], dtype=torch.float64)
    for b in range(B):
        for h in range(H):
            at = (row(b), slice(first[b], first[b] + n[b]))
            q, k = full["q"][(*at, h // share)], full["k"][(*at, h // share)]
            v, g = full["v"][(*at, h)], full["log_alpha"][(*at, h)]
            S0 = None if s["S0"] is None else s["S0"][b, h].double()
            leaves = [t.detach().clone().requires_grad_(back) for t in (q, k, v, g)] + ([] if S0 is None else [S0.requires_grad_(back)])
            q, k, v, g = leaves[:4]
            with torch.enable_grad():
                run = torch.cumsum(g, 0)
                w = torch.exp(torch.tril(run[:, None] - run[None, :])).tril()
                o = (w * (q @ k.T)) @ v
                S = (v * torch.exp(run[-1] - run)[:, None]).T @ k
                if S0 is not None:
                    o = o + torch.exp(run)[:, None] * (q @ S0.T)
                    S = S + torch.exp(run[-1]) * S0
                o = s["scale"] * o
                if back:
                    loss = (o * s["do"][(*at, h)].double()).sum() + (S * s["dS"][b, h].double()).sum()
            if not back:
                outs["o"][(*at, h)] = o
                outs["S"][b, h] = S
                continue
            got = torch.autograd.grad(loss, leaves)
            for m, d, i in (("q", got[0], h // share), ("k", got[1], h // share), ("v", got[2], h), ("log_alpha", got[3], h)):
                outs["d" + m][(*at, i)] += d
            if S0 is not None:
                outs["dS0"][b, h] = got[4]
    return outs


def _exact_norm(s, c):
    back = c["way"] == "bwd"
    names = [n for n in ("x", "gate", "weight", "bias") if s[n] is not None]
    leaf = {n: s[n].double().contiguous().requires_grad_(back) for n in names}
    with torch.enable_grad():
        x = leaf["x"]
        if c["center"]:
            n = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + EPS)
        else:
            n = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS)
        z = n * leaf["weight"] + leaf.get("bias", 0.0)
        f = {"none": lambda t: t, "silu": lambda t: t / (1 + torch.exp(-t)), "sigmoid": lambda t: 1 / (1 + torch.exp(-t))}[c["act"]]
        y = z * f(leaf["gate"]) if "gate" in leaf else f(z)
    if not back:
        return y
    got = dict(zip(names, torch.autograd.grad(y, [leaf[n] for n in names], s["dy"].double())))
    return {"dx": got["x"], "dgate": got.get("gate"), "dweight": got["weight"], "dbias": got.get("bias")}


def _exact_adjust(s, c):
    """Row by row, over the tokens that occur."""
    V, L = c["V"], c["L"]
    out = s["logits"].double().view(-1, V).clone()
    lengths, prompts = s["lengths"].tolist(), s["prompt"].tolist()
    for r in range(out.shape[0]):
        n, p = lengths[r], prompts[r]
        theta = s["repetition"][r].double()
        old = torch.unique(s["history"][r, :n]).long()
        x = out[r, old]
        out[r, old] = torch.where(x > 0, x / theta, x * theta)
        new, times = torch.unique(s["history"][r, p:n], return_counts=True)
        out[r, new.long()] -= s["frequency"][r].double() * times + s["presence"][r].double()
        if s["bias_token"] is not None:
            out[r].index_add_(0, s["bias_token"][r].long(), s["bias_value"][r].double())
        if s["allowed"] is not None:
            words = s["allowed"][r].long() & 0xFFFFFFFF
            bits = (words[:, None] >> torch.arange(32, device="cuda")) & 1
            out[r].masked_fill_(bits.flatten()[:V] == 0, -math.inf)
    return out.view(s["logits"].shape)
