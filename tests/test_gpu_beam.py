"""ccq_beam_select and ccq_beam_reorder on the GPU against their fp64 definitions.

Tokens and parents are equal; scores are rounded once from 64 bits, the normaliser's fp32 part adding
at most 2^-24 of itself (its terms and its sums of 64 at a time round apart from each other, 64 2^-24 at
worst of the tail's share): |error| <= 2^-24 |score| + 64 2^-24.  Reordering moves bits.
"""

import numpy as np
import pytest

from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _run(logits, scores, m, finished=None, pad=0, tag=""):
    import torch
    from curvature_conditioned_query_amd import ccq_beam_select
    print(f"beam {tag} {tuple(logits.shape)} {logits.dtype} m={m}", flush=True)
    out = ccq_beam_select(logits, scores, m, finished=finished, pad_token=pad)
    again = ccq_beam_select(logits, scores, m, finished=finished, pad_token=pad)
    t, p, s = layer.beam_select(logits.double().cpu().numpy(), scores.double().cpu().numpy(), m,
                                None if finished is None else finished.cpu().numpy(), pad)
    assert np.array_equal(out["parent"].cpu().numpy(), p), tag
    assert np.array_equal(out["token"].cpu().numpy(), t), tag
    got = out["score"].double().cpu().numpy()
    fin = np.isfinite(s)
    assert np.array_equal(got[~fin], s[~fin])
    assert (np.abs(got[fin] - s[fin]) <= U * np.abs(s[fin]) + 64 * U).all()
    assert all(torch.equal(out[n], again[n]) for n in out)
    return out


def _logits(N, K, V, dtype, seed, stride=None):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(seed)
    x = (2.5 * torch.randn(N, 1, V, generator=g) + torch.randn(N, K, V, generator=g)).to(dt)
    if stride:
        wide = torch.full((N, K, stride), 1e4, dtype=dt)
        wide[..., :V] = x
        return wide.cuda()[..., :V], g
    return x.cuda(), g


def _uniform(N, K, g):
    import torch
    return torch.rand(N, K, generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V,m,stride", [
    (1, 1, 1, 1, None), (1, 4, 3, 12, None), (2, 3, 17, 5, None), (3, 2, 255, 4, 256), (1, 4, 2048, 4, None),
    (2, 5, 2049, 10, None), (1, 8, 5003, 64, None), (5, 4, 32001, 8, None), (40, 16, 1000, 16, 1003), (1, 1, 70000, 64, None),
    (64, 8, 9001, 16, None), (1, 64, 333, 64, None), (3, 4, 16384, 7, 16385)])
def test_select(gpu_lib, dtype, N, K, V, m, stride):
    import torch
    logits, g = _logits(N, K, V, dtype, V + K, stride)
    scores = (-4 * torch.rand(N, K, generator=g) - 3).cuda()
    _run(logits, scores, m, tag="plain")
    fin = torch.rand(N, K, generator=g).cuda() < 0.3
    _run(logits, scores, m, finished=fin, pad=V // 2, tag="finished")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,m", [(100, 10), (4099, 16), (40000, 64)])
def test_ties_go_to_the_lowest(gpu_lib, dtype, V, m):
    """Rows of one value, of few values, rising and falling rows, equal beams."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    scores = torch.zeros(1, 3).cuda()
    _run(torch.zeros(1, 3, V, dtype=dt).cuda(), scores, m, tag="constant")
    g = torch.Generator().manual_seed(1)
    _run(torch.randint(0, 3, (1, 1, V), generator=g).to(dt).expand(1, 3, V).contiguous().cuda(), scores, m, tag="three values, equal beams")
    ramp = (torch.arange(V, dtype=torch.float64) / V * 8).to(dt).expand(1, 3, V).contiguous().cuda()
    _run(ramp, scores, m, tag="rising")
    _run(ramp.flip(-1).contiguous(), scores, m, tag="falling")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5000, 20011])
@pytest.mark.parametrize("allowed", [0, 1, 3, 40])
def test_masked_vocabulary(gpu_lib, dtype, V, allowed):
    """Only a few tokens are allowed, down to none; the picks run out into -inf, lowest first."""
    import torch
    logits, g = _logits(2, 3, V, dtype, V)
    keep = torch.randperm(V, generator=g)[:allowed].cuda()
    x = torch.full_like(logits, -float("inf"))
    x[..., keep] = logits[..., keep]
    _run(x, (-torch.rand(2, 3, generator=g)).cuda(), 16, tag=f"{allowed} allowed")


def test_lowest_finite_mask(gpu_lib):
    """A mask of the type's lowest value: those tokens count as far away, not as absent."""
    import torch
    logits, g = _logits(1, 2, 3001, "f32", 8)
    x = torch.full_like(logits, torch.finfo(torch.float32).min)
    x[..., 7:9] = logits[..., 7:9]
    _run(x, torch.tensor([[-1.0, -1.5]]).cuda(), 8, tag="lowest value")


def test_nan_inf_and_dead_beams(gpu_lib):
    import torch
    inf, nan = float("inf"), float("nan")
    logits, _ = _logits(1, 4, 6001, "f32", 9)
    logits[0, 0, 5:3000] = nan
    logits[0, 1, 17], logits[0, 1, 4000] = inf, inf
    _run(logits, torch.tensor([[-1.0, -2.0, -3.0, -4.0]]).cuda(), 8, tag="nan and inf")
    _run(logits, torch.tensor([[0.0, -inf, nan, -inf]]).cuda(), 12, tag="first step: one live beam")
    _run(logits, torch.full((1, 4), -inf).cuda(), 12, tag="no live beam")
    logits[0, 0] = nan
    fin = torch.tensor([[0, 1, 1, 0]], dtype=torch.uint8).cuda()
    _run(logits, torch.tensor([[-1.0, nan, -inf, -2.0]]).cuda(), 12, finished=fin, pad=3, tag="finished and nan")
    _run(logits, torch.tensor([[-1.0, -5.0, -0.1, -inf]]).cuda(), 30, finished=torch.ones_like(fin), pad=20, tag="all finished")


def test_peaked_rows_where_few_terms_carry_the_sum(gpu_lib):
    """Rows with one token far above, and rows whose large logits all lie on one thread."""
    import torch
    logits, g = _logits(4, 4, 40003, "f32", 10)
    logits[:, :, 12345] += 30.0
    logits[1, :, 8 : 8 + 4] += 25.0
    logits[2, :, 2048 * torch.arange(19)] += 20.0
    _run(logits, (-torch.rand(4, 4, generator=g)).cuda(), 32, tag="peaked")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,m", [(250, 64), (513, 1), (900, 64), (1532, 24), (2049, 64), (20857, 10)])
def test_rows_that_end_in_the_first_waves_of_a_piece(gpu_lib, dtype, V, m):
    logits, g = _logits(6, 12, V, dtype, V)
    _run(logits, (-_uniform(6, 12, g)).cuda(), m, tag="short")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 16, 64])
def test_long_rows_that_rise(gpu_lib, dtype, m):
    """Every later token is better, so that the wave's list fills again and again; equal values among them."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    N, K, V = 64, 16, 12001
    g = torch.Generator().manual_seed(m)
    x = (torch.arange(V, dtype=torch.float32) / V * 12 + 0.05 * torch.rand(V, generator=g)).to(dt).expand(N, K, V).contiguous().cuda()
    _run(x, (-_uniform(N, K, g)).cuda(), m, tag="rising")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 7, 64])
def test_rows_of_several_pieces(gpu_lib, dtype, m):
    """1024 rows, so that a workgroup goes through a whole row of 8192 tokens and 900 more: ties, masks, NaN and
    infinities that begin in the second part or end with the first."""
    import torch
    N, K, V, cut = 64, 16, 9092, 8192
    inf, nan = float("inf"), float("nan")
    x, g = _logits(N, K, V, dtype, m)
    rows = x.view(N * K, V)
    few = torch.randperm(cut, generator=g)[:5].cuda()
    late = cut + torch.randperm(V - cut, generator=g)[:5].cuda()
    rows[0::12] = 0.5
    rows[1::12] = torch.randint(0, 3, (V,), generator=g).cuda().to(x.dtype)
    for start, keep in ((2, few), (3, late), (4, few[:0])):
        kept = rows[start::12][:, keep].clone()
        rows[start::12] = -inf
        rows[start::12, keep] = kept
    rows[5::12, cut + 3] = nan
    rows[6::12, cut + 7] = inf
    rows[7::12, :cut] = torch.finfo(x.dtype).min
    rows[8::12, :cut] = -inf
    rows[9::12, cut:] = -inf
    rows[10::12] = torch.linspace(5, -5, V).cuda().to(x.dtype)
    _run(x, (-_uniform(N, K, g)).cuda(), m, tag="pieces")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V,m", [(64, 9001, 64), (40, 14337, 7), (16, 41115, 16), (64, 40000, 64), (3, 250001, 8)])
def test_one_request_of_many_beams(gpu_lib, dtype, K, V, m):
    """Its lists are kept to a workgroup's threads, so that stretches get longer: ties and masks at their ends."""
    import torch
    x, g = _logits(1, K, V, dtype, K)
    rows = x[0]
    rows[0] = 0.5
    rows[1] = torch.randint(0, 3, (V,), generator=g).cuda().to(x.dtype)
    rows[2, : V - 3] = -float("inf")
    if K > 8:
        rows[3, 2048] = float("nan")
        rows[4, 2047] = float("inf")
        rows[5, 2048:] = -float("inf")
        rows[6] = torch.linspace(-5, 5, V).cuda().to(x.dtype)
        rows[7] = rows[6]
    _run(x, (-_uniform(1, K, g)).cuda(), m, tag="one request")
    _run(x, torch.zeros(1, K).cuda(), m, tag="one request, equal scores")


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8, 13, 16, 17, 40, 64])
def test_reorder(gpu_lib, K):
    """States of many row sizes and types, moved in place by every kind of parents."""
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder
    print(f"reorder K={K}", flush=True)
    N = 3
    g = torch.Generator().manual_seed(K)
    make = lambda *shape: torch.randn(N * K, *shape, generator=g).cuda()  # noqa: E731
    states = [make(2, 16, 16), make(1), make(5, 3), make(4097), torch.randint(0, 1 << 40, (N * K, 3), generator=g).cuda(),
              make(2, 6).to(torch.bfloat16), torch.randint(0, 256, (N * K, 8), generator=g).to(torch.uint8).cuda()]
    for kind in ("random", "same", "all one", "cycle", "outside"):
        parent = {"random": torch.randint(0, K, (N, K), generator=g), "same": torch.arange(K).expand(N, K),
                  "all one": torch.full((N, K), K // 2), "cycle": (torch.arange(K) + 1).remainder(K).expand(N, K),
                  "outside": torch.randint(-2, K + 2, (N, K), generator=g)}[kind].to(torch.int32).contiguous()
        want = [torch.from_numpy(layer.beam_reorder(s.float().cpu().numpy() if s.dtype == torch.bfloat16 else s.cpu().numpy(),
                                                    parent.numpy())) for s in states]
        ccq_beam_reorder(states, parent.cuda())
        for s, w in zip(states, want):
            assert torch.equal(s.cpu().to(w.dtype), w), kind


def test_reorder_leaves_neighbours_alone(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder
    buf = torch.randn(12, 1000, device="cuda")
    keep = buf.clone()
    ccq_beam_reorder([buf[4:8]], torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device="cuda"))
    assert torch.equal(buf[:4], keep[:4]) and torch.equal(buf[8:], keep[8:])
    assert torch.equal(buf[4:8], keep[[5, 4, 7, 7]])


def test_other_stream_and_replayed_capture(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder, ccq_beam_select
    logits, g = _logits(3, 4, 9000, "bf16", 12)
    scores = -torch.rand(3, 4, generator=g).cuda()
    state, fresh = torch.randn(12, 700, device="cuda"), torch.randn(12, 700, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want, got = ccq_beam_select(logits, scores, 4), ccq_beam_select(logits, scores, 4, stream=side)
    side.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ccq_beam_select(logits, scores, 4)
        ccq_beam_reorder([state], out["parent"])
    for _ in range(4):
        logits.copy_(torch.randn(logits.shape, device="cuda"))
        want = ccq_beam_select(logits, scores, 4)
        state.copy_(fresh)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want)
        rows = (torch.arange(3, device="cuda")[:, None] * 4 + want["parent"]).flatten().long()
        assert torch.equal(state, fresh[rows])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V,m", [(8, 5, 16), (16, 3, 8), (4, 20, 32), (2, 40, 64), (32, 2, 4), (13, 3, 9)])
def test_lists_shorter_than_the_picks(gpu_lib, dtype, K, V, m):
    """No list has an entry at the depth that the join looks at first, and 65 to 128 entries in all, held by
    two waves: none of them may be lost."""
    logits, g = _logits(40, K, V, dtype, V + m)
    for i in range(3):
        _run(logits, (-_uniform(40, K, g)).cuda(), m, tag=f"short lists {i}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,m", [(50, 49, 8), (5000, 4999, 16), (5000, 3000, 64), (3, 2, 2)])
def test_finished_beams_without_a_score(gpu_lib, dtype, V, pad, m):
    """A finished beam at -inf or NaN has nothing but continuations at -inf, its pad token among them: they go
    in order of token, wherever that token stands."""
    import torch
    inf, nan = float("inf"), float("nan")
    logits, _ = _logits(4, 2, V, dtype, V)
    scores = torch.tensor([[-inf, -inf], [nan, -1.0], [-inf, nan], [-2.0, -inf]]).cuda()
    fin = torch.tensor([[1, 0], [1, 1], [1, 1], [1, 1]], dtype=torch.uint8).cuda()
    _run(logits, scores, m, finished=fin, pad=pad, tag="finished without a score")


MASKS = [-1e3, -1e4, -1e6, -1e7, -1e9, -1e10, -1e11, -1e12, -1e18, -1e20, -1e30, -1e38, 1e4]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V,m", [(1, 15, 32000, 8), (2, 15, 70001, 16), (70, 15, 9000, 16)])
def test_finite_masks_of_every_size(gpu_lib, dtype, N, K, V, m):
    """Rows, stretches and a row's first or last 8192 tokens at one far value: it counts as what it is, and what stands
    beside it as if it stood alone."""
    import torch
    for where in ("row", "first", "last", "all but a few"):
        logits, g = _logits(N, K, V, dtype, V)
        for i, value in enumerate(MASKS):
            part = {"row": slice(0, V), "first": slice(0, 8192), "last": slice(V - 8192, V), "all but a few": slice(3, V - 2)}[where]
            logits[:, i, part] = value
        _run(logits.view(N * K, 1, V), -torch.ones(N * K, 1).cuda(), m, tag=f"{where}, one beam a request")
        _run(logits, (-_uniform(N, K, g)).cuda(), m, tag=where)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [60.0, 1e3, -1e3, 1e4, -1e4, 1e6])
def test_scores_do_not_depend_on_an_offset(gpu_lib, dtype, offset):
    logits, g = _logits(2, 4, 32001, dtype, 5)
    moved = (logits.float() + offset).to(logits.dtype)
    _run(moved, (-_uniform(2, 4, g)).cuda(), 8, tag=f"offset {offset}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V,m", [(64, 16, 32003, 16), (64, 16, 24577, 1), (64, 16, 26000, 64), (1, 64, 100000, 16), (1, 8, 253000, 8)])
def test_pieces_far_above_the_first(gpu_lib, dtype, N, K, V, m):
    """A workgroup goes through three and more pieces, and the first tells nothing of the rest: at -inf, at a mask,
    or of a row that rises by several hundred.  Every later token is in the normaliser."""
    import torch
    x, g = _logits(N, K, V, dtype, V)
    rows = x.view(N * K, V)
    lowest = torch.finfo(x.dtype).min
    rows[0::8, :8192] = -float("inf")
    rows[1::8, :8192] = -1e4
    rows[2::8, :8192] = lowest
    rows[3::8] = rows[3::8] * 0.1 + torch.linspace(-300, 400, V).cuda().to(x.dtype)
    rows[4::8, : V // 2] = -float("inf")
    rows[5::8, 8192:16384] -= 200
    rows[6::8, :8192] -= 100
    rows[7::8] = torch.linspace(400, -300, V).cuda().to(x.dtype)
    _run(x, (-_uniform(N, K, g)).cuda(), m, tag="rising pieces")
    _run(x.view(N * K, 1, V), -torch.ones(N * K, 1).cuda(), m, tag="rising pieces, one beam a request")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-3.0, -0.0, -1e4, 2.0])
def test_rows_of_one_value_in_several_pieces(gpu_lib, dtype, value):
    """The bound is the row's one value, positive or negative: no token lies above it, and the lowest are looked up."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x = torch.full((64, 16, 20000), value, dtype=dt).cuda()
    x[5:, :, 17000] += 1
    _run(x, torch.zeros(64, 16).cuda(), 16, tag=f"all {value}")


def test_selections_in_flight_together(gpu_lib):
    """Calls on several streams at once, each with its own workspace, and one captured graph replayed among them."""
    import torch
    from curvature_conditioned_query_amd import ccq_beam_select
    sets = []
    for i, (N, K, V, m) in enumerate(((64, 16, 26000, 16), (1, 8, 32001, 8), (7, 5, 20, 32), (3, 64, 9001, 64))):
        logits, g = _logits(N, K, V, "bf16" if i % 2 else "f32", 40 + i)
        logits[..., : V // 2] = -1e10 if i % 2 else -float("inf")
        sets.append((logits, -_uniform(N, K, g).cuda(), m))
    want = [ccq_beam_select(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [ccq_beam_select(*s) for s in sets]
    for _ in range(4):
        graph.replay()
        got = [ccq_beam_select(*s, stream=t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, kept):
            assert all(torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]) for n in a)
