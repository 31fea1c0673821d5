"""The operators around the read step on tensors of more than 2^32 elements.

A token, channel, row or request is worked on alike wherever it stands, so the ends of a large call are
compared with a small call on the same values: equal bits, but for selection's scores, whose sums are cut
differently (each within 2^-24 |score| + 64 2^-24 of the score in 64 bits, so twice that apart).
"""

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _memory(gpu_lib):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def test_scan_and_gradient(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_scan, ccq_scan_backward
    T, D = 260, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(1)
    row = lambda: torch.randn(1, 1, D, device="cuda", generator=g).to(torch.bfloat16)
    x, la, dy = row().expand(1, T, D), (-row().abs()).expand(1, T, D), row().expand(1, T, D)
    y = ccq_scan(x, la)
    assert y.numel() > 1 << 32
    y2 = ccq_scan(y, la)  # reads past 2^32 elements too
    out = ccq_scan_backward(y, la, dy)
    for part in (slice(0, 136), slice(D // 2, D // 2 + 8), slice(D - 264, D)):
        cut = [t[..., part] for t in (x, la, dy)]
        small = ccq_scan(*cut[:2])
        assert torch.equal(y[..., part], small)
        assert torch.equal(y2[..., part], ccq_scan(small, cut[1]))
        back = ccq_scan_backward(small, cut[1], cut[2])
        assert torch.equal(out["dx"][..., part], back["dx"]) and torch.equal(out["dlog_alpha"][..., part], back["dlog_alpha"])


def test_qk_norm_rope_and_gradient(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_qk_norm_rope, ccq_qk_norm_rope_backward
    T, H, d = (1 << 20) + 3, 32, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(1, 1, H, d, device="cuda", generator=g).to(torch.bfloat16).expand(1, T, H, d)
    freq = torch.rand(32, device="cuda", generator=g)
    kw = dict(inv_freq=freq, q_norm="l2")
    out, _ = ccq_qk_norm_rope(q, None, **kw)
    assert out.numel() > 1 << 32
    grad = torch.zeros(1, H, T, d, device="cuda")
    for part in (slice(0, 7), slice(T - 9, T)):
        grad[:, :, part] = torch.randn(grad[:, :, part].shape, device="cuda", generator=g)
    dq = ccq_qk_norm_rope_backward(q, None, grad, None, **kw)["dq"]
    for part in (slice(0, 7), slice(T - 9, T)):
        here = dict(kw, position_offset=part.start)
        assert torch.equal(out[:, :, part], ccq_qk_norm_rope(q[:, part], None, **here)[0])
        small = ccq_qk_norm_rope_backward(q[:, part], None, grad[:, :, part].contiguous(), None, **here)["dq"]
        assert torch.equal(dq[:, part], small)
    assert not any(dq[0, at : at + 65536].any() for at in range(7, T - 9 - 65536, 65536))
    turned, _ = ccq_qk_norm_rope(out.transpose(1, 2), None, q_norm="none")  # reads past 2^32 elements too
    assert all(torch.equal(turned[0, h], out[0, h]) for h in range(H))


def test_beam_select(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_beam_select
    N, K, V = 65, 8, 1 << 23
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty(N, K, V, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    scores = -torch.rand(N, K, device="cuda", generator=g)
    out = ccq_beam_select(logits, scores, 16)
    for n in (0, N - 1):
        small = ccq_beam_select(logits[n : n + 1], scores[n : n + 1], 16)
        assert torch.equal(out["token"][n], small["token"][0]) and torch.equal(out["parent"][n], small["parent"][0])
        assert ((out["score"][n] - small["score"][0]).abs() <= 2 * (U * small["score"][0].abs() + 64 * U)).all()


def test_normaliser_of_very_long_rows(gpu_lib):
    """67 million tokens a row, 2048 pieces for a workgroup, all but one token at a value whose terms' fp32 sum
    drifts: the score is the closed form's to the same bound as a short row's."""
    import math
    import torch
    from curvature_conditioned_query_amd import ccq_beam_select
    N, V = 256, 1 << 26
    logits = torch.empty(N, 1, V, device="cuda", dtype=torch.bfloat16)
    for d in (1.5625, 1.75, 1.8125):
        logits.fill_(-d)
        logits[..., 77] = 0
        out = ccq_beam_select(logits, torch.zeros(N, 1, device="cuda"), 2)
        best = -math.log1p((V - 1) * math.exp(-d))
        assert (out["token"][:, 0] == 77).all() and (out["token"][:, 1] == 0).all()
        for i, want in enumerate((best, best - d)):
            assert ((out["score"][:, i].double() - want).abs() <= U * abs(want) + 64 * U).all(), (d, i)


def test_beam_reorder(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder
    for cols in ((1 << 30) + 4, (1 << 30) + 1):
        count = torch.arange(cols, device="cuda", dtype=torch.int32)
        state = torch.empty(4, cols, device="cuda", dtype=torch.int32)
        for j in range(4):
            state[j] = count + 11 * j
        assert state.numel() > 1 << 32
        ccq_beam_reorder([state], torch.tensor([[3, 0, 0, 2]], dtype=torch.int32, device="cuda"))
        for j, was in enumerate((3, 0, 0, 2)):
            assert torch.equal(state[j] - 11 * was, count)
        del state


@pytest.mark.parametrize("K", [1, 2, 3, 8, 11, 16, 33, 64])
@pytest.mark.parametrize("odd", [0, 1])
def test_beam_reorder_past_the_caches(gpu_lib, K, odd):
    """States of more than 128 MB, which are moved past the caches: rows of whole and of broken 16 bytes."""
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder
    N = 3
    cols = (150 << 20) // 4 // (N * K) // 4 * 4 + odd
    g = torch.Generator(device="cuda").manual_seed(K)
    state = torch.randint(-(1 << 31), 1 << 31, (N * K, cols), device="cuda", dtype=torch.int32, generator=g)
    small = torch.rand(N * K, 5, device="cuda", generator=g)
    parent = torch.randint(0, K, (N, K), device="cuda", dtype=torch.int32, generator=g)
    rows = (torch.arange(N, device="cuda")[:, None] * K + parent).view(-1)
    want, want_small = state[rows], small[rows]
    ccq_beam_reorder([small, state], parent)
    assert torch.equal(state, want) and torch.equal(small, want_small)


def test_launches_of_the_most_workgroups(gpu_lib):
    """The last sizes before the refusals: sequences, rows and requests by the million, alike or short, their ends
    compared with small calls."""
    import torch
    from curvature_conditioned_query_amd import ccq_beam_reorder, ccq_beam_select, ccq_scan, ccq_scan_backward
    g = torch.Generator(device="cuda").manual_seed(4)
    for dt, T, B in ((torch.bfloat16, 9, (1 << 26) - 8), (torch.bfloat16, 65, (1 << 23) - 1)):
        print(f"scan T{T} B{B}", flush=True)
        x, la = torch.randn(2, 1, T, 8, device="cuda", generator=g).to(dt)
        la = -la.abs()
        y = ccq_scan(x.expand(B, T, 8), la.expand(B, T, 8))
        small = ccq_scan(x, la)
        assert all(torch.equal(y[b : b + 1], small) for b in (0, 1, B // 2, B - 2, B - 1))
        del y
    T, B = 65, (1 << 22) - 1
    print(f"scan backward T{T} B{B}", flush=True)
    x, la, dy = torch.randn(3, 1, T, 8, device="cuda", generator=g)
    la = -la.abs()
    out, small = ccq_scan_backward(x.expand(B, T, 8), la.expand(B, T, 8), dy.expand(B, T, 8)), ccq_scan_backward(x, la, dy)
    assert all(torch.equal(out[n][b : b + 1], small[n]) for n in ("dx", "dlog_alpha") for b in (0, 1, B // 2, B - 1))
    del out
    torch.cuda.empty_cache()
    N = (1 << 24) - 1
    print(f"select and reorder N{N}", flush=True)
    logits = torch.randn(N, 1, 8, device="cuda", generator=g)
    scores = -torch.rand(N, 1, device="cuda", generator=g)
    out = ccq_beam_select(logits, scores, 2)
    for part in (slice(0, 500), slice(N // 2, N // 2 + 500), slice(N - 500, N)):
        small = ccq_beam_select(logits[part].clone(), scores[part].clone(), 2)
        assert torch.equal(out["token"][part], small["token"]) and torch.equal(out["parent"][part], small["parent"])
        assert ((out["score"][part] - small["score"]).abs() <= 2 * (U * small["score"].abs() + 64 * U)).all()
    N = 1 << 23
    state = torch.randn(2 * N, 1, device="cuda", generator=g)
    want = state.view(N, 2).flip(1).reshape(2 * N, 1)
    ccq_beam_reorder([state], torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").expand(N, 2).contiguous())
    assert torch.equal(state, want)


def test_qk_norm_rope_of_the_most_tokens(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_qk_norm_rope
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    T = (1 << 28) - 16
    print(f"qk T{T}", flush=True)
    q = torch.randn(1, 1, 1, 128, device="cuda").to(torch.bfloat16).expand(1, T, 1, 128)
    freq = torch.linspace(1, 0.1, 64, device="cuda")
    out, _ = ccq_qk_norm_rope(q, None, inv_freq=freq)
    for part in (slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 50, T)):
        assert torch.equal(out[:, :, part], ccq_qk_norm_rope(q[:, part], None, inv_freq=freq, position_offset=part.start)[0])
