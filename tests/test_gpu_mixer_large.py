"""Linear attention, group norm and adjusted logits on tensors of more than 2^32 elements, and in their largest launches.

A sequence, row or token is worked on alike wherever it stands, so the parts of a large call are compared with a small
call on the same values: equal bits.
"""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory(gpu_lib):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def _views(shape, strides, count):
    """Tensors of a shape side by side in one buffer of 2^33 bf16 elements."""
    import torch
    buf = torch.empty(1 << 33, dtype=torch.bfloat16, device="cuda")
    row = shape[2] * shape[3]
    reach = sum((n - 1) * s for n, s in zip(shape[:2], strides[:2])) + count * row
    assert 1 << 32 < reach <= 1 << 33
    return [buf.as_strided(shape, strides, i * row) for i in range(count)]


@pytest.mark.parametrize("B,T,far", [(2, 5, "batch"), (2, 200, "batch"), (1, 530, "token")])
def test_attention_and_gradient_of_far_rows(gpu_lib, B, T, far):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    H, d = 2, 64
    strides = ((1 << 32) + 2048, 1024, d, 1) if far == "batch" else (0, (1 << 23) + 1024, d, 1)
    q, k, v, d_o = _views((B, T, H, d), strides, 4)
    o, dq, dk, dv = _views((B, T, H, d), strides, 4)
    g = torch.Generator().manual_seed(1)
    near = [torch.randn(B, T, H, d, generator=g).bfloat16().cuda() for _ in range(4)]
    for dst, src in zip((q, k, v, d_o), near):
        dst.copy_(src)
    la = -torch.rand(B, T, H, generator=g).cuda()
    S, S2 = torch.empty(B, H, d, d, device="cuda"), torch.empty(B, H, d, d, device="cuda")
    ccq_linear_attn(q, k, v, la, o=o, S_out=S)
    assert torch.equal(o, ccq_linear_attn(*near[:3], la, S_out=S2)) and torch.equal(S, S2)
    got = ccq_linear_attn_backward(q, k, v, d_o, la, dq=dq, dk=dk, dv=dv)
    want = ccq_linear_attn_backward(*near, la)
    assert all(torch.equal(got[m], want[m]) for m in want)


def test_attention_of_the_last_of_many_packed_rows(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn
    rows, n, H, d = 1 << 23, 201, 2, 64
    q, k, v = _views((1, rows, H, d), (0, 1000, d, 1), 3)
    o, = _views((1, rows, H, d), (0, 1000, d, 1), 1)
    g = torch.Generator().manual_seed(2)
    near = [torch.randn(1, n, H, d, generator=g).bfloat16().cuda() for _ in range(3)]
    for dst, src in zip((q, k, v), near):
        dst[:, rows - n:] = src
    la = torch.full((1, rows, H), -0.1, device="cuda")
    o[:, rows - n - 5:] = 2.0
    at = torch.tensor([rows - n, rows], dtype=torch.int32, device="cuda")
    ccq_linear_attn(q, k, v, la, o=o, offsets=at, max_length=n)
    assert torch.equal(o[:, rows - n:], ccq_linear_attn(*near, la[:, :n])) and (o[:, rows - n - 5:rows - n] == 2.0).all()


@pytest.mark.parametrize("T", [1, 9])
def test_attention_of_the_most_chains(gpu_lib, T):
    """2^20 of them, whose states are 2^32 numbers; the gradient's launch has 6 workgroups for each."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn, ccq_linear_attn_backward
    B, H, d = 1 << 14, 64, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(B, T, 1, d, device="cuda", generator=g).bfloat16().expand(B, T, H, d) for _ in range(3))
    la = -torch.rand(1, 1, H, device="cuda", generator=g).expand(B, T, H)
    S = torch.empty(B, H, d, d, device="cuda")
    o = ccq_linear_attn(q, k, v, la, S_out=S)
    for part in (slice(0, 2), slice(B // 2, B // 2 + 2), slice(B - 2, B)):
        S2 = torch.empty(2, H, d, d, device="cuda")
        assert torch.equal(o[part], ccq_linear_attn(q[part], k[part], v[part], la[part], S_out=S2))
        assert torch.equal(S[part], S2)
    got = ccq_linear_attn_backward(q, k, v, o, la, grad_dtype=torch.float32)
    for part in (slice(0, 2), slice(B // 2, B // 2 + 2), slice(B - 2, B)):
        small = ccq_linear_attn_backward(q[part], k[part], v[part], o[part], la[part], grad_dtype=torch.float32)
        assert all(torch.equal(got[m][part], small[m]) for m in small)


def test_group_norm_of_the_most_rows(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_group_norm, ccq_group_norm_backward
    T, G, d = (1 << 28) - 1, 8, 8
    buf = torch.randn(1 << 20, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    x = torch.empty(1, T, G, d, dtype=torch.bfloat16, device="cuda")
    x[:, :1000] = buf[:1000 * G * d].view(1, 1000, G, d)
    x[:, T - 1000:] = buf[-1000 * G * d:].view(1, 1000, G, d)
    y = ccq_group_norm(x, activation="silu")
    for part in (slice(0, 1000), slice(T - 1000, T)):
        assert torch.equal(y[:, part], ccq_group_norm(x[:, part], activation="silu"))
    del y
    dx = ccq_group_norm_backward(x, x, activation="silu")["dx"]
    for part in (slice(0, 1000), slice(T - 1000, T)):
        assert torch.equal(dx[:, part], ccq_group_norm_backward(x[:, part], x[:, part], activation="silu")["dx"])


def test_logits_of_far_and_of_the_most_rows(gpu_lib):
    import torch
    from curvature_conditioned_query_amd import ccq_logits_adjust
    g = torch.Generator().manual_seed(5)
    R, V = 8, 20001
    wide = torch.empty(1 << 33, dtype=torch.bfloat16, device="cuda")[: R << 30].view(R, 1 << 30)[:, 8:8 + V]
    near = torch.randn(R, V, generator=g).bfloat16().cuda()
    wide.copy_(near)
    how = dict(history=torch.randint(0, V, (R, 500), generator=g).int().cuda(), repetition=1.5, frequency=0.2,
               bias_token=torch.randint(0, V, (R, 3), generator=g).int().cuda(), bias_value=torch.randn(R, 3, generator=g).cuda())
    assert torch.equal(ccq_logits_adjust(wide, out=wide, **how), ccq_logits_adjust(near, **how))
    del wide
    R, V = (1 << 24) - 1, 64
    rows = torch.randn(R, V, device="cuda").bfloat16()
    history = torch.arange(R, device="cuda", dtype=torch.int32)[:, None] % V
    out = ccq_logits_adjust(rows, history=history, presence=1.0)
    for part in (slice(0, 9), slice((1 << 22) - 9, (1 << 22) + 9), slice(R - 9, R)):
        assert torch.equal(out[part], ccq_logits_adjust(rows[part], history=history[part], presence=1.0))
        assert (out[part] != rows[part]).sum() == out[part].shape[0]
