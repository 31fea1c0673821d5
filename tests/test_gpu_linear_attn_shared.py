"""The attention's gradient where heads share queries and keys, in as many heads as a call may have."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,T,share", [(1 << 20, 9, 2), (1 << 18, 64, 4)])
def test_shared_heads_of_the_most_chains(gpu_lib, H, T, share):
    """A head is worked on alike wherever it stands: some heads of a large call give the bits of a small call.  A token's row of
    all heads is 2^29 bytes in fp32 (2^27), so eight tokens (32) lie 2^32 bytes apart."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    heads = lambda n, d: torch.randn(1, n, T, d, device="cuda", generator=g, dtype=torch.float32).bfloat16().transpose(1, 2)  # noqa: E731
    Hq, dk, dv = H // share, 128, 64
    q, k, v, d_o = heads(Hq, dk), heads(Hq, dk), heads(H, dv), heads(H, dv)
    la = -torch.rand(1, T, H, device="cuda", generator=g)
    new = lambda x: torch.empty(1, x.shape[2], T, x.shape[3], dtype=x.dtype, device="cuda").transpose(1, 2)  # noqa: E731
    got = ccq_linear_attn_backward(q, k, v, d_o, la, dq=new(q), dk=new(k), dv=new(v))
    for at in (0, Hq // 2, Hq - 2):
        few, many = slice(at, at + 2), slice(at * share, (at + 2) * share)
        want = ccq_linear_attn_backward(q[:, :, few], k[:, :, few], v[:, :, many], d_o[:, :, many], la[:, :, many].contiguous())
        for m, part in (("dq", few), ("dk", few), ("dv", many), ("dlog_alpha", many)):
            assert torch.equal(got[m][:, :, part], want[m]), (m, at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shares,dk,dv", [((1, 1, 1), 64, 64), ((2, 2, 1), 64, 128), ((1, 4, 2), 128, 64)])
@pytest.mark.parametrize("at,most", [([3, 3, 133, 134, 300], 200), ([3, 3, 133, 134, 300], 70), ([0, 0, 0], 90), ([310, 310], 5),
                                     ([200, 210], 400), ([0, 310], 310)])
def test_packed_rows_of_no_sequence_have_a_gradient_of_zero(gpu_lib, at, most, shares, dk, dv, dtype):
    """Before, between and behind the sequences, and past max_length, whatever the gradients' memory and the inputs held there;
    the sequences' rows have the bits of calls on one sequence each."""
    import torch
    from curvature_conditioned_query_amd import ccq_linear_attn_backward
    rows, H = 310, 4
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(6)
    rn = lambda h, d: torch.randn(1, rows, h, d, generator=g).to(dt).cuda()  # noqa: E731
    x = dict(q=rn(H // shares[0], dk), k=rn(H // shares[1], dk), v=rn(H // shares[2], dv), d_o=rn(H, dv),
             log_alpha=-torch.rand(1, rows, H, generator=g).to(dt).cuda())
    spans = [(a, min(b - a, most)) for a, b in zip(at, at[1:])]
    idle = torch.ones(rows, dtype=torch.bool)
    for a, n in spans:
        idle[a:a + n] = False
    for t in x.values():
        t[:, idle] = float("nan")
    grads = {"d" + m: torch.full_like(x[m], float("nan")) for m in "qkv"}
    junk = torch.full_like(x["log_alpha"], float("nan"))
    del junk  # memory that the decays' gradient is likely to get
    got = ccq_linear_attn_backward(**x, **grads, offsets=torch.tensor(at, dtype=torch.int32, device="cuda"), max_length=most)
    assert all(got[m] is grads[m] for m in grads)
    for m in got:
        assert (got[m][:, idle] == 0).all(), m
    for a, n in spans:
        if n:
            one = ccq_linear_attn_backward(**{m: t[:, a:a + n].contiguous() for m, t in x.items()})
            assert all(torch.equal(got[m][:, a:a + n], one[m]) for m in one)
