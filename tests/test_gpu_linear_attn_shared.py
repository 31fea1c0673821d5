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
