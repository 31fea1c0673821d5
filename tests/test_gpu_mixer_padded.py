"""Padded and packed batches through linear attention, group norm and both gradients, all tensors allocated by the calls."""

import numpy as np
import pytest

from oracle import mixer
from test_gpu_linear_attn import _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T", [6, 150])
def test_weights_take_nothing_from_rows_of_no_token(gpu_lib, T, packed):
    import torch
    import curvature_conditioned_query_amd as ccq
    B, H, d = 3, 2, 64
    n = [T, 0, T // 2]
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x = dict(q=rn(B, T, H, d), k=rn(B, T, H, d) / 8, v=rn(B, T, H, d), log_alpha=-rn(B, T, H).abs())
    gate, dy, weight, bias = rn(B, T, H, d), rn(B, T, H, d), 1 + 0.1 * rn(H, d), 0.1 * rn(H, d)
    live = torch.arange(T)[None] < torch.tensor(n)[:, None]
    how = dict(lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    if packed:  # rows behind the last sequence fill the batch up
        put = lambda t: torch.cat([t[live], t[:1, :7].reshape(-1, *t.shape[2:])])[None].contiguous()  # noqa: E731
        x, gate, dy = {m: put(t) for m, t in x.items()}, put(gate), put(dy)
        keep = torch.arange(gate.shape[1])[None] < sum(n)
        how = dict(offsets=torch.tensor([0] + n, device="cuda").cumsum(0).int(), max_length=T)
    else:
        keep = live
    dy[~keep] = 0.0
    norm = dict(weight=weight, bias=bias, gate=gate, center=True, activation="silu")
    for _ in range(3):  # memory that new tensors are likely to get
        junk = [torch.full_like(dy, float("nan")) for _ in range(6)]
        del junk
        o = ccq.ccq_linear_attn(**x, **how)
        assert (o[~keep] == 0).all()
        b = ccq.ccq_group_norm_backward(o, dy, **norm)
        a = ccq.ccq_linear_attn_backward(**x, d_o=b["dx"], **how)
        assert all(t.isfinite().all() for t in (*a.values(), b["dweight"], b["dbias"], ccq.ccq_group_norm(o, **norm)))
    live_rows = lambda t: _np(t)[keep.numpy()][None]  # noqa: E731
    _, _, dw, db = mixer.group_norm_backward(live_rows(o), live_rows(dy), _np(weight), _np(bias), live_rows(gate), True, 1e-6, "silu")
    for got, want in ((b["dweight"], dw), (b["dbias"], db)):
        # some hundred terms of a few units each, formed and summed in fp32
        assert np.abs(_np(got) - want).max() <= 1e-5 * np.abs(want).max() + 1e-4
