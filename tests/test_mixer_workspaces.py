"""Workspaces of linear attention: what the binding asks for, and in how many segments a sequence is cut.  No call here
reaches a kernel."""

import pytest

from curvature_conditioned_query_amd import binding
from test_mixer_abi import _la, _strides


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


class _Recorder:
    """What the binding looks up, with a library that wants 96 bytes for every call and notes what it is given."""

    def __init__(self):
        import torch
        self.torch, self.empty, self.empty_strided = torch, torch.empty, torch.empty_strided
        self.f32, self.i32, self.u8 = torch.float32, torch.int32, torch.uint8
        self.nowhere, self.asked, self.given = binding._NoContext(), 0, None

    def dtype_code(self, t):
        return {self.f32: 0, self.torch.bfloat16: 1}[t.dtype]

    def place(self, dev, stream):
        return self.nowhere

    def raw_stream(self, index):
        return 0

    def linear_attn_workspace_bytes(self, p):
        self.asked += 1
        return 96

    def linear_attn(self, p, stream):
        self.given = (p.workspace is not None, p.workspace_bytes)
        return 0


@pytest.mark.parametrize("T", [1, 2, 8, 9, 65])
def test_a_call_gets_the_workspace_that_the_library_asks_for(monkeypatch, T):
    """Only a single token is told in advance to need none: by the header, whatever T a kernel for few tokens takes."""
    import torch
    ops = _Recorder()
    monkeypatch.setattr(binding, "_ops", lambda: ops)
    x = torch.zeros(1, T, 2, 64)
    binding.ccq_linear_attn(x, x, x)
    assert (ops.asked, ops.given) == ((0, (False, 0)) if T == 1 else (1, (True, 96)))


def test_single_tokens_need_none(lib):
    for B in (1, 1000, 1 << 17):
        assert lib.ccq_linear_attn_workspace_bytes(_la(B=B, T=1, workspace=None)) == 0


@pytest.mark.parametrize("B,T,H,dk,dv,segments", [(4, 4096, 16, 128, 128, 1), (1, 20480, 16, 128, 128, 8), (7, 777, 6, 64, 128, 1),
                                                  (1, 4096, 16, 128, 128, 8), (1, 64, 1, 64, 64, 1)])
def test_segments(lib, B, T, H, dk, dv, segments):
    """By the workspace: a segment's states, and its log decays in 64 bits, each part in whole 256 bytes."""
    p = _la(B=B, T=T, H=H, H_q=H, H_k=H, H_v=H, d_k=dk, d_v=dv, workspace=None, lengths=None, S0=None, S_out=None, log_alpha=None,
            k=0x7E0000000000, v=0x7D0000000000, o=0x7C0000000000, **_strides("q", T, H, dk), **_strides("k", T, H, dk), **_strides("v", T, H, dv),
            **_strides("o", T, H, dv))
    whole = lambda n: (n + 255) // 256 * 256  # noqa: E731
    want = 0 if segments == 1 else whole(B * H * segments * dk * dv * 4) + whole(B * H * segments * 8)
    assert lib.ccq_linear_attn_workspace_bytes(p) == want
