"""Refusals of the operators around the read step, in the C ABI and in the binding, and the layout of
their argument structs.  No call here reaches a kernel, so these run without a GPU."""

import ctypes
import os
import shutil
import subprocess

import pytest

from curvature_conditioned_query_amd import binding
from curvature_conditioned_query_amd.binding import (BeamParams, QkBwdParams, QkParams, ScanBwdParams, ScanParams,
                                                      load_library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -5
BASE = 0x7F0000000000  # never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    return load_library()


def _places(names):
    """A fake pointer for every name, a GiB apart."""
    return {n: BASE + (i << 30) for i, n in enumerate(names)}


def _fill(p, values):
    for k, v in values.items():
        obj = p
        while "." in k:
            head, k = k.split(".", 1)
            obj = getattr(obj, head)
        setattr(obj, k, v)
    return p


def _qk(**kw):
    p = QkParams(dtype=1, B=2, T=10, H_q=4, H_k=2, d=64, q_norm=1, k_norm=2, rot=32, eps=1e-6, q_stride_b=2560,
                 q_stride_t=256, q_stride_h=64, k_stride_b=1280, k_stride_t=128, k_stride_h=64)
    _fill(p, _places(["q", "k", "positions", "inv_freq", "q_weight", "k_weight", "q_out", "k_out"]))
    return _fill(p, kw)


QK_BAD = [
    (dict(dtype=3), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H_q=-1), INVALID),
    (dict(H_q=0, H_k=0), INVALID), (dict(q_norm=3), INVALID), (dict(k_norm=-1), INVALID), (dict(interleaved=2), INVALID),
    (dict(expand_keys=1, H_q=3), INVALID), (dict(expand_keys=1, H_k=0, k=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(rot=-16), INVALID), (dict(rot=80), INVALID),
    (dict(rot=8), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(H_q=5000), UNSUPPORTED),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED), (dict(q=None), INVALID), (dict(H_k=0), INVALID), (dict(inv_freq=None), INVALID),
    (dict(rot=0), INVALID), (dict(q_stride_b=-8), INVALID), (dict(q_stride_t=1 << 60), INVALID),
    (dict(q_stride_t=257), MISALIGNED), (dict(k_stride_h=68), MISALIGNED), (dict(q=BASE + 2), MISALIGNED),
    (dict(positions=BASE + 8), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", QK_BAD + [
    (dict(q_out=None), INVALID), (dict(k_out=None), INVALID), (dict(q_out=BASE), INVALID),
    (dict(k_out=BASE + (1 << 30) + 64), INVALID), (dict(k_out=BASE + (6 << 30) + 16), INVALID),
    (dict(q_out=BASE + (4 << 30)), INVALID), (dict(q_out=BASE + (6 << 30) + 4), MISALIGNED)])
def test_qk_refusals(lib, kw, code):
    assert lib.ccq_qk_norm_rope(_qk(**kw), None) == code


def _qkb(**kw):
    p = QkBwdParams(fwd=_qk(q_out=None, k_out=None), dq_stride_b=2560, dq_stride_t=256, dq_stride_h=64, dk_stride_b=1280,
                    dk_stride_t=128, dk_stride_h=64, workspace_bytes=1 << 29)
    names = ["dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "workspace"]
    _fill(p, {n: BASE + ((10 + i) << 30) for i, n in enumerate(names)})
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", [({"fwd." + k: v for k, v in kw.items()}, c) for kw, c in QK_BAD] + [
    (dict(dq=None), INVALID), (dict(dk_out=None), INVALID), (dict(dq_weight=None), INVALID),
    ({"fwd.k_weight": None}, INVALID), (dict(dq_stride_h=32), INVALID), (dict(dq_stride_t=0), INVALID),
    (dict(dk_stride_b=64), INVALID), (dict(dq_stride_b=-8), INVALID), (dict(dk_stride_t=130), MISALIGNED),
    (dict(dq=BASE), INVALID), (dict(dk=BASE + (10 << 30)), INVALID), (dict(dk_weight=BASE + (4 << 30)), INVALID),
    (dict(workspace=BASE + (12 << 30)), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE),
    (dict(workspace=BASE + 8), MISALIGNED)])
def test_qk_backward_refusals(lib, kw, code):
    assert lib.ccq_qk_norm_rope_backward(_qkb(**kw), None) == code


def test_qk_backward_workspace(lib):
    assert lib.ccq_qk_backward_workspace_bytes(_qkb(workspace=None)) > 0
    none = {"fwd.q_weight": None, "fwd.k_weight": None, "dq_weight": None, "dk_weight": None}
    assert lib.ccq_qk_backward_workspace_bytes(_qkb(**none)) == 0
    assert lib.ccq_qk_backward_workspace_bytes(_qkb(dq=None)) == 0
    for fn in (lib.ccq_qk_norm_rope, lib.ccq_qk_norm_rope_backward, lib.ccq_scan, lib.ccq_scan_backward, lib.ccq_beam_select):
        assert fn(None, None) == INVALID
    for fn in (lib.ccq_qk_backward_workspace_bytes, lib.ccq_scan_workspace_bytes, lib.ccq_scan_backward_workspace_bytes,
               lib.ccq_beam_select_workspace_bytes):
        assert fn(None) == 0


def _scan(**kw):
    p = ScanParams(dtype=1, B=2, T=1000, D=64, x_stride_b=64000, x_stride_t=64, la_stride_b=64000, la_stride_t=64,
                   workspace_bytes=1 << 29)
    _fill(p, _places(["x", "log_alpha", "lengths", "h0", "y", "h_out", "chunk_carry", "workspace"]))
    return _fill(p, kw)


SCAN_BAD = [
    (dict(dtype=2), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(D=-8), INVALID), (dict(complement=2), INVALID),
    (dict(D=60), UNSUPPORTED), (dict(D=1 << 25), UNSUPPORTED), (dict(B=1 << 16, T=1 << 16), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(log_alpha=None), INVALID), (dict(x_stride_t=-64), INVALID), (dict(la_stride_b=1 << 60), INVALID),
    (dict(x_stride_t=65), MISALIGNED), (dict(la_stride_t=4), MISALIGNED), (dict(lengths=BASE + 4), MISALIGNED),
    (dict(h0=BASE + (3 << 30) + 4), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(y=None), INVALID), (dict(y=BASE), INVALID), (dict(y=BASE + (1 << 30) + 128), INVALID),
    (dict(h_out=BASE + (3 << 30) + 16), INVALID), (dict(h_out=BASE + (4 << 30)), INVALID),
    (dict(chunk_carry=BASE + (3 << 30)), INVALID), (dict(chunk_carry=BASE + (4 << 30)), INVALID)])
def test_scan_refusals(lib, kw, code):
    assert lib.ccq_scan(_scan(**kw), None) == code


def _scanb(**kw):
    p = ScanBwdParams(dtype=1, B=2, T=1000, D=64, x_stride_b=64000, x_stride_t=64, la_stride_b=64000, la_stride_t=64,
                      dy_stride_b=64000, dy_stride_t=64, workspace_bytes=1 << 29)
    _fill(p, _places(["x", "log_alpha", "lengths", "h0", "dy", "dh_out", "chunk_carry", "dx", "dlog_alpha", "dh0", "workspace"]))
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", SCAN_BAD + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dlog_alpha=None), INVALID), (dict(dy_stride_t=20), MISALIGNED),
    (dict(dx=BASE + (4 << 30)), INVALID), (dict(dlog_alpha=BASE + (7 << 30)), INVALID), (dict(dh0=BASE + (3 << 30)), INVALID),
    (dict(dh0=BASE + (5 << 30) + 16), INVALID), (dict(chunk_carry=None, workspace=None), WORKSPACE),
    (dict(chunk_carry=None, workspace_bytes=64), WORKSPACE)])
def test_scan_backward_refusals(lib, kw, code):
    assert lib.ccq_scan_backward(_scanb(**kw), None) == code


def _beam(**kw):
    p = BeamParams(dtype=1, N=2, K=4, V=1000, M=4, logits_stride=1000, pad_token=0, workspace_bytes=1 << 29)
    _fill(p, _places(["logits", "scores", "finished", "token", "parent", "score", "workspace"]))
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(M=0), INVALID),
    (dict(V=2, K=2, M=5), INVALID), (dict(logits_stride=999), INVALID), (dict(logits_stride=1 << 40), INVALID),
    (dict(pad_token=-1), INVALID), (dict(pad_token=1000), INVALID), (dict(K=65), UNSUPPORTED), (dict(M=65), UNSUPPORTED),
    (dict(K=64, V=1 << 25, logits_stride=1 << 25), UNSUPPORTED), (dict(N=1 << 23), UNSUPPORTED),
    (dict(K=16, V=1 << 23, logits_stride=1 << 23), UNSUPPORTED), (dict(logits=None), INVALID), (dict(scores=None), INVALID),
    (dict(token=None), INVALID), (dict(parent=None), INVALID), (dict(score=None), INVALID), (dict(logits=BASE + 2), MISALIGNED),
    (dict(finished=BASE + 1), MISALIGNED), (dict(token=BASE), INVALID), (dict(parent=BASE + (3 << 30)), INVALID),
    (dict(score=BASE + (1 << 30)), INVALID), (dict(workspace=BASE), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=16), WORKSPACE)])
def test_beam_select_refusals(lib, kw, code):
    assert lib.ccq_beam_select(_beam(**kw), None) == code


@pytest.mark.parametrize("states,rows,N,K,parent,code", [
    ([], [], 2, 4, BASE, INVALID), ([BASE] * 17, [16] * 17, 2, 4, BASE, INVALID), ([None], [16], 2, 4, BASE, INVALID),
    ([BASE], [0], 2, 4, BASE + 4096, INVALID), ([BASE], [6], 2, 4, BASE + 4096, INVALID), ([BASE], [16], 0, 4, BASE, INVALID),
    ([BASE], [16], 2, 0, BASE, INVALID), ([BASE], [16], 2, 4, None, INVALID), ([BASE], [16], 2, 65, BASE + 4096, UNSUPPORTED),
    ([BASE + 4], [16], 2, 4, BASE + 4096, MISALIGNED), ([BASE], [16], 2, 4, BASE + 4098, MISALIGNED),
    ([BASE], [1024], 2, 4, BASE + 4096, INVALID), ([BASE, BASE + 64], [16, 16], 2, 4, BASE + 4096, INVALID)])
def test_beam_reorder_refusals(lib, states, rows, N, K, parent, code):
    n = len(states)
    ptrs = (ctypes.c_void_p * max(1, n))(*states)
    sizes = (ctypes.c_size_t * max(1, n))(*rows)
    assert lib.ccq_beam_reorder(n, ptrs, sizes, N, K, parent, None) == code


def test_beam_reorder_needs_its_arrays(lib):
    one = (ctypes.c_size_t * 1)(16)
    ptr = (ctypes.c_void_p * 1)(BASE)
    assert lib.ccq_beam_reorder(1, None, one, 1, 1, BASE, None) == INVALID
    assert lib.ccq_beam_reorder(1, ptr, None, 1, 1, BASE, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        binding.ccq_scan(x, x)
    with pytest.raises(ValueError):
        binding.ccq_scan_backward(x, x, x)
    with pytest.raises(ValueError):
        binding.ccq_scan(x[0], x[0])
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        binding.ccq_qk_norm_rope(q, q)
    with pytest.raises(ValueError):
        binding.ccq_qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        binding.ccq_beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        binding.ccq_beam_select(torch.zeros(2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        binding.ccq_beam_reorder([], torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.ccq_beam_reorder([torch.zeros(2, 8)], torch.zeros(1, 2, dtype=torch.int32))


def test_param_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (("ccq_qk_params", QkParams), ("ccq_qk_bwd_params", QkBwdParams), ("ccq_scan_params", ScanParams),
               ("ccq_scan_bwd_params", ScanBwdParams), ("ccq_beam_params", BeamParams))
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "ccq.h"', "int main(void) {"]
    for cname, cls in structs:
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out if line}
    for cname, cls in structs:
        assert got[(cname, "size")] == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert got[(cname, f[0])] == getattr(cls, f[0]).offset, (cname, f[0])


# A launch counts its threads in 32 bits: what would pass that is refused, and what is just inside is not (the
# outputs overlap an input there, so no call goes on to a launch).
QK_DENSE = dict(q_stride_b=0, q_stride_t=0, q_stride_h=0, k_stride_b=0, k_stride_t=0, k_stride_h=0)


@pytest.mark.parametrize("d,most", [(128, (1 << 28) - 16), (64, (1 << 29) - 32)])
def test_qk_launch_limit(lib, d, most):
    for B, T in ((1, most), (most // 16, 16), (2, most // 2)):
        assert lib.ccq_qk_norm_rope(_qk(B=B, T=T, d=d, q_out=BASE, **QK_DENSE), None) == INVALID
    assert lib.ccq_qk_norm_rope(_qk(B=1, T=most + 1, d=d, **QK_DENSE), None) == UNSUPPORTED
    assert lib.ccq_qk_norm_rope(_qk(B=4, T=most // 4 + 4, d=d, **QK_DENSE), None) == UNSUPPORTED
    assert lib.ccq_qk_norm_rope_backward(_qkb(**{"fwd.B": 1, "fwd.T": 1 << 30, "fwd.d": d, "dq": BASE}), None) != UNSUPPORTED


SCAN_DENSE = dict(x_stride_b=0, x_stride_t=0, la_stride_b=0, la_stride_t=0)
N23 = 1 << 23


@pytest.mark.parametrize("dtype,T,D,inside,beyond", [
    (1, 65, 8, N23 - 1, N23), (1, 129, 8, N23 // 2 - 1, N23 // 2), (0, 65, 8, N23 - 1, N23), (1, 65, 264, N23 // 3, N23 // 3 + 1),
    (1, 9, 8, 8 * N23 - 8, 8 * N23 - 7), (0, 64, 8, 2 * N23 - 2, 2 * N23 - 1), (1, 33, 8, 2 * N23 - 2, 2 * N23 - 1)])
def test_scan_launch_limit(lib, dtype, T, D, inside, beyond):
    assert lib.ccq_scan(_scan(dtype=dtype, B=inside, T=T, D=D, y=BASE, **SCAN_DENSE), None) == INVALID
    assert lib.ccq_scan(_scan(dtype=dtype, B=beyond, T=T, D=D, y=BASE, **SCAN_DENSE), None) == UNSUPPORTED
    assert lib.ccq_scan_workspace_bytes(_scan(dtype=dtype, B=beyond, T=T, D=D, **SCAN_DENSE)) == 0


@pytest.mark.parametrize("dtype,T,D,inside,beyond", [
    (1, 65, 8, N23 - 1, N23), (1, 129, 8, N23 // 2 - 1, N23 // 2), (0, 65, 8, N23 // 2 - 1, N23 // 2), (0, 64, 8, N23 - 1, N23),
    (1, 64, 8, 2 * N23 - 2, 2 * N23 - 1), (0, 32, 8, 2 * N23 - 2, 2 * N23 - 1)])
def test_scan_backward_launch_limit(lib, dtype, T, D, inside, beyond):
    dense = dict(SCAN_DENSE, dy_stride_b=0, dy_stride_t=0)
    for carry in (BASE, None):
        assert lib.ccq_scan_backward(_scanb(dtype=dtype, B=inside, T=T, D=D, dx=BASE, chunk_carry=carry, **dense), None) == INVALID
        assert lib.ccq_scan_backward(_scanb(dtype=dtype, B=beyond, T=T, D=D, dx=BASE, chunk_carry=carry, **dense), None) == UNSUPPORTED


def test_beam_launch_limits(lib):
    few = dict(V=8, logits_stride=8, token=BASE)
    for N, K in (((1 << 24) - 1, 1), ((1 << 23) - 1, 2), ((1 << 18) - 1, 64)):
        assert lib.ccq_beam_select(_beam(N=N, K=K, **few), None) == INVALID
    for N, K in ((1 << 24, 1), (1 << 23, 2), (1 << 18, 64)):
        assert lib.ccq_beam_select(_beam(N=N, K=K, **few), None) == UNSUPPORTED

    def reorder(rows, N, K):
        n = len(rows)
        return lib.ccq_beam_reorder(n, (ctypes.c_void_p * n)(*[BASE] * n), (ctypes.c_size_t * n)(*rows), N, K, BASE, None)
    assert reorder([(1 << 36) - 4096], 1, 2) == INVALID  # parent inside the state
    assert reorder([1 << 36], 1, 2) == UNSUPPORTED
    assert reorder([(1 << 34) - 1028], 1, 2) == INVALID
    assert reorder([(1 << 34) - 1028, 4], 1, 2) == UNSUPPORTED
    assert reorder([(1 << 34) - 1024], 1, 17) == INVALID
    assert reorder([1 << 34], 1, 17) == UNSUPPORTED
    assert reorder([4], (1 << 24) - 1, 1) == INVALID
    assert reorder([4], 1 << 24, 1) == UNSUPPORTED
    assert reorder([16, 16], 1 << 23, 2) == UNSUPPORTED


def test_qk_backward_gradients_apart(lib):
    """One tensor for both gradients, or rows that overlap, are refused; the parts of a packed gradient are not (the
    workspace is too small here, so nothing is launched)."""
    dq = BASE + (12 << 30)
    packed = dict(dq_stride_b=3840, dq_stride_t=384, dk_stride_b=3840, dk_stride_t=384, workspace_bytes=0)
    for dk in (dq, dq + 16, dq + 112, dq - 112):
        assert lib.ccq_qk_norm_rope_backward(_qkb(dk=dk, **packed), None) == INVALID
    for dk in (dq + 4 * 128, dq - 2 * 128):
        assert lib.ccq_qk_norm_rope_backward(_qkb(dk=dk, **packed), None) == WORKSPACE
