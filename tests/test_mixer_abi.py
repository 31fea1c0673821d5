"""Refusals of the operators of a linear-attention layer, in the C ABI and in the binding, and the layout of their
argument structs.  No call here reaches a kernel, so these run without a GPU."""

import ctypes
import os
import shutil
import subprocess

import pytest

from curvature_conditioned_query_amd import binding
from curvature_conditioned_query_amd.binding import (GroupNormBwdParams, GroupNormParams, LinearAttnBwdParams,
                                                      LinearAttnParams, LogitsAdjustParams, load_library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -5
BASE = 0x7F0000000000  # never dereferenced: every call below fails validation
GIB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return load_library()


def _fill(p, values):
    for k, v in values.items():
        obj = p
        while "." in k:
            head, k = k.split(".", 1)
            obj = getattr(obj, head)
        setattr(obj, k, v)
    return p


def _places(names, first=0):
    """A fake pointer for every name, a GiB apart."""
    return {n: BASE + (first + i) * GIB for i, n in enumerate(names)}


def _strides(name, T, heads, d):
    return {f"{name}_stride_b": T * heads * d, f"{name}_stride_t": heads * d, f"{name}_stride_h": d}


LA = ["q", "k", "v", "log_alpha", "lengths", "S0", "o", "S_out", "workspace"]


def _la(**kw):
    p = LinearAttnParams(dtype=1, gate_dtype=1, B=2, T=1000, H=4, H_q=2, H_k=1, H_v=4, d_k=64, d_v=128, scale=0.5,
                         workspace_bytes=GIB // 2)
    _fill(p, _places(LA))
    for name, heads, d in (("q", 2, 64), ("k", 1, 64), ("v", 4, 128), ("o", 4, 128)):
        _fill(p, _strides(name, 1000, heads, d))
    _fill(p, dict(la_stride_b=4000, la_stride_t=4, la_stride_h=1))
    return _fill(p, kw)


at = lambda name: BASE + LA.index(name) * GIB  # noqa: E731

LA_BAD = [
    (dict(dtype=2), INVALID), (dict(gate_dtype=-1), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID),
    (dict(H_q=3), INVALID), (dict(H_k=0), INVALID), (dict(H_v=8), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(d_k=0), INVALID), (dict(d_k=96), UNSUPPORTED), (dict(d_v=256), UNSUPPORTED),
    (dict(B=1 << 19), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(rows=5), INVALID), (dict(offsets=BASE + 40 * GIB, rows=2000), INVALID),
    (dict(lengths=None, offsets=BASE + 40 * GIB), INVALID), (dict(lengths=None, offsets=BASE + 40 * GIB, rows=1 << 31), UNSUPPORTED),
    (dict(lengths=None, offsets=BASE + 40 * GIB, rows=-1), INVALID),
    (dict(q_stride_t=-8), INVALID), (dict(q_stride_t=1 << 24), UNSUPPORTED), (dict(k_stride_b=1 << 60), INVALID), (dict(v_stride_h=130), MISALIGNED),
    (dict(q_stride_t=132), MISALIGNED), (dict(la_stride_t=-1), INVALID), (dict(q=BASE + 2), MISALIGNED),
    (dict(gate_dtype=0, log_alpha=at("log_alpha") + 2), MISALIGNED), (dict(lengths=at("lengths") + 4), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", LA_BAD + [
    (dict(o=None), INVALID), (dict(o_stride_t=1 << 24, o_stride_b=1 << 36), UNSUPPORTED), (dict(o_stride_t=256), INVALID), (dict(o_stride_h=0), INVALID), (dict(o_stride_t=516), MISALIGNED),
    (dict(o=BASE), INVALID), (dict(o=at("v") + 256), INVALID), (dict(S_out=at("S0") + 16), INVALID), (dict(S_out=at("k")), INVALID),
    (dict(workspace=at("o")), INVALID), (dict(o=at("log_alpha")), INVALID), (dict(o=at("S0")), INVALID), (dict(o=at("lengths")), INVALID),
    (dict(S_out=at("S_out") + 4), MISALIGNED), (dict(T=30000, o=at("S0")), INVALID)])
def test_linear_attn_refusals(lib, kw, code):
    assert lib.ccq_linear_attn(_la(**kw), None) == code


def test_linear_attn_workspace(lib):
    """One sequence of few heads is cut along its tokens, which takes a workspace; many chains are not."""
    long = dict(B=1, T=20480, H=4, **_strides("q", 20480, 2, 64), **_strides("k", 20480, 1, 64), **_strides("v", 20480, 4, 128),
                **_strides("o", 20480, 4, 128))
    need = lib.ccq_linear_attn_workspace_bytes(_la(workspace=None, **long))
    assert need > 0
    assert lib.ccq_linear_attn(_la(workspace=None, **long), None) == WORKSPACE
    assert lib.ccq_linear_attn(_la(workspace_bytes=need - 1, **long), None) == WORKSPACE
    assert lib.ccq_linear_attn_workspace_bytes(_la(B=2048, T=200, workspace=None)) == 0
    assert lib.ccq_linear_attn_workspace_bytes(_la(T=1, workspace=None)) == 0
    assert lib.ccq_linear_attn_workspace_bytes(_la(d_k=96)) == 0
    for fn in (lib.ccq_linear_attn, lib.ccq_linear_attn_backward, lib.ccq_group_norm, lib.ccq_group_norm_backward,
               lib.ccq_logits_adjust):
        assert fn(None, None) == INVALID
    for fn in (lib.ccq_linear_attn_workspace_bytes, lib.ccq_linear_attn_backward_workspace_bytes,
               lib.ccq_group_norm_backward_workspace_bytes):
        assert fn(None) == 0


LAB = ["d_o", "dS_out", "dq", "dk", "dv", "dlog_alpha", "dS0", "workspace"]
bat = lambda name: BASE + (20 + LAB.index(name)) * GIB  # noqa: E731


def _lab(**kw):
    p = LinearAttnBwdParams(fwd=_la(o=None, S_out=None, workspace=None, workspace_bytes=0), grad_dtype=1, workspace_bytes=GIB // 2)
    _fill(p, _places(LAB, 20))
    for name, heads, d in (("dq", 2, 64), ("dk", 1, 64), ("dv", 4, 128), ("do", 4, 128)):
        _fill(p, _strides(name, 1000, heads, d))
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", [({"fwd." + k: v for k, v in kw.items()}, c) for kw, c in LA_BAD] + [
    (dict(grad_dtype=2), INVALID), ({"fwd.dtype": 0, "grad_dtype": 1}, INVALID), (dict(d_o=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dv=None), INVALID), ({"fwd.log_alpha": None}, INVALID), (dict(do_stride_t=-8), INVALID),
    (dict(do_stride_h=60), MISALIGNED), (dict(dq_stride_t=64), INVALID), (dict(dq_stride_t=1 << 24, dq_stride_b=1 << 36), UNSUPPORTED),
    (dict(dk_stride_t=0), INVALID), (dict(dv_stride_h=4), MISALIGNED),
    (dict(dq=bat("dk")), INVALID), (dict(dq=bat("dv") + 16), INVALID), (dict(dq=bat("d_o")), INVALID), (dict(dv=at("q")), INVALID),
    (dict(dS0=bat("dS_out")), INVALID), (dict(dS0=at("S0")), INVALID), (dict(dlog_alpha=at("log_alpha")), INVALID),
    (dict(dlog_alpha=bat("dq") + 64), INVALID), (dict(workspace=bat("dq")), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=64), WORKSPACE), (dict(dk=bat("dk") + 8), MISALIGNED), (dict(workspace=bat("workspace") + 8), MISALIGNED)])
def test_linear_attn_backward_refusals(lib, kw, code):
    assert lib.ccq_linear_attn_backward(_lab(**kw), None) == code


def test_linear_attn_backward_packed_gradient(lib):
    """dq, dk and dv as parts of one packed gradient are taken (the workspace is too small here)."""
    width = 2 * 64 + 64 + 4 * 128
    packed = {f"{m}_stride_{a}": s for m, d in (("dq", 64), ("dk", 64), ("dv", 128)) for a, s in (("b", 1000 * width), ("t", width), ("h", d))}
    dq = bat("dq")
    assert lib.ccq_linear_attn_backward(_lab(dq=dq, dk=dq + 2 * 128, dv=dq + 2 * 192, workspace_bytes=0, **packed), None) == WORKSPACE


NORM = ["x", "gate", "weight", "bias", "y"]


def _norm(**kw):
    p = GroupNormParams(dtype=1, B=2, T=100, G=4, d=80, center=1, activation=1, eps=1e-6)
    _fill(p, _places(NORM))
    for name in ("x", "gate", "y"):
        _fill(p, _strides(name, 100, 4, 80))
    return _fill(p, kw)


NORM_BAD = [
    (dict(dtype=5), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(G=0), INVALID), (dict(d=0), INVALID),
    (dict(center=2), INVALID), (dict(affine_shared=-1), INVALID), (dict(activation=3), INVALID), (dict(activation=-1), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(d=84), UNSUPPORTED),
    (dict(d=1032), UNSUPPORTED), (dict(G=1 << 16), UNSUPPORTED), (dict(B=1 << 15, T=1 << 15), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(x_stride_t=-8), INVALID), (dict(gate_stride_b=1 << 60), INVALID), (dict(x_stride_h=84), MISALIGNED),
    (dict(gate_stride_t=325), MISALIGNED), (dict(x=BASE + 8), MISALIGNED), (dict(weight=BASE + 2 * GIB + 4), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", NORM_BAD + [
    (dict(y=None), INVALID), (dict(y_stride_t=80), INVALID), (dict(y_stride_h=0), INVALID), (dict(y_stride_h=82), MISALIGNED),
    (dict(y=BASE + 160), INVALID), (dict(y=BASE, x_stride_h=8000, x_stride_t=80), INVALID), (dict(y=BASE + 2 * GIB), INVALID),
    (dict(y=BASE + GIB + 16), INVALID), (dict(y=BASE + 4 * GIB + 2), MISALIGNED)])
def test_group_norm_refusals(lib, kw, code):
    assert lib.ccq_group_norm(_norm(**kw), None) == code


NB = ["dy", "dx", "dgate", "dweight", "dbias", "workspace"]
nat = lambda name: BASE + (10 + NB.index(name)) * GIB  # noqa: E731


def _normb(**kw):
    p = GroupNormBwdParams(fwd=_norm(y=None), workspace_bytes=GIB // 2)
    _fill(p, _places(NB, 10))
    for name in ("dy", "dx", "dgate"):
        _fill(p, _strides(name, 100, 4, 80))
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", [({"fwd." + k: v for k, v in kw.items()}, c) for kw, c in NORM_BAD] + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dgate=None), INVALID), ({"fwd.gate": None}, INVALID),
    (dict(dweight=None), INVALID), ({"fwd.bias": None}, INVALID), (dict(dy_stride_t=-8), INVALID), (dict(dx_stride_t=160), INVALID),
    (dict(dgate_stride_h=12), MISALIGNED), (dict(dx=BASE), INVALID), (dict(dx=nat("dy") + 160), INVALID),
    (dict(dx=nat("dy"), dy_stride_t=0), INVALID), (dict(dgate=nat("dx")), INVALID), (dict(dweight=nat("dbias")), INVALID),
    (dict(workspace=nat("dy")), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE)])
def test_group_norm_backward_refusals(lib, kw, code):
    assert lib.ccq_group_norm_backward(_normb(**kw), None) == code


def test_group_norm_backward_workspace(lib):
    need = lib.ccq_group_norm_backward_workspace_bytes(_normb(workspace=None))
    none = {"fwd.weight": None, "dweight": None}
    assert need > 0 and lib.ccq_group_norm_backward_workspace_bytes(_normb(**none)) == need // 2
    assert lib.ccq_group_norm_backward_workspace_bytes(_normb(**none, **{"fwd.bias": None, "dbias": None})) == 0


ADJ = ["logits", "history", "lengths", "prompt_lengths", "repetition_rows", "presence_rows", "frequency_rows", "bias_token",
       "bias_value", "allowed", "out"]
aat = lambda name: BASE + ADJ.index(name) * GIB  # noqa: E731


def _adj(**kw):
    p = LogitsAdjustParams(dtype=1, R=8, V=1001, L=20, n_bias=4, logits_stride=1001, repetition=1.0, out_stride=1001)
    _fill(p, _places(ADJ))
    return _fill(p, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INVALID), (dict(R=0), INVALID), (dict(V=0), INVALID), (dict(L=-1), INVALID), (dict(n_bias=-1), INVALID),
    (dict(logits_stride=1000), INVALID), (dict(out_stride=1000), INVALID), (dict(logits_stride=1 << 40), INVALID),
    (dict(L=0), INVALID), (dict(history=None), INVALID), (dict(L=0, history=None), INVALID), (dict(n_bias=0), INVALID),
    (dict(bias_token=None), INVALID), (dict(bias_value=None), INVALID), (dict(repetition=0.0), INVALID),
    (dict(repetition=-1.0), INVALID), (dict(repetition=float("nan")), INVALID), (dict(repetition=float("inf")), INVALID),
    (dict(presence=float("inf")), INVALID), (dict(frequency=float("nan")), INVALID), (dict(n_bias=1025), UNSUPPORTED),
    (dict(V=(1 << 24) + 1, logits_stride=1 << 25, out_stride=1 << 25), UNSUPPORTED), (dict(L=(1 << 24) + 1), UNSUPPORTED),
    (dict(R=1 << 24), UNSUPPORTED), (dict(R=1 << 12, V=1 << 24, logits_stride=1 << 24, out_stride=1 << 24), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(out=None), INVALID), (dict(logits=BASE + 1), MISALIGNED),
    (dict(dtype=0, logits=BASE + 2), MISALIGNED), (dict(history=aat("history") + 2), MISALIGNED), (dict(out=aat("out") + 1), MISALIGNED), (dict(out=BASE, out_stride=1002), INVALID),
    (dict(out=BASE + 16), INVALID), (dict(out=aat("allowed")), INVALID), (dict(out=aat("lengths")), INVALID)])
def test_logits_adjust_refusals(lib, kw, code):
    assert lib.ccq_logits_adjust(_adj(**kw), None) == code


def test_logits_adjust_launch_limit(lib):
    few = dict(L=0, history=None, lengths=None, prompt_lengths=None, out=aat("allowed"))
    assert lib.ccq_logits_adjust(_adj(R=(1 << 24) - 1, **few), None) == INVALID  # out overlaps: no launch
    assert lib.ccq_logits_adjust(_adj(R=1 << 24, **few), None) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        binding.ccq_linear_attn(q, q, q)
    with pytest.raises(ValueError):
        binding.ccq_linear_attn_backward(q, q, q, q)
    with pytest.raises(ValueError):
        binding.ccq_group_norm(q)
    with pytest.raises(ValueError):
        binding.ccq_group_norm_backward(q, q)
    with pytest.raises(ValueError):
        binding.ccq_logits_adjust(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        binding.ccq_logits_adjust(torch.zeros(8))


def test_param_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (("ccq_linear_attn_params", LinearAttnParams), ("ccq_linear_attn_bwd_params", LinearAttnBwdParams),
               ("ccq_group_norm_params", GroupNormParams), ("ccq_group_norm_bwd_params", GroupNormBwdParams),
               ("ccq_logits_adjust_params", LogitsAdjustParams))
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
