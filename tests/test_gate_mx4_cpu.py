"""Host-side refusals of the gate and MX4 calls: checked before any HIP call, so no GPU is needed."""
import ctypes
import os
import subprocess

import pytest

import mixture_experts_layer_35_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20     # an aligned non-null address; rejected calls never dereference it
BAD, UNSUP, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from mixture_experts_layer_35_amd import build
        build.build()
    return moe.lib()


def rule(**kw):
    r = moe.make_gate_rule(16, 64, 6, n_groups=8, topk_groups=4)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def gate(lib, r, logits=FAKE, ld=64, bias=FAKE, scores=None, idx=FAKE, w=FAKE):
    return lib.moe_gate(None if r is None else ctypes.byref(r), logits, ld, bias, scores, idx, w, None)


def backward(lib, r, logits=FAKE, ld=64, idx=FAKE, w=FAKE, dw=FAKE, ds=None, dz=FAKE, dld=64):
    return lib.moe_gate_backward(None if r is None else ctypes.byref(r), logits, ld, idx, w, dw, ds, dz, dld, None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(n_experts=0), BAD), (dict(topk=0), BAD), (dict(n_groups=0), BAD), (dict(topk_groups=0), BAD),
    (dict(score=2), BAD), (dict(flags=4), BAD), (dict(logits_dtype=moe.MOE_E4M3), UNSUP), (dict(n_experts=1032), UNSUP),
    (dict(n_experts=60), UNSUP), (dict(topk_groups=9), UNSUP), (dict(n_groups=128, n_experts=128), UNSUP),
    (dict(topk=33), UNSUP), (dict(topk_groups=1, topk=9), UNSUP), (dict(T=1 << 29, topk=4), UNSUP),
])
def test_gate_rule_rejections(lib, change, want):
    r = rule(**change)
    big = max(r.n_experts, 64)
    assert gate(lib, r, ld=big) == want
    assert "moe_gate:" in moe.moe_last_error()
    assert backward(lib, r, ld=big, dld=big) == want
    assert "moe_gate_backward:" in moe.moe_last_error()


def test_gate_argument_rejections(lib):
    r = rule()
    assert gate(lib, None) == BAD and backward(lib, None) == BAD
    assert gate(lib, r, ld=63) == BAD and backward(lib, r, ld=63) == BAD and backward(lib, r, dld=63) == BAD
    for name in ("logits", "idx", "w"):
        assert gate(lib, r, **{name: None}) == BAD
        assert "must not be NULL" in moe.moe_last_error()
    for name in ("logits", "idx", "w", "dw", "dz"):
        assert backward(lib, r, **{name: None}) == BAD
    assert gate(lib, r, logits=FAKE + 2) == BAD and backward(lib, r, dz=FAKE + 1) == BAD
    assert gate(lib, rule(T=0), logits=None, idx=None, w=None) == OK
    assert backward(lib, rule(T=0), logits=None, idx=None, w=None, dw=None, dz=None) == OK
    with pytest.raises(ValueError):
        moe.make_gate_rule(1, 8, 2, score="relu")


def test_mx4_rejections(lib):
    q, dq = lib.moe_quantize_mx4, lib.moe_dequantize_mx4
    assert q(-1, 128, moe.MOE_BF16, FAKE, 128, FAKE, FAKE, None) == BAD
    assert q(1, 0, moe.MOE_BF16, FAKE, 128, FAKE, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE, 127, FAKE, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_E4M3, FAKE, 128, FAKE, FAKE, None) == UNSUP
    assert q(1, 128, moe.MOE_BF16, None, 128, FAKE, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE, 128, None, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE, 128, FAKE, None, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE + 1, 128, FAKE, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE, 128, FAKE + 8, FAKE, None) == BAD
    assert q(1, 128, moe.MOE_BF16, FAKE, 128, FAKE, FAKE + 2, None) == BAD
    assert q(0, 128, moe.MOE_BF16, None, 128, None, None, None) == OK
    assert dq(-1, 128, FAKE, FAKE, moe.MOE_BF16, FAKE, 128, None) == BAD
    assert dq(1, 128, FAKE, FAKE, moe.MOE_E4M3, FAKE, 128, None) == UNSUP
    assert dq(1, 128, FAKE, FAKE, moe.MOE_F32, FAKE, 100, None) == BAD
    assert dq(1, 128, FAKE, FAKE, moe.MOE_F32, FAKE + 2, 128, None) == BAD
    assert dq(1, 128, FAKE, FAKE, moe.MOE_F32, None, 128, None) == BAD
    assert dq(0, 128, None, None, moe.MOE_F32, None, 128, None) == OK


def test_experts_rejections(lib):
    def ffn(n=4, off=FAKE, rows=32, gather=None, d=256, inter=128, x=FAKE, xs=FAKE, w=(FAKE,) * 3, ws=(FAKE,) * 3,
            y=FAKE, scratch=FAKE, size=None):
        arr = [None if v is None else ctypes.cast((ctypes.c_void_p * 3)(*v), ctypes.c_void_p) for v in (w, ws)]
        need = lib.moe_ffn_mx4_workspace_bytes(max(rows, 0), max(inter, 1))
        return lib.moe_grouped_ffn_mx4(n, off, rows, gather, d, inter, x, xs, *arr, y, scratch,
                                       need if size is None else size, None)

    assert ffn(n=0) == BAD and ffn(rows=-1) == BAD and ffn(d=0) == BAD and ffn(inter=0) == BAD
    assert ffn(n=1025) == UNSUP and ffn(d=(1 << 20) + 1) == UNSUP and ffn(rows=1 << 31) == UNSUP
    assert ffn(rows=1 << 30, d=1 << 20) == UNSUP                    # more tiles than 32 bits count
    assert ffn(off=None) == BAD and ffn(x=None) == BAD and ffn(xs=None) == BAD and ffn(y=None) == BAD
    assert ffn(w=None) == BAD and ffn(ws=None) == BAD
    assert ffn(w=(FAKE, None, FAKE)) == BAD and ffn(ws=(FAKE, FAKE, None)) == BAD
    assert ffn(x=FAKE + 8) == BAD and ffn(xs=FAKE + 1) == BAD and ffn(w=(FAKE, FAKE, FAKE + 4)) == BAD
    assert ffn(y=FAKE + 1) == BAD
    need = lib.moe_ffn_mx4_workspace_bytes(32, 128)
    assert 32 * 68 <= need < 32 * 68 + 1024
    assert ffn(size=need - 1) == WS and ffn(scratch=None) == WS and ffn(scratch=FAKE + 16) == BAD
    assert ffn(rows=0, off=None, x=None, xs=None, w=None, ws=None, y=None, scratch=None) == OK
    assert lib.moe_ffn_mx4_workspace_bytes(-1, 128) == 0 and lib.moe_ffn_mx4_workspace_bytes(8, 0) == 0


def test_gate_rule_layout_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(moe_gate_rule), offsetof(moe_gate_rule, topk),'
                   ' offsetof(moe_gate_rule, logits_dtype), offsetof(moe_gate_rule, routed_scale),'
                   ' offsetof(moe_gate_rule, flags)); return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    R = moe.MoeGateRule
    assert [int(x) for x in out] == [ctypes.sizeof(R), R.topk.offset, R.logits_dtype.offset, R.routed_scale.offset,
                                     R.flags.offset]
