"""Grouped products and the SwiGLU checkpoint on a machine without a GPU: the
sizes and layout they report, and the arguments they refuse before any launch
(through the C ABI with pointers that are never followed, and in the binding)."""

import ctypes
import os
import subprocess

import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe
from mixture_experts_ffn_topk_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, DTYPE, VALUE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5, 6
F32, BF16, F16 = 0, 1, 2
FAKE = 0x7f0000000000          # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


def P(v):
    return ctypes.c_void_p(v)


def test_grouped_gemm_refusals(lib):
    def call(**kw):
        a = dict(a=P(FAKE), lda=64, off=P(FAKE), rows=10, w=P(FAKE), lay=0, E=4, N=40, K=64,
                 dt=BF16, out=P(FAKE), ldo=40, odt=BF16)
        a.update(kw)
        return lib.moe_grouped_gemm(a["a"], a["lda"], a["off"], a["rows"], a["w"], a["lay"],
                                    a["E"], a["N"], a["K"], a["dt"], a["out"], a["ldo"],
                                    a["odt"], P(None))
    assert call(dt=3) == DTYPE
    assert call(odt=F16) == DTYPE              # neither the operands' nor F32
    assert call(dt=F32, odt=BF16) == DTYPE
    assert call(lay=2) == VALUE
    assert call(rows=-1) == SHAPE
    assert call(rows=1 << 31) == SHAPE
    assert call(E=0) == SHAPE and call(E=1025) == SHAPE
    assert call(N=0) == SHAPE and call(K=0) == SHAPE
    assert call(N=(1 << 24) + 8, ldo=1 << 25) == SHAPE
    assert call(K=60, lda=64) == SHAPE         # 120 bytes
    assert call(dt=F32, odt=F32, K=62, lda=64) == SHAPE
    assert call(lay=1, N=41, ldo=41) == SHAPE  # N is contiguous in [E, K, N]
    assert call(lda=56) == SHAPE and call(lda=68) == SHAPE
    assert call(ldo=39) == SHAPE
    assert call(lda=(1 << 32) + 8) == SHAPE and call(ldo=(1 << 32) + 8) == SHAPE
    for p in ("a", "off", "w", "out"):
        assert call(**{p: P(None)}) == NULL
        assert call(**{p: P(FAKE + 8)}) == ALIGN
    # no rows: nothing to do, whatever the pointers
    assert call(rows=0, a=P(None), off=P(None), w=P(None), out=P(None)) == OK
    call(ldo=39)
    assert b"ldo" in lib.moe_last_error_detail()


def test_weight_grad_refusals(lib):
    def call(**kw):
        a = dict(g=P(FAKE), ldg=40, a=P(FAKE), lda=64, off=P(FAKE), rows=10, E=4, N=40, K=64,
                 dt=BF16, gw=P(FAKE), gdt=F32, acc=0)
        a.update(kw)
        return lib.moe_grouped_gemm_weight_grad(a["g"], a["ldg"], a["a"], a["lda"], a["off"],
                                                a["rows"], a["E"], a["N"], a["K"], a["dt"],
                                                a["gw"], a["gdt"], a["acc"], P(None))
    assert call(dt=7) == DTYPE and call(gdt=F16) == DTYPE
    assert call(rows=-1) == SHAPE and call(E=0) == SHAPE and call(E=1025) == SHAPE
    assert call(N=36) == SHAPE and call(K=60) == SHAPE
    assert call(ldg=32) == SHAPE and call(ldg=44) == SHAPE
    assert call(lda=56) == SHAPE and call(lda=68) == SHAPE
    for p in ("g", "a", "off", "gw"):
        assert call(**{p: P(None)}) == NULL
        assert call(**{p: P(FAKE + 8)}) == ALIGN
    # no rows, accumulating: grad_w stays as it is
    assert call(rows=0, acc=1, g=P(None), a=P(None), off=P(None)) == OK
    assert call(rows=0, acc=1, gw=P(None)) == NULL


def test_checkpoint_sizes(lib, tmp_path):
    for rows, I in [(1, 1), (3, 31), (3, 32), (3, 33), (1023, 2048), (24576, 1408), (7, 14336)]:
        p = moe.moe_swiglu_checkpoint_layout(rows, I)
        cols = (I + 31) // 32 * 32
        assert p.row_codes == cols and p.row_scales == cols // 32
        at = 0
        for name, n in (("gate_codes", rows * cols), ("up_codes", rows * cols),
                        ("gate_scales", rows * cols // 32), ("up_scales", rows * cols // 32)):
            assert getattr(p, name) == at and at % 256 == 0
            at += (n + 255) // 256 * 256
        assert p.total == at == moe.moe_swiglu_checkpoint_size(rows, I)
    # a checkpoint of more than 2^32 bytes
    assert moe.moe_swiglu_checkpoint_size(1 << 22, 14336) == 2 * (1 << 22) * (14336 + 448)
    assert moe.moe_swiglu_checkpoint_size(-1, 8) == 0
    assert moe.moe_swiglu_checkpoint_size(8, 0) == 0
    assert lib.moe_swiglu_checkpoint_layout(8, 0, ctypes.byref(moe.CheckpointLayout())) == SHAPE
    assert lib.moe_swiglu_checkpoint_layout(8, 8, None) == NULL
    # the structure is laid out as a C compiler lays out the header's
    fields = [n for n, _ in moe.CheckpointLayout._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {\n'
                   '    printf("%zu\\n", sizeof(moe_checkpoint_layout));\n'
                   + "".join(f'    printf("%zu\\n", offsetof(moe_checkpoint_layout, {n}));\n' for n in fields)
                   + "    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(moe.CheckpointLayout)] + [getattr(moe.CheckpointLayout, n).offset
                                                           for n in fields]


def test_checkpoint_refusals(lib):
    def fwd(**kw):
        a = dict(g=P(FAKE), u=P(FAKE), ld=40, off=P(None), E=0, rows=10, I=40, dt=BF16, h=P(FAKE),
                 ldh=40, ck=P(FAKE), nb=1 << 20)
        a.update(kw)
        return lib.moe_swiglu_checkpoint(a["g"], a["u"], a["ld"], a["off"], a["E"], a["rows"],
                                         a["I"], a["dt"], a["h"], a["ldh"], a["ck"], a["nb"], P(None))

    def bwd(**kw):
        a = dict(g=P(FAKE), ld=40, off=P(None), E=0, rows=10, I=40, dt=BF16, dg=P(FAKE), du=P(FAKE),
                 ldg=80, h=P(FAKE), ldh=40, ck=P(FAKE), nb=1 << 20)
        a.update(kw)
        return lib.moe_swiglu_checkpoint_backward(a["g"], a["ld"], a["ck"], a["nb"], a["off"], a["E"],
                                                  a["rows"], a["I"], a["dt"], a["dg"], a["du"],
                                                  a["ldg"], a["h"], a["ldh"], P(None))
    for call in (fwd, bwd):
        assert call(dt=5) == DTYPE
        assert call(rows=-1) == SHAPE and call(I=0) == SHAPE
        assert call(off=P(FAKE), E=0) == SHAPE and call(off=P(FAKE), E=1025) == SHAPE
        assert call(off=P(FAKE + 4), E=4) == ALIGN
        assert call(ld=39) == SHAPE and call(ldh=39) == SHAPE
        assert call(g=P(None)) == NULL and call(g=P(FAKE + 1)) == ALIGN
        assert call(ck=P(None)) == WORKSPACE and call(ck=P(FAKE + 16)) == WORKSPACE
        need = moe.moe_swiglu_checkpoint_size(10, 40)
        assert call(nb=need - 1) == WORKSPACE
        assert call(rows=0, g=P(None), ck=P(None), h=P(None)) == OK
    assert fwd(u=P(None)) == NULL and fwd(h=P(None)) == NULL
    assert bwd(dg=P(None)) == NULL and bwd(du=P(None)) == NULL and bwd(ldg=39) == SHAPE
    assert fwd(dt=F32, h=P(FAKE + 2)) == ALIGN


def test_binding_refusals(lib):
    """What the binding checks itself, before it needs a device."""
    off = torch.zeros(3, dtype=torch.int32)
    a, w = torch.zeros(4, 16), torch.zeros(2, 8, 16)
    with pytest.raises(ValueError):                    # CPU tensors
        moe.moe_grouped_gemm(a, off, w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off.long(), w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off[:1], w)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w[:1])            # E differs
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w, transposed=True)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w.double())
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w, out=torch.zeros(4, 9))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w, out=torch.zeros(4, 8), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a.T.contiguous().T, off, w)   # columns are not contiguous
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_weight_grad(a, a, off, accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_weight_grad(a, a[:3], off)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm_weight_grad(a, a, off, grad_w=torch.zeros(2, 16, 8))
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint(a, a[:, :8])
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint(a, torch.zeros(4, 32)[:, :16])   # strides differ
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint(a, a)
    ck = torch.zeros(moe.moe_swiglu_checkpoint_size(4, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint_backward(a, ck, grad_g=torch.zeros(4, 16))
    with pytest.raises(ValueError):
        moe.moe_swiglu_checkpoint_backward(a, ck)


def test_checkpoint_views(lib):
    rows, I = 5, 40
    p = moe.moe_swiglu_checkpoint_layout(rows, I)
    ck = torch.arange(p.total, dtype=torch.int64).to(torch.uint8)
    v = moe.swiglu_checkpoint_views(ck, rows, I)
    assert v["gate_codes"].shape == (5, 64) and v["gate_codes"].dtype == torch.float8_e4m3fn
    assert v["up_scales"].shape == (5, 2) and v["up_scales"].dtype == torch.uint8
    assert v["up_codes"].view(torch.uint8)[1, 3] == ck[p.up_codes + 64 + 3]
    assert v["up_scales"][4, 1] == ck[p.up_scales + 9]
