"""Experts in 8 bits and the few-token forward on a machine without a GPU: sizes, and
the arguments they refuse before any launch (through the C ABI with pointers that are
never followed, and in the binding)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe
from mixture_experts_ffn_topk_gb300 import build

OK, NULL, SHAPE, DTYPE, VALUE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5, 6
F32, BF16, F16 = 0, 1, 2
FAKE = 0x7f0000000000          # 256-byte aligned, never dereferenced
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


def P(v):
    return ctypes.c_void_p(v)


def test_quantize_refusals(lib):
    def rows(**kw):
        a = dict(x=P(FAKE), ld=40, off=P(None), E=0, rows=10, K=40, dt=BF16, c=P(FAKE), ldc=40, s=P(FAKE))
        a.update(kw)
        return lib.moe_quantize_rows(a["x"], a["ld"], a["off"], a["E"], a["rows"], a["K"], a["dt"],
                                     a["c"], a["ldc"], a["s"], P(None))

    def swiglu(**kw):
        a = dict(x=P(FAKE), u=P(FAKE), ld=40, off=P(None), E=0, rows=10, K=40, dt=BF16, c=P(FAKE), ldc=40,
                 s=P(FAKE))
        a.update(kw)
        return lib.moe_swiglu_quantize(a["x"], a["u"], a["ld"], a["off"], a["E"], a["rows"], a["K"],
                                       a["dt"], a["c"], a["ldc"], a["s"], P(None))
    for call in (rows, swiglu):
        assert call(dt=3) == DTYPE and call(dt=-1) == DTYPE
        assert call(rows=-1) == SHAPE and call(rows=1 << 31) == SHAPE
        assert call(K=0) == SHAPE and call(K=(1 << 24) + 1, ld=1 << 25, ldc=1 << 25) == SHAPE
        assert call(ld=39) == SHAPE and call(ldc=39) == SHAPE
        assert call(ld=(1 << 32) + 1) == SHAPE and call(ldc=(1 << 32) + 1) == SHAPE
        assert call(off=P(FAKE), E=0) == SHAPE and call(off=P(FAKE), E=1025) == SHAPE
        assert call(off=P(FAKE + 4), E=4) == ALIGN
        for p in ("x", "c", "s"):
            assert call(**{p: P(None)}) == NULL
        assert call(x=P(FAKE + 1)) == ALIGN and call(s=P(FAKE + 4)) == ALIGN
        assert call(dt=F32, x=P(FAKE + 2)) == ALIGN
        assert call(rows=0, x=P(None), c=P(None), s=P(None)) == OK
    assert swiglu(u=P(None)) == NULL and swiglu(u=P(FAKE + 1)) == ALIGN

    def weights(**kw):
        a = dict(w=P(FAKE), E=4, N=40, K=48, dt=BF16, c=P(FAKE), s=P(FAKE))
        a.update(kw)
        return lib.moe_quantize_weights(a["w"], a["E"], a["N"], a["K"], a["dt"], a["c"], a["s"], P(None))
    assert weights(dt=4) == DTYPE
    assert weights(E=0) == SHAPE and weights(E=1025) == SHAPE
    assert weights(N=0) == SHAPE and weights(K=0) == SHAPE and weights(N=(1 << 24) + 1) == SHAPE
    assert weights(E=1024, N=1 << 24, K=1 << 24) == SHAPE       # too many blocks
    for p in ("w", "c", "s"):
        assert weights(**{p: P(None)}) == NULL
    assert weights(w=P(FAKE + 1)) == ALIGN and weights(s=P(FAKE + 8)) == ALIGN


def test_grouped_gemm_f8_refusals(lib):
    def call(**kw):
        a = dict(a=P(FAKE), lda=64, sa=P(FAKE), off=P(FAKE), rows=10, w=P(FAKE), sw=P(FAKE), lay=0, E=4,
                 N=40, K=64, out=P(FAKE), ldo=40, odt=BF16)
        a.update(kw)
        return lib.moe_grouped_gemm_f8(a["a"], a["lda"], a["sa"], a["off"], a["rows"], a["w"], a["sw"],
                                       a["lay"], a["E"], a["N"], a["K"], a["out"], a["ldo"], a["odt"],
                                       P(None))
    assert call(odt=3) == DTYPE and call(odt=-1) == DTYPE
    assert call(lay=2) == VALUE
    assert call(rows=-1) == SHAPE and call(rows=1 << 31) == SHAPE
    assert call(E=0) == SHAPE and call(E=1025) == SHAPE
    assert call(N=0) == SHAPE and call(K=0) == SHAPE
    assert call(N=(1 << 24) + 1, ldo=1 << 25) == SHAPE
    assert call(K=56) == SHAPE and call(K=72, lda=80) == SHAPE
    assert call(lay=1) == SHAPE                       # N = 40 is contiguous in [E, K, N]
    assert call(lay=1, N=41, ldo=41) == SHAPE
    assert call(lda=48) == SHAPE and call(lda=72) == SHAPE and call(lda=(1 << 32) + 16) == SHAPE
    assert call(ldo=39) == SHAPE and call(ldo=(1 << 32) + 1) == SHAPE
    for p in ("a", "sa", "off", "w", "sw", "out"):
        assert call(**{p: P(None)}) == NULL
        assert call(**{p: P(FAKE + 8)}) == ALIGN
    assert call(rows=0, a=P(None), sa=P(None), off=P(None), w=P(None), sw=P(None), out=P(None)) == OK


def experts(**kw):
    a = dict(gate=FAKE, up=FAKE, down=FAKE, gate_scales=None, up_scales=None, down_scales=None)
    a.update(kw)
    return moe.FewExperts(*[a[n] for n, _ in moe.FewExperts._fields_])


def test_forward_few_refusals(lib):
    scales = dict(gate_scales=FAKE, up_scales=FAKE, down_scales=FAKE)

    def few(**kw):
        a = dict(x=P(FAKE), dt=BF16, r=P(FAKE), rdt=F32, e=experts(), T=3, H=48, I=64, E=8, k=2, y=P(FAKE),
                 ws=P(FAKE), n=1 << 20)
        a.update(kw)
        e = None if a["e"] is None else ctypes.byref(a["e"])
        return lib.moe_forward_few(a["x"], a["dt"], a["r"], a["rdt"], e, a["T"], a["H"], a["I"], a["E"],
                                   a["k"], 0, a["y"], a["ws"], a["n"], P(None))

    def routed(**kw):
        a = dict(x=P(FAKE), dt=BF16, i=P(FAKE), r=P(FAKE), rdt=F32, e=experts(), T=3, H=48, I=64, E=8, k=2,
                 y=P(FAKE), ws=P(FAKE), n=1 << 20)
        a.update(kw)
        e = None if a["e"] is None else ctypes.byref(a["e"])
        return lib.moe_forward_few_routed(a["x"], a["dt"], a["i"], a["r"], a["rdt"], e, a["T"], a["H"],
                                          a["I"], a["E"], a["k"], a["y"], a["ws"], a["n"], P(None))
    for call in (few, routed):
        assert call(dt=3) == DTYPE and call(rdt=5) == DTYPE
        assert call(dt=F32, e=experts(**scales)) == DTYPE
        assert call(T=-1) == SHAPE and call(T=33) == SHAPE
        assert call(E=0) == SHAPE and call(E=1025) == SHAPE
        assert call(k=0) == SHAPE and call(k=9) == SHAPE and call(E=64, k=33) == SHAPE
        assert call(H=0) == SHAPE and call(I=0) == SHAPE and call(H=44) == SHAPE and call(I=60) == SHAPE
        assert call(H=40, e=experts(**scales)) == SHAPE        # 8-bit weights: multiples of 16
        assert call(dt=F32, H=46) == SHAPE
        assert call(H=65536 + 16) == SHAPE and call(I=65536 + 16) == SHAPE
        assert call(e=None) == NULL
        for p in ("x", "r", "y"):
            assert call(**{p: P(None)}) == NULL and call(**{p: P(FAKE + 8)}) == ALIGN
        for p in ("gate", "up", "down"):
            assert call(e=experts(**{p: None})) == NULL and call(e=experts(**{p: FAKE + 8})) == ALIGN
        for p in scales:                                        # all scales or none
            assert call(e=experts(**{**scales, p: None})) == NULL
            assert call(e=experts(**{**scales, p: FAKE + 8})) == ALIGN
        need = moe.moe_forward_few_workspace_size(3, 64, 2, torch.bfloat16)
        assert need == 3 * 2 * 64 * 2
        assert call(n=need - 1) == WORKSPACE and call(ws=P(None)) == WORKSPACE and call(ws=P(FAKE + 16)) == WORKSPACE
        assert call(T=0, x=P(None), y=P(None), ws=P(None), n=0) == OK
    assert routed(i=P(None)) == NULL and routed(i=P(FAKE + 8)) == ALIGN
    for a in ((0, 64, 2), (33, 64, 2), (3, 0, 2), (3, 64, 0), (3, 64, 33)):
        assert moe.moe_forward_few_workspace_size(*a, torch.bfloat16) == 0
    # h's 5 * 3 * 72 values of 4 bytes, in whole 256 bytes
    assert moe.moe_forward_few_workspace_size(5, 72, 3, torch.float32) == 4352


def test_few_experts_layout(lib, tmp_path):
    """The structure is laid out as a C compiler lays out the header's."""
    import os
    import subprocess
    fields = [n for n, _ in moe.FewExperts._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {\n'
                   '    printf("%zu\\n", sizeof(moe_few_experts));\n'
                   + "".join(f'    printf("%zu\\n", offsetof(moe_few_experts, {n}));\n' for n in fields)
                   + "    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(build.ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(moe.FewExperts)] + [getattr(moe.FewExperts, n).offset for n in fields]


def test_binding_refusals(lib):
    """What the binding checks itself, before it needs a device."""
    x, off = torch.zeros(4, 16), torch.zeros(3, dtype=torch.int32)
    codes, scales = torch.zeros(4, 16).to(F8), torch.zeros(4, 1)
    w, ws = torch.zeros(2, 8, 16).to(F8), torch.zeros(2, 1, 1)
    for call in (lambda: moe.moe_quantize_rows(x), lambda: moe.moe_quantize_weights(x.view(1, 4, 16)),
                 lambda: moe.moe_swiglu_quantize(x, x),
                 lambda: moe.moe_grouped_gemm_f8(codes, scales, off, w, ws),
                 lambda: moe.moe_forward_few(x, x, x.view(1, 4, 16), x.view(1, 4, 16), x.view(1, 16, 4), 1, True),
                 lambda: moe.moe_forward_few_routed(x, off.view(3, 1), x[:, :1], x.view(1, 4, 16),
                                                    x.view(1, 4, 16), x.view(1, 16, 4))):
        with pytest.raises(ValueError):                # CPU tensors
            call()
