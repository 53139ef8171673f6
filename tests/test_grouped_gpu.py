"""Grouped products, their weight gradient and the SwiGLU checkpoint on the GPU,
against plain 64-bit implementations.

Tolerances. A product's FP32 sum of n terms is off by at most n * 2^-23 times
the sum of the terms' magnitudes, in any order (each of the n additions loses at
most one unit of a partial sum that is no larger; products of 16-bit values are
exact in FP32, those of FP32 values lose 2^-24 each, and n + 1 covers them); the
output is then rounded once, by half a step of its type. Both are computed per
element. The checkpoint's codes and scales are exact. h and the gradients of the
activation are a dozen FP32 operations: 16 * 2^-23 of the terms' magnitudes
(the fast exponential of the 16-bit types is within 2^-21 * (1 + |g|), counted
apart), then the output's rounding.
"""

import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BAD_INDEX = 9


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_topk_gb300 import build
    build.build()
    moe.moe_device_status(clear=True)


@pytest.fixture(autouse=True)
def status_stays_clear(request):
    yield
    torch.cuda.synchronize()
    if "bad_offsets" not in request.node.name:
        assert moe.moe_device_status(clear=True) == 0


def rounding(ref, dtype):
    """Half a step of dtype at |ref| (ref in 64 bits), its subnormals included."""
    f = torch.finfo(dtype)
    return torch.maximum(ref.abs() * (f.eps / 2), torch.tensor(f.tiny * f.eps / 2, dtype=torch.float64,
                                                               device=ref.device))


def check(got, ref, slack, dtype, what):
    """|got - ref| <= slack + half a step of what may be rounded, NaN where ref is."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    fine = torch.isfinite(ref)
    bound = slack + rounding(ref.abs() + slack, dtype)
    err = torch.where(fine, (got - ref).abs(), torch.zeros_like(ref))
    over = torch.where(fine, err - bound, torch.full_like(ref, -1.0))
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: error {err.flatten()[i]:.3e} > {bound.flatten()[i]:.3e} at {i} "
                             f"(ref {ref.flatten()[i]:.6e}, got {got.flatten()[i]:.6e}); "
                             f"{int((over > 0).sum())} of {over.numel()} over")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32, device="cuda")


def strided(rows, cols, dtype, g, pad, std=1.0):
    """A [rows, cols] matrix inside a wider one with NaN between its rows."""
    whole = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    whole[:, :cols] = torch.randn((rows, cols), generator=g, device="cuda") * std
    return whole[:, :cols]


def ref_product(a, off, w, transposed):
    rows, N = a.shape[0], w.shape[2 if transposed else 1]
    out = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    at = off.tolist()
    for e in range(len(at) - 1):
        s = slice(at[e], at[e + 1])
        m = w[e].double() if transposed else w[e].double().T
        out[s] = a[s].double() @ m
        size[s] = a[s].double().abs() @ m.abs()
    return out, size


COUNTS = {
    "one_row": [1],
    "one_of_many": [0, 0, 1, 0],
    "edges": [0, 15, 16, 17, 0, 31, 32, 33],
    "tiles": [63, 64, 65, 127, 0, 128, 129],
    "wide": [255, 0, 256, 257, 1, 300],
    "long": [700, 3, 1025],
    "empty": [0, 0, 0],
}

# N, K, transposed: tile edges in both, a single block, K that ends inside a block
SHAPES = [(8, 8, False), (8, 8, True), (72, 40, True), (130, 136, False), (1, 64, False),
          (250, 320, False), (256, 192, True), (264, 1000, True), (520, 72, False)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("N,K,transposed", SHAPES)
def test_product(dtype, counts, N, K, transposed):
    c = COUNTS[counts]
    g = gen(hash((N, K, len(c))) % 1000)
    first, rows, E = 3, 3 + sum(c) + 5, len(c)       # rows of no expert before and behind
    off = offsets_of(c, first)
    a = strided(rows, K, dtype, g, 8)
    a[:first], a[first + sum(c):] = float("nan"), float("inf")
    w = torch.randn((E, K, N) if transposed else (E, N, K), generator=g, device="cuda").to(dtype)
    ref, size = ref_product(a, off, w, transposed)
    for out_dtype in {dtype, F32}:
        for pad in (0, 3, 8):
            whole = torch.full((rows, N + pad), -7.0, dtype=out_dtype, device="cuda")
            out = moe.moe_grouped_gemm(a, off, w, transposed=transposed, out=whole[:, :N])
            assert torch.all(whole[:first] == -7) and torch.all(whole[first + sum(c):] == -7)
            assert torch.all(whole[:, N:] == -7)
            s = slice(first, first + sum(c))
            check(out[s], ref[s], size[s] * (K + 1) * 2.0 ** -23, out_dtype, f"{out_dtype} pad {pad}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [64], [65], [16, 1, 0, 40], [130]])
@pytest.mark.parametrize("N,K,transposed", [(8, 520, False), (8, 4104, True), (130, 2048, False),
                                            (250, 4096, False), (256, 1032, True), (1000, 1024, False),
                                            (1, 7168, False), (1032, 2056, True)])
def test_product_of_few_rows_over_a_long_k(dtype, counts, N, K, transposed):
    """Few units of work: their k is shared by 2, 4 or 8 CTAs whose sums are joined."""
    g = gen(N + K)
    first, rows, E = 2, sum(counts) + 5, len(counts)
    off = offsets_of(counts, first)
    a = strided(rows, K, dtype, g, 8)
    a[:first], a[first + sum(counts):] = float("nan"), float("inf")
    w = torch.randn((E, K, N) if transposed else (E, N, K), generator=g, device="cuda").to(dtype)
    ref, size = ref_product(a, off, w, transposed)
    s = slice(first, first + sum(counts))
    for out_dtype in {dtype, F32}:
        whole = torch.full((rows, N + 3), -7.0, dtype=out_dtype, device="cuda")
        out = moe.moe_grouped_gemm(a, off, w, transposed=transposed, out=whole[:, :N])
        assert torch.all(whole[:first] == -7) and torch.all(whole[s.stop:] == -7) and torch.all(whole[:, N:] == -7)
        check(out[s], ref[s], size[s] * (K + 1) * 2.0 ** -23, out_dtype, f"{out_dtype}")
        again = moe.moe_grouped_gemm(a, off, w, transposed=transposed, out_dtype=out_dtype)
        assert torch.equal(again[s], out[s])


def test_product_of_few_rows_with_bad_offsets():
    """The joined form also serves what is sound and touches nothing else."""
    g = gen(30)
    a = torch.randn((20, 2048), generator=g, device="cuda").to(BF16)
    w = torch.randn((3, 64, 2048), generator=g, device="cuda").to(BF16)
    out = torch.full((20, 64), -7.0, dtype=BF16, device="cuda")
    moe.moe_device_status(clear=True)
    moe.moe_grouped_gemm(a, torch.tensor([0, 5, 30, 20], dtype=torch.int32, device="cuda"), w, out=out)
    assert moe.moe_device_status(clear=True) == BAD_INDEX
    ref = a[:5].double() @ w[0].double().T
    size = a[:5].double().abs() @ w[0].double().abs().T
    check(out[:5], ref, size * 2049 * 2.0 ** -23, BF16, "the sound expert")
    assert torch.all(out[5:] == -7)


def test_fp32_outputs_do_not_drift_over_long_sums():
    """Positive terms, so that a sum that loses a little at each step loses it always. FP32 outputs of
    16-bit operands are summed in parts of 768 terms: at most 48 truncating steps of 16 and 17 roundings
    within a step, then one rounding per part, each of at most 2^-23 of the (positive) sum."""
    g = gen(40)
    pos = lambda *s: (torch.rand(s, generator=g, device="cuda") + 0.5).to(BF16)
    K = 14336
    tol = (48 + 17 + (K + 767) // 768) * 2.0 ** -23
    for E, rows, N in ((1, 3, 40), (2, 300, 264), (8, 48, 2100)):      # joined, pairs, single CTAs
        off = offsets_of([rows // E] * E)
        a, w = pos(rows, K), pos(E, N, K)
        ref, _ = ref_product(a, off, w, False)
        for got in (moe.moe_grouped_gemm(a, off, w, out_dtype=F32),
                    moe.moe_grouped_gemm(a, off, w.transpose(1, 2).contiguous(), transposed=True, out_dtype=F32)
                    if N % 8 == 0 else ref):
            assert float(((got.double() - ref).abs() / ref).max()) <= tol, (E, rows, N)
    for E, rows, N, K in ((1, 20000, 40, 72), (2, 12000, 264, 2048), (16, 16 * 500 + 3000, 1024, 1032)):
        c = [3500] + [500] * (E - 1) if E == 16 else [rows // E] * E   # joined, pairs, single CTAs
        off = offsets_of(c)
        a, d = pos(rows, K), pos(rows, N)
        at = off.tolist()
        got = moe.moe_grouped_gemm_weight_grad(d, a, off)
        old = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=got.clone(), accumulate=True)
        for e in range(E):
            s = slice(at[e], at[e + 1])
            ref = d[s].double().T @ a[s].double()
            tol = (48 + 17 + (c[e] + 767) // 768 + 8) * 2.0 ** -23     # and up to 8 joined CTAs
            assert float(((got[e].double() - ref).abs() / ref).max()) <= tol, (E, e)
            assert float(((old[e].double() - 2 * ref).abs() / ref).max()) <= 2 * tol, (E, e)


def test_product_many_experts():
    """1024 experts, most of them idle, and the last one busy."""
    g = gen(5)
    r = np.random.RandomState(5)
    c = np.where(r.rand(1024) < 0.15, r.randint(1, 40, 1024), 0)
    c[1023] = 70
    off, rows = offsets_of(c), int(c.sum())
    for dtype in (BF16, F32):
        a = torch.randn((rows, 64), generator=g, device="cuda").to(dtype)
        w = torch.randn((1024, 48, 64), generator=g, device="cuda").to(dtype)
        ref, size = ref_product(a, off, w, False)
        check(moe.moe_grouped_gemm(a, off, w), ref, size * 65 * 2.0 ** -23, dtype, str(dtype))


def test_product_nan_stays_in_its_row_and_expert():
    g = gen(6)
    for dtype in (BF16, F16, F32):
        off = offsets_of([70, 61, 130])
        a = torch.randn((261, 128), generator=g, device="cuda").to(dtype)
        w = torch.randn((3, 96, 128), generator=g, device="cuda").to(dtype)
        a[70, 5], a[130, 0], w[2, 7, 3] = float("nan"), float("-inf"), float("inf")
        bad = torch.zeros((261, 96), dtype=torch.bool, device="cuda")
        bad[70], bad[130] = True, True
        bad[131:, 7] = True
        for out in (moe.moe_grouped_gemm(a, off, w),
                    moe.moe_grouped_gemm(a, off, w.transpose(1, 2).contiguous(), transposed=True)):
            assert torch.equal(~torch.isfinite(out), bad)


def test_product_beyond_2_31_elements():
    """Element offsets past 2^31, in the rows, the output and the weights."""
    g = gen(7)
    rows, N, K = 263000, 8200, 64
    off = offsets_of([100, 262000, 900])
    a = torch.randn((rows, K), generator=g, device="cuda").to(BF16)
    w = torch.randn((3, N, K), generator=g, device="cuda").to(BF16)
    out = moe.moe_grouped_gemm(a, off, w)
    assert out.numel() > 2 ** 31
    for e, s in ((0, slice(0, 100)), (1, slice(261000, 262100)), (2, slice(262100, 263000))):
        ref = a[s].double() @ w[e].double().T
        size = a[s].double().abs() @ w[e].double().abs().T
        check(out[s], ref, size * 65 * 2.0 ** -23, BF16, f"rows {s}")
    del out
    whole = torch.zeros((rows, 8192 + 64), dtype=BF16, device="cuda")
    whole[:, 8192:] = a
    w2 = torch.randn((3, 24, K), generator=g, device="cuda").to(BF16)
    out = moe.moe_grouped_gemm(whole[:, 8192:], off, w2)
    ref, size = ref_product(a, off, w2, False)
    check(out, ref, size * 65 * 2.0 ** -23, BF16, "rows far apart")
    del whole
    E = 300
    w3 = torch.randn((8, 4000, 2048), generator=g, device="cuda").to(BF16)
    big = torch.empty((E, 4000, 2048), dtype=BF16, device="cuda")
    big[-8:] = w3
    assert big.numel() > 2 ** 31
    c = [0] * (E - 8) + [3, 0, 20, 1, 1, 0, 40, 5]
    a = torch.randn((sum(c), 2048), generator=g, device="cuda").to(BF16)
    got = moe.moe_grouped_gemm(a, offsets_of(c), big)
    ref, size = ref_product(a, offsets_of(c[-8:]), w3, False)
    check(got, ref, size * 2049 * 2.0 ** -23, BF16, "weights")


@pytest.mark.parametrize("bad", [[0, 40, 20, 60], [-1, 10, 20, 60], [0, 10, 20, 61],
                                 [0, 10, 2 ** 31 - 1, 60], [0, -5, 20, 60], [60, 0, 0, 60]])
def test_bad_offsets(bad):
    """An expert whose offsets fall or leave the matrix has no rows; the others are served."""
    g = gen(8)
    N = K = 64
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for dtype in (BF16, F32):
        moe.moe_device_status(clear=True)
        room = torch.full((180, N), -7.0, dtype=dtype, device="cuda")
        out = room[60:120]
        a = torch.randn((60, K), generator=g, device="cuda").to(dtype)
        w = torch.randn((3, N, K), generator=g, device="cuda").to(dtype)
        moe.moe_grouped_gemm(a, off, w, out=out)
        assert moe.moe_device_status(clear=True) == BAD_INDEX
        seen = torch.zeros(60, dtype=torch.bool, device="cuda")
        for e in range(3):
            lo, hi = bad[e], bad[e + 1]
            if 0 <= lo <= hi <= 60:
                s = slice(lo, hi)
                free = ~seen[s]                       # rows that two experts name hold either's product
                ref = a[s].double() @ w[e].double().T
                size = a[s].double().abs() @ w[e].double().abs().T
                if bad != [0, 40, 20, 60]:
                    check(out[s][free], ref[free], (size * 65 * 2.0 ** -23)[free], dtype, f"expert {e}")
                seen[s] = True
        assert torch.all(out[~seen] == -7) and torch.all(room[:60] == -7) and torch.all(room[120:] == -7)
        gw = moe.moe_grouped_gemm_weight_grad(out, a, off)
        assert moe.moe_device_status(clear=True) == BAD_INDEX
        for e in range(3):
            if not 0 <= bad[e] <= bad[e + 1] <= 60:
                assert torch.all(gw[e] == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,rows,K", [(64, 60, 2048), (1000, 100, 64), (6, 700, 128)])
def test_bad_offsets_that_name_rows_again_and_again(dtype, E, rows, K):
    """0, rows, 0, rows, ...: only the first expert has rows; the others neither write them a second
    time nor make more units than the launch was sized for."""
    g = gen(E)
    off = torch.tensor([0 if e % 2 == 0 else rows - 10 for e in range(E + 1)], dtype=torch.int32, device="cuda")
    a = torch.randn((rows, K), generator=g, device="cuda").to(dtype)
    w = torch.randn((E, 40, K), generator=g, device="cuda").to(dtype)
    out = torch.full((rows, 40), -7.0, dtype=dtype, device="cuda")
    moe.moe_device_status(clear=True)
    moe.moe_grouped_gemm(a, off, w, out=out)
    gw = moe.moe_grouped_gemm_weight_grad(a, a, off) if K <= 128 else None
    assert moe.moe_device_status(clear=True) == BAD_INDEX
    n = rows - 10
    ref = a[:n].double() @ w[0].double().T
    size = a[:n].double().abs() @ w[0].double().abs().T
    check(out[:n], ref, size * (K + 1) * 2.0 ** -23, dtype, "the first expert")
    assert torch.all(out[n:] == -7)
    if gw is not None:
        assert torch.all(gw[1:] == 0) and torch.any(gw[0] != 0)


def test_few_rows_captured_and_replayed():
    """The form that joins sums over a cluster, in two graphs on two streams."""
    g = gen(31)
    a = torch.randn((3, 4096), generator=g, device="cuda").to(BF16)
    w = torch.randn((2, 256, 4096), generator=g, device="cuda").to(BF16)
    off = offsets_of([1, 2])
    outs = [torch.zeros((3, 256), dtype=BF16, device="cuda") for _ in range(2)]
    moe.moe_grouped_gemm(a, off, w, out=outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_grouped_gemm(a, off, w, out=o)
            moe.moe_grouped_gemm(a, off, w, out=o)
        graphs.append(graph)
    for counts in ([2, 1], [0, 3], [3, 0]):
        off.copy_(offsets_of(counts))
        a.copy_(torch.randn((3, 4096), generator=g, device="cuda"))
        want = moe.moe_grouped_gemm(a, off, w)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            graphs[0].replay()
            with torch.cuda.stream(side):
                graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


GRAD_SHAPES = [(8, 8), (72, 40), (136, 264), (256, 320), (520, 72)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("N,K", GRAD_SHAPES)
def test_weight_grad(dtype, counts, N, K):
    c = COUNTS[counts]
    g = gen(hash((N, K, len(c), 3)) % 1000)
    first, rows, E = 2, 2 + sum(c) + 3, len(c)
    off = offsets_of(c, first)
    a, d = strided(rows, K, dtype, g, 8), strided(rows, N, dtype, g, 16)
    for m in (a, d):                                  # rows of no expert
        m[:first], m[first + sum(c):] = float("nan"), float("inf")
    at = off.tolist()
    ref = torch.stack([d[at[e]:at[e + 1]].double().T @ a[at[e]:at[e + 1]].double() for e in range(E)])
    size = torch.stack([d[at[e]:at[e + 1]].double().abs().T @ a[at[e]:at[e + 1]].double().abs()
                        for e in range(E)])
    terms = torch.tensor(c, device="cuda").view(E, 1, 1).double() + 1
    for out_dtype in {dtype, F32}:
        got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_dtype=out_dtype)
        check(got, ref, size * terms * 2.0 ** -23, out_dtype, f"{out_dtype}")
        old = torch.randn((E, N, K), generator=g, device="cuda").to(out_dtype)
        kept = old.clone()
        got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=kept, accumulate=True)
        assert got is kept
        sum_ = ref + old.double()
        slack = size * terms * 2.0 ** -23 + (ref.abs() + old.double().abs()) * 2.0 ** -24
        check(got, sum_, slack, out_dtype, f"accumulated {out_dtype}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", [[1000], [0, 3000, 5], [513, 512, 4097, 0], [40, 9000]])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 264), (136, 40), (256, 520)])
def test_weight_grad_of_narrow_matrices_over_long_segments(dtype, counts, N, K):
    """Few units of work: an expert's rows are shared by 2, 4 or 8 CTAs whose sums are joined."""
    g = gen(N + K + len(counts))
    first, rows, E = 3, sum(counts) + 8, len(counts)
    off = offsets_of(counts, first)
    a, d = strided(rows, K, dtype, g, 8), strided(rows, N, dtype, g, 8)
    for m in (a, d):
        m[:first], m[first + sum(counts):] = float("nan"), float("inf")
    at = off.tolist()
    ref = torch.stack([d[at[e]:at[e + 1]].double().T @ a[at[e]:at[e + 1]].double() for e in range(E)])
    size = torch.stack([d[at[e]:at[e + 1]].double().abs().T @ a[at[e]:at[e + 1]].double().abs()
                        for e in range(E)])
    terms = torch.tensor(counts, device="cuda").view(E, 1, 1).double() + 1
    for out_dtype in {dtype, F32}:
        room = torch.full((E + 2, N, K), -7.0, dtype=out_dtype, device="cuda")
        got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=room[1:E + 1])
        assert torch.all(room[0] == -7) and torch.all(room[-1] == -7)
        check(got, ref, size * terms * 2.0 ** -23, out_dtype, f"{out_dtype}")
        assert torch.equal(moe.moe_grouped_gemm_weight_grad(d, a, off, grad_dtype=out_dtype), got)
        old = torch.randn((E, N, K), generator=g, device="cuda").to(out_dtype)
        got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=old.clone(), accumulate=True)
        slack = size * terms * 2.0 ** -23 + (ref.abs() + old.double().abs()) * 2.0 ** -24
        check(got, ref + old.double(), slack, out_dtype, f"accumulated {out_dtype}")


def test_weight_grad_no_rows():
    gw = torch.full((3, 16, 24), 5.0, device="cuda")
    z = torch.zeros((0, 16), device="cuda", dtype=BF16)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_weight_grad(z, torch.zeros((0, 24), device="cuda", dtype=BF16), off, grad_w=gw,
                                     accumulate=True)
    assert torch.all(gw == 5)
    moe.moe_grouped_gemm_weight_grad(z, torch.zeros((0, 24), device="cuda", dtype=BF16), off, grad_w=gw)
    assert torch.all(gw == 0)
    assert moe.moe_grouped_gemm(z, off, torch.zeros((3, 24, 16), device="cuda", dtype=BF16)).shape == (0, 24)


def test_weight_grad_nan_stays_in_its_expert():
    """Experts that share a block of 64 rows: a NaN or infinity of one, in either operand, stays there."""
    g = gen(9)
    for dtype in (BF16, F16, F32):
        off = offsets_of([5, 3, 70, 1, 200])
        a = torch.randn((279, 72), generator=g, device="cuda").to(dtype)
        d = torch.randn((279, 136), generator=g, device="cuda").to(dtype)
        a[6], d[78] = float("nan"), float("inf")      # experts 1 and 3
        gw = moe.moe_grouped_gemm_weight_grad(d, a, off)
        fine = torch.isfinite(gw).all(dim=2).all(dim=1)
        assert fine.tolist() == [True, False, True, False, True]


def test_weight_grad_is_the_products_gradient():
    """sum(grad * product) changes by <grad_w, v> along v, and by <grad_a, v>: FP32, one
    direction each, against 64-bit differences of the (linear) product."""
    g = gen(10)
    c = [0, 33, 5, 90]
    off = offsets_of(c)
    a = torch.randn((128, 48), generator=g, device="cuda")
    w = torch.randn((4, 56, 48), generator=g, device="cuda")
    d = torch.randn((128, 56), generator=g, device="cuda")
    gw = moe.moe_grouped_gemm_weight_grad(d, a, off)
    ga = moe.moe_grouped_gemm(d, off, w, transposed=True)
    vw, va = torch.randn_like(w).double(), torch.randn_like(a).double()
    f = lambda aa, ww: (d.double() * ref_product(aa, off, ww, False)[0]).sum()
    for grad, diff in (((gw.double() * vw).sum(), f(a, w + vw) - f(a, w - vw)),
                       ((ga.double() * va).sum(), f(a + va, w) - f(a - va, w))):
        # 128 * 56 * 48 products: FP32 errors of 2^-23 * 91 terms each, random signs
        assert abs(grad - diff / 2) < 1e-4 * (128 * 56 * 48) ** 0.5


def test_products_repeat_bit_for_bit_on_any_stream():
    g = gen(11)
    c = [300, 0, 77, 513, 1, 2]
    off = offsets_of(c)
    for dtype in (BF16, F32):
        a = torch.randn((sum(c), 264), generator=g, device="cuda").to(dtype)
        w = torch.randn((6, 392, 264), generator=g, device="cuda").to(dtype)
        d = torch.randn((sum(c), 392), generator=g, device="cuda").to(dtype)
        calls = [lambda st=None: moe.moe_grouped_gemm(a, off, w, stream=st),
                 lambda st=None: moe.moe_grouped_gemm(d, off, w, transposed=True, stream=st),
                 lambda st=None: moe.moe_grouped_gemm_weight_grad(d, a, off, stream=st)]
        torch.cuda.synchronize()
        want = [f() for f in calls]
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        for _ in range(3):                            # two and more calls at once
            got = [f(st) for f, st in zip(calls, streams)]
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
        with torch.cuda.stream(streams[0]):
            got = [f() for f in calls]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_outputs_on_another_stream_take_that_streams_memory():
    """A block that the current stream has freed but still works on is not handed to a call on another
    stream: the output made there comes out right, and the pending work keeps its own values."""
    g = gen(50)
    rows, N, K = 4096, 2048, 256
    off = offsets_of([rows])
    a = torch.randn((rows, K), generator=g, device="cuda").to(BF16)
    w = torch.randn((1, N, K), generator=g, device="cuda").to(BF16)
    want = moe.moe_grouped_gemm(a, off, w)
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        busy = torch.ones((rows, N), dtype=BF16, device="cuda")
        for _ in range(30):                               # pending work on `busy`
            busy.mul_(1.0)
        total.add_(busy.sum(dtype=torch.float64))
        del busy                                          # free for the current stream's next tensor
        out = moe.moe_grouped_gemm(a, off, w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del out
    assert float(total) == 2.0 * rows * N


def test_captured_and_replayed():
    """Offsets, rows and weights may change between replays; two graphs run side by side."""
    g = gen(12)
    c1, c2 = [10, 200, 0, 46], [100, 0, 156, 0]
    a = torch.randn((256, 64), generator=g, device="cuda").to(BF16)
    w = torch.randn((4, 128, 64), generator=g, device="cuda").to(BF16)
    off = offsets_of(c1)
    h = torch.zeros((256, 64), dtype=BF16, device="cuda")
    out = torch.zeros((256, 128), dtype=BF16, device="cuda")
    gw = torch.zeros((4, 128, 64), device="cuda")
    ck = torch.zeros(moe.moe_swiglu_checkpoint_size(256, 64), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_grouped_gemm(a, off, w, out=out)
        moe.moe_swiglu_checkpoint(out[:, :64], out[:, 64:], off, h=h, ckpt=ck)
        moe.moe_grouped_gemm_weight_grad(out, a, off, grad_w=gw)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
    for counts in (c2, c1):
        off.copy_(offsets_of(counts))
        a.copy_(torch.randn((256, 64), generator=g, device="cuda"))
        want_out = moe.moe_grouped_gemm(a, off, w)
        want_gw = moe.moe_grouped_gemm_weight_grad(want_out, a, off)
        want_h = moe.moe_swiglu_checkpoint(want_out[:, :64], want_out[:, 64:], off)[0]
        torch.cuda.synchronize()
        for graph in graphs:
            out.zero_(), gw.zero_(), h.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want_out) and torch.equal(gw, want_gw) and torch.equal(h, want_h)
    # the same buffers, written by both with the same values, in any order
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()


# ------------------------------------------------------------ the checkpoint

def e4m3_values():
    b = torch.arange(128, dtype=torch.float64, device="cuda")
    ex, fr = torch.floor(b / 8), b % 8
    return torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * torch.exp2(ex - 7))[:127]


def ref_codes(v):
    """(values of the codes, scale exponents) of [rows, I], from the definition in 64 bits."""
    rows, I = v.shape
    cols = (I + 31) // 32 * 32
    x = torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
    x[:, :I] = v.double()
    x = x.view(rows, -1, 32)
    top = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    e = torch.full_like(top, -127.0)
    for k in range(-127, 119):                        # the smallest exponent that holds the block
        e = torch.where(top > 448 * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    y = (x / torch.exp2(e).unsqueeze(-1))
    grid = e4m3_values()
    m = y.abs().clamp(max=448)
    hi = torch.searchsorted(grid, m.nan_to_num(0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = m - grid[lo], grid[hi] - m
    # to nearest; halfway to the even code
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    val = torch.copysign(grid[code], y)
    val = torch.where(torch.isfinite(x), val, torch.full_like(val, float("nan")))
    return val.view(rows, cols), e


def loaded(ck, rows, I):
    v = moe.swiglu_checkpoint_views(ck, rows, I)
    out = []
    for n in ("gate", "up"):
        s = torch.exp2(v[n + "_scales"].double() - 127)
        out.append((v[n + "_codes"].double().view(rows, -1, 32) * s.unsqueeze(-1)).view(rows, -1)[:, :I])
    return out


def silu_slack(g, u, dtype):
    """Error of h = g t u before its rounding: a few FP32 roundings, and of the fast exponential."""
    rel = 16 * 2.0 ** -23 + (0 if dtype == F32 else 1) * 2.0 ** -21 * (1 + g.abs())
    # below FP32's normal range the result's rounding is absolute
    return (g * torch.sigmoid(g) * u).abs() * rel + 2.0 ** -120


def pairs(rows, I, dtype, seed, case):
    g = gen(seed)
    gu = torch.randn((rows, 2 * I), generator=g, device="cuda")
    if case == "spread":
        gu *= torch.exp(2 * torch.randn((1, 2 * I), generator=g, device="cuda"))
    if case == "small":
        gu *= 2.0 ** -10 if dtype == F16 else 2.0 ** -140
    if case == "large":
        gu *= 2.0 ** 12 if dtype == F16 else 2.0 ** 125
        gu = gu.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
    if case == "ties":       # values halfway between codes, and maxima on both sides of 448 s
        gu = torch.randint(-2000, 2000, (rows, 2 * I), generator=g, device="cuda").float() / 16
        gu[:, ::32] = 28.0
        gu[::2, ::32] = 28.125
    if case == "zeros":
        gu *= (torch.rand((rows, 2 * I), generator=g, device="cuda") < 0.02)
        gu[:, :: 3] *= -1
    if case == "nan":
        gu[torch.rand((rows, 2 * I), generator=g, device="cuda") < 0.05] = float("nan")
        gu[torch.rand((rows, 2 * I), generator=g, device="cuda") < 0.05] = float("inf")
        gu[torch.rand((rows, 2 * I), generator=g, device="cuda") < 0.05] = float("-inf")
    return gu.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,I", [(1, 1), (5, 7), (3, 8), (2, 31), (4, 32), (9, 33), (1, 100), (130, 160),
                                    (37, 1408), (3, 2047)])
@pytest.mark.parametrize("case", ["spread", "small", "large", "ties", "zeros", "nan"])
def test_checkpoint(dtype, rows, I, case):
    gu = pairs(rows, I, dtype, rows * 31 + I, case)
    stacked = (gu[:, :I], gu[:, I:])                  # the second half may start anywhere
    apart = (gu[:, :I].contiguous(), gu[:, I:].contiguous())
    for n, (g, u) in enumerate((stacked, apart)):
        whole = torch.full((rows + 2, I + 3 * n), -7.0, dtype=dtype, device="cuda")
        h, ck = moe.moe_swiglu_checkpoint(g, u, h=whole[1:rows + 1, :I])
        assert torch.all(whole[0] == -7) and torch.all(whole[-1] == -7) and torch.all(whole[:, I:] == -7)
        gd, ud = g.double(), u.double()
        ref = gd * torch.sigmoid(gd) * ud
        fits = ref.abs() < torch.finfo(dtype).max * 0.99
        ref = torch.where(fits | ~torch.isfinite(ref), ref, torch.full_like(ref, float("inf")))
        mask = torch.isfinite(gd) & torch.isfinite(ud)   # h of infinities is as the formula's FP32 has it
        check(torch.where(mask, h.double(), 0.0), torch.where(mask, ref, 0.0),
              torch.where(mask & torch.isfinite(ref), silu_slack(gd, ud, dtype), 0.0), dtype, "h")
        assert torch.all(torch.isnan(h.double())[torch.isnan(gd) | torch.isnan(ud)])
        v = moe.swiglu_checkpoint_views(ck, rows, I)
        for name, x in (("gate", g), ("up", u)):
            val, e = ref_codes(x)
            assert torch.equal(v[name + "_scales"].double() - 127, e)
            got = v[name + "_codes"].double()
            assert torch.equal(torch.isnan(got), torch.isnan(val))
            assert torch.equal(got.nan_to_num(0), val.nan_to_num(0))


def backward_ref(d, g, u):
    t = torch.sigmoid(g)
    return d * u * t * (1 + g * (1 - t)), d * g * t, g * t * u


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,I", [(1, 1), (5, 7), (3, 8), (9, 33), (1, 100), (130, 160), (37, 1408)])
@pytest.mark.parametrize("case", ["spread", "small", "ties", "zeros", "nan"])
def test_checkpoint_backward(dtype, rows, I, case):
    gu = pairs(rows, I, dtype, rows * 17 + I, case)
    ck = moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:])[1]
    g, u = loaded(ck, rows, I)
    for pad in (0, 1, 8):
        d = strided(rows, I, dtype, gen(rows + I), pad)
        # FP32 arithmetic on the checkpoint's values, as large as the largest term of each formula
        rg, ru, rh = backward_ref(d.double(), g, u)
        t = torch.sigmoid(g)
        rel = 16 * 2.0 ** -23 + (0 if dtype == F32 else 1) * 2.0 ** -21 * (1 + g.abs())
        sg = (d.double() * u).abs() * t * (1 + (g * (1 - t)).abs()) * rel + 2.0 ** -120
        su = ru.abs() * rel + 2.0 ** -120
        sh = rh.abs() * rel + 2.0 ** -120
        if pad == 8:
            room = torch.full((rows, 2 * I + 5), -7.0, dtype=dtype, device="cuda")
            dg, du, h = moe.moe_swiglu_checkpoint_backward(d, ck, grad_g=room[:, :I], grad_u=room[:, I:2 * I])
            assert torch.all(room[:, 2 * I:] == -7)
        else:
            dg, du, h = moe.moe_swiglu_checkpoint_backward(d, ck, need_h=pad == 0)
            assert (h is None) == (pad == 1)
        top = torch.finfo(dtype).max * 0.99
        for name, got, ref, slack in (("grad_g", dg, rg, sg), ("grad_u", du, ru, su), ("h", h, rh, sh)):
            if got is None:
                continue
            over = ref.abs() >= top                   # F16 may overflow there
            check(torch.where(over, 0.0, got.double()), torch.where(over, 0.0, ref),
                  torch.where(over, 0.0, slack), dtype, name)


def test_checkpoint_backward_against_differences():
    """The gradients along a direction equal differences of SiLU(g) u at the checkpoint's values."""
    rows, I = 64, 96
    gu = pairs(rows, I, F32, 3, "plain")
    ck = moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:])[1]
    g, u = loaded(ck, rows, I)
    d = torch.randn((rows, I), generator=gen(4), device="cuda")
    dg, du, _ = moe.moe_swiglu_checkpoint_backward(d, ck)
    f = lambda a, b: d.double() * (a * torch.sigmoid(a) * b)
    eps = 1e-5                                        # differences: eps^2 * third derivative, about 1e-10
    assert torch.allclose((f(g + eps, u) - f(g - eps, u)) / (2 * eps), dg.double(), rtol=1e-5, atol=1e-5)
    assert torch.allclose((f(g, u + eps) - f(g, u - eps)) / (2 * eps), du.double(), rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("end", [0, 1, 37, 64, 65, -3])
def test_checkpoint_leaves_rows_behind_the_last_expert(end):
    """Rows from offsets[E] on keep what h, the checkpoint and the gradients held."""
    rows, I = 64, 40
    do = min(max(end, 0), rows)
    off = torch.tensor([0, min(end, 1), end], dtype=torch.int32, device="cuda")
    gu = pairs(rows, I, BF16, 6, "spread")
    h = torch.full((rows, I), -7.0, dtype=BF16, device="cuda")
    ck = torch.full((moe.moe_swiglu_checkpoint_size(rows, I),), 0x55, dtype=torch.uint8, device="cuda")
    moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:], off, h=h, ckpt=ck)
    full_h, full = moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:])
    assert torch.equal(h[:do], full_h[:do]) and torch.all(h[do:] == -7)
    got, want = (moe.swiglu_checkpoint_views(c, rows, I) for c in (ck, full))
    for n in got:
        assert torch.equal(got[n].view(torch.uint8)[:do], want[n].view(torch.uint8)[:do])
        assert torch.all(got[n].view(torch.uint8)[do:] == 0x55)
    d = torch.randn((rows, I), generator=gen(7), device="cuda").to(BF16)
    outs = [torch.full((rows, I), -7.0, dtype=BF16, device="cuda") for _ in range(3)]
    moe.moe_swiglu_checkpoint_backward(d, full, off, grad_g=outs[0], grad_u=outs[1], h=outs[2])
    for got, want in zip(outs, moe.moe_swiglu_checkpoint_backward(d, full)):
        assert torch.equal(got[:do], want[:do]) and torch.all(got[do:] == -7)


def test_checkpoint_beyond_2_31_elements():
    rows, I = 150_000, 14_400
    gu = torch.empty((rows, 2 * I), dtype=BF16, device="cuda")
    g = gen(8)
    for s in range(0, rows, 10_000):
        gu[s:s + 10_000] = torch.randn((10_000, 2 * I), generator=g, device="cuda")
    h, ck = moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:])
    dg, du, h2 = moe.moe_swiglu_checkpoint_backward(h, ck)
    v = moe.swiglu_checkpoint_views(ck, rows, I)
    for s in (slice(0, 64), slice(149_100, 149_164), slice(rows - 64, rows)):
        one_h, one = moe.moe_swiglu_checkpoint(gu[s, :I], gu[s, I:])
        w = moe.swiglu_checkpoint_views(one, 64, I)
        assert torch.equal(h[s], one_h)
        assert all(torch.equal(v[n].view(torch.uint8)[s], w[n].view(torch.uint8)) for n in v)
        for x, y in zip((dg, du, h2), moe.moe_swiglu_checkpoint_backward(h[s], one)):
            assert torch.equal(x[s], y)


# ------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_layer_and_its_backward(dtype):
    """Routing, dispatch, the stacked gate/up product, the activation with its checkpoint, the down
    product and the combine; then the whole backward, against the same chain in 64 bits on the values
    the checkpoint holds."""
    T, H, I, E, k = 150, 72, 104, 8, 2
    g = gen(20)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)
    x, gy = rnd(T, H), rnd(T, H)
    gate_up, down = rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5)
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[:, 5] = -50.0                              # an expert without rows
    idx, wt = moe.moe_route(logits, k, True)
    d = moe.moe_dispatch(idx, x, E)
    off, xd = d["offsets"], d["x_disp"]
    gu = moe.moe_grouped_gemm(xd, off, gate_up)
    h, ck = moe.moe_swiglu_checkpoint(gu[:, :I], gu[:, I:], off)
    out = moe.moe_grouped_gemm(h, off, down, out_dtype=F32)
    y = moe.moe_combine(out, wt, d["row_of"], dtype=dtype)
    # backward
    gout, _ = moe.moe_combine_backward(out, wt, d["row_of"], gy)
    gh = moe.moe_grouped_gemm(gout, off, down, transposed=True)
    dg, du, h8 = moe.moe_swiglu_checkpoint_backward(gh, ck, off)
    both = dg.as_strided((T * k, 2 * I), (2 * I, 1))  # the two halves are one stacked matrix
    gdown = moe.moe_grouped_gemm_weight_grad(gout, h8, off)
    ggu = moe.moe_grouped_gemm_weight_grad(both, xd, off)
    gxd = moe.moe_grouped_gemm(both, off, gate_up, transposed=True)
    gx = moe.moe_dispatch_backward(gxd, d["row_of"], T, k)
    torch.cuda.synchronize()
    # 64 bits
    D = lambda t: t.double()
    row_of, src = d["row_of"].long(), d["src_of"].long()
    expert = torch.bucketize(torch.arange(T * k, device="cuda"), off[1:].long(), right=True)
    xr = D(x)[src // k]
    rgu = torch.einsum("rh,rnh->rn", xr, D(gate_up)[expert])
    rh = rgu[:, :I] * torch.sigmoid(rgu[:, :I]) * rgu[:, I:]
    rout = torch.einsum("ri,rhi->rh", rh, D(down)[expert])
    ry = (rout[row_of].view(T, k, H) * D(wt).unsqueeze(-1)).sum(1)
    rgo = torch.zeros_like(rout)
    rgo[row_of] = (D(wt).unsqueeze(-1) * D(gy).unsqueeze(1)).view(T * k, H)
    rgh = torch.einsum("rh,rhi->ri", rgo, D(down)[expert])
    g8, u8 = loaded(ck, T * k, I)
    rdg, rdu, rh8 = backward_ref(rgh, g8, u8)
    rboth = torch.cat([rdg, rdu], 1)
    onehot = torch.nn.functional.one_hot(expert, E).double()
    rgdown = torch.einsum("re,rh,ri->ehi", onehot, rgo, rh8)
    rggu = torch.einsum("re,rn,rh->enh", onehot, rboth, xr)
    rgxd = torch.einsum("rn,rnh->rh", rboth, D(gate_up)[expert])
    rgx = rgxd[row_of].view(T, k, H).sum(1)
    # each stage rounds to the dtype once (half a step, relative, of values of either sign): at most
    # six stages deep, so 6 steps of the tensor's own scale bound the error of a sum with random signs
    step = torch.finfo(dtype).eps if dtype != F32 else 2.0 ** -18
    for name, got, ref in (("y", y, ry), ("grad_down", gdown, rgdown), ("grad_gate_up", ggu, rggu),
                           ("grad_x", gx, rgx)):
        scale = ref.abs().max()
        assert torch.isfinite(got).all()
        assert float((got.double() - ref).abs().max() / scale) < 6 * step, name
    assert torch.all(gdown[5] == 0) and torch.all(ggu[5] == 0)
    # the checkpoint is near the products it was made from: half a step of e4m3
    for v8, v in ((g8, D(gu)[:, :I]), (u8, D(gu)[:, I:])):
        s = (v8 - v).abs() - v.abs() * 2.0 ** -4
        block = v.abs().amax(1, keepdim=True) / 448 * 2 * 2.0 ** -10
        assert torch.all(s <= block)


def test_another_device_is_refused_or_served():
    """With a second GPU the calls run on their tensors' device; a stream of another is refused."""
    if torch.cuda.device_count() < 2:
        a = torch.zeros((4, 16), dtype=BF16, device="cuda")
        off = offsets_of([4])
        w = torch.zeros((1, 8, 16), dtype=BF16)
        with pytest.raises(ValueError):
            moe.moe_grouped_gemm(a, off, w)           # weights on the host
        with pytest.raises(ValueError):
            moe.moe_grouped_gemm(a, off.cpu(), w.cuda())
        return
    a = torch.randn((4, 16), device="cuda:1").to(BF16)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda:1")
    w = torch.randn((1, 8, 16), device="cuda:1").to(BF16)
    out = moe.moe_grouped_gemm(a, off, w)
    assert torch.allclose(out.float(), a.float() @ w[0].float().T, atol=0.2)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(a, off, w, stream=torch.cuda.Stream("cuda:0"))
