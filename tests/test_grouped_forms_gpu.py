"""Every form that the grouped products and their weight gradients choose by
size, on integers: the sums are exact in FP32 whatever their order, so outputs
have to equal the 64-bit ones, rounded once.
"""

import re

import numpy as np
import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_topk_gb300 import build
    build.build()
    moe.moe_device_status(clear=True)
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert moe.moe_device_status(clear=True) == 0


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32, device="cuda")


def integers(shape, dtype, g, top=3):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    per = max(1, (1 << 26) // max(1, out[0].numel()))
    for s in range(0, shape[0], per):
        out[s:s + per] = torch.randint(-top, top + 1, (min(per, shape[0] - s),) + tuple(shape[1:]),
                                       generator=g, device="cuda").to(dtype)
    return out


def exact_matmul(a, b):
    """a @ b of integers whose sums stay below 2^24: exact in FP32."""
    allow = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        return a.float() @ b.float()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = allow


@pytest.mark.parametrize("counts,N,K,out", [
    ([8192, 33], 8192, 8192, BF16),             # the first foreign rows come after a long expert
    ([96] + [0] * 62 + [96], 4096, 4096, F32),  # loads wait until idle experts' zeros are stored
    ([96] + [0] * 62 + [100], 4096, 4096, F32)])
def test_waits_allow_for_the_launchs_own_work(counts, N, K, out):
    """A wait that only stands behind the launch's own progress does not expire, however short the limit:
    50 us here, where these launches take 0.4 ms and more."""
    g = generator(1)
    off, rows = offsets_of(counts), sum(counts)
    d, a = integers((rows, N), BF16, g), integers((rows, K), BF16, g)
    gw = torch.full((len(counts), N, K), -7.0, dtype=out, device="cuda")
    torch.cuda.synchronize()
    moe.moe_set_wait_limit_ns(50_000)
    try:
        moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=gw)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(0)
    assert moe.moe_device_status(clear=True) == 0
    at = off.tolist()
    for e in (0, 1, len(counts) - 1):
        ref = exact_matmul(d[at[e]:at[e + 1]].T, a[at[e]:at[e + 1]])
        assert torch.equal(gw[e], ref.to(out))


BAD_INDEX = 9


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("offsets,served", [([0, 40, 20, 60], [40, 0, 0]),          # falls, then overlaps
                                            ([0, 40, 20, 60, 70], [40, 0, 0, 10]),  # one behind both is served
                                            ([10, 30, 5, 25, 60, 61], [20, 0, 0, 0, 1]),
                                            ([0, 50, -1, 30, 40, 70], [50, 0, 0, 0, 0])])
def test_offsets_that_name_rows_twice(dtype, offsets, served):
    """Once offsets fall, an expert whose rows begin before an earlier one's end has none either: its rows
    keep what they held, and its gradient is zero."""
    g = generator(2)
    E, rows, N, K = len(offsets) - 1, 70, 72, 64
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    a, d = integers((rows, K), dtype, g), integers((rows, N), dtype, g)
    w = integers((E, N, K), dtype, g)
    out = torch.full((rows, N), -7.0, dtype=dtype, device="cuda")
    want, gw_want = out.clone(), torch.zeros((E, N, K), device="cuda")
    for e, n in enumerate(served):
        s = slice(offsets[e], offsets[e] + n) if n else slice(0, 0)
        want[s] = exact_matmul(a[s], w[e].T).to(dtype)
        gw_want[e] = exact_matmul(d[s].T, a[s])
    moe.moe_grouped_gemm(a, off, w, out=out)
    assert moe.moe_device_status(clear=True) == BAD_INDEX
    assert torch.equal(out, want)
    gw = moe.moe_grouped_gemm_weight_grad(d, a, off)
    assert moe.moe_device_status(clear=True) == BAD_INDEX
    assert torch.equal(gw, gw_want)


# ------------------------------------------------------------ every form

def forms_of(call):
    """The grouped kernels that `call` launches, as (name, template arguments)."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    found = []
    for e in prof.events():
        m = re.search(r"(grouped_gemm|grouped_wgrad|grouped_simt)_kernel<([^>]*)>", e.name)
        if m:
            args = re.sub(r"\((int|bool)\)", "", m.group(2)).replace("true", "1").replace("false", "0")
            found.append((m.group(1), tuple(int(v) for v in args.split(","))))
    return found


@pytest.fixture(scope="module")
def visible(ready):
    """Whether the profiler shows kernels here (its first session may come out empty)."""
    a, w = torch.zeros((4, 16), device="cuda"), torch.zeros((1, 8, 16), device="cuda")
    seen = [forms_of(lambda: moe.moe_grouped_gemm(a, offsets_of([4]), w)) for _ in range(3)]
    return len(seen[-1]) == 1


def check_form(call, visible, name, **want):
    """The call launches one kernel, of this form."""
    names = {"grouped_gemm": ("DT", "CG", "KN", "OUT_F32", "SPLIT", "PARTS"),
             "grouped_wgrad": ("DT", "CG", "OUT_F32", "SPLIT"),
             "grouped_simt": ("WG", "Y_MAJOR", "BM", "BN", "TM", "TN", "BK", "STAGES")}
    if not visible:
        call()
        return
    found = forms_of(call)
    assert [n for n, _ in found] == [name]
    got = dict(zip(names[name], found[0][1]))
    assert {k: got[k] for k in want} == {k: int(v) for k, v in want.items()}


def product_case(counts, N, K, dtype, transposed, seed):
    """Rows of a product with NaN between them and where they belong to no expert."""
    g = generator(seed)
    first, rows, E = 3, sum(counts) + 8, len(counts)
    whole = torch.full((rows, K + 8), float("nan"), dtype=dtype, device="cuda")
    a = whole[:, :K]
    a[first:rows - 5] = integers((rows - 8, K), dtype, g)
    w = integers((E, K, N) if transposed else (E, N, K), dtype, g)
    off = offsets_of(counts, first)
    at = off.tolist()
    ref = torch.cat([exact_matmul(a[at[e]:at[e + 1]], w[e] if transposed else w[e].T) for e in range(E)])
    return a, off, w, slice(first, rows - 5), ref


def check_product(counts, N, K, dtype, out_dtype, transposed, visible, form):
    a, off, w, s, ref = product_case(counts, N, K, dtype, transposed, N + K)
    whole = torch.full((a.shape[0], N + 3), -7.0, dtype=out_dtype, device="cuda")
    call = lambda: moe.moe_grouped_gemm(a, off, w, transposed=transposed, out=whole[:, :N])
    check_form(call, visible, **form)
    assert torch.equal(whole[s, :N], ref.to(out_dtype))
    assert torch.all(whole[:s.start] == -7) and torch.all(whole[s.stop:] == -7) and torch.all(whole[:, N:] == -7)
    # rows of out on 16 bytes
    out = moe.moe_grouped_gemm(a, off, w, transposed=transposed, out_dtype=out_dtype)
    assert torch.equal(out[s], ref.to(out_dtype))


MANY = [300, 0, 513, 64, 700, 129, 255, 1030]             # 16 row units of 256, 28 of 128
FEW = [40, 64, 65, 0, 1, 17, 33, 16, 15, 63, 50, 48, 31, 32, 30, 64, 2, 64, 64, 10, 20, 61, 62, 60]


@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("out", ["16-bit", "F32"])
@pytest.mark.parametrize("dtype", [BF16, F16])
class TestProducts:
    def run(self, visible, counts, N, K, dtype, out, transposed, **form):
        out_dtype = F32 if out == "F32" else dtype
        check_product(counts, N, K, dtype, out_dtype, transposed, visible,
                      dict(name="grouped_gemm", OUT_F32=out == "F32", KN=transposed, **form))

    @pytest.mark.parametrize("K", [72, 200, 832])          # one part, and (F32) two
    def test_pairs_with_several_units_each(self, visible, dtype, out, transposed, K):
        self.run(visible, MANY, 2064, K, dtype, out, transposed, CG=2, SPLIT=0, PARTS=out == "F32" and K > 768)

    def test_pairs_with_odd_rows_of_the_output(self, visible, dtype, out, transposed):
        N = 2064 if transposed else 2059
        self.run(visible, MANY, N, 136, dtype, out, transposed, CG=2, SPLIT=0)

    def test_blocks_of_row_units(self, visible, dtype, out, transposed):
        """More row units of an expert than stay in L2 together: 8 of 256 in blocks of 6, or (F32) 16 of 128
        in blocks of 13."""
        self.run(visible, [2000, 130], 4104, 14336, dtype, out, transposed, CG=2, SPLIT=0, PARTS=out == "F32")

    @pytest.mark.parametrize("K", [136, 776, 1544])
    def test_single_ctas_with_several_units_each(self, visible, dtype, out, transposed, K):
        self.run(visible, FEW, 1032, K, dtype, out, transposed, CG=1, SPLIT=0, PARTS=out == "F32" and K > 768)

    @pytest.mark.parametrize("counts,N,K", [([3, 0, 1], 136, 504), ([3, 0, 1], 136, 520),      # 8 k-blocks, 9
                                            ([64, 2], 264, 1016), ([65], 8, 1032),
                                            ([5], 128, 2040), ([5], 128, 2056), ([64], 136, 2112),
                                            ([1], 72, 6152), ([1, 1], 1032, 1152),
                                            # parts within a slice
                                            ([9, 0, 64], 136, 7168), ([2], 8, 14344)])
    def test_k_shared_by_a_cluster(self, visible, dtype, out, transposed, counts, N, K):
        """k slices that end on and beside blocks of 64, and inside one."""
        self.run(visible, counts, N, K, dtype, out, transposed, CG=1, SPLIT=1, PARTS=0)


@pytest.mark.parametrize("transposed", [False, True], ids=["NK", "KN"])
@pytest.mark.parametrize("counts,N,K,tile", [
    ([9, 0, 33, 1, 40], 264, 136, (16, 128)),
    ([100 + e % 7 for e in range(64)], 264, 72, (64, 128)),
    ([60 * (e % 5) for e in range(64)], 392, 1028, (64, 128)),
    ([100 + e % 7 for e in range(64)], 56, 68, (64, 64)),
    ([64 * (e % 4) + e % 3 for e in range(96)], 64, 516, (64, 64))])
def test_fp32_products(visible, transposed, counts, N, K, tile):
    N += 0 if transposed else -3                           # rows of w need only whole k
    check_product(counts, N, K, F32, F32, transposed, visible,
                  dict(name="grouped_simt", WG=0, Y_MAJOR=transposed, BM=tile[0], BN=tile[1]))


def check_gradient(counts, N, K, dtype, out_dtype, visible, form):
    g = generator(N + K + len(counts))
    first, rows, E = 3, sum(counts) + 8, len(counts)
    off = offsets_of(counts, first)
    d, a = (torch.full((rows, n + 8), float("nan"), dtype=dtype, device="cuda")[:, :n] for n in (N, K))
    for m in (d, a):
        m[first:rows - 5] = integers((rows - 8, m.shape[1]), dtype, g)
    at = off.tolist()
    ref = torch.stack([exact_matmul(d[at[e]:at[e + 1]].T, a[at[e]:at[e + 1]]) for e in range(E)])
    room = torch.full((E + 2, N, K), -7.0, dtype=out_dtype, device="cuda")
    check_form(lambda: moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=room[1:-1]), visible, **form)
    assert torch.equal(room[1:-1], ref.to(out_dtype))
    assert torch.all(room[0] == -7) and torch.all(room[-1] == -7)
    old = integers((E, N, K), out_dtype, g, top=100)
    want = (old.float() + ref).to(out_dtype)
    room[1:-1] = old
    check_form(lambda: moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=room[1:-1], accumulate=True), visible,
               **form)
    assert torch.equal(room[1:-1], want)
    assert torch.all(room[0] == -7) and torch.all(room[-1] == -7)


@pytest.mark.parametrize("out", ["16-bit", "F32"])
@pytest.mark.parametrize("dtype", [BF16, F16])
class TestGradients:
    def run(self, visible, counts, N, K, dtype, out, **form):
        check_gradient(counts, N, K, dtype, F32 if out == "F32" else dtype, visible,
                       dict(name="grouped_wgrad", OUT_F32=out == "F32", **form))

    @pytest.mark.parametrize("counts", [[1500, 777, 0, 30], [1, 2047, 0, 64], [768, 769, 767, 1537]])
    @pytest.mark.parametrize("N,K", [(1096, 1032), (1032, 1096), (520, 2056)])
    def test_pairs(self, visible, dtype, out, counts, N, K):
        self.run(visible, counts, N, K, dtype, out, CG=2, SPLIT=0)

    @pytest.mark.parametrize("counts", [[200] * 7 + [3500] + [200] * 8, [800, 0, 1537, 17] * 3 + [1, 0, 16, 768]])
    @pytest.mark.parametrize("N,K", [(1000, 1032), (392, 520)])
    def test_single_ctas_with_a_long_segment(self, visible, dtype, out, counts, N, K):
        """Under 512 rows on average; (F32) segments of several parts among short and empty ones."""
        counts = counts if sum(counts) < 512 * 16 else [c // 2 for c in counts[:-4]] + [1, 1700, 16, 0]
        self.run(visible, counts, N, K, dtype, out, CG=1, SPLIT=0)

    @pytest.mark.parametrize("counts", [[512], [511], [513], [1024 + 63], [4096 + 1], [2048, 0, 17],
                                        [6145, 15, 700], [0, 8 * 768 + 8]])
    @pytest.mark.parametrize("N,K", [(72, 264), (136, 40)])
    def test_rows_shared_by_a_cluster(self, visible, dtype, out, counts, N, K):
        """Slices of rows that end on and beside blocks of 64, and segments shorter than the cluster."""
        self.run(visible, counts, N, K, dtype, out, CG=1, SPLIT=1)


@pytest.mark.parametrize("counts,N,K,tile", [
    ([9, 0, 33, 1, 40], 264, 136, (16, 128)),
    ([17 * (e % 5) for e in range(64)], 200, 264, (64, 128)),
    ([1500, 0, 31, 700] * 16, 72, 132, (64, 128)),
    ([17 * (e % 5) for e in range(64)], 200, 56, (64, 64)),
    ([33, 0, 800] * 30, 132, 64, (64, 64)),
    ([17 * (e % 5) for e in range(64)], 36, 264, (16, 128))])
def test_fp32_gradients(visible, counts, N, K, tile):
    check_gradient(counts, N, K, F32, F32, visible,
                   dict(name="grouped_simt", WG=1, Y_MAJOR=1, BM=tile[0], BN=tile[1]))
