"""Long sums of the grouped products, against 64 bits at tolerances that do not
grow with the length.

The tensor cores' accumulator truncates: an instruction adds 16 products to the
accumulator, 17 values that may each lose a step of the partial sum, 2^-23 of it
at most. With positive terms of like size the partial sum after j of n
instructions is within a tenth of j / n of the sum, so n instructions lose at
most 17 * 0.55 n * 2^-23 of it. 16-bit outputs are summed in parts of 16384 (F16)
or 32768 (BF16) terms, FP32 outputs in parts of 768, joined by FP32 additions of
2^-24 each: the length of the sum itself enters by those alone.
"""

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


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def positive(shape, dtype, g, along=0, mean=0.03):
    """Values between mean / 2 and 3 mean, drawn slab by slab: of like size but for a factor of 1 to 2
    for each index of dimension `along`, so that sums over the others meet every place of a binade."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    view = [1] * len(shape)
    view[along] = shape[along]
    factor = (torch.rand(view, generator=g, device="cuda") + 1).expand((shape[0],) + tuple(view[1:]))
    per = max(1, (1 << 27) // out[0].numel())
    for s in range(0, shape[0], per):
        v = torch.rand((min(per, shape[0] - s),) + tuple(shape[1:]), generator=g, device="cuda")
        out[s:s + per] = (v + 0.5) * mean * factor[s:s + per]
    return out


def half_step(ref, dtype):
    """Half a step of dtype at ref (positive, normal)."""
    return torch.exp2(torch.floor(torch.log2(ref))) * (torch.finfo(dtype).eps / 2)


def part_slack(n, dtype):
    """Relative error of a sum of n positive terms, before its rounding (8: CTAs joined)."""
    part = {F16: 16384, BF16: 32768, F32: 768}[dtype]
    return (17 * 0.55 * min(n, part) / 16 + -(-n // part) + 8) * 2.0 ** -23


def check_long_sum(got, ref, n, dtype, what):
    slack = ref * part_slack(n, dtype)
    over = (got.double() - ref).abs() - slack - half_step(ref + slack, dtype)
    assert float(over.max()) <= 0, f"{what}: {float((got.double() / ref - 1).mean()):.2e} off on average"


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("counts,N,K", [([3], 40, 1 << 22),            # joined over a cluster
                                        ([640], 1000, 1 << 19),        # pairs
                                        ([40] * 16, 384, 1 << 19)],    # single CTAs
                         ids=["joined", "pairs", "singles"])
def test_16_bit_products_do_not_drift_over_long_k(dtype, counts, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    E, rows, off = len(counts), sum(counts), offsets_of(counts)
    at = off.tolist()
    a, w = positive((rows, K), dtype, g), positive((E, N, K), dtype, g, along=1)
    refs = []
    for e in range(E):
        ref = torch.zeros((counts[e], N), dtype=torch.float64, device="cuda")
        for k in range(0, K, 1 << 16):
            ref += a[at[e]:at[e + 1], k:k + (1 << 16)].double() @ w[e, :, k:k + (1 << 16)].double().T
        refs.append(ref)
    ref = torch.cat(refs)
    check_long_sum(moe.moe_grouped_gemm(a, off, w), ref, K, dtype, "[E, N, K]")
    wt = torch.empty((E, K, N), dtype=dtype, device="cuda")
    for e in range(E):
        wt[e] = w[e].T
    del w
    check_long_sum(moe.moe_grouped_gemm(a, off, wt, transposed=True), ref, K, dtype, "[E, K, N]")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("E,rows,N,K", [(1, 1 << 22, 72, 264),         # joined over a cluster
                                        (1, 1 << 19, 1544, 2048),      # pairs
                                        (1024, 500_000, 72, 72)],      # single CTAs
                         ids=["joined", "pairs", "singles"])
def test_16_bit_weight_gradients_do_not_drift_over_long_segments(dtype, E, rows, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    e = E // 3
    off = offsets_of([0] * e + [rows] + [0] * (E - e - 1))
    d, a = positive((rows, N), dtype, g, along=1), positive((rows, K), dtype, g, along=1)
    some = torch.arange(0, N, max(1, N // 64), device="cuda")
    ref = torch.zeros((some.numel(), K), dtype=torch.float64, device="cuda")
    for r in range(0, rows, 1 << 16):
        ref += d[r:r + (1 << 16)][:, some].double().T @ a[r:r + (1 << 16)].double()
    got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_dtype=dtype)
    check_long_sum(got[e][some], ref, rows, dtype, "gradient")
    assert int(torch.count_nonzero(got[:e])) == 0 and int(torch.count_nonzero(got[e + 1:])) == 0
    old = positive((E, N, K), dtype, g, mean=2000.0)
    kept = old[e][some].double()
    got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=old, accumulate=True)
    slack = ref * part_slack(rows, dtype) + (ref + kept) * 2.0 ** -24
    over = (got[e][some].double() - ref - kept).abs() - slack - half_step(ref + kept + slack, dtype)
    assert float(over.max()) <= 0


def test_fp32_gradients_of_single_ctas_are_added_to_once():
    """Integers, so that every sum up to the last addition is exact: with accumulate, old + sum rounded
    once, for a segment of several parts among short ones (no pairs, nothing joined)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    E, N, K = 16, 1000, 1032
    counts = [200] * E
    counts[5] = 3500
    off = offsets_of(counts)
    at = off.tolist()
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(BF16)
    d, a = ints(at[-1], N), ints(at[-1], K)
    # 2^25 and up: a step of FP32 is 4 there
    old = torch.randint(1 << 23, 1 << 24, (E, N, K), generator=g, device="cuda").float() * 4
    ref = torch.stack([d[at[e]:at[e + 1]].double().T @ a[at[e]:at[e + 1]].double() for e in range(E)])
    assert torch.equal(moe.moe_grouped_gemm_weight_grad(d, a, off).double(), ref)
    got = moe.moe_grouped_gemm_weight_grad(d, a, off, grad_w=old.clone(), accumulate=True)
    wrong = got != (old.double() + ref).float()
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {wrong.numel()} rounded otherwise"
