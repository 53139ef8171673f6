"""Every form that the grouped products and their weight gradients choose by
size, on integers: the sums are exact in FP32 whatever their order, so outputs
have to equal the 64-bit ones, rounded once.
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
