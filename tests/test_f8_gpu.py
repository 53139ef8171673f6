"""Experts in 8 bits on the GPU, against plain implementations.

Tolerances. The quantized rows and matrices are exact: every code and scale equals
the definition's FP32 operations (one division per block, one product per value, one
rounding). SwiGLU's h is a dozen FP32 operations, within 16 * 2^-23 of itself plus
2^-21 * (1 + |g|) for the 16-bit types' fast exponential; a code is then off by half
an e4m3 step: 2^-4 of the value, 2^-10 of the scale where it is subnormal, and 2^-22
of the value for the two roundings before. A product's inner FP32 sums of 128 exact
terms lose at most 128 * 2^-23 of the terms' magnitudes, the outer one a 2^-23 per
block, and the scales' product and its use 2 more; the output is then rounded once.
"""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
B = 128


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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


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
    over = torch.where(fine, (got - ref).abs() - bound, torch.full_like(ref, -1.0))
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {got.flatten()[i]:.6e} for {ref.flatten()[i]:.6e}, allowed "
                             f"{bound.flatten()[i]:.3e} off, at {i}; {int((over > 0).sum())} of {over.numel()}")


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32, device="cuda")


def up(n):
    return (n + B - 1) // B


def encode(x):
    """Codes (as bytes) and scales of [..., values of a block], FP32 on the CPU."""
    x = x.float().cpu()
    finite = torch.isfinite(x)
    m = torch.where(finite, x.abs(), torch.zeros(())).amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    q = (x * (torch.tensor(448.0) / m)).clamp(-448, 448)
    q = torch.where(finite, q, torch.full((), float("nan"))).to(F8)
    return q, (m / torch.tensor(448.0)).squeeze(-1)


def ref_rows(x):
    rows, K = x.shape
    p = torch.zeros((rows, up(K) * B), dtype=torch.float32)
    p[:, :K] = x.float().cpu()
    q, s = encode(p.view(rows, -1, B))
    return q.view(rows, -1)[:, :K], s


def same_codes(got, ref):
    """Equal values, NaN where the reference has it (of either sign)."""
    a, b = got.cpu().float(), ref.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a.nan_to_num(0), b.nan_to_num(0))


def values(rows, cols, dtype, seed, case):
    g = gen(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    if case == "spread":
        x *= torch.exp(2 * torch.randn((1, cols), generator=g, device="cuda"))
    if case == "small":
        x *= 2.0 ** -12 if dtype == F16 else 2.0 ** -110
    if case == "large":
        x *= 2.0 ** 13 if dtype == F16 else 2.0 ** 125
        x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
    if case == "zeros":
        x *= torch.rand((rows, cols), generator=g, device="cuda") < 0.01
    if case == "ties":                  # scale 1/4: values halfway between codes
        x = torch.randint(-1792, 1792, (rows, cols), generator=g, device="cuda").float() / 16
        x[:, ::B] = 112.0
    if case == "nan":
        for v in ("nan", "inf", "-inf"):
            x[torch.rand((rows, cols), generator=g, device="cuda") < 0.05] = float(v)
    return x.to(dtype)


SIZES = [(1, 1), (5, 7), (3, 16), (2, 127), (4, 128), (9, 129), (1, 100), (33, 264), (130, 1408), (7, 2047)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("case", ["spread", "small", "large", "zeros", "ties", "nan"])
def test_quantize_rows(dtype, rows, K, case):
    x = values(rows, K, dtype, rows * 31 + K, case)
    q, s = ref_rows(x)
    for pad, cpad in ((0, 0), (3, 1), (8, 8), (16, 0)):
        whole = torch.full((rows, K + pad), float("nan"), dtype=dtype, device="cuda")
        whole[:, :K] = x
        room = torch.full((rows + 2, K + cpad), 99, dtype=torch.uint8, device="cuda")
        codes, scales = moe.moe_quantize_rows(whole[:, :K], codes=room.view(F8)[1:rows + 1, :K])
        same_codes(codes, q)
        assert torch.equal(scales.cpu(), s)
        assert torch.all(room[0] == 99) and torch.all(room[-1] == 99) and torch.all(room[:, K:] == 99)
    codes, scales = moe.moe_quantize_rows(x)
    same_codes(codes, q)
    assert codes.dtype == F8 and codes.is_contiguous() and scales.shape == (rows, up(K))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 127, 16), (1, 128, 128), (3, 129, 136), (2, 40, 300),
                                   (5, 260, 513), (64, 72, 8)])
@pytest.mark.parametrize("case", ["spread", "small", "nan"])
def test_quantize_weights(dtype, E, N, K, case):
    w = values(E * N, K, dtype, E + N + K, case).view(E, N, K)
    codes, scales = moe.moe_quantize_weights(w)
    p = torch.zeros((E, up(N) * B, up(K) * B))
    p[:, :N, :K] = w.float().cpu()
    p = p.view(E, up(N), B, up(K), B).transpose(2, 3).reshape(E, up(N), up(K), B * B)
    q, s = encode(p)
    q = q.view(torch.uint8).view(E, up(N), up(K), B, B).transpose(2, 3).reshape(E, up(N) * B, -1)
    same_codes(codes, q[:, :N, :K].contiguous().view(F8))
    assert torch.equal(scales.cpu(), s)


def test_quantized_value_is_near():
    """code * scale is within half an e4m3 step of the value."""
    x = values(64, 1000, F32, 3, "spread")
    codes, scales = moe.moe_quantize_rows(x)
    s = scales.double().repeat_interleave(B, 1)[:, :1000]
    err = (codes.double() * s - x.double()).abs()
    assert torch.all(err <= torch.maximum(x.double().abs() * (2.0 ** -4 + 2.0 ** -22), s * 2.0 ** -10 * (1 + 2.0 ** -20)))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,I", SIZES)
@pytest.mark.parametrize("case", ["spread", "small", "zeros", "deep"])
def test_swiglu_quantize(dtype, rows, I, case):
    gu = values(rows, 2 * I, dtype, rows * 17 + I, case)
    if case == "deep":                 # gates whose sigmoid leaves FP32's normal range
        gu[:, :I] = (-85 + 30 * gu[:, :I].float().clamp(-0.9, 0.9)).to(dtype)
        gu[:, I:] *= 1000
    for g, u in ((gu[:, :I], gu[:, I:]), (gu[:, :I].contiguous(), gu[:, I:].contiguous())):
        codes, scales = moe.moe_swiglu_quantize(g, u)
        gd, ud = g.double(), u.double()
        h = gd * torch.sigmoid(gd) * ud
        rel = 16 * 2.0 ** -23 + (0 if dtype == F32 else 1) * 2.0 ** -21 * (1 + gd.abs())
        # a sigmoid below 2^-126 may count as 0, and so may an h
        slack = h.abs() * rel + 2.0 ** -126 * (1 + (gd * ud).abs())
        p = torch.zeros((rows, up(I) * B), dtype=torch.float64, device="cuda")
        p[:, :I] = h.abs()
        m = p.view(rows, -1, B).amax(-1).clamp(min=2.0 ** -100)
        p[:, :I] = slack
        ms = p.view(rows, -1, B).amax(-1)
        assert torch.all((scales.double() * 448 - m).abs() <= ms + m * 2.0 ** -23)
        s = scales.double().repeat_interleave(B, 1)[:, :I]
        err = (codes.double() * s - h).abs()
        top = h.abs() + slack
        assert torch.all(err <= slack + torch.maximum(top * (2.0 ** -4 + 2.0 ** -21), s * 2.0 ** -10 * 1.001))


def test_swiglu_quantize_nan_and_rows_behind_the_last_expert():
    g, u = torch.ones((40, 200), device="cuda"), torch.ones((40, 200), device="cuda")
    g[3, 5], u[4, 150], u[5, 0] = float("nan"), float("inf"), float("-inf")
    off = torch.tensor([0, 10, 23], dtype=torch.int32, device="cuda")
    for call, args in ((moe.moe_swiglu_quantize, (g, u)), (moe.moe_quantize_rows, (g * u,))):
        codes = torch.full((40, 200), 0x55, dtype=torch.uint8, device="cuda").view(F8)
        scales = torch.full((40, 2), -7.0, device="cuda")
        call(*args, off, codes=codes, scales=scales)
        c = codes.float()
        bad = torch.zeros((40, 200), dtype=torch.bool, device="cuda")
        bad[3, 5] = bad[4, 150] = bad[5, 0] = True
        assert torch.equal(torch.isnan(c), bad)
        assert torch.all(c[:23][~bad[:23]] == 448)
        assert torch.all(codes.view(torch.uint8)[23:] == 0x55) and torch.all(scales[23:] == -7)
        for end in (-3, 0, 40, 99):                   # a negative end is 0, one past the rows is all
            codes.view(torch.uint8).fill_(0x55)
            call(*args, torch.tensor([0, end], dtype=torch.int32, device="cuda"), codes=codes, scales=scales)
            n = min(max(end, 0), 40)
            assert torch.all(codes.view(torch.uint8)[n:] == 0x55)
            assert not torch.any(codes.view(torch.uint8)[:n] == 0x55)


def test_no_rows():
    codes, scales = moe.moe_quantize_rows(torch.empty((0, 64), dtype=BF16, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 1)
    w, ws = torch.zeros((2, 16, 64), device="cuda").to(F8), torch.ones((2, 1, 1), device="cuda")
    out = moe.moe_grouped_gemm_f8(codes, scales, torch.zeros(3, dtype=torch.int32, device="cuda"), w, ws)
    assert out.shape == (0, 16)


# ------------------------------------------------------------------ the product

def operands(rows, E, N, K, transposed, seed, pad=0):
    g = gen(seed)
    whole = torch.full((rows, K + pad), 0x7f, dtype=torch.uint8, device="cuda").view(F8)     # NaN between rows
    whole[:, :K] = (torch.randn((rows, K), generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
    a = whole[:, :K]
    sa = torch.exp(torch.randn((rows, up(K)), generator=g, device="cuda")) * 0.01
    r, c = (K, N) if transposed else (N, K)
    w = (torch.randn((E, r, c), generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)
    sw = torch.exp(torch.randn((E, up(r), up(c)), generator=g, device="cuda")) * 0.01
    return a, sa, w, sw


def dequantized(q, s):
    """[..., N, K] in 64 bits."""
    N, K = q.shape[-2:]
    s = s.double()
    return q.double() * s.repeat_interleave(B, -2)[..., :N, :].repeat_interleave(B, -1)[..., :K]


def dequantized_rows(q, s):
    return q.double() * s.double().repeat_interleave(B, 1)[:, :q.shape[1]]


def ref_product(a, sa, off, w, sw, transposed):
    x = dequantized_rows(a, sa)
    out = torch.zeros((a.shape[0], w.shape[2 if transposed else 1]), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    at = off.tolist()
    for e in range(len(at) - 1):
        s = slice(at[e], at[e + 1])
        m = dequantized(w[e], sw[e])
        m = m if transposed else m.T
        out[s] = x[s] @ m
        size[s] = x[s].abs() @ m.abs()
    return out, size


def slack_of(size, K):
    return size * (B + up(K) + 3) * 2.0 ** -23


COUNTS = {
    "one_row": [1],
    "one_of_many": [0, 0, 1, 0],
    "edges": [0, 15, 16, 17, 0, 31, 32, 33],
    "tiles": [63, 64, 65, 127, 0, 128, 129],
    "wide": [255, 0, 256, 257, 1, 300],
    "long": [700, 3, 1025],
    "empty": [0, 0, 0],
}
SHAPES = [(16, 16, False), (16, 16, True), (80, 48, True), (130, 144, False), (1, 64, False),
          (250, 320, False), (256, 192, True), (272, 1008, True), (520, 128, False), (128, 256, True)]


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("N,K,transposed", SHAPES)
def test_product(counts, N, K, transposed):
    c = COUNTS[counts]
    first, rows, E = 3, 3 + sum(c) + 5, len(c)       # rows of no expert before and behind
    off = offsets_of(c, first)
    a, sa, w, sw = operands(rows, E, N, K, transposed, N + K + len(c), pad=16)
    a.view(torch.uint8)[:first] = 0x7f
    sa[first + sum(c):] = float("nan")
    ref, size = ref_product(a, sa, off, w, sw, transposed)
    s = slice(first, first + sum(c))
    for out_dtype in (BF16, F16, F32):
        for pad in (0, 3, 8):
            whole = torch.full((rows, N + pad), -7.0, dtype=out_dtype, device="cuda")
            out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out=whole[:, :N])
            assert torch.all(whole[:first] == -7) and torch.all(whole[first + sum(c):] == -7)
            assert torch.all(whole[:, N:] == -7)
            check(out[s], ref[s], slack_of(size[s], K), out_dtype, f"{out_dtype} pad {pad}")


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [64], [65], [16, 1, 0, 40], [130]])
@pytest.mark.parametrize("N,K,transposed", [(8, 528, False), (16, 4112, True), (130, 2048, False),
                                            (250, 4096, False), (256, 1040, True), (1000, 1024, False),
                                            (1, 7168, False), (1040, 2064, True)])
def test_product_of_few_rows_over_a_long_k(counts, N, K, transposed):
    off = offsets_of(counts)
    a, sa, w, sw = operands(sum(counts), len(counts), N, K, transposed, N + K)
    ref, size = ref_product(a, sa, off, w, sw, transposed)
    for out_dtype in (BF16, F32):
        out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=out_dtype)
        check(out, ref, slack_of(size, K), out_dtype, str(out_dtype))


@pytest.mark.parametrize("E,rows,N,K,transposed", [(8, 4000, 2000, 1024, False), (64, 3001, 704, 512, True),
                                                   (256, 1024, 512, 1152, False), (16, 2048, 1500, 2048, False)])
def test_product_of_many_units(E, rows, N, K, transposed):
    counts = np.random.RandomState(E).multinomial(rows, np.random.RandomState(1).dirichlet(np.ones(E)))
    off = offsets_of(counts)
    a, sa, w, sw = operands(rows, E, N, K, transposed, E)
    ref, size = ref_product(a, sa, off, w, sw, transposed)
    for out_dtype in (BF16, F32):
        out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=out_dtype)
        check(out, ref, slack_of(size, K), out_dtype, str(out_dtype))
        again = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=out_dtype)
        assert torch.equal(out, again)                # bit-reproducible


@pytest.mark.parametrize("transposed", [False, True])
def test_small_integers_come_out_exactly(transposed):
    """Integers whose sums stay below 2^24, scales of powers of two: no rounding anywhere."""
    rows, E, N, K = 300, 2, 144, 400
    g = gen(1)
    a = torch.randint(-8, 9, (rows, K), generator=g, device="cuda").float().to(F8)
    w = torch.randint(-8, 9, (E, K, N) if transposed else (E, N, K), generator=g, device="cuda").float().to(F8)
    sa = torch.exp2(torch.randint(-2, 3, (rows, up(K)), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 3, (E, up(w.shape[1]), up(w.shape[2])), generator=g, device="cuda").float())
    for counts in ([100, 200], [7, 5]):
        off = offsets_of(counts)
        ref, _ = ref_product(a, sa, off, w, sw, transposed)
        out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=F32)
        assert torch.equal(out[:sum(counts)].double(), ref[:sum(counts)])


def test_nan_stays_in_its_row_and_column():
    rows, E, N, K = 70, 1, 140, 256
    off = offsets_of([rows])
    a, sa, w, sw = operands(rows, E, N, K, False, 4)
    a.view(torch.uint8)[5, 200] = 0x7f
    w.view(torch.uint8)[0, 7, 0] = 0xff
    sa[9, 1] = float("inf")
    out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, out_dtype=F32)
    bad = torch.zeros((rows, N), dtype=torch.bool, device="cuda")
    bad[5] = True
    bad[:, 7] = True
    fine = torch.isfinite(out)
    assert torch.all(~fine[bad]) and torch.all(~fine[9])
    bad[9] = True
    assert torch.all(fine[~bad])


def test_bad_offsets_are_refused_per_expert():
    a, sa, w, sw = operands(60, 3, 32, 64, False, 2)
    off = torch.tensor([0, 40, 20, 60], dtype=torch.int32, device="cuda")      # only the first has rows
    out = torch.full((60, 32), -7.0, dtype=F32, device="cuda")
    moe.moe_grouped_gemm_f8(a, sa, off, w, sw, out=out)
    torch.cuda.synchronize()
    assert moe.moe_device_status(clear=True) == 9
    ref, size = ref_product(a[:40], sa[:40], offsets_of([40]), w[:1], sw[:1], False)
    check(out[:40], ref, slack_of(size, 64), F32, "first expert")
    assert torch.all(out[40:] == -7)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_layer_in_8_bits_and_its_backward(dtype):
    """dispatch -> quantize -> product -> swiglu -> product -> combine, each step within its
    tolerance of 64 bits from the same inputs; then the input gradient through the same codes."""
    T, k, E, H, I = 50, 2, 4, 272, 144
    g = gen(11)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    logits = torch.randn((T, E), generator=g, device="cuda")
    gate_up = (torch.randn((E, 2 * I, H), generator=g, device="cuda") * H ** -0.5).to(dtype)
    down = (torch.randn((E, H, I), generator=g, device="cuda") * I ** -0.5).to(dtype)
    wq, ws = moe.moe_quantize_weights(gate_up)
    dq, ds = moe.moe_quantize_weights(down)
    idx, wt = moe.moe_route(logits, k, True)
    d = moe.moe_dispatch(idx, x, E)
    off = d["offsets"]
    xq, xs = moe.moe_quantize_rows(d["x_disp"], off)
    gu = moe.moe_grouped_gemm_f8(xq, xs, off, wq, ws, out_dtype=dtype)
    ref, size = ref_product(xq, xs, off, wq, ws, False)
    check(gu, ref, slack_of(size, H), dtype, "gate and up")
    hq, hs = moe.moe_swiglu_quantize(gu[:, :I], gu[:, I:], off)
    out = moe.moe_grouped_gemm_f8(hq, hs, off, dq, ds, out_dtype=F32)
    ref, size = ref_product(hq, hs, off, dq, ds, False)
    check(out, ref, slack_of(size, I), F32, "down")
    y = moe.moe_combine(out, wt, d["row_of"], dtype=dtype)
    rows = out.double()[d["row_of"].long()].view(T, k, H)
    terms = wt.double().unsqueeze(-1) * rows
    check(y, terms.sum(1), terms.abs().sum(1) * (k + 1) * 2.0 ** -23, dtype, "combine")
    # the layer as a whole against unquantized 64 bits: three roundings to e4m3 (x, h and the
    # weights, 2^-4 each at most, of random sign) on sums of hundreds of terms
    X, GU, D = d["x_disp"].double(), gate_up.double(), down.double()
    at = off.tolist()
    full = torch.zeros_like(out, dtype=torch.float64)
    for e in range(E):
        s = slice(at[e], at[e + 1])
        v = X[s] @ GU[e].T
        full[s] = (v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]) @ D[e].T
    assert (out.double() - full).norm() < 0.1 * full.norm()
    # backward of down and of gate and up: the same codes, read the other way
    gy = torch.randn(out.shape, generator=g, device="cuda").to(dtype)
    gq, gs = moe.moe_quantize_rows(gy, off)
    gh = moe.moe_grouped_gemm_f8(gq, gs, off, dq, ds, transposed=True, out_dtype=dtype)
    ref, size = ref_product(gq, gs, off, dq, ds, True)
    check(gh, ref, slack_of(size, H), dtype, "gradient of h")
    # against differences: the product is linear, so its gradient along a direction is the
    # product of the direction
    v = torch.randn((off[-1].item(), I), generator=g, device="cuda").to(dtype)
    vq, vs = moe.moe_quantize_rows(v, off)
    along = moe.moe_grouped_gemm_f8(vq, vs, off, dq, ds, out_dtype=F32)
    left = (dequantized_rows(gq, gs) * along.double()).sum()
    gh32 = moe.moe_grouped_gemm_f8(gq, gs, off, dq, ds, transposed=True, out_dtype=F32)
    right = (gh32.double() * dequantized_rows(vq, vs)).sum()
    _, sz = ref_product(vq, vs, off, dq, ds, False)
    room = (dequantized_rows(gq, gs).abs() * sz).sum() * 2 * (B + 6) * 2.0 ** -23
    assert (left - right).abs() <= room


def test_streams_graphs_and_overlapping_calls():
    rows, E, N, K = 500, 4, 400, 512
    off = offsets_of([100, 0, 150, 250])
    x = torch.randn((rows, K), generator=gen(1), device="cuda").to(BF16)
    w = torch.randn((E, N, K), generator=gen(2), device="cuda").to(BF16)

    def call(stream=None):
        xq, xs = moe.moe_quantize_rows(x, off, stream=stream)
        wq, ws = moe.moe_quantize_weights(w, stream=stream)
        gu = moe.moe_grouped_gemm_f8(xq, xs, off, wq, ws, stream=stream)
        hq, hs = moe.moe_swiglu_quantize(gu[:, :N // 2], gu[:, N // 2:], off, stream=stream)
        return xq, xs, wq, ws, gu, hq, hs
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [call(s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for t in r:
        t.view(torch.uint8).zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r, want))
    x.copy_(x.flip(0))                                # the graph reads its inputs anew
    graph.replay()
    again = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r, again))


def test_rows_behind_2_gib():
    """Offsets that pass 31 bits: the last rows of codes and outputs beyond 2^31 bytes."""
    rows, K, N = 150000, 14336 + 16, 64
    x = torch.zeros((rows, K), dtype=BF16, device="cuda")
    x[-3:] = torch.randn((3, K), generator=gen(5), device="cuda").to(BF16)
    codes, scales = moe.moe_quantize_rows(x)
    q, s = ref_rows(x[-3:])
    same_codes(codes[-3:], q)
    assert torch.equal(scales[-3:].cpu(), s)
    w, sw = operands(1, 2, N, K, False, 3)[2:]
    off = torch.tensor([0, 10, rows], dtype=torch.int32, device="cuda")
    whole = torch.zeros((rows, 16384), dtype=BF16, device="cuda")
    out = moe.moe_grouped_gemm_f8(codes, scales, off, w, sw, out=whole[:, :N])
    ref, size = ref_product(codes[-3:], scales[-3:], offsets_of([3]), w[1:], sw[1:], False)
    check(out[-3:], ref, slack_of(size, K), BF16, "last rows")
    assert torch.all(out[:-3] == 0) and torch.all(whole[:, N:] == 0)


# Three forms by sizes: a cluster shares k, few rows per expert, many.
FORMS = {"split": (1, 40, 144, 528), "few_rows": (64, 1300, 400, 528), "many_rows": (8, 1700, 1504, 528)}


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("case", ["small", "large", "zeros", "subnormal"])
def test_products_of_scales_outside_fp32s_range(form, transposed, case):
    """A block's contribution may be an ordinary number where the product of its two
    scales alone is below FP32's normal numbers or above its largest. Beside the usual
    slack, each block's use rounds to a multiple of 2^-149."""
    E, rows, N, K = FORMS[form]
    off = offsets_of(np.random.RandomState(3).multinomial(rows, np.ones(E) / E))
    a, sa, w, sw = operands(rows, E, N, K, transposed, 17)
    third = torch.arange(rows, device="cuda").view(-1, 1) % 3     # lanes of a warp differ
    pick = lambda *p: torch.tensor(p, dtype=torch.float64, device="cuda")[third]
    if case == "small":                # 2^-140 and less; sums of 2^-120
        sw *= 2.0 ** -63
        sa = (sa.double() * pick(2.0 ** 60, 2.0 ** -63, 2.0 ** -30)).float()
    elif case == "large":              # 2^129 to 2^131; codes of a few 2^-9: sums of a block below 2^-7
        a, w = (a.float() * 2.0 ** -13).to(F8), (w.float() * 2.0 ** -14).to(F8)
        sw = (1 + torch.rand(sw.shape, generator=gen(5), device="cuda")) * 2.0 ** 64
        sa = ((1 + torch.rand(sa.shape, generator=gen(6), device="cuda")).double() * pick(2.0 ** 65, 2.0 ** -60, 2.0 ** 40)).float()
    elif case == "zeros":              # blocks of zero codes under scales whose product is 2^150
        zero = (torch.arange(rows, device="cuda").view(-1, 1) + torch.arange(up(K), device="cuda")) % 2 == 0
        a = torch.where(zero.repeat_interleave(B, 1)[:, :K], torch.zeros((), device="cuda"), a.float()).to(F8)
        sa = torch.where(zero, sa * 2.0 ** 96, sa * 2.0 ** -54)
        sw *= 2.0 ** 67
    else:                              # scales that are subnormal or 0
        sa = (sa.double() * pick(2.0 ** -136, 0.0, 1.0)).float()
        sw *= 2.0 ** 100
    ref, size = ref_product(a, sa, off, w, sw, transposed)
    assert torch.isfinite(ref).all() and ref.abs().max() < 2.0 ** 126
    for out_dtype in (F32, BF16):
        out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=out_dtype)
        check(out, ref, slack_of(size, K) + (up(K) + 2) * 2.0 ** -149, out_dtype, f"{case} {out_dtype}")


@pytest.mark.parametrize("form", sorted(FORMS))
def test_scales_that_are_not_finite(form):
    """Infinite and NaN scales as FP32 arithmetic has them: a NaN scale, and an infinite
    one over a block of zeros, make the row NaN, an infinite one over other sums an
    infinity or NaN; other rows stay as they were."""
    E, rows, N, K = FORMS[form]
    off = offsets_of(np.random.RandomState(3).multinomial(rows, np.ones(E) / E))
    a, sa, w, sw = operands(rows, E, N, K, False, 18)
    want = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, out_dtype=F32)
    a.view(torch.uint8)[7, B:2 * B] = 0
    sa[3, 2], sa[7, 1], sa[11, 0] = float("nan"), float("inf"), float("-inf")
    got = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, out_dtype=F32)
    assert torch.isnan(got[3]).all() and torch.isnan(got[7]).all() and not torch.isfinite(got[11]).any()
    same = torch.ones(rows, dtype=torch.bool, device="cuda")
    same[[3, 7, 11]] = False
    assert torch.equal(got[same], want[same])


# At least 64 rows per expert: ten and more units per pair of CTAs, with one round of
# staged scales per unit (K up to 512), two and more.
@pytest.mark.parametrize("K", [16, 64, 128, 400, 512, 528, 1040])
@pytest.mark.parametrize("N,transposed", [(3000, False), (2992, True)])
@pytest.mark.parametrize("E", [16, 61])
def test_many_units_of_experts_of_many_rows(E, N, K, transposed):
    rows = 16384
    r = np.random.RandomState(E + K)
    counts = r.multinomial(rows - E, r.dirichlet(np.ones(E)))
    counts[0], counts[1] = counts[0] + counts[1], 0        # one without rows
    first = 5
    off = offsets_of(counts, first)
    a, sa, w, sw = operands(rows, E, N, K, transposed, E + N + K, pad=16)
    sa *= 0.25                                             # F16 outputs stay finite
    s = slice(first, first + int(counts.sum()))
    ref, size = ref_product(a, sa, off, w, sw, transposed)
    for out_dtype in (BF16, F16, F32):
        whole = torch.full((rows, N + 8), -7.0, dtype=out_dtype, device="cuda")
        out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out=whole[:, :N])
        check(out[s], ref[s], slack_of(size[s], K), out_dtype, str(out_dtype))
        assert torch.all(whole[:first] == -7) and torch.all(whole[s.stop:] == -7) and torch.all(whole[:, N:] == -7)
        again = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=out_dtype)
        assert torch.equal(out[s], again[s])               # bit-reproducible


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("E,rows,N,K", [(16, 16384, 2992, 400), (16, 16384, 2992, 128), (256, 6000, 2000, 400)])
def test_small_integers_over_many_units(E, rows, N, K, transposed):
    """As test_small_integers_come_out_exactly, with many units per CTA in both forms."""
    g = gen(2)
    a = torch.randint(-8, 9, (rows, K), generator=g, device="cuda").float().to(F8)
    w = torch.randint(-8, 9, (E, K, N) if transposed else (E, N, K), generator=g, device="cuda").float().to(F8)
    sa = torch.exp2(torch.randint(-2, 3, (rows, up(K)), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 3, (E, up(w.shape[1]), up(w.shape[2])), generator=g, device="cuda").float())
    off = offsets_of(np.random.RandomState(E).multinomial(rows, np.ones(E) / E))
    ref, _ = ref_product(a, sa, off, w, sw, transposed)
    out = moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, out_dtype=F32)
    assert torch.equal(out.double(), ref)


@pytest.mark.parametrize("transposed", [False, True])
def test_many_units_on_streams_and_in_graphs(transposed):
    """Overlapping, captured and replayed products of more than one unit per CTA, a long
    and a short k in turn."""
    E, rows, N = 16, 16384, 2992
    off = offsets_of(np.random.RandomState(4).multinomial(rows, np.ones(E) / E))
    sets = [operands(rows, E, N, K, transposed, K) for K in (128, 528)]

    def call(stream=None):
        return [moe.moe_grouped_gemm_f8(a, sa, off, w, sw, transposed=transposed, stream=stream)
                for a, sa, w, sw in sets]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    got = [call(s) for s in [torch.cuda.Stream() for _ in range(3)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for _ in range(3):
        for t in r:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r, want))
