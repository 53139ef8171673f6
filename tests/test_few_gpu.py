"""The few-token forward on the GPU, against a plain implementation in 64 bits.

Tolerances, per element. An FP32 sum of n products is off by at most (n + 2) * 2^-23 of
the terms' magnitudes, in any order. So g and u are off by (H + 2) 2^-23 sum|x w|; h by
what those bring (|SiLU'| <= 1.1) and 2^-20 of itself, then half a step of its type;
an expert's output by that through |Wd|, and (I + 2) 2^-23 of its own terms; y by the
k weighted ones and (k + 2) 2^-23 of them, and half a step. Softmax weights are off by
(E + 16) 2^-23 of themselves, and half a step of the logits' type.
"""

import numpy as np
import pytest
import torch

import mixture_experts_ffn_topk_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
B = 128
U = 2.0 ** -23


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
    if "bad_index" not in request.node.name:
        assert moe.moe_device_status(clear=True) == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def up_(n):
    return (n + B - 1) // B


class Layer:
    def __init__(self, E, H, I, dtype, f8, seed):
        g = gen(seed)
        self.E, self.H, self.I, self.dtype = E, H, I, dtype
        self.q, self.s, self.m = [], [], []
        for N, K in ((I, H), (I, H), (H, I)):
            w = torch.randn((E, N, K), generator=g, device="cuda")
            if f8:
                q = (w * 100).clamp(-448, 448).to(F8)
                s = torch.exp(0.5 * torch.randn((E, up_(N), up_(K)), generator=g, device="cuda")) * 0.01 * K ** -0.5
                self.m.append(q.double() * s.double().repeat_interleave(B, 1)[:, :N].repeat_interleave(B, 2)[..., :K])
            else:
                q, s = (w * K ** -0.5).to(dtype), None
                self.m.append(q.double())
            self.q.append(q)
            self.s.append(s)

    def scales(self):
        return dict(zip(("gate_scales", "up_scales", "down_scales"), self.s))

    def few(self, x, logits, k, renorm, **kw):
        return moe.moe_forward_few(x, logits, *self.q, k, renorm, **self.scales(), **kw)

    def routed(self, x, idx, w, **kw):
        return moe.moe_forward_few_routed(x, idx, w, *self.q, **self.scales(), **kw)

    def ref(self, x, ids, w, w_slack):
        """y and its slack: ids [T, k] (-1: no expert), w [T, k] and w_slack in 64 bits."""
        T, k = ids.shape
        y = torch.zeros((T, self.H), dtype=torch.float64, device="cuda")
        slack = torch.zeros_like(y)
        half = torch.finfo(self.dtype).eps / 2
        least = torch.finfo(self.dtype).tiny * half
        for t in range(T):
            size = torch.zeros(self.H, dtype=torch.float64, device="cuda")
            for j in range(k):
                e = int(ids[t, j])
                if e < 0:
                    y[t] = float("nan")
                    continue
                v = x[t].double()
                G, Up, D = (m[e] for m in self.m)
                g, u = G @ v, Up @ v
                eg, eu = ((m.abs() @ v.abs()) * (self.H + 2) * U for m in (G, Up))
                silu = g * torch.sigmoid(g)
                h = silu * u
                eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + h.abs() * 2.0 ** -20
                eh = eh + (h.abs() + eh) * half + least
                o = D @ h
                terms = D.abs() @ h.abs()
                eo = D.abs() @ eh + terms * (self.I + 2) * U
                y[t] += w[t, j] * o
                slack[t] += w[t, j].abs() * eo + w_slack[t, j] * (o.abs() + eo)
                size += w[t, j].abs() * o.abs()
            slack[t] += size * (k + 2) * U
        return y, slack


def check(got, ref, slack, dtype):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN in other places"
    f = torch.finfo(dtype)
    bound = slack + (ref.abs() + slack) * (f.eps / 2) + f.tiny * f.eps / 2
    over = torch.where(torch.isfinite(ref), (got - ref).abs() - bound, torch.full_like(ref, -1.0))
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{got.flatten()[i]:.6e} for {ref.flatten()[i]:.6e}, allowed {bound.flatten()[i]:.3e} "
                             f"off, at {i}; {int((over > 0).sum())} of {over.numel()}")


def softmax_routing(logits, k, renorm):
    """ids (by logit, lower id first), weights and their slack, in 64 bits."""
    l = logits.double()
    order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.gather(torch.softmax(l, 1), 1, order)
    if renorm:
        p = p / p.sum(1, keepdim=True)
    f = torch.finfo(logits.dtype)
    return order, p, p * ((logits.shape[1] + 16) * U + f.eps / 2) + f.tiny * f.eps / 2


KINDS = [(BF16, False), (F16, False), (F32, False), (BF16, True), (F16, True)]


@pytest.mark.parametrize("dtype,f8", KINDS)
@pytest.mark.parametrize("T,k,E,H,I,ldt", [
    (1, 1, 1, 16, 16, F32), (1, 2, 8, 128, 256, F32), (2, 6, 64, 272, 144, BF16), (5, 2, 8, 128, 256, F16),
    (7, 3, 5, 48, 1040, F32), (8, 8, 8, 512, 64, F32), (9, 1, 2, 160, 96, F32), (16, 4, 16, 256, 128, BF16),
    (17, 2, 3, 2048, 32, F32), (32, 8, 40, 144, 272, F32), (32, 2, 2, 96, 80, F16), (3, 32, 48, 64, 128, F32),
    (32, 32, 32, 32, 48, F32), (4, 2, 300, 64, 64, F32), (2, 3, 1000, 32, 32, BF16), (1, 8, 256, 1024, 512, F32)])
def test_forward_few(dtype, f8, T, k, E, H, I, ldt):
    L = Layer(E, H, I, dtype, f8, T + E + H)
    g = gen(I)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    logits = (2 * torch.randn((T, E), generator=g, device="cuda")).to(ldt)
    for renorm in (False, True):
        ids, w, ws = softmax_routing(logits, k, renorm)
        y, slack = L.ref(x, ids, w, ws)
        got = L.few(x, logits, k, renorm)
        check(got, y, slack, dtype)
        assert torch.equal(got, L.few(x, logits, k, renorm))       # bit-reproducible
        # the routed form on moe_route's result
        idx, wt = moe.moe_route(logits, k, renorm)
        assert torch.equal(idx.long(), ids)
        y, slack = L.ref(x, ids, wt.double(), torch.zeros_like(w))
        check(L.routed(x, idx, wt), y, slack, dtype)


@pytest.mark.parametrize("dtype,f8", KINDS)
def test_odd_multiples_and_block_borders(dtype, f8):
    """H and I of every residue of 128 that the type allows, in turn."""
    step = 16 if f8 else 16 // torch.tensor([], dtype=dtype).element_size()
    for i, H in enumerate(range(step, 300, step * 3)):
        I = 300 // step * step - H // step // 2 * step
        L = Layer(3, H, I, dtype, f8, H)
        x = torch.randn((3, H), generator=gen(i), device="cuda").to(dtype)
        logits = torch.randn((3, 3), generator=gen(i + 1), device="cuda")
        ids, w, ws = softmax_routing(logits, 2, True)
        y, slack = L.ref(x, ids, w, ws)
        check(L.few(x, logits, 2, True), y, slack, dtype)


@pytest.mark.parametrize("dtype,f8", KINDS)
def test_outputs_of_the_down_product_in_passes(dtype, f8):
    """1024 pairs: a CTA's outputs do not fit in shared memory at once."""
    T, k, E, H, I = 32, 32, 33, 7168, 32
    L = Layer(E, H, I, dtype, f8, 5)
    x = torch.randn((T, H), generator=gen(6), device="cuda").to(dtype)
    logits = torch.randn((T, E), generator=gen(7), device="cuda")
    ids, w, ws = softmax_routing(logits, k, True)
    y, slack = L.ref(x, ids, w, ws)
    check(L.few(x, logits, k, True), y, slack, dtype)


def test_the_largest_sizes():
    """H and I at their limit."""
    H = I = 65536
    x = torch.randn((2, H), generator=gen(1), device="cuda").to(BF16)
    gate = torch.empty((1, I, H), dtype=BF16, device="cuda").normal_(0, H ** -0.5, generator=gen(2))
    up = torch.empty((1, I, H), dtype=BF16, device="cuda").normal_(0, H ** -0.5, generator=gen(3))
    down = torch.empty((1, H, I), dtype=BF16, device="cuda").normal_(0, I ** -0.5, generator=gen(4))
    y = moe.moe_forward_few(x, torch.zeros((2, 1), device="cuda"), gate, up, down, 1, True)
    # the first and last columns against 64 bits (the products of all rows in FP32 first)
    g, u = x.float() @ gate[0].float().T, x.float() @ up[0].float().T
    h = g * torch.sigmoid(g) * u
    rows = torch.tensor([0, 1, 127, 128, H // 2, H - 2, H - 1], device="cuda")
    D = down[0, rows].double()
    ref = h.double() @ D.T
    # g and u of both sides: (H + 2) 2^-23 of terms of which sum |x w| is about 0.64 sqrt(H)
    size = h.double().abs() @ D.abs().T
    e = (H + 2) * U * 0.7 * H ** 0.5
    slack = size * ((I + 2) * U + 2.0 ** -8) + (e * (1.1 * u.abs() + g.abs() + 1).double()) @ D.abs().T
    check(y[:, rows], ref, slack, BF16)
    assert torch.all(torch.isfinite(y))


def test_ties_and_rows_without_a_softmax():
    E, H, I, k = 12, 64, 64, 3
    L = Layer(E, H, I, BF16, False, 3)
    x = torch.randn((7, H), generator=gen(1), device="cuda").to(BF16)
    logits = torch.randn((7, E), generator=gen(2), device="cuda")
    logits[0] = 0.5                                    # all equal: the lowest ids
    logits[1, 4], logits[1, 9] = 9.0, 9.0
    logits[2] = 0.0
    logits[2, 3:] = -0.0                               # equal to +0
    logits[3, 5] = float("nan")
    logits[4, 5] = float("inf")
    logits[5] = float("-inf")
    logits[6, 2:] = float("-inf")                      # fewer finite logits than top_k: weight 0
    ids, w, ws = softmax_routing(logits, k, False)
    idx, wt = moe.moe_route(logits, k, False)
    assert torch.equal(idx[[0, 1, 2, 6]].long(), ids[[0, 1, 2, 6]])
    for bad in (3, 4, 5):
        ids[bad] = torch.arange(k, device="cuda")
        w[bad] = float("nan")
    y, slack = L.ref(x, ids, w, ws)
    check(L.few(x, logits, k, False), y, slack, BF16)
    assert torch.all(torch.isnan(y[3:6])) and torch.all(torch.isfinite(y[[0, 1, 2, 6]]))


@pytest.mark.parametrize("dtype,f8", KINDS)
def test_an_expert_named_more_than_once(dtype, f8):
    """More pairs of one expert than a chunk has: 32 tokens, both slots on one expert."""
    T, k, E, H, I = 32, 2, 4, 96, 112
    L = Layer(E, H, I, dtype, f8, 5)
    x = torch.randn((T, H), generator=gen(6), device="cuda").to(dtype)
    idx = torch.full((T, k), 2, dtype=torch.int32, device="cuda")
    idx[7, 1] = 0
    w = torch.randn((T, k), generator=gen(7), device="cuda")       # weights of any sign
    y, slack = L.ref(x, idx.long(), w.double(), torch.zeros((T, k), dtype=torch.float64, device="cuda"))
    check(L.routed(x, idx, w), y, slack, dtype)
    for rows in (1, 8, 9, 17):
        check(L.routed(x[:rows], idx[:rows], w[:rows]), y[:rows], slack[:rows], dtype)


def test_bad_index_makes_the_row_nan():
    L = Layer(4, 64, 64, BF16, False, 5)
    x = torch.randn((3, 64), generator=gen(6), device="cuda").to(BF16)
    w = torch.rand((3, 2), generator=gen(7), device="cuda")
    for bad in (4, -1, 1 << 30, 65535, 65536):
        idx = torch.tensor([[0, 3], [bad, 1], [2, 2]], dtype=torch.int32, device="cuda")
        got = L.routed(x, idx, w)
        torch.cuda.synchronize()
        assert moe.moe_device_status(clear=True) == 9
        ids = idx.long()
        ids[1, 0] = -1
        y, slack = L.ref(x, ids, w.double(), torch.zeros((3, 2), dtype=torch.float64, device="cuda"))
        check(got, y, slack, BF16)
    idx = torch.full((3, 2), 9, dtype=torch.int32, device="cuda")
    assert torch.all(torch.isnan(L.routed(x, idx, w)))
    torch.cuda.synchronize()
    assert moe.moe_device_status(clear=True) == 9


@pytest.mark.parametrize("f8", [False, True])
def test_nan_stays_in_its_token(f8):
    """NaN and infinities of one token, and of an expert that only one token meets."""
    L = Layer(6, 128, 128, BF16, f8, 5)
    x = torch.randn((5, 128), generator=gen(6), device="cuda").to(BF16)
    x[1, 5], x[3, 100] = float("nan"), float("inf")
    idx = torch.tensor([[0, 1], [0, 1], [0, 1], [1, 0], [4, 0]], dtype=torch.int32, device="cuda")
    if f8:
        L.q[1].view(torch.uint8)[4, 7, 9] = 0x7f
    else:
        L.q[1][4, 7, 9] = float("nan")
    w = torch.rand((5, 2), generator=gen(7), device="cuda") + 0.1
    got = L.routed(x, idx, w)
    assert torch.equal(torch.isfinite(got).all(1).cpu(), torch.tensor([True, False, True, False, False]))
    assert torch.all(torch.isnan(got[4])) and torch.all(torch.isnan(got[1]))


def test_agrees_with_the_one_call_forward():
    """As moe_forward up to its rounding: the same products, h and combine."""
    L = Layer(16, 512, 256, BF16, False, 9)
    x = torch.randn((20, 512), generator=gen(1), device="cuda").to(BF16)
    logits = torch.randn((20, 16), generator=gen(2), device="cuda")
    a = L.few(x, logits, 4, True).double()
    b = moe.moe_forward(x, logits, *L.q, 4, True).double()
    # h may round the other way (2^-9 of a term, of 256 x 4 terms of random sign), y too
    assert (a - b).abs().max() <= b.abs().max() * 2.0 ** -7


def test_sigmoid_grouped_routing():
    L = Layer(32, 256, 128, F16, False, 9)
    x = torch.randn((6, 256), generator=gen(1), device="cuda").to(F16)
    logits = torch.randn((6, 32), generator=gen(2), device="cuda")
    bias = 0.1 * torch.randn((32,), generator=gen(3), device="cuda")
    idx, w = moe.moe_route_sigmoid_grouped(logits, bias, 4, 8, 4, True, True, 2.5)
    y, slack = L.ref(x, idx.long(), w.double(), torch.zeros((6, 4), dtype=torch.float64, device="cuda"))
    check(L.routed(x, idx, w), y, slack, F16)


def test_no_tokens():
    L = Layer(4, 64, 64, BF16, False, 5)
    y = L.few(torch.empty((0, 64), dtype=BF16, device="cuda"), torch.empty((0, 4), device="cuda"), 2, True)
    assert y.shape == (0, 64)


@pytest.mark.parametrize("dtype,f8", KINDS)
def test_streams_graphs_and_overlapping_calls(dtype, f8):
    L = Layer(16, 512, 384, dtype, f8, 9)
    xs = [torch.randn((n, 512), generator=gen(n), device="cuda").to(dtype) for n in (1, 8, 20)]
    ls = [torch.randn((len(x), 16), generator=gen(len(x) + 50), device="cuda") for x in xs]
    want = [L.few(x, l, 4, True).clone() for x, l in zip(xs, ls)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(5):                                 # back to back and side by side
        for s, x, l in zip(streams, xs, ls):
            got.append(L.few(x, l, 4, True, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
    # a decode loop's steps, each on the last one's output, in a graph
    ws = torch.empty(moe.moe_forward_few_workspace_size(8, 384, 4, dtype), dtype=torch.uint8, device="cuda")
    x0 = xs[1].clone()

    def steps(x):
        for _ in range(4):
            x = L.few(x, ls[1], 4, True, workspace=ws)
        return x
    eager = steps(x0).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = steps(x0)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    x0.copy_(x0.flip(0))
    graph.replay()
    assert torch.equal(out, steps(x0))


def test_outputs_given_and_refused():
    L = Layer(4, 64, 64, BF16, False, 5)
    x = torch.randn((3, 64), generator=gen(6), device="cuda").to(BF16)
    logits = torch.randn((3, 4), generator=gen(7), device="cuda")
    y = torch.full((5, 64), -7.0, dtype=BF16, device="cuda")
    ws = torch.full((3 * 2 * 64 * 2 + 512,), 0x55, dtype=torch.uint8, device="cuda")
    got = L.few(x, logits, 2, False, y=y[1:4], workspace=ws[:1024])
    assert got.data_ptr() == y[1:4].data_ptr()
    assert torch.equal(got, L.few(x, logits, 2, False))
    assert torch.all(y[0] == -7) and torch.all(y[4] == -7) and torch.all(ws[768:] == 0x55)
    with pytest.raises(moe.MoeError):
        L.few(x, logits, 2, False, workspace=ws[:512])
    with pytest.raises(ValueError):
        L.few(x, logits[:2], 2, False)
    with pytest.raises(ValueError):
        moe.moe_forward_few(x, logits, L.q[0], L.q[1], L.q[2].transpose(1, 2), 2, False)
    with pytest.raises(ValueError):
        moe.moe_forward_few(x, logits, *L.q, 2, False, gate_scales=torch.ones((4, 1, 1), device="cuda"))
    with pytest.raises(moe.MoeError):
        L.few(torch.zeros((33, 64), dtype=BF16, device="cuda"), torch.zeros((33, 4), device="cuda"), 2, False)
    with pytest.raises(moe.MoeError):
        L.few(x, logits, 5, False)


# ------------------------------------------------------------------ exact layers

class ExactLayer:
    """A layer in which nothing is rounded before y. x is 1 or 2. A row of gate has eight
    values of 8 (where some fall on one place, of 8, 16 or 32, so that g >= 32 all the
    same): FP32's SiLU(g) is then g itself, as exp(-g) < 2^-25 vanishes beside 1. A row
    of up has eight of +-1. g and u have four bits each (or are a power of two), so that
    h fits the 8 bits of BF16; |h| <= 2048. down is 0 or +-2^-6: an expert's sums are
    whole multiples of 2^-3. 8-bit weights: the same values, as codes times scales of
    2^-2 to 2^2."""

    def __init__(self, E, H, I, dtype, f8, seed):
        g = gen(seed)
        self.E, self.H, self.I, self.dtype = E, H, I, dtype
        kind = F8 if f8 else dtype
        self.q, self.s = [], []
        self.nonzero = []                                 # of gate and up: places and values
        for which, (N, K) in enumerate(((I, H), (I, H), (H, I))):
            r = torch.randint(-2, 3, (E, up_(N), up_(K)), generator=g, device="cuda") if f8 else None
            q = torch.empty((E, N, K), dtype=kind, device="cuda")
            if which < 2:
                at = torch.randint(0, K, (E, N, 8), generator=g, device="cuda").sort(-1).values
                first = torch.ones_like(at, dtype=torch.bool)
                first[..., 1:] = at[..., 1:] != at[..., :-1]
                if which == 0:
                    v = 8.0 * first
                    n = first.sum(-1, keepdim=True)      # x >= 1: g >= 8 n
                    v = v * torch.where(n >= 4, 1.0, torch.where(n >= 2, 2.0, 4.0))
                else:
                    v = torch.where(torch.rand(at.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0) * first
                self.nonzero.append((at, v))
                if f8:
                    e, n = torch.arange(E, device="cuda").view(-1, 1, 1), torch.arange(N, device="cuda").view(1, -1, 1)
                    v = v * torch.exp2(-r[e, n // B, at // B].float())
                for s in range(E):
                    m = torch.zeros((N, K), dtype=torch.float32 if N * K < 1 << 26 else BF16, device="cuda")
                    m.scatter_add_(1, at[s], v[s].to(m.dtype))
                    q[s] = m.to(kind)
            else:
                for s in range(E):
                    for n0 in range(0, N, 4096):
                        n1 = min(N, n0 + 4096)
                        m = torch.randint(-1, 2, (n1 - n0, K), generator=g, device="cuda", dtype=torch.int8).float() * 2.0 ** -6
                        if f8:
                            n, k = torch.arange(n0, n1, device="cuda") // B, torch.arange(K, device="cuda") // B
                            m *= torch.exp2(-r[s][n][:, k].float())
                        q[s, n0:n1] = m.to(kind)
            self.q.append(q)
            self.s.append(torch.exp2(r.float()) if f8 else None)

    def scales(self):
        return dict(zip(("gate_scales", "up_scales", "down_scales"), self.s))

    def x(self, T, seed):
        return torch.randint(1, 3, (T, self.H), generator=gen(seed), device="cuda").to(self.dtype)

    def ref(self, x, ids, w):
        """sum over j of w[t, j] times the expert's output, in 64 bits, before the last rounding."""
        T, k = ids.shape
        h = torch.zeros((T, k, self.I), dtype=torch.float64, device="cuda")
        for t in range(T):
            for j in range(k):
                g, u = ((x[t].double()[at[ids[t, j]]] * v[ids[t, j]].double()).sum(-1) for at, v in self.nonzero)
                assert g.min() >= 32
                h[t, j] = g * u
        assert torch.equal(h, h.to(self.dtype).double())
        y = torch.zeros((T, self.H), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(y)
        w = w.double()
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not t.numel():
                continue
            for n0 in range(0, self.H, 2048):
                m = self.q[2][e, n0:n0 + 2048].double()
                if self.s[2] is not None:
                    s = self.s[2][e].double().repeat_interleave(B, 0)[n0:n0 + m.shape[0]]
                    m = m * s.repeat_interleave(B, 1)[:, :self.I]
                # whole multiples of 2^-3, exact in FP32 in any order of summation
                assert (h[t, j].abs() @ m.abs().T).max() * 8 < 2.0 ** 24
                o = (h[t, j] @ m.T) * w[t, j].unsqueeze(-1)
                y[:, n0:n0 + 2048].index_add_(0, t, o)
                size[:, n0:n0 + 2048].index_add_(0, t, o.abs())
        assert size.max() * 32 < 2.0 ** 24                # and of 2^-5, with weights
        return y


def exact_layer(T, k, E, H, I, dtype, f8, same_expert=False):
    """Compares bit for bit. Routing weights: 2^-2 to 2^1, of either sign."""
    L = ExactLayer(E, H, I, dtype, f8, T + E + H + I)
    x = L.x(T, I)
    g = gen(H)
    ids = (torch.full((T, k), E - 1, device="cuda") if same_expert else
           torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k])
    w = torch.exp2(torch.randint(-2, 2, (T, k), generator=g, device="cuda").float())
    w *= torch.randint(0, 2, (T, k), generator=g, device="cuda") * 2 - 1
    ref = L.ref(x, ids, w)
    got = moe.moe_forward_few_routed(x, ids.int(), w, *L.q, **L.scales())
    assert torch.equal(got, ref.float().to(dtype))
    assert (ref != 0).double().mean() > 0.5               # zeros, or a pair left out, would not pass


@pytest.mark.parametrize("dtype,f8", KINDS)
@pytest.mark.parametrize("T,k,E,H,I", [
    (1, 1, 1, 128, 128), (2, 6, 64, 272, 144), (8, 8, 8, 512, 64), (5, 2, 8, 1024, 512), (7, 3, 5, 48, 1040),
    (17, 2, 3, 2048, 32), (32, 8, 40, 144, 272), (12, 8, 8, 640, 256), (24, 4, 4, 256, 640), (32, 8, 8, 1024, 384),
    (32, 32, 33, 7168, 32), (32, 32, 32, 8192, 64), (32, 16, 17, 16384, 96)])
def test_exact_layers(dtype, f8, T, k, E, H, I):
    """Bit for bit, also where an expert's pairs make several chunks and where a CTA's
    outputs take several passes (the last three)."""
    exact_layer(T, k, E, H, I, dtype, f8)


@pytest.mark.parametrize("dtype,f8", KINDS)
def test_exact_layer_of_one_expert(dtype, f8):
    """64 pairs of one expert: four to eight chunks."""
    exact_layer(32, 2, 3, 1024, 256, dtype, f8, same_expert=True)


@pytest.mark.parametrize("dtype,f8", [(BF16, False), (F32, False), (BF16, True)])
def test_the_largest_sizes_exactly(dtype, f8):
    """H and I at their limit, every output bit for bit."""
    exact_layer(2, 1, 1, 65536, 65536, dtype, f8)
    torch.cuda.empty_cache()
