"""Experts with 8-bit weights and activations, and the whole layer for a few
tokens, as measured cases.

A user who serves (or trains) large experts keeps their matrices in 8-bit
floating point with a scale for each block of 128, and a decode step of a few
tokens wants the layer in one call that does nothing but read the weights it
needs:

  rows     blocks of 128 columns of a row share the FP32 scale s = m / 448, m the
           block's largest magnitude (2^-100 at least); each value is kept as
           value / s rounded to e4m3
  weights  the same over blocks of 128 x 128 of each expert's matrix
  swiglu   h = SiLU(g) u, kept as `rows` keeps its input
  product  out[r, n] = sum over blocks b of K of
           sa[r, b] sw[e, n / 128, b] (sum over k in b of a[r, k] w[e][n, k])
           for the rows r of expert e (or w[e][k, n], the scales of whose blocks
           are [E, K / 128, N / 128])
  few      T <= 32 tokens: FP32 softmax of the logits, the top_k experts (ties to
           the lower id), their probabilities in the logits' type, and
           y = sum over the k experts of weight * Wd (SiLU(Wg x) * (Wu x)), with
           weights in x's type or in codes and block scales
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # the dispatched rows of a decode batch of 128 tokens, before the first product
        dict(name="rows_decode", op="rows", rows=1024, K=7168, dtype="bf16"),
        # the many-expert layer's matrices, after an optimizer step
        dict(name="weights_fine", op="weights", E=64, N=1408, K=2048, dtype="bf16"),
        # the activation of the many-expert layer on one stacked gate/up product
        dict(name="swiglu_fine", op="swiglu", rows=24576, I=1408, stacked=True, dtype="bf16"),
        # the activation of the few-expert layer, an odd number of rows
        dict(name="swiglu_coarse", op="swiglu", rows=32767, I=14336, stacked=False, dtype="bf16"),
        # a decode batch of 128 tokens on 256 experts, popular ones and idle ones
        dict(name="product_decode", op="product", T=128, top_k=8, E=256, N=2048, K=7168,
             transposed=False, spread="zipf", out="bf16"),
        # prefill of many small experts: 384 rows each on average
        dict(name="product_fine", op="product", T=4096, top_k=6, E=64, N=1408, K=2048,
             transposed=False, spread="even", out="bf16"),
        # prefill of a few large experts, up projection
        dict(name="product_coarse", op="product", T=16384, top_k=2, E=8, N=14336, K=4096,
             transposed=False, spread="normal", out="bf16"),
        # the input gradient of the many-expert layer, an odd number of tokens, FP32
        dict(name="product_fine_input_grad", op="product", T=4099, top_k=6, E=64, N=2048, K=1408,
             transposed=True, spread="even", out="f32"),
        # one token of the many-expert layer
        dict(name="few_one_token", op="few", T=1, top_k=6, E=64, H=2048, I=1408, renormalize=False,
             dtype="bf16", weights="plain", logits="bf16"),
        # eight sequences decoding on 256 experts
        dict(name="few_decode", op="few", T=8, top_k=8, E=256, H=7168, I=2048, renormalize=True,
             dtype="bf16", weights="plain", logits="f32"),
        # the same with 8-bit weights
        dict(name="few_decode_f8", op="few", T=8, top_k=8, E=256, H=7168, I=2048, renormalize=True,
             dtype="bf16", weights="f8", logits="f32"),
        # the small all-FP32 layer
        dict(name="few_tiny_f32", op="few", T=5, top_k=2, E=8, H=128, I=256, renormalize=True,
             dtype="f32", weights="plain", logits="f32"),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi, step):
    return max(step, _log_between(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["rows", "weights", "swiglu", "product", "product", "few", "few", "few"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "rows":
            c = dict(op=op, rows=_log_between(rng, 1, 32768), K=_log_between(rng, 16, 14336), dtype=dtype)
            if rng.random() < 0.6:
                c["K"] = max(16, c["K"] // 16 * 16)
            if c["rows"] * c["K"] <= 2 ** 27:
                return c
        elif op == "weights":
            c = dict(op=op, E=rng.choice([1, 2, 8, 16, 64]), N=_log_between(rng, 64, 14336),
                     K=_log_between(rng, 64, 14336), dtype=dtype)
            if rng.random() < 0.6:
                c["N"], c["K"] = max(16, c["N"] // 16 * 16), max(16, c["K"] // 16 * 16)
            if c["E"] * c["N"] * c["K"] <= 2 ** 28:
                return c
        elif op == "swiglu":
            c = dict(op=op, rows=_log_between(rng, 1, 32768), I=_log_between(rng, 16, 14336),
                     stacked=rng.random() < 0.5, dtype=dtype)
            if rng.random() < 0.6:
                c["I"] = max(16, c["I"] // 16 * 16)
            if c["rows"] * c["I"] <= 2 ** 27:
                return c
        elif op == "product":
            c = dict(op=op, T=_log_between(rng, 1, 16384), top_k=rng.randint(1, 8),
                     E=rng.choice([8, 16, 32, 64, 128, 256]), N=_dim(rng, 64, 14336, 16),
                     K=_dim(rng, 64, 14336, 16), transposed=rng.random() < 0.4,
                     spread=rng.choice(["even", "normal", "zipf"]),
                     out=rng.choice(["bf16", "bf16", "f16", "f32"]))
            if not c["transposed"] and rng.random() < 0.3:
                c["N"] += rng.randint(1, 15)
            rows, size = c["T"] * c["top_k"], c["N"] * c["K"]
            # no more than the largest listed case; the plain form's FP32 weights
            # and padded batch stay within a few GB too
            if 2 * rows * size > 3.5e12 or c["E"] * size > 3.8e9:
                continue
            if c["E"] * c["T"] * (c["N"] + c["K"]) > 8e9:
                continue
            return c
        else:
            weights = rng.choice(["plain", "f8"])
            if weights == "f8" and dtype == "f32":
                dtype = "bf16"
            E = rng.choice([8, 16, 32, 64, 128, 256])
            c = dict(op=op, T=_log_between(rng, 1, 32), top_k=rng.randint(1, 8), E=E,
                     H=_dim(rng, 64, 7168, 16), I=_dim(rng, 64, 14336, 16),
                     renormalize=rng.random() < 0.5, dtype=dtype, weights=weights,
                     logits=rng.choice(["f32", "bf16", "f16"]))
            if E * c["H"] * c["I"] > (1e9 if dtype == "f32" else 3.8e9):
                continue
            # no more weight passes than eight tokens of the 256-expert layer make
            if c["T"] * c["top_k"] * c["H"] * c["I"] > 9.5e8:
                continue
            return c


def _counts(case, seed):
    """How many rows the router gives each expert (int64 [E])."""
    r = np.random.RandomState(seed % (1 << 31))
    T, E = case["T"], case["E"]
    logits = r.standard_normal((T, E)).astype(np.float32)
    if case["spread"] == "normal":
        logits += math.sqrt(0.5) * r.standard_normal(E).astype(np.float32)
    elif case["spread"] == "zipf":
        logits -= 1.1 * np.log(r.permutation(E) + 1).astype(np.float32)
    picked = np.argpartition(-logits, case["top_k"] - 1, axis=1)[:, :case["top_k"]]
    return np.bincount(picked.reshape(-1), minlength=E)


def _normal(shape, g, dtype, std=1.0, limit=None):
    """N(0, std^2) values, drawn slab by slab so that a large tensor needs no FP32 copy."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    per = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for s in range(0, shape[0], per):
        v = torch.randn((min(per, shape[0] - s),) + tuple(shape[1:]), generator=g, device="cuda")
        if std != 1.0:
            v.mul_(std)
        out[s:s + per] = v if limit is None else v.clamp_(-limit, limit)
    return out


def _ceil(n):
    return -(-n // BLOCK)


def _codes(shape, g):
    """Codes of a normal matrix whose blocks' largest values land near e4m3's largest."""
    return _normal(shape, g, F8, 100.0, 448.0)


def _matrix_scales(E, N, K, std, g):
    """Scales of such a matrix's blocks: any positive FP32 numbers, as a checkpoint brings them."""
    s = torch.rand((E, _ceil(N), _ceil(K)), generator=g, device="cuda")
    return (0.7 + 0.6 * s) * (std / 100.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "product":
        counts = _counts(case, seed)
        rows, E, N, K = int(counts.sum()), case["E"], case["N"], case["K"]
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        st["most"] = int(counts.max())
        st["a"] = _codes((rows, K), g)
        # a row's blocks differ by a factor of a few
        st["a_scales"] = torch.randn((rows, _ceil(K)), generator=g, device="cuda").mul_(0.5).exp_().mul_(0.01)
        if case["transposed"]:
            st["w"] = _codes((E, K, N), g)
            st["w_scales"] = _matrix_scales(E, K, N, K ** -0.5, g)
        else:
            st["w"] = _codes((E, N, K), g)
            st["w_scales"] = _matrix_scales(E, N, K, K ** -0.5, g)
        return st
    dt = DTYPES[case["dtype"]]
    if op == "rows":
        # some columns carry much larger values than others
        spread = torch.randn((case["K"],), generator=g, device="cuda").mul_(0.7).exp_()
        st["x"] = (_normal((case["rows"], case["K"]), g, torch.float32) * spread).to(dt)
    elif op == "weights":
        st["w"] = _normal((case["E"], case["N"], case["K"]), g, dt, case["K"] ** -0.5)
    elif op == "swiglu":
        rows, I = case["rows"], case["I"]
        spread = torch.randn((2 * I,), generator=g, device="cuda").mul_(0.7).exp_()
        gu = torch.empty((rows, 2 * I), dtype=dt, device="cuda")
        for s in range(0, rows, 4096):
            gu[s:s + 4096] = torch.randn(gu[s:s + 4096].shape, generator=g, device="cuda") * spread
        st["g"], st["u"] = ((gu[:, :I], gu[:, I:]) if case["stacked"]
                            else (gu[:, :I].contiguous(), gu[:, I:].contiguous()))
    else:
        T, E, H, I = (case[k] for k in ("T", "E", "H", "I"))
        st["x"] = _normal((T, H), g, dt)
        st["logits"] = _normal((T, E), g, DTYPES[case["logits"]])
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            if case["weights"] == "f8":
                st[name] = _codes((E, N, K), g)
                st[name + "_scales"] = _matrix_scales(E, N, K, K ** -0.5, g)
            else:
                st[name] = _normal((E, N, K), g, dt, K ** -0.5)
                st[name + "_scales"] = None
    return st


# ------------------------------------------------------------------ the plain forms

def _store(x):
    """Codes and scales of [..., blocks, values of a block] in FP32."""
    top = x.abs().amax(-1).clamp(min=2.0 ** -100)
    q = (x * (448 / top).unsqueeze(-1)).clamp(-448, 448).to(F8)
    return q, top / 448


def _store_rows(v):
    rows, K = v.shape
    x = torch.zeros((rows, _ceil(K) * BLOCK), dtype=torch.float32, device=v.device)
    x[:, :K] = v
    q, s = _store(x.view(rows, -1, BLOCK))
    return q.view(rows, -1)[:, :K], s


def _store_matrices(w):
    E, N, K = w.shape
    n, k = _ceil(N), _ceil(K)
    x = torch.zeros((E, n * BLOCK, k * BLOCK), dtype=torch.float32, device=w.device)
    x[:, :N, :K] = w
    x = x.view(E, n, BLOCK, k, BLOCK).transpose(2, 3).reshape(E, n, k, BLOCK * BLOCK)
    q, s = _store(x)
    q = q.view(E, n, k, BLOCK, BLOCK).view(torch.uint8).transpose(2, 3).reshape(E, n * BLOCK, k * BLOCK)
    return q[:, :N, :K].contiguous().view(F8), s


def _load_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _load_matrices(q, s):
    """FP32 matrices of codes [..., N, K] and scales [..., N / 128, K / 128]."""
    N, K = q.shape[-2:]
    s = s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return q.float() * s


def _padded(x, expert, place, E, most):
    """The rows as a batch of E matrices, FP32, with zeros behind each expert's rows."""
    out = torch.zeros((E, most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[expert, place] = x
    return out


def _places(offsets, rows):
    r = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    expert = torch.searchsorted(offsets[1:], r, right=True)
    return expert, (r - offsets[expert]).long()


def _select(codes, scales, ids):
    """FP32 matrices of the experts `ids`."""
    if scales is None:
        return codes[ids].float()
    return _load_matrices(codes.view(torch.uint8)[ids].view(F8), scales[ids])


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rows":
        q, s = _store_rows(st["x"])
        return {"codes": q, "scales": s}
    if op == "weights":
        q, s = _store_matrices(st["w"])
        return {"codes": q, "scales": s}
    if op == "swiglu":
        g, u = st["g"].float(), st["u"].float()
        q, s = _store_rows(g / (1 + torch.exp(-g)) * u)
        return {"codes": q, "scales": s}
    if op == "product":
        expert, place = _places(st["offsets"], st["a"].shape[0])
        pa = _padded(_load_rows(st["a"], st["a_scales"]), expert, place, case["E"], st["most"])
        w = _load_matrices(st["w"], st["w_scales"])
        out = torch.bmm(pa, w if case["transposed"] else w.transpose(1, 2))
        return {"out": out[expert, place].to(DTYPES[case["out"]])}
    x, k = st["x"].float(), case["top_k"]
    p = torch.exp(st["logits"].float() - st["logits"].float().amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    order = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k]
    wt = torch.gather(p, 1, order)
    if case["renormalize"]:
        wt = wt / wt.sum(1, keepdim=True)
    wt = wt.to(st["logits"].dtype).float()
    y = torch.zeros_like(x)
    for j in range(k):
        ids = order[:, j]
        g = torch.bmm(_select(st["gate"], st["gate_scales"], ids), x.unsqueeze(2)).squeeze(2)
        u = torch.bmm(_select(st["up"], st["up_scales"], ids), x.unsqueeze(2)).squeeze(2)
        h = g / (1 + torch.exp(-g)) * u
        d = torch.bmm(_select(st["down"], st["down_scales"], ids), h.unsqueeze(2)).squeeze(2)
        y = y + wt[:, j:j + 1] * d
    return {"y": y.to(st["x"].dtype)}


def run(state):
    if not own:
        return _plain(state)
    import mixture_experts_ffn_topk_gb300 as moe
    case = state["case"]
    op = case["op"]
    if op == "rows":
        codes, scales = moe.moe_quantize_rows(state["x"])
        return {"codes": codes, "scales": scales}
    if op == "weights":
        codes, scales = moe.moe_quantize_weights(state["w"])
        return {"codes": codes, "scales": scales}
    if op == "swiglu":
        codes, scales = moe.moe_swiglu_quantize(state["g"], state["u"])
        return {"codes": codes, "scales": scales}
    if op == "product":
        return {"out": moe.moe_grouped_gemm_f8(state["a"], state["a_scales"], state["offsets"],
                                               state["w"], state["w_scales"],
                                               transposed=case["transposed"],
                                               out_dtype=DTYPES[case["out"]])}
    return {"y": moe.moe_forward_few(state["x"], state["logits"], state["gate"], state["up"],
                                     state["down"], case["top_k"], case["renormalize"],
                                     gate_scales=state["gate_scales"], up_scales=state["up_scales"],
                                     down_scales=state["down_scales"])}


def _touched(case):
    """Experts that T tokens of even routing meet, on average."""
    return case["E"] * (1 - (1 - case["top_k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    if op == "product":
        counts = _counts(case, 0)
        rows, touched = int(counts.sum()), int((counts > 0).sum())
        N, K = case["N"], case["K"]
        # the matrices of experts without rows are not read
        b = (rows * (K + 4 * _ceil(K)) + touched * (N * K + 4 * _ceil(N) * _ceil(K)) +
             rows * N * DTYPES[case["out"]].itemsize + 4 * (case["E"] + 1))
        return {"bytes": b, "flops": 2 * rows * N * K}
    es = DTYPES[case["dtype"]].itemsize
    if op == "rows":
        n = case["rows"] * case["K"]
        return {"bytes": n * (es + 1) + 4 * case["rows"] * _ceil(case["K"]), "flops": 3 * n}
    if op == "weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": n * (es + 1) + 4 * case["E"] * _ceil(case["N"]) * _ceil(case["K"]), "flops": 3 * n}
    if op == "swiglu":
        n = case["rows"] * case["I"]
        return {"bytes": n * (2 * es + 1) + 4 * case["rows"] * _ceil(case["I"]), "flops": 10 * n}
    T, H, I, E = (case[k] for k in ("T", "H", "I", "E"))
    ws = 1 + 4 / BLOCK ** 2 if case["weights"] == "f8" else es
    return {"bytes": int(_touched(case) * 3 * H * I * ws) + 2 * T * H * es +
            T * E * DTYPES[case["logits"]].itemsize,
            "flops": 6 * T * case["top_k"] * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_store(x):
    """e4m3 values and scales of [..., blocks, values], from the definition: rounding to
    multiples of the step of the value's binade (half to even)."""
    scale = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 448
    x = x / scale
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448), scale.squeeze(-1)


def _exact_rows(part, rows, K):
    """Of a matrix whose rows [s, t) in 64 bits are part(s, t)."""
    B = _ceil(K)
    codes = torch.empty((rows, K), dtype=torch.float64, device="cuda")
    scales = torch.empty((rows, B), dtype=torch.float64, device="cuda")
    per = max(1, (1 << 24) // (B * BLOCK))
    for s in range(0, rows, per):
        t = min(rows, s + per)
        x = torch.zeros((t - s, B * BLOCK), dtype=torch.float64, device="cuda")
        x[:, :K] = part(s, t)
        q, scales[s:t] = _exact_store(x.view(t - s, B, BLOCK))
        codes[s:t] = q.view(t - s, -1)[:, :K]
    return {"codes": codes, "scales": scales}


def _value_of_codes():
    """The value of every e4m3 byte: sign, exponent with bias 7, three bits of fraction."""
    b = torch.arange(256, device="cuda")
    ex, fr = (b >> 3) & 15, (b & 7).double()
    value = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * torch.exp2(ex.double() - 7))
    value = torch.where(b >= 128, -value, value)
    value[127] = value[255] = float("nan")
    return value


def _exact_matrix(q, s, table):
    """One matrix in 64 bits."""
    if s is None:
        return q.double()
    n, k = torch.arange(q.shape[0], device="cuda") // BLOCK, torch.arange(q.shape[1], device="cuda") // BLOCK
    return table[q.view(torch.uint8).long()] * s.double()[n][:, k]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        return _exact_rows(lambda s, t: st["x"][s:t].double(), case["rows"], case["K"])
    if op == "swiglu":
        def part(s, t):
            g = st["g"][s:t].double()
            return g * torch.sigmoid(g) * st["u"][s:t].double()
        return _exact_rows(part, case["rows"], case["I"])
    if op == "weights":
        E, N, K = st["w"].shape
        n, k = _ceil(N), _ceil(K)
        codes = torch.empty((E, N, K), dtype=torch.float64, device="cuda")
        scales = torch.empty((E, n, k), dtype=torch.float64, device="cuda")
        for e in range(E):
            for i in range(n):
                rows = slice(i * BLOCK, min(N, (i + 1) * BLOCK))
                x = torch.zeros((BLOCK, k * BLOCK), dtype=torch.float64, device="cuda")
                x[:rows.stop - rows.start, :K] = st["w"][e, rows].double()
                q, scales[e, i] = _exact_store(x.view(BLOCK, k, BLOCK).transpose(0, 1).reshape(k, -1))
                q = q.view(k, BLOCK, BLOCK).transpose(0, 1).reshape(BLOCK, -1)
                codes[e, rows] = q[:rows.stop - rows.start, :K]
        return {"codes": codes, "scales": scales}
    table = _value_of_codes()
    if op == "product":
        at, a = st["offsets"].tolist(), st["a"]
        if 2 * a.shape[0] * case["N"] * case["K"] > 5e12:
            return None
        out = torch.empty((a.shape[0], case["N"]), dtype=torch.float64, device="cuda")
        col = torch.arange(case["K"], device="cuda") // BLOCK
        for e in range(case["E"]):
            if at[e + 1] == at[e]:
                continue
            s = slice(at[e], at[e + 1])
            w = _exact_matrix(st["w"][e], st["w_scales"][e], table)
            x = table[a[s].view(torch.uint8).long()] * st["a_scales"][s].double()[:, col]
            out[s] = x @ (w if case["transposed"] else w.T)
        return {"out": out}
    x, logits = st["x"].double(), st["logits"].double()
    p = torch.softmax(logits, 1)
    y = torch.zeros_like(x)
    for t in range(case["T"]):
        row = logits[t].tolist()
        ids = sorted(range(case["E"]), key=lambda e: (-row[e], e))[:case["top_k"]]
        wt = p[t, ids]
        if case["renormalize"]:
            wt = wt / wt.sum()
        # routing weights are of the logits' type
        wt = wt.to(st["logits"].dtype).double()
        for j, e in enumerate(ids):
            m = [_exact_matrix(st[n][e], None if st[n + "_scales"] is None else st[n + "_scales"][e], table)
                 for n in ("gate", "up", "down")]
            g = m[0] @ x[t]
            y[t] += wt[j] * (m[2] @ (g * torch.sigmoid(g) * (m[1] @ x[t])))
    return {"y": y}
