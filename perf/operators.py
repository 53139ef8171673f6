"""The grouped products and the 8-bit SwiGLU checkpoint, as measured cases.

A user who trains or serves experts that are not the built-in SwiGLU block (a
stacked gate/up projection, an expert without a gate, a backward of their own)
needs the products of a ragged batch with each expert's matrix on their own,
in both directions, and an activation between them that keeps 8 bits per value
for the backward pass instead of the FP32 planes of the training cache:

  product      out[r] = a[r] w[e]^T (w [E, N, K]) or a[r] w[e] (w [E, K, N])
               for the rows r of expert e, offsets[e] <= r < offsets[e + 1]
  weight_grad  grad_w[e] = sum over the expert's rows of grad[r]^T a[r]
  swiglu       h = SiLU(g) u, and a checkpoint of g and u: blocks of 32
               columns share the smallest power of two s = 2^x (-127 <= x <=
               119) for which the block's largest magnitude is at most 448 s;
               each value is kept as value / s rounded to e4m3, the scale as
               the byte x + 127
  swiglu_grad  with g and u read back from the checkpoint, t = 1/(1+exp(-g)):
               grad_g = grad_h u t (1 + g (1 - t)), grad_u = grad_h g t,
               h = g t u

Rows come from a router: each of T tokens picks `top_k` of E experts.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32


def listed():
    return [
        # one token of a 256-expert model meets its eight experts' gate matrices
        dict(name="product_one_token", op="product", T=1, top_k=8, E=256, N=2048, K=7168,
             transposed=False, spread="zipf", dtype="bf16", out="bf16"),
        # a decode batch of 128 tokens on the same model, popular experts and idle ones
        dict(name="product_decode", op="product", T=128, top_k=8, E=256, N=2048, K=7168,
             transposed=False, spread="zipf", dtype="bf16", out="bf16"),
        # prefill of many small experts: 384 rows each on average
        dict(name="product_fine", op="product", T=4096, top_k=6, E=64, N=1408, K=2048,
             transposed=False, spread="even", dtype="bf16", out="bf16"),
        # prefill of a few large experts, up projection
        dict(name="product_coarse", op="product", T=16384, top_k=2, E=8, N=14336, K=4096,
             transposed=False, spread="normal", dtype="bf16", out="bf16"),
        # the input gradient of the many-expert layer, an odd number of tokens, F16
        dict(name="product_fine_input_grad", op="product", T=4099, top_k=6, E=64, N=2048, K=1408,
             transposed=True, spread="even", dtype="f16", out="f16"),
        # the small all-FP32 layer
        dict(name="product_tiny_f32", op="product", T=64, top_k=2, E=8, N=256, K=128,
             transposed=False, spread="even", dtype="f32", out="f32"),
        # weight gradient of the many-expert layer, FP32 as the optimizer takes it
        dict(name="weight_grad_fine", op="weight_grad", T=4096, top_k=6, E=64, N=1408, K=2048,
             spread="even", dtype="bf16", out="f32"),
        # weight gradient of the few-expert layer's down projection, in the weights' type
        dict(name="weight_grad_coarse", op="weight_grad", T=16383, top_k=2, E=8, N=4096, K=14336,
             spread="normal", dtype="bf16", out="bf16"),
        # the activation of the many-expert layer on one stacked gate/up product
        dict(name="swiglu_fine", op="swiglu", rows=24576, I=1408, stacked=True, dtype="bf16"),
        # the activation of the few-expert layer
        dict(name="swiglu_coarse", op="swiglu", rows=32768, I=14336, stacked=False, dtype="bf16"),
        # the backward of a decode-sized micro batch
        dict(name="swiglu_grad_small", op="swiglu_grad", rows=1023, I=2048, stacked=True, dtype="f16"),
        # the backward of the few-expert layer
        dict(name="swiglu_grad_coarse", op="swiglu_grad", rows=32766, I=14336, stacked=True,
             dtype="bf16"),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "weight_grad", "swiglu", "swiglu_grad"])
    if op in ("swiglu", "swiglu_grad"):
        while True:
            c = dict(op=op, rows=_log_between(rng, 1, 32768), I=_log_between(rng, 16, 14336),
                     stacked=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
            if rng.random() < 0.6:
                c["I"] = max(8, c["I"] // 8 * 8)
            if c["dtype"] == "f32" and c["rows"] * c["I"] > 2 ** 27:
                continue
            return c
    while True:
        E = rng.choice([8, 16, 32, 64, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        c = dict(op=op, T=_log_between(rng, 1, 16384), top_k=rng.randint(1, 8), E=E,
                 N=max(8, _log_between(rng, 64, 14336) // 8 * 8),
                 K=max(8, _log_between(rng, 64, 14336) // 8 * 8),
                 spread=rng.choice(["even", "normal", "zipf"]), dtype=dtype,
                 out="f32" if dtype == "f32" or rng.random() < 0.25 else dtype)
        if op == "product":
            c["transposed"] = rng.random() < 0.5
            if not c["transposed"] and rng.random() < 0.3:
                c["N"] += rng.randint(1, 7)
        rows, size = c["T"] * c["top_k"], c["N"] * c["K"]
        # no more than the largest listed case; the plain form's padded batch and
        # the FP32 weights stay within a few GB too
        if 2 * rows * size > (4e11 if dtype == "f32" else 3.8e12) or E * size > 2.5e9:
            continue
        if E * c["T"] * (c["N"] + c["K"]) > 8e9 or (op == "weight_grad" and c["T"] < 16):
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


def _normal(shape, g, dtype, std=1.0):
    """N(0, std^2) values, drawn slab by slab so that a large tensor needs no FP32 copy."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    per = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for s in range(0, shape[0], per):
        v = torch.randn((min(per, shape[0] - s),) + tuple(shape[1:]), generator=g, device="cuda")
        out[s:s + per] = v if std == 1.0 else v.mul_(std)
    return out


def _layout(rows, I):
    """Where the checkpoint keeps its four planes: (row codes, row scales, byte offsets, bytes)."""
    P = -(-I // BLOCK) * BLOCK
    S = P // BLOCK
    at, planes = 0, []
    for n in (rows * P, rows * P, rows * S, rows * S):
        planes.append(at)
        at += -(-n // 256) * 256
    return P, S, planes, at


def _planes(ckpt, rows, I):
    P, S, at, _ = _layout(rows, I)
    codes = [ckpt[a:a + rows * P].view(torch.float8_e4m3fn).view(rows, P) for a in at[:2]]
    scales = [ckpt[a:a + rows * S].view(rows, S) for a in at[2:]]
    return codes + scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("product", "weight_grad"):
        counts = _counts(case, seed)
        rows, E, N, K = int(counts.sum()), case["E"], case["N"], case["K"]
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        st["most"] = int(counts.max())
        st["a"] = _normal((rows, K), g, dt)
        if case["op"] == "product":
            shape = (E, K, N) if case["transposed"] else (E, N, K)
            st["w"] = _normal(shape, g, dt, K ** -0.5)
        else:
            st["grad"] = _normal((rows, N), g, dt)
        return st
    rows, I = case["rows"], case["I"]
    # gate and up products: some columns carry much larger values than others
    spread = torch.randn((2 * I,), generator=g, device="cuda").mul_(0.7).exp_()
    gu = (_normal((rows, 2 * I), g, torch.float32) * spread).to(dt)
    if case["op"] == "swiglu":
        st["g"], st["u"] = ((gu[:, :I], gu[:, I:]) if case["stacked"]
                            else (gu[:, :I].contiguous(), gu[:, I:].contiguous()))
        return st
    # any codes and scales a checkpoint may hold: here, those of gu
    P, _, _, size = _layout(rows, I)
    st["ckpt"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    codes_g, codes_u, scales_g, scales_u = _planes(st["ckpt"], rows, I)
    for part, codes, scales in ((gu[:, :I], codes_g, scales_g), (gu[:, I:], codes_u, scales_u)):
        q, s = _store(part)
        codes.view(torch.uint8).copy_(q.view(torch.uint8))
        scales.copy_(s)
    st["grad_h"] = _normal((rows, I), g, dt)
    # the gradients' destination: one stacked matrix (a product of both halves follows) or two
    both = torch.zeros((rows, 2 * I), dtype=dt, device="cuda")
    st["grad_g"], st["grad_u"] = ((both[:, :I], both[:, I:]) if case["stacked"] else
                                  (both.view(-1)[:rows * I].view(rows, I), both.view(-1)[rows * I:].view(rows, I)))
    return st


# ------------------------------------------------------------------ the plain forms

def _padded(x, expert, place, E, most):
    """The rows as a batch of E matrices, FP32, with zeros behind each expert's rows."""
    out = torch.zeros((E, most, x.shape[1]), dtype=torch.float32, device=x.device)
    out[expert, place] = x.float()
    return out


def _places(offsets, rows):
    r = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    expert = torch.searchsorted(offsets[1:], r, right=True)
    return expert, (r - offsets[expert]).long()


def _store(v):
    """Codes (e4m3, padded to whole blocks with zeros) and scale bytes of a matrix."""
    rows, I = v.shape
    P = -(-I // BLOCK) * BLOCK
    x = torch.zeros((rows, P), dtype=torch.float32, device=v.device)
    x[:, :I] = v
    x = x.view(rows, P // BLOCK, BLOCK)
    mant, expo = torch.frexp(x.abs().amax(-1))          # mant in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.where(mant == 0, -127, expo - 9 + (mant > 0.875).int()).clamp(-127, 119)
    q = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(rows, P), (e + 127).to(torch.uint8)


def _load(codes, scales, I):
    v = torch.ldexp(codes.float().view(codes.shape[0], -1, BLOCK), scales.int().unsqueeze(-1) - 127)
    return v.view(codes.shape[0], -1)[:, :I]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("product", "weight_grad"):
        a, E = st["a"], case["E"]
        expert, place = _places(st["offsets"], a.shape[0])
        pa = _padded(a, expert, place, E, st["most"])
        if op == "weight_grad":
            pg = _padded(st["grad"], expert, place, E, st["most"])
            return {"grad_w": torch.bmm(pg.transpose(1, 2), pa).to(DTYPES[case["out"]])}
        w = st["w"].float()
        out = torch.bmm(pa, w if case["transposed"] else w.transpose(1, 2))
        return {"out": out[expert, place].to(DTYPES[case["out"]])}
    if op == "swiglu":
        g, u = st["g"].float(), st["u"].float()
        h = (g / (1 + torch.exp(-g)) * u).to(st["g"].dtype)
        qg, sg = _store(st["g"])
        qu, su = _store(st["u"])
        return {"h": h, "gate": qg, "up": qu, "gate_scale": sg, "up_scale": su}
    gh = st["grad_h"]
    qg, qu, sg, su = _planes(st["ckpt"], gh.shape[0], gh.shape[1])
    g, u, d = _load(qg, sg, case["I"]), _load(qu, su, case["I"]), gh.float()
    t = 1 / (1 + torch.exp(-g))
    st["grad_g"].copy_(d * u * t * (1 + g * (1 - t)))
    st["grad_u"].copy_(d * g * t)
    return {"grad_g": st["grad_g"], "grad_u": st["grad_u"], "h": (g * t * u).to(gh.dtype)}


def run(state):
    if not own:
        return _plain(state)
    import mixture_experts_ffn_topk_gb300 as moe
    case = state["case"]
    op = case["op"]
    if op == "product":
        return {"out": moe.moe_grouped_gemm(state["a"], state["offsets"], state["w"],
                                            transposed=case["transposed"],
                                            out_dtype=DTYPES[case["out"]])}
    if op == "weight_grad":
        return {"grad_w": moe.moe_grouped_gemm_weight_grad(state["grad"], state["a"], state["offsets"],
                                                           grad_dtype=DTYPES[case["out"]])}
    if op == "swiglu":
        h, ckpt = moe.moe_swiglu_checkpoint(state["g"], state["u"])
        v = moe.swiglu_checkpoint_views(ckpt, *state["g"].shape)
        return {"h": h, "gate": v["gate_codes"], "up": v["up_codes"],
                "gate_scale": v["gate_scales"], "up_scale": v["up_scales"]}
    grad_g, grad_u, h = moe.moe_swiglu_checkpoint_backward(
        state["grad_h"], state["ckpt"], grad_g=state["grad_g"], grad_u=state["grad_u"])
    return {"grad_g": grad_g, "grad_u": grad_u, "h": h}


def work(case):
    es = DTYPES[case["dtype"]].itemsize
    if case["op"] in ("product", "weight_grad"):
        counts = _counts(case, 0)
        rows, touched, size = int(counts.sum()), int((counts > 0).sum()), case["N"] * case["K"]
        os_ = DTYPES[case["out"]].itemsize
        if case["op"] == "product":
            # the matrices of experts without rows are not read
            b = rows * case["K"] * es + touched * size * es + rows * case["N"] * os_
        else:
            # the gradient of an expert without rows is written too
            b = rows * (case["K"] + case["N"]) * es + case["E"] * size * os_
        return {"bytes": b + 4 * (case["E"] + 1), "flops": 2 * rows * size}
    rows, I = case["rows"], case["I"]
    P = -(-I // BLOCK) * BLOCK
    kept = 2 * rows * (P + P // BLOCK)
    if case["op"] == "swiglu":
        return {"bytes": 3 * rows * I * es + kept, "flops": 12 * rows * I}
    return {"bytes": 4 * rows * I * es + kept, "flops": 20 * rows * I}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_store(v, limit=1 << 24):
    """e4m3 values of one matrix's blocks, from the definition: exponent by comparison, value by
    rounding to multiples of the step of its binade (half to even)."""
    rows, I = v.shape
    P = -(-I // BLOCK) * BLOCK
    out = torch.zeros((rows, P), dtype=torch.float64, device=v.device)
    per = max(1, limit // P)
    for s in range(0, rows, per):
        x = torch.zeros((min(per, rows - s), P), dtype=torch.float64, device=v.device)
        x[:, :I] = v[s:s + per].double()
        x = x.view(x.shape[0], -1, BLOCK)
        top = x.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 10
        for _ in range(3):
            e = e + (top > 448 * torch.exp2(e)).double()
        x = x / torch.exp2(e.clamp(-127, 119))
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
        out[s:s + per] = (torch.round(x / step) * step).clamp(-448, 448).view(-1, P)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("product", "weight_grad"):
        if 2 * st["a"].shape[0] * case["N"] * case["K"] > 5e12:
            return None
        at, a = st["offsets"].tolist(), st["a"]
        if op == "weight_grad":
            out = torch.zeros((case["E"], case["N"], case["K"]), dtype=torch.float64, device=a.device)
            for e in range(case["E"]):
                s = slice(at[e], at[e + 1])
                torch.matmul(st["grad"][s].double().T, a[s].double(), out=out[e])
            return {"grad_w": out}
        out = torch.empty((a.shape[0], case["N"]), dtype=torch.float64, device=a.device)
        for e in range(case["E"]):
            s = slice(at[e], at[e + 1])
            if at[e + 1] > at[e]:
                w = st["w"][e].double()
                out[s] = a[s].double() @ (w if case["transposed"] else w.T)
        return {"out": out}
    if op == "swiglu":
        g, u = st["g"], st["u"]
        h = torch.empty(g.shape, dtype=torch.float64, device=g.device)
        for s in range(0, g.shape[0], 1024):
            x = g[s:s + 1024].double()
            h[s:s + 1024] = x * torch.sigmoid(x) * u[s:s + 1024].double()
        return {"h": h, "gate": _exact_store(g), "up": _exact_store(u), "gate_scale": None,
                "up_scale": None}
    rows, I = case["rows"], case["I"]
    P, S, at, _ = _layout(rows, I)
    outs = {k: torch.empty((rows, I), dtype=torch.float64, device="cuda") for k in ("grad_g", "grad_u", "h")}
    # the value of every e4m3 byte: sign, exponent with bias 7, three bits of fraction
    b = torch.arange(256, device="cuda")
    ex, fr = (b >> 3) & 15, (b & 7).double()
    value = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * torch.exp2(ex.double() - 7))
    value = torch.where(b >= 128, -value, value)
    value[127] = value[255] = float("nan")
    for s in range(0, rows, 1024):
        n = min(1024, rows - s)
        part = []
        for k in range(2):
            c = st["ckpt"][at[k] + s * P:at[k] + (s + n) * P].long()
            x = st["ckpt"][at[2 + k] + s * S:at[2 + k] + (s + n) * S].double()
            part.append((value[c].view(n, S, BLOCK) * torch.exp2(x - 127).view(n, S, 1)).view(n, P)[:, :I])
        g, u = part
        d, t = st["grad_h"][s:s + n].double(), torch.sigmoid(g)
        outs["grad_g"][s:s + n] = d * u * (t + g * t * (1 - t))
        outs["grad_u"][s:s + n] = d * g * t
        outs["h"][s:s + n] = g * t * u
    return outs
