"""Cases, inputs, plain forms and exact values of the 4-bit and expert operators.

Four operators of the library are measured here:

* ``quantize``  larosa_mx4_quantize and larosa_mx4_dequantize: values to the
                microscaled 4-bit format (blocks of 32 that share a power of
                two, elements in e2m1) and back to the values it stands for;
* ``linear``    larosa_mx4_quantize of the activations, then larosa_mx4_linear:
                the product of 4-bit activations and 4-bit weights in
                torch.nn.Linear layout, from one token to a prompt;
* ``sparse``    larosa_mx4_sparse_linear and larosa_mx4_topk_linear: the kept
                rows of a 4-bit weight, row-major [d_in, d_out], 1 to 16 tokens;
* ``moe``       larosa_moe_layer: router, chosen experts and their weighted
                sum for 1 to 16 tokens, experts in bf16, fp32 or 4 bits.

``own`` selects the library's kernels; otherwise ``run`` computes the same in
elementary torch operations with 32-bit (the router's scores: 64-bit)
arithmetic.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2.0, "f32": 4.0, "mx4": 0.5 + 1.0 / BLOCK}
_DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one token's activation of a 4096-wide layer to 4 bits
        {"name": "quantize_1x4096_bf16", "op": "quantize", "rows": 1, "cols": 4096, "axis": 1, "dtype": "bf16"},
        # offline: a gate|up weight (row-major) with its blocks along the input channels
        {"name": "quantize_4096x22016_axis0_bf16", "op": "quantize", "rows": 4096, "cols": 22016, "axis": 0,
         "dtype": "bf16"},
        # an odd number of fp32 rows (rotated activations are fp32)
        {"name": "quantize_777x11008_f32", "op": "quantize", "rows": 777, "cols": 11008, "axis": 1,
         "dtype": "f32"},
        # three tokens through the down projection: the weight's bytes count
        {"name": "linear_3x11008x4096", "op": "linear", "M": 3, "d_in": 11008, "d_out": 4096, "dtype": "bf16",
         "out": "f32"},
        # a ragged prompt through q|k|v
        {"name": "linear_1111x4096x12288", "op": "linear", "M": 1111, "d_in": 4096, "d_out": 12288,
         "dtype": "bf16", "out": "bf16"},
        # a long prompt through gate|up of the 13B shape: the tensor cores' rate counts
        {"name": "linear_4096x5120x27648", "op": "linear", "M": 4096, "d_in": 5120, "d_out": 27648,
         "dtype": "bf16", "out": "bf16"},
        # one decoded token, gate|up at 40 % sparsity: kept rows only
        {"name": "sparse_1x4096x22016", "op": "sparse", "M": 1, "d_in": 4096, "d_out": 22016, "K": 2458,
         "topk": True},
        # sixteen tokens through the 13B down projection on given kept lists
        {"name": "sparse_16x13824x5120", "op": "sparse", "M": 16, "d_in": 13824, "d_out": 5120, "K": 8295,
         "topk": False},
        # a small expert layer and one token: latency
        {"name": "moe_1x256x512_e8k2_bf16", "op": "moe", "M": 1, "d": 256, "f": 512, "E": 8, "k": 2,
         "dtype": "bf16", "experts": "bf16", "renormalize": True},
        # one token, many small experts
        {"name": "moe_1x2048x768_e128k8_bf16", "op": "moe", "M": 1, "d": 2048, "f": 768, "E": 128, "k": 8,
         "dtype": "bf16", "experts": "bf16", "renormalize": True},
        # five fp32 tokens, gates from the softmax over every expert
        {"name": "moe_5x1024x1408_e60k4_f32", "op": "moe", "M": 5, "d": 1024, "f": 1408, "E": 60, "k": 4,
         "dtype": "f32", "experts": "f32", "renormalize": False},
        # sixteen tokens, few large experts held in 4 bits
        {"name": "moe_16x4096x14336_e8k2_mx4", "op": "moe", "M": 16, "d": 4096, "f": 14336, "E": 8, "k": 2,
         "dtype": "bf16", "experts": "mx4", "renormalize": True},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "sparse", "moe"])
    if op == "quantize":
        axis = rng.choice([0, 1])
        cols = BLOCK * _log_int(rng, 1, 864)
        most = max(1, 90_000_000 // cols)
        rows = _log_int(rng, 1, min(8192, most))
        if axis == 0:
            rows = max(BLOCK, rows // BLOCK * BLOCK)
        return {"op": op, "rows": rows, "cols": cols, "axis": axis, "dtype": rng.choice(["bf16", "f32"])}
    if op == "linear":
        d_in = BLOCK * _log_int(rng, 2, 430)
        d_out = _log_int(rng, 1, 28000)
        most = max(1, int(5.7e11 / (d_in * d_out)))
        return {"op": op, "M": _log_int(rng, 1, min(4096, most)), "d_in": d_in, "d_out": d_out,
                "dtype": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}
    if op == "sparse":
        d_in = BLOCK * _log_int(rng, 1, 430)
        d_out = BLOCK * _log_int(rng, 1, max(1, min(864, 90_000_000 // d_in // BLOCK)))
        return {"op": op, "M": rng.choice([1, 1, 2, 3, 4, 7, 8, 11, 16]), "d_in": d_in, "d_out": d_out,
                "K": max(1, int(d_in * rng.choice([0.05, 0.3, 0.5, 0.6, 0.8, 1.0]))),
                "topk": rng.choice([True, False])}
    E = _log_int(rng, 2, 160)
    experts = rng.choice(["bf16", "f32", "mx4"])
    dtype = "f32" if experts == "f32" else "bf16" if experts == "bf16" else rng.choice(["bf16", "f32"])
    d = BLOCK * _log_int(rng, 2, 128)
    f = BLOCK * _log_int(rng, 2, max(2, min(448, int(1.2e8 / (d * E)) // BLOCK)))
    return {"op": op, "M": rng.choice([1, 1, 2, 3, 5, 8, 13, 16]), "d": d, "f": f, "E": E,
            "k": rng.randint(1, min(8, E)), "dtype": dtype, "experts": experts,
            "renormalize": rng.choice([True, False])}


def work(case):
    """Bytes: every input once (of the experts and kept rows, those that the call needs), every output once."""
    op = case["op"]
    if op == "quantize":
        # values in, codes and scales out; codes and scales in, values out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * _BYTES[case["dtype"]] + 2 * _BYTES["mx4"]), "flops": 4.0 * n}
    if op == "linear":
        M, K, N = case["M"], case["d_in"], case["d_out"]
        return {"bytes": M * K * _BYTES[case["dtype"]] + K * N * _BYTES["mx4"] + M * N * _BYTES[case["out"]],
                "flops": 2.0 * M * K * N}
    if op == "sparse":
        M, d, n, K = case["M"], case["d_in"], case["d_out"], case["K"]
        rows = d * (1.0 - (1.0 - K / d) ** M)  # expected union of the tokens' kept rows
        blocks = min(d / BLOCK, rows)
        return {"bytes": rows * n / 2 + blocks * n + M * (4 * d if case["topk"] else 8 * K) + 4.0 * M * n,
                "flops": 2.0 * M * K * n}
    M, d, f, E, k = (case[c] for c in ("M", "d", "f", "E", "k"))
    distinct = E * (1.0 - (1.0 - k / E) ** M)  # expected number of chosen experts
    return {"bytes": distinct * 3 * d * f * _BYTES[case["experts"]] + (E * d + M * d) * _BYTES[case["dtype"]]
            + M * d * 4.0 + M * k * 8.0,
            "flops": 2.0 * M * E * d + 6.0 * M * k * d * f}


# ---------------------------------------------------------------- inputs

def _activations(gen, M, d, dtype):
    """Heavy-tailed rows: falling channel scales and four outlier channels."""
    std = (torch.arange(d, device=_DEV, dtype=torch.float32) + 1.0) ** -0.25
    std[torch.randint(0, d, (4,), generator=gen, device=_DEV)] *= 20.0
    return (torch.randn((M, d), generator=gen, device=_DEV) * std).to(dtype).contiguous()


def _normal(gen, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=_DEV) * std).to(dtype)


def _weight_mx4(gen, rows, cols, axis, std):
    codes, scales = [], []
    step = max(BLOCK, (1 << 26) // cols // BLOCK * BLOCK)
    for r in range(0, rows, step):
        c, s = _plain_quantize(_normal(gen, (min(step, rows - r), cols), std), axis)
        codes.append(c)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        dt = _DT[case["dtype"]]
        if case["axis"] == 1:
            st["x"] = _activations(gen, case["rows"], case["cols"], dt)
        else:
            st["x"] = _normal(gen, (case["rows"], case["cols"]), 0.02, dt)
    elif op == "linear":
        st["x"] = _activations(gen, case["M"], case["d_in"], _DT[case["dtype"]])
        st["wc"], st["ws"] = _weight_mx4(gen, case["d_out"], case["d_in"], 1, 0.02)
    elif op == "sparse":
        M, d, K = case["M"], case["d_in"], case["K"]
        st["x"] = _normal(gen, (M, d), 1.0)
        st["wc"], st["ws"] = _weight_mx4(gen, d, case["d_out"], 0, 0.02)
        if not case["topk"]:
            keys = torch.rand((M, d), generator=gen, device=_DEV)
            idx = torch.sort(torch.sort(keys, dim=1, stable=True).indices[:, :K], dim=1).values
            st["idx"] = idx.to(torch.int32).contiguous()
            st["val"] = torch.gather(st["x"], 1, idx).contiguous()
        if own:
            import activation_sparsity_b200 as L
            st["work"] = L.Workspace(torch.device(_DEV, torch.cuda.current_device()))
    else:
        M, d, f, E = case["M"], case["d"], case["f"], case["E"]
        dt = _DT[case["dtype"]]
        st["x"] = _normal(gen, (M, d), 1.0, dt)
        st["wr"] = _normal(gen, (E, d), 0.02, dt)
        if case["experts"] == "mx4":
            c, s = _weight_mx4(gen, E * d, 2 * f, 0, d ** -0.5)
            st["gu"], st["gus"] = c.view(E, d, f), s.view(E, d // BLOCK, 2 * f)
            c, s = _weight_mx4(gen, E * f, d, 0, f ** -0.5)
            st["dn"], st["dns"] = c.view(E, f, d // 2), s.view(E, f // BLOCK, d)
        else:
            st["gu"] = _normal(gen, (E, d, 2 * f), d ** -0.5, dt)
            st["dn"] = _normal(gen, (E, f, d), f ** -0.5, dt)
            st["gus"] = st["dns"] = None
        if own:
            import activation_sparsity_b200 as L
            st["work"] = L.Workspace(torch.device(_DEV, torch.cuda.current_device()))
    return st


# ---------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    normal = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)
    return torch.where(e < -126, normal * 0.5, normal)


def _blocks(x, axis):
    if axis == 1:
        return x.reshape(x.shape[0], -1, BLOCK), 2
    return x.reshape(-1, BLOCK, x.shape[1]), 1


def _plain_quantize(x, axis):
    """Codes (two to a byte, the even column in the low half) and scale bytes of fp32 values."""
    rows, cols = x.shape
    v, dim = _blocks(x, axis)
    amax = v.abs().amax(dim=dim, keepdim=True)
    e = (amax.view(torch.int32) >> 23) - 127 - 2  # floor(log2 amax) - 2
    e = e.clamp(min=-127)
    mag = (v * _pow2(-e)).abs()
    code = ((mag > 0.25).to(torch.uint8) + (mag >= 0.75) + (mag > 1.25) + (mag >= 1.75) + (mag > 2.5)
            + (mag >= 3.5) + (mag > 5.0))
    code = (code + 8 * (v < 0)).to(torch.uint8).reshape(rows, cols)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8).squeeze(dim).contiguous()


def _plain_values(codes, scales, axis):
    """The fp32 values that codes and scales stand for."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    rows, cols = codes.shape[0], codes.shape[1] * 2
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1).reshape(rows, cols)
    s = _pow2(scales.int() - 127)
    v, dim = _blocks(v, axis)
    return (v * s.unsqueeze(dim)).reshape(rows, cols)


def _keep(x, K):
    """The K entries of largest magnitude of each row (ties: the lower index), the rest zero."""
    order = torch.sort(x.abs(), dim=1, descending=True, stable=True).indices[:, :K]
    return torch.zeros_like(x).scatter_(1, order, torch.gather(x, 1, order))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales = _plain_quantize(st["x"].float(), case["axis"])
        return _plain_values(codes, scales, case["axis"]).to(_DT[case["dtype"]])
    if op == "linear":
        x = _plain_values(*_plain_quantize(st["x"].float(), 1), 1)
        return (x @ _plain_values(st["wc"], st["ws"], 1).t()).to(_DT[case["out"]])
    if op == "sparse":
        if case["topk"]:
            c = _keep(st["x"], case["K"])
        else:
            c = torch.zeros_like(st["x"]).scatter_(1, st["idx"].long(), st["val"])
        return c @ _plain_values(st["wc"], st["ws"], 0)
    M, d, f, E, k = (case[c] for c in ("M", "d", "f", "E", "k"))
    logits = st["x"].double() @ st["wr"].double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = order.values[:, :k], order.indices[:, :k]
    weight = torch.exp(top - top[:, :1])
    over = weight if case["renormalize"] else torch.exp(logits - top[:, :1])
    gate = (weight / over.sum(dim=1, keepdim=True)).float()
    share = torch.zeros((M, E), device=gate.device).scatter_(1, idx, gate)
    if case["experts"] == "mx4":
        gu = _plain_values(st["gu"].view(E * d, f), st["gus"].view(E * d // BLOCK, 2 * f), 0).view(E, d, 2 * f)
    else:
        gu = st["gu"].float()
    a = st["x"].float() @ gu
    del gu
    g, u = a[..., :f], a[..., f:]
    h = g / (1.0 + torch.exp(-g)) * u
    if case["experts"] == "mx4":
        dn = _plain_values(st["dn"].view(E * f, d // 2), st["dns"].view(E * f // BLOCK, d), 0).view(E, f, d)
    else:
        dn = st["dn"].float()
    y = ((h @ dn) * share.t().unsqueeze(-1)).sum(dim=0)
    return y, idx.to(torch.int32), gate


# ---------------------------------------------------------------- the library's calls

def _run_own(st):
    import activation_sparsity_b200 as L
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales = L.larosa_mx4_quantize(st["x"], axis=case["axis"])
        return L.larosa_mx4_dequantize(codes, scales, axis=case["axis"], dtype=_DT[case["dtype"]])
    if op == "linear":
        codes, scales = L.larosa_mx4_quantize(st["x"])
        return L.larosa_mx4_linear(codes, scales, st["wc"], st["ws"], dtype=_DT[case["out"]])
    if op == "sparse":
        if case["topk"]:
            return L.larosa_mx4_topk_linear(st["x"], st["wc"], st["ws"], case["K"], ws=st["work"])
        return L.larosa_mx4_sparse_linear(st["idx"], st["val"], st["wc"], st["ws"])
    return L.larosa_moe_layer(st["x"], st["wr"], st["gu"], st["dn"], case["k"], S_gu=st["gus"], S_d=st["dns"],
                              renormalize=case["renormalize"], ws=st["work"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- exact values

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _unit(e):
    """2^e in 64 bits for whole e, by its exponent field (pow may be off in the last place)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(x, axis):
    """Each value of the matrix rounded to its block's 4-bit grid, in 64 bits."""
    rows, cols = x.shape
    a = x.double()
    a = a if axis == 1 else a.t()
    b = a.reshape(-1, BLOCK)
    top = b.abs().max(dim=1, keepdim=True).values
    _, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1
    e = torch.where(top > 0, e - 1 - 2, torch.full_like(e, -127)).clamp(-127, 127)
    unit = _unit(e)
    q = b.abs() / unit
    # spacing of the grid: 0.5 below 2, 1 from 2 to 4, 2 from 4 on; halves go to the even multiple
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0)).double()
    r = (torch.round(q / step) * step).clamp(max=6.0) * torch.sign(b) * unit
    r = r.reshape(a.shape)
    return (r if axis == 1 else r.t()).reshape(rows, cols)


def _exact_values(codes, scales, axis):
    grid = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=codes.device)
    lo, hi = grid[(codes % 16).long()], grid[torch.div(codes, 16, rounding_mode="floor").long()]
    v = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    v[:, 0::2], v[:, 1::2] = lo, hi
    return v * torch.repeat_interleave(_unit(scales.to(torch.int64) - 127), BLOCK, dim=axis)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_round(st["x"], case["axis"])
    if op == "linear":
        x = _exact_round(st["x"], 1)
        out = torch.empty((case["M"], case["d_out"]), dtype=torch.float64, device=_DEV)
        for j in range(0, case["d_out"], 4096):
            out[:, j:j + 4096] = x @ _exact_values(st["wc"][j:j + 4096], st["ws"][j:j + 4096], 1).T
        return out
    if op == "sparse":
        out = torch.zeros((case["M"], case["d_out"]), dtype=torch.float64, device=_DEV)
        W = _exact_values(st["wc"], st["ws"], 0)
        for m in range(case["M"]):
            row = st["x"][m].double()
            if case["topk"]:
                kept = torch.sort(-row.abs(), stable=True).indices[:case["K"]]
                out[m] = row[kept] @ W[kept]
            else:
                out[m] = st["val"][m].double() @ W[st["idx"][m].long()]
        return out
    M, d, f, k = case["M"], case["d"], case["f"], case["k"]
    score = (st["x"].double().unsqueeze(1) * st["wr"].double().unsqueeze(0)).sum(dim=-1)
    by_rank = torch.sort(-score, dim=1, stable=True).indices
    idx = by_rank[:, :k]
    among = torch.gather(score, 1, idx) if case["renormalize"] else score
    gate = torch.exp(torch.gather(score, 1, idx) - torch.logsumexp(among, dim=1, keepdim=True))
    y = torch.zeros((M, d), dtype=torch.float64, device=_DEV)
    for e in sorted(set(idx.flatten().tolist())):
        if case["experts"] == "mx4":
            gu, dn = _exact_values(st["gu"][e], st["gus"][e], 0), _exact_values(st["dn"][e], st["dns"][e], 0)
        else:
            gu, dn = st["gu"][e].double(), st["dn"][e].double()
        t, s = torch.nonzero(idx == e, as_tuple=True)
        a = st["x"][t].double() @ gu
        y[t] += gate[t, s].unsqueeze(1) * ((a[:, :f] * torch.sigmoid(a[:, :f]) * a[:, f:]) @ dn)
    return y, idx.to(torch.int32), gate
