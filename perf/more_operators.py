"""Microscaled 4-bit floating point, as measured workloads.

Three operators on the formats of 32 values that share a power of two (elements
of 4 bits, e2m1, or 8 bits, e4m3; the shared scale is an exponent of 8 bits):

  quant    rows to codes and scales, and back to the values they stand for
  linear   quantised rows times a weight of 4-bit elements
  grouped  the same product where each run of rows has a weight of its own: the
           experts of a layer, their rows read in place by index, the gated
           activation of an up projection in the same call

``run`` computes them with elementary torch operations in 32 bits (``own``
false) or through this package's entry points (``own`` true); ``exact``
computes them from their definitions in 64 bits.  Sizes: hidden 3584 and
intermediate 18944 are the decoder layer of this repository's benchmark; the
rest are generic powers of two and odd counts of blocks.
"""
import math

import torch

own = False

BLOCK = 32


def listed():
    return [
        # one decode token before a projection: pure latency
        dict(name="quant_token", op="quant", M=1, K=3584, dtype="bf16", fmt="fp4", rule="floor"),
        # rows of the down projection's input kept in 8 bits, no value clipped
        dict(name="quant_odd_fp8", op="quant", M=1003, K=18944, dtype="f32", fmt="fp8", rule="ceil"),
        # a prefill chunk: a stream through memory
        dict(name="quant_prefill", op="quant", M=16384, K=3584, dtype="bf16", fmt="fp4", rule="floor"),
        # one decode token through the up projection: latency and the weight stream
        dict(name="linear_token", op="linear", M=1, K=3584, N=18944, dtype="bf16", act="fp4",
             rule="floor"),
        # a decode batch through the down projection, activations in 8 bits
        dict(name="linear_decode_33", op="linear", M=33, K=18944, N=3584, dtype="bf16", act="fp8",
             rule="floor"),
        # a ragged chunk: odd numbers of rows, of blocks of inputs and of 16 channels
        dict(name="linear_ragged_517", op="linear", M=517, K=2912, N=4112, dtype="f32", act="fp4",
             rule="ceil"),
        # a prefill through the down projection, activations in 8 bits
        dict(name="linear_prefill_fp8", op="linear", M=2048, K=18944, N=3584, dtype="bf16", act="fp8",
             rule="floor"),
        # a prefill through the up projection, all in 4 bits
        dict(name="linear_prefill", op="linear", M=4096, K=3584, N=18944, dtype="bf16", act="fp4",
             rule="floor"),
        # one decode token's eight experts, gate and up in one call
        dict(name="grouped_token", op="grouped", M=1, k=8, E=128, K=2048, N=1536, dtype="bf16",
             act="fp4", rule="floor", gather=True, gated=True, tail=0),
        # a decode batch: most experts see a few rows, all weights are streamed
        dict(name="grouped_decode_64", op="grouped", M=64, k=8, E=128, K=2048, N=1536, dtype="bf16",
             act="fp8", rule="floor", gather=True, gated=True, tail=0),
        # the down products of a ragged chunk, rows in the experts' order; the last rows of the
        # buffer belong to no expert and stay as they were
        dict(name="grouped_ragged", op="grouped", M=517, k=4, E=32, K=1376, N=3584, dtype="bf16",
             act="fp4", rule="ceil", gather=False, gated=False, tail=111),
        # a prefill's gate and up products: hundreds of rows an expert
        dict(name="grouped_prefill", op="grouped", M=4096, k=6, E=64, K=3584, N=2560, dtype="bf16",
             act="fp4", rule="floor", gather=True, gated=True, tail=0),
    ]


# no drawn case costs more than the largest listed one of its operator
_CAP = {"quant": 16384 * 3584, "linear": 2.0 * 4096 * 3584 * 18944,
        "grouped": 2.0 * 4096 * 6 * 3584 * 2560}
_CAP_WEIGHT = 64 * 3584 * 2560


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "grouped", "grouped"])
    d = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rule=rng.choice(["floor", "ceil"]))
    fmt = rng.choice(["fp4", "fp8"])
    if op == "quant":
        d.update(fmt=fmt, M=_log(rng, 1, 16384), K=BLOCK * _log(rng, 1, 592))
        while d["M"] * d["K"] > _CAP["quant"]:
            d["M"] = d["M"] * 3 // 4
        return d
    if op == "linear":
        d.update(act=fmt, M=_log(rng, 1, 4096), K=BLOCK * _log(rng, 4, 592),
                 N=16 * _log(rng, 8, 1184))
        while 2.0 * d["M"] * d["N"] * d["K"] > _CAP["linear"]:
            d["M"] = d["M"] * 3 // 4
        return d
    E = _log(rng, 2, 128)
    d.update(act=fmt, E=E, k=rng.randint(1, min(8, E)), M=_log(rng, 1, 4096),
             K=BLOCK * rng.randint(4, 112), N=32 * rng.randint(4, 112),
             gather=rng.random() < 0.6, gated=rng.random() < 0.5,
             tail=rng.choice([0, 0, 1, 77]))
    while d["E"] * d["K"] * d["N"] > _CAP_WEIGHT:
        d["E"] = d["E"] * 3 // 4
    d["k"] = min(d["k"], d["E"])
    while 2.0 * (d["M"] * d["k"] + d["tail"]) * d["K"] * d["N"] > _CAP["grouped"]:
        d["M"] = d["M"] * 3 // 4
    return d


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K, dtype):
    """Tokens after a norm: unit variance, a few outlier channels."""
    x = _randn(g, M, K)
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 200)]
    x[:, cols] *= 20.0
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def _weight(g, N, K):
    """Codes, two to a byte (the even input in the low bits), and scales of N channels, as a
    checkpoint holds them; outputs of order one."""
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    mid = 127 + round(math.log2(1.0 / (2.9 * math.sqrt(K))))
    scales = torch.randint(mid - 2, mid + 2, (N, K // BLOCK), generator=g, device="cuda",
                           dtype=torch.uint8)
    return codes, scales


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    M, K = case["M"], case["K"]
    if op == "quant":
        return dict(x=_activations(g, M, K, case["dtype"]))
    if op == "linear":
        return dict(x=_activations(g, M, K, case["dtype"]), w=_weight(g, case["N"], K))
    E, k = case["E"], case["k"]
    # uneven popularity: some experts get many rows, some none
    pref = _randn(g, M, E) + 0.7 * _randn(g, 1, E)
    ids = torch.sort(pref, dim=1, descending=True).indices[:, :k].reshape(-1)
    order = torch.sort(ids, stable=True).indices
    ends = torch.cumsum(torch.bincount(ids, minlength=E), dim=0)
    offsets = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    P = M * k + case["tail"]
    rows = None
    if case["gather"]:
        rows = torch.cat([order // k, order.new_zeros(case["tail"])]).to(torch.int32)
    x = _activations(g, M if case["gather"] else P, K, case["dtype"])
    width = case["N"] // 2 if case["gated"] else case["N"]
    return dict(x=x, w=_weight(g, E * case["N"], K), offsets=offsets, rows=rows,
                out=_randn(g, P, width).to(torch.bfloat16))


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:
        import bit_quantized_amd as w4
        d["w4"] = w4
        if case["op"] == "linear":
            d["w"] = w4.mx_pack_weights(*d["w"])
            d["workspace"] = torch.empty(
                w4.mx_linear_workspace_bytes(case["M"], case["N"], case["K"], case["act"]),
                dtype=torch.uint8, device="cuda")
        elif case["op"] == "grouped":
            d["w"] = w4.mx_pack_weights(*d["w"], n_experts=case["E"])
            d["workspace"] = torch.empty(
                w4.mx_grouped_linear_workspace_bytes(d["x"].shape[0], d["out"].shape[0], case["E"],
                                                     case["N"], case["K"], case["act"]),
                dtype=torch.uint8, device="cuda")
    return d


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quant": _own_quant, "linear": _own_linear, "grouped": _own_grouped}[op](state)
    return {"quant": _plain_quant, "linear": _plain_linear, "grouped": _plain_grouped}[op](state)


# ------------------------------------------------- the package's operators

def _own_quant(st):
    w4 = st["w4"]
    c = st["case"]
    return w4.mx_dequant(w4.mx_quant(st["x"], c["fmt"], rule=c["rule"]), dtype=st["x"].dtype)


def _own_linear(st):
    w4 = st["w4"]
    c = st["case"]
    return w4.mx_linear(st["x"], st["w"], act=c["act"], rule=c["rule"], workspace=st["workspace"])


def _own_grouped(st):
    w4 = st["w4"]
    c = st["case"]
    return w4.mx_grouped_linear(st["x"], st["w"], st["offsets"], rows=st["rows"], gated=c["gated"],
                                act=c["act"], rule=c["rule"], out=st["out"],
                                workspace=st["workspace"])


# ------------------------------------------------------------ plain forms

def _plain_round(x, fmt, rule):
    """Values of 32-bit rows after the format: every block's scale, every element rounded to
    the nearest (ties to even)."""
    M, K = x.shape
    v = x.view(M, K // BLOCK, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    mant, e = torch.frexp(top)  # top = mant * 2^e, mant in [0.5, 1)
    e = e - 1
    if fmt == "fp4":
        e = e - 2
        above = mant > 0.75  # top > 6 * 2^e
    else:
        e = e - 8
        above = mant > 0.875  # top > 448 * 2^e
    if rule == "ceil":
        e = e + above.to(e.dtype)
    e = torch.where(top == 0, -127, e).clamp(-127, 127)
    a = torch.ldexp(v.abs(), -e)
    if fmt == "fp4":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp(max=6.0)
    else:
        a = a.clamp(max=448.0)
        step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp(min=-6) - 3)
        a = torch.round(a / step) * step
    return torch.ldexp(torch.where(v < 0, -a, a), e).view(M, K)


def _plain_weight(codes, scales):
    """Values [N][K] of packed codes and scales."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    N = codes.shape[0]
    q = torch.stack([codes & 15, codes >> 4], dim=2).view(N, -1)
    w = table[q.int()].view(N, -1, BLOCK)
    return torch.ldexp(w, scales.int()[:, :, None] - 127).view(N, -1)


def _plain_quant(st):
    c = st["case"]
    return _plain_round(st["x"].float(), c["fmt"], c["rule"]).to(st["x"].dtype)


def _plain_linear(st):
    c = st["case"]
    x = _plain_round(st["x"].float(), c["act"], c["rule"])
    return (x @ _plain_weight(*st["w"]).t()).to(torch.bfloat16)


def _plain_grouped(st):
    c = st["case"]
    N = c["N"]
    x = _plain_round(st["x"].float(), c["act"], c["rule"])
    ends = st["offsets"].tolist()
    codes, scales = st["w"]
    y = st["out"]
    for e in range(c["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        xe = x[lo:hi] if st["rows"] is None else x[st["rows"][lo:hi].long()]
        v = xe @ _plain_weight(codes[e * N:(e + 1) * N], scales[e * N:(e + 1) * N]).t()
        if c["gated"]:
            gate, up = v[:, : N // 2], v[:, N // 2:]
            v = gate / (1.0 + torch.exp(-gate)) * up
        y[lo:hi] = v.to(torch.bfloat16)
    return y


# ------------------------------------------------------------------ work

def work(case):
    M, K = case["M"], case["K"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quant":
        return {"bytes": 2 * M * K * size, "flops": 4 * M * K}
    weight = 0.5 + 1.0 / BLOCK  # bytes a weight: code, and its share of the scale
    N = case["N"]
    if case["op"] == "linear":
        return {"bytes": int(N * K * weight + M * K * size + M * N * 2), "flops": 2 * M * N * K}
    pairs = M * case["k"]
    E = case["E"]
    used = E * (1.0 - (1.0 - 1.0 / E) ** pairs) if M > 1 else min(E, pairs)
    width = N // 2 if case["gated"] else N
    return {"bytes": int(used * N * K * weight + (M if case["gather"] else pairs) * K * size
                         + pairs * (width * 2 + (4 if case["gather"] else 0))),
            "flops": 2 * pairs * N * K}


# --------------------------------------------------- definitions in 64 bits

def _exact_magnitudes(fmt, device):
    """The format's magnitudes in the order of their codes."""
    if fmt == "fp4":
        man, low, top = 1, 0, 6.0       # e2m1: smallest normal exponent 0
    else:
        man, low, top = 3, -6, 448.0    # e4m3: smallest normal exponent -6
    out, c = [], 0
    while True:
        e, m = c >> man, c & ((1 << man) - 1)
        v = m * 2.0 ** (low - man) if e == 0 else (1 + m / 2.0 ** man) * 2.0 ** (low + e - 1)
        if v > top:
            return torch.tensor(out, dtype=torch.float64, device=device)
        out.append(v)
        c += 1


def _exact_round(x, fmt, rule):
    x = x.double()
    M, K = x.shape
    mags = _exact_magnitudes(fmt, x.device)
    blocks = x.reshape(-1, BLOCK)
    out = torch.empty_like(blocks)
    for part in range(0, blocks.shape[0], 1 << 20):
        b = blocks[part: part + (1 << 20)]
        top = b.abs().max(dim=1).values
        # the exponent: floor: the largest value's own, less that of the format's largest;
        # ceil: the least at which the largest value needs no clipping
        limit = torch.exp2(torch.floor(torch.log2(mags[-1]))) if rule == "floor" else mags[-1]
        e = torch.floor(torch.log2(top.clamp(min=1e-300) / limit))
        for _ in range(2):  # (the logarithm may have rounded over a border)
            if rule == "floor":
                e = torch.where(limit * torch.exp2(e) > top, e - 1, e)
                e = torch.where(limit * torch.exp2(e + 1) <= top, e + 1, e)
            else:
                e = torch.where(limit * torch.exp2(e) < top, e + 1, e)
                e = torch.where(limit * torch.exp2(e - 1) >= top, e - 1, e)
        scale = torch.exp2(e.clamp(-127, 127))[:, None]
        a = (b.abs() / scale).clamp(max=float(mags[-1]))
        hi = torch.searchsorted(mags, a.contiguous()).clamp(max=len(mags) - 1)
        lo = (hi - 1).clamp(min=0)
        below, above = a - mags[lo], mags[hi] - a
        up = (above < below) | ((above == below) & (hi % 2 == 0))
        out[part: part + (1 << 20)] = torch.where(up, mags[hi], mags[lo]) * scale * torch.sign(b)
    return out.view(M, K)


def _exact_weight(codes, scales):
    mags = _exact_magnitudes("fp4", codes.device)
    N, half = codes.shape
    w = torch.empty(N, 2 * half, dtype=torch.float64, device=codes.device)
    for side in range(2):
        c = (codes // 16 if side else codes % 16).long()
        w[:, side::2] = torch.where(c >= 8, -1.0, 1.0) * mags[c % 8]
    return w * torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "quant":
        return _exact_round(d["x"], case["fmt"], case["rule"])
    x = _exact_round(d["x"], case["act"], case["rule"])
    if case["op"] == "linear":
        return x @ _exact_weight(*d["w"]).t().contiguous()
    y = d["out"].double()
    N = case["N"]
    offsets = d["offsets"].tolist()
    for e in range(case["E"]):
        run_of = slice(offsets[e], offsets[e + 1])
        xe = x[run_of] if d["rows"] is None else x[d["rows"][run_of].long()]
        if xe.shape[0] == 0:
            continue
        w = _exact_weight(*(t[e * N:(e + 1) * N] for t in d["w"]))
        v = xe @ w.t().contiguous()
        if case["gated"]:
            v = v[:, : N // 2] * torch.special.expit(v[:, : N // 2]) * v[:, N // 2:]
        y[run_of] = v
    return y
