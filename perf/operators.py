"""Operators whose weights depend on the row, as measured workloads.

Three operators of a served decoder layer in which the rows of one batch use
different weights:

  route  scores of a router -> the top-k experts of each token and their weights
  moe    the experts' gated MLP on W4A8 weights, combined by those weights
  lora   a shared W4A8 projection with a low-rank adapter chosen per row

``run`` computes them with elementary torch operations in 32 bits (``own``
false) or through this package's entry points (``own`` true); ``exact``
computes them from their definitions in 64 bits.  Sizes: hidden 3584 and
intermediate 18944 are the decoder layer of this repository's benchmark; the
rest are generic powers of two and odd counts.
"""
import math

import torch

own = False

GROUP = 128


def listed():
    return [
        # one decode token of a router over 128 experts: pure latency
        dict(name="route_token", op="route", M=1, E=128, k=8, dtype="bf16", score="softmax",
             bias=False, n_groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, masked=0),
        # a prefill chunk, sigmoid scores with a balance bias and limited groups
        dict(name="route_prefill_groups", op="route", M=16384, E=256, k=8, dtype="f32",
             score="sigmoid", bias=True, n_groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5, masked=0),
        # a mid-sized batch, odd number of experts, some of them switched off
        dict(name="route_batch_odd", op="route", M=1003, E=61, k=6, dtype="bf16", score="softmax",
             bias=False, n_groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, masked=7),
        # one decode token through many small experts: latency and a short weight stream
        dict(name="moe_token", op="moe", M=1, E=128, k=8, K=2048, I=768, dtype="bf16", drop=0.0),
        # a decode batch: most experts see a few rows, all weights are streamed
        dict(name="moe_decode_64", op="moe", M=64, E=128, k=8, K=2048, I=768, dtype="bf16", drop=0.0),
        # a ragged chunk with the benchmark's hidden size; a quarter of the slots belong to
        # experts held elsewhere
        dict(name="moe_chunk_ragged", op="moe", M=517, E=32, k=4, K=3584, I=1280, dtype="f32",
             drop=0.25),
        # a prefill: hundreds of rows an expert, bound by the matrix cores
        dict(name="moe_prefill", op="moe", M=4096, E=64, k=6, K=3584, I=1280, dtype="bf16", drop=0.0),
        # one decode token with its request's adapter on the up projection
        dict(name="lora_token", op="lora", M=1, K=3584, N=18944, L=8, R=16, dtype="bf16", seg=1),
        # a decode batch of different requests, long input
        dict(name="lora_decode_33", op="lora", M=33, K=18944, N=3584, L=32, R=64, dtype="bf16", seg=1),
        # a decode batch on the square projection, every row another request
        dict(name="lora_decode_16", op="lora", M=16, K=3584, N=3584, L=64, R=32, dtype="bf16", seg=1),
        # a prefill of some requests side by side, ragged lengths
        dict(name="lora_prefill", op="lora", M=2048, K=3584, N=18944, L=16, R=32, dtype="bf16",
             seg=300),
    ]


# no drawn case costs more than the largest listed one of its operator
_CAP = {"moe": 2.0 * 4096 * 6 * 3 * 3584 * 1280, "lora": 2.0 * 2048 * 3584 * 18944}
_CAP_SIZE = {"moe": 64 * 3584 * 1280, "lora": 32 * 64 * (3584 + 18944)}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd_out(v):
    return v + 128 if v == 3072 else v  # keep one much-used size out of the draw


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, _log(rng, 8, 512) // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(10, E * keep // groups))
        return dict(op=op, M=_odd_out(_log(rng, 1, 16384)), E=E, k=k, dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    n_groups=groups, topk_groups=keep,
                    group_top=rng.choice([1, 2]) if groups > 1 else 1,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0, 0, E // 3]))
    if op == "moe":
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        K = _odd_out(GROUP * rng.randint(2, 28))
        inter = GROUP * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 13, 16, 20])
        M = _odd_out(_log(rng, 1, 4096))
        while E * K * inter > _CAP_SIZE["moe"]:
            E = E * 3 // 4
        k = min(k, E)
        while 6.0 * M * k * K * inter > _CAP["moe"]:
            M = M * 3 // 4
        return dict(op=op, M=M, E=E, k=k, K=K, I=inter, dtype=dtype,
                    drop=rng.choice([0.0, 0.0, 0.3]))
    K = _odd_out(GROUP * _log(rng, 2, 148))
    N = _odd_out(16 * _log(rng, 16, 1184))
    M = _odd_out(_log(rng, 1, 2048))
    while 2.0 * M * N * K > _CAP["lora"]:
        M = M * 3 // 4
    L, R = _log(rng, 1, 64), 8 * _log(rng, 1, 16)
    while L * R * (K + N) > _CAP_SIZE["lora"]:
        L = L * 3 // 4
    return dict(op=op, M=M, K=K, N=N, L=L, R=R, dtype=dtype,
                seg=rng.choice([1, 1, 37, 300]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cast(x, dtype):
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def _activations(g, M, K, dtype):
    """Tokens after a norm: unit variance, a few outlier channels."""
    x = _randn(g, M, K)
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 200)]
    x[:, cols] *= 20.0
    return _cast(x, dtype)


def _weight(g, N, K):
    """int4 codes, zero points and scales of N output channels; outputs of order one."""
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    z = torch.randint(0, 16, (N, K // GROUP), generator=g, device="cuda", dtype=torch.uint8)
    s = _randn(g, N, K // GROUP).abs() * (0.15 / math.sqrt(K))
    return q, z, s


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "route":
        M, E = case["M"], case["E"]
        logits = _randn(g, M, E) * 1.5 + _randn(g, 1, E) * 0.5
        if case["masked"]:
            off = torch.randperm(E, generator=g, device="cuda")[: case["masked"]]
            logits[:, off] = float("-inf")
        bias = _randn(g, E) * 0.1 if case["bias"] else None
        return dict(logits=_cast(logits, case["dtype"]), bias=bias)
    if op == "moe":
        M, E, k, K, inter = (case[n] for n in ("M", "E", "k", "K", "I"))
        x = _activations(g, M, K, case["dtype"])
        up = _weight(g, E * 2 * inter, K)
        down = _weight(g, E * K, inter)
        # uneven popularity: some experts get many tokens, some none
        pref = _randn(g, M, E) + 0.7 * _randn(g, 1, E)
        val, ids = torch.sort(pref, dim=1, descending=True)
        weights = torch.softmax(val[:, :k], dim=1)
        ids = ids[:, :k].to(torch.int32)
        if case["drop"]:
            gone = torch.rand(M, k, generator=g, device="cuda") < case["drop"]
            ids = torch.where(gone, -1, ids)
        return dict(x=x, up=up, down=down, ids=ids.contiguous(), weights=weights.contiguous())
    M, K, N, L, R = (case[n] for n in ("M", "K", "N", "L", "R"))
    x = _activations(g, M, K, case["dtype"])
    w = _weight(g, N, K)
    A = (_randn(g, L, R, K) / math.sqrt(K)).to(torch.bfloat16)
    B = (_randn(g, L, N, R) / math.sqrt(R)).to(torch.bfloat16)
    scale = 0.25 + torch.rand(L, generator=g, device="cuda")
    # segments of rows of one request; -1: a request without an adapter
    nseg = -(-M // case["seg"])
    per = torch.randint(-1, L, (nseg,), generator=g, device="cuda", dtype=torch.int32)
    if nseg == 1:
        per.clamp_(min=0)
    ids = per.repeat_interleave(case["seg"])[:M].contiguous()
    return dict(x=x, w=w, A=A, B=B, scale=scale, ids=ids)


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:
        import bit_quantized_amd as w4
        d["w4"] = w4
        if case["op"] == "moe":
            E, K, inter = case["E"], case["K"], case["I"]
            d["up"] = w4.pack_experts(*d["up"], n_experts=E)
            d["down"] = w4.pack_experts(*d["down"], n_experts=E)
            d["workspace"] = torch.empty(
                w4.moe_mlp_workspace_bytes(case["M"], case["k"], E, inter, K), dtype=torch.uint8,
                device="cuda")
        elif case["op"] == "lora":
            d["w"] = w4.pack_weights(*d["w"])
            d["adapters"] = w4.LoraAdapters(d.pop("A"), d.pop("B"), d.pop("scale"))
            d["workspace"] = torch.empty(
                w4.lora_linear_workspace_bytes(case["M"], case["N"], case["K"], case["L"],
                                               case["R"]), dtype=torch.uint8, device="cuda")
    return d


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "moe": _own_moe, "lora": _own_lora}[op](state)
    return {"route": _plain_route, "moe": _plain_moe, "lora": _plain_lora}[op](state)


# ------------------------------------------------- the package's operators

def _own_route(st):
    w4 = st["w4"]
    c = st["case"]
    return w4.moe_route(st["logits"], c["k"], score=c["score"], bias=st["bias"],
                        n_groups=c["n_groups"], topk_groups=c["topk_groups"],
                        group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])


def _own_moe(st):
    w4 = st["w4"]
    return w4.moe_mlp(st["x"], st["up"], st["down"], st["ids"], st["weights"],
                      workspace=st["workspace"])


def _own_lora(st):
    w4 = st["w4"]
    return w4.lora_linear(st["x"], st["w"], st["adapters"], st["ids"], workspace=st["workspace"])


# ------------------------------------------------------------ plain forms

def _plain_route(st):
    c = st["case"]
    l = st["logits"].float()
    dead = torch.isneginf(l)
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        wide = torch.exp(l.double() - l.double().amax(dim=1, keepdim=True))
        wide = wide / wide.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
        wide = 1.0 / (1.0 + torch.exp(-l.double()))
    # which experts are chosen is decided in 64 bits: values next to a border
    sel = wide if st["bias"] is None else wide + st["bias"].double()
    sel = torch.where(dead, float("-inf"), sel)
    M, E = l.shape
    n = c["n_groups"]
    if n > 1:
        best = torch.sort(sel.view(M, n, E // n), dim=2, descending=True).values
        best = best[:, :, : c["group_top"]]
        value = torch.where(torch.isneginf(best), 0.0, best).sum(dim=2)
        value = torch.where(torch.isneginf(best[:, :, 0]), float("-inf"), value)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(M, n, dtype=torch.bool, device=l.device)
        keep.scatter_(1, order[:, : c["topk_groups"]], True)
        sel = torch.where(keep.repeat_interleave(E // n, dim=1), sel, float("-inf"))
    val, idx = torch.sort(sel, dim=1, descending=True, stable=True)
    val, idx = val[:, : c["k"]], idx[:, : c["k"]]
    w = torch.gather(p, 1, idx)
    none = torch.isneginf(val)
    w = torch.where(none, 0.0, w)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(none, -1, idx).to(torch.int32), w * c["scale"]


def _plain_quant(x):
    sa = x.abs().amax(dim=1, keepdim=True) / 127.0
    code = torch.round(x / torch.where(sa == 0, 1.0, sa)).clamp(-127, 127)
    return code, sa


def _plain_dequant(q, z, s):
    N, K = q.shape
    w = (q.view(N, -1, GROUP).float() - z.float()[:, :, None]) * s[:, :, None]
    return w.view(N, K)


def _plain_moe(st):
    c = st["case"]
    E, K, inter, k, M = c["E"], c["K"], c["I"], c["k"], c["M"]
    code, sa = _plain_quant(st["x"].float())
    flat = st["ids"].reshape(-1).long()
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1).tolist()
    parts = torch.zeros(M * k, K, dtype=torch.float32, device=code.device)
    qu, zu, su = st["up"]
    qd, zd, sd = st["down"]
    begin = 0
    for e in range(E):
        pairs = order[begin: begin + counts[e]]
        begin += counts[e]
        if counts[e] == 0:
            continue
        rows = pairs // k
        r = slice(e * 2 * inter, (e + 1) * 2 * inter)
        gu = (code[rows] @ _plain_dequant(qu[r], zu[r], su[r]).t()) * sa[rows]
        gate, up = gu[:, :inter], gu[:, inter:]
        h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float()
        hcode, hs = _plain_quant(h)
        r = slice(e * K, (e + 1) * K)
        parts[pairs] = (hcode @ _plain_dequant(qd[r], zd[r], sd[r]).t()) * hs
    y = (parts.view(M, k, K) * st["weights"][:, :, None]).sum(dim=1)
    return y.to(torch.bfloat16)


def _plain_lora(st):
    x = st["x"].float()
    code, sa = _plain_quant(x)
    y = (code @ _plain_dequant(*st["w"]).t()) * sa
    ids = st["ids"].long()
    for l in torch.unique(ids).tolist():
        if 0 <= l < st["A"].shape[0]:
            rows = torch.nonzero(ids == l).view(-1)
            hx = x[rows] @ st["A"][l].float().t()
            y[rows] += st["scale"][l] * (hx @ st["B"][l].float().t())
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "route":
        M, E, k = case["M"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * E * size + 8 * M * k + (4 * E if case["bias"] else 0),
                "flops": 8 * M * E}
    size = 2 if case["dtype"] == "bf16" else 4
    weight = 0.5 + (0.5 + 4.0) / GROUP  # bytes a weight: code, and its share of zero point and scale
    if op == "moe":
        M, E, k, K, inter = (case[n] for n in ("M", "E", "k", "K", "I"))
        pairs = M * k * (1.0 - case["drop"])
        used = E * (1.0 - (1.0 - 1.0 / E) ** pairs) if M > 1 else min(E, pairs)
        return {"bytes": int(used * 3 * inter * K * weight + M * K * (size + 2) + 8 * M * k),
                "flops": int(2 * pairs * 3 * inter * K)}
    M, K, N, L, R = (case[n] for n in ("M", "K", "N", "L", "R"))
    segs = -(-M // case["seg"])
    used = L * (1.0 - (1.0 - 1.0 / (L + 1)) ** segs) if segs > 1 else 1
    return {"bytes": int(N * K * weight + used * 2 * R * (K + N) + M * (K * size + N * 2 + 4)),
            "flops": int(2 * M * N * K + 2 * M * R * (K + N))}


# --------------------------------------------------- definitions in 64 bits

def _exact_codes(x):
    """Codes and scales of the rule sa = absmax / 127, code = rint(x / sa): both quotients are
    defined as correctly rounded float32 ones (a 64-bit quotient rounded once to 32 is that)."""
    x = x.double()
    sa = (x.abs().max(dim=1).values / 127.0).float().double()
    ratio = (x / sa.clamp(min=1e-300)[:, None]).float().double()
    return torch.clamp(torch.round(ratio), -127, 127), sa


def _exact_product(x, q, z, s):
    """sa * sum over groups of s * (integer group product), for every row of x."""
    code, sa = _exact_codes(x)
    N, K = q.shape
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
    for g in range(K // GROUP):
        span = slice(g * GROUP, (g + 1) * GROUP)
        steps = q[:, span].double() - z[:, g].double().unsqueeze(1)
        y += (code[:, span] @ steps.t().contiguous()) * s[:, g].double()
    return y * sa[:, None]


def _exact_route(case, d):
    l = d["logits"].double()
    M, E = l.shape
    if case["score"] == "softmax":
        p = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    else:
        p = torch.special.expit(l)
    c = p.clone() if d["bias"] is None else p + d["bias"].double()
    c[l == float("-inf")] = float("-inf")
    n = case["n_groups"]
    if n > 1:
        per = E // n
        alive = torch.zeros(M, n, dtype=torch.float64, device=l.device)
        for i in range(n):
            block = c[:, i * per:(i + 1) * per].clone()
            total = torch.zeros(M, dtype=torch.float64, device=l.device)
            empty = torch.isneginf(block.max(dim=1).values)
            for _ in range(min(case["group_top"], per)):
                top, at = block.max(dim=1)
                total += torch.where(torch.isneginf(top), torch.zeros_like(top), top)
                block.scatter_(1, at[:, None], float("-inf"))
            total[empty] = float("-inf")
            alive[:, i] = total
        rank = (alive[:, None, :] > alive[:, :, None]).sum(dim=2)
        lower = torch.tril(torch.ones(n, n, dtype=torch.bool, device=l.device), diagonal=-1)
        rank += ((alive[:, None, :] == alive[:, :, None]) & lower).sum(dim=2)
        gone = (rank >= case["topk_groups"]).repeat_interleave(per, dim=1)
        c[gone] = float("-inf")
    ids, ws = [], []
    column = torch.arange(E, device=l.device)
    for _ in range(case["k"]):
        top = c.max(dim=1, keepdim=True).values
        at = torch.where(c == top, column, E).min(dim=1).values  # ties: the lowest index
        none = torch.isneginf(top[:, 0])
        ids.append(torch.where(none, -1, at))
        ws.append(torch.where(none, 0.0, p.gather(1, at[:, None])[:, 0]))
        c.scatter_(1, at[:, None], float("-inf"))
    ids, w = torch.stack(ids, dim=1), torch.stack(ws, dim=1)
    if case["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), torch.zeros_like(w))
    return ids.to(torch.int32), w * case["scale"]


def _exact_moe(case, d):
    E, K, inter, M, k = (case[n] for n in ("E", "K", "I", "M", "k"))
    y = torch.zeros(M, K, dtype=torch.float64, device=d["x"].device)
    x = d["x"]
    for e in range(E):
        hit = d["ids"] == e
        rows = torch.nonzero(hit.any(dim=1))[:, 0]
        if rows.numel() == 0:
            continue
        up = [t[e * 2 * inter:(e + 1) * 2 * inter] for t in d["up"]]
        down = [t[e * K:(e + 1) * K] for t in d["down"]]
        gu = _exact_product(x[rows], *up)
        gate, value = gu[:, :inter], gu[:, inter:]
        h = (gate * torch.special.expit(gate) * value).to(torch.bfloat16)
        share = (d["weights"].double() * hit)[rows].sum(dim=1, keepdim=True)
        y[rows] += share * _exact_product(h, *down)
    return y


def _exact_lora(case, d):
    y = _exact_product(d["x"], *d["w"])
    x = d["x"].double()
    for m_id in range(case["L"]):
        rows = torch.nonzero(d["ids"] == m_id)[:, 0]
        if rows.numel():
            low = x[rows] @ d["A"][m_id].double().t().contiguous()
            y[rows] += float(d["scale"][m_id]) * (low @ d["B"][m_id].double().t().contiguous())
    return y


def exact(case, seed):
    d = _inputs(case, seed)
    return {"route": _exact_route, "moe": _exact_moe, "lora": _exact_lora}[case["op"]](case, d)
