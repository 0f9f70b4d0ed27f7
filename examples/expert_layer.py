"""A decoder layer's expert block and an adapted projection, as one served step.

    python examples/expert_layer.py --tokens 8 --steps 200

The step of a batch of tokens, each of its own request:

    scores  = x Wr^T                      the router (a plain product)
    ids, w  = moe_route(scores)           the experts of each token
    y       = x + moe_mlp(x, ids, w)      their gated MLP on W4A8 weights
    z       = lora_linear(y, adapters)    a W4A8 projection, an adapter a request

Weights are random.  The step is captured once as a graph, with its own
workspaces, and replayed with new tokens; every replay is compared with the
eager calls.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_amd as w4  # noqa: E402

GROUP = 128


def random_weight(g, n, k):
    """int4 codes, zero points and scales of n channels with k inputs."""
    q = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    z = torch.randint(0, 16, (n, k // GROUP), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand(n, k // GROUP, generator=g, device="cuda") * (0.2 / k ** 0.5)
    return q, z, s


class ExpertLayer:
    def __init__(self, g, hidden, inter, experts, top_k, out, adapters, rank):
        self.top_k = top_k
        self.router = torch.randn(experts, hidden, generator=g, device="cuda") / hidden ** 0.5
        self.balance = 0.1 * torch.randn(experts, generator=g, device="cuda")
        self.up = w4.pack_experts(*random_weight(g, experts * 2 * inter, hidden), n_experts=experts)
        self.down = w4.pack_experts(*random_weight(g, experts * hidden, inter), n_experts=experts)
        self.proj = w4.pack_weights(*random_weight(g, out, hidden))
        bf16 = torch.bfloat16
        self.adapters = w4.LoraAdapters(
            (torch.randn(adapters, rank, hidden, generator=g, device="cuda") / hidden ** 0.5).to(bf16),
            (torch.randn(adapters, out, rank, generator=g, device="cuda") / rank ** 0.5).to(bf16),
            torch.full((adapters,), 0.5, device="cuda"))

    def workspace(self, tokens):
        """One buffer for the step: its calls run one after another."""
        E, K, I = self.up.n_experts, self.up.K, self.down.K
        L, R, _ = self.adapters.A.shape
        need = max(w4.moe_mlp_workspace_bytes(tokens, self.top_k, E, I, K),
                   w4.lora_linear_workspace_bytes(tokens, self.proj.N, K, L, R))
        return torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(self, x, request_adapter, workspace=None):
        scores = x.float() @ self.router.t()
        ids, weights = w4.moe_route(scores, self.top_k, score="sigmoid", bias=self.balance)
        y = x + w4.moe_mlp(x, self.up, self.down, ids, weights, workspace=workspace)
        return y, w4.lora_linear(y, self.proj, self.adapters, request_adapter, workspace=workspace)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 8), ("steps", 100), ("hidden", 2048), ("inter", 768), ("experts", 64),
                        ("top-k", 8), ("out", 4096), ("adapters", 16), ("rank", 16), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(a.seed)
    layer = ExpertLayer(g, a.hidden, a.inter, a.experts, a.top_k, a.out, a.adapters, a.rank)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    req = torch.randint(-1, a.adapters, (a.tokens,), generator=g, device="cuda", dtype=torch.int32)
    ws = layer.workspace(a.tokens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, req, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = layer.step(x, req, ws)

    for _ in range(3):  # new tokens, other requests
        x.copy_(torch.randn(a.tokens, a.hidden, generator=g, device="cuda"))
        req.copy_(torch.randint(-1, a.adapters, (a.tokens,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), z.clone()
        want = layer.step(x, req)
        torch.cuda.synchronize()
        if not all(torch.equal(p, q) for p, q in zip(got, want)):
            raise SystemExit("a replay differs from the eager step")

    start = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / a.steps * 1e6
    print(f"{a.tokens} tokens: {us:.1f} us a step, replays equal the eager step")
    return us


if __name__ == "__main__":
    main()
