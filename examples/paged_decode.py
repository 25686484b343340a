"""A decode loop over the 4-bit K/V cache: one transformer layer of quantized
linears, attention over the cache and a sparse MoE, for requests that start with
prompts of their own lengths and then decode token by token.

Per step, all on the GPU and with no length read by the host:
  kv_plan       the step's pages, slots and query rows from the requests' lengths
  qgemv         x -> q | k | v (Q4_K weights)
  kv_append     k, v rows (fp32; v as the slice of that product) into the cache as Q4_0 blocks
  kv_attention  the query rows over the cache
  qgemv         attention output -> hidden
  moe_forward   the layer's experts
The prompts run first, through the same calls; the decode step is captured once in a
CUDA graph and replayed while every request grows.

  python examples/paged_decode.py [--steps 32] [--requests 8]
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dequant_gemv_moe_gb300 as dq  # noqa: E402
import synth  # noqa: E402


class Layer:
    """Synthetic weights: q|k|v and output projections and a small MoE in Q4_K."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, head_dim=128, experts=8, top_k=2, ffn=512, seed=1):
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.n_qkv = (heads + 2 * kv_heads) * head_dim
        g = synth.streams(synth.BASE_SEED + seed, 2)
        up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.w_qkv = up(synth.quant_matrix(g[0], dq.Q4_K, self.n_qkv, hidden))
        self.w_out = up(synth.quant_matrix(g[1], dq.Q4_K, hidden, heads * head_dim))
        w = synth.moe_weights(synth.BASE_SEED + seed + 1, experts, hidden, ffn, 0, dq.Q4_K)
        self.moe = {k: up(v) for k, v in w.items() if v is not None}
        self.desc = dq.ops.make_desc(experts, top_k, hidden, ffn, 0, dq.Q4_K, self.moe["router_W"],
                                     self.moe["w_gate"], self.moe["w_up"], self.moe["w_down"])

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def linear(self, w, rows, cols, x):
        """All rows of x, DQ_MAX_BATCH at a time."""
        y = torch.empty(x.shape[0], rows, dtype=torch.float32, device=x.device)
        for i in range(0, x.shape[0], 8):
            dq.qgemv(dq.Q4_K, w, rows, cols, x[i:i + 8], y=y[i:i + 8])
        return y

    def forward(self, x, cache, plan, table, max_q_len, ws):
        """x [T][hidden] fp32 -> (the layer's output, the q rows, the attention's output and lse)."""
        T, H, D = x.shape[0], self.heads, self.head_dim
        qkv = self.linear(self.w_qkv, self.n_qkv, self.hidden, self.norm(x))
        q, k, v = (t.view(T, -1, D) for t in qkv.split([H * D, self.kv_heads * D, self.kv_heads * D], 1))
        q, k = self.norm(q), self.norm(k).float() * 2.0     # per head, as recent models do
        dq.kv_append(cache, k, v, plan.slots)               # v: the slice of the product as it is
        att, lse = dq.kv_attention(cache, q, plan.q_start, plan.kv_len, table, max_q_len=max_q_len, ws=ws)
        x = x + 1e-2 * self.linear(self.w_out, self.hidden, H * D, att.view(T, H * D))
        return x + 1e-3 * dq.moe_forward(self.desc, self.norm(x)), q, att, lse


class Server:
    """The state a serving loop keeps: cache, block tables, free pages, lengths."""

    def __init__(self, layer, requests, max_len, page_size=16):
        self.layer, self.B, self.page_size = layer, requests, page_size
        width = -(-max_len // page_size)
        n_pages = requests * width
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache = dq.KvCache.empty(n_pages, page_size, layer.kv_heads, layer.head_dim)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device="cuda")
        self.count, self.length = i32([n_pages]), i32([0] * requests)
        self.ws = torch.empty(dq.kv_attention_workspace_size(self.cache, layer.heads, requests, requests * max_len),
                              dtype=torch.uint8, device="cuda")

    def step(self, x, new, plan=None, max_q_len=1):
        """new: int32 [B] tokens per request; x: their rows.  Returns (y, q, attention, lse, plan)."""
        plan = dq.kv_plan(self.length, new, self.table, self.free, self.count, self.page_size, x.shape[0], out=plan)
        out = self.layer.forward(x, self.cache, plan, self.table, max_q_len, self.ws)
        self.length.copy_(plan.kv_len)
        self.count.copy_(plan.free_count)
        return (*out, plan)


def run(requests=8, steps=32, seed=7, layer=None):
    """Prompts, then `steps` captured decode steps.  Returns the server, the last step's results and ms per step."""
    layer = layer or Layer()
    rng = np.random.default_rng(seed)
    prompts = [int(n) for n in rng.integers(1, 200, requests)]
    server = Server(layer, requests, max(prompts) + steps + 4)
    x = torch.tensor(rng.standard_normal((sum(prompts), layer.hidden)), dtype=torch.float32, device="cuda")
    y, *_, plan = server.step(x, torch.tensor(prompts, dtype=torch.int32, device="cuda"), max_q_len=max(prompts))
    last = (plan.q_start[1:] - 1).long()
    x = y[last].clone()
    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    # a step outside capture first: it allocates what the graph will reuse
    y, *_, plan = server.step(x, one)
    x.copy_(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            before = x.clone()
            y, q, att, lse, _ = server.step(x, one, plan=plan)
            x.copy_(y)
    torch.cuda.current_stream().wait_stream(side)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    assert dq.device_status() == 0 and plan.unserved.item() == 0
    return server, dict(x=before, y=y, q=q, att=att, lse=lse, prompts=prompts, plan=plan), a.elapsed_time(b) / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--requests", type=int, default=8)
    a = ap.parse_args()
    server, last, ms = run(a.requests, a.steps)
    print("prompts %s\nlengths %s\n%.3f ms per decode step of %d requests" %
          (last["prompts"], server.length.tolist(), ms, a.requests))


if __name__ == "__main__":
    main()
