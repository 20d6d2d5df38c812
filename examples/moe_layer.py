"""A mixture-of-experts block on 4-bit weights, as a model runs it.

Per token: a router (a small f32 product), top-k of E experts, the experts'
gate and up products with SwiGLU, their down products summed by weight, and a
dense shared expert beside them.  Prints the error against 64-bit arithmetic
and the time of a block as a CUDA graph, for a decode step, a small batch and
a prompt.

    python examples/moe_layer.py [--experts 64] [--top-k 8] [--hidden 2048] [--inner 1024] [--dtype bf16]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gguf_block_quantized_qmatmul_gb300 as q  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def random_weights(experts: int, N: int, K: int, group: int, gate_up: bool, gen: torch.Generator) -> q.Q4GWeights:
    """Checkpoint tensors of a 4-bit linear (codes, scales, zero points), laid out."""
    codes = torch.randint(0, 256, (experts, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand((experts, N, K // group), generator=gen, device="cuda")) * (0.2 / K ** 0.5)).half()
    zeros = torch.randint(6, 11, (experts, N, K // group), generator=gen, device="cuda", dtype=torch.uint8)
    return q.q4g_pack(codes, scales, zeros, gate_up=gate_up)


class MoeBlock:
    def __init__(self, experts: int, top_k: int, hidden: int, inner: int, group: int = 64, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.top_k, self.inner = top_k, inner
        self.router = torch.randn((experts, hidden), generator=gen, device="cuda") / hidden ** 0.5
        self.bias = 0.1 * torch.randn(experts, generator=gen, device="cuda")
        self.gate_up = random_weights(experts, 2 * inner, hidden, group, True, gen)
        self.down = random_weights(experts, hidden, inner, group, False, gen)
        self.shared_in = random_weights(1, 2 * inner, hidden, group, False, gen)
        self.shared_out = random_weights(1, hidden, inner, group, False, gen)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        route = q.moe_route(x.float() @ self.router.T, self.top_k, score="sigmoid", bias=self.bias)
        y = q.moe_down(self.down, q.moe_gate_up(self.gate_up, x, route), route)
        both = q.q4g_matmul(self.shared_in, x)
        h = torch.nn.functional.silu(both[:, :self.inner]) * both[:, self.inner:]
        return y + q.q4g_matmul(self.shared_out, h)

    def exact(self, x: torch.Tensor) -> torch.Tensor:
        """The same in 64 bits (for few tokens: an expert's weights per token and choice)."""
        route = q.moe_route(x.float() @ self.router.T, self.top_k, score="sigmoid", bias=self.bias)
        w = [q.q4g_dequantize(v) for v in (self.gate_up, self.down, self.shared_in, self.shared_out)]
        out = []
        for t in range(x.shape[0]):
            xt, F = x[t].double(), self.inner
            both = w[2][0].double() @ xt
            y = w[3][0].double() @ (both[:F] * torch.sigmoid(both[:F]) * both[F:])
            for e, p in zip(route.ids[t].tolist(), route.weights[t].tolist()):
                both = w[0][e].double() @ xt
                y = y + p * (w[1][e].double() @ (both[:F] * torch.sigmoid(both[:F]) * both[F:]))
            out.append(y)
        return torch.stack(out)


def graph_time(f, replays: int = 50) -> float:
    """Microseconds a replay of f captured in a CUDA graph."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    for _ in range(5):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(replays):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / replays


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--dtype", choices=list(DTYPES), default="bf16")
    a = ap.parse_args()
    block = MoeBlock(a.experts, a.top_k, a.hidden, a.inner)
    for tokens in (1, 16, 2048):
        x = torch.randn((tokens, a.hidden), device="cuda").to(DTYPES[a.dtype])
        y, few = block(x), min(tokens, 16)
        ref = block.exact(x[:few])
        err = float((y[:few].double() - ref).norm() / ref.norm())
        print(f"{tokens:5d} tokens: relative error {err:.1e}, {graph_time(lambda: block(x)):8.1f} us a block")
    if q.last_device_error():
        raise SystemExit("a device-side wait gave up")


if __name__ == "__main__":
    main()
