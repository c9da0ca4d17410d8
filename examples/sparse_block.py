"""One block of a sparse model, served with per-request adapters: the projection
with low-rank adapters, the router, the expert FFN, and the residuals, all on the
library's kernels.

    python examples/sparse_block.py [--tokens 16] [--steps 50]

    h   = x + proj_lora(x)                     W8A8, each row its request's adapter
    ids = top-k of h . Wr^T                    bf16 router
    out = h + sum of the chosen experts' FFN   W8A8

Every buffer is allocated once (a Block holds them for one number of tokens), so a
step is launches only and can be captured into a graph, as decode does here.
Weights and inputs are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_fp8_block_amd as fp8q  # noqa: E402


def fp8_weights(*shape, gen):
    """Random block-scaled FP8 weights [..., N, K]: codes and 128x128 scales."""
    w = torch.randn(*shape, generator=gen, device="cuda") / shape[-1] ** 0.5
    b = w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    scale = b.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(1e-12) / 448
    q = (b / scale).flatten(-2).flatten(-3, -2).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).contiguous(), scale.squeeze(-1).squeeze(-2).contiguous()


def dequantized(q, scale):
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, -2).repeat_interleave(128, -1)


class Weights:
    def __init__(self, H=1024, I=512, E=128, adapters=4, rank=16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.proj = fp8_weights(H, H, gen=g)
        self.lora_a = (torch.randn(adapters, rank, H, generator=g, device="cuda") / H ** 0.5).bfloat16()
        self.lora_b = (torch.randn(adapters, H, rank, generator=g, device="cuda") / rank ** 0.5).bfloat16()
        self.lora_scale = torch.full((adapters,), 0.5, device="cuda")
        self.router = (torch.randn(E, H, generator=g, device="cuda") / H ** 0.5).bfloat16()
        self.gate, self.up = fp8_weights(E, I, H, gen=g), fp8_weights(E, I, H, gen=g)
        self.down = fp8_weights(E, H, I, gen=g)
        self.H, self.I, self.E, self.rank = H, I, E, rank


class Block:
    """The block for T tokens: its buffers, and step() enqueueing one pass of the
    inputs in self.x and self.adapter_ids into self.out."""

    def __init__(self, weights, T, top_k=8):
        w, self.w = weights, weights
        bf16, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")

        def work(n):
            return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None

        self.x, self.h, self.ffn, self.out = (torch.empty(T, w.H, **bf16) for _ in range(4))
        self.adapter_ids = torch.full((T,), -1, **i32)
        self.scratch = fp8q.alloc_proj_scratch(T, w.H)
        self.lora_work = work(fp8q.fp8q_proj_lora_workspace_bytes(T, w.H, w.H, w.rank))
        self.logits = torch.empty(T, w.E, **bf16)
        self.ids = torch.empty(T, top_k, **i32)
        self.weights = torch.empty(T, top_k, device="cuda")
        self.order, self.pos = torch.empty(T * top_k, **i32), torch.empty(T * top_k, **i32)
        self.offsets = torch.empty(w.E + 1, **i32)
        self.route_work = work(fp8q.fp8q_moe_route_workspace_bytes(T, w.E, top_k))
        self.ffn_work = work(fp8q.fp8q_moe_ffn_workspace_bytes(T, w.E, top_k, w.H, w.I))

    def step(self):
        w = self.w
        fp8q.fp8q_proj_lora(self.x, *w.proj, w.lora_a, w.lora_b, w.lora_scale, self.adapter_ids, self.h,
                            *self.scratch, self.lora_work)
        self.h.add_(self.x)
        fp8q.fp8q_gemm_bf16(self.h, w.router, self.logits)
        fp8q.fp8q_moe_route(self.logits, self.ids, self.weights, self.order, self.pos, self.offsets,
                            self.route_work)
        fp8q.fp8q_moe_ffn(self.h, self.weights, self.order, self.pos, self.offsets, *w.gate, *w.up, *w.down,
                          self.ffn, self.ffn_work)
        torch.add(self.h, self.ffn, out=self.out)

    def plain(self):
        """The same in fp32 without quantized activations, with the experts that
        step() chose: (h, the experts' sum)."""
        w, x = self.w, self.x.float()
        h = x + x @ dequantized(*w.proj).T
        for a in range(len(w.lora_scale)):
            r = self.adapter_ids == a
            h[r] += w.lora_scale[a] * (x[r] @ w.lora_a[a].float().T) @ w.lora_b[a].float().T
        y = torch.zeros_like(h)
        for e in self.ids.unique().tolist():
            t, j = (self.ids == e).nonzero(as_tuple=True)
            g, u, d = (dequantized(q[e], s[e]) for q, s in (w.gate, w.up, w.down))
            y.index_add_(0, t, (torch.nn.functional.silu(h[t] @ g.T) * (h[t] @ u.T) @ d.T)
                         * self.weights[t, j, None])
        return h, y


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--steps", type=int, default=50)
    a = p.parse_args()
    w = Weights()
    block = Block(w, a.tokens)
    block.x.normal_()
    # a request is a run of rows; every fifth has no adapter
    block.adapter_ids.copy_((torch.arange(a.tokens, device="cuda") // 4) % 5 - 1)
    block.step()
    torch.cuda.synchronize()
    h, y = block.plain()
    for name, got, want in (("projection", block.h, h), ("experts", block.ffn, y)):
        print(f"{name}: relative difference to fp32 {((got.float() - want).norm() / want.norm()).item():.3f}")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step()
    for name, run in (("eager", block.step), ("graph", graph.replay)):
        run()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps * 1e3:.1f} us a step of {a.tokens} tokens")


if __name__ == "__main__":
    main()
