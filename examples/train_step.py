"""A training step through FP8 layers: the RMS norm with the residual's addition, an FP8
projection, and a router with its balance loss, forward and backward in the library.

    python examples/train_step.py

The master weights are fp32 torch tensors; the projection runs on their FP8 codes with a
scale per 128 x 128 block, which are formed anew after each update.  Autograd sees three
functions: NormProjection (norm, quantizer and product; its gradients are the two FP8
products and the norm's), Router (top-k weights and balance loss; one gradient of the
logits) and torch's own operations between them.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_fp8_block_amd as fp8q  # noqa: E402

EPS = 1e-6


def quantize_weights(w):
    """fp32 [N,K] -> (codes, scales [N/128,K/128])."""
    N, K = w.shape
    blocks = w.view(N // 128, 128, K // 128, 128)
    scale = (blocks.abs().amax(dim=(1, 3)) / 448.0).clamp(min=2.0 ** -100)
    codes = (blocks / scale[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(N, K), scale


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _workspace(nbytes):
    return _empty(nbytes, dtype=torch.uint8) if nbytes else None


class NormProjection(torch.autograd.Function):
    """(x, residual, norm weight, master weight, its codes, their scales) ->
    (h = x + residual, y = norm(h), norm(h) . W^T)."""

    @staticmethod
    def forward(ctx, x, residual, gain, master, w, w_scale):
        M, K = x.shape
        N = w.shape[0]
        h, y, q = _empty(M, K), _empty(M, K), _empty(M, K, dtype=torch.uint8)
        scale_km, rstd = _empty(K // 128, fp8q.fp8q_m_pad(M), dtype=torch.float32), _empty(M, dtype=torch.float32)
        fp8q.fp8q_add_rmsnorm_quant(x, residual, gain, h, y, q, None, scale_km, rstd, EPS)
        out = _empty(M, N)
        fp8q.fp8q_gemm_blockscaled(q, scale_km, w, w_scale, out)
        ctx.save_for_backward(h, y, gain, rstd, w, w_scale)
        return h, y, out

    @staticmethod
    def backward(ctx, dh, dy_more, dout):
        h, y, gain, rstd, w, w_scale = ctx.saved_tensors
        M, K = h.shape
        N, packs = w.shape[0], (M + 511) // 512
        # both codes of the output's gradient, the tokens' codes of the input
        dq, dscale = _empty(M, N, dtype=torch.uint8), _empty(N // 128, fp8q.fp8q_m_pad(M), dtype=torch.float32)
        dq_tok, dexp = _empty(M, N, dtype=torch.uint8), _empty(packs, N, 4, dtype=torch.uint8)
        fp8q.fp8q_quant_act_dual(dout.contiguous(), dq, dscale, dq_tok, dexp)
        y_tok, yexp = _empty(M, K, dtype=torch.uint8), _empty(packs, K, 4, dtype=torch.uint8)
        fp8q.fp8q_quant_act_dual(y, None, None, y_tok, yexp)
        dy, dw = _empty(M, K), _empty(N, K)
        fp8q.fp8q_gemm_dgrad(dq, dscale, w, w_scale, dy, _workspace(fp8q.fp8q_gemm_dgrad_workspace_bytes(M, N, K)))
        fp8q.fp8q_gemm_wgrad(dq_tok, dexp, y_tok, yexp, dw, _workspace(fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K)))
        if dy_more is not None:
            dy += dy_more
        dx, dgain = _empty(M, K), _empty(K, dtype=torch.float32)
        fp8q.fp8q_add_rmsnorm_grad(dy, None if dh is None else dh.contiguous(), h, gain, rstd, dx, dgain,
                                   _workspace(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K)))
        return dx, dx, dgain.to(gain.dtype), dw.float(), None, None


class Router(torch.autograd.Function):
    """logits [T,E] -> (weights [T,top_k] of the chosen experts, balance loss [1])."""

    @staticmethod
    def forward(ctx, logits, top_k, coef):
        T, E = logits.shape
        i32 = torch.int32
        ids, weights = _empty(T, top_k, dtype=i32), _empty(T, top_k, dtype=torch.float32)
        order, pos, offsets = _empty(T * top_k, dtype=i32), _empty(T * top_k, dtype=i32), _empty(E + 1, dtype=i32)
        fp8q.fp8q_moe_route(logits, ids, weights, order, pos, offsets,
                            _workspace(fp8q.fp8q_moe_route_workspace_bytes(T, E, top_k)), renormalize=False)
        counts, prob, loss = _empty(E + 1, dtype=i32), _empty(E, dtype=torch.float32), _empty(1, dtype=torch.float32)
        fp8q.fp8q_moe_balance(logits, ids, counts, prob, loss,
                              _workspace(fp8q.fp8q_moe_balance_workspace_bytes(T, E)), coef)
        ctx.save_for_backward(logits, ids, counts)
        ctx.coef = coef
        return weights, loss

    @staticmethod
    def backward(ctx, dweights, dloss):
        logits, ids, counts = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        fp8q.fp8q_moe_route_grad(logits, ids, dweights.contiguous(), counts, dloss.contiguous(), dlogits,
                                 renormalize=False, coef=ctx.coef)
        return dlogits, None, None


class Layer:
    def __init__(self, K=512, N=1024, E=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gain = torch.ones(K, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        self.w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).requires_grad_()
        self.router = (torch.randn(E, K, generator=g, device="cuda") * K ** -0.5).requires_grad_()
        self.top_k, self.coef = 4, 0.01

    def loss(self, x, residual, target):
        w, w_scale = quantize_weights(self.w.detach())
        h, y, out = NormProjection.apply(x, residual, self.gain, self.w, w, w_scale)
        weights, balance = Router.apply(y.float() @ self.router.t(), self.top_k, self.coef)
        mixed = out.float() * weights.sum(dim=1, keepdim=True)
        return (mixed - target).square().mean() + balance[0] + 1e-4 * h.float().square().mean()

    def parameters(self):
        return [self.gain, self.w, self.router]


def main(steps=20, tokens=777):
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(tokens, 512, generator=g, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    target = torch.randn(tokens, 1024, generator=g, device="cuda")
    for step in range(steps):
        loss = layer.loss(x, r, target)
        grads = torch.autograd.grad(loss, layer.parameters() + [x, r])
        with torch.no_grad():
            for p, d in zip(layer.parameters(), grads):
                p -= (20.0 * d).to(p.dtype)
        print(f"step {step}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
