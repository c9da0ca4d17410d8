"""A NaN among fp32 inputs stays a NaN in bf16 outputs, whichever of its bits are set:
memory filled with 0xFF holds the NaN 0xFFFFFFFF, whose rounding as an integer would carry
into the sign and leave a zero."""
import numpy as np
import pytest
import torch

import w8a8_fp8_block_amd as fp8q
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BITS = [0xFFFFFFFF, 0x7FFFFFFF, 0x7FC00000, 0x7F800001, 0xFFFF8000]


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _nan(t, at, bits):
    """t, fp32, with the NaN of these bits at `at`."""
    t.view(torch.int32)[at] = int(np.uint32(bits).view(np.int32))
    return t


def _work(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M", [5, 700])
def test_norm_gradient(M, bits):
    K = 640
    h, dy = torch.ones(M, K, dtype=torch.bfloat16, device="cuda"), torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    rstd = _nan(torch.ones(M, device="cuda"), 3, bits)
    dx, dw = torch.zeros_like(h), torch.zeros(K, device="cuda")
    fp8q.fp8q_add_rmsnorm_grad(dy, None, h, w, rstd, dx, dw, _work(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K)))
    assert torch.isnan(dx[3]).all() and torch.isnan(dw).all()
    assert not torch.isnan(dx[:3]).any() and not torch.isnan(dx[4:]).any()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_routing_gradient(dtype, renorm, bits):
    T, E, k = 20, 24, 3
    g = torch.Generator().manual_seed(1)
    l = torch.randn(T, E, generator=g).to(dtype).cuda()
    ids = torch.topk(l.float(), k, dim=1).indices.to(torch.int32)
    counts = torch.full((E + 1,), T, dtype=torch.int32, device="cuda")
    # through the weights: the row of the slot.  Renormalised, over the chosen experts alone.
    dw = _nan(torch.ones(T, k, device="cuda"), (6, 1), bits)
    d = torch.zeros_like(l)
    fp8q.fp8q_moe_route_grad(l, ids, dw, counts, None, d, renormalize=renorm)
    chosen = ids[6].long()
    assert torch.isnan(d[6, chosen]).all()
    assert renorm or torch.isnan(d[6]).all()
    keep = torch.arange(T) != 6
    assert not torch.isnan(d[keep]).any()
    # through the loss: everywhere
    loss = _nan(torch.ones(1, device="cuda"), 0, bits)
    fp8q.fp8q_moe_route_grad(l, None, None, counts, loss, d, top_k=k)
    assert torch.isnan(d).all()


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,N,K", [(20, 256, 384), (16, 5120, 1024), (300, 256, 16384)])
def test_products(M, N, K, bits):
    """dx (whole sums, and cut in ranges) and the forward product: scales that are NaN."""
    dy, w = (torch.full(s, 0x38, dtype=torch.uint8, device="cuda") for s in ((M, N), (N, K)))
    skm = _nan(torch.ones(N // 128, fp8q.fp8q_m_pad(M), device="cuda"), (1, 7), bits)
    ws = _nan(torch.ones(N // 128, K // 128, device="cuda"), (0, 2), bits)
    dx = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_dgrad(dy, skm, w, ws, dx, _work(fp8q.fp8q_gemm_dgrad_workspace_bytes(M, N, K)))
    want = torch.zeros(M, K, dtype=torch.bool, device="cuda")
    want[7] = True
    want[:, 256:384] = True
    assert torch.equal(torch.isnan(dx), want)

    x = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")
    xs = _nan(torch.ones(K // 128, fp8q.fp8q_m_pad(M), device="cuda"), (1, 7), bits)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    ws.fill_(1.0)
    fp8q.fp8q_gemm_blockscaled(x, xs, w, ws, out)
    assert torch.isnan(out[7]).all() and int(torch.isnan(out).sum()) == N


@pytest.mark.parametrize("bits", BITS)
def test_weighted_sum(bits):
    T, k, H = 6, 2, 256
    y = torch.ones(T * k, H, dtype=torch.bfloat16, device="cuda")
    weights = _nan(torch.ones(T, k, device="cuda"), (4, 1), bits)
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T * k], dtype=torch.int32, device="cuda")
    out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_moe_combine(y, weights, pos, offsets, out)
    assert torch.isnan(out[4]).all() and int(torch.isnan(out).sum()) == H


def test_every_bf16_value_and_its_neighbours():
    """1.0 times a scale, rounded to bf16: every bf16 value, the fp32 values next to it and
    those around the midpoint behind it, to the bit as torch rounds; NaN to NaN."""
    low = torch.tensor([0, 1, 0x7FFF, 0x8000, 0x8001, 0xFFFF])
    u = (torch.arange(1 << 16)[:, None] * 65536 + low).reshape(-1)
    s = torch.from_numpy(u.numpy().astype(np.uint32).view(np.float32))
    N = s.numel()
    w, dst = torch.full((N, 128), 0x38, dtype=torch.uint8, device="cuda"), torch.empty(N, 128, dtype=torch.bfloat16,
                                                                                       device="cuda")
    fp8q.fp8q_dequant_fp8_bf16(w, s.cuda(), dst, per_row=True)
    out, want = dst[:, 5].cpu(), s.to(torch.bfloat16)
    nan = torch.isnan(s)
    assert torch.isnan(out[nan]).all()
    assert torch.equal(out[~nan].view(torch.int16), want[~nan].view(torch.int16))
