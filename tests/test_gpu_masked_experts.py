"""The routing's gradient where experts cannot be chosen (logits of -inf or NaN): exactly
0, whatever the gradients that come in."""
import math

import pytest
import torch

import w8a8_fp8_block_amd as fp8q
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), math.inf])
@pytest.mark.parametrize("E", [12, 70, 300])
def test_zero_with_nan_and_infinite_gradients(E, bad, renorm, dtype):
    T, k = 21, 3
    g = torch.Generator().manual_seed(E)
    l = torch.randn(T, E, generator=g)
    l[:, 1::4] = -math.inf
    l[:, 2::4] = float("nan")
    l[7] = -math.inf
    ids = torch.topk(torch.nan_to_num(l, nan=-math.inf), k, dim=1).indices.to(torch.int32)
    ids[3, 1] = 1  # a slot that holds an expert that cannot be chosen
    dw = torch.randn(T, k, generator=g)
    dw[3] = dw[7] = dw[20, 2] = bad
    l = l.to(dtype)
    never = ~(l > -math.inf)
    counts = torch.full((E + 1,), T - 1, dtype=torch.int32)
    for loss in (1.0, bad):
        d = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
        fp8q.fp8q_moe_route_grad(l.cuda(), ids.cuda(), dw.cuda(), counts.cuda(), torch.tensor([loss], device="cuda"), d,
                                 renormalize=renorm)
        d = d.cpu()
        assert (d[never] == 0).all()
        finite = torch.isfinite(d) | never
        if loss == 1.0:
            assert finite[[t for t in range(T) if t not in (3, 20)]].all()
            assert not finite[20].all()  # a bad gradient of an expert's weight is not lost
        else:
            assert not finite[~never].any()
