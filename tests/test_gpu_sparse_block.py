"""The example block (examples/sparse_block.py) runs the adapter, routing and expert
operators together: against fp32 without quantized activations.

Bound: an e4m3 rounding is at most 2^-4 of a value, about 2.6% in the mean
square, and as much of a product's norm.  The projection carries one (beside
the unquantized residual); gate and up add one to what h brings, 3.7% each, their
product 5.2%, and the intermediate's rounding makes it 5.8%: bounds 0.05, 0.1.
"""
import importlib.util
import os

import pytest
import torch

from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_block.py")


@pytest.mark.parametrize("tokens", [1, 16, 300])
def test_block(tokens):
    require_gpu()
    log(f"sparse block tokens={tokens}")
    spec = importlib.util.spec_from_file_location("sparse_block", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.Block(ex.Weights(H=512, I=256, E=128), tokens, top_k=4)
    block.x.copy_(torch.randn(tokens, 512, generator=torch.Generator().manual_seed(tokens)))
    block.adapter_ids.copy_(torch.arange(tokens) // 2 % 5 - 1)
    block.step()
    torch.cuda.synchronize()
    h, y = block.plain()
    assert ((block.h.float() - h).norm() / h.norm()).item() <= 0.05
    assert ((block.ffn.float() - y).norm() / y.norm()).item() <= 0.1
    assert torch.equal(block.out, block.h + block.ffn)
