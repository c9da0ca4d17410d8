"""dW over long sums, and over ranges of tokens that start and end anywhere.

A matrix instruction adds the products of 64 tokens, aligned to the largest of them, to
about 16 bits, and its sum to an fp32 accumulator that runs over all tokens of the range.
A product is off by at most 2^-16 of the largest of its 64; that one is 8 times the
products' RMS at most for normal data (two factors, each within 4 standard deviations,
both near them once in 10^5).  Errors and products add up alike, random signs or one
sign, so a sum is off by 8 * 2^-16 = 2^-13 of its norm whatever the number of tokens.
The accumulator's own roundings are 1024 at 65536 tokens, 2^-24 of the running sum each:
2^-14 where all go one way."""
import pytest
import torch

import train_ref as ref
import w8a8_fp8_block_amd as fp8q
from gpu_util import log, require_gpu
from test_gpu_grad import _check, _dual, _values, _wgrad, _wgrad_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _codes(M, C, g, one_sign):
    q = torch.empty(M, C, dtype=ref.F8, device="cuda")
    e = torch.empty((M + 511) // 512, C, 4, dtype=torch.uint8, device="cuda")
    x = torch.randn(M, C, generator=g, device="cuda")
    fp8q.fp8q_quant_act_dual((x.abs() if one_sign else x).bfloat16(), None, None, q, e)
    return q, e


def _part(q, e, first, last):
    """The values of token blocks first .. last - 1, float64."""
    b = torch.arange(first, last, device="cuda")
    scale = torch.exp2(e[b // 4, :, b % 4].double() - 127.0)
    v = q[128 * first:128 * last].double()
    return v * scale.repeat_interleave(128, 0)[:v.shape[0]]


@pytest.mark.parametrize("tokens", [4608, 16384, 65536])  # of one accumulator
@pytest.mark.parametrize("one_sign", [False, True])
def test_long_sums(tokens, one_sign):
    """The ranges' fp32 sums, before their one rounding to bf16 (they stand in the
    workspace).  The longest call has 64 ranges."""
    M, N, K = 64 * tokens, 128, 128
    g = torch.Generator(device="cuda").manual_seed(tokens)
    y, x = _codes(M, N, g, one_sign), _codes(M, K, g, one_sign)
    work = torch.empty(fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    dw = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_wgrad(*y, *x, dw, work)
    sums = work.view(torch.float32).view(-1, N, K)
    assert len(sums) == 64
    total = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for i in range(64):
        a, b = (_part(*t, i * tokens // 128, (i + 1) * tokens // 128) for t in (y, x))
        r = a.t().contiguous() @ b
        total += r
        if i < 2:
            off = float((sums[i].double() - r).norm() / r.norm())
            log(f"  tokens={tokens} one_sign={one_sign}: {off:.2e}")
            assert off <= 2.0 ** -13 + 2.0 ** -14
    off = (dw.double() - total).abs()
    assert (off <= 2.0 ** -8 * total.abs() + 2.0 ** -12 * total.norm() / 128).all()


def test_long_sum_of_a_whole_tile():
    """16384 and more tokens, uncut, value by value."""
    M, N, K = 40000, 1152, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    y, x = _codes(M, N, g, False), _codes(M, K, g, False)
    assert fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K) == 0
    dw = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_wgrad(*y, *x, dw, None)
    a, b = (_part(*t, 0, (M + 127) // 128) for t in (y, x))
    r = a.t().contiguous() @ b
    assert ((dw.double() - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -13 * r.norm() / (N * K) ** 0.5 * 6).all()


# 25 blocks in ranges of 12 and 13; 30 in two of 15; 37 in 12, 12 and 13: they start inside a
# dword of four blocks' bytes, end in the middle of one, and have an odd length.
@pytest.mark.parametrize("M", [3200, 3840, 4736, 4700, 3085])
@pytest.mark.parametrize("scales", ["own", "random"])
def test_ranges_that_start_anywhere(M, scales):
    N, K = 256, 256
    y, x = _dual(_values(M, N, M), rows=False), _dual(_values(M, K, M + 1), rows=False)
    if scales == "random":
        g = torch.Generator().manual_seed(M)
        for o in (y, x):
            o["et"].copy_(torch.randint(100, 150, o["et"].shape, generator=g, dtype=torch.int32).to(torch.uint8))
    assert fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K) >= 2 * 4 * N * K
    dw = _wgrad(y, x, M, N, K)
    r, size = _wgrad_ref(y, x)
    if scales == "own":
        _check(dw, r, size, f"M={M}")
    assert ((dw.double().cpu() - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -9 * size).all()


def test_nan_in_a_range():
    """A NaN in one range, at its edges: its rows and columns of dW, no others."""
    M, N, K = 3200, 256, 256
    yv, xv = _values(M, N, 5), _values(M, K, 6)
    a = _wgrad(_dual(yv, False), _dual(xv, False), M, N, K)
    yv[12 * 128 - 1, 9] = float("nan")  # the first range's last token
    xv[12 * 128, 200] = float("inf")  # the second one's first
    b = _wgrad(_dual(yv, False), _dual(xv, False), M, N, K).cpu()
    assert torch.isnan(b[9]).all() and torch.isnan(b[:, 200]).all()
    keep = torch.ones(N, K, dtype=torch.bool)
    keep[9], keep[:, 200] = False, False
    assert torch.equal(b[keep], a.cpu()[keep])
