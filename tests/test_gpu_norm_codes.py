"""Scales and codes of the norm's FP8 output where its arithmetic is delicate.

Here rstd is exactly 1 and y an exact fp32 number, so scale = fl(amax / 448) and
q = e4m3_rne_sat(fl(y / scale)) are known to the last bit: no tolerance."""
import pytest
import torch

import train_ref as ref
import w8a8_fp8_block_amd as fp8q
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -126  # lost beside a mean of 1


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _norm(h, w):
    M, K = h.shape
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s, rstd = torch.empty(M, K // 128, device="cuda"), torch.empty(M, device="cuda")
    fp8q.fp8q_add_rmsnorm_quant(h.cuda(), None, w.cuda(), None, None, q, s, None, rstd, EPS)
    torch.cuda.synchronize()
    assert (rstd == 1.0).all()
    return q.cpu(), s.cpu()


def _expected(h, w):
    """(codes' values, scales) of y = h * w."""
    y = (h.double() * w.double()).view(h.shape[0], -1, 128)
    assert torch.equal(y.float().double(), y)
    s = (y.abs().amax(2) / 448.0).float()
    d = s.double()[:, :, None]
    v = torch.where(d > 0, y / torch.where(d > 0, d, 1.0), 0.0).float().double().clamp(-448.0, 448.0)
    return ref.nearest_code(v).view(h.shape), s


@pytest.mark.parametrize("M", [255, 600])  # a workgroup a row, several rows a workgroup
def test_tiny_groups(M):
    """Group maxima from 2^-149 to 5e4 times that: scales of a few units of 2^-149, whose
    rounding makes y / scale as large as 672 (which the code saturates to 448) or the
    scale 0."""
    g = torch.Generator().manual_seed(M)
    top = torch.arange(M) % 255 + 1
    n = torch.randint(-255, 256, (M, 512), generator=g) % (top[:, None] + 1)
    n = n * (2 * torch.randint(0, 2, n.shape, generator=g) - 1)
    for k in range(3):
        n[torch.arange(M), 128 * k + torch.randint(0, 128, (M,), generator=g)] = top
    h = n.float() * 2.0 ** -24
    h[:, 384:] = 2.0  # the mean of the squares: 128 * 4 / 512, the others lost beside it
    w = torch.ones(512)
    for k, m in enumerate((1, 6, 200)):
        w[128 * k:128 * k + 128] = m * 2.0 ** -125
    h, w = h.bfloat16(), w.bfloat16()
    q, s = _norm(h, w)
    rq, rs = _expected(h, w)
    nan = (q & 0x7F) == 0x7F
    assert not nan.any(), nan.nonzero()[:8].tolist()
    assert torch.equal(s, rs)
    bad = (ref.code_values(q) != rq).nonzero()
    assert not len(bad), [(i, int(q[tuple(i)]), float(rq[tuple(i)])) for i in bad[:8].tolist()]


@pytest.mark.parametrize("M", [64, 600])
def test_codes_and_scales_are_correctly_rounded(M):
    """Ordinary maxima: fp32 products of two bf16 numbers, 16 significant bits."""
    g = torch.Generator().manual_seed(M)
    h = torch.ones(M, 1024)
    h[:, 512:] = torch.where(torch.rand(M, 512, generator=g) < 0.5, -1.0, 1.0)
    w = torch.randn(1024, generator=g) * torch.exp(2 * torch.randn(1024, generator=g))
    h, w = h.bfloat16(), w.bfloat16()
    q, s = _norm(h, w)
    rq, rs = _expected(h, w)
    assert torch.equal(s, rs)
    assert torch.equal(ref.code_values(q), rq)


def test_groups_do_not_change_each_other():
    """A group of zeros or of tiny values takes the wave's division another way; the other
    groups' codes stay the same."""
    g = torch.Generator().manual_seed(3)
    M, K = 40, 1024
    h = torch.where(torch.rand(M, K, generator=g) < 0.5, -1.0, 1.0).bfloat16()
    w = (torch.randn(K, generator=g) * torch.exp(torch.randn(K, generator=g))).bfloat16()
    q, s = _norm(h, w)
    for value in (0.0, 2.0 ** -130, float("inf")):
        v = w.clone()
        v[256:384] = value
        q2, s2 = _norm(h, v)
        keep = torch.ones(K, dtype=torch.bool)
        keep[256:384] = False
        assert torch.equal(q2[:, keep], q[:, keep])
        assert torch.equal(s2[:, keep[::128]], s[:, keep[::128]])
