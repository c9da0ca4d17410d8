"""Balance loss and the routing's gradient against 64-bit forms.

Tolerances: e^x is within 2 ulp, a token's sum joins 8 + 10 terms, a probability's
sum over the tokens T / 2048 + 16 + 128 of one sign: under 2^-17 of the value for up
to 30000 tokens (256 additions of 2^-24 each, and 2^-18 for the exponentials' sums).
A gradient's terms are products of such: 2^-17 of the magnitudes it adds, and 2^-8 of
the result where it is rounded to bf16."""
import math

import pytest
import torch

import train_ref as ref
import w8a8_fp8_block_amd as fp8q
from gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -17


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _router(T, E, k, dtype, seed, masked=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    l[:, torch.randperm(E, generator=g)[:masked]] = -math.inf
    l = l.to(dtype)
    best, ids = torch.sort(l.float(), dim=1, descending=True, stable=True)
    ids = torch.where(best > -math.inf, ids, -1)[:, :k].to(torch.int32)
    return l, ids, torch.randn(T, k, generator=g)


def _balance(l, ids, coef):
    T, E = l.shape
    counts, prob = Guarded((E + 1,), torch.int32), Guarded((E,), torch.float32)
    loss = Guarded((1,), torch.float32)
    n = fp8q.fp8q_moe_balance_workspace_bytes(T, E)
    work = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    fp8q.fp8q_moe_balance(l.cuda(), ids.cuda(), counts.t, prob.t, loss.t, work, coef)
    torch.cuda.synchronize()
    for o in (counts, prob, loss):
        o.check_canary()
    return counts.t.cpu(), prob.t.cpu(), float(loss.t)


def _grad(l, ids, dw, counts, dloss, coef, renorm, top_k):
    d = Guarded(tuple(l.shape), l.dtype)
    fp8q.fp8q_moe_route_grad(l.cuda(), None if ids is None else ids.cuda(), None if dw is None else dw.cuda(),
                             None if counts is None else counts.int().cuda(),
                             None if dloss is None else torch.tensor([dloss], device="cuda"), d.t, renorm, coef, top_k)
    torch.cuda.synchronize()
    d.check_canary()
    return d.t.cpu()


def _near(d, r, size):
    half = 2.0 ** -8 if d.dtype is torch.bfloat16 else 0.0
    off = (d.double() - r).abs() - (half * r.abs() + F32 * size + 1e-38)
    bad = (~(off <= 0)).nonzero()
    assert not len(bad), [(i, float(d[tuple(i)]), float(r[tuple(i)]), float(size[tuple(i)])) for i in bad[:8].tolist()]


CASES = [(1, 8, 1), (3, 64, 8), (16, 128, 8), (25, 65, 3), (128, 160, 6), (129, 192, 2), (130, 7, 7), (1000, 256, 8),
         (5000, 16, 2), (700, 512, 32), (2049, 300, 5), (30000, 40, 4)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance(T, E, k, dtype):
    l, ids, _ = _router(T, E, k, dtype, T + E, masked=E // 8)
    counts, prob, loss = _balance(l, ids, 0.5)
    rc, rp, rl, _ = ref.balance(l, ids, 0.5)
    assert torch.equal(counts.long(), rc)
    assert ((prob.double() - rp).abs() <= F32 * rp).all()
    assert abs(loss - rl) <= 4 * F32 * rl


@pytest.mark.parametrize("T,E,k", [c for c in CASES if c[0] <= 2100])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("parts", ["weights", "loss", "both"])
def test_route_grad(T, E, k, renorm, parts):
    dtype = torch.bfloat16 if (T + E) % 2 else torch.float32
    l, ids, dw = _router(T, E, k, dtype, 3 * T + E, masked=E // 8)
    counts = ref.balance(l, ids, 1.0)[0] if parts != "weights" else None
    use = parts != "loss"
    d = _grad(l, ids if use else None, dw if use else None, counts, 1.5, 20.0, renorm, k)
    r, size = ref.route_grad(l, ids if use else None, dw, counts, 1.5, 20.0, renorm, k)
    _near(d, r, size)
    assert (d[l == -math.inf] == 0).all()


def test_nothing_to_choose_nan_and_infinity():
    T, E, k = 40, 20, 4
    l, ids, dw = _router(T, E, k, torch.float32, 8)
    l[3] = -math.inf
    l[5] = float("nan")
    l[7, 4] = float("nan")
    l[9, 6] = math.inf
    l[11] = torch.finfo(torch.float32).min
    ids[3] = ids[5] = -1
    dw[3] = dw[5] = float("nan")  # slots without an expert
    ids[7] = torch.tensor([1, 2, 3, 5])
    ids[13] = torch.tensor([2, 2, 2, 9])  # an expert twice and thrice
    ids[15] = torch.tensor([1000, -7, 20, 0])  # outside, but the last
    ids[17] = torch.tensor([4, 4, 4, 4])
    counts, prob, loss = _balance(l, ids, 2.0)
    rc, rp, rl, _ = ref.balance(l, ids, 2.0)
    assert torch.equal(counts.long(), rc) and int(counts[E]) == T - 2
    assert ((prob.double() - rp).abs() <= F32 * rp).all() and abs(loss - rl) <= 4 * F32 * rl
    for renorm in (True, False):
        d = _grad(l, ids, dw, rc, None, 2.0, renorm, k)
        r, size = ref.route_grad(l, ids, dw, rc, 1.0, 2.0, renorm, k)
        _near(d, r, size)
        assert (d[3] == 0).all() and (d[5] == 0).all() and d[7, 4] == 0


def test_empty():
    E = 12
    counts = torch.full((E + 1,), 9, dtype=torch.int32, device="cuda")
    prob, loss = torch.full((E,), 9.0, device="cuda"), torch.full((1,), 9.0, device="cuda")
    none, ids = torch.empty(0, E, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    fp8q.fp8q_moe_balance(none, ids, counts, prob, loss, None)
    assert (counts == 0).all() and (prob == 0).all() and (loss == 0).all()
    fp8q.fp8q_moe_route_grad(none, ids, torch.empty(0, 2, device="cuda"), counts, None, none)
    l = torch.full((4, E), -math.inf)
    c, p, s = _balance(l, torch.full((4, 2), -1, dtype=torch.int32), 1.0)
    assert (c == 0).all() and (p == 0).all() and s == 0
    assert (_grad(l, None, None, c, None, 1.0, True, 2) == 0).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit forms (counts and choices held) in random
    directions against the kernel's gradient."""
    T, E, k = 30, 24, 4
    l, ids, dw = _router(T, E, k, torch.float32, 12)
    counts = ref.balance(l, ids, 1.0)[0]
    g = torch.Generator().manual_seed(3)
    for renorm in (True, False):
        d = _grad(l, ids, dw, counts, 0.7, 30.0, renorm, k)
        size = ref.route_grad(l, ids, dw, counts, 0.7, 30.0, renorm, k)[1]

        def value(x):
            p, _ = ref.softmax(x)
            loss = 30.0 * E * float((counts[:E] / (T * k) * p.sum(0) / T).sum())
            chosen = torch.gather(x, 1, ids.long())
            w = ref.softmax(chosen)[0] if renorm else torch.gather(p, 1, ids.long())
            return 0.7 * loss + float((w * dw.double()).sum())

        for _ in range(6):
            u = torch.randn(T, E, generator=g, dtype=torch.float64)
            num = (value(l.double() + 1e-5 * u) - value(l.double() - 1e-5 * u)) / 2e-5
            assert abs(float((d.double() * u).sum()) - num) <= (F32 + 1e-6) * float((size * u.abs()).sum())


def test_scalars_anywhere():
    """The loss and its gradient are single floats: elements of a program's own tensor of
    losses serve, at any of its places."""
    T, E, k = 30, 24, 4
    l, ids, _ = _router(T, E, k, torch.float32, 12)
    lc, ic = l.cuda(), ids.cuda()
    losses, grads = torch.zeros(7, device="cuda"), torch.arange(1.0, 8.0, device="cuda")
    counts, prob = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda")
    rl = ref.balance(l, ids, 0.5)[2]
    d, first = torch.empty_like(lc), None
    for i in range(7):
        fp8q.fp8q_moe_balance(lc, ic, counts, prob, losses[i:i + 1], None, 0.5)
        fp8q.fp8q_moe_route_grad(lc, None, None, counts, grads[i:i + 1], d, top_k=k)
        first = d.clone() if i == 0 else first
        assert ((d - (i + 1) * first).abs() <= 2.0 ** -20 * (i + 1) * first.abs().max()).all()
    assert ((losses.cpu().double() - rl).abs() <= 4 * F32 * rl).all() and (losses == losses[0]).all()


# Both sides of every border of the numbers of logits a lane holds, and of the workgroups'
# sums: slices cut at 16 (few experts), and fewer of them with more rounds (many).
@pytest.mark.parametrize("E", [1, 31, 32, 33, 63, 95, 96, 97, 127, 129, 159, 161, 191, 193, 223, 224, 225, 255, 257,
                               383, 384, 385, 511])
@pytest.mark.parametrize("T", [129, 1100])
def test_every_number_of_experts(T, E):
    k = min(E, 3)
    dtype = torch.bfloat16 if E % 2 else torch.float32
    l, ids, dw = _router(T, E, k, dtype, T + E, masked=E // 8)
    counts, prob, loss = _balance(l, ids, 0.5)
    rc, rp, rl, _ = ref.balance(l, ids, 0.5)
    assert torch.equal(counts.long(), rc)
    assert ((prob.double() - rp).abs() <= F32 * rp).all() and abs(loss - rl) <= 4 * F32 * rl
    if T < 1000:
        for renorm in (True, False):
            d = _grad(l, ids, dw, rc, 1.5, 20.0, renorm, k)
            _near(d, *ref.route_grad(l, ids, dw, rc, 1.5, 20.0, renorm, k))


def test_many_tokens_of_few_and_of_many_experts():
    """256 workgroups' sums, in 16 slices and in 3."""
    for T, E in ((20000, 8), (20000, 512)):
        l, ids, _ = _router(T, E, 2, torch.float32, E)
        counts, prob, loss = _balance(l, ids, 0.5)
        rc, rp, rl, _ = ref.balance(l, ids, 0.5)
        assert torch.equal(counts.long(), rc)
        assert ((prob.double() - rp).abs() <= F32 * rp).all() and abs(loss - rl) <= 4 * F32 * rl
