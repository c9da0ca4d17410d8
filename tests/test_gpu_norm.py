"""RMS norm with the residual's addition and FP8 output, and its gradient, against
64-bit forms.

Tolerances.  A lane adds at most 8 * 4 squares one after the other, then 6 + 15 sums
join them: under 64 fp32 additions, each off by at most 2^-24 of the running sum, so
a sum of one sign is within 2^-18; a rounding to bf16 adds 2^-8 of the value, one to
e4m3 2^-4 of it, or half the step of the smallest codes, 2^-10.  The weights'
gradient adds M / 256 rows, then 16 and 16 parts: under 64 additions here too."""
import pytest
import torch

import train_ref as ref
import w8a8_fp8_block_amd as fp8q
from gpu_util import Guarded, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -18
BF16 = 2.0 ** -8


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _inputs(M, K, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    x[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20.0
    r = torch.randn(M, K, generator=g) if residual else None
    w = 1.0 + 0.3 * torch.randn(K, generator=g)
    return x.bfloat16(), None if r is None else r.bfloat16(), w.bfloat16()


def _mp(M):
    return (M + 15) // 16 * 16


def _forward(x, r, w, eps=EPS):
    M, K = x.shape
    out = dict(h=Guarded((M, K), torch.bfloat16) if r is not None else None, y=Guarded((M, K), torch.bfloat16),
               q=Guarded((M, K), ref.F8), srm=Guarded((M, K // 128), torch.float32),
               skm=Guarded((K // 128, _mp(M)), torch.float32), rstd=Guarded((M,), torch.float32))
    t = {k: None if v is None else v.t for k, v in out.items()}
    fp8q.fp8q_add_rmsnorm_quant(x.cuda(), None if r is None else r.cuda(), w.cuda(), t["h"], t["y"], t["q"], t["srm"],
                                t["skm"], t["rstd"], eps)
    torch.cuda.synchronize()
    for v in out.values():
        if v is not None:
            v.check_canary()
    return {k: None if v is None else v.cpu() for k, v in t.items()}


SHAPES = [(1, 128), (1, 5120), (3, 256), (7, 384), (16, 1024), (17, 1408), (25, 5120), (33, 2048), (65, 2176),
          (130, 6144), (5, 8320), (9, 17408), (2, 32768), (409, 640), (1168, 1152)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(M, K, residual):
    x, r, w = _inputs(M, K, M * 7 + K, residual)
    o = _forward(x, r, w)
    h, rstd, y, scale, q = ref.norm(x, r, w, EPS)
    if residual:
        assert torch.equal(o["h"].view(torch.int16), h.view(torch.int16))
    assert ((o["rstd"].double() - rstd).abs() <= F32 * rstd).all()
    assert ((o["y"].double() - y).abs() <= (BF16 + F32) * y.abs()).all()
    assert torch.equal(o["srm"], o["skm"][:, :M].t()) and (o["skm"][:, M:] == 0).all()
    assert ((o["srm"].double() - scale).abs() <= F32 * scale).all()
    err = (ref.code_values(o["q"]) - q).abs()
    assert (err <= q.abs() * (2.0 ** -4 + F32) + 2.0 ** -10).all()


def test_zero_rows_and_small_values():
    K = 1408
    x, r, w = _inputs(6, K, 5)
    x[1] = 0
    r[1] = 0
    x[2] = -r[2]  # cancels
    x[3] *= 2.0 ** -90  # far below eps: y is x / sqrt(eps)
    r[3] = 0
    w[:128] = 0  # a group of zeros
    o = _forward(x, r, w)
    h, rstd, y, scale, q = ref.norm(x, r, w, EPS)
    assert torch.equal(o["h"].view(torch.int16) & 0x7FFF, h.view(torch.int16) & 0x7FFF)
    assert ((o["rstd"].double() - rstd).abs() <= F32 * rstd).all()
    assert (o["srm"][1:3] == 0).all() and (o["srm"][:, 0] == 0).all()
    assert (ref.code_values(o["q"])[1:3] == 0).all() and (ref.code_values(o["q"])[:, :128] == 0).all()
    s = o["srm"].double()
    assert ((s - scale).abs() <= F32 * scale + 2.0 ** -149).all()
    assert ((o["y"].double() - y).abs() <= (BF16 + F32) * y.abs() + 2.0 ** -133).all()


def test_one_output_or_the_other():
    """Every choice of outputs gives the same bits; h may lie over x or the residual."""
    M, K = 37, 2304
    x, r, w = _inputs(M, K, 11)
    full = _forward(x, r, w)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    for rm, km in ((True, False), (False, True)):
        h, q = torch.empty_like(xd), torch.empty(M, K, dtype=torch.uint8, device="cuda")
        s = torch.empty((M, K // 128) if rm else (K // 128, _mp(M)), device="cuda")
        fp8q.fp8q_add_rmsnorm_quant(xd, rd, wd, h, None, q, s if rm else None, s if km else None, None, EPS)
        assert torch.equal(q.cpu(), full["q"].view(torch.uint8))
        assert torch.equal(s.cpu(), full["srm" if rm else "skm"])
    for over in ("x", "residual"):
        a, b = xd.clone(), rd.clone()
        q, s = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, _mp(M), device="cuda")
        fp8q.fp8q_add_rmsnorm_quant(a, b, wd, a if over == "x" else b, None, q, None, s, None, EPS)
        assert torch.equal(q.cpu(), full["q"].view(torch.uint8)) and torch.equal(s.cpu(), full["skm"])
        assert torch.equal((a if over == "x" else b).cpu(), full["h"])


def test_rows_do_not_depend_on_their_batch():
    """A row's results are the same alone and among others, whichever workgroup has it."""
    K = 5120
    x, r, w = _inputs(300, K, 3)
    full = _forward(x, r, w)
    for m in (0, 1, 150, 299):
        one = _forward(x[m:m + 1], r[m:m + 1], w)
        for k in ("h", "y", "q", "srm", "rstd"):
            a, b = one[k], full[k][m:m + 1]
            if k == "rstd":  # other numbers of waves a row add in another order
                assert ((a - b).abs() <= F32 * b).all()
            elif k == "h":
                assert torch.equal(a, b)


def test_nan_and_infinity_stay_in_their_row():
    K = 1152
    x, r, w = _inputs(9, K, 21)
    clean = _forward(x, r, w)
    x[2, 5] = float("nan")
    x[4, 700] = float("inf")
    x[6, 3] = 1e30  # the squares leave fp32's range
    o = _forward(x, r, w)
    for m in range(9):
        if m in (2, 4, 6):
            assert torch.isnan(o["srm"][m]).all()
        else:
            assert torch.equal(o["srm"][m], clean["srm"][m]) and torch.equal(o["q"].view(torch.uint8)[m],
                                                                            clean["q"].view(torch.uint8)[m])


def _backward(dy, dh, h, w, rstd):
    M, K = h.shape
    dx, dw = Guarded((M, K), torch.bfloat16), Guarded((K,), torch.float32)
    work = torch.full((fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    fp8q.fp8q_add_rmsnorm_grad(dy.cuda(), None if dh is None else dh.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dx.t,
                               dw.t, work)
    torch.cuda.synchronize()
    dx.check_canary()
    dw.check_canary()
    return dx.t.cpu(), dw.t.cpu()


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_backward(M, K, residual):
    h, dh, w = _inputs(M, K, M * 5 + K, residual)
    dy, _, _ = _inputs(M, K, M * 3 + K, False)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dw = _backward(dy, dh, h, w, rstd)
    rx, rw, sx, sw = ref.norm_grad(dy, dh, h, w, rstd)
    assert ((dx.double() - rx).abs() <= BF16 * rx.abs() + F32 * sx).all()
    assert ((dw.double() - rw).abs() <= F32 * sw).all()


def test_backward_many_rows_is_reproducible():
    M, K = 3000, 640
    h, dh, w = _inputs(M, K, 77)
    dy, _, _ = _inputs(M, K, 78, False)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    a, b = _backward(dy, dh, h, w, rstd), _backward(dy, dh, h, w, rstd)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    rx, rw, sx, sw = ref.norm_grad(dy, dh, h, w, rstd)
    assert ((a[0].double() - rx).abs() <= BF16 * rx.abs() + F32 * sx).all()
    assert ((a[1].double() - rw).abs() <= F32 * sw).all()


def test_backward_in_place_and_empty():
    M, K = 50, 1408
    h, dh, w = _inputs(M, K, 1)
    dy, _, _ = _inputs(M, K, 2, False)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dw = _backward(dy, dh, h, w, rstd)
    work = torch.empty(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    for over in range(3):
        t = [v.cuda() for v in (dy, dh, h)]
        dw2 = torch.empty(K, device="cuda")
        fp8q.fp8q_add_rmsnorm_grad(t[0], t[1], t[2], w.cuda(), rstd.cuda(), t[over], dw2, work)
        assert torch.equal(t[over].cpu(), dx) and torch.equal(dw2.cpu(), dw)
    none = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    dw2 = torch.full((K,), 7.0, device="cuda")
    fp8q.fp8q_add_rmsnorm_grad(none, None, none, w.cuda(), torch.empty(0, device="cuda"), none, dw2, None)
    assert (dw2 == 0).all()
    fp8q.fp8q_add_rmsnorm_quant(none, None, w.cuda(), None, None, torch.empty(0, K, dtype=torch.uint8, device="cuda"),
                                None, torch.empty(K // 128, 0, device="cuda"), None)


def test_gradient_against_differences():
    """The kernel's gradient against central differences of the 64-bit forward form,
    in random directions: <dx, u> = d/dt <y(x + t u), dy> + <x + t u, dh>."""
    M, K = 4, 384
    h, dh, w = _inputs(M, K, 31)
    dy, _, _ = _inputs(M, K, 32, False)

    def value(x, wt):
        y = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * wt
        return float((y * dy.double()).sum() + (x * dh.double()).sum())

    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dw = _backward(dy, dh, h, w, rstd)
    _, _, sx, sw = ref.norm_grad(dy, dh, h, w, rstd)
    g = torch.Generator().manual_seed(4)
    for _ in range(8):
        u, v = torch.randn(M, K, generator=g, dtype=torch.float64), torch.randn(K, generator=g, dtype=torch.float64)
        t = 1e-5
        nx = (value(h.double() + t * u, w.double()) - value(h.double() - t * u, w.double())) / (2 * t)
        nw = (value(h.double(), w.double() + t * v) - value(h.double(), w.double() - t * v)) / (2 * t)
        # the roundings of dx, and the difference's own: t^2 and 2^-53 / t of the terms, far below
        size = float(((BF16 * dx.double().abs() + F32 * sx) * u.abs()).sum())
        assert abs(float((dx.double() * u).sum()) - nx) <= size + 1e-6 * float((sx * u.abs()).sum())
        assert abs(float((dw.double() * v).sum()) - nw) <= (F32 + 1e-6) * float((sw * v.abs()).sum())


@pytest.mark.parametrize("K", [384, 5120, 17408])
def test_a_row_alone_and_in_a_batch(K):
    """Calls of up to 256 rows add a row's squares in one order and larger ones in another,
    since a row has twice the waves there: within each kind a row's results are the same bits
    in every batch, and between the two they agree as two results within the tolerances
    do."""
    x, r, w = _inputs(600, K, K + 1)
    many, more, few, one = (_forward(x[:n], r[:n], w) for n in (300, 600, 200, 1))
    for a, b, n in ((one, few, 1), (many, more, 300)):
        for k in ("h", "y", "q", "srm", "rstd"):
            assert torch.equal(a[k][:n].contiguous().view(torch.uint8), b[k][:n].contiguous().view(torch.uint8)), k
    last = _forward(x[199:200], r[199:200], w)
    for k in ("h", "y", "q", "srm", "rstd"):
        assert torch.equal(last[k].view(torch.uint8), few[k][199:].contiguous().view(torch.uint8)), k
    _, _, y, scale, q = ref.norm(x[:200], r[:200], w, EPS)
    for o in (few, {k: v[:200] for k, v in many.items()}):
        assert ((o["y"].double() - y).abs() <= (BF16 + F32) * y.abs()).all()
        assert ((o["srm"].double() - scale).abs() <= F32 * scale).all()
        assert ((ref.code_values(o["q"]) - q).abs() <= q.abs() * (2.0 ** -4 + F32) + 2.0 ** -10).all()
    assert torch.equal(few["h"], many["h"][:200])
    assert ((few["rstd"].double() - many["rstd"][:200].double()).abs() <= 2 * F32 * few["rstd"].double()).all()
    assert ((few["y"].double() - many["y"][:200].double()).abs() <= 2 * (BF16 + F32) * y.abs()).all()
    assert ((few["srm"].double() - many["srm"][:200].double()).abs() <= 2 * F32 * scale).all()
    off = (ref.code_values(few["q"]) - ref.code_values(many["q"][:200])).abs()
    assert (off <= 2 * (q.abs() * (2.0 ** -4 + F32) + 2.0 ** -10)).all()
    # a code moves where the two values lie on two sides of a border: 2^-17 of the value apart,
    # the borders 2^-4 of it, so one in 2^13
    assert (off != 0).double().mean() < 1e-3


def test_gradient_of_a_row_alone_and_in_a_batch():
    """dx in the same way: the same bits within a kind of launch."""
    K = 5120
    h, dh, w = _inputs(600, K, 9)
    dy, _, _ = _inputs(600, K, 10, False)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx = {n: _backward(dy[:n], dh[:n], h[:n], w, rstd[:n])[0] for n in (20, 200, 300, 600)}
    assert torch.equal(dx[20], dx[200][:20]) and torch.equal(dx[300], dx[600][:300])
    rx, _, sx, _ = ref.norm_grad(dy[:200], dh[:200], h[:200], w, rstd[:200])
    for n in (200, 600):
        assert ((dx[n][:200].double() - rx).abs() <= BF16 * rx.abs() + F32 * sx).all()


@pytest.mark.parametrize("M,K", [(1, 384), (30, 17408), (300, 8320), (300, 17408), (270, 32768)])
def test_in_place_at_every_kind_of_row(M, K):
    """dx over dy, dh or h, and h over x or the residual, where a row takes one launch or two,
    a workgroup or a part of one, and where dh is loaded behind the row's sum."""
    x, r, w = _inputs(M, K, M + K)
    dy, dh, _ = _inputs(M, K, M + K + 1)
    o = _forward(x, r, w)
    dx, dw = _backward(dy, dh, o["h"], w, o["rstd"])
    work = torch.empty(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    for over in range(3):
        t = [v.cuda() for v in (dy, dh, o["h"])]
        dw2 = torch.empty(K, device="cuda")
        fp8q.fp8q_add_rmsnorm_grad(*t, w.cuda(), o["rstd"].cuda(), t[over], dw2, work)
        assert torch.equal(t[over].cpu(), dx) and torch.equal(dw2.cpu(), dw)
    for over in range(2):
        t = [x.cuda(), r.cuda()]
        q, s = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, _mp(M), device="cuda")
        fp8q.fp8q_add_rmsnorm_quant(t[0], t[1], w.cuda(), t[over], None, q, None, s, None, EPS)
        assert torch.equal(t[over].cpu(), o["h"]) and torch.equal(q.cpu(), o["q"].view(torch.uint8))
        assert torch.equal(s.cpu(), o["skm"])
