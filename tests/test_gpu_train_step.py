"""The operators of a training step together: the example's gradients, one step's calls
eager, on another stream and captured, and sizes past 32 bits."""
import importlib.util
import os

import pytest
import torch

import train_ref as ref
import w8a8_fp8_block_amd as fp8q
from gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _example():
    spec = importlib.util.spec_from_file_location("train_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


@pytest.mark.parametrize("tokens", [1, 16, 300, 777])
def test_example_gradients(tokens):
    """Against autograd in 64 bits on the dequantized weights.  An e4m3 rounding is 2.6% of
    the values in the mean square at most: the forward product carries one, which reaches
    every gradient through the loss, and each gradient product one or two more: 2.6% *
    sqrt(3) = 4.5%, bf16's 0.2% beside it.  Bound 0.08.  (One token: fewer values to average
    over, and no more roundings.)"""
    ex = _example()
    layer = ex.Layer(seed=tokens)
    g = torch.Generator().manual_seed(tokens)
    x, r = (torch.randn(tokens, 512, generator=g).bfloat16().cuda().requires_grad_() for _ in range(2))
    target = torch.randn(tokens, 1024, generator=g).cuda()
    leaves = layer.parameters() + [x, r]
    loss = layer.loss(x, r, target)
    grads = torch.autograd.grad(loss, leaves)

    codes, scale = ex.quantize_weights(layer.w.detach())
    w = codes.double().cpu() * scale.double().cpu().repeat_interleave(128, 0).repeat_interleave(128, 1)
    leaf = [t.detach().double().cpu().requires_grad_() for t in (layer.gain, w, layer.router, x, r)]
    gain, w, router, xd, rd = leaf
    h = xd + rd
    y = h * (h.square().mean(1, keepdim=True) + ex.EPS).rsqrt() * gain
    out = y @ w.t()
    p = torch.softmax(y @ router.t(), dim=1)
    top = p.topk(layer.top_k, dim=1)
    E = router.shape[0]
    f = torch.bincount(top.indices.reshape(-1), minlength=E).double() / (tokens * layer.top_k)
    plain = ((out * top.values.sum(1, keepdim=True) - target.double().cpu()).square().mean()
             + layer.coef * E * (f * p.mean(0)).sum() + 1e-4 * h.square().mean())
    want = torch.autograd.grad(plain, leaf)
    assert abs(loss.item() - plain.item()) <= 0.02 * plain.item()
    for name, a, b in zip(("gain", "w", "router", "x", "residual"), grads, want):
        off = float((a.double().cpu() - b).norm() / b.norm())
        log(f"  tokens={tokens} d{name}: {off:.4f}")
        assert off <= 0.08, (name, off)
    assert torch.equal(grads[3], grads[4])


class _Step:
    """One step's buffers and calls: norm, product, both codes, both gradients, the norm's
    gradient, the router's loss and gradient."""

    def __init__(self, M, N, K, E, top_k, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        Mp, packs = fp8q.fp8q_m_pad(M), (M + 511) // 512
        work = lambda n: new(n, dtype=u8) if n else None  # noqa: E731
        self.x, self.r, self.gain = rnd(M, K).bfloat16(), rnd(M, K).bfloat16(), (1 + 0.1 * rnd(K)).bfloat16()
        self.dout, self.dh = (rnd(M, N) * 1e-3).bfloat16(), (rnd(M, K) * 1e-3).bfloat16()
        q = torch.randint(0, 256, (N, K), generator=g, device="cuda").to(u8)
        self.w = torch.where((q & 0x7F) == 0x7F, 0x18, q.to(i32)).to(u8)
        self.ws = torch.rand(N // 128, K // 128, generator=g, device="cuda") * 1e-3
        self.logits, self.dweights = rnd(M, E), rnd(M, top_k)
        self.ids = torch.topk(self.logits, top_k, dim=1).indices.to(i32)
        self.h, self.y, self.q, self.skm, self.rstd = new(M, K), new(M, K), new(M, K, dtype=u8), \
            new(K // 128, Mp, dtype=f32), new(M, dtype=f32)
        self.out = new(M, N)
        self.dq, self.ds, self.dqt, self.de = new(M, N, dtype=u8), new(N // 128, Mp, dtype=f32), new(M, N, dtype=u8), \
            new(packs, N, 4, dtype=u8)
        self.yt, self.ye = new(M, K, dtype=u8), new(packs, K, 4, dtype=u8)
        self.dy, self.dw, self.dx, self.dgain = new(M, K), new(N, K), new(M, K), new(K, dtype=f32)
        self.counts, self.prob, self.loss = new(E + 1, dtype=i32), new(E, dtype=f32), new(1, dtype=f32)
        self.dlogits = new(M, E, dtype=f32)
        self.works = [work(n) for n in (
            fp8q.fp8q_gemm_dgrad_workspace_bytes(M, N, K), fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K),
            fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K), fp8q.fp8q_moe_balance_workspace_bytes(M, E))]

    OUT = ("h", "y", "q", "skm", "rstd", "out", "dq", "ds", "dqt", "de", "yt", "ye", "dy", "dw", "dx", "dgain",
           "counts", "prob", "loss", "dlogits")

    def run(self, stream=None):
        s = self
        fp8q.fp8q_add_rmsnorm_quant(s.x, s.r, s.gain, s.h, s.y, s.q, None, s.skm, s.rstd, stream=stream)
        fp8q.fp8q_gemm_blockscaled(s.q, s.skm, s.w, s.ws, s.out, stream=stream)
        fp8q.fp8q_moe_balance(s.logits, s.ids, s.counts, s.prob, s.loss, s.works[3], 0.1, stream=stream)
        fp8q.fp8q_quant_act_dual(s.dout, s.dq, s.ds, s.dqt, s.de, stream=stream)
        fp8q.fp8q_quant_act_dual(s.y, None, None, s.yt, s.ye, stream=stream)
        fp8q.fp8q_gemm_dgrad(s.dq, s.ds, s.w, s.ws, s.dy, s.works[0], stream=stream)
        fp8q.fp8q_gemm_wgrad(s.dqt, s.de, s.yt, s.ye, s.dw, s.works[1], stream=stream)
        fp8q.fp8q_add_rmsnorm_grad(s.dy, s.dh, s.h, s.gain, s.rstd, s.dx, s.dgain, s.works[2], stream=stream)
        fp8q.fp8q_moe_route_grad(s.logits, s.ids, s.dweights, s.counts, None, s.dlogits, coef=0.1, stream=stream)

    def take(self):
        return {k: getattr(self, k).clone() for k in self.OUT}

    def clear(self):
        for k in self.OUT:
            getattr(self, k).view(torch.uint8).fill_(0xFF)


def _same(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


def _product(o, form, a, a_scale, b, b_scale):
    """Value by value: the matrix instruction's alignment, 2^-9 of the products' magnitudes,
    and the rounding to bf16, 2^-8 of the result.  (Not by the whole's RMS: two correct results
    on either side of a rounding boundary are a whole bf16 step apart, 2^-7 of the value, and
    exponents that differ by 2^18 let a single value make up the norm.)"""
    r, size = form(a, a_scale, b, b_scale), form(a.abs(), a_scale, b.abs(), b_scale)
    assert ((o.double().cpu() - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -9 * size).all()


SIZES = [(1, 256, 128, 8, 2), (25, 512, 384, 64, 8), (409, 640, 1152, 40, 4), (1500, 1024, 640, 160, 6),
         (4000, 512, 512, 16, 2)]


@pytest.mark.parametrize("size", SIZES)
def test_step_eager_stream_and_graph(size):
    s = _Step(*size, seed=3)
    s.run()
    torch.cuda.synchronize()
    want = s.take()
    # every output's definition, from the step's own inputs to each call
    M, N, K, E, top_k = size
    h, rstd, y, scale, _ = ref.norm(s.x.cpu(), s.r.cpu(), s.gain.cpu(), 1e-6)
    assert torch.equal(want["h"].cpu(), h)
    _product(want["dy"], ref.dgrad, ref.code_values(want["dq"]), want["ds"].cpu()[:, :M].t(), ref.code_values(s.w),
             s.ws.cpu())
    _product(want["dw"], ref.wgrad, ref.code_values(want["dqt"]), want["de"].cpu(), ref.code_values(want["yt"]),
             want["ye"].cpu())

    side = torch.cuda.Stream()
    for explicit in (False, True):
        s.clear()
        torch.cuda.synchronize()
        if explicit:
            s.run(stream=side)
        else:
            with torch.cuda.stream(side):
                s.run()
        side.synchronize()
        _same(want, s.take())

    other = _Step(*size, seed=4)  # a second captured step, with workspaces of its own
    other.run()
    torch.cuda.synchronize()
    want2 = other.take()
    graphs = []
    for step in (s, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.run()
        graphs.append(graph)
    for turn in range(4):
        s.clear()
        other.clear()
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        _same(want, s.take())
        _same(want2, other.take())
        if turn == 1:  # new inputs in the captured buffers, and eager work between the replays
            s.x.neg_()
            s.dout.mul_(2.0)
            s.run()
            torch.cuda.synchronize()
            want = s.take()


def test_results_repeat():
    s = _Step(2000, 384, 1024, 48, 3, seed=9)
    s.run()
    first = s.take()
    for _ in range(3):
        s.clear()
        s.run()
        _same(first, s.take())


def test_refused_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w, q, s = x[0].clone(), torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 16, device="cuda")
    norm = fp8q.fp8q_add_rmsnorm_quant
    with pytest.raises(TypeError, match="x must be"):
        norm(x.float(), None, w, None, None, q, None, s, None)
    with pytest.raises(ValueError, match="weight must be of shape"):
        norm(x, None, w[:128], None, None, q, None, s, None)
    with pytest.raises(ValueError, match="scale_km must be of shape"):
        norm(x, None, w, None, None, q, None, s[:, :4], None)
    with pytest.raises(ValueError, match="contiguous"):
        norm(x, None, w, None, None, torch.zeros(256, 4, dtype=torch.uint8, device="cuda").t(), None, s, None)
    with pytest.raises(ValueError, match="current GPU"):
        norm(x, None, w.cpu(), None, None, q, None, s, None)
    with pytest.raises(fp8q.Fp8qError, match="eps"):
        norm(x, None, w, None, None, q, None, s, None, 0.0)
    with pytest.raises(fp8q.Fp8qError, match="without residual"):
        norm(x, None, w, x.clone(), None, q, None, s, None)
    with pytest.raises(fp8q.Fp8qError, match="aligned"):
        norm(torch.zeros(4 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 256), None, w, None, None, q,
             None, s, None)
    e = torch.zeros(1, 256, 4, dtype=torch.uint8, device="cuda")
    with pytest.raises(fp8q.Fp8qError, match="NULL"):
        fp8q.fp8q_quant_act_dual(x, q, None, q.clone(), e)
    with pytest.raises(TypeError, match="workspace"):
        fp8q.fp8q_add_rmsnorm_grad(x, None, x, w, s[0, :4].contiguous(), x.clone(), torch.zeros(256, device="cuda"),
                                   torch.zeros(1024, device="cuda"))
    with pytest.raises(fp8q.Fp8qError, match="workspace"):
        fp8q.fp8q_add_rmsnorm_grad(x, None, x, w, s[0, :4].contiguous(), x.clone(), torch.zeros(256, device="cuda"),
                                   torch.zeros(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(4, 256) - 1,
                                               dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="top_k"):
        fp8q.fp8q_moe_route_grad(s, None, None, torch.zeros(17, dtype=torch.int32, device="cuda"), None, s.clone())


# ---------------------------------------------------- offsets past 32 bits
def _big_codes(M, N, seed):
    q = torch.randint(0, 119, (M, N), dtype=torch.uint8, device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(seed))
    return q.view(ref.F8)


def test_dw_past_32_bits():
    """2.5e9 elements, 5 GB of bf16: the last rows and columns."""
    M, N, K = 130, 40960, 61440
    y, x = _big_codes(M, N, 1), _big_codes(M, K, 2)
    e = lambda n: torch.randint(110, 120, (1, n, 4), dtype=torch.uint8, device="cuda")  # noqa: E731
    ey, ex = e(N), e(K)
    dw = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_wgrad(y, ey, x, ex, dw, None)
    torch.cuda.synchronize()
    rows, cols = [0, 17000, 35000, N - 1], slice(K - 300, K)
    _product(dw[rows, cols], ref.wgrad, ref.code_values(y[:, rows].contiguous()), ey.cpu()[:, rows],
             ref.code_values(x[:, cols].contiguous()), ex.cpu()[:, cols])


def test_dx_past_32_bits():
    M, N, K = 66000, 128, 40960  # 2.7e9 elements of dx
    dy, s = _big_codes(M, N, 1), torch.rand(1, M, device="cuda")
    w, ws = _big_codes(N, K, 2), torch.rand(1, K // 128, device="cuda")
    n = fp8q.fp8q_gemm_dgrad_workspace_bytes(M, N, K)
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_dgrad(dy, s, w, ws, dx, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    torch.cuda.synchronize()
    rows, cols = [0, 33000, 52500, M - 1], slice(K - 256, K)
    _product(dx[rows, cols], ref.dgrad, ref.code_values(dy[rows]), s.cpu()[:, rows].t(),
             ref.code_values(w[:, cols].contiguous()), ws.cpu()[:, -2:])


def test_norm_and_dual_past_32_bits():
    M, K = 70000, 32768  # 2.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    h, y, q = torch.empty_like(x), torch.empty_like(x), torch.empty(M, K, dtype=ref.F8, device="cuda")
    s, rstd = torch.empty(K // 128, fp8q.fp8q_m_pad(M), device="cuda"), torch.empty(M, device="cuda")
    fp8q.fp8q_add_rmsnorm_quant(x, x, w, h, y, q, None, s, rstd, 1e-6)
    rows = [0, 32768, 65537, M - 1]
    rh, rr, ry, rs, _ = ref.norm(x[rows].cpu(), x[rows].cpu(), w.cpu(), 1e-6)
    assert torch.equal(h[rows].cpu(), rh)
    assert ((y[rows].cpu().double() - ry).abs() <= (2.0 ** -8 + 2.0 ** -18) * ry.abs()).all()
    assert ((s[:, rows].t().cpu().double() - rs).abs() <= 2.0 ** -18 * rs).all()
    del y
    dx, dw = torch.empty_like(x), torch.empty(K, device="cuda")
    work = torch.empty(fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_add_rmsnorm_grad(x, None, h, w, rstd, dx, dw, work)
    rx, _, sx, _ = ref.norm_grad(x[rows].cpu(), None, h[rows].cpu(), w.cpu(), rstd[rows].cpu())
    assert ((dx[rows].cpu().double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 2.0 ** -18 * sx).all()
    del dx, h
    qt, et = torch.empty(M, K, dtype=ref.F8, device="cuda"), torch.empty((M + 511) // 512, K, 4, dtype=torch.uint8,
                                                                        device="cuda")
    fp8q.fp8q_quant_act_dual(x, q, s, qt, et)
    last = M // 128 * 128
    rq, rb = ref.token_codes(x[last:, -64:].cpu())
    assert torch.equal(ref.code_values(qt[last:, -64:].contiguous()), rq)
    assert torch.equal(et.cpu()[last // 512, -64:, last // 128 % 4], rb[0, :, 0])
