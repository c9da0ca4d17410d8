"""Cases of the operators of a training step: the RMS norm with the residual's
addition and FP8 output (and its gradient), the quantizer along rows and along
tokens, the two gradients of the block-scaled FP8 product, and the router's
balance loss with its gradient.

``listed()`` names the cases, ``draw(rng)`` gives one more of the same ranges,
``prepare(case, seed)`` makes what a program holds before the call,
``run(state)`` is one call, ``work(case)`` the bytes and operations it cannot
do without, ``exact(case, seed)`` the result in 64 bits.  With ``own`` false
``run`` computes the operators from elementary torch operations in 32 bits;
with ``own`` true it calls this package's entry points.

Shared definitions:

* Row codes: e4m3 codes [M, K] with one fp32 scale, amax / 448, per row and
  128 columns; the scales K-major, [K/128, ceil16(M)], pad slots zero.
* Token codes: e4m3 codes [M, K] with one power of two, 2^(b - 127), per column
  and 128 rows, the least with amax / 2^(b - 127) <= 448 (and b >= 0).  The bytes
  b lie in [ceil(M/512), K, 4]: entry [i // 4, k, i % 4] for rows 128 i and on;
  entries past the last row are zero.
* FP8 weights: e4m3 codes [N, K] with one fp32 scale per 128 x 128 block.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
COEF = 0.01


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # Serving, one token: the norm in front of a projection, latency.
        dict(name="norm_one_token", op="norm", M=1, K=5120, residual=True, y=False),
        # A long prompt, or a training batch whose norm also feeds a router in bf16.
        dict(name="norm_long", op="norm", M=4576, K=5120, residual=True, y=True),
        # The norm's backward pass: a short batch of odd size without a residual's gradient, and a long one with it.
        dict(name="norm_grad_short", op="norm_grad", M=409, K=6144, residual=False),
        dict(name="norm_grad_long", op="norm_grad", M=4576, K=5120, residual=True),
        # Activations kept for the weights' gradient alone (token codes), few and narrow.
        dict(name="dual_short", op="dual", M=409, K=1408, rows=False),
        # A wide gradient, codes both ways from one pass.
        dict(name="dual_long", op="dual", M=4576, K=17408, rows=True),
        # The activations' gradient: a small batch of odd size, and a long one.
        dict(name="dgrad_short", op="dgrad", M=409, N=5120, K=6144),
        dict(name="dgrad_long", op="dgrad", M=4576, N=17408, K=5120),
        # The weights' gradient: an expert-sized matrix over few tokens, and a large one over many.
        dict(name="wgrad_short", op="wgrad", M=409, N=2048, K=1408),
        dict(name="wgrad_long", op="wgrad", M=4576, N=17408, K=5120),
        # The router's backward pass: a small batch, and a long one in bf16 with some experts masked out.
        dict(name="balance_short", op="balance", T=25, E=64, top_k=8, logits="f32", renorm=True, masked=0),
        dict(name="balance_long", op="balance", T=16384, E=160, top_k=6, logits="bf16", renorm=False, masked=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _blocks(rng, lo, hi):
    """A multiple of 128 in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, _log(rng, lo, hi) // 128 * 128))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dual", "dgrad", "wgrad", "balance"])
    if op == "balance":
        E = _log(rng, 8, 256)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, top_k=rng.randint(1, min(8, E)),
                    logits=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0, rng.randint(0, E // 2)]))
    while True:
        c = dict(op=op, M=_log(rng, 1, 4576))
        if op in ("dgrad", "wgrad"):
            c |= dict(N=_blocks(rng, 512, 17408), K=_blocks(rng, 512, 17408))
            if c["N"] * c["K"] <= 17408 * 5120:
                return c
        else:
            c["K"] = _blocks(rng, 256, 17408)
            c["rows" if op == "dual" else "residual"] = rng.random() < 0.6
            if op == "norm":
                c["y"] = rng.random() < 0.4
            if op == "dual" or c["M"] * c["K"] <= 4576 * 5120:
                return c


# --------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 64 + 5)
    return g


def _acts(rows, K, g):
    """bf16 activations: normal, 1% outlier channels of 20 times the size."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20.0
    return x.to(torch.bfloat16)


def _grads(rows, K, g):
    """bf16 gradients: small, tokens of different weight."""
    size = 1e-3 * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    return (torch.randn(rows, K, generator=g, device=DEV) * size).to(torch.bfloat16)


def _weights(N, K, g):
    """(codes [N, K], block scales [N/128, K/128]) of normal weights."""
    w = (torch.randn(N, K, generator=g, device=DEV) * 0.02).view(N // 128, 128, K // 128, 128)
    s = w.abs().amax(dim=(1, 3)) / 448.0
    q = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(N, K), s


def _ceil16(m):
    return (m + 15) // 16 * 16


def _row_codes(x):
    """(codes [M, K], scales [M, K/128]) of rows; 448 as a tensor: by a number the
    GPU would multiply with its rounded reciprocal."""
    v = x.float().view(x.shape[0], -1, 128)
    s = v.abs().amax(dim=2, keepdim=True) / torch.full((1,), 448.0, device=DEV)
    codes = torch.where(s > 0, v / s, v).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(x.shape), s[:, :, 0]


def _k_major(s):
    km = torch.zeros(s.shape[1], _ceil16(s.shape[0]), device=DEV)
    km[:, :s.shape[0]] = s.t()
    return km


def _power(b):
    """2^(b - 127) in fp32 of bytes b < 255, exact (a function of the exponent would round)."""
    return torch.where(b > 0, b.to(torch.int32) << 23, 1 << 22).view(torch.float32)


def _token_codes(x):
    """(codes [M, K], bytes [ceil(M/512), K, 4]) of columns."""
    M, K = x.shape
    blocks, packs = -(-M // 128), -(-M // 512)
    v = torch.zeros(blocks * 128, K, device=DEV)
    v[:M] = x.float()
    v = v.view(blocks, 128, K)
    m, e = torch.frexp(v.abs().amax(dim=1))  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    b = torch.where(m > 0, e - 9 + (m > 0.875) + 127, 0).clamp(min=0)
    codes = (v * _power(254 - b)[:, None, :]).to(torch.float8_e4m3fn)
    packed = torch.zeros(packs * 4, K, dtype=torch.uint8, device=DEV)
    packed[:blocks] = b.to(torch.uint8)
    return codes.view(-1, K)[:M].contiguous(), packed.view(packs, 4, K).transpose(1, 2).contiguous()


def prepare(case, seed):
    c, op = case, case["op"]
    g = _gen(seed)
    s = {"case": c}
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "balance":
        T, E, k = c["T"], c["E"], c["top_k"]
        logits = torch.randn(T, E, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(E, generator=g, device=DEV)
        logits[:, torch.randperm(E, generator=g, device=DEV)[:c["masked"]]] = -math.inf
        s["logits"] = logits.to(torch.float32 if c["logits"] == "f32" else torch.bfloat16)
        best, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        s["ids"] = torch.where(best > -math.inf, ids, -1)[:, :k].to(torch.int32).contiguous()
        s["dweights"] = torch.randn(T, k, generator=g, device=DEV) * 1e-2
        s["dloss"] = torch.ones(1, device=DEV)
        s["counts"] = new(E + 1, dtype=torch.int32)
        s["prob"], s["loss"] = new(E, dtype=torch.float32), new(1, dtype=torch.float32)
        s["dlogits"] = torch.empty_like(s["logits"])
        return s
    M, K = c["M"], c["K"]
    if op == "norm":
        s["x"] = _acts(M, K, g)
        s["residual"] = _acts(M, K, g) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
        s["h"] = new(M, K) if c["residual"] else None
        s["y"] = new(M, K) if c["y"] else None
        s["q"] = new(M, K, dtype=torch.float8_e4m3fn)
        s["scale_km"] = new(K // 128, _ceil16(M), dtype=torch.float32)
        s["rstd"] = new(M, dtype=torch.float32)
    elif op == "norm_grad":
        s["h"] = _acts(M, K, g)
        s["dy"] = _grads(M, K, g)
        s["dh"] = _grads(M, K, g) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
        s["dx"] = new(M, K)
        s["dweight"] = new(K, dtype=torch.float32)
    elif op == "dual":
        s["x"] = _grads(M, K, g) if c["rows"] else _acts(M, K, g)
        s["q"] = new(M, K, dtype=torch.float8_e4m3fn) if c["rows"] else None
        s["scale_km"] = new(K // 128, _ceil16(M), dtype=torch.float32) if c["rows"] else None
        s["q_tok"] = new(M, K, dtype=torch.float8_e4m3fn)
        s["exp_tok"] = new(-(-M // 512), K, 4, dtype=torch.uint8)
    elif op == "dgrad":
        s["dy"], scale = _row_codes(_grads(M, c["N"], g))
        s["dy_scale_km"] = _k_major(scale)
        s["w"], s["w_scale"] = _weights(c["N"], K, g)
        s["dx"] = new(M, K)
    else:
        s["dy_tok"], s["dy_exp"] = _token_codes(_grads(M, c["N"], g))
        s["x_tok"], s["x_exp"] = _token_codes(_acts(M, K, g))
        s["dw"] = new(c["N"], K)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _work_buffer(s, query, *sizes):
    """The workspace a program keeps between calls of one size."""
    if "work" not in s:
        nbytes = query(*sizes)
        s["work"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return s["work"]


def _own_norm(s):
    import w8a8_fp8_block_amd as fp8q
    fp8q.fp8q_add_rmsnorm_quant(s["x"], s["residual"], s["weight"], s["h"], s["y"], s["q"], None, s["scale_km"],
                                s["rstd"], EPS)
    return {n: s[n] for n in ("h", "y", "q", "scale_km", "rstd")}


def _own_norm_grad(s):
    import w8a8_fp8_block_amd as fp8q
    work = _work_buffer(s, fp8q.fp8q_add_rmsnorm_grad_workspace_bytes, *s["h"].shape)
    fp8q.fp8q_add_rmsnorm_grad(s["dy"], s["dh"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], work)
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_dual(s):
    import w8a8_fp8_block_amd as fp8q
    fp8q.fp8q_quant_act_dual(s["x"], s["q"], s["scale_km"], s["q_tok"], s["exp_tok"])
    return {n: s[n] for n in ("q", "scale_km", "q_tok", "exp_tok")}


def _own_dgrad(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, fp8q.fp8q_gemm_dgrad_workspace_bytes, c["M"], c["N"], c["K"])
    fp8q.fp8q_gemm_dgrad(s["dy"], s["dy_scale_km"], s["w"], s["w_scale"], s["dx"], work)
    return s["dx"]


def _own_wgrad(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, fp8q.fp8q_gemm_wgrad_workspace_bytes, c["M"], c["N"], c["K"])
    fp8q.fp8q_gemm_wgrad(s["dy_tok"], s["dy_exp"], s["x_tok"], s["x_exp"], s["dw"], work)
    return s["dw"]


def _own_balance(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, fp8q.fp8q_moe_balance_workspace_bytes, c["T"], c["E"])
    fp8q.fp8q_moe_balance(s["logits"], s["ids"], s["counts"], s["prob"], s["loss"], work, COEF)
    fp8q.fp8q_moe_route_grad(s["logits"], s["ids"], s["dweights"], s["counts"], s["dloss"], s["dlogits"],
                             renormalize=c["renorm"], coef=COEF)
    return {n: s[n] for n in ("counts", "prob", "loss", "dlogits")}


_run_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "dual": _own_dual, "dgrad": _own_dgrad,
            "wgrad": _own_wgrad, "balance": _own_balance}


# ------------------------------------------------------- the plain forms
def _plain_norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    v = h.float()
    rstd = 1.0 / torch.sqrt(v.square().mean(dim=1) + EPS)
    y = v * rstd[:, None] * s["weight"].float()
    q, scale = _row_codes(y)
    return {"h": None if s["residual"] is None else h, "y": y.to(torch.bfloat16) if s["case"]["y"] else None,
            "q": q, "scale_km": _k_major(scale), "rstd": rstd}


def _plain_norm_grad(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * xhat).sum(dim=0)}


def _plain_dual(s):
    out = {"q": None, "scale_km": None}
    if s["case"]["rows"]:
        out["q"], scale = _row_codes(s["x"])
        out["scale_km"] = _k_major(scale)
    out["q_tok"], out["exp_tok"] = _token_codes(s["x"])
    return out


def _plain_dgrad(s):
    M, N = s["dy"].shape
    K = s["w"].shape[1]
    dy = s["dy"].float().view(M, -1, 128) * s["dy_scale_km"][:, :M].t()[:, :, None]
    w = s["w"].float().view(N // 128, 128, K // 128, 128) * s["w_scale"][:, None, :, None]
    return (dy.view(M, N) @ w.view(N, K)).to(torch.bfloat16)


def _token_values(q, b):
    """Token codes and their bytes -> fp32."""
    M, K = q.shape
    scale = _power(b.transpose(1, 2).reshape(-1, K))
    return q.float() * scale.repeat_interleave(128, dim=0)[:M]


def _plain_wgrad(s):
    dy, x = _token_values(s["dy_tok"], s["dy_exp"]), _token_values(s["x_tok"], s["x_exp"])
    return (dy.t() @ x).to(torch.bfloat16)


def _plain_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["top_k"]
    l = s["logits"].float()
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    chosen = torch.zeros(T, E + 1, device=DEV).scatter_(1, torch.where(s["ids"] < 0, E, s["ids"]).long(), 1.0)[:, :E]
    d = torch.zeros(T, E + 1, device=DEV).scatter_(1, torch.where(s["ids"] < 0, E, s["ids"]).long(), s["dweights"])[:, :E]
    n = (total > 0).sum()
    counts = chosen.sum(dim=0)
    prob = p.sum(dim=0) / n
    f = counts / (n * k)
    loss = COEF * E * (f * prob).sum()
    w = p if not c["renorm"] else e * chosen / torch.where(total > 0, (e * chosen).sum(dim=1, keepdim=True), 1.0)
    dl = w * (d - (w * d).sum(dim=1, keepdim=True))
    share = COEF * E * f / n * s["dloss"]
    dl = dl + p * (share - (p * share).sum(dim=1, keepdim=True))
    return {"counts": torch.cat([counts, n[None]]).to(torch.int32), "prob": prob, "loss": loss[None],
            "dlogits": dl.to(s["logits"].dtype)}


_run_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dual": _plain_dual, "dgrad": _plain_dgrad,
              "wgrad": _plain_wgrad, "balance": _plain_balance}


# ------------------------------------------------------------------ the work
def work(case):
    c, op = case, case["op"]
    if op == "balance":
        T, E, k = c["T"], c["E"], c["top_k"]
        return {"bytes": 2 * T * E * (4 if c["logits"] == "f32" else 2) + 8 * T * k + 8 * E, "flops": 12 * T * E}
    M, K = c["M"], c["K"]
    if op == "norm":
        return {"bytes": M * K * (3 + 4 * c["residual"] + 2 * c["y"]) + 4 * M * (K // 128) + 2 * K + 4 * M, "flops": 6 * M * K}
    if op == "norm_grad":
        return {"bytes": M * K * (6 + 2 * c["residual"]) + 6 * K + 4 * M, "flops": 10 * M * K}
    if op == "dual":
        blocks = (M + 127) // 128
        return {"bytes": M * K * (3 + c["rows"]) + 4 * c["rows"] * M * (K // 128) + blocks * K, "flops": 6 * M * K}
    N = c["N"]
    if op == "dgrad":
        return {"bytes": M * N + N * K + 2 * M * K + 4 * M * (N // 128), "flops": 2 * M * N * K}
    return {"bytes": M * N + M * K + 2 * N * K + (M + 127) // 128 * (N + K), "flops": 2 * M * N * K}


# ------------------------------------------------------ the result in 64 bits
def _two_to(e):
    """2^e in 64 bits, exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_code(x):
    """Nearest e4m3 value, ties to even, of float64 values of at most 448."""
    _, e = torch.frexp(x)
    step = _two_to((e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_norm(s):
    h = s["x"].double() if s["residual"] is None else (s["x"].double() + s["residual"].double()).bfloat16().double()
    rstd = (h.pow(2).sum(1) / h.shape[1] + EPS).pow(-0.5)
    y = h * rstd[:, None] * s["weight"].double()
    groups = y.view(y.shape[0], -1, 128)
    scale = groups.abs().amax(dim=2) / 448.0
    km = torch.zeros(scale.shape[1], _ceil16(scale.shape[0]), dtype=torch.float64, device=DEV)
    km[:, :scale.shape[0]] = scale.t()
    # the codes' own target: y over its scale, before the rounding to 8 bits
    q = (groups / torch.where(scale > 0, scale, 1.0)[:, :, None]).view(y.shape)
    return {"h": None if s["residual"] is None else h, "y": y if s["case"]["y"] else None, "q": q, "scale_km": km,
            "rstd": rstd}


def _exact_norm_grad(s):
    h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    g = dy * s["weight"].double()
    dx = r * g - h * r.pow(3) * ((g * h).sum(1, keepdim=True) / h.shape[1])
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"dx": dx, "dweight": (dy * h * r).sum(0)}


def _exact_dual(s):
    x = s["x"].double()
    M, K = x.shape
    out = {"q": None, "scale_km": None}
    if s["case"]["rows"]:
        v = x.view(M, -1, 128)
        scale = (v.abs().amax(dim=2) / 448.0).float().double()  # a 32-bit number by definition, as is x / scale
        km = torch.zeros(K // 128, _ceil16(M), dtype=torch.float64, device=DEV)
        km[:, :M] = scale.t()
        out["scale_km"] = km
        out["q"] = _nearest_code((v / torch.where(scale > 0, scale, 1.0)[:, :, None]).float().double()).view(M, K)
    packed = torch.zeros(-(-M // 512), K, 4, dtype=torch.uint8, device=DEV)
    q = torch.empty_like(x)
    for i in range(-(-M // 128)):
        rows = x[128 * i:128 * i + 128]
        amax = rows.abs().amax(dim=0)
        e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448.0))
        e = torch.where(448.0 * _two_to(e - 1) >= amax, e - 1, e)  # the logarithm's own rounding
        e = torch.where(amax > 0, e, -127.0).clamp(min=-127.0)
        packed[i // 4, :, i % 4] = (e + 127).to(torch.uint8)
        q[128 * i:128 * i + 128] = _nearest_code(rows * _two_to(-e))
    out["q_tok"], out["exp_tok"] = q, packed
    return out


def _exact_dgrad(s):
    M, N = s["dy"].shape
    K = s["w"].shape[1]
    out = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for i in range(0, N, 1024):  # pieces of the sum
        scale = s["dy_scale_km"][i // 128:(i + 1024) // 128, :M].double().t().repeat_interleave(128, 1)
        block = s["w_scale"][i // 128:(i + 1024) // 128].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        out += (s["dy"][:, i:i + 1024].double() * scale) @ (s["w"][i:i + 1024].double() * block)
    return out


def _exact_wgrad(s):
    M, N = s["dy_tok"].shape
    K = s["x_tok"].shape[1]
    out = torch.zeros(N, K, dtype=torch.float64, device=DEV)
    for i in range(-(-M // 128)):
        rows = slice(128 * i, 128 * i + 128)
        part = s["dy_tok"][rows].double().t().contiguous() @ s["x_tok"][rows].double()
        eb, ek = (_two_to(s[n][i // 4, :, i % 4].long() - 127) for n in ("dy_exp", "x_exp"))
        out += part * eb[:, None] * ek[None, :]
    return out


def _exact_balance(s):
    c = s["case"]
    l = s["logits"].double()
    T, E = l.shape
    p = torch.softmax(l, dim=1)
    ids = s["ids"].long()
    some = ids >= 0
    counts = torch.bincount(ids[some], minlength=E)
    prob, f = p.mean(0), counts.double() / (T * c["top_k"])
    d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    rows = torch.arange(T, device=DEV)[:, None].expand_as(ids)
    d[rows[some], ids[some]] = s["dweights"].double()[some]
    if c["renorm"]:
        keep = torch.full((T, E), -math.inf, dtype=torch.float64, device=DEV)
        keep[rows[some], ids[some]] = 0.0
        w = torch.softmax(l + keep, dim=1)
    else:
        w = p
    share = COEF * E * f / T * s["dloss"].double()
    dl = w * d - w * (w * d).sum(1, keepdim=True) + p * share - p * (p @ share)[:, None]
    return {"counts": torch.cat([counts, counts.new_tensor([T])]), "prob": prob, "loss": COEF * E * (f @ prob)[None],
            "dlogits": dl}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "dual": _exact_dual, "dgrad": _exact_dgrad,
            "wgrad": _exact_wgrad, "balance": _exact_balance}[case["op"]](s)
