"""Plain 64-bit forms (torch, on the CPU) of the operators of a training step,
written from their formulas.  Imported only by tests."""
from __future__ import annotations

import math

import torch

F8 = torch.float8_e4m3fn


def code_values(q):
    """e4m3 codes -> float64."""
    return q.cpu().view(torch.uint8).view(F8).double()


def norm(x, residual, weight, eps):
    """(h, rstd, y, scale, y / scale) in float64; h is rounded to bf16 first."""
    h = x if residual is None else (x.double() + residual.double()).to(torch.bfloat16)
    v = h.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    y = v * rstd[:, None] * weight.double()
    g = y.view(y.shape[0], -1, 128)
    scale = g.abs().amax(2) / 448.0
    q = (g / torch.where(scale > 0, scale, 1.0)[:, :, None]).view(y.shape)
    return h, rstd, y, scale, q


def norm_grad(dy, dh, h, weight, rstd):
    """(dx, dweight) and the sums of magnitudes that bound their fp32 errors."""
    xhat = h.double() * rstd.double()[:, None]
    g = dy.double() * weight.double()
    r = rstd.double()[:, None]
    dx = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
    size = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    t = dy.double() * xhat
    return dx, t.sum(0), size, t.abs().sum(0)


def token_codes(x):
    """(codes' values float64 [M,K], bytes [ceil(M/512),K,4]) of finite x."""
    M, K = x.shape
    q = torch.empty(M, K, dtype=torch.float64)
    b = torch.zeros(-(-M // 512), K, 4, dtype=torch.uint8)
    for i in range(-(-M // 128)):
        v = x[128 * i:128 * i + 128].double()
        amax = v.abs().amax(0)
        for k in range(K):
            a = float(amax[k])
            e = -127
            if a:
                m, e = math.frexp(a)  # a = m * 2^e, 448 = 0.875 * 2^9
                e = max(e - 9 + (m > 0.875), -127)
            b[i // 4, k, i % 4] = e + 127
            q[128 * i:128 * i + 128, k] = v[:, k] * 2.0 ** -e
    return nearest_code(q), b


def nearest_code(x):
    """Nearest e4m3 value, ties to even, of float64 values of at most 448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def dgrad(dy, dy_scale, w, w_scale):
    """codes' values [M,N], [N,K] and scales [M,N/128], [N/128,K/128] -> [M,K]."""
    a = dy * dy_scale.double().repeat_interleave(128, 1)
    b = w * w_scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return a @ b


def wgrad(dy, dy_exp, x, x_exp):
    """codes' values [M,N], [M,K] and bytes -> [N,K]."""
    out = torch.zeros(dy.shape[1], x.shape[1], dtype=torch.float64)
    for i in range(-(-dy.shape[0] // 128)):
        r = slice(128 * i, 128 * i + 128)
        ey, ex = (torch.exp2(b[i // 4, :, i % 4].double() - 127.0) for b in (dy_exp, x_exp))
        out += (dy[r].t() @ x[r]) * ey[:, None] * ex[None, :]
    return out


def clean(logits):
    l = logits.double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    return l.clamp(max=float(torch.finfo(torch.float32).max))


def softmax(l):
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top > -math.inf, top, 0.0))
    e = torch.where(l > -math.inf, e, 0.0)
    s = e.sum(1, keepdim=True)
    return torch.where(s > 0, e / torch.where(s > 0, s, 1.0), 0.0), (s[:, 0] > 0)


def balance(logits, ids, coef):
    """(counts with n behind them, prob, loss, p)."""
    T, E = logits.shape
    p, some = softmax(clean(logits))
    n = int(some.sum())
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    prob = p.sum(0) / max(n, 1)
    loss = coef * E * float((counts / (max(n, 1) * ids.shape[1]) * prob).sum())
    return torch.cat([counts, torch.tensor([n])]), prob, loss, p


def route_grad(logits, ids, dweights, counts, dloss, coef, renormalize, top_k):
    """dlogits, and the magnitudes that bound its fp32 error."""
    T, E = logits.shape
    l = clean(logits)
    p, _ = softmax(l)
    out, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    if counts is not None and int(counts[E]):
        n = float(counts[E])
        c = dloss * coef * E * counts[:E].double() / (n * top_k) / n
        out += p * (c - (p * c).sum(1, keepdim=True))
        size += p * (c.abs() + (p * c.abs()).sum(1, keepdim=True))
    if ids is not None:
        for t in range(T):
            slots = [j for j in range(ids.shape[1]) if 0 <= int(ids[t, j]) < E]
            e = [int(ids[t, j]) for j in slots]
            d = dweights[t].double()[slots]
            if not e:
                continue
            if renormalize:
                le = l[t, e]
                if not bool((le > -math.inf).any()):
                    continue
                w = torch.where(le > -math.inf, torch.exp(le - le.max()), 0.0)
                w = w / w.sum()
                dl, sz = w * (d - (w * d).sum()), w * (d.abs() + (w * d.abs()).sum())
                out[t].index_add_(0, torch.tensor(e), dl)
                size[t].index_add_(0, torch.tensor(e), sz)
            else:
                full = torch.zeros(E, dtype=torch.float64).index_add_(0, torch.tensor(e), d)
                out[t] += p[t] * (full - (p[t] * full).sum())
                size[t] += p[t] * (full.abs() + (p[t] * full.abs()).sum())
    return out, size
