"""Cases of the routed and per-request operators: expert routing, matrix
products grouped by expert, the expert FFN, and low-rank adapters beside a
shared FP8 projection.

``listed()`` names the cases, ``draw(rng)`` gives one more of the same
ranges, ``prepare(case, seed)`` makes what a serving program holds before the
call, ``run(state)`` is one call, ``work(case)`` the bytes and operations it
cannot do without, ``exact(case, seed)`` the result in 64 bits.  With ``own``
false ``run`` computes the operators from elementary torch operations in 32
bits; with ``own`` true it calls this package's entry points.

Shared definitions:

* FP8 activations: e4m3 codes of bf16 rows with one fp32 scale, amax / 448,
  per row and 128-wide group; the scales K-major, [K/128, ceil16(rows)].
* FP8 weights: e4m3 codes with one fp32 scale per 128 x 128 block.
* Routing: slot s = t * top_k + j is the j-th choice of token t.  ``order``
  lists the slots sorted by expert (stable), ``pos`` is its inverse and
  ``offsets[e] .. offsets[e + 1]`` are the sorted rows of expert e.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # One decode step's routing for a small batch: launch latency.
        dict(name="route_decode", op="route", T=16, E=128, top_k=8, logits="f32", renorm=True, masked=0),
        # A long prompt's routing, bf16 router output, some experts masked out,
        # weights taken from the softmax over all experts.
        dict(name="route_prefill", op="route", T=4576, E=160, top_k=6, logits="bf16", renorm=False, masked=9),
        # A single token through a few experts: latency.
        dict(name="grouped_one_token", op="grouped", T=1, E=16, top_k=4, K=1024, N=2048, gather=True),
        # A decode batch: every expert holds a few rows, the weights stream once.
        dict(name="grouped_decode", op="grouped", T=25, E=64, top_k=8, K=5120, N=2048, gather=True),
        # A short prompt in odd numbers: some tens of rows an expert, rows already in expert order.
        dict(name="grouped_short_prompt", op="grouped", T=409, E=40, top_k=5, K=1408, N=5120, gather=False),
        # A long prompt: hundreds of rows an expert.
        dict(name="grouped_prefill", op="grouped", T=4576, E=64, top_k=8, K=5120, N=2048, gather=True),
        # The expert FFN for a decode batch and for a prompt.
        dict(name="ffn_decode", op="ffn", T=16, E=64, top_k=6, H=5120, I=1408),
        dict(name="ffn_prefill", op="ffn", T=4576, E=32, top_k=4, H=5120, I=2048),
        # One token with its own adapter beside the projection.
        dict(name="lora_one_token", op="lora", M=1, K=5120, N=6144, adapters=4, rank=16, requests=1, bare=0),
        # A decode batch, each row of another request with its own adapter.
        dict(name="lora_decode", op="lora", M=25, K=5120, N=17408, adapters=32, rank=64, requests=25, bare=3),
        # Two prompts and decode rows in one batch of odd size.
        dict(name="lora_mixed", op="lora", M=1168, K=5120, N=6144, adapters=8, rank=24, requests=19, bare=2),
        # Long prompts of a few requests.
        dict(name="lora_prefill", op="lora", M=4576, K=17408, N=5120, adapters=4, rank=32, requests=5, bare=1),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + 1 if v == 24 * 128 else v


def _blocks(rng, lo, hi):
    """A multiple of 128 in [lo, hi], spread over its logarithm."""
    v = max(lo, min(hi, _log(rng, lo, hi) // 128 * 128))
    return v + 128 if v == 24 * 128 else v


def draw(rng):
    op = rng.choice(["route", "grouped", "ffn", "lora"])
    if op == "route":
        E = _log(rng, 8, 256)
        return dict(op=op, T=_log(rng, 1, 4576), E=E, top_k=rng.randint(1, min(8, E)),
                    logits=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0, rng.randint(0, E - 1)]))
    if op == "lora":
        while True:
            c = dict(op=op, M=_log(rng, 1, 4576), K=_blocks(rng, 512, 17408), N=_blocks(rng, 512, 17408),
                     adapters=_log(rng, 1, 64), rank=8 * rng.randint(1, 16), requests=0, bare=0)
            c["requests"] = rng.randint(1, min(c["M"], 64))
            c["bare"] = rng.randint(0, c["requests"] // 2)
            if c["K"] * c["N"] <= 17408 * 5120 and c["adapters"] * c["rank"] <= 2048:
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 4576), E=_log(rng, 4, 64), top_k=rng.randint(1, 8))
        c["top_k"] = min(c["top_k"], c["E"])
        if op == "grouped":
            c |= dict(K=_blocks(rng, 512, 5120), N=_blocks(rng, 512, 5120), gather=rng.random() < 0.7)
            if c["T"] * c["top_k"] * c["K"] * c["N"] <= 36608 * 5120 * 2048 and c["E"] * c["K"] * c["N"] <= 64 * 5120 * 2048:
                return c
        else:
            c |= dict(H=_blocks(rng, 512, 5120), I=_blocks(rng, 256, 2048))
            if c["T"] * c["top_k"] * c["H"] * c["I"] <= 18304 * 5120 * 2048 and c["E"] * c["H"] * c["I"] <= 64 * 5120 * 1408:
                return c


# --------------------------------------------------------------- the inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 64 + salt)
    return g


def _acts(rows, K, g):
    """bf16 activations: normal, 1% outlier channels of 20 times the size."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20.0
    return x.to(torch.bfloat16)


def _weights(N, K, g):
    """(codes [N, K], block scales [N/128, K/128]) of normal weights."""
    w = (torch.randn(N, K, generator=g, device=DEV) * 0.02).view(N // 128, 128, K // 128, 128)
    s = w.abs().amax(dim=(1, 3)) / 448.0
    q = (w / s[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(N, K), s


def _expert_weights(E, N, K, g):
    both = [_weights(N, K, g) for _ in range(E)]
    q = torch.stack([q.view(torch.uint8) for q, _ in both]).view(torch.float8_e4m3fn)
    return q, torch.stack([s for _, s in both])


def _routing(T, E, top_k, seed):
    """Choices of T tokens: experts differ in popularity, a token's are distinct."""
    r = np.random.default_rng(seed)
    liking = r.normal(0.0, 0.5, E)
    ids = np.argsort(-(liking + r.gumbel(size=(T, E))), axis=1)[:, :top_k]
    return np.ascontiguousarray(ids).astype(np.int32)


def _plan(ids, E):
    """(order, pos, offsets, rows of the largest group) of choices [T, top_k], on the host."""
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    pos = np.empty_like(order)
    pos[order] = np.arange(flat.size, dtype=np.int32)
    counts = np.bincount(flat, minlength=E)
    return order, pos, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), int(counts.max())


def _ceil16(m):
    return (m + 15) // 16 * 16


def _adapter_of_rows(c, seed):
    """Adapter of each row: requests of contiguous rows, `bare` of them without one."""
    r = np.random.default_rng(seed)
    cuts = np.sort(r.choice(np.arange(1, c["M"]), c["requests"] - 1, replace=False)) if c["requests"] > 1 else np.zeros(0, int)
    rows = np.diff(np.concatenate([[0], cuts, [c["M"]]]))
    who = r.permutation(np.arange(c["requests"]) % c["adapters"])
    who[r.permutation(c["requests"])[:c["bare"]]] = -1
    return np.repeat(who, rows).astype(np.int32)


def prepare(case, seed):
    c, op = case, case["op"]
    g = _gen(seed, 1)
    s = {"case": c}
    if op == "route":
        T, E, k = c["T"], c["E"], c["top_k"]
        logits = torch.randn(T, E, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(E, generator=g, device=DEV)
        off = torch.randperm(E, generator=g, device=DEV)[:c["masked"]]
        logits[:, off] = -math.inf
        s["logits"] = logits.to(torch.float32 if c["logits"] == "f32" else torch.bfloat16)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(T, k, device=DEV)
        s["order"], s["pos"] = (torch.empty(T * k, dtype=torch.int32, device=DEV) for _ in range(2))
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        return s
    if op == "lora":
        M, K, N, n, R = c["M"], c["K"], c["N"], c["adapters"], c["rank"]
        s["x"] = _acts(M, K, g)
        s["w"], s["w_scale"] = _weights(N, K, g)
        s["lora_a"] = (torch.randn(n, R, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
        s["lora_b"] = (torch.randn(n, N, R, generator=g, device=DEV) * 0.05).to(torch.bfloat16)
        s["lora_scale"] = 0.5 + 1.5 * torch.rand(n, generator=g, device=DEV)
        s["ids"] = torch.from_numpy(_adapter_of_rows(c, seed)).to(DEV)
        s["out"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        s["act_q"] = torch.empty(M, K, dtype=torch.uint8, device=DEV)
        s["act_scale"] = torch.empty(M, K // 128, device=DEV)
        s["act_scale_km"] = torch.empty(K // 128, _ceil16(M), device=DEV)
        return s
    T, E, k = c["T"], c["E"], c["top_k"]
    ids = _routing(T, E, k, seed)
    order, pos, offsets, s["rows_max"] = _plan(ids, E)
    s["order"], s["pos"], s["offsets"] = (torch.from_numpy(a).to(DEV) for a in (order, pos, offsets))
    if op == "grouped":
        K, N = c["K"], c["N"]
        x = _acts(T if c["gather"] else T * k, K, g)
        rows = x.shape[0]
        grouped = x.float().view(rows, K // 128, 128)
        scale = grouped.abs().amax(dim=2) / 448.0
        s["a"] = (grouped / scale[:, :, None]).to(torch.float8_e4m3fn).view(rows, K)
        s["a_scale_km"] = torch.zeros(K // 128, _ceil16(rows), device=DEV)
        s["a_scale_km"][:, :rows] = scale.t()
        s["w"], s["w_scale"] = _expert_weights(E, N, K, g)
        s["out"] = torch.empty(T * k, N, dtype=torch.bfloat16, device=DEV)
        return s
    H, I = c["H"], c["I"]
    s["x"] = _acts(T, H, g)
    s["w_gate"], s["w_gate_scale"] = _expert_weights(E, I, H, g)
    s["w_up"], s["w_up_scale"] = _expert_weights(E, I, H, g)
    s["w_down"], s["w_down_scale"] = _expert_weights(E, H, I, g)
    s["weights"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), dim=1)
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _work_buffer(s, nbytes):
    """The workspace a serving program keeps between calls of one size."""
    if "work" not in s:
        s["work"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return s["work"]


def _own_route(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, 0 if "work" in s else fp8q.fp8q_moe_route_workspace_bytes(c["T"], c["E"], c["top_k"]))
    fp8q.fp8q_moe_route(s["logits"], s["ids"], s["weights"], s["order"], s["pos"], s["offsets"], work,
                        renormalize=c["renorm"])
    return {n: s[n] for n in ("ids", "weights", "order", "pos", "offsets")}


def _own_grouped(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    fp8q.fp8q_gemm_grouped(s["a"], s["a_scale_km"], s["w"], s["w_scale"], s["offsets"], s["out"],
                           order=s["order"] if c["gather"] else None, top_k=c["top_k"])
    return s["out"]


def _own_ffn(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, 0 if "work" in s else
                        fp8q.fp8q_moe_ffn_workspace_bytes(c["T"], c["E"], c["top_k"], c["H"], c["I"]))
    fp8q.fp8q_moe_ffn(s["x"], s["weights"], s["order"], s["pos"], s["offsets"], s["w_gate"], s["w_gate_scale"],
                      s["w_up"], s["w_up_scale"], s["w_down"], s["w_down_scale"], s["out"], work)
    return s["out"]


def _own_lora(s):
    import w8a8_fp8_block_amd as fp8q
    c = s["case"]
    work = _work_buffer(s, 0 if "work" in s else
                        fp8q.fp8q_proj_lora_workspace_bytes(c["M"], c["N"], c["K"], c["rank"]))
    fp8q.fp8q_proj_lora(s["x"], s["w"], s["w_scale"], s["lora_a"], s["lora_b"], s["lora_scale"], s["ids"], s["out"],
                        s["act_q"], s["act_scale"], s["act_scale_km"], work)
    return s["out"]


_run_own = {"route": _own_route, "grouped": _own_grouped, "ffn": _own_ffn, "lora": _own_lora}


# ------------------------------------------------------- the plain forms
def _dequant_weights(w, s):
    """FP8 weights [..., N, K] with block scales -> fp32."""
    N, K = w.shape[-2:]
    blocks = w.float().view(*w.shape[:-2], N // 128, 128, K // 128, 128)
    return (blocks * s[..., :, None, :, None]).view(w.shape)


def _quantized(x):
    """bf16 rows -> the fp32 values their FP8 codes and scales stand for (448 as a
    tensor: by a number the GPU would multiply with its rounded reciprocal)."""
    v = x.float().view(*x.shape[:-1], -1, 128)
    s = v.abs().amax(dim=-1, keepdim=True) / torch.full((1,), 448.0, device=DEV)
    codes = torch.where(s > 0, v / s, v).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (codes.float() * s).view(x.shape)


def _padded_rows(offsets, rows_max):
    """(sorted row of each place of each group [E, rows_max], whether the group reaches it)."""
    p = offsets[:-1, None].long() + torch.arange(rows_max, device=DEV)
    return p, p < offsets[1:, None]


def _grouped_product(rows, inside, w):
    """[E, rows_max, K] x [E, N, K] -> [E, rows_max, N] (places outside a group are zero)."""
    return torch.bmm(rows * inside[:, :, None], w.transpose(1, 2))


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["top_k"]
    l = s["logits"].float()
    best, ids = torch.sort(l, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    taken = best > -math.inf
    top = torch.where(taken[:, :1], best[:, :1], 0.0)
    e = torch.exp(best - top) * taken
    total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(l - top).sum(1, keepdim=True)
    weights = e / torch.where(taken[:, :1], total, 1.0)
    ids = torch.where(taken, ids, -1).to(torch.int32)
    key = torch.where(taken, ids, E).reshape(-1)
    order = torch.sort(key, stable=True)[1].to(torch.int32)
    pos = torch.empty_like(order).scatter_(0, order.long(), torch.arange(T * k, dtype=torch.int32, device=DEV))
    counts = torch.zeros(E + 1, device=DEV, dtype=torch.int32).scatter_add_(0, key.long(), torch.ones_like(order))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:E], 0, dtype=torch.int32)])
    return {"ids": ids, "weights": weights, "order": order, "pos": pos, "offsets": offsets}


def _plain_grouped(s):
    c = s["case"]
    rows = c["T"] if c["gather"] else c["T"] * c["top_k"]
    scale = s["a_scale_km"][:, :rows].t()
    a = (s["a"].float().view(rows, -1, 128) * scale[:, :, None]).view(rows, -1)
    p, inside = _padded_rows(s["offsets"], s["rows_max"])
    at = torch.where(inside, p, 0)
    src = s["order"][at].long() // c["top_k"] if c["gather"] else at
    y = _grouped_product(a[src], inside, _dequant_weights(s["w"], s["w_scale"]))
    return y[inside].to(torch.bfloat16)  # groups follow one another: the places inside, in order, are the sorted rows


def _plain_ffn(s):
    c = s["case"]
    p, inside = _padded_rows(s["offsets"], s["rows_max"])
    src = s["order"][torch.where(inside, p, 0)].long() // c["top_k"]
    x = _quantized(s["x"])[src]
    gate = _grouped_product(x, inside, _dequant_weights(s["w_gate"], s["w_gate_scale"])).bfloat16().float()
    up = _grouped_product(x, inside, _dequant_weights(s["w_up"], s["w_up_scale"])).bfloat16().float()
    h = _quantized((gate / (1.0 + torch.exp(-gate)) * up).bfloat16())
    y = _grouped_product(h, inside, _dequant_weights(s["w_down"], s["w_down_scale"]))[inside]
    slots = y[s["pos"].long()].view(c["T"], c["top_k"], -1)
    return (slots * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)


def _plain_lora(s):
    c = s["case"]
    n, R = c["adapters"], c["rank"]
    base = _quantized(s["x"]) @ _dequant_weights(s["w"], s["w_scale"]).t()
    v = s["x"].float() @ s["lora_a"].float().view(n * R, -1).t()
    mine = s["ids"][:, None] == torch.arange(n, device=DEV, dtype=torch.int32)
    v = v.view(-1, n, R) * (mine * s["lora_scale"])[:, :, None]
    b = s["lora_b"].float().transpose(0, 1).reshape(-1, n * R)
    return (base + v.view(-1, n * R) @ b.t()).to(torch.bfloat16)


_run_plain = {"route": _plain_route, "grouped": _plain_grouped, "ffn": _plain_ffn, "lora": _plain_lora}


# ------------------------------------------------------------------ the work
def _active(T, E, top_k):
    """Experts that T tokens reach, at one seed of the routing."""
    return len(np.unique(_routing(T, E, top_k, 0)))


def work(case):
    c, op = case, case["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["top_k"]
        return {"bytes": T * E * (4 if c["logits"] == "f32" else 2) + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if op == "lora":
        M, K, N, R = c["M"], c["K"], c["N"], c["rank"]
        used = min(c["adapters"], c["requests"] - c["bare"])
        return {"bytes": N * K + 4 * (N // 128) * (K // 128) + 2 * used * R * (K + N) + 2 * M * (K + N),
                "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    R = c["T"] * c["top_k"]
    experts = _active(c["T"], c["E"], c["top_k"])
    if op == "grouped":
        K, N = c["K"], c["N"]
        rows = c["T"] if c["gather"] else R
        return {"bytes": experts * N * K + rows * K + 2 * R * N, "flops": 2 * R * N * K}
    return {"bytes": 3 * experts * c["H"] * c["I"] + 4 * c["T"] * c["H"], "flops": 6 * R * c["H"] * c["I"]}


# ------------------------------------------------------ the result in 64 bits
def _code_values(x):
    """Nearest e4m3 value, ties to even, of float64 values of at most 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _row_values(x):
    """bf16 rows as FP8 holds them: amax / 448 and x / scale are 32-bit numbers by definition."""
    v = x.double().view(x.shape[0], -1, 128)
    s = (v.abs().amax(dim=2, keepdim=True) / 448.0).float().double()
    codes = _code_values((v / torch.where(s > 0, s, 1.0)).float().double())
    return (codes * s).view(x.shape)


def _block_values(q, s):
    return q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_route(s):
    c = s["case"]
    l = s["logits"].double().cpu().numpy()
    ids = np.argsort(-l, axis=1, kind="stable")[:, :c["top_k"]].astype(np.int32)
    best = np.take_along_axis(l, ids.astype(np.int64), 1)
    e = np.exp(best - best[:, :1])
    total = e.sum(1, keepdims=True) if c["renorm"] else np.exp(l - best[:, :1]).sum(1, keepdims=True)
    ids[best == -math.inf] = -1
    flat = np.where(ids < 0, c["E"], ids).reshape(-1)
    order, pos, offsets, _ = _plan(flat, c["E"] + 1)
    return {"ids": ids, "weights": e / total, "order": order, "pos": pos, "offsets": offsets[:c["E"] + 1]}


def _exact_grouped(s):
    c = s["case"]
    R = c["T"] * c["top_k"]
    out = torch.zeros(R, c["N"], dtype=torch.float64, device=DEV)
    src = s["order"].long() // c["top_k"] if c["gather"] else torch.arange(R, device=DEV)
    ends = s["offsets"].tolist()
    for e in range(c["E"]):
        rows = src[ends[e]:ends[e + 1]]
        if len(rows):
            scale = s["a_scale_km"].double()[:, rows].t().repeat_interleave(128, 1)
            out[ends[e]:ends[e + 1]] = (s["a"].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() * scale) @ \
                _block_values(s["w"][e], s["w_scale"][e]).t()
    return out


def _exact_ffn(s):
    c = s["case"]
    x = _row_values(s["x"])
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    for e in range(c["E"]):
        slots = s["order"][ends[e]:ends[e + 1]].long()
        if len(slots):
            rows = x[slots // c["top_k"]]
            gate = (rows @ _block_values(s["w_gate"][e], s["w_gate_scale"][e]).t()).bfloat16().double()
            up = (rows @ _block_values(s["w_up"][e], s["w_up_scale"][e]).t()).bfloat16().double()
            h = _row_values((gate * torch.sigmoid(gate) * up).bfloat16())
            y = h @ _block_values(s["w_down"][e], s["w_down_scale"][e]).t()
            out.index_add_(0, slots // c["top_k"], y * s["weights"].double().reshape(-1)[slots, None])
    return out


def _exact_lora(s):
    out = _row_values(s["x"]) @ _block_values(s["w"], s["w_scale"]).t()
    for a in s["ids"].unique().tolist():
        if a >= 0:
            rows = (s["ids"] == a).nonzero()[:, 0]
            v = s["x"][rows].double() @ s["lora_a"][a].double().t()
            out[rows] += s["lora_scale"][a].double() * (v @ s["lora_b"][a].double().t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "grouped": _exact_grouped, "ffn": _exact_ffn, "lora": _exact_lora}[case["op"]](s)
