"""GPU tests of the expert operators: routing, grouping, products grouped by
expert, the weighted sum and the expert FFN.

References are plain numpy in 64 bits (and the oracle's GEMM on each expert's
rows).  Tolerances, derived:

* routing: ids, order, pos and offsets are whole numbers and must be equal.
  A weight is exp(l - lmax) / sum in fp32: l - lmax carries a rounding of at
  most 2^-24 |l - lmax| (below 110: an exponent beyond is a weight below
  1e-47), the exponential 2 ulp, the sum of at most 512 positive terms 16
  roundings (a tree over lanes and registers), the quotient one:
  (110 + 4 + 16 + 1) 2^-24 < 1e-5 relative, and results below 1e-37 may be
  flushed.
* grouped products: the GEMM contract of gpu_util.assert_tol.
* weighted sum: fp32 fmas of at most 32 terms are within err = 32 * 2^-24 of the
  sum of the terms' magnitudes; rounding is monotonic, so the result lies
  between the bf16 roundings of ref - err and ref + err.
* expert FFN: see test_ffn_against_the_definition.
"""
import numpy as np
import pytest
import torch

import synth
from gpu_util import Guarded, assert_tol, bf16_bits_to_f64, dev, host, log, require_gpu

pytestmark = pytest.mark.gpu

fp8q = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global fp8q
    require_gpu()
    import w8a8_fp8_block_amd as m
    fp8q = m
    yield


def _work(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


# ------------------------------------------------------------------ routing
def _route_ref(l, k, renorm):
    """(ids, weights, order, pos, offsets) of float64 logits."""
    T, E = l.shape
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max)) + 0.0
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    best = np.take_along_axis(l, ids.astype(np.int64), 1)
    top = np.where(np.isfinite(best[:, :1]), best[:, :1], 0.0)
    with np.errstate(over="ignore"):
        e = np.exp(best - top)
        total = e.sum(1, keepdims=True) if renorm else np.exp(l - top).sum(1, keepdims=True)
    w = np.where(best == -np.inf, 0.0, e / np.where(total > 0, total, 1.0))
    ids[best == -np.inf] = -1
    return (ids, w) + _group_ref(ids.reshape(-1), E)


def _group_ref(ids, groups):
    key = np.where((ids < 0) | (ids >= groups), groups, ids)
    order = np.argsort(key, kind="stable").astype(np.int32)
    pos = np.empty_like(order)
    pos[order] = np.arange(len(ids), dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return order, pos, offsets.astype(np.int32)


def _route_gpu(t, k, renorm, stream=None):
    T, E = t.shape
    out = dict(ids=Guarded((T, k), torch.int32), weights=Guarded((T, k), torch.float32),
               order=Guarded((T * k,), torch.int32), pos=Guarded((T * k,), torch.int32),
               offsets=Guarded((E + 1,), torch.int32))
    work = _work(fp8q.fp8q_moe_route_workspace_bytes(T, E, k))
    fp8q.fp8q_moe_route(t, *(out[n].t for n in ("ids", "weights", "order", "pos", "offsets")), work,
                        renormalize=renorm, stream=stream)
    torch.cuda.synchronize()
    for g in out.values():
        g.check_canary()
    return [host(g.t) for g in out.values()]


def _check_route(t, k, renorm):
    got = _route_gpu(t, k, renorm)
    want = _route_ref(t.float().cpu().numpy().astype(np.float64), k, renorm)
    for name, g, w in zip(("ids", "weights", "order", "pos", "offsets"), got, want):
        if name == "weights":
            assert np.all(np.abs(g - w) <= 1e-5 * w + 1e-37), name
        else:
            np.testing.assert_array_equal(g, w, err_msg=name)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 7, 7), (16, 64, 4), (63, 65, 6),
                                   (64, 512, 32), (65, 16, 2), (300, 160, 6), (1000, 3, 2),
                                   (9001, 40, 5), (20000, 8, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, dtype, renorm):
    log(f"route T={T} E={E} k={k} {dtype} renorm={renorm}")
    t = torch.randn(T, E, generator=torch.Generator().manual_seed(T * 1000 + E + k)) * 2
    # (bf16 logits tie often: the lowest index comes first)
    _check_route(t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda(), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(renorm):
    inf, low = float("inf"), float(np.finfo(np.float32).min)
    rows = [[-inf] * 6,                                # nothing to choose
            [-inf, 2.0, -inf, -inf, 1.0, -inf],        # fewer than k
            [float("nan")] * 6, [float("nan"), 0.5, float("nan"), 0.25, 0.5, -inf],
            [low] * 6,                                 # the type's lowest value is a value
            [low, -inf, low, 0.0, -inf, low],
            [inf, 1.0, inf, 3.0, -inf, 2.0],           # +inf: the largest finite value
            [0.0, -0.0, -0.0, 0.0, -0.0, 0.0],         # signed zeros tie
            [1.0] * 6, [-200.0, 100.0, 3e38, -3e38, 99.0, 0.0]]
    log("route special values")
    _check_route(torch.tensor(rows * 9, dtype=torch.float32).cuda(), 3, renorm)
    _check_route(torch.tensor(rows, dtype=torch.float32).cuda(), 3, renorm)


def test_route_without_tokens():
    log("route T=0")
    got = _route_gpu(torch.empty(0, 9, device="cuda"), 2, True)
    assert not got[4].any()


@pytest.mark.parametrize("n,groups", [(0, 5), (1, 1), (5, 7), (64, 64), (2048, 65), (2049, 3), (5000, 512),
                                      (100003, 130), (1 << 20, 31)])
def test_group_rows(n, groups):
    log(f"group_rows n={n} groups={groups}")
    rng = np.random.default_rng(n + groups)
    ids = rng.integers(-2, groups + 2, n).astype(np.int32)
    ids[rng.random(n) < 0.3] = min(1, groups - 1)  # one popular group
    if n > 10:
        ids[3], ids[7] = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    order, pos, offs = Guarded((n,), torch.int32), Guarded((n,), torch.int32), Guarded((groups + 1,), torch.int32)
    fp8q.fp8q_group_rows(dev(ids), order.t, pos.t, offs.t, _work(fp8q.fp8q_group_rows_workspace_bytes(n, groups)))
    torch.cuda.synchronize()
    for g, w in zip((order, pos, offs), _group_ref(ids, groups)):
        g.check_canary()
        np.testing.assert_array_equal(host(g.t), w)


# ------------------------------------------------------------ grouped products
def _experts(orc, E, N, K, rng):
    q, s = zip(*(orc.quant_weight_block(rng.normal(0, 0.02, (N, K)).astype(np.float32)) for _ in range(E)))
    return np.stack(q), np.stack(s)


def _acts(orc, rows, K, rng):
    x = rng.laplace(0, 1, (rows, K)).astype(np.float32)
    x[:, rng.choice(K, max(1, K // 100), replace=False)] *= 20
    return synth.f32_to_bf16_bits(x)


def _grouped_case(orc, sizes, N, K, top_k, gather, dropped, seed):
    """Codes, scales, plan and fp64 result of groups of the given sizes."""
    rng = np.random.default_rng(seed)
    E, R = len(sizes), sum(sizes) + dropped
    assert R % top_k == 0
    ids = np.repeat(np.arange(E + 1, dtype=np.int32), list(sizes) + [dropped])
    ids = rng.permutation(ids) if gather else ids
    order, pos, offsets = _group_ref(ids, E)
    rows = R // top_k if gather else R
    a, a_s = orc.quant_act(_acts(orc, rows, K, rng))
    wq, ws = _experts(orc, E, N, K, rng)
    ref = np.zeros((R, N))
    for e in range(E):
        p = np.arange(offsets[e], offsets[e + 1])
        r = order[p] // top_k if gather else p
        if len(p):
            ref[p] = orc.gemm_ref(a[r], a_s[r], wq[e], ws[e])
    return a, a_s, wq, ws, order, offsets, ref


SIZES = [  # group sizes, N, K, top_k, slots of no expert
    ([1], 128, 128, 1, 0),
    ([0, 3, 0, 0, 1, 0], 256, 384, 2, 2),          # empty experts around, ends inside a tile
    ([16, 17, 15, 0, 33, 1, 2], 384, 1408, 4, 0),  # tile edges, odd N / 128, K blocks not of a stage
    ([5, 60, 129, 0, 300, 128, 2], 640, 640, 3, 6),  # several row tiles
    ([0] * 65 + [7] + [0] * 200 + [40, 1], 128, 512, 1, 1),  # more experts than lanes, most empty
    ([2] * 300, 128, 256, 4, 0),                   # more experts than the persistent kernel's tables
]


@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("gather", [True, False])
def test_gemm_grouped(orc, case, gather):
    sizes, N, K, top_k, dropped = SIZES[case]
    a, a_s, wq, ws, order, offsets, ref = _grouped_case(orc, sizes, N, K, top_k, gather, dropped, 11 + case)
    R, used = len(order), int(offsets[-1])
    ad, kmd, wqd, wsd = dev(a), dev(orc.scale_to_kmajor(a_s)), dev(wq), dev(ws)
    for kernel in (0, 1, 2, 3):
        log(f"gemm_grouped case={case} gather={gather} kernel={kernel}")
        out = Guarded((R, N), torch.int16)
        before = host(out.t).copy()
        fp8q.fp8q_gemm_grouped(ad, kmd, wqd, wsd, dev(offsets), out.t, order=dev(order) if gather else None,
                               top_k=top_k if gather else 1, kernel=kernel)
        torch.cuda.synchronize()
        out.check_canary()
        got = host(out.t)
        assert np.array_equal(got[used:], before[used:]), "rows of no expert must be left alone"
        assert_tol(bf16_bits_to_f64(got[:used]), ref[:used], f"grouped case {case} kernel {kernel}")


@pytest.mark.parametrize("E,T,top_k,N,K", [(40, 25, 6, 1408, 1024), (4, 9, 2, 512, 5120), (8, 700, 2, 896, 1536),
                                          (24, 90, 8, 256, 2048)])
def test_gemm_grouped_routed(orc, E, T, top_k, N, K):
    """Rows routed on the device, each kernel choice; 2 and 3 give the same bits."""
    log(f"gemm_grouped routed E={E} T={T} k={top_k} N={N} K={K}")
    rng = np.random.default_rng(E + T)
    ids, _, order, pos, offsets = _route_gpu(torch.from_numpy(rng.normal(0, 1, (T, E)).astype(np.float32)).cuda(),
                                             top_k, True)
    a, a_s = orc.quant_act(_acts(orc, T, K, rng))
    wq, ws = _experts(orc, E, N, K, rng)
    ref = np.zeros((T * top_k, N))
    for e in range(E):
        r = order[offsets[e]:offsets[e + 1]] // top_k
        if len(r):
            ref[offsets[e]:offsets[e + 1]] = orc.gemm_ref(a[r], a_s[r], wq[e], ws[e])
    ad, kmd, wqd, wsd = dev(a), dev(orc.scale_to_kmajor(a_s)), dev(wq), dev(ws)
    outs = {}
    for kernel in (1, 2, 3):
        out = Guarded((T * top_k, N), torch.int16)
        for _ in range(2):
            fp8q.fp8q_gemm_grouped(ad, kmd, wqd, wsd, dev(offsets), out.t, order=dev(order), top_k=top_k,
                                   kernel=kernel)
            torch.cuda.synchronize()
            got = host(out.t).copy()
            assert kernel not in outs or np.array_equal(outs[kernel], got), "two runs differ"
            outs[kernel] = got
        out.check_canary()
        assert_tol(bf16_bits_to_f64(outs[kernel]), ref, f"routed kernel {kernel}")
    assert np.array_equal(outs[2], outs[3])


@pytest.mark.parametrize("K", [512, 640, 768, 896])
@pytest.mark.parametrize("gather", [True, False])
def test_gemm_grouped_many_tiles(orc, K, gather):
    """More tiles than CUs: the persistent kernels' workgroups run several, whose
    first blocks fall on every slot of the ring (K / 128 = 4 .. 7)."""
    sizes, N, top_k = [130, 0, 257, 1, 128, 700, 60, 500], 3840, 4
    a, a_s, wq, ws, order, offsets, ref = _grouped_case(orc, sizes, N, K, top_k, gather, 0, K)
    ad, kmd, wqd, wsd = dev(a), dev(orc.scale_to_kmajor(a_s)), dev(wq), dev(ws)
    for kernel in (1, 2, 3):
        log(f"gemm_grouped many tiles K={K} gather={gather} kernel={kernel}")
        out = Guarded((len(order), N), torch.int16)
        fp8q.fp8q_gemm_grouped(ad, kmd, wqd, wsd, dev(offsets), out.t, order=dev(order) if gather else None,
                               top_k=top_k if gather else 1, kernel=kernel)
        torch.cuda.synchronize()
        out.check_canary()
        assert_tol(bf16_bits_to_f64(host(out.t)), ref, f"many tiles K {K} kernel {kernel}")


def test_gemm_grouped_weights_past_32_bits(orc):
    """180 experts of 5120 x 5120: 4.7e9 codes; rows in the first and last experts."""
    E, N, K = 180, 5120, 5120
    rng = np.random.default_rng(4)
    used = (0, 1, 163, 164, 179)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(E, N // 128, K // 128, device="cuda")
    hosts = {e: orc.quant_weight_block(rng.normal(0, 0.02, (N, K)).astype(np.float32)) for e in used}
    for e, (q, s) in hosts.items():
        w[e], ws[e] = dev(q), dev(s)
    ids = np.repeat(np.array(used, np.int32), 3)
    _, _, offsets = _group_ref(ids, E)
    a, a_s = orc.quant_act(_acts(orc, len(ids), K, rng))
    ref = np.concatenate([orc.gemm_ref(a[3 * i:3 * i + 3], a_s[3 * i:3 * i + 3], *hosts[e]) for i, e in enumerate(used)])
    for kernel in (1, 2, 3):
        log(f"gemm_grouped weights past 32 bits kernel={kernel}")
        out = Guarded((len(ids), N), torch.int16)
        fp8q.fp8q_gemm_grouped(dev(a), dev(orc.scale_to_kmajor(a_s)), w, ws, dev(offsets), out.t, kernel=kernel)
        torch.cuda.synchronize()
        out.check_canary()
        assert_tol(bf16_bits_to_f64(host(out.t)), ref, f"past 32 bits kernel {kernel}")


# --------------------------------------------------------------- weighted sum
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (5, 3, 136), (33, 8, 5120), (2, 32, 2056)])
def test_combine(T, k, H):
    log(f"combine T={T} k={k} H={H}")
    rng = np.random.default_rng(T + k)
    E = 6
    ids = rng.integers(-1, E, T * k).astype(np.int32)
    if T > 1:
        ids[:k] = -1  # a token without any expert
    order, pos, offsets = _group_ref(ids, E)
    y = synth.f32_to_bf16_bits(rng.normal(0, 3, (T * k, H)).astype(np.float32))
    y[offsets[-1]:] = 0x7FC0  # rows of no expert: NaN, never read into a result
    w = rng.random((T, k)).astype(np.float32)
    out = Guarded((T, H), torch.int16)
    fp8q.fp8q_moe_combine(dev(y), dev(w), dev(pos), dev(offsets), out.t)
    torch.cuda.synchronize()
    out.check_canary()
    terms = bf16_bits_to_f64(y)[pos].reshape(T, k, H) * w.astype(np.float64)[:, :, None]
    terms[(pos >= offsets[-1]).reshape(T, k)] = 0
    ref, mag = terms.sum(1), np.abs(terms).sum(1)
    got = bf16_bits_to_f64(host(out.t))
    err = 32 * 2.0 ** -24 * mag
    assert np.all((_bf16(ref - err) <= got) & (got <= _bf16(ref + err)))
    if T > 1:
        assert not got[0].any()


@pytest.mark.parametrize("taken", [12, 17, 2 ** 31 - 1, -1])
def test_combine_keeps_to_the_rows(taken):
    """Whatever offsets[E] and pos hold, rows past the T * top_k of y are not read: such
    slots add nothing.  (The rows behind y here are NaN.)"""
    log(f"combine with offsets[E]={taken}")
    T, k, H, E = 4, 3, 264, 5
    rng = np.random.default_rng(3)
    pos = rng.permutation(T * k).astype(np.int32)
    pos[[0, 4, 5, 10]] = [T * k, T * k + 4, -1, np.iinfo(np.int32).min]
    offsets = np.array([0, 2, 4, 6, 8, taken], np.int32)
    behind = torch.full((2 * T * k, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = behind[:T * k]
    y.copy_(torch.from_numpy(rng.normal(0, 3, (T * k, H)).astype(np.float32)))
    w = rng.random((T, k)).astype(np.float32)
    out = Guarded((T, H), torch.int16)
    fp8q.fp8q_moe_combine(y, dev(w), dev(pos), dev(offsets), out.t)
    torch.cuda.synchronize()
    out.check_canary()
    inside = ((pos >= 0) & (pos < T * k)).reshape(T, k)
    rows = y.float().cpu().numpy().astype(np.float64)[np.where(inside.reshape(-1), pos, 0)].reshape(T, k, H)
    terms = rows * np.where(inside, w, 0).astype(np.float64)[:, :, None]
    ref, err = terms.sum(1), 32 * 2.0 ** -24 * np.abs(terms).sum(1)
    got = bf16_bits_to_f64(host(out.t))
    assert np.all((_bf16(ref - err) <= got) & (got <= _bf16(ref + err)))


def test_combine_of_many_tokens():
    """More tokens than one dimension of a launch has workgroups for (2^24 of 256
    threads): weights are powers of two, so the results are exact."""
    log("combine of 2^24 + 5 tokens")
    T, H = (1 << 24) + 5, 8
    g = torch.Generator("cuda").manual_seed(1)
    y = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.tensor([0.5, 2.0, 1.0], device="cuda")[torch.arange(T, device="cuda") % 3].view(T, 1)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = Guarded((T, H), torch.int16)
    fp8q.fp8q_moe_combine(y, w, pos, offsets, out.t)
    torch.cuda.synchronize()
    assert torch.equal(out.t.view(torch.bfloat16), (y.flip(0).float() * w).bfloat16())
    out.check_canary()


# ----------------------------------------------------------------- expert FFN
def _ffn_inputs(orc, T, E, k, H, I, seed, holes=False):
    rng = np.random.default_rng(seed)
    logits = rng.normal(0, 1.5, (T, E))
    ids, w, order, pos, offsets = _route_ref(logits, k, True)
    if holes:  # some choices belong to another rank
        ids = np.where(rng.random(ids.shape) < 0.3, -1, ids).astype(np.int32)
        if T > 1:
            ids[0] = -1
        order, pos, offsets = _group_ref(ids.reshape(-1), E)
    x = _acts(orc, T, H, rng)
    return x, ids, w.astype(np.float32), order, pos, offsets, _experts(orc, E, I, H, rng), \
        _experts(orc, E, I, H, rng), _experts(orc, E, H, I, rng)


def _bf16(a):
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(a.astype(np.float32))).astype(np.float64)


def _ffn_ref(orc, x, ids, w, wg, wu, wd):
    """The definition in 64 bits, each intermediate in its format."""
    a, a_s = orc.quant_act(x)
    out = np.zeros((x.shape[0], wd[0].shape[1]))
    for e in range(wg[0].shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t):
            g = _bf16(orc.gemm_ref(a[t], a_s[t], wg[0][e], wg[1][e]))
            u = _bf16(orc.gemm_ref(a[t], a_s[t], wu[0][e], wu[1][e]))
            h = synth.f32_to_bf16_bits((g / (1 + np.exp(-g)) * u).astype(np.float32))
            hq, hs = orc.quant_act(h)
            np.add.at(out, t, orc.gemm_ref(hq, hs, wd[0][e], wd[1][e]) * w[t, j].astype(np.float64)[:, None])
    return out


def _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, variant, stream=None):
    T, H = x.shape
    E, I, _ = wg[0].shape
    out = Guarded((T, H), torch.int16)
    work = _work(fp8q.fp8q_moe_ffn_workspace_bytes(T, E, w.shape[1], H, I, variant))
    work.fill_(0xFF)  # NaN in every format: nothing in it may be read before it is written
    fp8q.fp8q_moe_ffn(dev(x), dev(w), dev(order), dev(pos), dev(offsets), dev(wg[0]), dev(wg[1]), dev(wu[0]),
                      dev(wu[1]), dev(wd[0]), dev(wd[1]), out.t, work, variant=variant, stream=stream)
    torch.cuda.synchronize()
    out.check_canary()
    return bf16_bits_to_f64(host(out.t))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 3, 1, 128, 128), (2, 8, 3, 512, 384), (16, 24, 4, 1024, 640),
                                       (70, 5, 2, 640, 256), (300, 4, 3, 512, 512),
                                       (500, 3, 2, 512, 4096), (450, 3, 2, 768, 4096)])
@pytest.mark.parametrize("holes", [False, True])
def test_ffn_against_the_definition(orc, T, E, k, H, I, holes):
    """Against the 64-bit definition: bf16 roundings of each expert's output and
    of the sum, 1.7e-3 of the norm each, 2.4e-3 together; and the codes of
    the intermediate that fall on the other side of a rounding.  The FP8 MFMA
    moves gate and up by 2e-5 of their RMS, so that about 2% of them round to
    the neighbouring bf16 (2^-8 away), 4% of the h; of those one in ten takes
    the next e4m3 code, on average 8% away, or, where h is its group's maximum,
    moves the scale: up to 0.5% of the codes, sqrt(0.005) * 0.08 = 5.7e-3 of the
    norm.  Bound: 8e-3 (few elements average little)."""
    x, ids, w, order, pos, offsets, wg, wu, wd = _ffn_inputs(orc, T, E, k, H, I, T + E, holes)
    ref = _ffn_ref(orc, x, ids, w, wg, wu, wd)
    for variant in (0, 1, 2):
        log(f"moe_ffn T={T} E={E} k={k} H={H} I={I} holes={holes} variant={variant}")
        got = _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, variant)
        rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
        log(f"  relative error {rel:.2e}")
        assert rel <= 8e-3
        assert not got[(ids < 0).all(1)].any()


def test_ffn_is_its_parts(orc):
    """The separate variant on 128 x 128 tiles gives the bits of the public
    steps: quantizer, grouped products, intermediate, grouped product, sum."""
    T, E, k, H, I = 120, 4, 2, 512, 256
    log("moe_ffn against its parts")
    x, ids, w, order, pos, offsets, wg, wu, wd = _ffn_inputs(orc, T, E, k, H, I, 5)
    got = _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, 1)
    R = T * k
    xq, xs = Guarded((T, H), torch.uint8), Guarded((H // 128, synth.ceil16(T)), torch.float32)
    fp8q.fp8q_quant_act_kmajor(dev(x), xq.t, None, xs.t)
    g, u, y = (Guarded((R, n), torch.int16) for n in (I, I, H))
    for wt, o in ((wg, g), (wu, u)):
        fp8q.fp8q_gemm_grouped(xq.t, xs.t, dev(wt[0]), dev(wt[1]), dev(offsets), o.t, order=dev(order), top_k=k, kernel=2)
    hq, hs = Guarded((R, I), torch.uint8), Guarded((I // 128, synth.ceil16(R)), torch.float32)
    fp8q.fp8q_silu_mul_quant(g.t, u.t, hq.t, hs.t)
    fp8q.fp8q_gemm_grouped(hq.t, hs.t, dev(wd[0]), dev(wd[1]), dev(offsets), y.t, kernel=2)
    out = Guarded((T, H), torch.int16)
    fp8q.fp8q_moe_combine(y.t, dev(w), dev(pos), dev(offsets), out.t)
    torch.cuda.synchronize()
    want = bf16_bits_to_f64(host(out.t))
    # (the fused kernel's intermediate has the same bits; the down product may
    # take another kernel, equal up to the order of its fp32 sums)
    assert np.linalg.norm(got - want) <= 1e-3 * np.linalg.norm(want)


# (T, E, k, H, I) by the streaming instance that gate and up (f16 products), and the
# down product (FP8), take on 256 CUs: rows a tile, columns x K blocks of a stage
STREAMED = [(2, 8, 3, 512, 384),       # 16 rows, 32 x 4 both
            (16, 24, 4, 1024, 640),    # 16 rows, 64 x 2 both
            (20, 8, 2, 512, 512),      # 32 rows, 32 x 4 both
            (30, 8, 2, 2048, 1024),    # 32 rows, 64 x 2 both
            (64, 64, 6, 640, 256)]     # 32 rows, 128 x 1 both


@pytest.mark.parametrize("T,E,k,H,I", STREAMED)
@pytest.mark.parametrize("holes", [False, True])
def test_streamed_ffn_against_the_definition(orc, T, E, k, H, I, holes):
    """Every streaming instance.  Gate and up come from f16 products, off by 1e-7 of
    their RMS at most, so that hardly one in 10^4 rounds to another bf16 value or code:
    what is left are the bf16 roundings of each expert's output and of the sum, each
    2^-7 / sqrt(12) of the value's power of two, up to 1.7e-3 of the norm, 2.4e-3
    together; bound 3e-3 for the scatter of few elements."""
    log(f"streamed moe_ffn T={T} E={E} k={k} H={H} I={I} holes={holes}")
    assert fp8q.fp8q_gemm_grouped_select(T * k, E, 2 * I) == 1 and fp8q.fp8q_gemm_grouped_select(T * k, E, H) == 1
    x, ids, w, order, pos, offsets, wg, wu, wd = _ffn_inputs(orc, T, E, k, H, I, 3 * T + E, holes)
    ref = _ffn_ref(orc, x, ids, w, wg, wu, wd)
    got = _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, 2)
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    log(f"  relative error {rel:.2e}")
    assert rel <= 3e-3
    assert not got[(ids < 0).all(1)].any()


@pytest.mark.parametrize("sizes,N", [([1, 0, 4, 2], 1024), ([3, 1, 0, 4] * 4, 2048),           # 16-row tiles
                                     ([33, 0, 9, 17], 1024), ([40, 3, 0, 16, 17, 5, 32, 1], 2048),
                                     ([20, 1, 0, 33] * 4, 2048)])                              # 32-row tiles
@pytest.mark.parametrize("K", [640, 1408])
def test_streamed_products(orc, sizes, N, K):
    """Every streaming instance of the FP8 product, K blocks that do not fill the last stage."""
    a, a_s, wq, ws, order, offsets, ref = _grouped_case(orc, sizes, N, K, 1, True, 0, N + K)
    log(f"streamed product E={len(sizes)} R={len(order)} N={N} K={K}")
    out = Guarded((len(order), N), torch.int16)
    fp8q.fp8q_gemm_grouped(dev(a), dev(orc.scale_to_kmajor(a_s)), dev(wq), dev(ws), dev(offsets), out.t,
                           order=dev(order), kernel=1)
    torch.cuda.synchronize()
    out.check_canary()
    assert_tol(bf16_bits_to_f64(host(out.t)), ref, f"streamed product E {len(sizes)} N {N} K {K}")


def _ffn_by_parts(x, w, order, pos, offsets, wg, wu, wd):
    """The public steps: quantizer, gate and up on 128 x 128 tiles, intermediate, down
    product on the automatic kernel, weighted sum."""
    (T, H), k, (E, I, _) = x.shape, w.shape[1], wg[0].shape
    R = T * k
    xq, xs = Guarded((T, H), torch.uint8), Guarded((H // 128, synth.ceil16(T)), torch.float32)
    fp8q.fp8q_quant_act_kmajor(dev(x), xq.t, None, xs.t)
    g, u, y = (Guarded((R, n), torch.int16) for n in (I, I, H))
    for wt, o in ((wg, g), (wu, u)):
        fp8q.fp8q_gemm_grouped(xq.t, xs.t, dev(wt[0]), dev(wt[1]), dev(offsets), o.t, order=dev(order), top_k=k, kernel=2)
    hq, hs = Guarded((R, I), torch.uint8), Guarded((I // 128, synth.ceil16(R)), torch.float32)
    fp8q.fp8q_silu_mul_quant(g.t, u.t, hq.t, hs.t)
    fp8q.fp8q_gemm_grouped(hq.t, hs.t, dev(wd[0]), dev(wd[1]), dev(offsets), y.t)
    out = Guarded((T, H), torch.int16)
    fp8q.fp8q_moe_combine(y.t, dev(w), dev(pos), dev(offsets), out.t)
    torch.cuda.synchronize()
    return host(out.t)


@pytest.mark.parametrize("T,E,k,H,I", [(120, 4, 2, 512, 256),    # persistent fused gate/up
                                       (500, 3, 2, 640, 4096),   # the same, several tiles a workgroup
                                       (300, 4, 2, 256, 384),    # H < 512: a workgroup a tile
                                       (700, 3, 2, 384, 256), (257, 2, 1, 128, 640),
                                       (600, 300, 2, 512, 256),  # more experts than the tables
                                       (90, 300, 4, 256, 128)])
@pytest.mark.parametrize("holes", [False, True])
def test_fused_ffn_has_the_bits_of_its_parts(orc, T, E, k, H, I, holes):
    """Both fused gate/up kernels, and the separate form on 128 x 128 tiles, give the
    output of the public steps bit for bit; against the 64-bit definition as in
    test_ffn_against_the_definition."""
    log(f"fused moe_ffn T={T} E={E} k={k} H={H} I={I} holes={holes}")
    x, ids, w, order, pos, offsets, wg, wu, wd = _ffn_inputs(orc, T, E, k, H, I, 7 * T + E, holes)
    want = bf16_bits_to_f64(_ffn_by_parts(x, w, order, pos, offsets, wg, wu, wd))
    variants = (1, 2) if fp8q.fp8q_gemm_grouped_select(T * k, E, 2 * I) != 1 else (1,)
    for variant in variants:
        got = _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, variant)
        assert np.array_equal(got, want), f"variant {variant}"
    ref = _ffn_ref(orc, x, ids, w, wg, wu, wd)
    rel = np.linalg.norm(want - ref) / np.linalg.norm(ref)
    log(f"  relative error {rel:.2e}, variants {variants}")
    assert rel <= 8e-3


# ------------------------------------------------------- streams and capture
def test_side_stream_and_graph(orc):
    """The whole path on a stream of its own, then captured once and replayed with
    new inputs, with eager work between the replays."""
    T, E, k, H, I = 24, 6, 2, 512, 256
    log("expert path on a side stream and in a graph")
    x, ids, w, order, pos, offsets, wg, wu, wd = _ffn_inputs(orc, T, E, k, H, I, 9)
    want = _ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, 0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert np.array_equal(_ffn_gpu(x, w, order, pos, offsets, wg, wu, wd, 0), want)

    logits = torch.randn(T, E, device="cuda")
    xd, out = dev(x), torch.empty(T, H, dtype=torch.int16, device="cuda")
    wts = [dev(t) for t in (*wg, *wu, *wd)]
    i32 = dict(dtype=torch.int32, device="cuda")
    r = [torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(T * k, **i32),
         torch.empty(T * k, **i32), torch.empty(E + 1, **i32)]
    rw = _work(fp8q.fp8q_moe_route_workspace_bytes(T, E, k))
    fw = _work(fp8q.fp8q_moe_ffn_workspace_bytes(T, E, k, H, I))

    def path():
        fp8q.fp8q_moe_route(logits, *r, rw)
        fp8q.fp8q_moe_ffn(xd, r[1], r[2], r[3], r[4], *wts, out, fw)

    path()  # (kernel attributes are set outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path()
    for i in range(4):
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(i)))
        xd.copy_(dev(_acts(orc, T, H, np.random.default_rng(i))))
        path()
        torch.cuda.synchronize()
        eager = host(out).copy()
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), eager), f"replay {i}"
