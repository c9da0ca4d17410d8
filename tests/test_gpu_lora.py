"""GPU tests of fp8q_proj_lora: the projection with each row's low-rank adapter.

Reference: the oracle's fp64 projection of the oracle's quantized x, plus the
adapter's two products in fp64, under the GEMM contract of gpu_util.assert_tol
(the adapter's part is formed to about 2^-16: x . A^T in fp32, split into two
bf16 terms for the second product, so the contract's 1e-3 covers it).  The
codes and scales the call leaves in its scratch must be the quantizer's, bit
for bit.
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


def _ids(kind, M, n, rng):
    if kind == "each":
        return rng.integers(0, n, M)
    if kind == "runs":  # contiguous requests, some without an adapter
        cuts = np.sort(rng.integers(0, M, 3))
        who = rng.integers(-1, n, 4)
        return np.repeat(who, np.diff(np.concatenate([[0], cuts, [M]])))
    if kind == "none":
        return np.full(M, -1)
    ids = rng.integers(0, n, M)  # "outside": ids that name no adapter among the rows
    ids[rng.random(M) < 0.5] = rng.choice([-1, n, n + 5, np.iinfo(np.int32).max, np.iinfo(np.int32).min])
    return ids


def _run(orc, M, N, K, n, R, kind, seed, pad_rank=0):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    x[:, rng.choice(K, max(1, K // 100), replace=False)] *= 20
    x = synth.f32_to_bf16_bits(x)
    wq, ws = orc.quant_weight_block(rng.normal(0, 0.02, (N, K)).astype(np.float32))
    A = synth.f32_to_bf16_bits((rng.normal(0, 1, (n, R, K)) / np.sqrt(K)).astype(np.float32))
    B = synth.f32_to_bf16_bits(rng.normal(0, 0.05, (n, N, R)).astype(np.float32))
    if pad_rank:  # an adapter of smaller rank, padded with zeros
        A[0, pad_rank:], B[0, :, pad_rank:] = 0, 0
    s = (0.5 + rng.random(n)).astype(np.float32)
    ids = _ids(kind, M, n, rng).astype(np.int32)
    out, q = Guarded((M, N), torch.int16), Guarded((M, K), torch.uint8)
    rm, km = Guarded((M, K // 128), torch.float32), Guarded((K // 128, synth.ceil16(M)), torch.float32)
    nbytes = fp8q.fp8q_proj_lora_workspace_bytes(M, N, K, R)
    work = Guarded((nbytes,), torch.uint8, fill=0xFF)  # NaN: nothing may be read before it is written
    args = (dev(x), dev(wq), dev(ws), dev(A), dev(B), dev(s), dev(ids), out.t, q.t, rm.t, km.t, work.t)
    fp8q.fp8q_proj_lora(*args)
    torch.cuda.synchronize()
    for g in (out, q, rm, km, work):
        g.check_canary()
    a, a_s = orc.quant_act(x)
    np.testing.assert_array_equal(host(q.t), a)
    np.testing.assert_array_equal(host(rm.t), a_s)
    np.testing.assert_array_equal(host(km.t), orc.scale_to_kmajor(a_s))
    ref = orc.gemm_ref(a, a_s, wq, ws)
    for m in range(M):
        if 0 <= ids[m] < n:
            v = bf16_bits_to_f64(x[m]) @ bf16_bits_to_f64(A[ids[m]]).T
            ref[m] += s[ids[m]].astype(np.float64) * (bf16_bits_to_f64(B[ids[m]]) @ v)
    got = host(out.t).copy()
    assert_tol(bf16_bits_to_f64(got), ref, f"lora M{M}N{N}K{K}n{n}R{R}{kind}")
    fp8q.fp8q_proj_lora(*args)
    torch.cuda.synchronize()
    assert np.array_equal(host(out.t), got), "two runs differ"
    return args, got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 48, 64, 65, 100, 129, 257, 300, 520])
@pytest.mark.parametrize("kind", ["each", "runs"])
def test_rows(orc, M, kind):
    log(f"lora M={M} {kind}")
    _run(orc, M, 384, 640, 5, 24, kind, M)


@pytest.mark.parametrize("N,K", [(128, 128), (256, 1408), (1152, 512), (5120, 5120)])
@pytest.mark.parametrize("M", [3, 40, 100])
def test_shapes(orc, M, N, K):
    log(f"lora M={M} N={N} K={K}")
    _run(orc, M, N, K, 3, 16, "each", N + K)


def test_split_k(orc):
    """Long K: the projection's split forms, whose first part (tiled) or all
    parts (skinny) add the adapters."""
    for M in (12, 50, 90):
        log(f"lora split-K M={M}")
        assert fp8q.fp8q_gemm_splitk_select(M, 1024, 8192) >= 2
        _run(orc, M, 1024, 8192, 4, 32, "each", M)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("M", [5, 70])
def test_ranks(orc, M, R):
    log(f"lora M={M} rank={R}")
    _run(orc, M, 256, 512, 3, R, "each", R, pad_rank=4)


@pytest.mark.parametrize("kind", ["none", "outside"])
@pytest.mark.parametrize("M", [1, 30, 64, 200])
def test_rows_without_adapter(orc, M, kind):
    log(f"lora M={M} ids {kind}")
    _run(orc, M, 256, 512, 2, 16, kind, M)


def test_more_adapters_than_rows(orc):
    """As many adapters as rows and more; every row its own."""
    for M, n in ((64, 70), (16, 16), (130, 200)):
        log(f"lora M={M} adapters={n}")
        _run(orc, M, 256, 384, n, 8, "each", n)


@pytest.mark.parametrize("M,N,K", [(3, 256, 384), (16, 5120, 512), (40, 512, 640), (100, 1024, 8192), (200, 384, 512),
                                   (1024, 5120, 384)])
@pytest.mark.parametrize("where", ["a", "b", "scale"])
def test_adapters_do_not_reach_other_rows(orc, M, N, K, where):
    """Infinities and NaN in one adapter leave the rows of the others, and those
    without one, bit for bit as they were."""
    log(f"lora M={M} N={N} K={K} non-finite {where}")
    args, want = _run(orc, M, N, K, 3, 16, "outside" if M < 1000 else "runs", M + K)
    x, wq, ws, A, B, s, ids, out = args[:8]
    who = host(ids)
    ids.copy_(torch.from_numpy(np.where(np.arange(M) % 3 == 0, 1, who).astype(np.int32)))
    fp8q.fp8q_proj_lora(*args)
    torch.cuda.synchronize()
    clean, others = host(out).copy(), host(ids) != 1
    if where == "a":
        A[1, :, ::7], A[1, :, 3] = 0x7F80, 0x7FC0
    elif where == "b":
        B[1, ::3], B[1, 1::3] = 0x7F80, 0x7FC0
    else:
        s[1] = float("nan")
    fp8q.fp8q_proj_lora(*args)
    torch.cuda.synchronize()
    assert np.array_equal(host(out)[others], clean[others])
    if others.sum() < M:
        assert not np.array_equal(host(out), clean)


@pytest.mark.parametrize("M,N,K", [(3, 256, 384), (16, 5120, 512), (40, 512, 640), (100, 1024, 8192), (200, 384, 512),
                                   (1024, 5120, 384)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scaled_v_at_the_end_of_the_range(orc, M, N, K, sign):
    """scale * (x . A^T) of 6e38 is an infinity, and so is the output, with the sign of
    B; of 3.4e38, which bf16 rounds to an infinity, it is a number like others
    (B there 2^-120 .. 2^-122: the adapter adds up to 256)."""
    log(f"lora M={M} N={N} K={K} scaled v at the end of the range, sign {sign}")
    rng = np.random.default_rng(M + K)
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    x[:, 0] = 2.0
    x = synth.f32_to_bf16_bits(x)
    wq, ws = orc.quant_weight_block(rng.normal(0, 0.02, (N, K)).astype(np.float32))
    n, R = 3, 16
    A = np.zeros((n, R, K), np.float32)
    A[:, 5, 0] = 1.0  # v = 2 at rank 5, 0 elsewhere
    B = rng.choice([-1, 1], (n, N, R)) * 2.0 ** rng.integers(-2, 1, (n, N, R))
    B[2] *= 2.0 ** -120
    A, B = synth.f32_to_bf16_bits(A), synth.f32_to_bf16_bits(B.astype(np.float32))
    s = np.array([1.0, sign * 3e38, sign * 1.7e38], np.float32)
    ids = (np.arange(M) % 4 - 1).astype(np.int32)
    out = Guarded((M, N), torch.int16)
    work = torch.empty(fp8q.fp8q_proj_lora_workspace_bytes(M, N, K, R), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_proj_lora(dev(x), dev(wq), dev(ws), dev(A), dev(B), dev(s), dev(ids), out.t,
                        *fp8q.alloc_proj_scratch(M, K), work)
    torch.cuda.synchronize()
    out.check_canary()
    got, b = bf16_bits_to_f64(host(out.t)), bf16_bits_to_f64(B)[:, :, 5]
    ref = orc.gemm_ref(*orc.quant_act(x), wq, ws)
    ref += np.where((ids >= 0)[:, None], 2.0 * s.astype(np.float64)[ids][:, None] * b[ids], 0)
    over = ids == 1
    assert np.array_equal(got[over], sign * np.sign(b[1]) * np.full((over.sum(), N), np.inf))
    assert_tol(got[~over], ref[~over], "lora at the end of the range")


@pytest.mark.parametrize("M,N,K", [(3, 256, 384), (200, 384, 512)])
@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, 0xFFFFFFFF])
def test_nan_scale_of_any_payload(orc, M, N, K, bits):
    """A NaN stays one in its rows, whatever its payload."""
    log(f"lora M={M} scale {bits:#x}")
    args, _ = _run(orc, M, N, K, 3, 16, "each", M)
    args[5].copy_(torch.from_numpy(np.array([1, 1, bits], np.uint32).view(np.float32)))
    fp8q.fp8q_proj_lora(*args)
    torch.cuda.synchronize()
    nan = np.isnan(bf16_bits_to_f64(host(args[7])))
    assert np.array_equal(nan, np.repeat((host(args[6]) == 2)[:, None], N, 1))


@pytest.mark.parametrize("M,N", [(1024, 5120), (1100, 4096)])
@pytest.mark.parametrize("kind", ["each", "runs"])
def test_prompts(orc, M, N, kind):
    """The ping-pong kernel's tiles, the last one partial."""
    log(f"lora M={M} N={N} {kind}")
    assert fp8q.fp8q_gemm_select(M, N, 384) == 5
    _run(orc, M, N, 384, 4, 40, kind, M)


def test_stacks_past_32_bits(orc):
    """2000 adapters of 17408 x 128 B: 4.5e9 numbers; rows of the first and last."""
    M, N, K, n, R = 6, 17408, 128, 2000, 128
    log("lora stacks past 32 bits")
    rng = np.random.default_rng(8)
    x = synth.f32_to_bf16_bits(rng.normal(0, 1, (M, K)).astype(np.float32))
    wq, ws = orc.quant_weight_block(rng.normal(0, 0.02, (N, K)).astype(np.float32))
    ids = np.array([0, 1999, 1930, -1, 1, 1928], np.int32)
    A = torch.zeros(n, R, K, dtype=torch.int16, device="cuda")
    B = torch.zeros(n, N, R, dtype=torch.int16, device="cuda")
    s = (0.5 + rng.random(n)).astype(np.float32)
    a, a_s = orc.quant_act(x)
    ref = orc.gemm_ref(a, a_s, wq, ws)
    for m, i in enumerate(ids):
        if i >= 0:
            Ai = synth.f32_to_bf16_bits((rng.normal(0, 1, (R, K)) / np.sqrt(K)).astype(np.float32))
            Bi = synth.f32_to_bf16_bits(rng.normal(0, 0.05, (N, R)).astype(np.float32))
            A[int(i)], B[int(i)] = dev(Ai), dev(Bi)
            ref[m] += float(s[i]) * (bf16_bits_to_f64(Bi) @ (bf16_bits_to_f64(Ai) @ bf16_bits_to_f64(x[m])))
    out = Guarded((M, N), torch.int16)
    work = torch.empty(fp8q.fp8q_proj_lora_workspace_bytes(M, N, K, R), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_proj_lora(dev(x), dev(wq), dev(ws), A, B, dev(s), dev(ids), out.t, *fp8q.alloc_proj_scratch(M, K), work)
    torch.cuda.synchronize()
    out.check_canary()
    assert_tol(bf16_bits_to_f64(host(out.t)), ref, "lora stacks past 32 bits")


def test_without_adapters_is_the_projection(orc):
    """Rows without an adapter get fp8q_proj's bits where it takes the same kernel."""
    M, N, K = 20, 512, 640
    log("lora against proj")
    (x, wq, ws, *_), got = _run(orc, M, N, K, 2, 16, "none", 1)
    out = torch.empty(M, N, dtype=torch.int16, device="cuda")
    fp8q.fp8q_proj(x, wq, ws, out, *fp8q.alloc_proj_scratch(M, K))
    torch.cuda.synchronize()
    assert np.array_equal(host(out), got)


def test_side_stream_and_graph(orc):
    M, N, K = 30, 512, 1024
    log("lora on a side stream and in a graph")
    args, want = _run(orc, M, N, K, 4, 16, "each", 3)
    out = args[7]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.fill_(0)
    torch.cuda.synchronize()
    fp8q.fp8q_proj_lora(*args, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(host(out), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8q.fp8q_proj_lora(*args)
    x, ids = args[0], args[6]
    for i in range(4):
        x.copy_(dev(synth.f32_to_bf16_bits(np.random.default_rng(i).normal(0, 1, (M, K)).astype(np.float32))))
        ids.copy_(torch.from_numpy(np.random.default_rng(i).integers(-1, 5, M).astype(np.int32)))
        fp8q.fp8q_proj_lora(*args)
        torch.cuda.synchronize()
        eager = host(out).copy()
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), eager), f"replay {i}"
