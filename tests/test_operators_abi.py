"""Refusals and host-side sizes of the expert and adapter operators (no GPU
needed, no kernel launched): every call here fails a check, or is an empty call
that returns before anything is enqueued."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import w8a8_fp8_block_amd as fp8q

P = ctypes.c_void_p
BAD, G = P(0x1001), P(0x1000)  # misaligned; aligned but never dereferenced
NULL, SHAPE, ALIGN, VARIANT = 1, 2, 3, 6
BIG = 1 << 40


def _err():
    return fp8q.lib().fp8q_last_error().decode()


def _each_pointer(call, args, names):
    """Every pointer refused as NULL (with its name) and misaligned."""
    for i, name in names.items():
        for bad, want in ((None, NULL), (BAD, ALIGN)):
            a = list(args)
            a[i] = bad
            assert call(*a) == want, name
            assert name in _err()


def test_route_refusals():
    L = fp8q.lib()

    def route(T=4, E=8, k=2, bf16=0, renorm=1, ws=G, nb=BIG, ptrs=(G,) * 6):
        lo, ids, w, order, pos, offs = ptrs
        return L.fp8q_moe_route(lo, bf16, ids, w, order, pos, offs, ws, nb, T, E, k, renorm, None)

    for kw, what in ((dict(E=0, k=1), "0 groups"), (dict(E=513), "513 groups"), (dict(k=0), "top_k=0"),
                     (dict(k=9), "top_k=9"), (dict(E=64, k=33), "top_k=33"),
                     (dict(T=1 << 31, k=1), "2^31"), (dict(T=1 << 24, E=512, k=1), "T*E")):
        assert route(**kw) == SHAPE, kw
        assert what in _err()
    for kw in (dict(bf16=2), dict(bf16=-1), dict(renorm=2), dict(renorm=-1)):
        assert route(**kw) == VARIANT
    for i, name in enumerate(("logits", "ids", "weights", "order", "pos", "offsets")):
        for bad, want in ((None, NULL), (BAD, ALIGN)):
            ptrs = [G] * 6
            ptrs[i] = bad
            assert route(ptrs=ptrs) == want
            assert name in _err()
    need = fp8q.fp8q_moe_route_workspace_bytes(100000, 8, 2)
    assert need > 0 and fp8q.fp8q_moe_route_workspace_bytes(1, 8, 2) == 0
    assert route(T=100000, nb=need - 1) == SHAPE and "workspace" in _err()
    assert route(T=100000, ws=None) == NULL
    assert route(T=100000, ws=BAD) == ALIGN


def test_group_rows_refusals():
    L = fp8q.lib()

    def group(n=100, groups=4, ids=G, order=G, pos=G, offs=G, ws=G, nb=BIG):
        return L.fp8q_group_rows(ids, order, pos, offs, ws, nb, n, groups, None)

    assert group(groups=0) == SHAPE and group(groups=513) == SHAPE and group(n=1 << 31) == SHAPE
    for name in ("ids", "order", "pos"):
        assert group(**{name: None}) == NULL and group(**{name: BAD}) == ALIGN
    assert group(offs=None) == NULL and group(n=0, offs=BAD) == ALIGN
    need = fp8q.fp8q_group_rows_workspace_bytes(1 << 20, 4)
    assert need > 0 and group(n=1 << 20, nb=need - 1) == SHAPE


def test_combine_refusals():
    L = fp8q.lib()

    def combine(y=G, w=G, pos=G, offs=G, out=G, T=4, E=8, k=2, H=128):
        return L.fp8q_moe_combine(y, w, pos, offs, out, T, E, k, H, None)

    for kw in (dict(E=0), dict(E=513), dict(k=0), dict(k=33), dict(H=0), dict(H=12),
               dict(T=1 << 20, k=8, H=5120)):
        assert combine(**kw) == SHAPE, kw
    _each_pointer(L.fp8q_moe_combine, (G, G, G, G, G, 4, 8, 2, 128, None),
                  {0: "y_bf16", 1: "weights", 2: "pos", 3: "offsets", 4: "out_bf16"})
    assert combine(T=0) == 0


def test_gemm_grouped_refusals():
    L = fp8q.lib()

    def grouped(order=G, rows=8, R=16, E=4, k=2, N=256, K=256, kernel=0):
        return L.fp8q_gemm_grouped(G, G, G, G, G, order, G, rows, R, E, k, N, K, kernel, None)

    for kw in (dict(E=0), dict(E=513), dict(k=0), dict(rows=1, R=33, k=33), dict(N=0), dict(N=200), dict(K=0),
               dict(K=192), dict(rows=9), dict(order=None), dict(rows=1 << 25, R=1 << 26),
               dict(R=1 << 31, rows=1 << 30, K=128), dict(N=1 << 17, K=1 << 15)):
        assert grouped(**kw) == SHAPE, kw
    for kernel in (-1, 4):
        assert grouped(kernel=kernel) == VARIANT
    assert grouped(order=BAD) == ALIGN
    _each_pointer(L.fp8q_gemm_grouped, (G, G, G, G, G, G, G, 8, 16, 4, 2, 256, 256, 0, None),
                  {0: "a_e4m3", 1: "a_scale_km", 2: "w_e4m3", 3: "w_scale", 4: "offsets", 6: "out_bf16"})
    assert grouped(rows=0, R=0) == 0


def test_grouped_select():
    sel = fp8q.fp8q_gemm_grouped_select
    assert sel(8, 0, 256) == 0 and sel(8, 4, 0) == 0 and sel(8, 4, 200) == 0
    assert sel(8, 128, 2048) == 1               # one row an expert: streaming
    assert sel(32 * 13, 32, 2048) == 1 and sel(32 * 14, 32, 2048) == 3
    assert sel(8 * 63, 8, 2048) == 1 and sel(8 * 64, 8, 2048) == 2   # few tiles: streaming further
    assert sel(8 * 500, 8, 2048) == 2 and sel(4 * 500, 4, 5120) == 2  # 1.5 rounds of 128x256 tiles at most
    assert sel(8 * 500, 8, 5120) == 3 and sel(64 * 572, 64, 2048) == 3
    assert sel(0, 8, 2048) == 1


def test_ffn_refusals():
    L = fp8q.lib()

    def ffn(T=4, E=8, k=2, H=256, I=128, variant=0, ws=G, nb=BIG):
        return L.fp8q_moe_ffn(G, G, G, G, G, G, G, G, G, G, G, G, ws, nb, T, E, k, H, I, variant, None)

    for kw in (dict(E=0), dict(E=513), dict(k=0), dict(k=33), dict(H=0), dict(H=130), dict(I=0), dict(I=64),
               dict(T=1 << 22, k=8, H=1024)):
        assert ffn(**kw) == SHAPE, kw
    assert ffn(variant=3) == VARIANT and ffn(variant=-1) == VARIANT
    names = ("x_bf16", "weights", "order", "pos", "offsets", "w_gate", "w_gate_scale", "w_up", "w_up_scale",
             "w_down", "w_down_scale", "out_bf16", "workspace")
    _each_pointer(L.fp8q_moe_ffn, (G,) * 13 + (BIG, 4, 8, 2, 256, 128, 0, None), dict(enumerate(names)))
    for variant in (0, 1, 2):
        need = fp8q.fp8q_moe_ffn_workspace_bytes(4, 8, 2, 256, 128, variant)
        assert need > 0 and ffn(variant=variant, nb=need - 1) == SHAPE and "workspace" in _err()
    assert ffn(T=0) == 0
    # the automatic variant's workspace is that variant's
    for T, I, want in ((4, 2048, 2), (5000, 2048, 1), (5000, 128, 2)):
        v = fp8q.fp8q_moe_ffn_select(T, 8, 2, I)
        assert v == want
        assert fp8q.fp8q_moe_ffn_workspace_bytes(T, 8, 2, 256, I) == \
            fp8q.fp8q_moe_ffn_workspace_bytes(T, 8, 2, 256, I, v)


def test_lora_refusals():
    L = fp8q.lib()

    def lora(M=4, N=256, K=256, n=3, r=16, ws=G, nb=BIG):
        return L.fp8q_proj_lora(G, G, G, G, G, G, G, G, G, G, G, ws, nb, M, N, K, n, r, None)

    for kw in (dict(N=0), dict(N=100), dict(K=0), dict(K=130), dict(r=0), dict(r=12), dict(r=136), dict(n=0),
               dict(M=1 << 25, K=256), dict(N=1 << 26, K=128, r=128)):
        assert lora(**kw) == SHAPE, kw
    names = ("x_bf16", "w_e4m3", "w_scale", "lora_a", "lora_b", "lora_scale", "adapter_ids", "out_bf16",
             "act_q_scratch", "act_scale_scratch", "act_scale_km_scratch", "workspace")
    _each_pointer(L.fp8q_proj_lora, (G,) * 12 + (BIG, 4, 256, 256, 3, 16, None), dict(enumerate(names)))
    need = fp8q.fp8q_proj_lora_workspace_bytes(4, 256, 256, 16)
    assert need > 0 and lora(nb=need - 1) == SHAPE and "workspace" in _err()
    assert lora(M=0) == 0


def test_binding_refusals():
    """Shapes and types that disagree end in ValueError before the C call."""
    i32 = dict(dtype=torch.int32)
    T, E, k = 4, 8, 2
    good = dict(logits=torch.zeros(T, E), ids=torch.zeros(T, k, **i32), weights=torch.zeros(T, k),
                order=torch.zeros(T * k, **i32), pos=torch.zeros(T * k, **i32),
                offsets=torch.zeros(E + 1, **i32))
    for name, bad in (("logits", torch.zeros(T, E, dtype=torch.float16)), ("ids", torch.zeros(T, k)),
                      ("weights", torch.zeros(T, k, dtype=torch.float64)), ("order", torch.zeros(T, **i32)),
                      ("pos", torch.zeros(T * k, dtype=torch.int64)), ("offsets", torch.zeros(E, **i32)),
                      ("logits", torch.zeros(E, T).t())):
        with pytest.raises((ValueError, TypeError)):
            fp8q.fp8q_moe_route(*{**good, name: bad}.values(), None)


def test_size_queries_of_any_numbers():
    """The size and selection queries return for an empty batch and for numbers that no
    call accepts (in a process of their own: a division by zero ends it)."""
    code = """
import itertools
import w8a8_fp8_block_amd as fp8q
L = fp8q.lib()
rows = [0, 1, 16, 17, 256, 257, (1 << 31) - 1, 1 << 31, 2**32 - 256, 2**32 - 128, 2**32 - 32, 2**32 - 16, 2**32 - 1]
cols = [0, 1, 128, 5120, 2**32 - 128, 2**32 - 1]
few = [0, 1, 8, 128, 512, 2**32 - 1]
for m, n, k, r in itertools.product(rows, cols, cols, few):
    L.fp8q_proj_lora_workspace_bytes(m, n, k, r)
    L.fp8q_moe_ffn_workspace_bytes(m, r, 2, n, k, 0)
    L.fp8q_moe_ffn_workspace_bytes(m, 8, r, n, k, 2)
for m, r, n in itertools.product(rows, few, cols):
    L.fp8q_moe_route_workspace_bytes(m, r, n)
    L.fp8q_group_rows_workspace_bytes(m, r)
    L.fp8q_gemm_grouped_select(m, r, n)
    L.fp8q_moe_ffn_select(m, r, 2, n)
assert fp8q.fp8q_proj_lora_workspace_bytes(0, 512, 512, 16) == 0
assert fp8q.fp8q_moe_ffn_workspace_bytes(0, 8, 2, 512, 512) == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root).returncode == 0


@pytest.fixture
def no_device(monkeypatch):
    """The binding with any tensor's pointer taken and no call made: its checks alone."""
    class Accepts:
        def __getattr__(self, name):
            return lambda *args: 0
    monkeypatch.setattr(fp8q, "_ptr", lambda t: 0x1000)
    monkeypatch.setattr(fp8q, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(fp8q, "lib", Accepts)


def _each_refused(call, good, bad):
    """The good arguments pass; with each bad one in turn the error names it."""
    call(**good)
    for name, t, error, what in bad:
        with pytest.raises(error, match=what):
            call(**{**good, name: t})


def _fp8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i32(n):
    return torch.zeros(n, dtype=torch.int32)


def test_lora_binding_refusals(no_device):
    M, N, K, n, R = 20, 256, 384, 3, 16
    good = dict(x=_bf16(M, K), w=_fp8(N, K), w_scale=torch.zeros(2, 3), lora_a=_bf16(n, R, K), lora_b=_bf16(n, N, R),
                lora_scale=torch.zeros(n), adapter_ids=_i32(M), out=_bf16(M, N), act_q=_fp8(M, K),
                act_scale=torch.zeros(M, 3), act_scale_km=torch.zeros(3, 32), workspace=None)
    bad = [(name, good[name].to(dt), TypeError, f"{name} must be") for name, dt in (
        ("x", torch.float16), ("x", torch.float32), ("w", torch.bfloat16), ("w_scale", torch.float64),
        ("lora_a", torch.float16), ("lora_a", torch.float32), ("lora_b", torch.float16), ("lora_b", torch.float32),
        ("lora_scale", torch.bfloat16), ("adapter_ids", torch.int64), ("out", torch.uint8), ("out", torch.float32),
        ("act_q", torch.float32), ("act_scale", torch.bfloat16), ("act_scale_km", torch.float16))]
    bad += [("w_scale", torch.zeros(3, 2), ValueError, "w_scale"), ("act_q", _fp8(M - 1, K), ValueError, "act_q has"),
            ("act_scale", torch.zeros(M - 1, 3), ValueError, "act_scale has"),
            ("act_scale_km", torch.zeros(3, 16), ValueError, "act_scale_km has"),
            ("adapter_ids", _i32(M + 1), ValueError, "adapter_ids has"), ("out", _bf16(M, N + 1), ValueError, "disagree"),
            ("lora_scale", torch.zeros(n - 1), ValueError, "lora_scale has"), ("x", None, AttributeError, "shape")]
    _each_refused(fp8q.fp8q_proj_lora, good, bad)
    # scratch of a larger batch serves a smaller one
    larger = dict(act_q=_fp8(M + 9, K), act_scale=torch.zeros(M + 9, 3), act_scale_km=torch.zeros(3, 48))
    _each_refused(fp8q.fp8q_proj_lora, {**good, **larger}, [])


def test_expert_binding_refusals(no_device):
    T, E, k, H, I = 20, 4, 2, 256, 128
    R = T * k
    combine = dict(y=_bf16(R, H), weights=torch.zeros(T, k), pos=_i32(R), offsets=_i32(E + 1), out=_bf16(T, H))
    _each_refused(fp8q.fp8q_moe_combine, combine, [
        ("y", torch.zeros(R, H), TypeError, "y must be"), ("out", _fp8(T, H), TypeError, "out must be"),
        ("y", _bf16(R, H).half(), TypeError, "y must be"), ("pos", _i32(R - 1), ValueError, "pos has"),
        ("weights", _bf16(T, k), TypeError, "weights must be")])
    grouped = dict(a=_fp8(T, H), a_scale_km=torch.zeros(2, 32), w=_fp8(E, I, H), w_scale=torch.zeros(E, 1, 2),
                   offsets=_i32(E + 1), out=_bf16(R, I), order=_i32(R), top_k=k)
    _each_refused(fp8q.fp8q_gemm_grouped, grouped, [
        ("out", _fp8(R, I), TypeError, "out must be"), ("out", torch.zeros(R, I), TypeError, "out must be"),
        ("a", _bf16(T, H), TypeError, "a must be"), ("w", _bf16(E, I, H), TypeError, "w must be"),
        ("w_scale", _bf16(E, 1, 2), TypeError, "w_scale must be"), ("a_scale_km", torch.zeros(2, 16), ValueError, "scale"),
        ("a_scale_km", _bf16(2, 32), TypeError, "a_scale_km must be"), ("offsets", _i32(E), ValueError, "offsets has")])
    ffn = dict(x=_bf16(T, H), weights=torch.zeros(T, k), order=_i32(R), pos=_i32(R), offsets=_i32(E + 1),
               w_gate=_fp8(E, I, H), w_gate_scale=torch.zeros(E, 1, 2), w_up=_fp8(E, I, H),
               w_up_scale=torch.zeros(E, 1, 2), w_down=_fp8(E, H, I), w_down_scale=torch.zeros(E, 2, 1),
               out=_bf16(T, H), workspace=None)
    _each_refused(fp8q.fp8q_moe_ffn, ffn, [
        ("x", torch.zeros(T, H), TypeError, "x must be"), ("x", _bf16(T, H).half(), TypeError, "x must be"),
        ("out", _fp8(T, H), TypeError, "out must be"), ("w_gate", _bf16(E, I, H), TypeError, "w_gate must be"),
        ("w_up", _bf16(E, I, H), TypeError, "w_up must be"), ("w_down", _bf16(E, H, I), TypeError, "w_down must be"),
        ("w_up_scale", _bf16(E, 1, 2), TypeError, "w_up_scale must be"), ("order", _i32(R + 1), ValueError, "order has"),
        ("weights", _bf16(T, k), TypeError, "weights must be")])
