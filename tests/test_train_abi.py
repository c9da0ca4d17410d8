"""Refusals and host-side sizes of the operators of a training step (no GPU needed,
no kernel launched): every call here fails a check, or is an empty call that returns
before anything is enqueued."""
import ctypes

import pytest
import torch

import w8a8_fp8_block_amd as fp8q

P = ctypes.c_void_p
BAD, G = P(0x1001), P(0x1000)  # misaligned; aligned but never dereferenced
NULL, SHAPE, ALIGN, VARIANT = 1, 2, 3, 6
BIG = 1 << 40


def _err():
    return fp8q.lib().fp8q_last_error().decode()


def _refused(call, args, names, optional=()):
    """Every pointer refused misaligned, and as NULL (with its name) unless optional."""
    for i, name in names.items():
        for bad, want in ((None, NULL), (BAD, ALIGN)):
            if bad is None and name in optional:
                continue
            a = list(args)
            a[i] = bad
            assert call(*a) == want, name
            assert name in _err()


def test_norm_refusals():
    f = fp8q.lib().fp8q_add_rmsnorm_quant

    def call(x=G, r=G, w=G, h=G, y=G, q=G, srm=G, skm=G, rstd=G, eps=1e-6, M=4, K=256):
        return f(x, r, w, h, y, q, srm, skm, rstd, eps, M, K, None)

    for kw in (dict(K=0), dict(K=200), dict(K=32896), dict(M=1 << 25, K=128), dict(M=0xFFFFFFFF, K=128)):
        assert call(**kw) == SHAPE, kw
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-39):
        assert call(eps=eps) == VARIANT and "eps" in _err()
    _refused(f, (G,) * 9 + (1e-6, 4, 256, None),
             dict(enumerate(("x_bf16", "residual_bf16", "weight_bf16", "h_bf16", "y_bf16", "q_e4m3", "scale_rm",
                             "scale_km", "rstd"))),
             optional=("residual_bf16", "y_bf16", "scale_rm", "scale_km", "rstd"))
    assert call(r=None) == NULL and "without residual" in _err()
    assert call(srm=None, skm=None) == NULL and "scale" in _err()
    assert call(M=0) == 0 and call(M=0, x=None, q=None) == 0
    assert call(M=0, K=100) == SHAPE


def test_norm_grad_refusals():
    f = fp8q.lib().fp8q_add_rmsnorm_grad
    args = [G] * 8 + [BIG, 300, 256, None]
    _refused(f, args, dict(enumerate(("dy_bf16", "dh_bf16", "h_bf16", "weight_bf16", "rstd", "dx_bf16", "dweight",
                                      "workspace"))), optional=("dh_bf16",))
    need = fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(300, 256)
    assert need > 0
    assert f(*(args[:8] + [need - 1] + args[9:])) == SHAPE and "workspace" in _err()
    for K in (0, 130, 32896):
        assert f(*(args[:10] + [K, None])) == SHAPE
        assert fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(300, K) == 0
    assert fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(0, 256) == 0


def test_dual_refusals():
    f = fp8q.lib().fp8q_quant_act_dual
    args = [G] * 5 + [4, 256, None]
    _refused(f, args, dict(enumerate(("x_bf16", "q_e4m3", "scale_km", "q_tok", "exp_tok"))))
    for M, K in ((4, 0), (4, 64), (1 << 25, 128), (0xFFFFFFFF, 128)):
        assert f(*([G] * 5 + [M, K, None])) == SHAPE
    assert f(*([None] * 5 + [0, 256, None])) == 0


@pytest.mark.parametrize("name,args", [
    ("fp8q_gemm_dgrad", ("dy_e4m3", "dy_scale_km", "w_e4m3", "w_scale", "dx_bf16")),
    ("fp8q_gemm_wgrad", ("dy_tok", "dy_exp", "x_tok", "x_exp", "dw_bf16"))])
def test_gradient_product_refusals(name, args):
    f, size = getattr(fp8q.lib(), name), getattr(fp8q, name + "_workspace_bytes")
    _refused(f, [G] * 6 + [BIG, 4, 256, 384, None], dict(enumerate(args)))
    for M, N, K in ((4, 0, 128), (4, 128, 0), (4, 192, 128), (4, 128, 130), (1 << 25, 128, 128), (4, 1 << 25, 128),
                    (4, 128, 1 << 25), (4, 1 << 16, 1 << 16), (0xFFFFFFFF, 128, 128)):
        assert f(*([G] * 6 + [BIG, M, N, K, None])) == SHAPE, (M, N, K)
        assert size(M, N, K) == 0
    some = [(M, N, K) for M in (1, 200, 4576) for N in (128, 5120) for K in (128, 2048) if size(M, N, K)]
    for M, N, K in some:
        need = size(M, N, K)
        assert f(*([G] * 6 + [need - 1, M, N, K, None])) == SHAPE and "workspace" in _err()
        assert f(*([G] * 5 + [None, need, M, N, K, None])) == NULL
        assert f(*([G] * 5 + [BAD, need, M, N, K, None])) == ALIGN


def test_dgrad_empty():
    assert fp8q.lib().fp8q_gemm_dgrad(None, None, None, None, None, None, 0, 0, 128, 128, None) == 0


def test_balance_refusals():
    f = fp8q.lib().fp8q_moe_balance

    def call(lo=G, bf16=0, ids=G, counts=G, prob=G, loss=G, ws=G, nb=BIG, coef=1.0, T=4, E=8, k=2):
        return f(lo, bf16, ids, counts, prob, loss, ws, nb, coef, T, E, k, None)

    for kw in (dict(E=0, k=1), dict(E=513), dict(k=0), dict(k=9), dict(E=64, k=33), dict(T=1 << 31, k=1),
               dict(T=1 << 24, E=512, k=1)):
        assert call(**kw) == SHAPE, kw
    assert call(bf16=2) == VARIANT and call(bf16=-1) == VARIANT
    for name, arg in (("logits", "lo"), ("ids", "ids"), ("counts", "counts"), ("prob", "prob"), ("loss", "loss")):
        assert call(**{arg: None}) == NULL and name in _err()
        assert call(**{arg: BAD}) == ALIGN and name in _err()
    need = fp8q.fp8q_moe_balance_workspace_bytes(100000, 8)
    assert need > 0 and call(T=100000, nb=need - 1) == SHAPE and "workspace" in _err()
    assert fp8q.fp8q_moe_balance_workspace_bytes(1, 8) == 0 and fp8q.fp8q_moe_balance_workspace_bytes(9, 513) == 0


def test_route_grad_refusals():
    f = fp8q.lib().fp8q_moe_route_grad

    def call(lo=G, bf16=0, ids=G, dw=G, counts=G, dloss=G, dl=G, coef=1.0, T=4, E=8, k=2, renorm=1):
        return f(lo, bf16, ids, dw, counts, dloss, dl, coef, T, E, k, renorm, None)

    for kw in (dict(E=0, k=1), dict(E=513), dict(k=0), dict(k=9), dict(T=1 << 24, E=512, k=1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(bf16=2), dict(bf16=-1), dict(renorm=2), dict(renorm=-1)):
        assert call(**kw) == VARIANT
    for name, arg, optional in (("logits", "lo", False), ("ids", "ids", False), ("dweights", "dw", False),
                                ("counts", "counts", True), ("dloss", "dloss", True), ("dlogits", "dl", False)):
        assert call(**{arg: BAD}) == ALIGN and name in _err()
        if not optional:
            assert call(**{arg: None}) == NULL and name in _err()
    assert call(ids=None, dw=None, counts=None) == NULL
    assert call(T=0, lo=None, dl=None) == 0


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 16)
    with pytest.raises(ValueError, match="current GPU"):
        fp8q.fp8q_add_rmsnorm_quant(x, None, w, None, None, q, None, s, None)
    with pytest.raises(ValueError, match="current GPU"):
        fp8q.fp8q_quant_act_dual(x, None, None, q, torch.zeros(1, 256, 4, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2-d"):
        fp8q.fp8q_quant_act_dual(x[0], None, None, q, torch.zeros(1, 256, 4, dtype=torch.uint8))


def test_scalars_need_their_own_alignment_only():
    """loss and dloss are single floats: any multiple of 4 passes their check (here the next
    check refuses the call), no other address does."""
    lib = fp8q.lib()
    for at, want in ((0x1004, "logits"), (0x1008, "logits"), (0x100C, "logits"), (0x1002, "loss"), (0x1006, "loss")):
        st = lib.fp8q_moe_balance(None if want == "logits" else G, 0, G, G, G, P(at), G, BIG, 1.0, 4, 8, 2, None)
        assert st == (NULL if want == "logits" else ALIGN) and want in _err(), hex(at)
    for at, want in ((0x1004, "dlogits"), (0x1008, "dlogits"), (0x100C, "dlogits"), (0x1002, "dloss"), (0x1006, "dloss")):
        st = lib.fp8q_moe_route_grad(G, 0, G, G, G, P(at), None if want == "dlogits" else G, 1.0, 4, 8, 2, 1, None)
        assert st == (NULL if want == "dlogits" else ALIGN) and want in _err(), hex(at)


SIZES = sorted({1, 2, 3, 5, 8, 12, 13, 24, 25, 63, 64, 100, 127, 128, 129, 200, 255, 256, 257, 300, 384, 385, 409, 511,
                512, 513, 700, 1024, 1168, 1500, 2000, 2500, 4096, 4576, 10000, 16384, 40000, 131072})


def test_workspaces_for_several_batch_sizes():
    """What the header promises a program that keeps one buffer: sizes that serve every batch,
    and which sizes never fall as the batch grows."""
    cus = 256
    for K in (128, 256, 384, 640, 1408, 2048, 5120, 6144, 17408, 32768):
        need = [fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, K) for M in SIZES]
        assert max(need) == 1024 * K and all(need)
        assert need[SIZES.index(256)] == 1024 * K
        for N in (128, 512, 2048, 5120, 17408):
            dx = [fp8q.fp8q_gemm_dgrad_workspace_bytes(M, N, K) for M in SIZES]
            assert max(dx) <= cus * 128 * 1024
            dw = [fp8q.fp8q_gemm_wgrad_workspace_bytes(M, N, K) for M in SIZES]
            assert max(dw) <= cus * 64 * 1024 and dw == sorted(dw)
    for E in (1, 8, 64, 160, 512):
        need = [fp8q.fp8q_moe_balance_workspace_bytes(T, E) for T in SIZES]
        assert need == sorted(need)
    # the sizes that do fall, of which the header warns
    assert fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(256, 640) > fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(257, 640)
    assert fp8q.fp8q_gemm_dgrad_workspace_bytes(16, 5120, 6144) > fp8q.fp8q_gemm_dgrad_workspace_bytes(409, 5120, 6144) == 0


def test_one_byte_less_is_refused():
    """At batch sizes on both sides of the rules' borders."""
    f = fp8q.lib().fp8q_add_rmsnorm_grad
    for M in (1, 4, 24, 25, 256, 257, 4576):
        need = fp8q.fp8q_add_rmsnorm_grad_workspace_bytes(M, 640)
        assert f(*([G] * 8 + [need - 1, M, 640, None])) == SHAPE and "workspace" in _err()
    f, size = fp8q.lib().fp8q_gemm_dgrad, fp8q.fp8q_gemm_dgrad_workspace_bytes
    for M in (1, 16, 128, 129, 200):
        need = size(M, 5120, 6144)
        assert need and f(*([G] * 6 + [need - 1, M, 5120, 6144, None])) == SHAPE and "workspace" in _err()
