"""Refusals and plans of the MXFP4 entry points on the CPU: every argument is checked before anything is
enqueued, so CPU tensors serve (nothing is dereferenced)."""
import pytest
import torch

import dense_gemm_19_amd as dg

F32, F16, BF16, I32, U8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.uint8
M, N, K, E = 6, 48, 96, 4
LIMIT = 2 ** 31 - 4096


def z(*shape, dt=U8):
    return torch.zeros(*shape, dtype=dt)


def one(*shape, dt=U8):
    return z(1, dt=dt).expand(*shape)


def refused(status, f, *args, **kw):
    with pytest.raises(dg.DGError) as e:
        f(*args, stream=0, **kw)
    assert dg.STATUS[e.value.status] == "DG_ERR_" + status


def quant(**kw):
    a = dict(X=z(M, K, dt=BF16), Q=z(M, K // 2), S=z(M, K // 32))
    a.update(kw)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(mode=2), "INVALID_ARG"), (dict(mode=-1), "INVALID_ARG"), (dict(X=z(M, K, dt=I32)), "DTYPE"), (dict(X=z(M, K)), "DTYPE"),
    (dict(Q=z(M, K // 2, dt=torch.float8_e4m3fn)), "DTYPE"), (dict(S=z(M, K // 32, dt=F32)), "DTYPE"),
    (dict(Q=z(M, K)), "SHAPE_MISMATCH"), (dict(Q=z(M + 1, K // 2)), "SHAPE_MISMATCH"), (dict(S=z(M, K // 16)), "SHAPE_MISMATCH"),
    (dict(S=z(M - 1, K // 32)), "SHAPE_MISMATCH"), (dict(X=z(M, K + 1, dt=F16)), "SHAPE_MISMATCH"),
    (dict(Q=z(1, M, K // 2), X=z(2, M, K, dt=BF16)), "SHAPE_MISMATCH"), (dict(Q=z(M, K)[:, ::2]), "UNSUPPORTED_VIEW"),
    (dict(Q=z(K // 2, M).t()), "UNSUPPORTED_VIEW"), (dict(Q=one(M, 1).expand(M, K // 2)), "UNSUPPORTED_VIEW"),
    (dict(Q=z(1, K // 2).expand(M, K // 2)), "STRIDE"), (dict(S=z(1, K // 32).expand(M, K // 32)), "STRIDE"), (dict(X=None), "NULL"),
    (dict(Q=None), "NULL"), (dict(S=None), "NULL"),
])
def test_quant(change, status):
    refused(status, dg.quant_mx4, **quant(**change))


@pytest.mark.parametrize("change,status", [
    (dict(Y=z(M, K, dt=I32)), "DTYPE"), (dict(Q=z(M, K // 2, dt=F16)), "DTYPE"), (dict(Y=z(M, K + 1, dt=F32)), "SHAPE_MISMATCH"),
    (dict(S=z(M, K // 32 + 1)), "SHAPE_MISMATCH"), (dict(Q=z(K // 2, M).t()), "UNSUPPORTED_VIEW"), (dict(Y=one(M, K, dt=F32)), "STRIDE"),
    (dict(Y=z(2, M, K, dt=F32)), "SHAPE_MISMATCH"), (dict(Y=None), "NULL"),
])
def test_dequant(change, status):
    a = dict(Q=z(M, K // 2), S=z(M, K // 32), Y=z(M, K, dt=BF16))
    a.update(change)
    refused(status, dg.dequant_mx4, **a)


def test_alias():
    b = z(M * K * 2)
    x, q = b.view(BF16).view(M, K), b[:M * K // 2].view(M, K // 2)
    refused("ALIAS", dg.quant_mx4, x, q, z(M, K // 32))
    refused("ALIAS", dg.quant_mx4, x, z(M, K // 2), b[-M * 3:].view(M, 3))
    refused("ALIAS", dg.quant_mx4, z(M, K, dt=F32), q, b[M:4 * M].view(M, 3))
    refused("ALIAS", dg.dequant_mx4, q, z(M, K // 32), x)
    c = b[:2 * M * N].view(BF16).view(M, N)
    refused("ALIAS", dg.gemm_mx4, q, z(N, K // 2), z(N, K // 32), c, SA=z(M, K // 32))
    refused("ALIAS", dg.gemm_mx4, z(M, K // 2), z(N, K // 2), z(N, K // 32), c, SA=b[:M * 3].view(M, 3))
    stack = z(2 * M * K // 2).as_strided((2, M, K // 2), (K // 2, K // 2, 1))      # matrices that overlap
    refused("STRIDE", dg.quant_mx4, z(2, M, K, dt=F32), stack, z(2, M, K // 32))


def gemm(codes, experts, **kw):
    lead = (E,) if experts else ()
    a = dict(A=z(M, K // 2) if codes else z(M, K, dt=BF16), Q=z(*lead, N, K // 2), S=z(*lead, N, K // 32), C=z(M, N, dt=F32),
             SA=z(M, K // 32) if codes else None)
    if experts:
        a["offsets"] = z(E + 1, dt=I32)
    a.update(kw)
    return a


@pytest.mark.parametrize("experts", [False, True])
@pytest.mark.parametrize("codes,change,status", [
    (True, dict(SA=None), "NULL"), (False, dict(SA=z(M, K // 32)), "INVALID_ARG"), (True, dict(act=3), "INVALID_ARG"),
    (True, dict(A=z(M, K // 2, dt=F32)), "DTYPE"), (True, dict(A=z(M, K // 2, dt=torch.float8_e4m3fn)), "DTYPE"),
    (True, dict(SA=z(M, K // 32, dt=F32)), "DTYPE"), (False, dict(A=z(M, K, dt=F32)), "DTYPE"), (True, dict(C=z(M, N)), "DTYPE"),
    (True, dict(C=z(M, N, dt=I32)), "DTYPE"), (True, dict(A=z(M, K // 2 + 1)), "SHAPE_MISMATCH"), (True, dict(SA=z(M, K // 32 + 1)), "SHAPE_MISMATCH"),
    (True, dict(SA=z(M + 1, K // 32)), "SHAPE_MISMATCH"), (False, dict(A=z(M, K + 1, dt=F16)), "SHAPE_MISMATCH"),
    (False, dict(A=z(M, K - 2, dt=F16)), "SHAPE_MISMATCH"), (True, dict(C=z(M + 1, N, dt=F32)), "SHAPE_MISMATCH"),
    (True, dict(C=z(M, N + 1, dt=F32)), "SHAPE_MISMATCH"), (True, dict(A=z(K // 2, M).t()), "UNSUPPORTED_VIEW"),
    (False, dict(A=z(K, M, dt=F16).t()), "UNSUPPORTED_VIEW"), (True, dict(C=one(M, N, dt=F32)), "STRIDE"),
    (True, dict(C=z(M, 1, dt=F32).expand(M, N)), "STRIDE"), (True, dict(A=None), "NULL"), (True, dict(Q=None), "NULL"), (True, dict(C=None), "NULL"),
])
def test_gemm(experts, codes, change, status):
    refused(status, dg.moe_gemm_mx4 if experts else dg.gemm_mx4, **gemm(codes, experts, **change))


@pytest.mark.parametrize("change,status", [
    (dict(Q=z(N, K // 2)), "NDIM"), (dict(S=z(N, K // 32)), "NDIM"), (dict(Q=z(E + 1, N, K // 2)), "SHAPE_MISMATCH"),
    (dict(S=z(E + 1, N, K // 32)), "SHAPE_MISMATCH"), (dict(offsets=z(E, dt=I32)), "SHAPE_MISMATCH"),
    (dict(offsets=z(E + 1, dt=torch.int64)), "DTYPE"), (dict(offsets=None), "NULL"), (dict(Q=z(E, K // 2, N).transpose(1, 2)), "UNSUPPORTED_VIEW"),
    (dict(Q=z(0, N, K // 2), S=z(0, N, K // 32)), "SHAPE_MISMATCH"),
])
def test_experts(change, status):
    refused(status, dg.moe_gemm_mx4, **gemm(True, True, **change))


def test_long_and_wide():
    refused("OVERFLOW", dg.gemm_mx4, torch.empty(1, 1 << 21, dtype=BF16), torch.empty(1, 1 << 20, dtype=U8), torch.empty(1, 1 << 16, dtype=U8),
            z(1, 1, dt=F32))
    wide = torch.empty_strided((2, 64), (1 << 24, 1), dtype=BF16)
    refused("OVERFLOW", dg.gemm_mx4, wide, z(N, 32), z(N, 2), z(2, N, dt=F32))
    for size, status in ((LIMIT, "STRIDE"), (LIMIT + 1, "OVERFLOW")):
        refused(status, dg.dequant_mx4, z(1, 16).expand(size, 16), one(size, 1), one(size, 32, dt=F32))
        refused(status, dg.quant_mx4, one(size, 32, dt=F32), z(1, 16).expand(size, 16), one(size, 1))
        refused(status, dg.gemm_mx4, z(1, 16).expand(size, 16), z(N, 16), z(N, 1), one(size, N, dt=F32), SA=one(size, 1))
        refused(status, dg.gemm_mx4, z(M, 16), z(1, 16).expand(size, 16), one(size, 1), one(M, size, dt=F32), SA=z(M, 1))
    for rows, status in ((2 ** 28, "STRIDE"), (2 ** 28 + 1, "OVERFLOW")):
        refused(status, dg.moe_gemm_mx4, z(1, 16).expand(rows, 16), z(2, dt=I32), z(1, N, 16), z(1, N, 1), one(rows, N, dt=F32), SA=one(rows, 1))
    for experts, status in ((16384, "STRIDE"), (16385, "OVERFLOW")):
        refused(status, dg.moe_gemm_mx4, z(M, 16), one(experts + 1, dt=I32), z(1, N, 16).expand(experts, N, 16), one(experts, N, 1),
                one(M, N, dt=F32), SA=z(M, 1))


def test_nothing_to_do():
    # no rows or columns: success without a device
    dg.quant_mx4(z(0, K, dt=F32), z(0, K // 2), z(0, K // 32), stream=0)
    dg.quant_mx4(z(M, 0, dt=F32), z(M, 0), z(M, 0), stream=0)
    dg.quant_mx4(z(0, M, K, dt=F32), z(0, M, K // 2), z(0, M, K // 32), stream=0)
    dg.dequant_mx4(z(0, K // 2), z(0, K // 32), z(0, K, dt=F32), stream=0)
    dg.gemm_mx4(z(0, K // 2), z(N, K // 2), z(N, K // 32), z(0, N, dt=F32), SA=z(0, K // 32), stream=0)
    dg.gemm_mx4(z(M, K, dt=BF16), z(0, K // 2), z(0, K // 32), z(M, 0, dt=F32), stream=0)
    assert dg.gemm_mx4_plan(z(0, K, dt=F16), z(N, K // 2), z(N, K // 32), z(0, N, dt=F32)) == "nothing to do"


def test_plans_refuse_what_the_calls_refuse():
    with pytest.raises(dg.DGError, match="NULL"):
        dg.gemm_mx4_plan(z(M, K // 2), z(N, K // 2), z(N, K // 32), z(M, N, dt=F32))
    with pytest.raises(dg.DGError, match="NDIM"):
        dg.moe_gemm_mx4_plan(z(M, K // 2), z(E + 1, dt=I32), z(N, K // 2), z(E, N, K // 32), z(M, N, dt=F32), SA=z(M, K // 32))
    assert dg.STATUS[dg.lib().dg_gemm_mx4_plan(None, None, None, None, None, None, 8)] == "DG_ERR_INVALID_ARG"
    assert dg.STATUS[dg.lib().dg_moe_gemm_mx4_plan(None, None, None, None, None, None, None, 0)] == "DG_ERR_NULL"


def test_gather_takes_codes():
    dg.moe_gather(z(M, K // 2), z(0, dt=I32), 2, z(0, K // 2), stream=0)
    refused("DTYPE", dg.moe_gather, z(M, K // 2), z(8, dt=I32), 2, z(8, K // 2, dt=torch.float8_e4m3fn))
