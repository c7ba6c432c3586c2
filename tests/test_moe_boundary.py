"""Refusals of the mixture-of-experts and 4-bit entry points on the CPU: every
argument is checked before anything is enqueued, so CPU tensors serve (nothing
is dereferenced)."""
import pytest
import torch

import dense_gemm_19_amd as dg

F32, F16, BF16, I32, I64, U8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64, torch.uint8
T, K, E, H, N = 6, 2, 4, 32, 48
R = T * K


def z(*shape, dt=BF16):
    return torch.zeros(*shape, dtype=dt)


def refused(status, f, *args, **kw):
    with pytest.raises(dg.DGError) as e:
        f(*args, stream=0, **kw)
    assert dg.STATUS[e.value.status] == "DG_ERR_" + status


def overlapping(*shape, dt=BF16):
    return z(shape[-1], dt=dt).expand(*shape)


def sort_args(**kw):
    a = dict(ids=z(T, K, dt=I64), E=E, offsets=z(E + 1, dt=I32), order=z(R, dt=I32), pos=z(T, K, dt=I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(E=0), "INVALID_ARG"), (dict(E=2049), "INVALID_ARG"), (dict(ids=z(T, K, dt=F32)), "DTYPE"),
    (dict(ids=z(T, K, dt=U8)), "DTYPE"), (dict(offsets=z(E + 1, dt=I64)), "DTYPE"), (dict(pos=z(T, K, dt=I64)), "DTYPE"),
    (dict(offsets=z(E, dt=I32)), "SHAPE_MISMATCH"), (dict(order=z(R - 1, dt=I32)), "SHAPE_MISMATCH"),
    (dict(order=z(T, K, dt=I32)), "SHAPE_MISMATCH"), (dict(pos=z(K, T, dt=I32)), "SHAPE_MISMATCH"),
    (dict(order=z(2 * R, dt=I32)[::2]), "UNSUPPORTED_VIEW"), (dict(pos=z(K, T, dt=I32).t()), "UNSUPPORTED_VIEW"),
    (dict(offsets=z(2 * E + 2, dt=I32)[::2]), "UNSUPPORTED_VIEW"),
])
def test_sort(change, status):
    refused(status, dg.moe_sort, **sort_args(**change))


def test_sort_alias():
    p = z(R, dt=I32)
    refused("ALIAS", dg.moe_sort, **sort_args(order=p, pos=p.view(T, K)))
    refused("ALIAS", dg.moe_sort, **sort_args(ids=p.view(T, K), order=p))


@pytest.mark.parametrize("X,order,k,Xs,status", [
    (z(T, H), z(R, dt=I32), 0, z(R, H), "INVALID_ARG"), (z(T, H), z(R, dt=I32), 2, z(R, H, dt=F16), "DTYPE"),
    (z(T, H, dt=I32), z(R, dt=I32), 2, z(R, H, dt=I32), "DTYPE"), (z(T, H), z(R, dt=I64), 2, z(R, H), "DTYPE"),
    (z(T, H), z(R, dt=I32), 2, z(R, H + 1), "SHAPE_MISMATCH"), (z(T, H), z(R + 1, dt=I32), 2, z(R, H), "SHAPE_MISMATCH"),
    (z(T, H), z(R, dt=I32), 2, overlapping(R, H), "STRIDE"),
])
def test_gather(X, order, k, Xs, status):
    refused(status, dg.moe_gather, X, order, k, Xs)


def test_gather_alias():
    X = z(R, H)
    refused("ALIAS", dg.moe_gather, X[:T], z(R, dt=I32), 2, X)


@pytest.mark.parametrize("change,status", [
    (dict(Ys=z(R, H, dt=F16)), "DTYPE"), (dict(Ys=z(R, H, dt=I32), Y=z(T, H, dt=I32)), "DTYPE"),
    (dict(pos=z(T, K, dt=I64)), "DTYPE"), (dict(w=z(T, K, dt=I32)), "DTYPE"), (dict(Y=z(T, H + 1)), "SHAPE_MISMATCH"),
    (dict(pos=z(T + 1, K, dt=I32)), "SHAPE_MISMATCH"), (dict(w=z(T, K + 1)), "SHAPE_MISMATCH"),
    (dict(Y=overlapping(T, H)), "STRIDE"),
])
def test_combine(change, status):
    a = dict(Ys=z(R, H), pos=z(T, K, dt=I32), Y=z(T, H), w=z(T, K, dt=F32))
    a.update(change)
    refused(status, dg.moe_combine, **a)


@pytest.mark.parametrize("change,status", [
    (dict(dYs=z(R, H, dt=F16)), "DTYPE"), (dict(dw=z(T, K, dt=F16)), "DTYPE"), (dict(dYs=z(R + 1, H)), "SHAPE_MISMATCH"),
    (dict(dw=z(T, K + 1, dt=F32)), "SHAPE_MISMATCH"), (dict(dYs=overlapping(R, H)), "STRIDE"), (dict(w=None), "NULL"),
    (dict(dw=overlapping(T, K, dt=F32)), "STRIDE"),
])
def test_combine_grad(change, status):
    a = dict(dY=z(T, H), Ys=z(R, H), pos=z(T, K, dt=I32), w=z(T, K, dt=F32), dYs=z(R, H), dw=z(T, K, dt=F32))
    a.update(change)
    refused(status, dg.moe_combine_grad, **a)


def test_combine_grad_alias():
    Ys = z(R, H)
    refused("ALIAS", dg.moe_combine_grad, z(T, H), Ys, z(T, K, dt=I32), z(T, K, dt=F32), Ys, z(T, K, dt=F32))


@pytest.mark.parametrize("change,status", [
    (dict(A=z(R, H, dt=F32), W=z(E, H, N, dt=F32)), "DTYPE"), (dict(W=z(E, H, N, dt=F16)), "DTYPE"),
    (dict(C=z(R, N, dt=I32)), "DTYPE"), (dict(offsets=z(E + 1, dt=I64)), "DTYPE"), (dict(W=z(H, N)), "NDIM"),
    (dict(W=z(E, H + 1, N)), "SHAPE_MISMATCH"), (dict(C=z(R, N + 1)), "SHAPE_MISMATCH"), (dict(C=z(R + 1, N)), "SHAPE_MISMATCH"),
    (dict(offsets=z(E, dt=I32)), "SHAPE_MISMATCH"), (dict(W=z(0, H, N), offsets=z(1, dt=I32)), "SHAPE_MISMATCH"),
    (dict(C=overlapping(R, N)), "STRIDE"), (dict(act=3), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"),
])
def test_moe_gemm(change, status):
    a = dict(A=z(R, H), offsets=z(E + 1, dt=I32), W=z(E, H, N), C=z(R, N))
    a.update(change)
    refused(status, dg.moe_gemm, **a)


def test_moe_gemm_alias():
    buf = z(E * H * N)
    W = buf.view(E, H, N)
    refused("ALIAS", dg.moe_gemm, z(R, H), z(E + 1, dt=I32), W, buf[-R * N:].view(R, N))   # only the last expert's weights


@pytest.mark.parametrize("change,status", [
    (dict(D=z(R, N, dt=F16)), "DTYPE"), (dict(dW=z(E, H, N, dt=I32)), "DTYPE"), (dict(dW=z(H, N)), "NDIM"),
    (dict(D=z(R + 1, N)), "SHAPE_MISMATCH"), (dict(dW=z(E, N, H)), "SHAPE_MISMATCH"), (dict(offsets=z(E + 2, dt=I32)), "SHAPE_MISMATCH"),
    (dict(dW=z(1, H, N).expand(E, H, N)), "STRIDE"), (dict(dW=z(E, H, 1).expand(E, H, N)), "STRIDE"),
])
def test_moe_gemm_wgrad(change, status):
    a = dict(A=z(R, H), D=z(R, N), offsets=z(E + 1, dt=I32), dW=z(E, H, N, dt=F32))
    a.update(change)
    refused(status, dg.moe_gemm_wgrad, **a)


@pytest.mark.parametrize("experts", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(A=z(R, 64, dt=F32)), "DTYPE"), (dict(Q=z(N, 32, dt=I32)), "DTYPE"), (dict(S=z(N, 2, dt=U8)), "DTYPE"),
    (dict(Z=z(N, 2)), "DTYPE"), (dict(C=z(R, N, dt=U8)), "DTYPE"), (dict(group=16), "INVALID_ARG"), (dict(group=0), "INVALID_ARG"),
    (dict(group=-32), "INVALID_ARG"), (dict(group=48), "INVALID_ARG"), (dict(act=7), "INVALID_ARG"),
    (dict(Q=z(N, 33, dt=U8)), "SHAPE_MISMATCH"), (dict(S=z(N, 3)), "SHAPE_MISMATCH"), (dict(Z=z(N, 1, dt=U8)), "SHAPE_MISMATCH"),
    (dict(C=z(R, N + 1)), "SHAPE_MISMATCH"), (dict(A=z(64, R).t()), "UNSUPPORTED_VIEW"),
    (dict(Q=z(N, 64, dt=U8)[:, ::2]), "UNSUPPORTED_VIEW"), (dict(C=overlapping(R, N)), "STRIDE"),
])
def test_w4(change, status, experts):
    a = dict(A=z(R, 64), Q=z(N, 32, dt=U8), S=z(N, 2), C=z(R, N), group=32)
    a.update(change)
    if experts:
        for key in ("Q", "S", "Z"):
            if a.get(key) is not None:
                a[key] = torch.stack([a[key]] * E) if a[key].is_contiguous() else a[key].unsqueeze(0).expand(E, *a[key].shape)
        refused(status, dg.moe_gemm_w4, offsets=z(E + 1, dt=I32), **a)
    else:
        refused(status, dg.gemm_w4, **a)


def test_w4_experts_count():
    a = dict(A=z(R, 64), offsets=z(E + 1, dt=I32), Q=z(E, N, 32, dt=U8), S=z(E, N, 2), C=z(R, N), group=32)
    refused("SHAPE_MISMATCH", dg.moe_gemm_w4, **{**a, "S": z(E + 1, N, 2)})
    refused("SHAPE_MISMATCH", dg.moe_gemm_w4, **{**a, "offsets": z(E, dt=I32)})
    refused("NDIM", dg.moe_gemm_w4, **{**a, "Q": z(N, 32, dt=U8)})


def test_w4_too_long():
    refused("OVERFLOW", dg.gemm_w4, torch.empty(1, 1 << 21, dtype=BF16), torch.empty(1, 1 << 20, dtype=U8),
            torch.empty(1, 1 << 14), z(1, 1), 128)
    refused("OVERFLOW", dg.gemm_w4, torch.empty_strided((2, 64), (1 << 24, 1), dtype=BF16), z(N, 32, dt=U8), z(N, 2), z(2, N), 32)


def test_views_of_the_binding_match_the_struct():
    view = dg._bind().view
    for t in (z(3), z(3, 4).t(), z(2, 3, 4)[:, ::2], z(1, 2, 3, 4, dt=F32), torch.tensor(1.0), z(0, 4, dt=U8), z(2, dt=I64),
              z(5, dt=I32), z(2, dt=F16), z(4, dt=torch.float8_e4m3fn)):
        a, b = dg.View.from_buffer_copy(view(t)), dg.view_of(t)
        assert (a.ptr, a.ndim, list(a.shape), list(a.stride), a.dtype) == (b.ptr, b.ndim, list(b.shape), list(b.stride), b.dtype)


@pytest.mark.parametrize("bad,error", [(torch.zeros(2, dtype=torch.int16), TypeError), ([1, 2], TypeError),
                                       (torch.zeros(1, 1, 1, 1, 1), ValueError)])
def test_arguments_that_are_no_views(bad, error):
    with pytest.raises(error):
        dg.moe_gather(z(T, H), bad, 2, z(R, H), stream=0)
    with pytest.raises(TypeError):
        dg._bind().moe_gather(z(T, H), z(R, dt=I32), 2)
    with pytest.raises(OverflowError):
        dg.moe_gather(z(T, H), z(R, dt=I32), 1 << 40, z(R, H), stream=0)
    refused("NULL", dg.moe_gather, z(T, H), None, 2, z(R, H))


def test_nothing_to_do():
    # no rows or columns: success without a device
    dg.moe_gemm(z(0, H), z(E + 1, dt=I32), z(E, H, N), z(0, N), stream=0)
    dg.gemm_w4(z(3, 64), z(0, 32, dt=U8), z(0, 2), z(3, 0), 32, stream=0)
    dg.moe_gather(z(T, H), z(0, dt=I32), 2, z(0, H), stream=0)
    dg.moe_combine(z(0, H), z(0, K, dt=I32), z(0, H), stream=0)
    dg.moe_gemm_wgrad(z(R, 0), z(R, N), z(E + 1, dt=I32), z(E, 0, N), stream=0)


# An extent that a kernel's 32-bit walk could step past 2^31 is refused; the next smaller one is not (an
# output of one repeated element is then refused for that).
LIMIT = 2 ** 31 - 4096


def one(*shape, dt=BF16):
    return z(1, dt=dt).expand(*shape)


@pytest.mark.parametrize("size,status", [(LIMIT, "STRIDE"), (LIMIT + 1, "OVERFLOW"), (2 ** 31 - 1, "OVERFLOW")])
def test_extents_next_to_32_bits(size, status):
    i32 = lambda *s: z(*s, dt=I32)   # noqa: E731
    for dt in (F32, BF16):
        refused(status, dg.moe_gather, one(2, size, dt=dt), i32(2), 1, one(2, size, dt=dt))
        refused(status, dg.moe_combine, one(2, size, dt=dt), i32(2, 1), one(2, size, dt=dt))
        refused(status, dg.moe_combine_grad, one(2, size, dt=dt), one(2, size, dt=dt), i32(2, 1), z(2, 1, dt=F32),
                one(2, size, dt=dt), z(2, 1, dt=F32))
    many = one(2, size, dt=I32)
    refused(status, dg.moe_combine, z(2, H), many, one(2, H))
    refused(status, dg.moe_combine_grad, z(2, H), z(2, H), many, one(2, size, dt=F32), z(2, H), one(2, size, dt=F32))
    refused(status, dg.moe_gemm, one(2, size), i32(2), one(1, size, 8), one(2, 8))
    refused(status, dg.moe_gemm, one(2, 8), i32(2), one(1, 8, size), one(2, size))
    refused(status, dg.moe_gemm_wgrad, one(size, 8), one(size, 8), i32(2), one(1, 8, 8))
    refused(status, dg.moe_gemm_wgrad, one(2, size), one(2, 8), i32(2), one(1, size, 8))
    refused(status, dg.moe_gemm_wgrad, one(2, 8), one(2, size), i32(2), one(1, 8, size))
    refused(status, dg.gemm_w4, z(2, 32), z(1, 16, dt=U8).expand(size, 16), one(size, 1), one(2, size), 32)
    refused(status, dg.gemm_w4, z(1, 32).expand(size, 32), z(8, 16, dt=U8), z(8, 1), one(size, 8), 32)


def test_plans_refuse_what_the_calls_refuse():
    i32 = lambda *s: z(*s, dt=I32)   # noqa: E731
    with pytest.raises(dg.DGError, match="INVALID_ARG"):
        dg.moe_sort_plan(i32(T, K), 0, i32(1), i32(R), i32(T, K))
    with pytest.raises(dg.DGError, match="SHAPE_MISMATCH"):
        dg.moe_gemm_plan(z(R, H), i32(E), z(E, H, N), z(R, N))
    with pytest.raises(dg.DGError, match="STRIDE"):
        dg.moe_gemm_wgrad_plan(z(R, H), z(R, N), i32(E + 1), z(1, H, N).expand(E, H, N))
    with pytest.raises(dg.DGError, match="DTYPE"):
        dg.gemm_w4_plan(z(R, 64), z(N, 32), z(N, 2), z(R, N), 32)
    with pytest.raises(dg.DGError, match="NDIM"):
        dg.moe_gemm_w4_plan(z(R, 64), i32(E + 1), z(N, 32, dt=U8), z(E, N, 2), z(R, N), 32)
    # a grid of 2^32 threads and the largest below it
    for experts, ok in ((2 ** 24, False), (2 ** 24 - 1, True)):
        args = (one(16, 8), one(16, 8), torch.empty(experts + 1, dtype=I32), torch.empty(experts, 8, 8, dtype=BF16))
        if ok:
            assert dg.moe_gemm_wgrad_plan(*args).endswith(f"{experts} workgroups")
        else:
            with pytest.raises(dg.DGError, match="OVERFLOW"):
                dg.moe_gemm_wgrad_plan(*args)
    assert dg.moe_gemm_plan(z(0, H), i32(E + 1), z(E, H, N), z(0, N)) == "nothing to do"
    assert dg.STATUS[dg.lib().dg_gemm_w4_plan(None, None, None, None, None, 32, None, 8)] == "DG_ERR_INVALID_ARG"
    assert dg.STATUS[dg.lib().dg_gemm_w4_plan(None, None, None, None, None, 32, None, 0)] == "DG_ERR_NULL"


def test_experts_whose_offsets_are_scanned_are_bounded():
    for E, status in ((16384, "STRIDE"), (16385, "OVERFLOW"), (1 << 30, "OVERFLOW")):
        off = one(E + 1, dt=I32)
        refused(status, dg.moe_gemm, z(R, H), off, one(E, H, N), one(R, N))
        refused(status, dg.moe_gemm_w4, z(R, 64), off, z(1, N, 32, dt=U8).expand(E, N, 32), one(E, N, 2), one(R, N), 32)
