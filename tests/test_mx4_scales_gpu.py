"""GPU tests of the MXFP4 products over the whole range of scales and activations: in every kernel that the plans
choose, single weights read to the bit, whose numbers may lie outside the range of the 16-bit type or of FP32 while
their products do not, and sums of the largest and least operands against the definition in 64 bits."""
import pytest
import torch

from oracle import moe as om
from oracle import mx4 as ox
from test_mx4_gpu import BF16, DEV, F16, F32, NAN, U8, coded, gen, in_ones, normal
from test_mx4_kernels_gpu import few, many

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()
    return m


def odd_rows(t):
    """Rows at odd multiples of 2 bytes, NaN between them; codes and scales inside bytes of 0xff."""
    if t.dtype == U8:
        return in_ones(t)
    M, K = t.shape
    buf = torch.full((M * (K + 1 + K % 2) + 1,), NAN, dtype=t.dtype, device=DEV)
    v = buf[1:].view(M, -1)[:, :K]
    v.copy_(t)
    return v


def here(t):
    return t.to(DEV)


def any_address(*plan):
    return many(*plan).replace("rows,", "rows at any address,")


# every kernel for 16-bit rows, and every way through it: whole units and an end of K, K in pieces, 16 and 32 columns
# (the last shape of each kernel that takes any K ends inside a block)
KERNELS = [
    (5, 300, 1100, few(16, 16), here), (1, 90, 512, few(16, 16), here), (3, 72, 9000, few(16, 16, 4), here), (5, 300, 1101, few(16, 16), odd_rows),
    (13, 300, 1100, few(16, 16), here), (13, 8200, 520, few(16, 32), here), (16, 100, 8300, few(16, 16, 4), here), (30, 300, 1100, few(32, 16), here),
    (29, 4096, 8200, few(32, 32, 2), here), (35, 300, 1100, few(36, 16), here), (33, 4096, 8192, few(36, 32, 2), here),
    (40, 300, 1120, "aligned words, 48x64", here), (20, 4200, 1120, "aligned words, 32x64", here), (40, 300, 8192, "aligned words, 48x64 tiles, K in 8", here),
    (40, 300, 1100, "any layout, 48x64", here), (20, 4200, 333, "any layout, 32x64", here),
    (140, 200, 1024, many(64, 128), here), (140, 200, 1056, many(64, 128), here), (140, 200, 1000, many(64, 128), here), (129, 100, 1001, any_address(64, 128), here),
    (100, 4096, 4096, many(64, 128, 4), here), (1100, 4096, 256, many(128, 256), here), (1100, 4096, 584, many(128, 256), here),
    (1100, 4096, 333, any_address(128, 256), here)]


def scale_bytes(g, lo, hi, *shape):
    """lo .. hi, the three at either end in a third of them."""
    ends = torch.tensor([lo, lo + 1, lo + 2, hi - 2, hi - 1, hi], dtype=U8)
    S = torch.randint(lo, hi + 1, shape, generator=g, dtype=U8)
    return torch.where(torch.rand(shape, generator=g) < 1 / 3, ends[torch.randint(0, 6, shape, generator=g)], S)


def one_weight_each(g, M, K, dtype, exponents):
    """Rows of zeros but for a power of two, at K's end in the first of them, and where it is."""
    at = torch.randint(0, K, (M,), generator=g)
    at[0] = K - 1
    A = torch.zeros(M, K, dtype=dtype)
    A[torch.arange(M), at] = torch.ldexp(torch.ones(M), torch.randint(exponents[0], exponents[1] + 1, (M,), generator=g)).to(dtype)
    return A, at


@pytest.mark.parametrize("M,N,K,plan,place", KERNELS)
@pytest.mark.parametrize("dtype,lo,hi,exponents", [
    (BF16, 0, 130, (0, 20)), (BF16, 124, 254, (-40, 0)), (F16, 0, 130, (0, 15)), (F16, 124, 254, (-14, 0)), (F16, 104, 140, (0, 15))])
def test_single_weights(dg, M, N, K, plan, place, dtype, lo, hi, exponents):
    # a product of two numbers of few bits: FP32 holds it, or it is infinite there; all other products are zeros
    g = gen(M, N, K, lo)
    A, at = one_weight_each(g, M, K, dtype, exponents)
    Q, _ = coded(g, N, K)
    S = scale_bytes(g, lo, hi, N, -(-K // 32))
    a, q, s = place(A), place(Q), place(S)
    C = torch.full((M, N), NAN, device=DEV)
    assert dg.gemm_mx4_plan(a, q, s, C).startswith(plan), dg.gemm_mx4_plan(a, q, s, C)
    dg.gemm_mx4(a, q, s, C)
    want = (A[torch.arange(M), at].double()[:, None] * ox.values(Q, S, K)[:, at].t()).to(F32)
    C = C.cpu()
    assert torch.equal(C, want), f"{int((C != want).sum())} of {C.numel()} differ, {int(C.isnan().sum())} NaN"


@pytest.mark.parametrize("dtype,lo,hi,exponents", [(BF16, 124, 254, (-40, 0)), (BF16, 0, 130, (0, 20)), (F16, 124, 254, (-14, 0)), (F16, 104, 140, (0, 15))])
@pytest.mark.parametrize("counts,N,K,plan", [
    ([1, 5, 0, 30, 2, 9], 4096, 1100, few(16, 32)), ([1, 0, 0, 1], 70, 1100, few(16, 16)), ([40, 9, 20, 22, 21], 512, 1120, "aligned words, 32x64"),
    ([40, 39, 20, 32, 41], 512, 1101, "any layout, 48x64"), ([60, 70, 0, 90, 64], 4096, 640, many(64, 128)),
    ([300, 0, 520, 200], 4096, 333, any_address(128, 256))])
def test_single_weights_of_experts(dg, counts, N, K, plan, dtype, lo, hi, exponents):
    g = gen(sum(counts), N, lo)
    E, n = len(counts), sum(counts) + 1
    off = torch.tensor([0] + counts).cumsum(0).int()
    A, at = one_weight_each(g, n, K, dtype, exponents)
    Q, _ = coded(g, E * N, K)
    Q, S = Q.view(E, N, -1), scale_bytes(g, lo, hi, E, N, -(-K // 32))
    C = torch.full((n, N), NAN, device=DEV)
    args = here(A), here(off), here(Q), here(S), C
    assert dg.moe_gemm_mx4_plan(*args).startswith(plan), dg.moe_gemm_mx4_plan(*args)
    dg.moe_gemm_mx4(*args)
    want = torch.zeros(n, N, dtype=torch.float64)
    for e, c in enumerate(counts):
        r = torch.arange(int(off[e]), int(off[e]) + c)
        want[r] = A[r, at[r]].double()[:, None] * ox.values(Q[e], S[e], K)[:, at[r]].t()
    C, want = C.cpu(), want.to(F32)
    assert torch.equal(C, want), f"{int((C != want).sum())} of {C.numel()} differ, {int(C.isnan().sum())} NaN"


@pytest.mark.parametrize("M,N,K,plan,place", KERNELS)
def test_scales_past_bf16_here_and_there(dg, M, N, K, plan, place):
    # a few blocks of scales 253 and 254, one of them zeros, others with one weight that a small activation meets: every
    # other sum is what it would be without them, of all kinds of scales
    g = gen(M, N, K, 3)
    A = normal(g, M, K, dtype=BF16, spread=0.5)
    Q, S = coded(g, N, K, (100, 140))
    blocks = S.shape[1]
    for n, b, k, byte, code in ((7, 0, None, 254, 0), (N - 3, blocks - 1, K - 1, 253, 0x6), (N // 2, blocks // 2, 32 * (blocks // 2), 254, 0xF)):
        Q[n, 16 * b:16 * b + 16] = 0
        S[n, b] = byte
        if k is not None:
            Q[n, k // 2] = code << (4 * (k % 2))
            A[:, k] = torch.randn(M, generator=g).to(BF16) * 2.0 ** -100
    a, q, s = place(A), place(Q), place(S)
    C = torch.full((2, M, N), NAN, device=DEV)
    assert dg.gemm_mx4_plan(a, q, s, C[0]).startswith(plan), dg.gemm_mx4_plan(a, q, s, C[0])
    for c in C:
        dg.gemm_mx4(a, q, s, c)
    om.check(C[0], ox.gemm(A, None, Q, S, K, 0, F32), plan)
    assert torch.equal(C[0], C[1])


@pytest.mark.parametrize("M,N,K,plan,place", KERNELS)
@pytest.mark.parametrize("size,scales", [(2.0 ** 120, (40, 61)), (2.0 ** 20, (0, 3)), (2.0 ** -100, (225, 255))])
def test_largest_and_least_operands(dg, M, N, K, plan, place, size, scales):
    # BF16 rows whose sums without the scales pass FP32, the least weights, and the largest against small rows
    g = gen(M, N, K, 4)
    A = ((1 + torch.rand(M, K, generator=g)) * size * (2 * torch.randint(0, 2, (M, K), generator=g) - 1)).to(BF16)
    if size > 1e30:
        A *= 2.0 ** torch.randint(0, 7, (M, K), generator=g).to(BF16)       # up to 2^127
    Q, S = coded(g, N, K, scales)
    a, q, s = place(A), place(Q), place(S)
    C = torch.full((M, N), NAN, device=DEV)
    assert dg.gemm_mx4_plan(a, q, s, C).startswith(plan), dg.gemm_mx4_plan(a, q, s, C)
    dg.gemm_mx4(a, q, s, C)
    assert A.isfinite().all() and C.isfinite().all(), f"{int((~C.isfinite()).sum())} not finite"
    om.check(C, ox.gemm(A, None, Q, S, K, 0, F32), plan)


def test_the_largest_number_quantised(dg):
    # DG_MX4_CEIL gives FP32's largest number 4 times 2^126: infinite read back, finite in every product with small rows
    f = torch.finfo(F32)
    W = torch.full((40, 64), f.max, device=DEV)
    W[1:, 3] = 1.75 * 2.0 ** 127
    W[::2] *= -1
    Q, S = torch.zeros(40, 32, dtype=U8, device=DEV), torch.zeros(40, 2, dtype=U8, device=DEV)
    dg.quant_mx4(W, Q, S, dg.DG_MX4_CEIL)
    assert (S == 253).all() and ((Q & 0x77) == 0x66).all()
    assert torch.equal(dg.dequant_mx4(Q, S, torch.zeros_like(W)), W * float("inf"))
    for M in (1, 13, 40, 200):
        A = torch.zeros(M, 64, dtype=BF16, device=DEV)
        A[:, ::2] = 2.0 ** -30
        C = dg.gemm_mx4(A, Q, S, torch.full((M, 40), NAN, device=DEV))
        assert torch.equal(C, (torch.sign(W[:, 0]) * 2.0 ** 103).expand(M, -1))                      # 32 times 2^128 times 2^-30


def zeros_of_both_signs(g, *shape):
    return (torch.randint(0, 2, shape, generator=g) * 8 + torch.randint(0, 2, shape, generator=g) * 128).to(U8)


@pytest.mark.parametrize("M,N,K,plan,place", KERNELS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_zeros_under_any_scale(dg, M, N, K, plan, place, dtype):
    # blocks of zeros of both signs count nothing, whatever scale they are under (but NaN)
    g = gen(M, N, K, 5)
    A = normal(g, M, K, dtype=dtype, spread=0.5)
    Q, S = coded(g, N, K, (118, 128))
    blocks = S.shape[1]
    zero = torch.rand(N, blocks, generator=g) < 0.2
    S = torch.where(zero, scale_bytes(g, 0, 254, N, blocks), S)
    mask = zero.repeat_interleave(16, 1)[:, :Q.shape[1]]
    Q = torch.where(mask, zeros_of_both_signs(g, *Q.shape), Q)
    if K % 2:
        Q[:, -1] &= 15
    a, q, s = place(A), place(Q), place(S)
    C = torch.full((M, N), NAN, device=DEV)
    assert dg.gemm_mx4_plan(a, q, s, C).startswith(plan)
    dg.gemm_mx4(a, q, s, C)
    om.check(C, ox.gemm(A, None, Q, S, K, 0, F32), plan)


@pytest.mark.parametrize("M,N,K,plan", [
    (5, 300, 1100, few(16, 16)), (30, 300, 1101, few(32, 16)), (50, 300, 1024, few(64, 16)), (70, 300, 90, "element loads"), (70, 300, 777, "vector loads, 64x64"),
    (70, 300, 1000, "direct loads, 64x64"), (1030, 2900, 512, "ring loads, 128x128"), (1030, 2900, 500, "vector loads, 128x128"), (1030, 2900, 1000, "direct loads, 128x128"),
    (4000, 3300, 512, "ring loads, 256x256"), (4000, 3300, 304, "direct loads, 256x256")])
def test_zeros_of_codes_under_any_scale(dg, M, N, K, plan):
    # and so for blocks of either operand in products of codes, the other's largest scale against them
    g = gen(M, N, K, 6)
    ops = []
    for rows in (M, N):
        Q, S = coded(g, rows, K, (118, 128))
        zero = torch.rand(rows, S.shape[1], generator=g) < 0.2
        S = torch.where(zero, scale_bytes(g, 0, 254, rows, S.shape[1]), S)
        Q = torch.where(zero.repeat_interleave(16, 1)[:, :Q.shape[1]], zeros_of_both_signs(g, *Q.shape), Q)
        if K % 2:
            Q[:, -1] &= 15
        ops += [Q, S]
    A, SA, Q, S = ops
    # the last block of either operand: zeros of one under the largest scale, codes of the other under it
    A[0, 16 * (S.shape[1] - 1):], SA[0, -1], S[:, -1] = 0, 254, 254
    if M > 1:
        SA[1:, -1] = 1
    C = torch.full((M, N), NAN, device=DEV)
    args = here(A), here(Q), here(S), C
    assert dg.gemm_mx4_plan(*args, SA=here(SA)).startswith(plan), dg.gemm_mx4_plan(*args, SA=here(SA))
    dg.gemm_mx4(*args, SA=here(SA))
    om.check(C, ox.gemm(A, SA, Q, S, K, 0, F32), plan)
