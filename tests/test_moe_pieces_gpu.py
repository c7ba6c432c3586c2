"""GPU tests of the expert and 4-bit products where K is cut into pieces over workgroups, of
the two ways 4-bit operands are loaded (aligned words and any other layout), of ragged experts
in their rings, and of offsets that overlap; against the definitions in 64 bits (oracle/moe.py)."""
import pytest
import torch

from oracle import moe as om

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()   # raises if the library is missing: there is no fallback
    return m


def normal(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets(counts):
    return torch.tensor([0] + counts).cumsum(0).int()


def nan(*shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def same_again(f, out):
    """A second and third call give the same bits (the pieces are added in a fixed order)."""
    first = out.clone()
    for _ in range(2):
        out.fill_(3)
        f()
        assert torch.equal(out, first)


# few tiles and a long K: aligned, odd N, odd K, any strides
@pytest.mark.parametrize("counts", [[3], [1, 0, 7], [40, 30], [0, 90, 0, 5]], ids=str)
@pytest.mark.parametrize("K,N", [(2048, 64), (1600, 136), (1601, 70), (1032, 33)])
@pytest.mark.parametrize("dtype,act", [(BF16, 2), (F16, 0)])
def test_experts_in_pieces(dg, counts, K, N, dtype, act):
    g = torch.Generator().manual_seed(K + N + sum(counts))
    off, n, E = offsets(counts), sum(counts) + 2, len(counts)
    A, W = normal(g, n, K, dtype=dtype), normal(g, E, K, N, dtype=dtype, scale=K ** -0.5)
    A[n - 2:] = float("nan")                                     # rows of no expert: zero
    v, b = om.experts(A[:n - 2], off, W, act, F32)
    want = torch.cat([v, torch.zeros(2, N, dtype=torch.float64)]), torch.cat([b, torch.zeros(2, N, dtype=torch.float64)])
    o = off.to(DEV)
    for a, w in [(A.to(DEV), W.to(DEV)), (A.to(DEV), W.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)),
                 (A.t().contiguous().to(DEV).t(), W.to(DEV))]:
        C = nan(n, N)
        dg.moe_gemm(a, o, w, C, act)
        om.check(C, want, f"{counts} {K}x{N}")
        same_again(lambda: dg.moe_gemm(a, o, w, C, act), C)


@pytest.mark.parametrize("counts", [[700], [0, 1200, 3], [513, 64, 900]], ids=str)
@pytest.mark.parametrize("K,N", [(64, 128), (72, 33), (5, 130)])
def test_weight_gradient_in_pieces(dg, counts, K, N):
    g = torch.Generator().manual_seed(K + N + sum(counts))
    off, n = offsets(counts), sum(counts) + 2
    A, D = normal(g, n, K), normal(g, n, N)
    A[n - 2:], D[n - 2:] = float("nan"), float("nan")
    want = om.wgrad(A, D, off, F32)
    o = off.to(DEV)
    for a, d in [(A.to(DEV), D.to(DEV)), (A.t().contiguous().to(DEV).t(), D.to(DEV))]:
        dW = nan(len(counts), K, N)
        dg.moe_gemm_wgrad(a, d, o, dW)
        om.check(dW, want, f"{counts} {K}x{N}")
        same_again(lambda: dg.moe_gemm_wgrad(a, d, o, dW), dW)


def weights(g, N, K, G, zeros, st, lead=()):
    groups = -(-K // G)
    Q = torch.randint(0, 256, (*lead, N, (K + 1) // 2), generator=g, dtype=torch.uint8)
    S = ((0.5 + torch.rand(*lead, N, groups, generator=g)) * K ** -0.5).to(st)
    return Q, S, torch.randint(0, 256, (*lead, N, groups), generator=g, dtype=torch.uint8) if zeros else None


def moved(t, by):
    """t on the device, its elements `by` places past an aligned address."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=DEV)[by:].view(t.shape)
    return flat.copy_(t)


# groups that fill whole words or do not, chunks from one to many, all row tiles
@pytest.mark.parametrize("M", [1, 12, 20, 40, 48, 49, 100])
@pytest.mark.parametrize("N,K,G", [(40, 512, 64), (70, 2080, 32), (33, 6176, 96), (96, 9216, 128), (16, 1184, 256)])
def test_w4_layouts(dg, M, N, K, G):
    g = torch.Generator().manual_seed(M + K)
    for dtype, st in ((BF16, BF16), (F16, F32)):
        A = normal(g, M, K, dtype=dtype)
        Q, S, Z = weights(g, N, K, G, True, st)
        want = om.w4(A, Q, S, Z, G, 0, F32)
        for by in ((0, 0, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 0, 0, 0), (0, 3, 0, 0)):   # A, Q, S, Z off their alignment
            a, q, s, z = (moved(t, b) for t, b in zip((A, Q, S, Z), by))
            C = nan(M, N)
            dg.gemm_w4(a, q, s, C, group=G, Z=z)
            om.check(C, want, f"{M}x{N}x{K} moved {by}")
            same_again(lambda: dg.gemm_w4(a, q, s, C, group=G, Z=z), C)


@pytest.mark.parametrize("counts", [[1, 15, 2, 30, 0, 7], [16, 1, 1, 1], [48, 3, 100], [9] * 9], ids=str)
@pytest.mark.parametrize("K", [1024, 5120, 4128])
def test_w4_experts_with_ragged_rows(dg, counts, K):
    # rows above the mean leave the rings fewer slots
    g = torch.Generator().manual_seed(sum(counts) + K)
    n, E, N, G = sum(counts) + 1, len(counts), 40, 32
    off = offsets(counts)
    A = normal(g, n, K)
    Q, S, Z = weights(g, N, K, G, True, BF16, (E,))
    C = nan(n, N)
    dg.moe_gemm_w4(A.to(DEV), off.to(DEV), Q.to(DEV), S.to(DEV), C, group=G, Z=Z.to(DEV))
    v, b = om.w4_experts(A, off, Q, S, Z, G, 0, F32)
    v[n - 1:], b[n - 1:] = 0, 0
    om.check(C, (v, b), f"{counts}")


def test_overlapping_offsets_stay_inside(dg):
    # every expert claims every row: more tiles than the grid has; some result or none, in bounds
    g = torch.Generator().manual_seed(1)
    E, n, K, N = 9, 40, 1024, 64
    off = torch.tensor([0, n] * 5, dtype=torch.int32, device=DEV)
    guard = torch.full((3 * n, N), 7.0, device=DEV)
    A, W = normal(g, n, K).to(DEV), normal(g, E, K, N, scale=0.03).to(DEV)
    Q, S, _ = weights(g, N, K, 64, False, BF16, (E,))
    for _ in range(2):
        dg.moe_gemm(A, off, W, guard[n:2 * n])
        dg.moe_gemm_wgrad(A, A[:, :N].contiguous(), off, torch.zeros(E, K, N, device=DEV))
        dg.moe_gemm_w4(A, off, Q.to(DEV), S.to(DEV), guard[n:2 * n], group=64)
    torch.cuda.synchronize()
    assert (guard[:n] == 7).all() and (guard[2 * n:] == 7).all()
    # and the pieces' counters are as they were: an ordinary call is right
    C = nan(n, N)
    dg.moe_gemm(A, torch.tensor([0] * 9 + [n], dtype=torch.int32, device=DEV), W, C)
    om.check(C, om.experts(A.cpu(), torch.tensor([0] * 9 + [n]), W.cpu(), 0, F32), "after")


def test_gather_of_a_large_batch(dg):
    # an output large enough to be stored past the caches, with rows whose last chunk is partial
    g = torch.Generator().manual_seed(2)
    T, k, H = 12000, 2, 2101
    order = torch.randperm(T * k, generator=g).int()
    order[::97] = -1
    X = normal(g, T, H)
    Xs = dg.moe_gather(X.to(DEV), order.to(DEV), k, torch.full((T * k, H), float("nan"), dtype=BF16, device=DEV))
    want = torch.where((order >= 0)[:, None], X[order.clamp(min=0).long() // k], torch.zeros(1, dtype=BF16))
    assert torch.equal(Xs.cpu(), want)


@pytest.mark.parametrize("M", [1, 16, 30, 90])
@pytest.mark.parametrize("N,K,G", [(68, 2080, 32), (36, 4640, 32), (44, 5920, 128), (20, 1312, 96)])
@pytest.mark.parametrize("st", [F32, F16, BF16])
def test_w4_rows_of_scales_off_words(dg, M, N, K, G, st):
    # odd counts of groups: rows of scales and zero points begin anywhere in a word, the whole run does not
    g = torch.Generator().manual_seed(M + N + K)
    A = normal(g, M, K)
    Q, S, Z = weights(g, N, K, G, True, st)
    for z in (Z, None):
        C = nan(M, N)
        dg.gemm_w4(A.to(DEV), Q.to(DEV), S.to(DEV), C, group=G, Z=None if z is None else z.to(DEV))
        om.check(C, om.w4(A, Q, S, z, G, 0, F32), f"{M}x{N}x{K}")
    E, n = 3, 3 * M + 1
    off = offsets([M, 0, 2 * M])
    A = normal(g, n, K)
    Q, S, Z = weights(g, N, K, G, True, st, (E,))
    C = nan(n, N)
    dg.moe_gemm_w4(A.to(DEV), off.to(DEV), Q.to(DEV), S.to(DEV), C, group=G, Z=Z.to(DEV))
    v, b = om.w4_experts(A, off, Q, S, Z, G, 0, F32)
    v[n - 1:], b[n - 1:] = 0, 0
    om.check(C, (v, b), "experts")
