"""GPU tests of the products with 4-bit weights (dg.gemm_w4, dg.moe_gemm_w4)
against the definition in 64 bits (oracle/moe.py) with the bounds derived there."""
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


def weights(g, N, K, G, zeros, st, lead=()):
    groups = -(-K // G)
    Q = torch.randint(0, 256, (*lead, N, (K + 1) // 2), generator=g, dtype=torch.uint8)
    S = ((0.5 + torch.rand(*lead, N, groups, generator=g)) * K ** -0.5).to(st)
    return Q, S, torch.randint(0, 256, (*lead, N, groups), generator=g, dtype=torch.uint8) if zeros else None


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 130, 300])
@pytest.mark.parametrize("N,K,G", [(64, 128, 128), (33, 256, 32), (48, 1024, 64), (100, 200, 128), (17, 333, 32), (1, 1, 32),
                                   (65, 2176, 256), (40, 1000, 96), (96, 4096, 128), (130, 288, 160)])
def test_w4(dg, M, N, K, G):
    g = torch.Generator().manual_seed(M * N + K)
    dtype, st, out, act, zeros = [(BF16, BF16, BF16, 0, False), (F16, F16, F32, 0, True), (BF16, F32, F32, 2, True),
                                  (F16, F32, F16, 1, True)][(M + N + K) % 4]
    A = torch.randn(M, K, generator=g).to(dtype)
    Q, S, Z = weights(g, N, K, G, zeros, st)
    C = dg.gemm_w4(*dev(A, Q, S), torch.full((M, N), float("nan"), dtype=out, device=DEV), group=G, Z=dev(Z)[0], act=act)
    om.check(C, om.w4(A, Q, S, Z, G, act, out), f"w4 {M}x{N}x{K} G {G}")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("st", [F32, F16, BF16])
@pytest.mark.parametrize("G", [32, 64, 96, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_types(dg, dtype, st, G, zeros):
    g = torch.Generator().manual_seed(G)
    M, N, K = 5, 50, 1600
    A = torch.randn(M, K, generator=g).to(dtype)
    Q, S, Z = weights(g, N, K, G, zeros, st)
    for out in (F32, F16, BF16):
        C = dg.gemm_w4(*dev(A, Q, S), torch.empty(M, N, dtype=out, device=DEV), group=G, Z=dev(Z)[0])
        om.check(C, om.w4(A, Q, S, Z, G, 0, out), f"{dtype} {st} {G} {out}")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_code_and_zero_point(dg, dtype):
    # a one-hot A reads single weights: q - z for every q and z, to the bit
    N, K = 256, 32
    Q = (torch.arange(16, dtype=torch.uint8).repeat(N, 1) * 17).contiguous()   # byte i: code i twice
    Z = torch.arange(N, dtype=torch.uint8).reshape(N, 1)
    A = torch.eye(K, dtype=dtype)
    C = dg.gemm_w4(*dev(A, Q, torch.ones(N, 1)), torch.empty(K, N, device=DEV), group=32, Z=Z.to(DEV))
    want = torch.arange(16).repeat_interleave(2)[:, None] - Z.int().t()
    assert torch.equal(C.cpu(), want.float())


def test_w4_strides(dg):
    g = torch.Generator().manual_seed(2)
    M, N, K, G = 20, 70, 640, 64
    A = torch.randn(M, K, generator=g).to(BF16)
    Q, S, Z = weights(g, N, K, G, True, BF16)
    want = om.w4(A, Q, S, Z, G, 0, F32)
    wide = lambda t: torch.cat([t, t, t], 1).to(DEV)[:, t.shape[1]:2 * t.shape[1]]   # noqa: E731  rows apart
    C = torch.zeros(N, M, device=DEV).t()
    om.check(dg.gemm_w4(wide(A), wide(Q), wide(S), C, group=G, Z=wide(Z)), want, "rows apart")
    a1 = torch.zeros(M * K + 1, dtype=BF16, device=DEV)[1:].view(M, K)               # 2-byte aligned only
    a1.copy_(A)
    q1 = torch.zeros(N * K // 2 + 1, dtype=torch.uint8, device=DEV)[1:].view(N, K // 2)
    q1.copy_(Q)
    om.check(dg.gemm_w4(a1, q1, S.to(DEV), torch.zeros(M, N, device=DEV), group=G, Z=Z.to(DEV)), want, "unaligned")
    s2, z2 = S.t().contiguous().to(DEV).t(), Z.t().contiguous().to(DEV).t()          # groups apart
    om.check(dg.gemm_w4(A.to(DEV), Q.to(DEV), s2, torch.zeros(M, N, device=DEV), group=G, Z=z2), want, "groups apart")


def test_non_finite_activations(dg):
    # Inf times a weight keeps the weight's sign, Inf times an exact zero is NaN, as in the definition
    g = torch.Generator().manual_seed(4)
    M, N, K, G = 4, 40, 256, 128
    A = torch.randn(M, K, generator=g).to(BF16)
    A[1, 7], A[2, 200] = float("inf"), float("nan")
    Q, S, _ = weights(g, N, K, G, False, F32)
    C = dg.gemm_w4(*dev(A, Q, S), torch.empty(M, N, device=DEV), group=G)
    W = om.dense4(Q, S, None, K, G)
    row = A[1].double()[None] * W
    want = om.w4(A[[0, 3]], Q, S, None, G, 0, F32)
    om.check(C[[0, 3]], want, "finite rows")
    assert torch.isnan(C[2]).all()
    inf = row.sum(1)
    assert torch.equal(torch.isnan(C[1].cpu()), torch.isnan(inf)) and torch.equal(C[1].cpu().nan_to_num(0, 1, -1), inf.float().nan_to_num(0, 1, -1))


@pytest.mark.parametrize("G", [32, 64, 96, 128, 160, 224, 384, 4096, 1 << 20])
def test_group_of_every_element(dg, G):
    # a one-hot A reads one weight: the scale of its group at the group's ends, along a long K
    K, N = 8192 + 40, 3
    Q = torch.full((N, K // 2), 0x99, dtype=torch.uint8)            # q - 8 = 1
    groups = -(-K // G)
    S = (torch.arange(N * groups, dtype=torch.float32) + 1).reshape(N, groups)
    at = sorted({min(max(k, 0), K - 1) for g in range(0, groups, max(1, groups // 7)) for k in (g * G - 1, g * G, g * G + G - 1)})
    for dtype in (BF16, F16):
        A = torch.zeros(len(at), K, dtype=dtype)
        for m, k in enumerate(at):
            A[m, k] = 1
        C = dg.gemm_w4(*dev(A, Q, S), torch.empty(len(at), N, device=DEV), group=G)
        want = torch.stack([S[:, k // G] for k in at])
        assert torch.equal(C.cpu(), want)


@pytest.mark.parametrize("zeros", [False, True])
def test_split_k(dg, zeros):
    # few columns and a long K: the sum meets in the workspace; twice gives the same bits
    g = torch.Generator().manual_seed(3)
    M, N, K, G = 6, 72, 9000, 64
    A = torch.randn(M, K, generator=g).to(BF16)
    Q, S, Z = weights(g, N, K, G, zeros, BF16)
    args = dev(A, Q, S)
    C = [dg.gemm_w4(*args, torch.empty(M, N, device=DEV), group=G, Z=dev(Z)[0]) for _ in range(3)]
    om.check(C[0], om.w4(A, Q, S, Z, G, 0, F32), "split")
    assert torch.equal(C[0], C[1]) and torch.equal(C[0], C[2])


def test_empty(dg):
    Q, S = torch.zeros(8, 0, dtype=torch.uint8, device=DEV), torch.zeros(8, 0, device=DEV)
    C = torch.full((3, 8), 7.0, device=DEV)
    dg.gemm_w4(torch.zeros(3, 0, dtype=F16, device=DEV), Q, S, C, group=32)
    assert (C == 0).all()                                       # K = 0: an empty sum
    dg.gemm_w4(torch.zeros(0, 64, dtype=F16, device=DEV), torch.zeros(8, 32, dtype=torch.uint8, device=DEV),
               torch.zeros(8, 2, device=DEV), torch.zeros(0, 8, device=DEV), group=32)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 20], [2] * 9, [40, 0, 17, 1], [1, 0] * 40, [200, 30]])
@pytest.mark.parametrize("N,K,G,zeros,act", [(64, 256, 128, False, 0), (45, 300, 32, True, 2), (32, 1024, 64, True, 1)])
def test_w4_experts(dg, counts, N, K, G, zeros, act):
    g = torch.Generator().manual_seed(sum(counts) + N)
    E, n = len(counts), sum(counts) + 2
    off = torch.tensor([0] + counts).cumsum(0).int()
    dtype, out = (BF16, BF16) if act else (F16, F32)
    A = torch.randn(n, K, generator=g).to(dtype)
    Q, S, Z = weights(g, N, K, G, zeros, dtype, (E,))
    C = dg.moe_gemm_w4(*dev(A, off, Q, S), torch.full((n, N), float("nan"), dtype=out, device=DEV), group=G, Z=dev(Z)[0], act=act)
    v, b = om.w4_experts(A, off, Q, S, Z, G, act, out)
    v[n - 2:], b[n - 2:] = 0, 0                                  # rows of no expert
    om.check(C, (v, b), f"{counts}")


def test_w4_in_a_graph(dg):
    g = torch.Generator().manual_seed(9)
    M, N, K, G = 3, 96, 1024, 128
    A = torch.zeros(M, K, dtype=BF16, device=DEV)
    Q, S, _ = weights(g, N, K, G, False, BF16)
    Q, S = dev(Q, S)
    C = torch.zeros(M, N, device=DEV)
    dg.gemm_w4(A, Q, S, C, group=G)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.gemm_w4(A, Q, S, C, group=G)
    for rep in range(3):
        A.copy_(torch.randn(M, K, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = C.clone()
        dg.gemm_w4(A, Q, S, C, group=G)
        torch.cuda.synchronize()
        assert torch.equal(C, got), rep


@pytest.mark.parametrize("K,G", [(160, 32), (320, 64), (288, 96), (333, 32), (2080, 32), (1096, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
def test_infinite_scale_of_the_last_group(dg, K, G, dtype, zeros):
    # the last 128 elements of K hold less than their groups: what lies past K adds nothing, not Inf times 0
    g = torch.Generator().manual_seed(K + G)
    N = 40
    Q, S, Z = weights(g, N, K, G, zeros, F32)
    Q = (Q | 0x99)                                               # q - z is not 0, and above it
    if zeros:
        Z = Z % 9
    S[::3, -1], S[1::3, -1] = float("inf"), float("-inf")
    S[0, 0] = float("inf")
    for M in (3, 20, 40):
        A = (0.5 + torch.rand(M, K, generator=g)).to(dtype)
        a1 = torch.zeros(M * K + 1, dtype=dtype, device=DEV)[1:].view(M, K).copy_(A)   # any other layout
        want = om.w4(A, Q, S, Z, G, 0, F32)
        for a in (A.to(DEV), a1):
            C = dg.gemm_w4(a, *dev(Q, S), torch.empty(M, N, device=DEV), group=G, Z=dev(Z)[0])
            om.check(C, want, f"{M}x{N}x{K} G {G}")
    off = torch.tensor([0, 15, 40], dtype=torch.int32)
    Q, S, Z = (None if t is None else torch.stack([t, t]) for t in (Q, S, Z))
    C = dg.moe_gemm_w4(*dev(A, off, Q, S), torch.empty(40, N, device=DEV), group=G, Z=dev(Z)[0])
    om.check(C, want, "experts")


@pytest.mark.parametrize("M", [1, 5, 20])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("zeros", [False, True])
def test_zero_weights_meet_large_activations(dg, M, dtype, zeros):
    # most codes equal their zero point, a few activations are a thousand times the others: the sum's bound is
    # that of the weights that are not zero
    g = torch.Generator().manual_seed(M)
    N, K, G = 70, 2048, 64
    A = torch.randn(M, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.02, 1000.0, 1.0)
    _, S, Z = weights(g, N, K, G, zeros, F32)
    z = torch.full((N, K), 8) if Z is None else (Z % 16).repeat_interleave(G, 1).long()
    q = torch.where(torch.rand(N, K, generator=g) < 0.97, z, torch.randint(0, 16, (N, K), generator=g))
    q[7] = z[7]                                                  # nothing but zeros
    Q = (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8)
    Z = None if Z is None else Z % 16
    A = A.to(dtype)
    C = dg.gemm_w4(*dev(A, Q, S), torch.empty(M, N, device=DEV), group=G, Z=dev(Z)[0])
    om.check(C, om.w4(A, Q, S, Z, G, 0, F32), f"{M}")
    assert (C[:, 7] == 0).all()
