"""Every kernel that the mixture-of-experts and 4-bit entry points choose among, by shapes whose
plan is asserted (on the CPU too, where the plan is that of a 256-CU device): a changed rule
cannot leave one of them without a test.  Results against the definitions in 64 bits (oracle/moe.py).
"""
import pytest
import torch

import dense_gemm_19_amd as dg
from oracle import moe as om

gpu = pytest.mark.gpu
DEV = "cuda:0"
F32, F16, BF16, I32, I64, U8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64, torch.uint8


def empty(*shape, dt=BF16, dev="cpu"):
    return torch.empty(*shape, dtype=dt, device=dev)


def normal(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets(counts):
    return torch.tensor([0] + counts).cumsum(0).int()


# ---------------------------------------------------------------- sort

# tokens, choices, experts, share of dropped ids, what runs
SORTS = [(1000, 1, 64, 0.1, "one workgroup, up to 1 ids"), (999, 3, 5, 0.2, "one workgroup, up to 4 ids"),
         (1000, 5, 2000, 0.1, "one workgroup, up to 16 ids"), (8191, 1, 2, 0.0, "one workgroup, up to 16 ids"),
         (1024, 8, 2048, 0.0, "two launches of 4 workgroups, 2048 ids"), (131073, 1, 8, 0.3, "two launches of 33 workgroups, 4096 ids"),
         (20001, 7, 256, 0.1, "two launches of 35 workgroups, 4096 ids"), (60000, 8, 200, 0.0, "two launches of 118 workgroups, 4096 ids"),
         (20001, 7, 2000, 0.1, "three launches of 35 workgroups"), (100000, 6, 700, 0.0, "three launches of 147 workgroups")]


@pytest.mark.parametrize("T,k,E,drop,plan", SORTS)
def test_sort_plan(T, k, E, drop, plan):
    assert dg.moe_sort_plan(empty(T, k, dt=I64), E, empty(E + 1, dt=I32), empty(T * k, dt=I32), empty(T, k, dt=I32)).startswith(plan)


def sorted_quick(ids, E):
    flat = ids.reshape(-1).long()
    by = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    kept = int((flat >= 0).sum())
    order = torch.where(torch.arange(flat.numel()) < kept, by, -1).int()
    pos = torch.full_like(order, -1)
    pos[by[:kept]] = torch.arange(kept, dtype=I32)
    off = torch.cat([torch.zeros(1, dtype=I64), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0)]).int()
    return off, order, pos.reshape(ids.shape)


@gpu
@pytest.mark.parametrize("T,k,E,drop,plan", SORTS)
@pytest.mark.parametrize("dtype", [I32, I64])
def test_sort(T, k, E, drop, plan, dtype):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E, (T, k), generator=g)
    ids = torch.where(torch.rand(T, k, generator=g) < drop, -1, ids).to(dtype)
    out = [torch.full(s, 77, dtype=I32, device=DEV) for s in ((E + 1,), (T * k,), (T, k))]
    d = ids.to(DEV)
    assert dg.moe_sort_plan(d, E, *out).startswith(plan)
    for _ in range(2):
        dg.moe_sort(d, E, *out)
        for a, b in zip(out, sorted_quick(ids, E)):
            assert torch.equal(a.cpu(), b)


@gpu
def test_sort_by_one_workgroup_in_a_graph():
    # 16000 ids: two launches with the workspace, one workgroup without it
    g = torch.Generator().manual_seed(4)
    ids = torch.zeros(8000, 2, dtype=I64, device=DEV)
    out = [torch.zeros(s, dtype=I32, device=DEV) for s in ((130,), (16000,), (8000, 2))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_sort(ids, 129, *out)
    for _ in range(3):
        host = torch.randint(-5, 129, (8000, 2), generator=g)
        host = torch.where(host < 0, -1, host)
        ids.copy_(host)
        for t in out:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, sorted_quick(host, 129)):
            assert torch.equal(a.cpu(), b)


# ---------------------------------------------------------------- gather past the caches

@gpu
@pytest.mark.parametrize("H,dtype", [(2101, BF16), (4202, torch.float8_e4m3fn), (1050, F32)])
def test_gather_of_outputs_above_160_mb(H, dtype):
    g = torch.Generator().manual_seed(2)
    T, k = 20500, 2
    order = torch.randperm(T * k, generator=g).int()
    order[::97] = -1
    assert T * k * H * dtype.itemsize > 160 << 20
    X = torch.randint(0, 120, (T, H * dtype.itemsize), generator=g, dtype=U8).view(dtype)   # finite in every type
    out = torch.full((T * k, H * dtype.itemsize), 0x7f, dtype=U8, device=DEV).view(dtype)
    dg.moe_gather(X.to(DEV), order.to(DEV), k, out)
    want = torch.where((order >= 0)[:, None], X.view(U8)[order.clamp(min=0).long() // k], 0)
    assert torch.equal(out.cpu().view(U8), want)


# ---------------------------------------------------------------- experts' products

# rows of each expert, K, N, what runs; K and the rows are no whole tiles
FORWARD = [([2600, 1800], 520, 2056, "direct loads, 192x256 tiles, K in 1 pieces"),
           ([2600, 1800], 520, 4104, "direct loads, 256x256 tiles, K in 1 pieces"),
           ([150, 0, 333], 520, 2056, "direct loads, 128x128 tiles, K in 2 pieces"),
           ([2000, 1500, 900], 136, 1032, "direct loads, 128x128 tiles, K in 1 pieces"),
           ([9, 40, 0, 3], 136, 1032, "direct loads, 32x128 tiles, K in 1 pieces"),
           ([9, 40, 0, 3], 1096, 136, "direct loads, 32x128 tiles, K in 4 pieces"),
           ([300, 500], 641, 4097, "vector loads, 128x128 tiles, K in 1 pieces"),
           ([30, 50], 641, 97, "vector loads, 64x64 tiles, K in 2 pieces")]


def experts_plan(counts, K, N, dtype, transposed, dev):
    n, E = sum(counts) + 2, len(counts)
    W = empty(E, N, K, dt=dtype, dev=dev).transpose(1, 2) if transposed else empty(E, K, N, dt=dtype, dev=dev)
    return dg.moe_gemm_plan(empty(n, K, dt=dtype, dev=dev), empty(E + 1, dt=I32, dev=dev), W, empty(n, N, dt=dtype, dev=dev))


@pytest.mark.parametrize("counts,K,N,plan", FORWARD)
@pytest.mark.parametrize("transposed", [False, True])
def test_experts_plan(counts, K, N, plan, transposed):
    assert experts_plan(counts, K, N, BF16, transposed, "cpu").startswith(plan)


@gpu
@pytest.mark.parametrize("counts,K,N,plan", FORWARD)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype,out,act", [(BF16, BF16, 0), (F16, F32, 2)])
def test_experts(counts, K, N, plan, transposed, dtype, out, act):
    assert experts_plan(counts, K, N, dtype, transposed, DEV).startswith(plan)
    g = torch.Generator().manual_seed(K + N)
    off, kept, E = offsets(counts), sum(counts), len(counts)
    A, W = normal(g, kept + 2, K, dtype=dtype), normal(g, E, K, N, dtype=dtype, scale=K ** -0.5)
    A[kept:] = float("nan")                                      # rows of no expert: zero
    w = W.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if transposed else W.to(DEV)
    C = torch.full((kept + 2, N), float("nan"), dtype=out, device=DEV)
    dg.moe_gemm(A.to(DEV), off.to(DEV), w, C, act)
    om.check(C[:kept], om.experts(A[:kept], off, W, act, out), plan)
    assert (C[kept:] == 0).all()
    first = C.clone()
    dg.moe_gemm(A.to(DEV), off.to(DEV), w, C.fill_(3), act)
    assert torch.equal(C, first)


WGRAD = [([300, 0, 517, 129], 2056, 2056, "direct loads, 256x256 tiles, K in 1 pieces"),
         ([300, 0, 517, 129], 520, 264, "direct loads, 128x128 tiles, K in 1 pieces"),
         ([700, 450], 136, 72, "direct loads, 128x128 tiles, K in 2 pieces"),
         ([300, 0, 517, 129], 1025, 1023, "vector loads, 128x128 tiles, K in 1 pieces"),
         ([700, 450], 65, 129, "vector loads, 64x64 tiles, K in 2 pieces")]


def wgrad_plan(counts, K, N, dtype, dev):
    n, E = sum(counts) + 2, len(counts)
    return dg.moe_gemm_wgrad_plan(empty(n, K, dt=dtype, dev=dev), empty(n, N, dt=dtype, dev=dev), empty(E + 1, dt=I32, dev=dev),
                                  empty(E, K, N, dt=F32, dev=dev))


@pytest.mark.parametrize("counts,K,N,plan", WGRAD)
def test_weight_gradient_plan(counts, K, N, plan):
    assert wgrad_plan(counts, K, N, BF16, "cpu").startswith(plan)


@gpu
@pytest.mark.parametrize("counts,K,N,plan", WGRAD)
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16)])
def test_weight_gradient(counts, K, N, plan, dtype, out):
    assert wgrad_plan(counts, K, N, dtype, DEV).startswith(plan)
    g = torch.Generator().manual_seed(K + N)
    off, n = offsets(counts), sum(counts) + 2
    A, D = normal(g, n, K, dtype=dtype), normal(g, n, N, dtype=dtype)
    A[n - 2:], D[n - 2:] = float("nan"), float("inf")
    dW = torch.full((len(counts), K, N), float("nan"), dtype=out, device=DEV)
    dg.moe_gemm_wgrad(A.to(DEV), D.to(DEV), off.to(DEV), dW)
    om.check(dW, om.wgrad(A, D, off, out), plan)


# ---------------------------------------------------------------- 4-bit products

def weights(g, N, K, G, zeros, st, lead=()):
    groups = -(-K // G)
    Q = torch.randint(0, 256, (*lead, N, (K + 1) // 2), generator=g, dtype=U8)
    S = ((0.5 + torch.rand(*lead, N, groups, generator=g)) * K ** -0.5).to(st)
    return Q, S, torch.randint(0, 256, (*lead, N, groups), generator=g, dtype=U8) if zeros else None


# half: the layout whose LDS lets two workgroups share a CU
W4 = [(1, 9000, 4192, 128, "aligned words, 16x32 tiles, K in 1 pieces", True), (5, 9000, 2080, 32, "aligned words, 16x32 tiles, K in 1 pieces", True),
      (5, 1000, 4192, 64, "aligned words, 16x32 tiles, K in 2 pieces", False), (3, 72, 9024, 64, "aligned words, 16x32 tiles, K in 3 pieces", False),
      (3, 72, 9001, 64, "any layout, 16x32 tiles, K in 3 pieces", None), (30, 1000, 2080, 96, "aligned words, 32x64 tiles, K in 1 pieces", False),
      (45, 200, 6176, 64, "aligned words, 48x64 tiles, K in 5 pieces", False), (100, 200, 6175, 64, "any layout, 48x64 tiles, K in 5 pieces", None)]


def is_half(plan):
    return int(plan.split(" of ")[1].split()[0]) <= 80 * 1024


def w4_plan(M, N, K, G, dtype, dev):
    groups = -(-K // G)
    return dg.gemm_w4_plan(empty(M, K, dt=dtype, dev=dev), empty(N, (K + 1) // 2, dt=U8, dev=dev), empty(N, groups, dt=dtype, dev=dev),
                           empty(M, N, dt=dtype, dev=dev), G, empty(N, groups, dt=U8, dev=dev))


@pytest.mark.parametrize("M,N,K,G,plan,half", W4)
def test_w4_plan(M, N, K, G, plan, half):
    got = w4_plan(M, N, K, G, BF16, "cpu")
    assert got.startswith(plan) and half in (None, is_half(got)), got


@gpu
@pytest.mark.parametrize("M,N,K,G,plan,half", W4)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_w4(M, N, K, G, plan, half, dtype):
    got = w4_plan(M, N, K, G, dtype, DEV)
    assert got.startswith(plan) and half in (None, is_half(got)), got
    g = torch.Generator().manual_seed(M + K)
    A = normal(g, M, K, dtype=dtype)
    Q, S, Z = weights(g, N, K, G, True, dtype)
    C = torch.full((M, N), float("nan"), device=DEV)
    args = [t.to(DEV) for t in (A, Q, S)]
    dg.gemm_w4(*args, C, group=G, Z=Z.to(DEV))
    om.check(C, om.w4(A, Q, S, Z, G, 0, F32), plan)
    first = C.clone()
    dg.gemm_w4(*args, C.fill_(3), group=G, Z=Z.to(DEV))
    assert torch.equal(C, first)


# a mean of at most 10 rows in the two-workgroup layout: tiles of 16 rows leave the rings of A one slot
W4_EXPERTS = [([40, 1, 0, 3, 16, 2, 0, 1], 3000, 3168, 32, "aligned words, 16x32 tiles", True),
              ([33, 0, 2, 1, 1, 0, 2, 3], 3000, 1024, 128, "aligned words, 16x32 tiles", True),
              ([20, 3, 1], 96, 3168, 64, "aligned words, 16x32 tiles", False), ([60, 1, 20, 0], 200, 1568, 32, "aligned words, 32x64 tiles", False),
              ([100, 1, 20, 0], 200, 1568, 32, "aligned words, 48x64 tiles", False), ([20, 3, 1], 96, 3167, 64, "any layout, 16x32 tiles", None)]


def w4_experts_plan(counts, N, K, G, dtype, dev):
    n, E, groups = sum(counts) + 1, len(counts), -(-K // G)
    return dg.moe_gemm_w4_plan(empty(n, K, dt=dtype, dev=dev), empty(E + 1, dt=I32, dev=dev), empty(E, N, (K + 1) // 2, dt=U8, dev=dev),
                               empty(E, N, groups, dt=dtype, dev=dev), empty(n, N, dt=dtype, dev=dev), G, empty(E, N, groups, dt=U8, dev=dev))


@pytest.mark.parametrize("counts,N,K,G,plan,half", W4_EXPERTS)
def test_w4_experts_plan(counts, N, K, G, plan, half):
    got = w4_experts_plan(counts, N, K, G, BF16, "cpu")
    assert got.startswith(plan) and half in (None, is_half(got)), got


@gpu
@pytest.mark.parametrize("counts,N,K,G,plan,half", W4_EXPERTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_w4_experts(counts, N, K, G, plan, half, dtype):
    got = w4_experts_plan(counts, N, K, G, dtype, DEV)
    assert got.startswith(plan) and half in (None, is_half(got)), got
    g = torch.Generator().manual_seed(N + K)
    off, n = offsets(counts), sum(counts) + 1
    A = normal(g, n, K, dtype=dtype)
    A[n - 1] = float("nan")
    Q, S, Z = weights(g, N, K, G, True, dtype, (len(counts),))
    C = torch.full((n, N), float("nan"), device=DEV)
    dg.moe_gemm_w4(*[t.to(DEV) for t in (A, off, Q, S)], C, group=G, Z=Z.to(DEV))
    v, b = om.w4_experts(A[:n - 1], off, Q, S, Z, G, 0, F32)
    om.check(C[:n - 1], (v, b), plan)
    assert (C[n - 1] == 0).all()


# ---------------------------------------------------------------- products whose K is cut, captured (whole there)

@gpu
def test_products_in_a_graph_that_are_cut_outside():
    g = torch.Generator().manual_seed(6)
    off = torch.tensor([0, 3, 40], dtype=I32)
    A, W = normal(g, 40, 2048), normal(g, 2, 2048, 64, scale=2048 ** -0.5)
    off2 = torch.tensor([0, 1200, 1205], dtype=I32)
    X, D = normal(g, 1205, 64), normal(g, 1205, 128)
    B = normal(g, 3, 9024)
    Q, S, Z = weights(g, 72, 9024, 64, True, BF16)
    a, w, x, d, b, q, s, z, o, o2 = (t.to(DEV) for t in (A, W, X, D, B, Q, S, Z, off, off2))
    C, dW, Y = torch.zeros(40, 64, device=DEV), torch.zeros(2, 64, 128, device=DEV), torch.zeros(3, 72, device=DEV)
    for plan in (dg.moe_gemm_plan(a, o, w, C), dg.moe_gemm_wgrad_plan(x, d, o2, dW), dg.gemm_w4_plan(b, q, s, Y, 64, z)):
        assert "K in 1 pieces" not in plan

    def calls():
        dg.moe_gemm(a, o, w, C)
        dg.moe_gemm_wgrad(x, d, o2, dW)
        dg.gemm_w4(b, q, s, Y, group=64, Z=z)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for rep in range(3):
        for host, dev in ((A, a), (X, x), (B, b)):
            host.copy_(normal(g, *host.shape))
            dev.copy_(host)
        for t in (C, dW, Y):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        om.check(C, om.experts(A, off, W, 0, F32), f"C {rep}")
        om.check(dW, om.wgrad(X, D, off2, F32), f"dW {rep}")
        om.check(Y, om.w4(B, Q, S, Z, 64, 0, F32), f"Y {rep}")
        calls()                                                  # the program's own work between the replays
        torch.cuda.synchronize()
        om.check(Y, om.w4(B, Q, S, Z, 64, 0, F32), f"Y {rep} outside")
