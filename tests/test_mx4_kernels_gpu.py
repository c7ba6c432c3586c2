"""GPU tests of the MXFP4 products, kernel by kernel: for every kernel and way through it that the sizes,
types and layouts choose, a call that its plan says takes it, against the definition in 64 bits."""
import pytest
import torch

from oracle import moe as om
from oracle import mx4 as ox
from test_mx4_gpu import BF16, DEV, F16, F32, I32, NAN, U8, coded, gen, in_ones, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()
    return m


def run(dg, kind, M, N, K, plan, place=lambda t: t.to(DEV), scales=(118, 128), out=F32, change=None):
    """Three calls on a stream of their own (whose workspace is new): the plan, the values, the same bits."""
    g = gen(M, N, K)
    A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
    Q, S = coded(g, N, K, scales)
    if change:
        change(Q, S)
    want = ox.gemm(A, SA, Q, S, K, 0, out)
    a, q, s, sa = place(A), place(Q), place(S), None if SA is None else place(SA)
    C = torch.full((4, M, N), NAN, dtype=out, device=DEV)
    assert dg.gemm_mx4_plan(a, q, s, C[0], SA=sa).startswith(plan), dg.gemm_mx4_plan(a, q, s, C[0], SA=sa)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for i in range(3):
        dg.gemm_mx4(a, q, s, C[i], SA=sa, stream=stream)
    stream.synchronize()
    om.check(C[0], want, f"{kind} {M}x{N}x{K}")
    assert torch.equal(C[0], C[1]) and torch.equal(C[0], C[2]) and C[3].isnan().all()


def few(rows, cols, pieces=1):
    return f"few rows, {rows}x{cols} tiles, K in {pieces} pieces"


def many(rows, cols, pieces=1):
    return f"many rows, {rows}x{cols} tiles, K in {pieces} pieces"


# ---------------------------------------------------------------- few rows

@pytest.mark.parametrize("M,N,K,rows,cols,pieces", [
    (1, 40, 512, 16, 16, 1), (16, 33, 4096, 16, 16, 1), (13, 8200, 1024, 16, 32, 1), (5, 100, 5000, 16, 16, 1), (17, 50, 4608, 32, 16, 1),
    (32, 8192, 520, 32, 32, 1), (16, 1000, 8192, 16, 16, 4), (3, 70, 40000, 16, 16, 16), (20, 4096, 8192, 32, 32, 2), (16, 4100, 9000, 16, 32, 0),
    (33, 40, 512, 64, 16, 1), (50, 1000, 5000, 64, 16, 1), (64, 4096, 8192, 64, 32, 2), (63, 1024, 8200, 64, 16, 4)])
def test_few_rows_of_codes(dg, M, N, K, rows, cols, pieces):
    plan = few(rows, cols, pieces) if pieces else f"few rows, {rows}x{cols} tiles"
    run(dg, "codes", M, N, K, plan)
    run(dg, "codes", M, N, K, plan, in_ones)


@pytest.mark.parametrize("M,N,K,rows,cols,pieces", [
    (1, 40, 512, 16, 16, 1), (8, 33, 4096, 16, 16, 1), (7, 60, 4700, 16, 16, 1), (3, 72, 9000, 16, 16, 4),              # whole rows
    (9, 33, 4096, 16, 16, 1), (16, 70, 600, 16, 16, 1), (13, 8200, 1024, 16, 32, 1), (16, 4096, 8192, 16, 32, 2),      # steps of 128
    (17, 50, 4608, 32, 16, 1), (32, 4096, 520, 32, 16, 1), (29, 4096, 8200, 32, 32, 2), (21, 72, 9000, 32, 16, 4),
    (33, 50, 4608, 36, 16, 1), (36, 130, 1000, 36, 16, 1), (33, 4096, 14336, 36, 32, 2), (35, 700, 8192, 36, 16, 4)])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_few_rows_of_16_bits(dg, M, N, K, rows, cols, pieces, kind):
    run(dg, kind, M, N, K, few(rows, cols, pieces))


@pytest.mark.parametrize("M,N,K", [(1, 40, 512), (16, 70, 1600), (11, 4100, 9000), (9, 30, 77)])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_few_rows_at_odd_addresses(dg, M, N, K, kind):
    def place(t):
        if t.dtype == U8:
            return in_ones(t)
        buf = torch.full((M * (K + 1) + 3,), NAN, dtype=kind, device=DEV)      # rows at odd multiples of 2 bytes
        v = buf[1:1 + M * (K + 1)].view(M, K + 1)[:, :K]
        v.copy_(t)
        return v
    run(dg, kind, M, N, K, "few rows, 16x16", place)


# ---------------------------------------------------------------- the scales that FP16 holds, and others

def ends(Q, S):
    S[:, 0], S[:, -1] = 104, 140                   # 2^-23 and 2^13: the outermost that FP16 holds all codes times


def one_far(Q, S):
    S[S.shape[0] // 2, S.shape[1] // 2] = 150


def zero_blocks(Q, S):
    Q[1, :16], S[1, 0], Q[-1], S[-1] = 0x80, 0, 0x08, 0      # zeros of both signs under a scale of 2^-127


@pytest.mark.parametrize("M,N,K,plan", [
    (12, 90, 2048, few(16, 16)), (30, 90, 1024, few(32, 16)), (34, 4096, 8192, few(36, 32, 2)), (4, 90, 1024, few(16, 16)),
    (130, 2000, 512, many(64, 128)), (100, 4096, 4096, many(64, 128, 4)), (1100, 4096, 256, many(128, 256)), (40, 90, 512, "aligned")])
@pytest.mark.parametrize("change", [None, ends, one_far, zero_blocks])
def test_scales_of_fp16(dg, M, N, K, plan, change):
    run(dg, F16, M, N, K, plan, scales=(104, 141) if change is None else (118, 128), change=change)


# ---------------------------------------------------------------- many rows, 16 bits

@pytest.mark.parametrize("M,N,K,rows,cols,pieces", [
    (65, 8200, 512, 64, 128, 1), (129, 100, 640, 64, 128, 1), (200, 1000, 1160, 64, 128, 1), (129, 70, 32, 64, 128, 1), (200, 300, 8200, 64, 128, 8),
    (70, 4096, 4096, 64, 128, 4), (64, 4096, 4096, 64, 128, 4), (150, 200, 2568, 64, 128, 4), (1030, 4400, 384, 128, 256, 1), (1100, 4096, 584, 128, 256, 1)])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_many_rows_of_16_bits(dg, M, N, K, rows, cols, pieces, kind):
    run(dg, kind, M, N, K, many(rows, cols, pieces), out=[F32, kind][M % 2])


@pytest.mark.parametrize("kind", [F16, BF16])
def test_scales_at_odd_addresses(dg, kind):
    # byte by byte where the scales do not lie at whole words, or K ends within a word of them
    place = lambda t: in_ones(t) if t.dtype == U8 and t.shape[1] < 200 else t.to(DEV)   # noqa: E731
    run(dg, kind, 140, 200, 1024, many(64, 128), place)
    run(dg, kind, 1100, 4096, 512, many(128, 256), place)
    run(dg, kind, 140, 200, 1056, many(64, 128))


@pytest.mark.parametrize("M,N,K,rows,cols,pieces", [
    (65, 8200, 333, 64, 128, 1), (129, 100, 1001, 64, 128, 1), (140, 70, 33, 64, 128, 1), (200, 300, 8201, 64, 128, 16), (150, 130, 2564, 64, 128, 5),
    (1030, 4400, 614, 128, 256, 1), (1100, 4096, 260, 128, 256, 1), (1100, 4096, 75, 128, 256, 1)])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_many_rows_of_16_bits_at_any_address(dg, M, N, K, rows, cols, pieces, kind):
    plan = many(rows, cols, pieces).replace("rows,", "rows at any address,")
    run(dg, kind, M, N, K, plan, lambda t: in_ones(t) if t.dtype == U8 else t.to(DEV), out=[F32, kind][M % 2])


@pytest.mark.parametrize("K", [256, 320, 584, 1024, 1152])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_many_rows_whose_addresses_are_odd(dg, K, kind):
    # a K that would do, rows that do not: A at odd multiples of 2 bytes, what lies between its rows NaN
    def place(t):
        if t.dtype == U8:
            return in_ones(t)
        buf = torch.full((t.shape[0] * (K + 3) + 1,), NAN, dtype=kind, device=DEV)
        v = buf[1:].view(-1, K + 3)[:, :K]
        v.copy_(t)
        return v
    run(dg, kind, 140, 300, K, "many rows at any address, 64x128", place)
    run(dg, kind, 1100, 4096, K, "many rows at any address, 128x256", place)


@pytest.mark.parametrize("M,N,K", [(40, 100, 1024), (48, 5000, 333), (20, 4200, 512), (33, 70, 1001)])
@pytest.mark.parametrize("kind", [F16, BF16])
def test_between_few_and_many(dg, M, N, K, kind):
    run(dg, kind, M, N, K, "")


# ---------------------------------------------------------------- many rows of codes

@pytest.mark.parametrize("M,N,K,plan", [
    (4096, 3300, 512, "ring loads, 256x256"), (1030, 2900, 512, "ring loads, 128x128"),
    (4096, 4200, 512, "ring loads, 256x256 tiles, K in 1 pieces, 256 workgroups; direct loads, 64x64 tiles"),
    (4000, 4500, 304, "direct loads, 256x256 tiles, K in 1 pieces, 256 workgroups; direct loads, 64x64 tiles"),
    (1100, 2900, 1536, "ring loads, 128x128"),
    (4000, 3300, 304, "direct loads, 256x256"), (1030, 2900, 1000, "direct loads, 128x128"), (70, 50, 264, "direct loads, 64x64"), (40, 4200, 264, "direct loads, 64x64"),
    (70, 130, 9000, "direct loads, 64x64"), (1100, 2900, 333, "vector loads, 128x128"), (70, 130, 777, "vector loads, 64x64"), (70, 50, 90, "element loads")])
def test_many_rows_of_codes(dg, M, N, K, plan):
    run(dg, "codes", M, N, K, plan, out=[F32, BF16][M * N > 1 << 20])


# ---------------------------------------------------------------- experts

@pytest.mark.parametrize("counts,N,K,kinds", [
    ([300, 0, 520, 200], 4096, 512, {"codes": "ring loads, 128x128", F16: many(128, 256), BF16: many(128, 256)}),
    ([300, 0, 520, 200], 4096, 333, {"codes": "vector loads, 128x128", F16: "many rows at any address, 128x256", BF16: "many rows at any address, 128x256"}),
    ([60, 70, 0, 90, 64], 4096, 640, {"codes": "direct loads, 64x64", F16: many(64, 128), BF16: many(64, 128)}),
    ([1, 5, 0, 30, 2, 9], 4096, 1024, {"codes": few(16, 32), F16: few(16, 32), BF16: few(16, 32)}),
    ([1, 0, 0, 1], 70, 4096, {"codes": few(16, 16), F16: few(16, 16), BF16: few(16, 16)}),
    ([1, 0, 7, 2, 0, 4, 0, 0], 4096, 1100, {"codes": few(16, 32), F16: few(16, 32), BF16: few(16, 32)}),
    ([40, 9, 20, 22, 21], 2048, 520, {"codes": few(32, 32), F16: "", BF16: ""})])
def test_experts(dg, counts, N, K, kinds):
    g = gen(sum(counts), N)
    E, n = len(counts), sum(counts) + 1
    off = torch.tensor([0] + counts).cumsum(0).int()
    Q, S = coded(g, E * N, K, (118, 128))
    Q, S = Q.view(E, N, -1), S.view(E, N, -1)
    for kind, plan in kinds.items():
        A, SA = coded(g, n, K, (118, 128)) if kind == "codes" else (normal(g, n, K, dtype=kind, spread=0.5), None)
        args = A.to(DEV), off.to(DEV), Q.to(DEV), S.to(DEV)
        C = torch.full((2, n, N), NAN, device=DEV)
        sa = None if SA is None else SA.to(DEV)
        assert dg.moe_gemm_mx4_plan(*args, C[0], SA=sa).startswith(plan), dg.moe_gemm_mx4_plan(*args, C[0], SA=sa)
        for c in C:
            dg.moe_gemm_mx4(*args, c, SA=sa)
        om.check(C[0], ox.experts(A, SA, off, Q, S, K, 0, F32), f"{kind} {counts}")
        assert torch.equal(C[0], C[1]) and (C[:, n - 1] == 0).all()


# ---------------------------------------------------------------- workspaces

def test_pieces_of_every_kernel_on_one_stream(dg):
    # kernels whose K meets in the same workspace, one after another and twice over, growing and shrinking
    g = gen(77)
    calls = []
    for kind, M, N, K in [(F16, 33, 4096, 8192), (BF16, 70, 4096, 4096), ("codes", 16, 1000, 8192), (F16, 3, 72, 9000), ("codes", 70, 130, 9000),
                          (BF16, 21, 72, 9000), (F16, 40, 300, 9000)]:
        A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
        Q, S = coded(g, N, K, (118, 128))
        calls.append(([t.to(DEV) for t in (A, Q, S)], None if SA is None else SA.to(DEV), ox.gemm(A, SA, Q, S, K, 0, F32), (M, N)))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for order in (calls, calls[::-1], calls):
        outs = []
        for args, sa, want, shape in order:
            outs.append(torch.full(shape, NAN, device=DEV))
            torch.cuda.synchronize()
            dg.gemm_mx4(*args, outs[-1], SA=sa, stream=stream)
        stream.synchronize()
        for C, (_, _, want, shape) in zip(outs, order):
            om.check(C, want, str(shape))


def test_every_kernel_in_a_graph(dg):
    # captured together (whole, without workspaces), replayed with other inputs between the program's own calls
    g = gen(78)
    calls = []
    for kind, M, N, K in [("codes", 16, 1000, 8192), (F16, 33, 300, 8192), (BF16, 5, 300, 1024), (BF16, 70, 4096, 4096), (F16, 140, 200, 1001),
                          ("codes", 70, 130, 2000), ("codes", 4096, 4200, 512), (F16, 40, 300, 2048)]:
        A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
        Q, S = coded(g, N, K, (118, 128))
        calls.append(([t.to(DEV) for t in (A, Q, S)], None if SA is None else SA.to(DEV), torch.zeros(M, N, device=DEV), K))

    def step():
        for args, sa, C, _ in calls:
            dg.gemm_mx4(*args, C, SA=sa)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for (A, Q, S), sa, C, K in calls:
            A.copy_(A.roll(rep + 1, 0))
            C.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        got = [C.clone() for _, _, C, _ in calls]
        step()
        torch.cuda.synchronize()
        for (args, sa, C, K), once in zip(calls, got):
            A, Q, S = (t.cpu() for t in args)
            want = ox.gemm(A, None if sa is None else sa.cpu(), Q, S, K, 0, F32)
            om.check(once, want, f"replay {rep}: {tuple(C.shape)} {K}")
            om.check(C, want, f"call {rep}: {tuple(C.shape)} {K}")
