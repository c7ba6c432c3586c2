"""GPU tests of the MXFP4 operators (dg.quant_mx4, dequant_mx4, gemm_mx4, moe_gemm_mx4) against the
definitions in 64 bits (oracle/mx4.py): codes, scales and values to the bit, products within the
bounds derived in oracle/moe.py."""
import numpy as np
import pytest
import torch

from oracle import moe as om
from oracle import mx4 as ox

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16, I32, U8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.uint8
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()   # raises if the library is missing: there is no fallback
    return m


def gen(*seed):
    return torch.Generator().manual_seed(sum((i + 1) * s for i, s in enumerate(seed)))


def normal(g, *shape, dtype=F32, spread=1.0):
    return (torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(shape[-1], generator=g))).to(dtype)


def codes(M, K, fill=0):
    return (torch.full((M, (K + 1) // 2), fill, dtype=U8, device=DEV), torch.full((M, -(-K // 32)), fill, dtype=U8, device=DEV))


def coded(g, M, K, scales=(110, 140)):
    """Random codes and scale bytes of a range; the spare half of an odd K is zero."""
    Q = torch.randint(0, 256, (M, (K + 1) // 2), generator=g, dtype=U8)
    if K % 2:
        Q[:, -1] &= 15
    return Q, torch.randint(*scales, (M, -(-K // 32)), generator=g, dtype=U8)


def in_ones(t, before=7, after=33, pitch=None):
    """The same matrix inside a buffer of 0xff bytes: NaN scales, codes of -6, wherever a load goes astray."""
    rows, cols = t.shape[-2:]
    pitch = cols if pitch is None else pitch
    n = t[..., 0, 0].numel() * rows
    buf = torch.full((before + n * pitch + after,), 255, dtype=U8, device=DEV)
    view = buf[before:before + n * pitch].view(n, pitch)[:, :cols]
    view.copy_(t.reshape(n, cols))
    return view if t.dim() == 2 else view.unflatten(0, t.shape[:-1])


# ---------------------------------------------------------------- quantiser

def check_quant(dg, X, ceil, x=None):
    """x: X on the device, in whatever layout."""
    M, K = X.shape
    Q, S = codes(M, K, 0xA5)
    dg.quant_mx4(X.to(DEV) if x is None else x, Q, S, dg.DG_MX4_CEIL if ceil else dg.DG_MX4_FLOOR)
    q, s = ox.quant(X, ceil)
    assert torch.equal(S.cpu(), s), f"{int((S.cpu() != s).sum())} scales differ"
    assert torch.equal(Q.cpu(), q), f"{int((Q.cpu() != q).sum())} bytes of codes differ"


@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (1, 32), (3, 33), (5, 64), (2, 257), (70, 96), (17, 1000), (129, 250), (300, 40), (4, 4096), (1, 9000)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("ceil", [False, True])
def test_quant(dg, M, K, dtype, ceil):
    X = normal(gen(M, K), M, K, dtype=dtype)
    check_quant(dg, X, ceil)
    check_quant(dg, X, ceil, X.t().contiguous().to(DEV).t())                     # columns contiguous
    if M * K < 20000:
        check_quant(dg, X, ceil, X.to(DEV).repeat_interleave(2, 1)[:, ::2])      # neither
        pad = torch.full((M * K + 3,), NAN, dtype=dtype, device=DEV)
        pad[1:-2].view(M, K).copy_(X)
        check_quant(dg, X, ceil, pad[1:-2].view(M, K))                           # at any element's address
        wide = torch.full((K, M + 5), NAN, dtype=dtype, device=DEV)
        wide[:, 3:-2].copy_(X.t())
        check_quant(dg, X, ceil, wide[:, 3:-2].t())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quant_of_midpoints_and_ends(dg, dtype):
    # every midpoint and its neighbours in the type, at scales over the type's range; tops that both rules tell apart
    f = torch.finfo(dtype)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0]).to(dtype)
    step = torch.tensor([1 - f.eps, 1.0, 1 + f.eps]).to(dtype)
    row = (mids[:, None] * step).reshape(-1)[:31]
    rows = []
    for top in (4.0, 6.0, 6.0 * (1 + f.eps), 7.5, 8.0 * (1 - f.eps)):
        for e in (-8, -3, 0, 5, 11) + (() if dtype == F16 else (-120, -100, 90, 124)):
            r = torch.cat([torch.tensor([top]), row.float()]).to(dtype).double() * 2.0 ** e
            rows.append(torch.cat([r, -r]))
    check_quant(dg, torch.stack(rows).to(dtype), False)
    check_quant(dg, torch.stack(rows).to(dtype), True)
    check_quant(dg, torch.stack(rows).to(dtype), True, torch.stack(rows).to(dtype).t().contiguous().to(DEV).t())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("ceil", [False, True])
def test_quant_of_special_values(dg, dtype, ceil):
    f = torch.finfo(dtype)
    X = normal(gen(3), 12, 160, dtype=dtype)
    X[0] = 0
    X[1] = -0.0
    X[2, 5], X[3, 40], X[4, 159], X[5, 64] = NAN, INF, -INF, -NAN
    X[6] = f.tiny * f.eps                                          # the least subnormal
    X[7] = f.tiny / 2
    X[8] = f.max
    X[9, :32] = f.tiny * f.eps * torch.arange(1, 33).to(dtype)
    X[10, 32:64] = 0
    check_quant(dg, X, ceil)
    check_quant(dg, X, ceil, X.t().contiguous().to(DEV).t())
    check_quant(dg, X, ceil, X.to(DEV).repeat_interleave(3, 1)[:, ::3])


def test_quant_of_stacks_and_pitches(dg):
    g = gen(11)
    for E, M, K in ((3, 40, 75), (5, 1, 32), (2, 300, 260), (700, 2, 33)):
        W = normal(g, E * M, K, dtype=BF16).view(E, M, K)
        want = [torch.stack(t) for t in zip(*(ox.quant(w) for w in W[:: max(1, E // 5)]))]
        pick = slice(None, None, max(1, E // 5))
        for x in (W.to(DEV), W.transpose(1, 2).contiguous().to(DEV).transpose(1, 2), torch.cat([W, W], 1).to(DEV)[:, :M]):
            Qb, Sb = torch.full((E, M + 1, (K + 1) // 2 + 5), 0x5A, dtype=U8, device=DEV), torch.full((E, -(-K // 32), M + 2), 0x5A, dtype=U8, device=DEV)
            Q, S = Qb[:, :M, 2:2 + (K + 1) // 2], Sb[:, :, :M].transpose(1, 2)
            dg.quant_mx4(x, Q, S)
            assert torch.equal(Q[pick].cpu(), want[0]) and torch.equal(S[pick].cpu(), want[1])
            Q.fill_(0x5A), S.fill_(0x5A)
            assert (Qb == 0x5A).all() and (Sb == 0x5A).all()      # nothing else was written
        # the transposes of the stack: what a gradient sums over
        Q, S = torch.zeros(E, K, (M + 1) // 2, dtype=U8, device=DEV), torch.zeros(E, K, -(-M // 32), dtype=U8, device=DEV)
        dg.quant_mx4(W.to(DEV).transpose(1, 2), Q, S)
        q, s = ox.quant(W[E - 1].t())
        assert torch.equal(Q[E - 1].cpu(), q) and torch.equal(S[E - 1].cpu(), s)


# ---------------------------------------------------------------- what codes stand for

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_every_code_and_scale_read_back(dg, dtype):
    Q = torch.arange(256, dtype=U8).repeat(256, 2)[:, :272].contiguous()     # 544 elements, every pair of codes
    S = torch.arange(256, dtype=U8).repeat_interleave(17).view(256, 17).contiguous()
    want = ox.values(Q, S, 544)
    Y = dg.dequant_mx4(Q.to(DEV), S.to(DEV), torch.zeros(256, 544, dtype=dtype, device=DEV)).cpu()
    ref = want.to(F32).to(dtype)                                             # (exact in FP32 but where it is infinite)
    assert torch.equal(torch.isnan(Y), torch.isnan(ref)) and torch.equal(Y.nan_to_num(0, 1, -1), ref.nan_to_num(0, 1, -1))
    assert torch.equal(torch.signbit(Y)[:255], torch.signbit(ref)[:255])


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 33), (40, 250), (9, 1000), (300, 64), (1, 20000)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_dequant(dg, M, K, dtype):
    g = gen(M, K)
    Q, S = coded(g, M, K)
    want = ox.values(Q, S, K).to(dtype)
    for q, s in ((Q.to(DEV), S.to(DEV)), (in_ones(Q, pitch=Q.shape[1] + 3), in_ones(S.t(), pitch=M + 1).t())):
        Y = dg.dequant_mx4(q, s, torch.full((M, K), NAN, dtype=dtype, device=DEV))
        assert torch.equal(Y.cpu(), want)
        buf = torch.full((K, M + 3), 7.0, dtype=dtype, device=DEV)
        dg.dequant_mx4(q, s, buf[:, 2:2 + M].t())
        assert torch.equal(buf[:, 2:2 + M].t().cpu(), want) and (buf[:, :2] == 7).all() and (buf[:, 2 + M:] == 7).all()
        buf = torch.full((M, K + 3), 7.0, dtype=dtype, device=DEV)
        dg.dequant_mx4(q, s, buf[:, 1:1 + K])
        assert torch.equal(buf[:, 1:1 + K].cpu(), want) and (buf[:, :1] == 7).all() and (buf[:, 1 + K:] == 7).all()
    Q3, S3 = torch.stack([Q, Q]).to(DEV), torch.stack([S, S]).to(DEV)
    Y = dg.dequant_mx4(Q3, S3, torch.zeros(2, M, K, dtype=dtype, device=DEV))
    assert torch.equal(Y[0].cpu(), want) and torch.equal(Y[1].cpu(), want)


# ---------------------------------------------------------------- products

SHAPES = [(1, 1, 1), (1, 64, 32), (2, 33, 64), (7, 100, 250), (16, 96, 256), (17, 130, 333), (33, 48, 1024), (64, 64, 512), (65, 200, 300),
          (100, 257, 1056), (130, 70, 2600), (200, 300, 776), (300, 129, 520)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["codes", F16, BF16])
def test_gemm(dg, M, N, K, kind):
    g = gen(M, N, K)
    out, act = [(F32, 0), (BF16, 2), (F16, 1), (F32, 2)][(M + N + K) % 4]
    A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
    Q, S = coded(g, N, K, (118, 128))
    want = ox.gemm(A, SA, Q, S, K, act, out)
    for place in (lambda t: t.to(DEV), in_ones):
        a = place(A) if kind == "codes" else A.to(DEV)
        C = torch.full((M, N), NAN, dtype=out, device=DEV)
        dg.gemm_mx4(a, place(Q), place(S), C, SA=None if SA is None else place(SA), act=act)
        om.check(C, want, f"{kind} {M}x{N}x{K}")


@pytest.mark.parametrize("K", [256, 264, 500, 1000, 1024, 1031, 2048, 5000])
@pytest.mark.parametrize("M,N", [(40, 50), (150, 300), (256, 256), (513, 770)])
def test_ragged_ends_of_codes(dg, M, N, K):
    # rows at multiples of 4 bytes, in a pitch of their own and one after another, every end of a tile of K; what
    # lies behind the rows' ends are codes of -6 and NaN scales
    g = gen(M, N, K)
    A, SA = coded(g, M, K, (118, 128))
    Q, S = coded(g, N, K, (118, 128))
    want = ox.gemm(A, SA, Q, S, K, 0, F32)
    row, blocks = A.shape[1], SA.shape[1]
    places = [(0, row, row), (4, row + (-row) % 4, row + (-row) % 4 + 8), (16, row + (-row) % 16, row + (-row) % 16), (3, row, row + 1)]
    for before, pa, pq in places:
        C = torch.full((M, N), NAN, device=DEV)
        args = in_ones(A, before, 0, pa), in_ones(Q, before, 0, pq), in_ones(S, 5, 0), C
        dg.gemm_mx4(*args, SA=in_ones(SA, 1, 0))
        om.check(C, want, f"{M}x{N}x{K} pitch {pa} {pq}")


def test_gemm_of_strides(dg):
    g = gen(8)
    M, N, K = 90, 150, 800
    A, SA = coded(g, M, K, (118, 128))
    X = normal(g, M, K, dtype=BF16)
    Q, S = coded(g, N, K, (118, 128))
    for a, sa, w in ((A, SA, ox.gemm(A, SA, Q, S, K, 0, F32)), (X, None, ox.gemm(X, None, Q, S, K, 0, F32))):
        apart = lambda t: t.to(DEV).t().contiguous().t()   # noqa: E731  columns apart
        buf = torch.full((N + 2, 3 * M), 7.0, device=DEV)
        C = buf[1:1 + N, ::3].t()
        dg.gemm_mx4(a.to(DEV), Q.to(DEV), apart(S), C, SA=None if sa is None else apart(sa))
        om.check(C, w, "strides")
        assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, 1::3] == 7).all() and (buf[:, 2::3] == 7).all()
        same = a[:1].to(DEV).expand(M, -1), None if sa is None else sa[:1].to(DEV).expand(M, -1)     # a broadcast row
        C = dg.gemm_mx4(same[0], Q.to(DEV), S.to(DEV), torch.zeros(M, N, device=DEV), SA=same[1])
        om.check(C, (w[0][:1].expand(M, N), w[1][:1].expand(M, N)), "broadcast")
        last = Q[-1:].to(DEV).expand(N, -1), S[-1:].to(DEV).expand(N, -1)
        C = dg.gemm_mx4(a.to(DEV), *last, torch.zeros(M, N, device=DEV), SA=None if sa is None else sa.to(DEV))
        om.check(C, (w[0][:, -1:].expand(M, N), w[1][:, -1:].expand(M, N)), "broadcast weights")


@pytest.mark.parametrize("kind", ["codes", F16, BF16])
@pytest.mark.parametrize("M", [1, 20, 70, 150])
def test_split_k(dg, M, kind):
    # few columns and a long K: twice gives the same bits
    g = gen(M)
    N, K = 72, 9000
    A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
    Q, S = coded(g, N, K, (118, 128))
    args = A.to(DEV), Q.to(DEV), S.to(DEV)
    C = [dg.gemm_mx4(*args, torch.empty(M, N, device=DEV), SA=None if SA is None else SA.to(DEV)) for _ in range(3)]
    om.check(C[0], ox.gemm(A, SA, Q, S, K, 0, F32), "split")
    assert torch.equal(C[0], C[1]) and torch.equal(C[0], C[2])


@pytest.mark.parametrize("kind", ["codes", F16, BF16])
def test_empty(dg, kind):
    dt = U8 if kind == "codes" else kind
    sa = lambda *s: torch.zeros(*s, dtype=U8, device=DEV) if kind == "codes" else None   # noqa: E731
    z = lambda *s: torch.zeros(*s, dtype=U8, device=DEV)   # noqa: E731
    C = torch.full((3, 8), 7.0, device=DEV)
    dg.gemm_mx4(torch.zeros(3, 0, dtype=dt, device=DEV), z(8, 0), z(8, 0), C, SA=sa(3, 0))
    assert (C == 0).all()                                       # K = 0: an empty sum
    dg.moe_gemm_mx4(torch.zeros(3, 0, dtype=dt, device=DEV), torch.tensor([0, 1, 3], dtype=I32, device=DEV), z(2, 8, 0), z(2, 8, 0),
                    C.fill_(7.0), SA=sa(3, 0))
    assert (C == 0).all()
    k = 32 if kind == "codes" else 64
    dg.gemm_mx4(torch.zeros(0, k, dtype=dt, device=DEV), z(8, 32), z(8, 2), torch.zeros(0, 8, device=DEV), SA=sa(0, 2))


@pytest.mark.parametrize("kind", ["codes", F16, BF16])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_one_block_at_a_time(dg, M, kind):
    # rows of A that are zero but for one element read single weights, to the bit, each with its own scales
    K, N = 1100, 70
    g = gen(M)
    at = torch.randint(0, K, (M,), generator=g)
    at[0] = K - 1
    Q, S = coded(g, N, K, (0, 255) if kind == "codes" else (100, 150))
    if kind == "codes":
        A, SA = torch.zeros(M, K // 2, dtype=U8), torch.zeros(M, -(-K // 32), dtype=U8)
        A[torch.arange(M), at // 2] = torch.where(at % 2 == 0, 2, 32).to(U8)
        SA[torch.arange(M), at // 32] = 127
    else:
        A, SA = torch.zeros(M, K, dtype=kind), None
        A[torch.arange(M), at] = 1
    C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.to(DEV), torch.empty(M, N, device=DEV), SA=None if SA is None else SA.to(DEV))
    want = ox.values(Q, S, K)[:, at].t().to(F32)
    assert torch.equal(C.cpu(), want)


@pytest.mark.parametrize("kind", ["codes", BF16, F16])
@pytest.mark.parametrize("M,K", [(3, 96), (3, 2080), (100, 96), (100, 2080), (300, 1056)])
def test_nan_scales(dg, M, K, kind):
    # a NaN scale makes its row's or column's sums NaN, whatever the codes, and no other
    g = gen(M, K)
    N = 300
    A, SA = coded(g, M, K, (118, 128)) if kind == "codes" else (normal(g, M, K, dtype=kind, spread=0.5), None)
    Q, S = coded(g, N, K, (118, 128))
    S[5, 0], S[N - 1, -1] = 255, 255
    Q[5, :16] = 0
    rows = []
    if SA is not None:
        SA[M - 1, -1] = 255
        rows = [M - 1]
    C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.to(DEV), torch.empty(M, N, device=DEV), SA=None if SA is None else SA.to(DEV))
    om.check(C, ox.gemm(A, SA, Q, S, K, 0, F32), "NaN scales")
    assert torch.isnan(C[:, [5, N - 1]]).all() and torch.isnan(C[rows]).all() and int(torch.isnan(C).sum()) == 2 * M + (N - 2) * len(rows)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_non_finite_activations(dg, dtype):
    # Inf times a weight keeps the weight's sign, Inf times zero is NaN, as in the definition
    g = gen(4)
    M, N, K = 4, 40, 256
    A = normal(g, M, K, dtype=dtype, spread=0.5)
    A[1, 7], A[2, 200] = INF, NAN
    Q, S = coded(g, N, K, (118, 128))
    C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.to(DEV), torch.empty(M, N, device=DEV)).cpu()
    om.check(C[[0, 3]], ox.gemm(A[[0, 3]], None, Q, S, K, 0, F32), "finite rows")
    assert torch.isnan(C[2]).all()
    inf = (A[1].double()[None] * ox.values(Q, S, K)).sum(1).float()
    assert torch.equal(torch.isnan(C[1]), torch.isnan(inf)) and torch.equal(C[1].nan_to_num(0, 1, -1), inf.nan_to_num(0, 1, -1))


@pytest.mark.parametrize("M", [2, 100])
def test_ends_of_the_scales(dg, M):
    # scales whose product is moderate, from the least to the largest; both least give nothing, both largest infinities
    g = gen(M)
    N, K = 40, 320
    A, _ = coded(g, M, K)
    Q, _ = coded(g, N, K)
    for sa, sw in ((0, 254), (254, 0), (1, 253), (200, 54), (127, 127)):
        SA, S = torch.full((M, 10), sa, dtype=U8), torch.full((N, 10), sw, dtype=U8)
        C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.to(DEV), torch.empty(M, N, device=DEV), SA=SA.to(DEV))
        want = ox.gemm(A, SA, Q, S, K, 0, F32)                     # whole quarters below 2^24: exact
        assert torch.equal(C.cpu().double(), want[0]), (sa, sw)
    SA, S = torch.zeros(M, 10, dtype=U8), torch.zeros(N, 10, dtype=U8)
    assert (dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.to(DEV), torch.empty(M, N, device=DEV), SA=SA.to(DEV)) == 0).all()
    A.fill_(0x22), Q.fill_(0xAA)                                   # 1 times -1
    C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.fill_(254).to(DEV), torch.empty(M, N, device=DEV), SA=SA.fill_(254).to(DEV))
    assert (C == -INF).all()
    C = dg.gemm_mx4(A.to(DEV), Q.to(DEV), S.fill_(60).to(DEV), torch.empty(M, N, device=DEV), SA=SA.fill_(60).to(DEV))
    assert (C == -K * 2.0 ** -134).all()                           # subnormal in FP32


# ---------------------------------------------------------------- experts

@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 20], [2] * 9, [40, 0, 17, 1], [1, 0] * 40, [200, 30], [0, 0, 300], [70, 64, 65, 130, 5]])
@pytest.mark.parametrize("N,K,act", [(64, 256, 0), (45, 300, 2), (130, 1030, 1), (33, 62, 0)])
@pytest.mark.parametrize("kind", ["codes", F16, BF16])
def test_experts(dg, counts, N, K, act, kind):
    g = gen(sum(counts), N)
    E, n = len(counts), sum(counts) + 2
    out = [F32, BF16, F16][act]
    off = torch.tensor([0] + counts).cumsum(0).int()
    A, SA = coded(g, n, K, (118, 128)) if kind == "codes" else (normal(g, n, K, dtype=kind, spread=0.5), None)
    Q, S = coded(g, E * N, K, (118, 128))
    Q, S = Q.view(E, N, -1), S.view(E, N, -1)
    want = ox.experts(A, SA, off, Q, S, K, act, out)
    place = in_ones if kind == "codes" else lambda t: t.to(DEV)   # noqa: E731
    C = dg.moe_gemm_mx4(place(A), off.to(DEV), in_ones(Q), in_ones(S), torch.full((n, N), NAN, dtype=out, device=DEV),
                        SA=None if SA is None else in_ones(SA), act=act)
    om.check(C, want, f"{kind} {counts}")
    assert (C[n - 2:] == 0).all()


def test_experts_apart_and_offsets_astray(dg):
    g = gen(21)
    E, N, K, n = 3, 70, 512, 50
    A, SA = coded(g, n, K, (118, 128))
    Q, S = coded(g, 2 * E * N, K, (118, 128))
    Q, S = Q.view(2 * E, N, -1)[::2], S.view(2 * E, N, -1)[::2]
    off = torch.tensor([0, 20, 20, 44], dtype=I32)
    want = ox.experts(A, SA, off, Q, S, K, 0, F32)
    both = torch.zeros(2 * E, N, K // 2, dtype=U8, device=DEV)[::2], torch.zeros(2 * E, N, K // 32, dtype=U8, device=DEV)[::2]
    both[0].copy_(Q), both[1].copy_(S)
    om.check(dg.moe_gemm_mx4(A.to(DEV), off.to(DEV), *both, torch.full((n, N), NAN, device=DEV), SA=SA.to(DEV)), want, "experts apart")
    # offsets past the rows, or negative: no row outside is touched
    wild = torch.tensor([-5, 20, 1 << 30, 60], dtype=I32)
    buf = torch.full((n + 4, N), 7.0, device=DEV)
    dg.moe_gemm_mx4(A.to(DEV), wild.to(DEV), *both, buf[2:-2], SA=SA.to(DEV))
    torch.cuda.synchronize()
    assert (buf[:2] == 7).all() and (buf[-2:] == 7).all()
    om.check(buf[2:22], (want[0][:20], want[1][:20]), "the first expert's rows")


# ---------------------------------------------------------------- together

def quantised(dg, x, ceil=False):
    Q, S = torch.zeros(*x.shape[:-1], (x.shape[-1] + 1) // 2, dtype=U8, device=DEV), torch.zeros(*x.shape[:-1], -(-x.shape[-1] // 32), dtype=U8, device=DEV)
    return dg.quant_mx4(x, Q, S, dg.DG_MX4_CEIL if ceil else dg.DG_MX4_FLOOR)


@pytest.mark.parametrize("T,K,N", [(100, 300, 130), (37, 64, 96), (260, 512, 257)])
def test_training_step_of_a_linear_layer(dg, T, K, N):
    # Y = X W^T, dX = dY W, dW = dY^T X, each of operands quantised along what it sums over; each gradient is the
    # product of what the quantised operands stand for
    g = gen(T, K, N)
    X, W, dY = normal(g, T, K, dtype=BF16), normal(g, N, K, dtype=F32), normal(g, T, N, dtype=BF16)
    x, w, dy = X.to(DEV), W.to(DEV), dY.to(DEV)
    for (a, a_ref), (b, b_ref), shape in (((x, X), (w, W), (T, N)), ((dy, dY), (w.t(), W.t()), (T, K)), ((dy.t(), dY.t()), (x.t(), X.t()), (N, K))):
        (qa, sa), (qb, sb) = quantised(dg, a), quantised(dg, b)
        C = dg.gemm_mx4(qa, qb, sb, torch.empty(shape, device=DEV), SA=sa)
        (ra, rsa), (rb, rsb) = ox.quant(a_ref), ox.quant(b_ref)
        om.check(C, ox.gemm(ra, rsa, rb, rsb, a_ref.shape[1], 0, F32), f"{shape}")


def test_gradients_against_differences(dg):
    # numbers of the format itself are exact along every direction, and so are their products here: the loss
    # <X W^T, G> moves by its gradient times the step
    g = gen(77)
    T, K, N = 40, 96, 64
    numbers = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    X, W, G = (numbers[torch.randint(0, 8, s, generator=g)] * (2 * torch.randint(0, 2, s, generator=g) - 1) for s in ((T, K), (N, K), (T, N)))
    X, W, G = X.to(DEV), W.to(DEV), G.to(DEV)

    def matmul_t(a, b):
        (qa, sa), (qb, sb) = quantised(dg, a), quantised(dg, b)
        return dg.gemm_mx4(qa, qb, sb, torch.empty(a.shape[0], b.shape[0], device=DEV), SA=sa)

    loss = lambda x, w: float((matmul_t(x, w).double() * G.double()).sum())   # noqa: E731
    dX, dW = matmul_t(G, W.t()), matmul_t(G.t(), X.t())
    at = loss(X, W)
    for i in range(12):
        t, k, n = (int(torch.randint(0, m, (), generator=g)) for m in (T, K, N))
        x, w = X.clone(), W.clone()
        x[t, k], w[n, k] = -X[t, k] if i % 2 else 6.0, 1.5
        assert loss(x, W) - at == float(dX[t, k]) * float(x[t, k] - X[t, k])
        assert loss(X, w) - at == float(dW[n, k]) * float(w[n, k] - W[n, k])


def test_a_layer_of_experts(dg):
    # route, quantise every token once, gather codes and scales, both products of every expert, combine
    g = gen(5)
    T, k, E, H, F = 60, 2, 6, 256, 320
    X = normal(g, T, H, dtype=BF16, spread=0.3)
    W1, W2 = normal(g, E * F, H, dtype=BF16, spread=0.3).view(E, F, H) * H ** -0.5, normal(g, E * H, F, dtype=BF16, spread=0.3).view(E, H, F) * F ** -0.5
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices
    w = torch.rand(T, k, generator=g)
    n = T * k
    i32 = lambda *s: torch.zeros(*s, dtype=I32, device=DEV)   # noqa: E731
    off, order, pos = dg.moe_sort(ids.to(DEV), E, i32(E + 1), i32(n), i32(T, k))
    qx, sx = quantised(dg, X.to(DEV))
    q1, s1 = quantised(dg, W1.to(DEV))
    q2, s2 = quantised(dg, W2.to(DEV))
    qs = dg.moe_gather(qx, order, k, torch.zeros(n, H // 2, dtype=U8, device=DEV))
    ss = dg.moe_gather(sx, order, k, torch.zeros(n, H // 32, dtype=U8, device=DEV))
    h = dg.moe_gemm_mx4(qs, off, q1, s1, torch.zeros(n, F, dtype=BF16, device=DEV), SA=ss, act=dg.DG_ACT_GELU_TANH)
    qh, sh = quantised(dg, h)
    y = dg.moe_gemm_mx4(qh, off, q2, s2, torch.zeros(n, H, device=DEV), SA=sh)
    out = dg.moe_combine(y, pos, torch.zeros(T, H, device=DEV), w.to(DEV))
    # stage by stage against the definitions, each from what the stage before gave
    o = order.cpu().long()
    rq, rs = ox.quant(X)
    assert torch.equal(qs.cpu(), rq[o // k]) and torch.equal(ss.cpu(), rs[o // k])
    om.check(h, ox.experts(qs.cpu(), ss.cpu(), off.cpu(), q1.cpu(), s1.cpu(), H, 2, BF16), "up")
    om.check(y, ox.experts(qh.cpu(), sh.cpu(), off.cpu(), q2.cpu(), s2.cpu(), F, 0, F32), "down")
    om.check(out, om.combine(y.cpu(), pos.cpu(), w, F32), "combine")


@pytest.mark.parametrize("kind", ["codes", BF16])
def test_in_a_graph(dg, kind):
    # quantise and multiply, captured, replayed with other inputs between the program's own calls
    g = gen(9)
    M, N, K = 24, 96, 1024
    X = torch.zeros(M, K, dtype=BF16, device=DEV)
    Q, S = (t.to(DEV) for t in coded(g, N, K, (118, 128)))
    qx, sx = codes(M, K)
    C, Y = torch.zeros(M, N, device=DEV), torch.zeros(M, K, device=DEV)

    def step():
        dg.quant_mx4(X, qx, sx)
        dg.dequant_mx4(qx, sx, Y)
        if kind == "codes":
            dg.gemm_mx4(qx, Q, S, C, SA=sx)
        else:
            dg.gemm_mx4(X, Q, S, C)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        X.copy_(normal(g, M, K, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qx, sx, Y, C)]
        a, sa = ox.quant(X.cpu())
        assert torch.equal(qx.cpu(), a) and torch.equal(sx.cpu(), sa)
        om.check(C, ox.gemm(a, sa, Q.cpu(), S.cpu(), K, 0, F32) if kind == "codes" else ox.gemm(X.cpu(), None, Q.cpu(), S.cpu(), K, 0, F32), f"replay {rep}")
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got[:3], (qx, sx, Y)))


def test_streams(dg):
    # two streams at once, each with products whose K meets in its own workspace
    g = gen(31)
    jobs = []
    for i in range(2):
        A, SA = coded(g, 30 + i, 8000, (118, 128))
        Q, S = coded(g, 80, 8000, (118, 128))
        jobs.append((torch.cuda.Stream(), [t.to(DEV) for t in (A, Q, S, SA)], torch.zeros(30 + i, 80, device=DEV), ox.gemm(A, SA, Q, S, 8000, 0, F32)))
    torch.cuda.synchronize()
    for _ in range(8):
        for s, (a, q, sc, sa), C, _ in jobs:
            dg.gemm_mx4(a, q, sc, C, SA=sa, stream=s)
    torch.cuda.synchronize()
    for _, _, C, want in jobs:
        om.check(C, want, "stream")
    with torch.cuda.stream(jobs[0][0]):
        C = dg.gemm_mx4(*jobs[1][1][:3], torch.zeros(31, 80, device=DEV), SA=jobs[1][1][3])
    torch.cuda.synchronize()
    om.check(C, jobs[1][3], "another stream")
