"""GPU tests of the mixture-of-experts operators (dg.moe_*) against the definitions
in 64 bits (oracle/moe.py), with the bounds derived there: row counts from
none to many, odd and unaligned sizes, strides, dropped choices, every type,
values that are not finite, wrong indices, streams and graphs.
"""
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


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def choices(g, T, k, E, drop=0.0):
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k] if E >= k else torch.randint(0, E, (T, k), generator=g)
    return torch.where(torch.rand(T, k, generator=g) < drop, torch.full_like(ids, -1), ids)


def odd_rows(t):
    """t in rows two elements longer than its own, on the device (any alignment)."""
    big = torch.full((*t.shape[:-1], t.shape[-1] + 2), float("nan"), dtype=t.dtype, device=DEV)
    v = big[..., 1:-1]
    v.copy_(t)
    return v


def sort_dev(dg, ids, E):
    n = ids.numel()
    out = [torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((E + 1,), (n,), tuple(ids.shape))]
    return dg.moe_sort(ids, E, *out)


# ---------------------------------------------------------------- sort

@pytest.mark.parametrize("T,k,E,drop", [(0, 2, 4, 0), (1, 1, 1, 0), (1, 8, 64, 0), (64, 8, 64, 0), (300, 2, 7, 0.2),
                                        (999, 3, 5, 1.0), (2048, 8, 256, 0.1), (5, 3, 2048, 0), (8193, 2, 129, 0.05),
                                        (9001, 5, 2000, 0.3), (40000, 1, 3, 0.0), (6000, 8, 64, 0.0)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(dg, T, k, E, drop, dtype):
    ids = choices(gen(T + k), T, k, E, drop).to(dtype)
    got = sort_dev(dg, ids.to(DEV), E)
    flat = ids.reshape(-1).long()
    for a, b in zip(got, om.sort(ids, E) if flat.numel() * E < 1 << 22 else _sort_quick(ids, E)):
        assert torch.equal(a.cpu(), b)


def _sort_quick(ids, E):
    flat = ids.reshape(-1).long()
    by = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    kept = int((flat >= 0).sum())
    order = torch.where(torch.arange(flat.numel()) < kept, by, -1).int()
    pos = torch.full_like(order, -1)
    pos[by[:kept]] = torch.arange(kept, dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0)]).int()
    return offsets, order, pos.reshape(ids.shape)


def test_sort_strided_and_wrong_ids(dg):
    g = gen(3)
    ids = torch.randint(-3, 12, (500, 4), generator=g)          # ids outside 0..7 are dropped
    ids[0, 0], ids[1, 1] = 2 ** 40, -2 ** 40                    # also where 32 bits would fold them into range
    want = om.sort(torch.where((ids < 0) | (ids >= 8), torch.full_like(ids, -1), ids), 8)
    wide = torch.zeros(500, 9, dtype=torch.int64, device=DEV)
    wide[:, 1::2].copy_(ids)
    for dev in (ids.to(DEV), wide[:, 1::2], ids.t().contiguous().to(DEV).t()):
        for a, b in zip(sort_dev(dg, dev, 8), want):
            assert torch.equal(a.cpu(), b)


# ---------------------------------------------------------------- gather, combine and its gradient

SIZES = [(1, 1, 1, 1, 0.0), (3, 2, 4, 7, 0.3), (48, 8, 64, 2048, 0.0), (33, 6, 8, 1000, 0.1), (130, 3, 9, 65, 0.0),
         (17, 9, 16, 512, 0.2), (20, 20, 32, 24, 0.5), (5, 4, 4, 4097, 0.0), (9, 2, 3, 64, 1.0)]


@pytest.mark.parametrize("T,k,E,H,drop", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("strided", [False, True])
def test_rows(dg, T, k, E, H, drop, dtype, strided):
    g = gen(T * H + k)
    _, order, pos = om.sort(choices(g, T, k, E, drop), E)
    put = odd_rows if strided else (lambda t: t.to(DEV))
    X, Ys, dY = (normal(g, r, H, dtype=dtype) for r in (T, T * k, T))
    empty = lambda *s, dt=dtype: put(torch.full(s, float("nan"), dtype=dt))   # noqa: E731
    Xs = dg.moe_gather(put(X), order.to(DEV), k, empty(T * k, H))
    want = torch.zeros(T * k, H, dtype=dtype)
    want[order >= 0] = X[order[order >= 0].long() // k]
    assert torch.equal(Xs.cpu(), want)
    for wt in (F32, dtype, None):
        w = None if wt is None else torch.rand(T, k, generator=g).to(wt)
        wd = None if w is None else put(w)
        Y = dg.moe_combine(put(Ys), pos.to(DEV), empty(T, H), wd)
        om.check(Y, om.combine(Ys, pos, w, dtype), "combine")
        dYs, dw = dg.moe_combine_grad(put(dY), put(Ys), pos.to(DEV), wd, empty(T * k, H),
                                      None if w is None else empty(T, k, dt=wt))
        a, b = om.combine_grad(dY, Ys, pos, w)
        om.check(dYs, a, "dYs")
        if w is not None:
            om.check(dw, b, "dw")


def test_gather_fp8_and_strided_columns(dg):
    g = gen(5)
    _, order, _ = om.sort(choices(g, 20, 2, 4), 4)
    X = torch.randint(0, 120, (20, 33), generator=g, dtype=torch.uint8).view(torch.float8_e4m3fn)
    out = dg.moe_gather(X.to(DEV), order.to(DEV), 2, torch.zeros(40, 33, device=DEV).to(torch.float8_e4m3fn))
    assert torch.equal(out.cpu().view(torch.uint8), X.view(torch.uint8)[order.long() // 2])
    Xt = normal(g, 33, 20).to(DEV).t()                           # column-major
    out = dg.moe_gather(Xt, order.to(DEV), 2, torch.zeros(40, 66, device=DEV, dtype=BF16)[:, ::2])
    assert torch.equal(out.cpu(), Xt.cpu()[order.long() // 2])


def test_dropped_and_wrong_places_add_nothing(dg):
    # what a dropped choice would have read holds NaN: neither its weight nor a row may count
    g = gen(6)
    Ys, dY = normal(g, 6, 96), normal(g, 4, 96)
    pos = torch.tensor([[0, -1], [5, 1 << 30], [-7, -1], [2, 6]], dtype=torch.int32)
    w = torch.rand(4, 2, generator=g)
    w[0, 1] = float("nan")
    w[1, 1] = float("inf")
    Ys[3] = float("nan")
    Y = dg.moe_combine(Ys.to(DEV), pos.to(DEV), torch.empty(4, 96, dtype=BF16, device=DEV), w.to(DEV))
    om.check(Y, om.combine(Ys, pos, w, BF16), "combine")
    assert (Y[2] == 0).all()
    dYs, dw = dg.moe_combine_grad(dY.to(DEV), Ys.to(DEV), pos.to(DEV), w.to(DEV),
                                  torch.full((6, 96), float("nan"), dtype=BF16, device=DEV), torch.empty(4, 2, device=DEV))
    a, b = om.combine_grad(dY, Ys, pos, w)
    om.check(dYs, a, "dYs")
    om.check(dw, b, "dw")
    order = torch.tensor([3, -1, 8, 1 << 30, 0, -5], dtype=torch.int32)   # choices 8 and up do not exist (T k = 8)
    Xs = dg.moe_gather(dY.to(DEV), order.to(DEV), 2, torch.full((6, 96), float("nan"), dtype=BF16, device=DEV))
    want = torch.zeros(6, 96, dtype=BF16)
    want[0], want[4] = dY[1], dY[0]
    assert torch.equal(Xs.cpu(), want)


def test_combine_grad_against_differences(dg):
    # d/dYs and d/dw of <combine(Ys, w), dY>, by central differences in 64 bits
    g = gen(7)
    T, k, H = 5, 3, 19
    _, _, pos = om.sort(choices(g, T, k, 6, 0.2), 6)
    Ys, dY, w = normal(g, T * k, H, dtype=F32), normal(g, T, H, dtype=F32), torch.rand(T, k, generator=g)
    dYs, dw = dg.moe_combine_grad(dY.to(DEV), Ys.to(DEV), pos.to(DEV), w.to(DEV), torch.empty(T * k, H, device=DEV),
                                  torch.empty(T, k, device=DEV))

    def loss(ys, ww):
        s = 0.0
        for t in range(T):
            for j in range(k):
                if pos[t, j] >= 0:
                    s += float(ww[t, j] * (ys[pos[t, j]] * dY[t].double()).sum())
        return s
    h = 1e-3                                                     # the loss is linear in each: exact up to 64-bit rounding
    for (r, c) in [(0, 0), (4, 18), (14, 7)]:
        d = torch.zeros(T * k, H, dtype=torch.float64)
        d[r, c] = h
        num = (loss(Ys.double() + d, w.double()) - loss(Ys.double() - d, w.double())) / (2 * h)
        assert abs(num - float(dYs[r, c])) <= om.U * abs(num) * 2 + 1e-9
    for (t, j) in [(0, 0), (4, 2), (2, 1)]:
        d = torch.zeros(T, k, dtype=torch.float64)
        d[t, j] = h
        num = (loss(Ys.double(), w.double() + d) - loss(Ys.double(), w.double() - d)) / (2 * h)
        size = float((dY[t].double() * Ys[max(int(pos[t, j]), 0)].double()).abs().sum())
        assert abs(num - float(dw[t, j])) <= 2 * H * om.U * size + 1e-9


# ---------------------------------------------------------------- expert products

def counts_to_offsets(counts):
    return torch.tensor([0] + counts).cumsum(0).int()


COUNTS = [[1], [0, 0, 3], [5, 0, 1, 40], [64, 64], [33, 0, 0, 129, 2], [300, 7], [1] * 70, [0] * 65 + [9] + [0] * 70 + [4],
          [260, 0, 513]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("K,N,dtype,out,act", [(64, 128, BF16, BF16, 0), (192, 264, F16, F32, 2), (200, 72, BF16, F32, 1),
                                               (65, 129, F16, F16, 0), (8, 8, BF16, F32, 0), (3, 5, BF16, BF16, 2),
                                               (72, 300, F16, F16, 2)])
def test_experts(dg, counts, K, N, dtype, out, act):
    g = gen(sum(counts) + K)
    E, n = len(counts), sum(counts) + 3                          # three rows of no expert: zero
    off = counts_to_offsets(counts)
    A, W, D = normal(g, n, K, dtype=dtype), normal(g, E, K, N, dtype=dtype, scale=K ** -0.5), normal(g, n, N, dtype=dtype)
    A[n - 3:], D[n - 3:] = float("nan"), float("nan")            # which nothing may read into a result
    o = off.to(DEV)
    nan = lambda *s, dt=out: torch.full(s, float("nan"), dtype=dt, device=DEV)   # noqa: E731
    C = dg.moe_gemm(A.to(DEV), o, W.to(DEV), nan(n, N), act)
    om.check(C, _tailed(om.experts, A, off, W, act, out), "C")
    dA = dg.moe_gemm(D.to(DEV), o, W.to(DEV).transpose(1, 2), nan(n, K, dt=dtype))
    om.check(dA, _tailed(om.experts, D, off, W.transpose(1, 2), 0, dtype), "dA")
    dW = dg.moe_gemm_wgrad(A.to(DEV), D.to(DEV), o, nan(E, K, N))
    om.check(dW, om.wgrad(A, D, off, out), "dW")


def _tailed(f, A, off, *rest):
    """The oracle on the experts' rows, and zeros (to the bit) for the rows after them."""
    kept = int(off[-1])
    v, b = f(A[:kept], off, *rest)
    z = torch.zeros(A.shape[0] - kept, v.shape[1], dtype=torch.float64)
    return torch.cat([v, z]), torch.cat([b, z])


@pytest.mark.parametrize("K,N,counts", [(512, 768, [600, 0, 300]), (1032, 520, [1500, 700]), (641, 1001, [300, 500])])
def test_experts_larger_tiles(dg, K, N, counts):
    test_experts(dg, counts, K, N, BF16, BF16, 0)


def test_experts_any_strides(dg):
    g = gen(11)
    off, n, K, N = counts_to_offsets([10, 0, 37]), 47, 96, 88
    A, W, D = normal(g, n, K), normal(g, 3, K, N, scale=0.1), normal(g, n, N)
    o2 = torch.zeros(4, 3, dtype=torch.int32, device=DEV)
    o2[:, 1].copy_(off)
    o = o2[:, 1]                                                 # strided offsets
    for a, w, c in [(odd_rows(A), odd_rows(W), odd_rows(torch.zeros(n, N))),
                    (A.t().contiguous().to(DEV).t(), W.to(DEV), torch.zeros(N, n, device=DEV).t()),
                    (A.to(DEV), W.permute(1, 2, 0).contiguous().to(DEV).permute(2, 0, 1), torch.zeros(n, 2 * N, device=DEV)[:, ::2]),
                    (A.to(DEV), W.transpose(1, 2).contiguous().to(DEV).transpose(1, 2), torch.zeros(n, N, device=DEV))]:
        om.check(dg.moe_gemm(a, o, w, c, 2), om.experts(A, off, W, 2, F32), "C")
    for a, d, w in [(odd_rows(A), odd_rows(D), odd_rows(torch.zeros(3, K, N))),
                    (A.t().contiguous().to(DEV).t(), D.to(DEV), torch.zeros(3, N, K, device=DEV).transpose(1, 2)),
                    (A.to(DEV), D.to(DEV), torch.zeros(5, K, N, device=DEV)[::2])]:
        om.check(dg.moe_gemm_wgrad(a, d, o, w), om.wgrad(A, D, off, F32), "dW")
    # one matrix of weights for every expert (stride 0)
    om.check(dg.moe_gemm(A.to(DEV), o, W[:1].to(DEV).expand(3, K, N), torch.zeros(n, N, device=DEV)),
             om.experts(A, off, W[:1].expand(3, K, N), 0, F32), "C")


def test_infinities_stay_with_their_expert(dg):
    # ragged row counts end inside a tile; a neighbour's Inf and NaN must not leak across
    g = gen(12)
    off, n, K, N = counts_to_offsets([5, 70, 9]), 84, 136, 144
    A, W, D = normal(g, n, K), normal(g, 3, K, N, scale=0.1), normal(g, n, N)
    A[5:75], D[5:75] = float("inf"), float("nan")
    C = dg.moe_gemm(A.to(DEV), off.to(DEV), W.to(DEV), torch.zeros(n, N, device=DEV))
    assert torch.isfinite(C[:5]).all() and torch.isfinite(C[75:]).all()
    dW = dg.moe_gemm_wgrad(A.to(DEV), D.to(DEV), off.to(DEV), torch.zeros(3, K, N, device=DEV))
    assert torch.isfinite(dW[0]).all() and torch.isfinite(dW[2]).all() and torch.isnan(dW[1]).all()
    B = normal(g, n, K)
    B[7, 130] = float("inf")                                     # in the last, partial K tile
    C = dg.moe_gemm(B.to(DEV), off.to(DEV), W.to(DEV), torch.zeros(n, N, device=DEV))
    om.check(C, om.experts(B, off, W, 0, F32), "C")


@pytest.mark.parametrize("bad", [[0, 9, 4, 20], [0, -5, 30, 10], [0, 100, 200, 300], [-3, 5, 5, 1 << 30]])
def test_wrong_offsets_stay_inside(dg, bad):
    # decreasing or out-of-range offsets give some result, in bounds
    g = gen(13)
    A, W, D = normal(g, 20, 64).to(DEV), normal(g, 3, 64, 72).to(DEV), normal(g, 20, 72).to(DEV)
    guard = torch.full((60, 72), 7.0, device=DEV)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    dg.moe_gemm(A, off, W, guard[20:40])
    dg.moe_gemm_wgrad(A, D, off, torch.zeros(3, 64, 72, device=DEV))
    torch.cuda.synchronize()
    assert (guard[:20] == 7).all() and (guard[40:] == 7).all()


# ---------------------------------------------------------------- together

def layer(dg, s):
    """An MoE layer forward and backward on the state's buffers."""
    dg.moe_sort(s["ids"], s["E"], s["off"], s["order"], s["pos"])
    dg.moe_gather(s["X"], s["order"], s["k"], s["Xs"])
    dg.moe_gemm(s["Xs"], s["off"], s["W"], s["Ys"])
    dg.moe_combine(s["Ys"], s["pos"], s["Y"], s["w"])
    dg.moe_combine_grad(s["dY"], s["Ys"], s["pos"], s["w"], s["dYs"], s["dw"])
    dg.moe_gemm(s["dYs"], s["off"], s["W"].transpose(1, 2), s["dXs"])
    dg.moe_gemm_wgrad(s["Xs"], s["dYs"], s["off"], s["dW"])
    dg.moe_combine(s["dXs"], s["pos"], s["dX"])


def layer_state(g, T=300, k=2, E=8, H=128, N=192, dtype=BF16):
    n = T * k
    z = lambda *sh, dt=dtype: torch.zeros(*sh, dtype=dt, device=DEV)   # noqa: E731
    s = {"k": k, "E": E, "ids": choices(g, T, k, E, 0.1).to(DEV), "X": normal(g, T, H, dtype=dtype).to(DEV),
         "W": normal(g, E, H, N, dtype=dtype, scale=H ** -0.5).to(DEV), "w": torch.rand(T, k, generator=g).to(DEV),
         "dY": normal(g, T, N, dtype=dtype).to(DEV), "off": z(E + 1, dt=torch.int32), "order": z(n, dt=torch.int32),
         "pos": z(T, k, dt=torch.int32), "Xs": z(n, H), "Ys": z(n, N), "Y": z(T, N), "dYs": z(n, N), "dw": z(T, k, dt=F32),
         "dXs": z(n, H), "dW": z(E, H, N, dt=F32), "dX": z(T, H)}
    return s


OUTS = ("off", "order", "pos", "Xs", "Ys", "Y", "dYs", "dw", "dXs", "dW", "dX")


def test_layer_on_a_side_stream_and_repeats(dg):
    s = layer_state(gen(20))
    layer(dg, s)
    torch.cuda.synchronize()
    first = {o: s[o].clone() for o in OUTS}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in OUTS:
            s[o].zero_()
        layer(dg, s)
    side.synchronize()
    for o in OUTS:
        assert torch.equal(s[o], first[o]), o                    # bitwise


def test_layer_in_a_graph(dg):
    g = gen(21)
    s = layer_state(g)
    layer(dg, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(dg, s)
    for rep in range(3):
        s["ids"].copy_(choices(g, 300, 2, 8, 0.1))
        s["X"].copy_(normal(g, 300, 128))
        for o in OUTS:
            s[o].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = {o: s[o].clone() for o in OUTS}
        for o in OUTS:
            s[o].fill_(5)
        layer(dg, s)
        torch.cuda.synchronize()
        for o in OUTS:
            assert torch.equal(s[o], got[o]), (rep, o)


def test_large_sort_in_a_graph(dg):
    g = gen(22)
    ids = torch.zeros(9000, 4, dtype=torch.int64, device=DEV)
    out = [torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((65,), (36000,), (9000, 4))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_sort(ids, 64, *out)
    for rep in range(3):
        host = choices(g, 9000, 4, 64, 0.1)
        ids.copy_(host)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, _sort_quick(host, 64)):
            assert torch.equal(a.cpu(), b)
