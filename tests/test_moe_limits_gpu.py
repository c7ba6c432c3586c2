"""GPU tests of the mixture-of-experts operators at the ends of what they accept."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()   # raises if the library is missing: there is no fallback
    return m


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def test_sort_of_as_many_ids_as_there_are_numbers(dg):
    # 2^31 - 1 choices of one expert (one id, read again and again): every place up to the last
    room(24)
    n = 2 ** 31 - 1
    order, pos = (torch.full((n,), -7, dtype=I32, device=DEV) for _ in range(2))
    offsets = torch.zeros(2, dtype=I32, device=DEV)
    dg.moe_sort(torch.zeros(1, 1, dtype=I32, device=DEV).expand(n, 1), 1, offsets, order, pos.view(n, 1))
    assert offsets.tolist() == [0, n]
    for t in (order, pos):
        for i in range(0, n, 1 << 28):
            part = t[i:i + (1 << 28)]
            assert torch.equal(part, torch.arange(i, i + part.numel(), dtype=I32, device=DEV)), i


# 2^32 threads do not fit one launch: 64 threads a row of 264, 2^26 rows and a few
MANY, H = 2 ** 26 + 3, 264


def test_gather_and_combine_of_more_rows_than_a_launch_holds(dg):
    room(48)
    X = torch.randn(1000, H, device=DEV).to(BF16)
    place = torch.arange(MANY, dtype=I32, device=DEV) % 1000
    out = torch.empty(MANY, H, dtype=BF16, device=DEV)
    step = 1 << 22

    def check():
        for i in range(0, MANY, step):
            assert torch.equal(out[i:i + step], X[place[i:i + step].long()]), i
    dg.moe_gather(X, place, 1, out)
    check()
    out.fill_(7)
    dg.moe_combine(X, place.view(MANY, 1), out)
    check()


@pytest.mark.parametrize("T,H", [(2 ** 24 + 5, 1024), (MANY, H)])   # a workgroup, 64 threads a token
@pytest.mark.parametrize("weighted", [False, True])
def test_combine_gradient_of_more_tokens_than_a_launch_holds(dg, T, H, weighted):
    room(8)
    named = {T - 1: 0, T // 2 + 1: 2, 0: 4}                     # token -> its row; every other choice is dropped
    pos = torch.full((T, 1), -1, dtype=I32, device=DEV)
    for t, r in named.items():
        pos[t, 0] = r
    g = torch.Generator().manual_seed(1)
    dY = torch.randint(-8, 9, (1, H), generator=g).to(DEV, BF16)    # the same for every token
    Ys = torch.randint(-8, 9, (6, H), generator=g).to(DEV, BF16)
    w = torch.full((1, 1), 0.5, device=DEV).expand(T, 1) if weighted else None
    dw = torch.full((T, 1), float("nan"), device=DEV) if weighted else None
    dYs = torch.full((6, H), float("nan"), dtype=BF16, device=DEV)
    dg.moe_combine_grad(dY.expand(T, H), Ys, pos, w, dYs, dw)
    want = torch.zeros(6, H, device=DEV)
    want[[0, 2, 4]] = dY[0].float() * (0.5 if weighted else 1.0)
    assert torch.equal(dYs.float(), want)
    if weighted:                                                 # whole numbers: the sums are exact
        for t, r in named.items():
            assert float(dw[t, 0]) == float((dY[0].double() * Ys[r].double()).sum())
            dw[t, 0] = 0
        assert int(dw.count_nonzero()) == 0


def test_products_of_more_tiles_than_a_launch_holds(dg):
    room(8)
    E = 2 ** 24
    A, D = (torch.ones(16, 8, dtype=BF16, device=DEV) for _ in range(2))
    off = torch.zeros(E + 1, dtype=I32, device=DEV)
    dW = torch.full((E, 8, 8), 3.0, dtype=BF16, device=DEV)
    with pytest.raises(dg.DGError, match="OVERFLOW"):
        dg.moe_gemm_wgrad(A, D, off, dW)
    torch.cuda.synchronize()
    assert int((dW != 3).sum()) == 0
