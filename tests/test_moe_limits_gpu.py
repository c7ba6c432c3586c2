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
