"""GPU tests of MXFP4 products whose rows of codes begin at whole words but are no whole words long: the end of K of
the last row of either operand, in every tile that loads straight to LDS."""
import pytest
import torch

from oracle import moe as om
from oracle import mx4 as ox
from test_mx4_gpu import DEV, F32, NAN, coded, gen, in_ones

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_19_amd as m
    m.lib()
    return m


def words(t, extra=0):
    """Rows in a pitch of whole words; NaN scales and codes of -6 between them, nothing behind the last one."""
    cols = t.shape[-1]
    return in_ones(t, 4, 0, cols + (-cols) % 4 + extra)


# rows of 129, 167, 389, 501 and 1301 bytes (1 and 3 past a word, 1 to 13 past 16), of 250, 502 and 2510 (2 past a word)
@pytest.mark.parametrize("K", [257, 333, 778, 1001, 2602, 500, 1004, 5019])
@pytest.mark.parametrize("M,N,tile", [(70, 50, 64), (129, 300, 64), (1030, 2900, 128), (4000, 3300, 256)])
def test_rows_of_no_whole_words(dg, M, N, K, tile):
    if tile == 256 and K > 1100:
        K = 1003
    g = gen(M, N, K)
    (A, SA), (Q, S) = coded(g, M, K, (118, 128)), coded(g, N, K, (118, 128))
    want = ox.gemm(A, SA, Q, S, K, 0, F32)
    for extra in (0, 12):
        a, q, s, sa = words(A, extra), words(Q), in_ones(S, 5, 0), in_ones(SA, 1, 0)
        C = torch.full((M, N), NAN, device=DEV)
        plan = dg.gemm_mx4_plan(a, q, s, C, SA=sa)
        assert plan.startswith(f"direct loads, {tile}x{tile}"), plan
        dg.gemm_mx4(a, q, s, C, SA=sa)
        om.check(C, want, f"{M}x{N}x{K}")


@pytest.mark.parametrize("K", [333, 778, 2602])
@pytest.mark.parametrize("counts,N,tile", [([70, 0, 90, 33], 130, 64), ([300, 520, 0, 200], 4096, 128)])
def test_experts(dg, counts, N, K, tile):
    # the last row of every expert's A has the next expert's behind it, the last of every W the next W
    g = gen(sum(counts), N, K)
    E, n = len(counts), sum(counts)
    off = torch.tensor([0] + counts).cumsum(0).int()
    A, SA = coded(g, n, K, (118, 128))
    Q, S = coded(g, E * N, K, (118, 128))
    want = ox.experts(A, SA, off, Q.view(E, N, -1), S.view(E, N, -1), K, 0, F32)
    a, q, s, sa = words(A), words(Q).unflatten(0, (E, N)), in_ones(S.view(E, N, -1)), in_ones(SA)
    C = torch.full((n, N), NAN, device=DEV)
    plan = dg.moe_gemm_mx4_plan(a, off.to(DEV), q, s, C, SA=sa)
    assert plan.startswith(f"direct loads, {tile}x{tile}"), plan
    dg.moe_gemm_mx4(a, off.to(DEV), q, s, C, SA=sa)
    om.check(C, want, f"{counts} {K}")
