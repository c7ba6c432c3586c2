"""Pins of the MXFP4 oracle (oracle/mx4.py) on the CPU: closed forms and torch's own decoders where it has them."""
import itertools

import numpy as np
import pytest
import torch

from oracle import mx4 as ox

POWERS = np.ldexp(1.0, np.arange(-20, 21))


def test_numbers_of_the_format():
    assert ox.MAGNITUDES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]        # OCP Microscaling Formats v1.0, table of E2M1
    assert ox.scale(np.array([0, 1, 127, 130, 254], np.uint8)).tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 8.0, 2.0 ** 127]
    assert np.isnan(ox.scale(np.array([255], np.uint8))).all()
    e8m0 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e8m0fnu).float().double().numpy()
    assert np.array_equal(ox.scale(np.arange(256, dtype=np.uint8)), e8m0, equal_nan=True)


def test_every_number_is_its_own_code():
    v = np.concatenate([ox.MAGNITUDES, -ox.MAGNITUDES])
    assert ox.encode(v).tolist() == list(range(16))                     # -0.0 is code 8


def test_midpoints_go_to_the_even_code_and_their_neighbours_apart():
    for lo, hi in itertools.pairwise(range(8)) if hasattr(itertools, "pairwise") else zip(range(7), range(1, 8)):
        mid = (ox.MAGNITUDES[lo] + ox.MAGNITUDES[hi]) / 2
        assert ox.encode(mid) == (lo if lo % 2 == 0 else hi)
        assert ox.encode(np.nextafter(mid, 0)) == lo and ox.encode(np.nextafter(mid, 9)) == hi
    assert ox.encode(1e9) == 7


def test_block_exponents():
    for p in POWERS:
        for a, floor, ceil in ((1.0, -2, -2), (1.5, -2, -2), (np.nextafter(1.5, 2), -2, -1), (1.9, -2, -1), (2.0, -1, -1), (6.0, 0, 0), (7.9, 0, 1)):
            e = int(np.log2(p))
            assert ox.block_exponent(a * p, False) == floor + e
            assert ox.block_exponent(a * p, True) == ceil + e
    g = np.random.default_rng(1)
    for a in np.exp(g.normal(0, 5, 500)):
        e = ox.block_exponent(a, False)
        assert 4 * 2.0 ** e <= a < 8 * 2.0 ** e
        e = ox.block_exponent(a, True)
        assert a <= 6 * 2.0 ** e and a > 6 * 2.0 ** (e - 1)


def test_quantised_values():
    X = torch.tensor([[6.0, -3.0, 0.2, 0.25, 0.75, -0.0] + [0.0] * 26 + [1.0, 0.5, 0.1]])
    Q, S = ox.quant(X)
    assert S.tolist() == [[127, 125]] and Q.shape == (1, 18)
    v = ox.values(Q, S, 35)
    assert v[0, :6].tolist() == [6.0, -3.0, 0.0, 0.0, 1.0, -0.0] and torch.signbit(v[0, 5])
    assert v[0, 32:].tolist() == [1.0, 0.5, 0.125] and Q[0, 17] == 0x01   # the spare half is zero
    Q, S = ox.quant(torch.tensor([[7.0, 1.0]]))
    assert ox.values(Q, S, 2).tolist() == [[6.0, 1.0]]                   # saturated
    Q, S = ox.quant(torch.tensor([[7.0, 1.0]]), True)
    assert ox.values(Q, S, 2).tolist() == [[8.0, 1.0]]                   # 3.5 of the next power, a tie


@pytest.mark.parametrize("ceil", [False, True])
def test_error_of_a_block(ceil):
    # within a block the nearest number is at most half the widest step (2) of the scale away, saturation apart
    g = torch.Generator().manual_seed(3)
    X = torch.randn(20, 64, generator=g, dtype=torch.float64) * torch.exp(torch.randn(20, 1, generator=g))
    Q, S = ox.quant(X, ceil)
    step = torch.from_numpy(ox.scale(S.numpy())).repeat_interleave(32, 1)
    assert ((ox.values(Q, S, 64) - X).abs() <= step * (1.0 if ceil else 2.0)).all()
    assert torch.equal(ox.quant(X * 2.0 ** 9, ceil)[0], Q)               # a power of two moves the scales alone
    again = ox.quant(ox.values(Q, S, 64), ceil)                          # what is of the format stays (a top of 3 at half the scale is 6)
    assert torch.equal(ox.values(*again, 64), ox.values(Q, S, 64)) and (ceil or torch.equal(again[0], Q))


def test_blocks_that_are_not_finite():
    X = torch.ones(3, 64)
    X[0, 3], X[1, 40], X[2, 63] = float("nan"), float("inf"), float("-inf")
    Q, S = ox.quant(X)
    assert (S == 255).tolist() == [[True, False], [False, True], [False, True]]
    assert torch.isnan(ox.values(Q, S, 64)).sum() == 96 and Q[0, :16].sum() == 0


def test_small_blocks():
    for x, b in ((2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** -149, 0), (0.0, 0)):
        assert int(ox.quant(torch.full((1, 32), x))[1]) == b


def test_the_product_rejects_planted_mistakes():
    from oracle.moe import check
    g = torch.Generator().manual_seed(5)
    A, W = torch.randn(9, 96, generator=g), torch.randn(7, 96, generator=g)
    (qa, sa), (qw, sw) = ox.quant(A), ox.quant(W)
    want = ox.gemm(qa, sa, qw, sw, 96, 0, torch.float32)
    a, w = ox.values(qa, sa, 96), ox.values(qw, sw, 96)
    check((a @ w.t()).float(), want, "itself")
    wrong = [a[:, :95] @ w[:, :95].t(), ox.values(qa, sa.roll(1, 1), 96) @ w.t(), ox.values(qa >> 4 | qa << 4, sa, 96) @ w.t(),
             2 * a @ w.t(), a.abs() @ w.t(), A.double() @ w.t()]
    for x in wrong:
        with pytest.raises(AssertionError):
            check(x.float(), want, "a mistake")
