"""Oracle of the microscaled 4-bit (MXFP4) operators: the definitions in 64 bits, on the CPU
(no code shared with the library).  Products return (value, bound) as oracle/moe.py does.

The numbers of an element are decoded from its fields, and an element is encoded by a search
over them, so that encoder and decoder do not rest on a common table of borders.
"""
import numpy as np
import torch

from oracle.moe import product

F64 = torch.float64


def magnitude(code):
    """The size of an E2M1 number: exponent field of 2 bits (bias 1), fraction of 1 bit."""
    e, m = (code >> 1) & 3, code & 1
    return m * 0.5 if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)


MAGNITUDES = np.array([magnitude(c) for c in range(8)])


def scale(b):
    """What a scale byte stands for."""
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.minimum(b, 254).astype(np.int64) - 127))


def encode(y):
    """The code nearest to each y; of two equally near, the even one."""
    y = np.asarray(y, dtype=np.float64)
    off = np.abs(np.abs(y)[..., None] - MAGNITUDES)
    best = off.min(-1, keepdims=True)
    near = off == best                                  # one, or two neighbours, one of them even
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, near)
    return (pick.argmax(-1) + 8 * np.signbit(y)).astype(np.uint8)


def block_exponent(a, ceil):
    """e of a block whose largest size is a > 0."""
    _, e = np.frexp(a)                                  # a = m 2^e, m in [1/2, 1)
    if not ceil:
        return e - 1 - 2
    e = e - 4                                           # 6 2^e < a: count up to the least that holds it
    while a > 6 * 2.0 ** e:
        e += 1
    return e


def quant(X, ceil=False):
    """Codes and scale bytes of X [M, K] as uint8 tensors, block by block."""
    x = X.detach().cpu().double().numpy()
    M, K = x.shape
    blocks = -(-K // 32)
    codes = np.zeros((M, 2 * ((K + 1) // 2)), np.uint8)
    S = np.zeros((M, blocks), np.uint8)
    for j in range(blocks):
        part = x[:, 32 * j:32 * j + 32]
        for m in range(M):
            row = part[m]
            if not np.isfinite(row).all():
                S[m, j] = 255
                continue
            a = np.abs(row).max()
            b = max(int(block_exponent(a, ceil)) + 127, 0) if a > 0 else 0
            S[m, j] = b
            codes[m, 32 * j:32 * j + row.size] = encode(np.ldexp(row, 127 - b))
    return torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4), torch.from_numpy(S)


def values(Q, S, K):
    """What codes and scales [..., rows, .] stand for, [..., rows, K] in 64 bits (a negative zero keeps its sign)."""
    q, s = Q.cpu().numpy(), S.cpu().numpy()
    k = np.arange(K)
    code = (q[..., k // 2] >> (4 * (k % 2)).astype(np.uint8)) & 15
    v = np.where(code & 8, -MAGNITUDES[code & 7], MAGNITUDES[code & 7])
    return torch.from_numpy(v * scale(s)[..., k // 32])


def gemm(A, SA, Q, S, K, act, out):
    """act(A @ W.T): A codes with scales SA, or 16-bit with SA None."""
    a = A.double() if SA is None else values(A, SA, K)
    # a block's sum, then its scale: one more product and sum per block
    return product(a, values(Q, S, K).t(), act, out, terms=K + 2 * S.shape[-1])


def experts(A, SA, offsets, Q, S, K, act, out):
    """gemm of every expert's rows, zeros from offsets[E] on."""
    v = torch.zeros(A.shape[0], Q.shape[1], dtype=F64)
    bound = torch.zeros_like(v)
    o = offsets.tolist()
    for e in range(Q.shape[0]):
        r = slice(o[e], o[e + 1])
        v[r], bound[r] = gemm(A[r], None if SA is None else SA[r], Q[e], S[e], K, act, out)
    return v, bound
