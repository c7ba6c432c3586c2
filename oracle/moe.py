"""Oracle of the mixture-of-experts and 4-bit operators: the definitions in 64 bits,
on the CPU, one expert or token at a time (no code shared with the library).

Every function returns (value, bound): the exact value and, element by element,
how far a right FP32 computation rounded once to `out` may be from it.
  - A sum of m products in FP32, in any order, is off by at most 2 m u S, with
    u = 2^-24 and S the sum of the terms' sizes (the factor 2 covers a matrix
    core that cuts instead of rounding).
  - Rounding to `out` adds half a step: eps/2 of the value, or half the smallest
    step of the type near zero.
  - GELU (tanh form) has slopes of at most 1.13 and is evaluated in FP32 to
    8 u |y|.
"""
import numpy as np
import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(value, dtype):
    """Half a step of dtype at the value (or at zero)."""
    f = torch.finfo(dtype)
    return torch.clamp(value.abs() * (f.eps / 2), min=f.tiny * f.eps / 2)


def act64(y, act):
    if act == 1:
        return torch.where(y < 0, torch.zeros_like(y), y)
    if act == 2:
        return 0.5 * y * (1 + torch.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))
    return y


def finish(y, err, act, out):
    """The activated value and its bound, from a sum and its bound."""
    v = act64(y, act)
    if act == 2:
        err = 1.13 * err + 8 * U * y.abs()
    return v, err + half_step(v.abs() + err, out)


def sort(ids, E):
    """offsets, order, pos by walking the choices expert by expert."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    order, offsets = [], [0]
    for e in range(E):
        order += [i for i, x in enumerate(flat) if x == e]
        offsets.append(len(order))
    pos = [-1] * len(flat)
    for r, i in enumerate(order):
        pos[i] = r
    order += [-1] * (len(flat) - len(order))
    t = lambda x: torch.tensor(x, dtype=torch.int32)   # noqa: E731
    return t(offsets), t(order), t(pos).reshape(T, k)


def combine(Ys, pos, w, out):
    T, k = pos.shape
    y = torch.zeros(T, Ys.shape[1], dtype=F64)
    size = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            r = int(pos[t, j])
            if 0 <= r < Ys.shape[0]:
                term = Ys[r].double() * (1.0 if w is None else float(w[t, j]))
                y[t] += term
                size[t] += term.abs()
    return finish(y, 2 * k * U * size, 0, out)


def combine_grad(dY, Ys, pos, w):
    """(dYs, bound), (dw, bound)."""
    T, k = pos.shape
    dYs = torch.zeros(Ys.shape, dtype=F64)
    dw, size = torch.zeros(T, k, dtype=F64), torch.zeros(T, k, dtype=F64)
    for t in range(T):
        for j in range(k):
            r = int(pos[t, j])
            if 0 <= r < Ys.shape[0]:
                dYs[r] = dY[t].double() * (1.0 if w is None else float(w[t, j]))
                p = dY[t].double() * Ys[r].double()
                dw[t, j], size[t, j] = p.sum(), p.abs().sum()
    a = finish(dYs, U * dYs.abs(), 0, Ys.dtype)
    return a, None if w is None else finish(dw, 2 * Ys.shape[1] * U * size, 0, w.dtype)


def product(a, b, act, out, terms=None):
    """act(a @ b) of 64-bit matrices."""
    y = a.double() @ b.double()
    size = a.double().abs() @ b.double().abs()
    return finish(y, 2 * (a.shape[1] if terms is None else terms) * U * size, act, out)


def experts(A, offsets, W, act, out):
    """act(A[r] @ W[e]) of every expert's rows, zeros from offsets[E] on."""
    v = torch.zeros(A.shape[0], W.shape[2], dtype=F64)
    bound = torch.zeros_like(v)
    o = offsets.tolist()
    for e in range(W.shape[0]):
        v[o[e]:o[e + 1]], bound[o[e]:o[e + 1]] = product(A[o[e]:o[e + 1]], W[e], act, out)
    return v, bound


def wgrad(A, D, offsets, out):
    o = offsets.tolist()
    parts = [product(A[o[e]:o[e + 1]].t(), D[o[e]:o[e + 1]], 0, out) for e in range(len(o) - 1)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def dense4(Q, S, Z, K, G):
    """The weights [N][K] of 4-bit codes, code by code (exact)."""
    N = Q.shape[0]
    W = torch.zeros(N, K, dtype=F64)
    for k in range(K):
        q = (Q[:, k // 2].int() >> (4 * (k % 2))) & 15
        z = 8 if Z is None else Z[:, k // G].int()
        W[:, k] = S[:, k // G].double() * (q - z).double()
    return W


def w4(A, Q, S, Z, G, act, out):
    K = A.shape[1]
    # each group's sum, then its scale: one more product and sum per group
    return product(A, dense4(Q, S, Z, K, G).t(), act, out, terms=K + 2 * S.shape[1])


def w4_experts(A, offsets, Q, S, Z, G, act, out):
    v = torch.zeros(A.shape[0], Q.shape[1], dtype=F64)
    bound = torch.zeros_like(v)
    o = offsets.tolist()
    for e in range(Q.shape[0]):
        r = slice(o[e], o[e + 1])
        v[r], bound[r] = w4(A[r], Q[e], S[e], None if Z is None else Z[e], G, act, out)
    return v, bound


def check(got, want, what=""):
    """Every element within its bound; non-finite values have to agree."""
    v, bound = want
    g = got.detach().cpu().double()
    assert g.shape == v.shape, (what, g.shape, v.shape)
    finite = torch.isfinite(v)
    assert torch.equal(torch.isnan(g), torch.isnan(v)), f"{what}: NaN places differ"
    assert torch.equal(g[~finite & ~torch.isnan(v)], v[~finite & ~torch.isnan(v)]), f"{what}: infinities differ"
    err = (g - v).abs()[finite]
    over = err > bound[finite]
    worst = float((err / bound[finite].clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"[{what}] worst err/bound {worst:.3g}", flush=True)
    assert not bool(over.any()), f"{what}: {int(over.sum())} of {over.numel()} outside, worst {worst:.3g}"
