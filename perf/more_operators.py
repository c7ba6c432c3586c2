"""Cases of the microscaled 4-bit (MXFP4) operators: their inputs, plain forms and 64-bit values.

A case names one operator (`op`) and its sizes.  `prepare` makes the inputs that
a program holds before the call, `run` makes one pass: the operator's plain form
in elementary torch operations, or (`own`) the library's calls.  `exact` gives
the same outputs from the definition in 64 bits.

A matrix in MXFP4 is codes and scales: two 4-bit codes a byte along K (even k in the
low half: sign, then 0, .5, 1, 1.5, 2, 3, 4, 6) and for every 32 of them a byte b, the
power of two 2^(b - 127) (255: NaN).

  round    X -> codes and scales -> Y: quantised, and what the codes stand for read back
  read     codes and scales -> Y
  codes    C = act(A . W^T), A [M][K] and W [N][K] in MXFP4
  weights  the same with A in 16 bits
  experts  C[r] = act(A[r] . W[e(r)]^T) for rows in expert order, A in MXFP4 or 16 bits
"""
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "mx4": 17 / 32}


def listed():
    return [
        # the hidden states of one decoding step: latency alone
        {"name": "round step", "op": "round", "M": 16, "K": 4096, "t": "bf16", "out": "bf16", "columns": False, "ceil": False},
        # activations of a training batch along their tokens, for the gradient of the weights
        {"name": "round columns", "op": "round", "M": 4096, "K": 8192, "t": "bf16", "out": "bf16", "columns": True, "ceil": True},
        # an FFN matrix read back in 16 bits
        {"name": "read weights", "op": "read", "M": 14336, "K": 4096, "out": "bf16"},
        # a small matrix with an odd number of columns
        {"name": "read odd", "op": "read", "M": 777, "K": 2055, "out": "f32"},
        # FFN up-projection of one decoding step of 16 sequences, activations in 4 bits too
        {"name": "codes step", "op": "codes", "M": 16, "K": 4096, "N": 14336, "out": "bf16", "act": "gelu"},
        # the same FFN for a prompt batch: matrix work
        {"name": "codes prompt", "op": "codes", "M": 4096, "K": 4096, "N": 14336, "out": "bf16", "act": "none"},
        # gradient of a weight matrix, summed over a ragged number of tokens, kept in 32 bits for the optimizer
        {"name": "codes train", "op": "codes", "M": 4096, "K": 5000, "N": 4096, "out": "f32", "act": "none"},
        # one token through the FFN up-projection, activations in 16 bits: the weights' bytes
        {"name": "weights token", "op": "weights", "M": 1, "K": 4096, "N": 14336, "t": "bf16", "out": "bf16", "act": "none"},
        # an odd number of sequences through the down-projection
        {"name": "weights batch", "op": "weights", "M": 33, "K": 14336, "N": 4096, "t": "f16", "out": "f32", "act": "none"},
        # a prompt through a projection, activations in 16 bits
        {"name": "weights prompt", "op": "weights", "M": 2048, "K": 4096, "N": 4096, "t": "bf16", "out": "bf16", "act": "none"},
        # one decoding step of 8 sequences, 2 of 16 experts each
        {"name": "experts step", "op": "experts", "T": 8, "k": 2, "E": 16, "K": 4096, "N": 7168, "t": "bf16", "out": "bf16", "act": "gelu"},
        # a prompt batch over 8 experts, everything in 4 bits
        {"name": "experts prompt", "op": "experts", "T": 8192, "k": 2, "E": 8, "K": 4096, "N": 14336, "t": "mx4", "out": "bf16", "act": "none"},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        """A size spread over the logarithm of lo..hi, a multiple of step."""
        return min(hi, max(step, int(round(lo * (hi / lo) ** rng.random() / step)) * step))

    op = rng.choice(["round", "round", "read", "codes", "codes", "codes", "weights", "weights", "weights", "experts", "experts"])
    t = rng.choice(["bf16", "f16"])
    if op in ("round", "read"):
        case = {"op": op, "M": size(1, 8192), "K": size(32, 8192, rng.choice([32, 128, 8, 1])), "out": rng.choice([t, "f32"])}
        if op == "round":
            case.update(t=rng.choice([t, t, "f32"]), columns=rng.random() < 0.4, ceil=rng.random() < 0.5)
        return case
    K = size(64, 8192, rng.choice([256, 128, 32, 1]))
    N = size(32, 8192, rng.choice([64, 16, 1]))
    case = {"op": op, "K": K, "N": N, "out": rng.choice([t, "f32"]), "act": rng.choice(["none", "none", "gelu", "relu"])}
    if op == "experts":
        E = size(2, 32)
        case.update(T=size(1, 4096), k=rng.randint(1, min(4, E)), E=E, K=min(K, 4096), N=min(N, 4096), t=rng.choice(["mx4", t]))
        return case
    case.update(M=size(1, 4096))
    if op == "weights":
        case.update(t=t)
    return case


# ------------------------------------------------------------------ inputs

def _generator(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1) + sum(map(ord, case["op"])))
    return g


def _values(g, rows, K, scale=1.0):
    """Normal values whose columns differ in size, as activations' and weights' do."""
    return torch.randn(rows, K, generator=g, device=DEV) * (scale * torch.exp(0.5 * torch.randn(K, generator=g, device=DEV)))


def _offsets(case, g):
    """Where each expert's rows end: the k largest of E router logits, some experts more liked than others."""
    logits = torch.randn(case["T"], case["E"], generator=g, device=DEV) + 0.5 * torch.randn(case["E"], generator=g, device=DEV)
    ids = logits.topk(case["k"], dim=1).indices.reshape(-1)
    return torch.cat([ids.new_zeros(1), (ids[:, None] == torch.arange(case["E"], device=DEV)).sum(0).cumsum(0)]).int()


def prepare(case, seed):
    g, op = _generator(case, seed), case["op"]
    s = {"case": case}
    if op in ("round", "read"):
        M, K = case["M"], case["K"]
        x = _values(g, M, K)
        if op == "read":
            s["Q"], s["S"] = _quantised(x, False)
        else:
            x = x.to(TYPES[case["t"]])
            s["X"] = x.t().contiguous().t() if case["columns"] else x
            s["Q"] = torch.zeros(M, (K + 1) // 2, device=DEV, dtype=torch.uint8)
            s["S"] = torch.zeros(M, -(-K // 32), device=DEV, dtype=torch.uint8)
        s["Y"] = torch.zeros(M, K, device=DEV, dtype=TYPES[case["out"]])
        return s
    K, N = case["K"], case["N"]
    if op == "experts":
        s["offsets"] = _offsets(case, g)
        s["Q"] = torch.empty(case["E"], N, (K + 1) // 2, device=DEV, dtype=torch.uint8)
        s["S"] = torch.empty(case["E"], N, -(-K // 32), device=DEV, dtype=torch.uint8)
        for e in range(case["E"]):
            s["Q"][e], s["S"][e] = _quantised(_values(g, N, K, K ** -0.5), False)
    else:
        s["Q"], s["S"] = _quantised(_values(g, N, K, K ** -0.5), False)
    rows = case["T"] * case["k"] if op == "experts" else case["M"]
    s["A"], s["SA"] = torch.randn(rows, K, generator=g, device=DEV), None
    if case.get("t", "mx4") == "mx4":
        s["A"], s["SA"] = _quantised(s["A"], False)
    else:
        s["A"] = s["A"].to(TYPES[case["t"]])
    s["C"] = torch.zeros(rows, N, device=DEV, dtype=TYPES[case["out"]])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_19_amd as dg
    case = s["case"]
    op, act = case["op"], {"none": dg.DG_ACT_NONE, "relu": dg.DG_ACT_RELU, "gelu": dg.DG_ACT_GELU_TANH}[case.get("act", "none")]
    if op == "round":
        dg.quant_mx4(s["X"], s["Q"], s["S"], dg.DG_MX4_CEIL if case["ceil"] else dg.DG_MX4_FLOOR)
    if op in ("round", "read"):
        return {"Y": dg.dequant_mx4(s["Q"], s["S"], s["Y"])}
    if op == "experts":
        return {"C": dg.moe_gemm_mx4(s["A"], s["offsets"], s["Q"], s["S"], s["C"], SA=s["SA"], act=act)}
    return {"C": dg.gemm_mx4(s["A"], s["Q"], s["S"], s["C"], SA=s["SA"], act=act)}


def _blocks(x):
    """[M][K] as [M][blocks][32], zeros past K."""
    M, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 32)).reshape(M, -1, 32)


def _quantised(x, ceil):
    """Codes and scales of x [M][K]."""
    M, K = x.shape
    b = _blocks(x.float())
    bits = b.abs().amax(-1).view(torch.int32)                       # of the largest value
    field = (bits >> 23) - 2 + (((bits & 0x7FFFFF) > 0x400000).int() if ceil else 0)
    field = field.clamp(min=0)
    y = b * torch.exp2(127.0 - field)[..., None]
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)) + 8 * torch.signbit(y)
    code = torch.where(torch.arange(code.shape[1] * 32, device=x.device).reshape(-1, 32) < K, code, 0).reshape(M, -1, 2)
    return (code[..., 0] + 16 * code[..., 1])[:, :(K + 1) // 2].to(torch.uint8).contiguous(), field.to(torch.uint8)


def _dense(Q, S, K):
    """What codes and scales [..., rows, .] stand for, in 32 bits (exact)."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=Q.device)
    v = table[torch.stack([Q & 15, Q >> 4], dim=-1).flatten(-2)[..., :K].int()]
    return v * torch.exp2(S.float() - 127.0).repeat_interleave(32, dim=-1)[..., :K]


def _activated(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x))) if act == "gelu" else x


def _plain(s):
    case = s["case"]
    op, K, out = case["op"], case["K"], TYPES[case["out"]]
    if op == "round":
        return {"Y": _dense(*_quantised(s["X"], case["ceil"]), K).to(out)}
    if op == "read":
        return {"Y": _dense(s["Q"], s["S"], K).to(out)}
    A = s["A"].float() if s["SA"] is None else _dense(s["A"], s["SA"], K)
    W = _dense(s["Q"], s["S"], K)
    if op != "experts":
        return {"C": _activated(A @ W.t(), case["act"]).to(out)}
    # every expert's rows padded to the longest, one batched product, the rows back
    off, n = s["offsets"], A.shape[0]
    r = torch.arange(n, device=DEV)
    expert = (r[:, None] >= off[None, 1:]).sum(1)
    table = off[:-1, None] + torch.arange(int((off[1:] - off[:-1]).max()), device=DEV)
    padded = A[table.clamp(max=n - 1)] * (table < off[1:, None])[..., None]
    C = torch.bmm(padded, W.transpose(1, 2).contiguous())[expert, r - off[expert]]
    return {"C": _activated(C, case["act"]).to(out)}


# ------------------------------------------------------------------ work

def work(case):
    op, K, out = case["op"], case["K"], SIZE[case["out"]]
    if op in ("round", "read"):
        n = case["M"] * K
        # X read, codes and scales written, Y written; or codes and scales read, Y written
        return {"bytes": n * ((SIZE[case["t"]] if op == "round" else 0) + SIZE["mx4"] + out), "flops": n}
    N, rows = case["N"], case["T"] * case["k"] if op == "experts" else case["M"]
    used = min(case["E"], rows) if op == "experts" else 1
    return {"bytes": rows * K * SIZE[case.get("t", "mx4")] + used * N * K * SIZE["mx4"] + rows * N * out, "flops": 2 * rows * K * N}


# ------------------------------------------------------------------ the values in 64 bits

def _magnitudes():
    """The eight sizes of an E2M1 number from its fields: exponent e, one bit m."""
    return torch.tensor([m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1) for e in range(4) for m in range(2)], device=DEV, dtype=torch.float64)


def _matrix(Q, S, K):
    k = torch.arange(K, device=DEV)
    code = (Q[:, k // 2].int() >> (4 * (k % 2))) & 15
    v = _magnitudes()[code & 7] * (1 - 2 * (code >> 3)).double()
    return torch.ldexp(v, S[:, k // 32].int() - 127)


def exact(case, seed):
    s, op, K = prepare(case, seed), case["op"], case["K"]
    if op == "read":
        return {"Y": _matrix(s["Q"], s["S"], K)}
    if op == "round":
        x = _blocks(s["X"].double())
        top = x.abs().amax(-1)
        if case["ceil"]:
            m, e = torch.frexp(top / 6)                              # top / 6 = m 2^e, m in [1/2, 1)
            e = torch.where(m == 0.5, e - 1, e)
        else:
            e = torch.frexp(top)[1] - 3
        e = torch.where(top == 0, -127, e).clamp(min=-127)[..., None]
        y, near, sizes = torch.ldexp(x.abs(), -e), torch.full_like(x, float("inf")), _magnitudes()
        value = torch.zeros_like(x)
        for c in (0, 2, 4, 6, 1, 3, 5, 7):                           # of two equally near the even code, which is first
            off = (y - sizes[c]).abs()
            value, near = torch.where(off < near, sizes[c], value), torch.minimum(off, near)
        return {"Y": (torch.ldexp(value, e) * torch.where(x < 0, -1.0, 1.0)).reshape(x.shape[0], -1)[:, :K].contiguous()}
    C = torch.zeros(s["C"].shape, device=DEV, dtype=torch.float64)
    bounds = s["offsets"].tolist() if op == "experts" else [0, case["M"]]
    for e in range(len(bounds) - 1):
        rows = slice(bounds[e], bounds[e + 1])
        W = _matrix(s["Q"][e], s["S"][e], K) if op == "experts" else _matrix(s["Q"], s["S"], K)
        A = s["A"][rows].double() if s["SA"] is None else _matrix(s["A"][rows], s["SA"][rows], K)
        C[rows] = A @ W.t()
    if case["act"] == "relu":
        C = torch.clamp(C, min=0)
    elif case["act"] == "gelu":
        C = C * torch.sigmoid(2 * 0.7978845608028654 * (C + 0.044715 * C ** 3))
    return {"C": C}
