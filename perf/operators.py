"""Cases of the mixture-of-experts and 4-bit operators: their inputs, plain forms and 64-bit values.

A case names one operator (`op`) and its sizes.  `prepare` makes the inputs that
a program holds before the call, `run` makes one pass: the operator's plain form
in elementary torch operations, or (`own`) the library's call.  `exact` gives
the same outputs from the definition in 64 bits.

Operators (rows of Xs, Ys, A, C are in expert order: expert 0's rows, then expert 1's, ...):
  sort          expert ids [T][k] -> offsets [E+1], order [T*k], pos [T][k] (stable counting sort;
                ids outside 0..E-1 are dropped: order and pos are -1 there)
  gather        Xs[r] = X[order[r] / k]
  combine       Y[t] = sum_j w[t][j] * Ys[pos[t][j]]  (no weights: the gradient of gather)
  combine_grad  dYs[pos[t][j]] = w[t][j] * dY[t],  dw[t][j] = <dY[t], Ys[pos[t][j]]>
  experts       C[r] = act(A[r] . W[e(r)])            (the products of every expert)
  experts_dx    dA[r] = dC[r] . W[e(r)]^T
  experts_dw    dW[e] = sum of A[r]^T dC[r] over the rows of expert e
  w4            C = act(A . W^T), W[n][k] = s[n][k/G] * (q[n][k] - z[n][k/G]), q in 4 bits
  w4_experts    the same with the weights of every expert, A's rows in expert order
"""
import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i32": 4, "i64": 8}


def listed():
    return [
        # one decoding step of 64 sequences, 8 of 64 experts each: the call is latency alone
        {"name": "sort step", "op": "sort", "T": 64, "k": 8, "E": 64, "ids": "i64", "drop": 0.0},
        # the tokens of a long prompt batch over many small experts, some past their expert's capacity
        {"name": "sort prompt", "op": "sort", "T": 32768, "k": 8, "E": 256, "ids": "i32", "drop": 0.05},
        # hidden states of a prompt batch copied into expert order
        {"name": "gather prompt", "op": "gather", "T": 8192, "k": 2, "E": 8, "H": 4096, "t": "bf16", "drop": 0.0},
        # the experts' outputs of one decoding step back in token order, weighted
        {"name": "combine step", "op": "combine", "T": 48, "k": 8, "E": 64, "H": 2048, "t": "bf16", "wt": "f32", "drop": 0.0},
        # the backward pass of that step in training: gradients of rows and router weights
        {"name": "combine train", "op": "combine_grad", "T": 4096, "k": 8, "E": 64, "H": 2048, "t": "bf16", "wt": "f32", "drop": 0.0},
        # FFN up-projection of 8 experts for 16 sequences at decode: the weights' bytes
        {"name": "experts step", "op": "experts", "T": 16, "k": 2, "E": 8, "K": 4096, "N": 14336, "t": "bf16", "out": "bf16", "act": "gelu"},
        # the same FFN for a prompt batch: matrix work
        {"name": "experts prompt", "op": "experts", "T": 8192, "k": 2, "E": 8, "K": 4096, "N": 14336, "t": "bf16", "out": "bf16", "act": "none"},
        # gradient of the inputs of 64 small experts, ragged row counts
        {"name": "experts train dx", "op": "experts_dx", "T": 2500, "k": 6, "E": 64, "K": 512, "N": 4096, "t": "f16", "out": "f16", "act": "none"},
        # gradient of the weights, kept in 32 bits for the optimizer
        {"name": "experts train dw", "op": "experts_dw", "T": 4096, "k": 2, "E": 8, "K": 4096, "N": 4096, "t": "bf16", "out": "f32", "act": "none"},
        # one token through a 4-bit FFN up-projection
        {"name": "w4 token", "op": "w4", "M": 1, "K": 4096, "N": 14336, "G": 128, "zeros": False, "t": "bf16", "st": "bf16", "out": "bf16", "act": "none"},
        # an odd number of sequences through the down-projection, asymmetric codes in small groups
        {"name": "w4 batch", "op": "w4", "M": 33, "K": 14336, "N": 4096, "G": 64, "zeros": True, "t": "f16", "st": "f16", "out": "f32", "act": "none"},
        # a decoding step of 8 sequences over 16 experts held in 4 bits
        {"name": "w4 experts step", "op": "w4_experts", "T": 8, "k": 2, "E": 16, "K": 4096, "N": 7168, "G": 32, "zeros": True, "t": "bf16", "st": "bf16", "out": "bf16", "act": "gelu"},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        """A size spread over the logarithm of lo..hi, a multiple of step."""
        n = 3072
        while n == 3072:
            n = max(step, int(round(lo * (hi / lo) ** rng.random() / step)) * step)
        return min(n, hi)

    op = rng.choice(["sort", "gather", "combine", "combine_grad", "experts", "experts", "experts_dx", "experts_dw", "w4", "w4", "w4_experts"])
    t = rng.choice(["bf16", "f16"])
    if op == "sort":
        E = size(2, 256)
        return {"op": op, "T": size(1, 32768), "k": rng.randint(1, min(8, E)), "E": E, "ids": rng.choice(["i32", "i64"]), "drop": rng.choice([0.0, 0.1, 1.0 / 3])}
    if op in ("gather", "combine", "combine_grad"):
        E = size(4, 128)
        case = {"op": op, "T": size(1, 4096), "k": rng.randint(1, min(8, E)), "E": E, "H": size(64, 4096, rng.choice([1, 8, 64])),
                "t": rng.choice(["bf16", "f16", "f32"]), "drop": rng.choice([0.0, 0.1])}
        if op != "gather":
            case["wt"] = rng.choice(["f32", case["t"]] + (["none"] if op == "combine" else []))
        return case
    group = rng.choice([32, 64, 128])
    K = size(64, 4096, rng.choice([64, 64, 8, 1]))
    N = size(64, 4096, rng.choice([64, 64, 8, 1]))
    out = rng.choice([t, "f32"])
    act = rng.choice(["none", "none", "gelu", "relu"])
    if op == "w4":
        K = size(128, 14336, rng.choice([128, 32, 32, 1]))
        return {"op": op, "M": size(1, 256), "K": K, "N": size(64, 7168, rng.choice([16, 64, 1])), "G": group,
                "zeros": rng.random() < 0.5, "t": t, "st": rng.choice([t, "f32"]), "out": out, "act": act}
    E = size(2, 64)
    k = rng.randint(1, min(4, E))
    if op == "w4_experts":
        K = size(128, 4096, rng.choice([128, 32, 32, 1]))
        return {"op": op, "T": size(1, 512), "k": k, "E": min(E, 32), "K": K, "N": N, "G": group, "zeros": rng.random() < 0.5,
                "t": t, "st": rng.choice([t, "f32"]), "out": out, "act": act}
    return {"op": op, "T": size(1, 4096), "k": k, "E": E, "K": K, "N": N, "t": t,
            "out": "f32" if op == "experts_dw" and out == "f32" else t, "act": act if op == "experts" else "none"}


# ------------------------------------------------------------------ inputs

def _generator(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1) + sum(map(ord, case["op"])))
    return g


def _normal(g, shape, t, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPES[t])


def _ids(case, g):
    """The k experts of every token: the largest of E router logits, some experts more liked than others."""
    logits = torch.randn(case["T"], case["E"], generator=g, device=DEV) + 0.5 * torch.randn(case["E"], generator=g, device=DEV)
    ids = logits.topk(case["k"], dim=1).indices
    if case.get("drop"):
        ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < case["drop"], torch.full_like(ids, -1), ids)
    return ids


def _sorted(ids, E):
    """offsets, order, pos of the definition, on the host."""
    flat = ids.reshape(-1).cpu().numpy()
    order = np.full(flat.size, -1, np.int32)
    pos = np.full(flat.size, -1, np.int32)
    kept = np.nonzero((flat >= 0) & (flat < E))[0]
    by = kept[np.argsort(flat[kept], kind="stable")]
    order[:by.size] = by
    pos[by] = np.arange(by.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))]).astype(np.int32)
    return [torch.from_numpy(x).to(DEV) for x in (offsets, order, pos.reshape(ids.shape))]


def prepare(case, seed):
    g, op = _generator(case, seed), case["op"]
    s = {"case": case}
    if op in ("w4", "w4_experts"):
        E = (case["E"],) if op == "w4_experts" else ()
        N, K, groups = case["N"], case["K"], -(-case["K"] // case["G"])
        s["Q"] = torch.randint(0, 256, E + (N, (K + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["S"] = ((0.5 + torch.rand(E + (N, groups), generator=g, device=DEV)) * (0.2 / K ** 0.5)).to(TYPES[case["st"]])
        s["Z"] = torch.randint(5, 12, E + (N, groups), generator=g, device=DEV, dtype=torch.uint8) if case["zeros"] else None
        rows = case["T"] * case["k"] if op == "w4_experts" else case["M"]
        if op == "w4_experts":
            s["offsets"] = _sorted(_ids(case, g), case["E"])[0]
        s["A"] = _normal(g, (rows, K), case["t"])
        s["C"] = torch.zeros(rows, N, device=DEV, dtype=TYPES[case["out"]])
        return s
    ids = _ids(case, g)
    n, E = ids.numel(), case["E"]
    if op == "sort":
        s["ids"] = ids.to({"i32": torch.int32, "i64": torch.int64}[case["ids"]])
        s["offsets"], s["order"], s["pos"] = (torch.zeros(z, device=DEV, dtype=torch.int32) for z in ((E + 1,), (n,), ids.shape))
        return s
    offsets, order, pos = _sorted(ids, E)
    if op == "gather":
        s["order"], s["X"] = order, _normal(g, (case["T"], case["H"]), case["t"])
        s["Xs"] = torch.zeros(n, case["H"], device=DEV, dtype=TYPES[case["t"]])
    elif op in ("combine", "combine_grad"):
        s["pos"], s["Ys"] = pos, _normal(g, (n, case["H"]), case["t"])
        s["w"] = None if case["wt"] == "none" else torch.rand(ids.shape, generator=g, device=DEV).to(TYPES[case["wt"]])
        s["Y"] = torch.zeros(case["T"], case["H"], device=DEV, dtype=TYPES[case["t"]])
        if op == "combine_grad":
            s["Y"] = _normal(g, (case["T"], case["H"]), case["t"])
            s["dYs"], s["dw"] = torch.zeros_like(s["Ys"]), torch.zeros_like(s["w"])
    else:
        K, N = case["K"], case["N"]
        s["offsets"] = offsets
        if op != "experts_dw":
            s["W"] = _normal(g, (E, K, N), case["t"], K ** -0.5)
        if op != "experts_dx":
            s["A"] = _normal(g, (n, K), case["t"])
        if op != "experts":
            s["D"] = _normal(g, (n, N), case["t"])
        s["C"] = torch.zeros({"experts": (n, N), "experts_dx": (n, K), "experts_dw": (E, K, N)}[op], device=DEV, dtype=TYPES[case["out"]])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_19_amd as dg
    case = s["case"]
    op, act = case["op"], {"none": dg.DG_ACT_NONE, "relu": dg.DG_ACT_RELU, "gelu": dg.DG_ACT_GELU_TANH}[case.get("act", "none")]
    if op == "sort":
        dg.moe_sort(s["ids"], case["E"], s["offsets"], s["order"], s["pos"])
        return {"offsets": s["offsets"], "order": s["order"], "pos": s["pos"]}
    if op == "gather":
        return {"Xs": dg.moe_gather(s["X"], s["order"], case["k"], s["Xs"])}
    if op == "combine":
        return {"Y": dg.moe_combine(s["Ys"], s["pos"], s["Y"], s["w"])}
    if op == "combine_grad":
        dg.moe_combine_grad(s["Y"], s["Ys"], s["pos"], s["w"], s["dYs"], s["dw"])
        return {"dYs": s["dYs"], "dw": s["dw"]}
    if op == "experts":
        return {"C": dg.moe_gemm(s["A"], s["offsets"], s["W"], s["C"], act)}
    if op == "experts_dx":
        return {"dA": dg.moe_gemm(s["D"], s["offsets"], s["W"].transpose(1, 2), s["C"])}
    if op == "experts_dw":
        return {"dW": dg.moe_gemm_wgrad(s["A"], s["D"], s["offsets"], s["C"])}
    if op == "w4":
        return {"C": dg.gemm_w4(s["A"], s["Q"], s["S"], s["C"], group=case["G"], Z=s["Z"], act=act)}
    return {"C": dg.moe_gemm_w4(s["A"], s["offsets"], s["Q"], s["S"], s["C"], group=case["G"], Z=s["Z"], act=act)}


def _activated(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    return 0.5 * x * (1 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x))) if act == "gelu" else x


def _rows_of(offsets, n):
    """The expert of every row (E past the last one), its place there, and [E][most] row numbers with their mask."""
    E = offsets.numel() - 1
    r = torch.arange(n, device=offsets.device)
    expert = (r[:, None] >= offsets[None, 1:]).sum(1)
    first = offsets[expert.clamp(max=E - 1)]
    most = max(int((offsets[1:] - offsets[:-1]).max()), 1)
    table = offsets[:-1, None] + torch.arange(most, device=offsets.device)
    return expert.clamp(max=E - 1), r - first, table.clamp(max=n - 1), table < offsets[1:, None]


def _products(A, offsets, W):
    """A[r] . W[e(r)] in 32 bits: every expert's rows padded to the longest, one batched product, the rows back."""
    expert, place, table, inside = _rows_of(offsets, A.shape[0])
    padded = A.float()[table] * inside[..., None]
    return torch.bmm(padded, W)[expert, place.clamp(max=table.shape[1] - 1)]


def _dense(case, Q, S, Z):
    """The 4-bit weights [..., N, K] in 32 bits."""
    codes = torch.stack([Q & 15, Q >> 4], dim=-1).flatten(-2)[..., :case["K"]].float()
    rep = lambda x: x.float().repeat_interleave(case["G"], dim=-1)[..., :case["K"]]  # noqa: E731
    return rep(S) * (codes - (8.0 if Z is None else rep(Z)))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        ids, E = s["ids"], case["E"]
        flat = ids.reshape(-1).long()
        key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
        by = torch.argsort(key, stable=True)
        in_order = key[by]
        r = torch.arange(flat.numel(), device=flat.device)
        offsets = torch.searchsorted(in_order, torch.arange(E + 1, device=flat.device))
        pos = torch.empty_like(flat)
        pos[by] = torch.where(in_order < E, r, -1)
        return {"offsets": offsets.int(), "order": torch.where(in_order < E, by, -1).int(), "pos": pos.reshape(ids.shape).int()}
    if op == "gather":
        rows = s["X"][torch.div(s["order"].clamp(min=0), case["k"], rounding_mode="floor")]
        return {"Xs": torch.where((s["order"] >= 0)[:, None], rows, torch.zeros_like(rows))}
    if op in ("combine", "combine_grad"):
        kept = (s["pos"] >= 0)[..., None]
        rows = torch.where(kept, s["Ys"][s["pos"].clamp(min=0)].float(), 0.0)
        w = kept.float() if s["w"] is None else s["w"].float()[..., None]
        if op == "combine":
            return {"Y": (w * rows).sum(1).to(s["Ys"].dtype)}
        dY = s["Y"].float()[:, None]
        n = s["Ys"].shape[0]
        buffer = torch.zeros(n + 1, case["H"], device=dY.device)
        buffer[torch.where(s["pos"] < 0, n, s["pos"])] = w * dY
        return {"dYs": buffer[:n].to(s["Ys"].dtype), "dw": (rows * dY).sum(-1).to(s["w"].dtype)}
    out = TYPES[case["out"]]
    if op == "experts":
        return {"C": _activated(_products(s["A"], s["offsets"], s["W"].float()), case["act"]).to(out)}
    if op == "experts_dx":
        return {"dA": _products(s["D"], s["offsets"], s["W"].float().transpose(1, 2).contiguous()).to(out)}
    if op == "experts_dw":
        _, _, table, inside = _rows_of(s["offsets"], s["A"].shape[0])
        padded = (s["A"].float()[table] * inside[..., None]).transpose(1, 2).contiguous()
        return {"dW": torch.bmm(padded, s["D"].float()[table] * inside[..., None]).to(out)}
    W = _dense(case, s["Q"], s["S"], s["Z"]).transpose(-1, -2).contiguous()
    product = s["A"].float() @ W if op == "w4" else _products(s["A"], s["offsets"], W)
    return {"C": _activated(product, case["act"]).to(out)}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op in ("w4", "w4_experts"):
        rows = case["M"] if op == "w4" else case["T"] * case["k"]
        used = 1 if op == "w4" else min(case["E"], rows)
        K, N, groups = case["K"], case["N"], -(-case["K"] // case["G"])
        weights = N * ((K + 1) // 2) + N * groups * (SIZE[case["st"]] + (1 if case["zeros"] else 0))
        return {"bytes": used * weights + rows * (K * SIZE[case["t"]] + N * SIZE[case["out"]]), "flops": 2 * rows * K * N}
    n = case["T"] * case["k"]
    if op == "sort":
        return {"bytes": n * (SIZE[case["ids"]] + 8) + 4 * (case["E"] + 1), "flops": n}
    if op in ("gather", "combine", "combine_grad"):
        row = case["H"] * SIZE[case["t"]]
        kept = int(n * (1 - case["drop"]))
        w = 0 if case.get("wt", "none") == "none" else n * SIZE[case["wt"]]
        if op == "gather":
            return {"bytes": (case["T"] + kept) * row + 4 * n, "flops": 0}
        if op == "combine":
            return {"bytes": (case["T"] + kept) * row + 4 * n + w, "flops": 2 * kept * case["H"]}
        return {"bytes": (case["T"] + 2 * kept) * row + 4 * n + 2 * w, "flops": 3 * kept * case["H"]}
    K, N, t, o = case["K"], case["N"], SIZE[case["t"]], SIZE[case["out"]]
    weights = K * N * min(case["E"], n)
    moved = {"experts": t * (weights + n * K) + o * n * N, "experts_dx": t * (weights + n * N) + o * n * K,
             "experts_dw": t * n * (K + N) + o * K * N * case["E"]}[op]
    return {"bytes": moved, "flops": 2 * n * K * N}


# ------------------------------------------------------------------ the values in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "sort":
        offsets, order, pos = _sorted(s["ids"], case["E"])
        return {"offsets": offsets, "order": order, "pos": pos}
    if op == "gather":
        out = torch.zeros_like(s["Xs"], dtype=torch.float64)
        kept = torch.nonzero(s["order"] >= 0)[:, 0]
        out[kept] = s["X"].double()[s["order"][kept].long() // case["k"]]
        return {"Xs": out}
    if op in ("combine", "combine_grad"):
        t, j = torch.nonzero(s["pos"] >= 0, as_tuple=True)
        r = s["pos"][t, j].long()
        w = torch.ones(len(t), device=DEV, dtype=torch.float64) if s["w"] is None else s["w"].double()[t, j]
        if op == "combine":
            y = torch.zeros(s["Y"].shape, device=DEV, dtype=torch.float64)
            return {"Y": y.index_add_(0, t, s["Ys"].double()[r] * w[:, None])}
        dYs = torch.zeros(s["Ys"].shape, device=DEV, dtype=torch.float64)
        dYs[r] = s["Y"].double()[t] * w[:, None]
        dw = torch.zeros(s["pos"].shape, device=DEV, dtype=torch.float64)
        dw[t, j] = torch.linalg.vecdot(s["Y"].double()[t], s["Ys"].double()[r])
        return {"dYs": dYs, "dw": dw}
    C = torch.zeros(s["C"].shape, device=DEV, dtype=torch.float64)
    bounds = [0, case["M"]] if op == "w4" else s["offsets"].tolist()
    for e in range(len(bounds) - 1):
        rows = slice(bounds[e], bounds[e + 1])
        if op == "experts_dw":
            C[e] = s["A"][rows].double().t() @ s["D"][rows].double()
            continue
        if op == "experts":
            W = s["W"][e].double()
        elif op == "experts_dx":
            W = s["W"][e].double().t()
        else:
            Q, S, Z = (x if x is None or op == "w4" else x[e] for x in (s["Q"], s["S"], s["Z"]))
            k = torch.arange(case["K"], device=DEV)
            q = ((Q[:, k // 2].int() >> (4 * (k % 2))) & 15).double()
            z = 8.0 if Z is None else Z.double()[:, k // case["G"]]
            W = (S.double()[:, k // case["G"]] * (q - z)).t()
        C[rows] = (s["A"] if op != "experts_dx" else s["D"])[rows].double() @ W
    if case["act"] == "relu":
        C = torch.clamp(C, min=0)
    elif case["act"] == "gelu":
        C = C * torch.sigmoid(2 * 0.7978845608028654 * (C + 0.044715 * C ** 3))
    return {{"experts": "C", "experts_dx": "dA", "experts_dw": "dW"}.get(op, "C"): C}
