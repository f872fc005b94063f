"""What the scoring operators of the head are measured on: their cases, their plain forms and their exact values.

q4_pack                  4-bit codes and group scales of a head's weights, and the weights that they stand for
q4_scores                the scores of a few queries against a head held in 4 bits
score_logprobs           log probabilities of given labels, log-sum-exp, entropy and the k best labels of rows of scores
score_logprobs_backward  the gradient of those log probabilities, log-sum-exps and entropies with regard to the scores
label_logprobs           the same statistics straight from the head, without the scores ever being stored
"""
import math

import torch

own = False

BF16, FP32, E4M3, E5M2 = "bf16", "fp32", "e4m3", "e5m2"
_TYPES = {BF16: torch.bfloat16, FP32: torch.float32, E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
_MOST = {"pack": 500_000 * 768, "q4": 3_000_000 * 768, "scores": 256 * 500_000, "label": 256 * 3_000_000 * 768}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a small head's copy, made again whenever the head has moved a little: the launch counts
        {"name": "pack_tiny_e4m3", "op": "q4_pack", "L": 4096, "d": 64, "group": 32, "w": E4M3},
        # the whole 500K-label head of the text-tagging workload, laid out once for serving
        {"name": "pack_text500k_bf16", "op": "q4_pack", "L": 500_000, "d": 768, "group": 64, "w": BF16},
        # one query against a small head
        {"name": "q4_one_tiny", "op": "q4_scores", "L": 4096, "d": 64, "group": 32, "B": 1, "pad": 0},
        # one query against the 3M-label product head: the time is that of reading the head
        {"name": "q4_one_3m", "op": "q4_scores", "L": 3_000_000, "d": 768, "group": 64, "B": 1, "pad": 0},
        # a handful of queries, an odd number of labels, rows of scores with a pitch
        {"name": "q4_odd_500k", "op": "q4_scores", "L": 500_001, "d": 768, "group": 128, "B": 7, "pad": 3},
        # one query's scores over 3M labels: few rows, a long axis
        {"name": "lp_one_3m_fp32", "op": "score_logprobs", "L": 3_000_000, "B": 1, "z": FP32, "pad": 0, "lam": 35, "k": 5, "masked": 0.0},
        # an evaluation batch of the text-tagging workload, some labels masked out
        {"name": "lp_text500k_bf16", "op": "score_logprobs", "L": 500_000, "B": 256, "z": BF16, "pad": 0, "lam": 4, "k": 10, "masked": 0.1},
        # few labels, an odd number of them, a pitch that keeps rows off 16 bytes, the longest lists
        {"name": "lp_odd_4k_fp32", "op": "score_logprobs", "L": 4099, "B": 33, "z": FP32, "pad": 2, "lam": 5, "k": 64, "masked": 0.0},
        # the gradient of the same evaluation batch's scores
        {"name": "bwd_text500k_bf16", "op": "score_logprobs_backward", "L": 500_000, "B": 256, "z": BF16, "pad": 0, "lam": 4, "masked": 0.1},
        {"name": "bwd_odd_4k_fp32", "op": "score_logprobs_backward", "L": 4099, "B": 33, "z": FP32, "pad": 2, "lam": 5, "masked": 0.0},
        # a training-sized batch against the whole 3M-label product head
        {"name": "label_3m_e4m3", "op": "label_logprobs", "L": 3_000_000, "d": 768, "w": E4M3, "B": 256, "lam": 35, "k": 5},
        # a few served queries against the 500K-label head
        {"name": "label_serve_bf16", "op": "label_logprobs", "L": 500_000, "d": 768, "w": BF16, "B": 4, "lam": 4, "k": 5},
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["q4_pack", "q4_scores", "score_logprobs", "score_logprobs_backward", "label_logprobs"])
    lam = rng.choice([1, 4, 10, 35])
    if op == "q4_pack":
        d = 64 * rng.randint(1, 16)
        group = rng.choice([g for g in (32, 64, 128) if d % g == 0])
        return {"op": op, "L": _between(rng, 1000, _MOST["pack"] // d), "d": d, "group": group, "w": rng.choice([BF16, E4M3, E5M2])}
    if op == "q4_scores":
        d = 64 * rng.randint(1, 16)
        group = rng.choice([g for g in (32, 64, 128) if d % g == 0])
        B = _between(rng, 1, 64)
        most = min(_MOST["q4"] // d, 3_000_000 * 16 // B)
        return {"op": op, "L": _between(rng, 1000, most), "d": d, "group": group, "B": B, "pad": rng.choice([0, 0, 1, 4])}
    if op == "label_logprobs":
        d = 64 * rng.randint(1, 16)
        B = _between(rng, 1, 256)
        L = _between(rng, 1000, min(3_000_000, _MOST["label"] // (d * B)))
        return {"op": op, "L": L, "d": d, "w": rng.choice([BF16, E4M3, E5M2]), "B": B, "lam": lam, "k": rng.choice([1, 5, 10, 64])}
    B = _between(rng, 1, 512)
    case = {"op": op, "L": _between(rng, 100, min(3_000_000, _MOST["scores"] // B)), "B": B, "z": rng.choice([FP32, BF16]),
            "pad": rng.choice([0, 0, 1, 8]), "lam": lam, "masked": rng.choice([0.0, 0.1, 0.9])}
    if op == "score_logprobs":
        case["k"] = rng.choice([0, 1, 5, 10, 64])
    return case


# ---------------------------------------------------------------- inputs
def _labels(case, seed):
    """CSR label lists: 1 + lam labels a row on average, some of them twice, some rows without any."""
    g = torch.Generator().manual_seed(seed + 7)
    owner = torch.randint(0, case["B"], (case["B"] * (1 + case["lam"]),), generator=g)
    rowptr = torch.zeros(case["B"] + 1, dtype=torch.int32)
    rowptr[1:] = torch.cumsum(torch.bincount(owner, minlength=case["B"]), 0)
    cols = torch.randint(0, case["L"], (int(rowptr[-1]),), generator=g, dtype=torch.int32)
    return rowptr.cuda(), cols.cuda()


def _weights(case, g):
    """N(0, 0.02^2) on the head's grid."""
    return torch.randn(case["L"], case["d"], generator=g, device="cuda").mul_(0.02).to(_TYPES[case["w"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, L = case["op"], case["L"]
    s = {"case": case}
    if op == "q4_pack":
        s["W"] = _weights(case, g)
        s["codes"] = torch.empty(L, case["d"] // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(L, case["d"] // case["group"], dtype=torch.bfloat16, device="cuda")
        s["values"] = torch.empty(L, case["d"], dtype=torch.bfloat16, device="cuda")
    elif op == "q4_scores":
        s["codes"], s["scales"] = _quantised(_weights({**case, "w": BF16}, g), case["group"])
        s["X"] = torch.randn(case["B"], case["d"], generator=g, device="cuda").to(torch.bfloat16)
        s["Z"] = torch.empty(case["B"], L + case["pad"], device="cuda")[:, :L]
    elif op == "label_logprobs":
        s["W"] = _weights(case, g)
        s["X"] = torch.randn(case["B"], case["d"], generator=g, device="cuda").to(torch.bfloat16)
        s["rowptr"], s["cols"] = _labels(case, seed)
        _outputs(s, case)
    else:
        s["rowptr"], s["cols"] = _labels(case, seed)
        Z = torch.randn(case["B"], L + case["pad"], generator=g, device="cuda").mul_(2).to(_TYPES[case["z"]])
        if case["masked"]:
            hidden = torch.rand(Z.shape, generator=g, device="cuda") < case["masked"]
            hidden[case["B"] // 2] |= case["B"] > 2      # a row with no label left, as padding leaves one
            Z.masked_fill_(hidden, -math.inf)
        s["Z"] = Z[:, :L]
        if op == "score_logprobs":
            _outputs(s, case)
        else:
            rows = torch.randn(3, case["B"], generator=g, device="cuda")
            s["g_logp"] = torch.randn(s["cols"].numel(), generator=g, device="cuda")
            s["g_lse"], s["g_entropy"] = rows[0], rows[1]
            s["lse"], s["entropy"] = _statistics(s["Z"].float())[:2]
            s["dZ"] = torch.empty_like(Z)[:, :L]
    return s


def _outputs(s, case):
    s["logp"] = torch.empty(s["cols"].numel(), device="cuda")
    s["lse"], s["entropy"] = torch.empty(2, case["B"], device="cuda").unbind(0)
    s["idx"] = torch.empty(case["B"], min(case["k"], case["L"]), dtype=torch.int32, device="cuda")
    s["top"] = torch.empty(case["B"], min(case["k"], case["L"]), device="cuda")


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "q4_pack":
        codes, scales = _quantised(s["W"], s["case"]["group"])
        return {"scales": scales, "values": _dequantised(codes, scales).to(torch.bfloat16)}
    if op == "q4_scores":
        return {"Z": s["X"].float() @ _dequantised(s["codes"], s["scales"]).T}
    if op == "score_logprobs":
        return _scored(s["Z"].float(), s["rowptr"], s["cols"], s["idx"].shape[1])
    if op == "score_logprobs_backward":
        return _backward(s)
    # the order of the best labels has to be that of the exact scores: in 64 bits
    return _scored(s["X"].double() @ s["W"].double().T, s["rowptr"], s["cols"], s["idx"].shape[1])


def _own(s, op):
    import precision_label_chunk_b200 as elmo
    if op == "q4_pack":
        elmo.elmo_q4_pack(s["W"], s["case"]["w"], s["case"]["group"], s["codes"], s["scales"])
        elmo.elmo_q4_unpack(s["codes"], s["scales"], s["values"])
        return {"scales": s["scales"], "values": s["values"]}
    if op == "q4_scores":
        elmo.elmo_q4_scores(s["codes"], s["scales"], s["X"], s["Z"])
        return {"Z": s["Z"]}
    if op == "score_logprobs_backward":
        elmo.elmo_score_logprobs_backward(s["Z"], s["rowptr"], s["cols"], s["lse"], s["entropy"], s["g_logp"], s["g_lse"],
                                          s["g_entropy"], s["dZ"])
        return {"dZ": s["dZ"]}
    out = {n: s[n] for n in ("logp", "lse", "entropy", "idx", "top")}
    if op == "score_logprobs":
        if "work" not in s:
            n = elmo.elmo_score_logprobs_workspace_bytes(s["Z"].shape[0], s["Z"].shape[1], s["idx"].shape[1])
            s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        elmo.elmo_score_logprobs(s["Z"], s["rowptr"], s["cols"], s["logp"], s["lse"], s["entropy"], s["idx"], s["top"], s["work"])
    else:
        if "head" not in s:
            s["head"] = elmo.elmo_init_head(s["W"], s["case"]["w"])
        elmo.elmo_label_logprobs(s["head"], s["X"], s["rowptr"], s["cols"], s["logp"], s["lse"], s["entropy"], s["idx"], s["top"])
    return out


# ---------------------------------------------------------------- plain forms
def _quantised(W, group):
    """Codes (two a byte, the even element low, code c for c - 8) and bf16 scales of groups along a row: the scale is
    a seventh of the group's largest magnitude, the code the nearest whole number of scales, ties to even."""
    w = W.float().view(W.shape[0], -1, group)
    scales = (w.abs().amax(2) / 7).to(torch.bfloat16)
    by = scales.float().unsqueeze(2)
    q = torch.where(by > 0, torch.round(w / by), torch.zeros_like(w)).clamp_(-8, 7)
    q = (q + 8).to(torch.uint8).view(W.shape[0], -1)
    return q[:, 0::2] | (q[:, 1::2] << 4), scales


def _dequantised(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], scales.shape[1], -1)
    return ((q.float() - 8) * scales.float().unsqueeze(2)).view(codes.shape[0], -1)


def _statistics(Z):
    """lse, entropy and log sum exp's parts of each row; a row with nothing left has lse -inf and entropy 0."""
    m = Z.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(Z - m)
    s = e.sum(1)
    t = torch.where(e > 0, e * (Z - m), torch.zeros_like(e)).sum(1)
    logs = torch.log(s)
    entropy = torch.where(s > 0, logs - t / s, torch.zeros_like(s))
    return m[:, 0] + logs, entropy, m[:, 0], logs


def _rows_of(rowptr, n):
    return torch.bucketize(torch.arange(n, device=rowptr.device), rowptr[1:], right=True)


def _scored(Z, rowptr, cols, k):
    lse, entropy, m, logs = _statistics(Z)
    r = _rows_of(rowptr, cols.numel())
    logp = Z[r, cols.long()]
    logp = torch.where(torch.isinf(logp), logp, logp - m[r] - logs[r])
    if Z.dtype == torch.float64:
        top, idx = torch.topk(Z, k, dim=1)
    else:
        # equal scores go to the lowest label: (score's order, label) as one whole number
        key = (Z + 0.0).view(torch.int32)
        key = torch.where(key < 0, key ^ 0x7FFFFFFF, key).long() << 24
        key += (1 << 24) - 1 - torch.arange(Z.shape[1], device=Z.device)
        idx = (1 << 24) - 1 - (torch.topk(key, k, dim=1).values & ((1 << 24) - 1))
        top = torch.gather(Z, 1, idx)
    none = top == -math.inf
    top = torch.where(none, top, top - m[:, None] - logs[:, None])
    return {"logp": logp.float(), "lse": lse.float(), "entropy": entropy.float(), "idx": torch.where(none, -1, idx).int(),
            "top": top.float()}


def _backward(s):
    Z = s["Z"].float()
    lse = s["lse"][:, None]
    logp = torch.where(torch.isinf(lse), -math.inf, Z - lse)
    p = torch.exp(logp)
    r = _rows_of(s["rowptr"], s["cols"].numel())
    each = s["g_lse"].index_add(0, r, s["g_logp"], alpha=-1)[:, None]
    spread = torch.where(p > 0, p * (each - s["g_entropy"][:, None] * (logp + s["entropy"][:, None])), 0.0)
    dZ = spread.index_put((r, s["cols"].long()), s["g_logp"], accumulate=True)
    dZ = torch.where(torch.isinf(lse), 0.0, dZ)          # a row with nothing left has no gradient
    return {"dZ": dZ.to(s["Z"].dtype)}


# ---------------------------------------------------------------- the work of one pass
def work(case):
    op, L, B, d, k = case["op"], case["L"], case.get("B", 1), case.get("d", 0), case.get("k", 0)
    nnz = B * (1 + case.get("lam", 0))
    lists = nnz * 8 + (B + 1) * 4 + B * (8 + 8 * k)
    if op == "q4_pack":
        packed = L * d // 2 + 2 * L * d // case["group"]
        return {"bytes": L * d * (2 if case["w"] == BF16 else 1) + packed + 2 * L * d, "flops": 4 * L * d}
    if op == "q4_scores":
        return {"bytes": L * d // 2 + 2 * L * d // case["group"] + 2 * B * d + 4 * B * L, "flops": 2 * B * L * d}
    if op == "label_logprobs":
        return {"bytes": L * d * (2 if case["w"] == BF16 else 1) + 2 * B * d + lists, "flops": 2 * B * L * d + 6 * B * L}
    size = 2 if case["z"] == BF16 else 4
    if op == "score_logprobs":
        return {"bytes": B * L * size + lists, "flops": 6 * B * L}
    return {"bytes": 2 * B * L * size + lists, "flops": 8 * B * L}


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    op, L = case["op"], case["L"]
    if op == "q4_pack":
        # the scale is what the format rounds: given it, each value is a whole number of scales
        W = s["W"].double()
        big = torch.stack([W[:, a:a + case["group"]].abs().amax(1) for a in range(0, case["d"], case["group"])], 1)
        scale = (big.float() / 7).bfloat16()
        step = scale.double().repeat_interleave(case["group"], 1)
        values = torch.nan_to_num(torch.round(W / step)).clamp(-8, 7) * step
        return {"scales": scale.double(), "values": values}
    if op == "q4_scores":
        out, X = torch.empty(case["B"], L, dtype=torch.float64, device="cuda"), s["X"].double()
        for a in range(0, L, 1 << 18):
            c = s["codes"][a:a + (1 << 18)]
            w = torch.empty(c.shape[0], case["d"], dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = (c % 16).double() - 8, (c // 16).double() - 8
            w *= s["scales"][a:a + (1 << 18)].double().repeat_interleave(case["group"], 1)
            out[:, a:a + (1 << 18)] = torch.mm(X, w.t())
        return {"Z": out}
    ptr = s["rowptr"].tolist()
    owner = torch.tensor([b for b in range(case["B"]) for _ in range(ptr[b + 1] - ptr[b])], device="cuda")
    if op == "score_logprobs_backward":
        # rows one after another: the definition's sums over the labels, with nothing shared with the plain form
        out = torch.zeros(case["B"], L, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            lse = float(s["lse"][b])
            if math.isinf(lse):
                continue
            given, ids = s["g_logp"][ptr[b]:ptr[b + 1]].double(), s["cols"][ptr[b]:ptr[b + 1]].long()
            logs = (s["Z"][b].double() - lse).clamp(min=-1e4)
            p = logs.exp()
            out[b] = p * (float(s["g_lse"][b]) - given.sum() - float(s["g_entropy"][b]) * (logs + float(s["entropy"][b])))
            out[b].scatter_add_(0, ids, given)
        return {"dZ": out}
    if op == "label_logprobs":
        X = s["X"].double()
        Z = torch.cat([torch.mm(X, s["W"][a:a + (1 << 18)].double().t()) for a in range(0, L, 1 << 18)], 1)
    else:
        Z = s["Z"]
    lse = torch.stack([torch.logsumexp(Z[b].double(), 0) for b in range(case["B"])])
    entropy = torch.stack([-torch.special.xlogy(p, p).sum() for b in range(case["B"])
                           for p in [torch.exp(Z[b].double() - (lse[b] if math.isfinite(lse[b]) else 0.0))]])
    given = Z[owner, s["cols"].long()].double()
    logp = torch.where(torch.isinf(given), given, given - lse[owner])
    best = torch.stack([torch.sort(Z[b].double(), descending=True, stable=True).values[:s["idx"].shape[1]] for b in range(case["B"])])
    top = torch.where(torch.isinf(best), best, best - lse[:, None])
    return {"logp": logp, "lse": lse, "entropy": entropy, "idx": None, "top": top}
