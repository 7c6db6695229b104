"""Performance cases of the router's balance loss (per-expert counts, loss, gradient) and of the experts' 4-bit weights
with group scales (quantisation, and the product with 16-bit activations for few rows).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library's
entry points.  Inputs come from the case and a seed alone.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "ue8m0": 1}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
CLAMP, ALPHA, UP_BIAS = 7.0, 1.702, 1.0  # the parameterised SwiGLU's


# ---------------------------------------------------------------------------------------
# cases

def _router(name, op, tokens, experts, topk, dtype, seqs=1, padded=False, score="softmax", z=False, add=False):
    """add: the gradient is added to that of the routing weights"""
    c = {"name": name, "op": op, "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype, "seqs": seqs,
         "padded": padded, "score": score, "z": z}
    return dict(c, add=add) if op == "balance_grad" else c


def _weights(name, rows, k, group, dtype, scale, zeros):
    return {"name": name, "op": "quantize", "rows": rows, "k": k, "group": group, "dtype": dtype, "scale": scale,
            "zeros": zeros}


def _product(name, rows, used, experts, n, k, group, form, scale, zeros, dtype, out, act="none", zipf=0.0):
    return {"name": name, "op": "product", "rows": rows, "used": used, "experts": experts, "n": n, "k": k,
            "group": group, "form": form, "scale": scale, "zeros": zeros, "dtype": dtype, "out": out, "act": act,
            "zipf": zipf}


def listed():
    return [
        # a micro-batch of a small model's router
        _router("balance_small", "balance", 128, 32, 4, "f32"),
        # a training step of 65536 tokens, 256 experts, with the logits' squared log-sum as a second loss
        _router("balance_train", "balance", 65536, 256, 8, "f32", z=True),
        # packed sequences of uneven lengths with padding, a balance loss for each, sigmoid scores, an odd expert count
        _router("balance_sequences", "balance", 16385, 129, 6, "bf16", seqs=24, padded=True, score="sigmoid"),
        # the gradient of a small step in float16, three sequences
        _router("balance_grad_small", "balance_grad", 500, 60, 4, "f16", seqs=3, padded=True),
        # the gradient of the large step, added to the one that the routing weights already have
        _router("balance_grad_train", "balance_grad", 65536, 256, 8, "f32", z=True, add=True),
        # one projection of a small expert, an odd number of rows, groups of 32
        _weights("quantize_projection", 1027, 2080, 32, "bf16", "bf16", False),
        # float32 master weights of four experts (4096 x 7168 each) for serving, with zero points
        _weights("quantize_experts", 16384, 7168, 128, "f32", "bf16", True),
        # one token through one expert's projection
        _product("product_one_token", 1, 1, 1, 4096, 7168, 128, "int4", "bf16", True, "bf16", "bf16"),
        # a decoding step's rows through 32 experts' gate and up projections, the activation applied
        _product("product_decode_up", 256, 128, 32, 2048, 7168, 128, "int4", "bf16", True, "bf16", "bf16", act="swiglu"),
        # the same rows through the down projections, the weights in the layer's own MXFP4
        _product("product_decode_down", 256, 128, 32, 7168, 2048, 32, "mxfp4", "ue8m0", False, "bf16", "f32"),
        # odd sizes: few uneven rows, groups of 32, float16 with float32 scales, the parameterised activation
        _product("product_odd", 40, 37, 5, 1027, 2080, 32, "int4", "f32", False, "f16", "f32", act="swigluoai", zipf=0.8),
        # a larger batch, about 64 rows for each of 32 experts
        _product("product_batch", 2048, 2000, 32, 4096, 4096, 64, "int4", "f16", False, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance", "balance_grad", "balance_grad", "quantize", "product", "product", "product"])
    if op in ("balance", "balance_grad"):
        experts = _log(rng, 2, 512)
        tokens = max(1, min(_log(rng, 1, 65536), 65536 * 256 // experts))
        c = _router("", op, tokens, experts, rng.randint(1, min(8, experts)), rng.choice(["f32", "f32", "bf16", "f16"]),
                    seqs=rng.choice([1, 1, _log(rng, 1, min(64, tokens))]), padded=rng.random() < 0.5,
                    score=rng.choice(["softmax", "softmax", "sigmoid"]), add=rng.random() < 0.5)
        c["z"] = c["score"] == "softmax" and rng.random() < 0.5
    elif op == "quantize":
        group = rng.choice([32, 64, 128, 128, 256])
        k = group * _log(rng, 1, 8192 // group)
        c = _weights("", min(_log(rng, 1, 40000), 16384 * 7168 // k), k, group, rng.choice(["bf16", "f16", "f32"]),
                     rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5)
    else:
        form = rng.choice(["int4", "int4", "mxfp4"])
        group = 32 if form == "mxfp4" else rng.choice([32, 64, 128, 128, 256])
        act = rng.choice(["none", "none", "swiglu", "swigluoai"])
        experts, k = _log(rng, 1, 64), group * _log(rng, 1, 8192 // group)
        n = max(1, min(_log(rng, 1, 8192), 32 * 4096 * 7168 // (experts * k * (1 if act == "none" else 2))))
        most = max(1, 2 * 2000 * 4096 * 4096 // (n * k * (1 if act == "none" else 2)))  # operations of the largest listed case
        rows = min(_log(rng, 1, 64 * experts), most)
        c = _product("", rows, rng.randint(max(1, rows - rows // 4), rows), experts, n, k, group, form,
                     "ue8m0" if form == "mxfp4" else rng.choice(["bf16", "f16", "f32"]),
                     form == "int4" and rng.random() < 0.5, rng.choice(["bf16", "bf16", "f16"]),
                     rng.choice(["bf16", "f16", "f32"]), act=act, zipf=rng.choice([0.0, 0.0, 0.8]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# inputs

def _sizes(case, seed):
    """Rows of each expert: a multinomial over even or Zipf shares, the experts in a random order."""
    r = np.random.RandomState(seed % (1 << 31))
    p = np.arange(1, case["experts"] + 1, dtype=np.float64) ** -case["zipf"]
    return r.multinomial(case["used"], r.permutation(p / p.sum()))


def _ends(case, seed):
    """Where sequences of uneven lengths end, one after the other; some tokens belong to none where there is padding."""
    r = np.random.RandomState(seed % (1 << 31))
    last = case["tokens"] - (case["tokens"] // 16 if case["padded"] else 0)
    cuts = np.sort(r.randint(0, last + 1, case["seqs"] - 1))
    return np.concatenate([[0], cuts, [last]]).astype(np.int32)


def _plan(case):
    """The descriptor (and the workspace) that a program keeps for its sizes."""
    from moe_expert_layer_amd import binding as B
    op = case["op"]
    if op == "quantize":
        return B.make_int4_desc(case["rows"], case["k"], case["group"], dtype=case["dtype"], scale_dtype=case["scale"],
                                zeros=case["zeros"]), None
    if op == "product":
        return B.make_w4_gemm_desc(case["rows"], case["n"], case["k"], groups=case["experts"], weight_format=case["form"],
                                   group_size=case["group"], scale_dtype=case["scale"], zeros=case["zeros"],
                                   dtype=case["dtype"], out_dtype=case["out"],
                                   activation=None if case["act"] == "none" else case["act"], activation_clamp=CLAMP,
                                   activation_alpha=ALPHA, activation_up_bias=UP_BIAS), None
    d = B.make_balance_desc(case["tokens"], case["experts"], case["topk"], num_seqs=case["seqs"], dtype=case["dtype"],
                            score=case["score"])
    return d, B.alloc_balance_workspace(d)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, "plan": _plan(case) if own else None}
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if op in ("balance", "balance_grad"):
        T, E, k, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
        # experts of uneven popularity, as before the loss has evened them out
        logits = (1.5 * normal(T, E) + normal(E)).to(DTYPES[case["dtype"]])
        s["logits"] = logits
        s["ids"] = torch.topk(logits.float(), k, dim=1)[1].to(torch.int32)
        s["mask"] = torch.rand(T, generator=g, device="cuda") < 0.9 if case["padded"] else None
        s["ends"] = torch.from_numpy(_ends(case, seed)).cuda() if S > 1 else None
        if op == "balance":
            s["out"] = {"counts": torch.zeros(S, E, dtype=torch.int32, device="cuda"),
                        "tokens": torch.zeros(S, dtype=torch.int32, device="cuda"),
                        "prob_sums": torch.zeros(S, E, device="cuda"), "balance": torch.zeros(S, device="cuda")}
            if case["z"]:
                s["out"]["z"] = torch.zeros(S, device="cuda")
            return s
        # what the forward pass left: how often each expert was chosen, and by how many tokens
        seq, live = _sequences(s)
        s["counts"], s["tokens"] = _counts(s, seq, live)
        s["dbalance"] = 0.01 * torch.rand(S, generator=g, device="cuda") + 0.005
        s["dz"] = 0.001 * torch.rand(S, generator=g, device="cuda") + 0.0005 if case["z"] else None
        # gradients of the routing weights, of the size that the balance loss's has
        s["add"] = normal(T, E) * (3e-5 / T) if case["add"] else None
        s["dlogits"] = torch.zeros(T, E, device="cuda")
        return s
    K, group = case["k"], case["group"]
    if op == "quantize":
        M, scale = case["rows"], DTYPES[case["scale"]]
        # rows of different magnitude, as a weight's output channels have
        s["v"] = (0.02 * normal(M, K) * torch.exp(0.5 * normal(M, 1))).to(DTYPES[case["dtype"]])
        s["codes"] = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(M, K // group, dtype=scale, device="cuda")
        s["zeros"] = torch.zeros(M, K // group, dtype=torch.uint8, device="cuda") if case["zeros"] else None
        s["out"] = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        return s
    R, E, N = case["rows"], case["experts"], case["n"] * (1 if case["act"] == "none" else 2)
    s["a"] = normal(R, K).to(DTYPES[case["dtype"]])
    s["b"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):  # codes as the quantisation of normal weights leaves them
        v = normal(N, K)
        if case["form"] == "mxfp4":
            q = torch.bucketize(2.0 * v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda"))
            q = q.to(torch.uint8) | (v < 0).to(torch.uint8) << 3
        else:
            q = torch.clamp(torch.round(2.5 * v + 7.5), 0, 15).to(torch.uint8)
        s["b"][e] = q[:, 0::2] | q[:, 1::2] << 4
    if case["form"] == "mxfp4":
        s["scales"] = (119 + 3 * torch.rand(E, N, K // group, generator=g, device="cuda")).to(torch.uint8)
    else:
        s["scales"] = (0.01 * torch.exp(0.3 * normal(E, N, K // group))).to(DTYPES[case["scale"]])
    s["zeros"] = None
    if case["zeros"]:
        s["zeros"] = torch.clamp(torch.round(normal(E, N, K // group) + 7.5), 0, 15).to(torch.uint8)
    sizes = _sizes(case, seed)
    s["most"] = max(1, int(sizes.max()))
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    s["out"] = torch.zeros(R, case["n"], dtype=DTYPES[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from moe_expert_layer_amd import binding as B
    d, ws = s["plan"]
    op = s["case"]["op"]
    if op == "balance":
        o = s["out"]
        B.moe_balance_loss(d, s["logits"], s["ids"], o["counts"], o["tokens"], o["prob_sums"], o["balance"], ws,
                           z=o.get("z"), mask=s["mask"], seq_offsets=s["ends"])
        return o
    if op == "balance_grad":
        B.moe_balance_loss_backward(d, s["logits"], s["counts"], s["tokens"], s["dbalance"], s["dlogits"], dz=s["dz"],
                                    mask=s["mask"], seq_offsets=s["ends"], add=s["add"])
        return {"dlogits": s["dlogits"]}
    if op == "quantize":
        B.moe_quantize_int4(d, s["v"], s["codes"], s["scales"], s["zeros"])
        B.moe_dequantize_int4(d, s["codes"], s["scales"], s["zeros"], s["out"], dtype="bf16")
        return {"scales": s["scales"], "values": s["out"]}
    B.moe_w4_gemm(d, s["a"], s["b"], s["scales"], s["zeros"], s["offsets"], s["out"])
    return {"c": s["out"]}


def _sequences(s):
    """The sequence of each token (0 where it has none) and whether it counts."""
    T = s["logits"].shape[0]
    live = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device="cuda")
    if s["ends"] is None:
        return torch.zeros(T, dtype=torch.int64, device="cuda"), live
    t = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["ends"], t, right=True) - 1
    live = live & (seq < s["case"]["seqs"])
    return torch.where(live, seq, 0), live


def _counts(s, seq, live):
    """How often the tokens of each sequence chose each expert, and how many tokens it has."""
    S, E = s["case"]["seqs"], s["case"]["experts"]
    at = torch.where(live[:, None], seq[:, None] * E + s["ids"], S * E).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device="cuda").scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    tokens = torch.zeros(S, dtype=torch.int32, device="cuda").scatter_add_(0, seq, live.to(torch.int32))
    return counts[:S * E].reshape(S, E), tokens


def _probabilities(s):
    """Each token's probabilities, and its log-sum of exponentials."""
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    if s["case"]["score"] == "sigmoid":
        v = 1 / (1 + torch.exp(-x))
        return v / v.sum(1, keepdim=True), None
    v = torch.exp(x - top)
    n = v.sum(1, keepdim=True)
    return v / n, (top + torch.log(n)).squeeze(1)


def _balance(s):
    c = s["case"]
    seq, live = _sequences(s)
    counts, tokens = _counts(s, seq, live)
    p, lse = _probabilities(s)
    # sums over up to 65536 tokens: in 64 bits, a product with the sequences' members
    member = (torch.arange(c["seqs"], device="cuda")[:, None] == seq) & live
    member = member.double()
    sums = member @ p.double()
    n = tokens.double().clamp(min=1)
    o = {"counts": counts, "tokens": tokens, "prob_sums": sums.float(),
         "balance": ((counts * sums).sum(1) * c["experts"] / (c["topk"] * n * n)).float()}
    if c["z"]:
        o["z"] = ((member @ (lse.double() ** 2)) / n).float()
    return o


def _balance_grad(s):
    c = s["case"]
    seq, live = _sequences(s)
    p, lse = _probabilities(s)
    n = s["tokens"].double().clamp(min=1)
    # the counts differ little from their mean: the difference in 64 bits
    w = s["counts"].double()[seq]
    w = (w - (p.double() * w).sum(1, keepdim=True)).float()
    scale = s["dbalance"].double() * c["experts"] / (c["topk"] * n * n)
    g = p * w * scale[seq].float()[:, None]
    if c["score"] == "sigmoid":
        g = g / (1 + torch.exp(s["logits"].float()))
    if c["z"]:
        g = g + p * (lse * (2 * s["dz"].double() / n)[seq].float())[:, None]
    g = torch.where(live[:, None], g, 0.0)
    return {"dlogits": g if s["add"] is None else s["add"] + g}


def _stored(q, scales, zeros):
    """float32 values of 4-bit codes [M, K / 2] with a scale (and a zero point, else 8) for each group of a row."""
    M, G = scales.shape
    v = torch.stack([q & 15, q >> 4], -1).reshape(M, G, -1)
    if scales.dtype == torch.uint8:  # MXFP4
        table = torch.tensor(E2M1, device="cuda")
        return torch.ldexp(table[v.long()], scales.to(torch.int32)[..., None] - 127).reshape(M, -1)
    v = v.float() - (8.0 if zeros is None else zeros.float()[..., None])
    return (v * scales.float()[..., None]).reshape(M, -1)


def _quantize(s):
    c = s["case"]
    v = s["v"].float().reshape(c["rows"], -1, c["group"])
    if c["zeros"]:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        scale = ((hi.double() - lo.double()) / 15).float().to(DTYPES[c["scale"]])
    else:
        scale = (v.abs().amax(-1) / 7).to(DTYPES[c["scale"]])
    d = scale.double()  # quotients next to a border of two codes: in 64 bits
    d = torch.where(d > 0, d, 1.0)
    zero = torch.round(-lo / d).clamp(0, 15) if c["zeros"] else torch.full_like(d, 8.0)
    q = (torch.round(v / d[..., None]) + zero[..., None]).clamp(0, 15).to(torch.uint8).reshape(c["rows"], -1)
    return {"scales": scale, "values": _stored(q[:, 0::2] | q[:, 1::2] << 4, scale, zero if c["zeros"] else None).to(torch.bfloat16)}


def _product_plain(s):
    """The experts' rows padded to the longest, one batched float32 product, the activation, the rows back in place."""
    c = s["case"]
    R, E, K = c["rows"], c["experts"], c["k"]
    N = s["b"].shape[1]
    a, o = s["a"].float(), s["offsets"].long()
    b = _stored(s["b"].reshape(E * N, -1), s["scales"].reshape(E * N, -1), None if s["zeros"] is None else s["zeros"].reshape(E * N, -1))
    b = b.reshape(E, N, K).transpose(1, 2).contiguous()
    at = o[:-1, None] + torch.arange(s["most"], device="cuda")
    p = torch.where((at < o[1:, None])[..., None], a[at.clamp(max=R - 1)], 0.0)
    p = torch.bmm(p, b)
    if c["act"] != "none":
        gate, up = p[..., :c["n"]], p[..., c["n"]:]
        alpha = 1.0
        if c["act"] == "swigluoai":
            gate, up, alpha = gate.clamp(max=CLAMP), up.clamp(-CLAMP, CLAMP) + UP_BIAS, ALPHA
        p = gate / (1 + torch.exp(-alpha * gate)) * up
    r = torch.arange(R, device="cuda")
    e = (torch.searchsorted(o, r, right=True) - 1).clamp(max=E - 1)
    mine = r < o[-1]
    return {"c": torch.where(mine[:, None], p[e, torch.where(mine, r - o[e], 0)], 0.0).to(s["out"].dtype)}


_PLAIN = {"balance": _balance, "balance_grad": _balance_grad, "quantize": _quantize, "product": _product_plain}


# ---------------------------------------------------------------------------------------
# bytes and operations that a pass cannot do without

def work(case):
    op = case["op"]
    if op == "balance":
        T, E = case["tokens"], case["experts"]
        return {"bytes": T * (E * BYTES[case["dtype"]] + 4 * case["topk"] + case["padded"]) + case["seqs"] * (8 * E + 16),
                "flops": 6.0 * T * E}
    if op == "balance_grad":
        T, E = case["tokens"], case["experts"]
        return {"bytes": T * E * (BYTES[case["dtype"]] + (8 if case["add"] else 4)) + case["seqs"] * (4 * E + 12),
                "flops": 9.0 * T * E}
    groups = case["k"] // case["group"]
    per = case["k"] / 2 + groups * (BYTES[case["scale"]] + case["zeros"])  # a row of weights
    if op == "quantize":
        return {"bytes": case["rows"] * (case["k"] * (BYTES[case["dtype"]] + 2) + per), "flops": 0}
    N = case["n"] * (1 if case["act"] == "none" else 2)
    experts = min(case["experts"], case["used"])  # an expert without rows is not read
    return {"bytes": experts * N * per + case["used"] * (2 * case["k"] + case["n"] * BYTES[case["out"]]),
            "flops": 2.0 * case["used"] * N * case["k"]}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence or expert by expert

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("balance", "balance_grad"):
        T, E, k, S = case["tokens"], case["experts"], case["topk"], case["seqs"]
        ends = [0, T] if S == 1 else s["ends"].tolist()
        mask = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        sums, balance, z = [], [], []
        d = torch.zeros(T, E, dtype=torch.float64, device="cuda") if s.get("add") is None else s["add"].double().clone()
        for i in range(S):
            at = torch.nonzero(mask[ends[i]:ends[i + 1]]).squeeze(1) + ends[i]
            x, n = s["logits"][at].double(), max(1, at.numel())
            lse = torch.logsumexp(x, 1)
            logp = x - lse[:, None]
            if case["score"] == "sigmoid":
                logp = torch.nn.functional.logsigmoid(x)
                logp = logp - torch.logsumexp(logp, 1, keepdim=True)
            p = torch.exp(logp)
            f = torch.bincount(s["ids"][at].long().reshape(-1), minlength=E).double() * (E / (k * n))  # E f_e
            sums.append(p.sum(0))
            balance.append((f * sums[-1]).sum() / n)
            z.append((lse * lse).sum() / n)
            if op == "balance_grad":
                u = s["dbalance"][i].double() / n * f
                gp = p * u - p * (p @ u)[:, None]
                if case["score"] == "sigmoid":
                    gp = gp * torch.sigmoid(-x)
                if case["z"]:
                    gp = gp + s["dz"][i].double() * 2 / n * lse[:, None] * p
                d[at] += gp
        if op == "balance_grad":
            return {"dlogits": d}
        o = {"counts": None, "tokens": None, "prob_sums": torch.stack(sums), "balance": torch.stack(balance)}
        return dict(o, z=torch.stack(z)) if case["z"] else o
    if op == "quantize":
        # a group spans 15 steps of its scale, from its smallest to its largest value, or 7 to either side of zero
        v = s["v"].double().reshape(case["rows"], -1, case["group"])
        if case["zeros"]:
            low = torch.minimum(v.min(-1)[0], torch.zeros((), dtype=torch.float64, device="cuda"))
            span = torch.maximum(v.max(-1)[0], torch.zeros((), dtype=torch.float64, device="cuda")) - low
            step = (span / 15).float().to(DTYPES[case["scale"]]).double()
            first = -torch.round(-low / step.clamp(min=1e-300)).clamp(0, 15)
        else:
            step = (torch.maximum(v.max(-1)[0], -v.min(-1)[0]) / 7).float().to(DTYPES[case["scale"]]).double()
            first = torch.full_like(step, -8.0)
        n = torch.round(v / step.clamp(min=1e-300)[..., None])
        n = torch.maximum(torch.minimum(n, first[..., None] + 15), first[..., None])
        return {"scales": step, "values": (n * step[..., None]).reshape(case["rows"], case["k"])}
    o = s["offsets"].tolist()
    out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        if o[e + 1] == o[e]:
            continue
        byte, step = s["b"][e].long(), s["scales"][e].double()
        w = torch.empty(byte.shape[0], case["k"], dtype=torch.float64, device="cuda")
        for half in (0, 1):
            code = (byte >> (4 * half)) & 15
            if case["form"] == "mxfp4":
                w[:, half::2] = table[code]
            elif s["zeros"] is None:
                w[:, half::2] = code.double() - 8
            else:
                w[:, half::2] = code.double() - s["zeros"][e].double().repeat_interleave(case["group"] // 2, 1)
        w *= (torch.exp2(step - 127) if case["form"] == "mxfp4" else step).repeat_interleave(case["group"], 1)
        y = s["a"][o[e]:o[e + 1]].double() @ w.t().contiguous()
        if case["act"] != "none":
            gate, up = y.chunk(2, 1)
            if case["act"] == "swigluoai":
                gate, up = torch.clamp(gate, max=CLAMP), torch.clamp(up, -CLAMP, CLAMP)
                y = gate * torch.sigmoid(ALPHA * gate) * (up + UP_BIAS)
            else:
                y = torch.nn.functional.silu(gate) * up
        out[o[e]:o[e + 1]] = y
    return {"c": out}
