"""Performance cases of the operators beside the expert layer: tokens sorted by expert and brought
back with their routing weights (each with its gradient), and microscaled 4-bit floating point
(quantisation and the grouped product).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library's
entry points.  Inputs come from the case and a seed alone.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------
# cases

def _route(name, op, tokens, hidden, experts, local, topk, dtype, rows, zipf=0.0, first=0):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "experts": experts, "first": first,
            "local": local, "topk": topk, "dtype": dtype, "rows": rows, "zipf": zipf}


def _product(name, rows, used, groups, n, k, out, zipf=0.0):
    return {"name": name, "op": "product", "rows": rows, "used": used, "groups": groups, "n": n, "k": k, "out": out,
            "zipf": zipf}


def listed():
    return [
        # one decoding step of 128 requests on a GPU that holds 32 of 256 experts: its tokens in expert order
        _route("dispatch_decode", "dispatch", 128, 7168, 256, 32, 8, "bf16", 512),
        # a prefill chunk of 4096 tokens whose experts are unevenly popular
        _route("dispatch_prefill", "dispatch", 4096, 7168, 256, 32, 8, "bf16", 8192, zipf=1.1, first=64),
        # the tokens' gradient in a float32 training step of a small model, every expert on this GPU, odd sizes
        _route("dispatch_grad_f32", "dispatch_grad", 4097, 2050, 32, 32, 4, "f32", 4097 * 4),
        # one token of one request, all of its experts on this GPU
        _route("combine_one_token", "combine", 1, 7168, 256, 256, 8, "bf16", 8),
        # a large prefill batch: the share of 32 of 256 experts brought back into token order
        _route("combine_batch", "combine", 32768, 7168, 256, 32, 8, "bf16", 40000),
        # a small training step in float16, every expert on this GPU
        _route("combine_grad_small", "combine_grad", 512, 2048, 32, 32, 4, "f16", 2048),
        # a training step of 16384 tokens in bfloat16, eight experts of 64 a token
        _route("combine_grad_train", "combine_grad", 16384, 4096, 64, 64, 8, "bf16", 16384 * 8),
        # the activations of a decoding step, an odd number of rows
        {"name": "quantize_tokens", "op": "quantize", "rows": 129, "k": 7168, "dtype": "bf16"},
        # float32 master weights of four experts (4096 x 7168 each) for serving
        {"name": "quantize_weights", "op": "quantize", "rows": 16384, "k": 7168, "dtype": "f32"},
        # one token through one linear layer with an odd width, float32 results
        _product("product_one_token", 1, 1, 1, 4099, 7168, "f32"),
        # the decoding step's rows against 32 experts: the weights are what is read
        _product("product_decode", 256, 128, 32, 4096, 7168, "bf16"),
        # the large batch's rows against 32 experts
        _product("product_batch", 32768, 32500, 32, 4096, 7168, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "quantize", "product", "product"])
    if op == "quantize":
        k = 32 * _log(rng, 1, 256)
        return {"op": op, "rows": min(_log(rng, 1, 40000), 16384 * 7168 // k), "k": k,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "product":
        groups, n, k = _log(rng, 1, 64), _log(rng, 1, 8192), 32 * _log(rng, 1, 256)
        n = max(1, min(n, 32 * 4096 * 7168 // (groups * k)))
        rows = max(1, min(_log(rng, 1, 16384), 32768 * 4096 * 7168 // (16 * n * k)))
        c = _product("", rows, rng.randint(max(0, rows - rows // 4), rows), groups, n, k, rng.choice(["bf16", "f32", "f16"]),
                     zipf=rng.choice([0.0, 0.0, 0.8]))
        del c["name"]
        return c
    experts = _log(rng, 1, 256)
    local = experts if rng.random() < 0.5 else rng.randint(1, experts)
    topk = rng.randint(1, min(8, experts))
    hidden = _log(rng, 16, 8192)
    tokens = max(1, min(_log(rng, 1, 32768), 16384 * 8 * 2048 // (hidden * topk)))
    rows = tokens * topk if local == experts else max(1, min(tokens * topk, 2 * tokens * topk * local // experts + 64))
    c = _route("", op, tokens, hidden, experts, local, topk, rng.choice(["bf16", "f16", "f32"]), rows,
               zipf=rng.choice([0.0, 0.0, 1.1]), first=rng.randint(0, experts - local))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# inputs

def _routing(case, g):
    """Expert ids and softmax weights of each token: the top k of normal logits plus a Zipf prior's logarithm."""
    T, E, k = case["tokens"], case["experts"], case["topk"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["zipf"]:
        logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _sort(ids, first, local):
    """counts, offsets, row_to_slot, slot_to_row of the (token, slot) pairs grouped by local expert, stable by slot."""
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < local), flat, local)
    key, slots = torch.sort(key, stable=True)
    counts = torch.bincount(key, minlength=local + 1)[:local]
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    ours = key < local
    row_to_slot = torch.where(ours, slots, -1)
    slot_to_row = torch.empty_like(slots)
    slot_to_row[slots] = torch.where(ours, torch.arange(slots.numel(), device=slots.device), -1)
    return tuple(v.to(torch.int32) for v in (counts, offsets, row_to_slot, slot_to_row))


def _codes_of(v):
    """E2M1 codes and UE8M0 bytes of [M, K] values in blocks of 32: the smallest power of two that brings a block's
    largest magnitude within 6, then the nearest of the format's values, ties to the even code."""
    b = v.float().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = torch.where(top > 0, e - 3 + (m > 0.75), torch.zeros_like(e)).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e)
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c |= torch.signbit(b).to(torch.uint8) << 3
    return c.reshape(v.shape), (e + 127).to(torch.uint8).squeeze(-1)


def _nibbles(c):
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _packed(sf):
    """UE8M0 bytes [M, G] as int32 words [ceil(G / 4), M rounded up to 4], zero in the padding."""
    m, g = sf.shape
    j, am = (g + 3) // 4, (m + 3) // 4 * 4
    p = torch.zeros(am, 4 * j, dtype=torch.uint8, device=sf.device)
    p[:m, :g] = sf
    return p.reshape(am, j, 4).permute(1, 0, 2).contiguous().view(torch.int32).reshape(j, am)


def _sizes(case, seed):
    """Rows of each group: a multinomial over even or Zipf shares, the groups in a random order."""
    r = np.random.RandomState(seed % (1 << 31))
    p = np.arange(1, case["groups"] + 1, dtype=np.float64) ** -case["zipf"]
    return r.multinomial(case["used"], r.permutation(p / p.sum()))


def _plan(case):
    """The descriptor (and the sort's workspace) that a program keeps for its sizes."""
    from moe_expert_layer_amd import binding as B
    if case["op"] == "quantize":
        return B.make_mxfp4_desc(case["rows"], case["k"], dtype=case["dtype"], scale_layout="packed"), None
    if case["op"] == "product":
        return B.make_mxfp4_gemm_desc(case["rows"], case["n"], case["k"], groups=case["groups"], out_dtype=case["out"],
                                      a_scale_layout="packed", b_scale_layout="packed"), None
    d = B.make_dispatch_desc(case["tokens"], case["hidden"], case["experts"], case["topk"], local_begin=case["first"],
                             num_local=case["local"], dtype=case["dtype"], max_rows=case["rows"])
    return d, B.alloc_sort_workspace(d)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, "plan": _plan(case) if own else None}
    op = case["op"]

    def normal(*shape, dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    if op == "quantize":
        M, K = case["rows"], case["k"]
        # columns of different magnitude, as the channels of an activation or a weight have
        s["v"] = (normal(M, K, dtype=torch.float32)
                  * torch.exp(normal(K, dtype=torch.float32))).to(DTYPES[case["dtype"]])
        s["codes"] = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
        s["sf"] = torch.zeros((K // 32 + 3) // 4, (M + 3) // 4 * 4, dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "product":
        M, N, K, G = case["rows"], case["n"], case["k"], case["groups"]
        a, a_sf = _codes_of(normal(M, K, dtype=torch.bfloat16))
        s["a"], s["a_sf"] = _nibbles(a), _packed(a_sf)
        b = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
        b_sf = torch.empty(G, N, K // 32, dtype=torch.uint8, device="cuda")
        for e in range(G):
            c, b_sf[e] = _codes_of(normal(N, K, dtype=torch.bfloat16, scale=0.02))
            b[e] = _nibbles(c)
        s["b"], s["b_sf"] = b, _packed(b_sf.reshape(G * N, K // 32))
        sizes = _sizes(case, seed)
        s["most"] = max(1, int(sizes.max()))
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        s["out"] = torch.zeros(M, N, dtype=DTYPES[case["out"]], device="cuda")
        return s
    T, H, k, R, dt = case["tokens"], case["hidden"], case["topk"], case["rows"], DTYPES[case["dtype"]]
    ids, w = _routing(case, g)
    s["ids"], s["w"] = ids, w
    if op == "dispatch":
        s["x"] = normal(T, H, dtype=dt)
        s["maps"] = [torch.zeros(n, dtype=torch.int32, device="cuda")
                     for n in (case["local"], case["local"] + 1, T * k, T * k)]
        s["out"] = torch.zeros(R, H, dtype=dt, device="cuda")
        return s
    s["s2r"] = _sort(ids, case["first"], case["local"])[3]
    if op in ("combine", "combine_grad", "dispatch_grad"):
        s["rows"] = normal(R, H, dtype=dt)
    if op == "combine_grad":
        s["dy"] = normal(T, H, dtype=dt)
        s["drows"] = torch.zeros(R, H, dtype=dt, device="cuda")
        s["dw"] = torch.zeros(T, k, dtype=torch.float32, device="cuda")
        s["dlogits"] = torch.zeros(T, case["experts"], dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.zeros(T, H, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from moe_expert_layer_amd import binding as B
    d, ws = s["plan"]
    op = s["case"]["op"]
    if op == "dispatch":
        B.moe_sort_tokens(d, s["ids"], *s["maps"], ws)
        B.moe_dispatch(d, s["x"], s["maps"][3], s["out"])
        return {"counts": s["maps"][0], "offsets": s["maps"][1], "row_to_slot": s["maps"][2],
                "slot_to_row": s["maps"][3], "rows": s["out"]}
    if op == "dispatch_grad":
        B.moe_dispatch_backward(d, s["rows"], s["s2r"], s["out"])
        return {"dx": s["out"]}
    if op == "combine":
        B.moe_combine(d, s["rows"], s["s2r"], s["w"], s["out"])
        return {"y": s["out"]}
    if op == "combine_grad":
        B.moe_combine_backward(d, s["dy"], s["rows"], s["s2r"], s["w"], s["drows"], s["dw"], topk_ids=s["ids"],
                               dlogits=s["dlogits"])
        return {"drows": s["drows"], "dw": s["dw"], "dlogits": s["dlogits"]}
    if op == "quantize":
        B.moe_quantize_mxfp4(d, s["v"], s["codes"], s["sf"])
        B.moe_dequantize_mxfp4(d, s["codes"], s["sf"], s["out"], dtype="bf16")
        return {"values": s["out"]}
    B.moe_mxfp4_gemm(d, s["a"], s["a_sf"], s["b"], s["b_sf"], s["offsets"], s["out"])
    return {"c": s["out"]}


def _slots(s):
    """Row of each (token, slot), 0 where it has none, and whether it has one: [T, k]."""
    c = s["case"]
    r = s["s2r"].reshape(c["tokens"], c["topk"])
    has = (r >= 0) & (r < c["rows"])
    return torch.where(has, r, 0).long(), has


def _dispatch(s):
    c = s["case"]
    counts, offsets, r2s, s2r = _sort(s["ids"], c["first"], c["local"])
    slot = r2s[:c["rows"]].long()
    rows = torch.where((slot >= 0)[:, None], s["x"][slot.clamp(min=0) // c["topk"]], 0)
    return {"counts": counts, "offsets": offsets, "row_to_slot": r2s, "slot_to_row": s2r, "rows": rows}


def _dispatch_grad(s):
    r, has = _slots(s)
    return {"dx": torch.where(has[..., None], s["rows"][r].float(), 0.0).sum(1).to(s["rows"].dtype)}


def _combine(s):
    r, has = _slots(s)
    v = torch.where(has[..., None], s["rows"][r].float() * s["w"][..., None], 0.0)
    return {"y": v.sum(1).to(s["rows"].dtype)}


def _combine_grad(s):
    r, has = _slots(s)
    dy = s["dy"].float()
    dw = torch.where(has, (s["rows"][r].float() * dy[:, None]).sum(-1), 0.0)
    drows = torch.zeros_like(s["drows"])
    drows[r[has]] = (s["w"][..., None] * dy[:, None])[has].to(drows.dtype)
    g = s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True))
    dlogits = torch.zeros_like(s["dlogits"]).scatter_add_(1, s["ids"].long(), g)
    return {"drows": drows, "dw": dw, "dlogits": dlogits}


def _quantize(s):
    c, b = _codes_of(s["v"])
    return {"values": _values(c, b).to(torch.bfloat16)}


def _values(c, b):
    """float32 values of E2M1 codes [M, K] with UE8M0 bytes [M, K / 32]."""
    m = (c & 7).float()
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))  # 0 .5 1 1.5 2 3 4 6
    v = torch.where(c > 7, -v, v).reshape(c.shape[0], -1, 32)
    return torch.ldexp(v, b.to(torch.int32).unsqueeze(-1) - 127).reshape(c.shape)


def _stored(codes, packed):
    """float32 values of packed codes [M, K / 2] and packed scales."""
    m, g = codes.shape[0], codes.shape[1] // 16
    b = packed.view(torch.uint8).reshape(packed.shape[0], packed.shape[1], 4).permute(1, 0, 2).reshape(packed.shape[1], -1)
    return _values(torch.stack([codes & 15, codes >> 4], -1).reshape(m, -1), b[:m, :g])


def _product_plain(s):
    """The groups' rows padded to the longest group, one batched float32 product, the rows back in their places."""
    c = s["case"]
    G, N, M, K = c["groups"], c["n"], c["rows"], c["k"]
    a, o = _stored(s["a"], s["a_sf"]), s["offsets"].long()
    b = _stored(s["b"].reshape(G * N, K // 2), s["b_sf"]).reshape(G, N, K).transpose(1, 2).contiguous()
    at = o[:-1, None] + torch.arange(s["most"], device=a.device)
    p = torch.where((at < o[1:, None])[..., None], a[at.clamp(max=M - 1)], 0.0)
    p = torch.bmm(p, b)
    r = torch.arange(M, device=a.device)
    e = (torch.searchsorted(o, r, right=True) - 1).clamp(max=G - 1)
    mine = r < o[-1]
    out = p[e, torch.where(mine, r - o[e], 0)]
    return {"c": torch.where(mine[:, None], out, 0.0).to(s["out"].dtype)}


_PLAIN = {"dispatch": _dispatch, "dispatch_grad": _dispatch_grad, "combine": _combine, "combine_grad": _combine_grad,
          "quantize": _quantize, "product": _product_plain}


# ---------------------------------------------------------------------------------------
# bytes and operations that a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["k"]
        return {"bytes": n * (BYTES[case["dtype"]] + 0.5 + 1 / 32 + 2), "flops": 0}
    if op == "product":
        per = case["k"] / 2 + case["k"] / 32
        groups = min(case["groups"], case["used"])  # a group without rows is not read
        return {"bytes": case["used"] * (per + case["n"] * BYTES[case["out"]]) + groups * case["n"] * per,
                "flops": 2.0 * case["used"] * case["n"] * case["k"]}
    T, H, k, E = case["tokens"], case["hidden"], case["topk"], case["experts"]
    share = case["local"] / E
    rows = min(case["rows"], T * k * share)  # expected with evenly chosen experts
    some = T * (1 - (1 - share) ** k)        # tokens with a local expert
    row = H * BYTES[case["dtype"]]
    if op == "dispatch":
        return {"bytes": some * row + rows * row + 3 * 4 * T * k, "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": rows * row + T * row + 4 * T * k, "flops": rows * H}
    if op == "combine":
        return {"bytes": rows * row + T * row + 8 * T * k, "flops": 2 * rows * H}
    return {"bytes": 2 * rows * row + some * row + 16 * T * k + 4 * T * E, "flops": 3 * rows * H}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, row by row or group by group

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v = s["v"].double().reshape(case["rows"], -1, 32)
        top = v.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 6.0))
        e = e + (top > 6.0 * torch.exp2(e)).double() - (top <= 6.0 * torch.exp2(e - 1)).double()
        scale = torch.exp2(torch.where(top > 0, e.clamp(-127, 127), torch.zeros_like(e)))
        a = (v / scale).abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
        q = torch.clamp(torch.round(a / step) * step, max=6.0)
        return {"values": (torch.copysign(q, v) * scale).reshape(case["rows"], case["k"])}
    if op == "product":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                             device="cuda")

        def of(codes, packed, lo, hi):
            words = packed[:, lo:hi].long()
            by = torch.stack([(words >> (8 * i)) & 255 for i in range(4)], -1)  # [J, rows, 4]
            by = by.permute(1, 0, 2).reshape(hi - lo, -1)[:, :case["k"] // 32]
            c = codes.long()
            v = torch.empty(hi - lo, case["k"], dtype=torch.float64, device="cuda")
            v[:, 0::2], v[:, 1::2] = table[c & 15], table[c >> 4]
            return v * torch.exp2(by.double() - 127).repeat_interleave(32, 1)

        o = s["offsets"].tolist()
        out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["groups"]):
            if o[e + 1] > o[e]:
                a = of(s["a"][o[e]:o[e + 1]], s["a_sf"], o[e], o[e + 1])
                out[o[e]:o[e + 1]] = a @ of(s["b"][e], s["b_sf"], e * case["n"], (e + 1) * case["n"]).t().contiguous()
        return {"c": out}
    # the maps, by counting on the host
    T, H, k, E = case["tokens"], case["hidden"], case["topk"], case["experts"]
    ids = s["ids"].cpu().numpy().reshape(-1)
    order = [np.flatnonzero(ids == e) for e in range(case["first"], case["first"] + case["local"])]
    slots = np.concatenate(order)[:case["rows"]] if order else np.zeros(0, np.int64)
    slot = torch.from_numpy(slots.astype(np.int64)).cuda()
    R, tok = slot.numel(), slot // k
    if op == "dispatch":
        rows = torch.zeros(case["rows"], H, dtype=torch.float64, device="cuda")
        rows[:R] = s["x"].double()[tok]
        return {"counts": None, "offsets": None, "row_to_slot": None, "slot_to_row": None, "rows": rows}
    rows = s["rows"][:R].double()
    w = s["w"].double().reshape(-1)[slot]
    if op == "dispatch_grad":
        return {"dx": torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, tok, rows)}
    if op == "combine":
        return {"y": torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, tok, rows * w[:, None])}
    dy = s["dy"].double()[tok]
    drows = torch.zeros(case["rows"], H, dtype=torch.float64, device="cuda")
    drows[:R] = dy * w[:, None]
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    dw[slot] = (dy * rows).sum(1)
    dw = dw.reshape(T, k)
    # softmax over the chosen logits: d logit_j = sum_i dw_i w_i ([i = j] - w_j)
    wk = s["w"].double()
    jac = torch.diag_embed(wk) - wk[:, :, None] * wk[:, None, :]
    g = torch.matmul(jac, dw[:, :, None]).squeeze(-1)
    dlogits = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    dlogits.index_put_((torch.arange(T, device="cuda")[:, None].expand(T, k), s["ids"].long()), g, accumulate=True)
    return {"drows": drows, "dw": dw, "dlogits": dlogits}
