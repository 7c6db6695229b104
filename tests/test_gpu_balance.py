"""The router's balance loss and its gradient against float64 on the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24  # half a float32 step


# ---- the definition in float64 ----

def spans(case):
    """The tokens of each sequence that count."""
    T, ends, mask = case["T"], case["ends"], case["mask"]
    out = []
    for s in range(case["S"]):
        lo, hi = (0, T) if ends is None else (min(max(int(ends[s]), 0), T), min(max(int(ends[s + 1]), 0), T))
        t = np.arange(lo, max(lo, hi))
        out.append(t if mask is None else t[mask[t] != 0])
    return out


def probabilities(l, score):
    """p, log-sum-exp and a bound of p's relative error in float32: the rounded exponent (the difference, its product with
    log2 e and that constant, half a step each), the exponential and the reciprocal (a step each), and a sum of up to 1024
    positive terms in at most 32 steps a lane and 6 over lanes."""
    with np.errstate(all="ignore"):
        top = np.max(l, 1, keepdims=True)
        top = np.where(top == -np.inf, 0.0, top)
        v = np.exp(l - top)
        n = v.sum(1, keepdims=True)
        lse = np.where(n[:, 0] == 0, 0.0, top[:, 0] + np.log(np.where(n[:, 0] == 0, 1.0, n[:, 0])))
        d = np.minimum(np.abs(l - top), 150.0)
        if score == "sigmoid":
            logs = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
            top = np.max(logs, 1, keepdims=True)
            top = np.where(top == -np.inf, 0.0, top)
            v = np.exp(logs - top)
            n = v.sum(1, keepdims=True)
            d = d + np.minimum(np.abs(l), 150.0)
        p = np.where(n == 0, 0.0, v / np.where(n == 0, 1.0, n))
        rel = (4 * d + 4 + 2 * 40 + 4) * U
    return p, lse, np.where(np.isfinite(rel), rel, 1e-3)


def reference(case, logits, ids, k, score, counts=None, tokens=None, db=None, dz=None, add=None):
    T, E = logits.shape
    S = case["S"]
    r = {"counts": np.zeros((S, E), np.int64), "tokens": np.zeros(S, np.int64), "psum": np.zeros((S, E)),
         "psum_tol": np.zeros((S, E)), "balance": np.zeros(S), "balance_tol": np.zeros(S), "z": np.zeros(S),
         "z_tol": np.zeros(S)}
    grad = np.zeros((T, E)) if add is None else add.astype(np.float64).copy()
    tol = np.abs(grad) * 2 * U
    for s, t in enumerate(spans(case)):
        n = len(t)
        chosen = ids[t].reshape(-1)
        chosen = chosen[(chosen >= 0) & (chosen < E)]
        c = np.bincount(chosen, minlength=E)
        p, lse, rel = probabilities(logits[t], score)
        r["counts"][s], r["tokens"][s], r["psum"][s] = c, n, p.sum(0)
        # a lane adds up to 128 tokens, then 4 groups and 8 waves; the rest in float64
        r["psum_tol"][s] = (p * rel).sum(0) + p.sum(0) * (min(n, 4096) + 16) * U + 1e-37
        f = E / (k * max(n, 1) ** 2)
        r["balance"][s] = f * (c * p.sum(0)).sum()
        r["balance_tol"][s] = f * (c * r["psum_tol"][s]).sum() + r["balance"][s] * 2 * U
        with np.errstate(all="ignore"):
            lerr = rel.mean(1) + np.abs(lse) * 2 * U  # the sum's error is a mean of its terms' by their shares; bounded below
            lerr = np.maximum(lerr, (p * rel).sum(1) + np.abs(lse) * 2 * U)
        r["z"][s] = (lse ** 2).sum() / max(n, 1)
        r["z_tol"][s] = (2 * np.abs(lse) * lerr).sum() / max(n, 1) + r["z"][s] * (min(n, 4096) + 16) * U
        if db is None or n == 0:
            continue
        cs, ns = (c, n) if counts is None else (counts[s], int(tokens[s]))
        A = float(db[s]) * E / (k * float(ns) ** 2)
        mean = ns * k // E
        w = (cs - mean).astype(np.float64)  # a constant off every count changes nothing
        dot = (p * w).sum(1, keepdims=True)
        q = 1.0 if score == "softmax" else 1 / (1 + np.exp(np.minimum(logits[t], 700)))
        g = A * p * q * (w - dot)
        # the probabilities' errors, also in the dot product (which takes 64 terms a lane at most, then 6 steps)
        err = np.abs(A) * p * q * (np.abs(w - dot) * (2 * rel + 8 * U) + (p * np.abs(w) * (rel + 72 * U)).sum(1, keepdims=True)
                                   + np.abs(w) * 4 * U)
        if dz is not None:
            zc = 2 * float(dz[s]) / ns
            g = g + zc * lse[:, None] * p
            err = err + np.abs(zc) * p * (np.abs(lse[:, None]) * (rel + 8 * U) + lerr[:, None])
        grad[t] += g
        tol[t] += err + np.abs(g) * 4 * U + 1e-40
        tol[t] += np.abs(grad[t]) * 2 * U
    r["grad"], r["grad_tol"] = grad, tol
    return r


def make_case(T, S, padded, seed):
    r = np.random.RandomState(seed)
    ends = None
    if S > 1 or padded == "ends":
        lo, hi = (T // 7, T - T // 5) if padded else (0, T)
        ends = np.concatenate([[lo], np.sort(r.randint(lo, hi + 1, S - 1)), [hi]]).astype(np.int32)
        if S > 3:
            ends[2] = ends[1]  # an empty sequence
    mask = (r.rand(T) < 0.7).astype(np.uint8) * 3 if padded else None  # any byte but 0 counts
    return {"T": T, "S": S, "ends": ends, "mask": mask}


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def place(v, pad, shift, fill):
    """v [T, E] in rows pad elements longer, shift elements into its buffer, with fill in between."""
    T, E = v.shape
    buf = torch.full((shift + T * (E + pad) + 8,), fill, dtype=v.dtype, device="cuda")
    m = buf[shift:shift + T * (E + pad)].view(T, E + pad)[:, :E]
    m.copy_(v)
    return buf, m


def call_forward(d, logits, ids, case, z, ws=None):
    S, E = case["S"], d.num_experts
    out = {"counts": torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
           "tokens": torch.full((S,), -7, dtype=torch.int32, device="cuda"),
           "psum": torch.full((S, E), -7.0, device="cuda"), "balance": torch.full((S,), -7.0, device="cuda")}
    if z:
        out["z"] = torch.full((S,), -7.0, device="cuda")
    if ws is None:
        ws = torch.full((max(B.moe_balance_workspace_size(d), 256),), 0xa5, dtype=torch.uint8, device="cuda")
    B.moe_balance_loss(d, logits, ids, out["counts"], out["tokens"], out["psum"], out["balance"], ws, z=out.get("z"),
                       mask=dev(case["mask"]), seq_offsets=dev(case["ends"]))
    return out


def check_forward(out, r):
    assert np.array_equal(out["counts"].cpu().numpy(), r["counts"])
    assert np.array_equal(out["tokens"].cpu().numpy(), r["tokens"])
    for name in ("psum", "balance") + (("z",) if "z" in out else ()):
        got = out[name].cpu().numpy().astype(np.float64)
        off = np.abs(got - r[name]) - r[name + "_tol"]
        assert off.max() <= 0, (name, off.max(), np.unravel_index(off.argmax(), off.shape))


SHAPES = [  # T, E, k, S, padded
    (1, 1, 1, 1, False), (1, 2, 2, 1, False), (7, 3, 1, 3, True), (64, 4, 2, 1, False), (33, 5, 3, 5, True),
    (129, 16, 4, 1, True), (130, 17, 4, 2, False), (1000, 31, 6, 4, True), (1024, 32, 16, 1, False),
    (1025, 33, 8, 6, True), (2000, 64, 2, 1, True), (1500, 66, 8, 40, False), (5000, 127, 8, 3, True),
    (3000, 129, 6, 24, True), (4097, 192, 4, 1, False), (2048, 193, 8, 7, True), (20000, 256, 8, 1, False),
    (1100, 257, 8, 2, True), (1030, 385, 8, 1, False), (1300, 511, 1, 9, True), (1700, 513, 8, 4, True),
    (1111, 1023, 16, 2, True), (40, 1024, 8, 1, False), (2100, 1024, 8, 33, False), (1025, 8, 2, 700, True)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,S,padded", SHAPES)
def test_loss_and_gradient(T, E, k, S, padded, dtype, score):
    seed = T + 7 * E + S
    g = torch.Generator().manual_seed(seed)
    case = make_case(T, S, padded, seed)
    logits = (3 * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).to(DT[dtype])
    ids = torch.randint(-2 if padded else 0, E + (2 if padded else 0), (T, k), generator=g, dtype=torch.int32)
    if padded:  # padding may hold anything
        counted = np.zeros(T, bool)
        for t in spans(case):
            counted[t] = True
        logits[~torch.from_numpy(counted)] = float("nan")
        ids[~torch.from_numpy(counted)] = 2 ** 31 - 1
    pad, shift = (3, 1) if T % 2 else (0, 0)
    _, l = place(logits.cuda(), pad, shift, float("nan"))
    d = B.make_balance_desc(T, E, k, S, dtype, score, logit_stride=E + pad, grad_stride=E + pad)
    z = score == "softmax"
    out = call_forward(d, l, ids.cuda(), case, z)
    db = np.random.RandomState(seed).rand(S).astype(np.float32) - 0.3
    dz = (np.random.RandomState(seed + 1).rand(S).astype(np.float32) - 0.3) if z and T % 3 else None
    add = (torch.randn(T, E, generator=g) * float(np.abs(db).max()) / T).numpy() if k % 2 else None
    x, i = logits.double().numpy(), ids.numpy()
    r = reference(case, x, i, k, score, db=db, dz=dz, add=add)
    check_forward(out, r)
    buf, dl = place(torch.full((T, E), 55.0), pad, shift, 77.0)
    base = None
    if add is not None:
        base = torch.from_numpy(add).cuda()
        base = place(base, pad, shift, float("nan"))[1]
        if k % 4 == 1:  # in place
            dl.copy_(base)
            base = dl
    B.moe_balance_loss_backward(d, l, out["counts"], out["tokens"], dev(db), dl, dz=dev(dz), mask=dev(case["mask"]),
                                seq_offsets=dev(case["ends"]), add=base)
    off = np.abs(dl.cpu().double().numpy() - r["grad"]) - r["grad_tol"]
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    dl.fill_(77.0)
    assert (buf == 77).all()  # nothing between the rows


def test_gradient_against_differences():
    """The gradient of sum_s db[s] balance[s] + dz[s] z[s] along random directions, with the counts held: central
    differences of the float64 definition."""
    T, E, k, S = 200, 24, 4, 3
    case = make_case(T, S, True, 5)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, E, generator=g) * 2
    ids = torch.topk(x, k)[1].to(torch.int32)
    db, dz = np.array([0.5, -1.0, 2.0], np.float32), np.array([0.25, 0.5, -0.125], np.float32)
    for score in ("softmax", "sigmoid"):
        d = B.make_balance_desc(T, E, k, S, "f32", score)
        l = x.cuda()
        out = call_forward(d, l, ids.cuda(), case, False)
        dl = torch.empty(T, E, device="cuda")
        zz = dz if score == "softmax" else None
        B.moe_balance_loss_backward(d, l, out["counts"], out["tokens"], dev(db), dl, dz=dev(zz), mask=dev(case["mask"]),
                                    seq_offsets=dev(case["ends"]))

        def loss(v):
            r = reference(case, v, ids.numpy(), k, score)
            return (db * r["balance"]).sum() + (0 if zz is None else (zz * r["z"]).sum())

        for i in range(3):
            u = torch.randn(T, E, generator=g, dtype=torch.float64).numpy()
            h = 1e-4
            num = (loss(x.double().numpy() + h * u) - loss(x.double().numpy() - h * u)) / (2 * h)
            ana = (dl.cpu().double().numpy() * u).sum()
            size = np.abs(dl.cpu().double().numpy() * u).sum()
            # h^2 / 6 of the third derivative (of order 1 in the logits), and the gradient's own relative error
            assert abs(num - ana) <= 1e-4 * size, (num, ana)


def test_infinities_and_the_lowest_value():
    T, E, k = 12, 10, 2
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    inf = float("inf")
    x[1, 3] = -inf                      # an expert that is masked off
    x[2, :] = -inf                      # all of them
    x[3, :9] = -inf                     # all but one
    x[4, :] = torch.finfo(torch.float32).min
    x[5, :5] = torch.finfo(torch.float32).min
    x[6, :] = -300.0                    # sigmoids that all underflow
    x[6, 2] = -299.0
    x[7, 0] = 1e30
    ids = torch.topk(torch.randn(T, E), k)[1].to(torch.int32)
    for score in ("softmax", "sigmoid"):
        for T0 in (T, 3 * 512):  # both forward paths
            l = x.repeat(T0 // T, 1)
            i = ids.repeat(T0 // T, 1)
            case = {"T": T0, "S": 1, "ends": None, "mask": None}
            d = B.make_balance_desc(T0, E, k, 1, "f32", score)
            out = call_forward(d, l.cuda(), i.cuda(), case, False)
            db = np.ones(1, np.float32)
            r = reference(case, l.double().numpy(), i.numpy(), k, score, db=db)
            check_forward(out, r)
            dl = torch.empty(T0, E, device="cuda")
            B.moe_balance_loss_backward(d, l.cuda(), out["counts"], out["tokens"], dev(db), dl)
            got = dl.cpu().double().numpy()
            assert (np.abs(got - r["grad"]) <= r["grad_tol"]).all()
            assert (got[2] == 0).all() and (got[1, 3] == 0)


@pytest.mark.parametrize("T", [100, 3000])
def test_nan_stays_in_its_sequence(T):
    E, k, S = 20, 3, 2
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(2))
    x[T // 4, 7] = float("nan")
    ids = torch.randint(0, E, (T, k), dtype=torch.int32)
    case = {"T": T, "S": S, "ends": np.array([0, T // 2, T], np.int32), "mask": None}
    d = B.make_balance_desc(T, E, k, S)
    out = call_forward(d, x.cuda(), ids.cuda(), case, True)
    assert torch.isnan(out["psum"][0]).all() and torch.isnan(out["balance"][0]) and torch.isnan(out["z"][0])
    assert torch.isfinite(out["psum"][1]).all() and torch.isfinite(out["balance"][1]) and torch.isfinite(out["z"][1])
    dl = torch.empty(T, E, device="cuda")
    B.moe_balance_loss_backward(d, x.cuda(), out["counts"], out["tokens"], dev(np.ones(2, np.float32)), dl,
                                dz=dev(np.ones(2, np.float32)), seq_offsets=dev(case["ends"]))
    bad = torch.isnan(dl).any(1).cpu()
    assert bad[T // 4] and bad.sum() == 1


@pytest.mark.parametrize("T", [50, 4000])
def test_offsets_are_cut_and_sequences_may_be_empty(T):
    E, k = 12, 2
    x, ids = torch.randn(T, E), torch.randint(0, E, (T, k), dtype=torch.int32)
    ends = np.array([-5, 0, T // 3, T // 3, T + 100, T + 100, 2 ** 31 - 1], np.int32)
    case = {"T": T, "S": 6, "ends": ends, "mask": None}
    d = B.make_balance_desc(T, E, k, 6)
    out = call_forward(d, x.cuda(), ids.cuda(), case, True)
    db, dz = np.ones(6, np.float32), np.ones(6, np.float32)
    r = reference(case, x.double().numpy(), ids.numpy(), k, "softmax", db=db, dz=dz)
    check_forward(out, r)
    assert r["tokens"].tolist() == [0, T // 3, 0, T - T // 3, 0, 0]
    dl = torch.empty(T, E, device="cuda")
    B.moe_balance_loss_backward(d, x.cuda(), out["counts"], out["tokens"], dev(db), dl, dz=dev(dz), seq_offsets=dev(ends))
    assert (np.abs(dl.cpu().double().numpy() - r["grad"]) <= r["grad_tol"]).all()
    # nothing but padding
    case["mask"] = np.zeros(T, np.uint8)
    out = call_forward(d, x.cuda(), ids.cuda(), case, True)
    assert all((v == 0).all() for v in out.values())


def test_counts_of_a_larger_batch():
    """Counts and tokens summed over two parts of a batch give each part the gradient of the whole batch's loss."""
    T, E, k = 600, 40, 4
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2 * T, E, generator=g) + torch.randn(E, generator=g)
    ids = torch.topk(x, k)[1].to(torch.int32)
    db = np.ones(1, np.float32)
    outs = [call_forward(B.make_balance_desc(T, E, k), x[i * T:(i + 1) * T].cuda(), ids[i * T:(i + 1) * T].cuda(),
                         {"T": T, "S": 1, "ends": None, "mask": None}, False) for i in range(2)]
    counts, tokens = outs[0]["counts"] + outs[1]["counts"], outs[0]["tokens"] + outs[1]["tokens"]
    whole = reference({"T": 2 * T, "S": 1, "ends": None, "mask": None}, x.double().numpy(), ids.numpy(), k, "softmax", db=db)
    for i in range(2):
        dl = torch.empty(T, E, device="cuda")
        B.moe_balance_loss_backward(B.make_balance_desc(T, E, k), x[i * T:(i + 1) * T].cuda(), counts, tokens, dev(db), dl)
        at = slice(i * T, (i + 1) * T)
        assert (np.abs(dl.cpu().double().numpy() - whole["grad"][at]) <= whole["grad_tol"][at]).all()


def test_same_bits_on_every_run_stream_and_replay():
    """Eager calls, two streams at once and a captured graph's replays (with other work on the workspace in between) give
    the same bits."""
    T, E, k, S = 9000, 96, 6, 5
    case = make_case(T, S, True, 3)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(4)).cuda()
    ids = torch.topk(x, k)[1].to(torch.int32)
    mask, ends, one = dev(case["mask"]), dev(case["ends"]), dev(np.ones(S, np.float32))
    d = B.make_balance_desc(T, E, k, S)

    def buffers():
        return {"counts": torch.zeros(S, E, dtype=torch.int32, device="cuda"),
                "tokens": torch.zeros(S, dtype=torch.int32, device="cuda"), "psum": torch.zeros(S, E, device="cuda"),
                "balance": torch.zeros(S, device="cuda"), "z": torch.zeros(S, device="cuda"),
                "dl": torch.zeros(T, E, device="cuda"), "ws": B.alloc_balance_workspace(d)}

    def call(o, stream=None):
        B.moe_balance_loss(d, x, ids, o["counts"], o["tokens"], o["psum"], o["balance"], o["ws"], z=o["z"], mask=mask,
                           seq_offsets=ends, stream=stream)
        B.moe_balance_loss_backward(d, x, o["counts"], o["tokens"], one, o["dl"], dz=one, mask=mask, seq_offsets=ends,
                                    stream=stream)

    def same(o):
        torch.cuda.synchronize()
        return all(torch.equal(first[n], o[n]) for n in first if n != "ws")

    first = buffers()
    call(first)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(), buffers()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            call(o, s)
    assert same(outs[0]) and same(outs[1])
    o = buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(o)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o)
    for i in range(4):
        for n in o:
            o[n].fill_(i)
        graph.replay()
        assert same(o)


def test_far_rows():
    """Rows whose distance takes the offsets past 32 bits (the stride is the distance; four rows of a large buffer)."""
    T, E, k = 4, 8, 2
    stride = (1 << 30) + 1
    buf = torch.empty(3 * stride + E, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, E).bfloat16()
    l = buf.as_strided((T, E), (stride, 1))
    l.copy_(x)
    ids = torch.topk(x.float(), k)[1].to(torch.int32)
    case = {"T": T, "S": 1, "ends": None, "mask": None}
    d = B.make_balance_desc(T, E, k, 1, "bf16", logit_stride=stride)
    out = call_forward(d, l, ids.cuda(), case, True)
    db = np.ones(1, np.float32)
    r = reference(case, x.double().numpy(), ids.numpy(), k, "softmax", db=db)
    check_forward(out, r)
    dl = torch.empty(T, E, device="cuda")
    B.moe_balance_loss_backward(d, l, out["counts"], out["tokens"], dev(db), dl)
    assert (np.abs(dl.cpu().double().numpy() - r["grad"]) <= r["grad_tol"]).all()


def test_refusals():
    T, E, k = 8, 6, 2
    d = B.make_balance_desc(T, E, k, 2)
    x, ids = torch.zeros(T, E, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    c, t, f = torch.zeros(2, E, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, E, device="cuda")
    b, ws = torch.zeros(2, device="cuda"), B.alloc_balance_workspace(d)

    def forward(logits=x, i=ids, counts=c, tokens=t, psum=f, bal=b, w=ws, desc=d, **kw):
        kw.setdefault("seq_offsets", ends)
        B.moe_balance_loss(desc, logits, i, counts, tokens, psum, bal, w, **kw)

    forward()
    bad = [dict(logits=x.half()), dict(logits=x[:, :5]), dict(logits=x[:4]), dict(i=ids.long()), dict(i=ids[:3]),
           dict(counts=c[:1]), dict(tokens=t.float()), dict(psum=f[0]), dict(bal=b[:1]), dict(z=b[:1]), dict(mask=b),
           dict(mask=torch.ones(T - 1, dtype=torch.bool, device="cuda")), dict(seq_offsets=ends[:2]),
           dict(seq_offsets=ends.long()), dict(seq_offsets=None), dict(i=ids.cpu()), dict(logits=x.t().contiguous().t())]
    for kw in bad:
        with pytest.raises(B.MoeError):
            forward(**kw)
    with pytest.raises(B.MoeError) as e:
        forward(desc=B.make_balance_desc(T, E, k, 2, score="sigmoid"), z=b)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
    dl = torch.zeros(T, E, device="cuda")
    B.moe_balance_loss_backward(d, x, c, t, b, dl, seq_offsets=ends)
    for kw in (dict(dlogits=dl.half()), dict(dlogits=dl[:4]), dict(dbalance=b[:1]), dict(dz=b[:1]), dict(add=dl[:3]),
               dict(add=dl.double()), dict(seq_offsets=None)):
        a = dict(dbalance=b, dlogits=dl, seq_offsets=ends)
        a.update(kw)
        with pytest.raises(B.MoeError):
            B.moe_balance_loss_backward(d, x, c, t, a.pop("dbalance"), a.pop("dlogits"), **a)


def test_most_sequences():
    """As many sequences as there may be, most of them of one token or none, in both directions."""
    T, E, k, S = 70001, 5, 2, 65536
    r = np.random.RandomState(3)
    ends = np.concatenate([[0], np.sort(r.randint(0, T + 1, S - 1)), [T]]).astype(np.int32)
    case = {"T": T, "S": S, "ends": ends, "mask": None}
    logits = r.randn(T, E).astype(np.float32)
    ids = r.randint(0, E, (T, k)).astype(np.int32)
    db, dz = r.randn(S).astype(np.float32), r.randn(S).astype(np.float32)
    ref = reference(case, logits.astype(np.float64), ids, k, "softmax", db=db, dz=dz)
    d = B.make_balance_desc(T, E, k, S, "f32")
    out = call_forward(d, dev(logits), dev(ids), case, True)
    check_forward(out, ref)
    grad = torch.full((T, E), 7.0, device="cuda")
    B.moe_balance_loss_backward(d, dev(logits), out["counts"], out["tokens"], dev(db), grad, dz=dev(dz), seq_offsets=dev(ends))
    assert (np.abs(grad.cpu().numpy() - ref["grad"]) <= ref["grad_tol"]).all()


def test_millions_of_tokens():
    """More tokens than 512 chunks of 8192 hold.  |l| < 4, so a probability is (4 * 8 + 88) U off relatively; a lane then adds up to 1024, and 16
    sums follow."""
    T, E, k = 4_500_001, 3, 2
    g = torch.Generator().manual_seed(1)
    logits = (8 * torch.rand(T, E, generator=g) - 4)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    out = call_forward(B.make_balance_desc(T, E, k, 1, "f32"), logits.cuda(), ids.cuda(), {"T": T, "S": 1, "ends": None, "mask": None}, False)
    p = torch.softmax(logits.double(), 1).sum(0)
    c = torch.bincount(ids[ids >= 0].long(), minlength=E)
    assert torch.equal(out["counts"][0].cpu().long(), c) and int(out["tokens"][0]) == T
    tol = (120 + 1024 + 16 + 1) * U
    assert ((out["psum"][0].cpu().double() - p).abs() <= p * tol).all()
    want = float((c * p).sum()) * E / (k * float(T) ** 2)
    assert abs(float(out["balance"][0]) - want) <= want * (tol + 2 * U)
