"""Tokens sorted by expert and back, with gradients, against float64 on the CPU.

Tolerances: a float32 sum of n terms of the values v is within n 2^-24 sum|v| of the exact one, a
product or a rounding to a type within half a step (finfo.eps / 2 of the value; half the smallest
subnormal near zero)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def half_step(dtype, ref):
    """Largest rounding error of ref to dtype, plus one float32 rounding."""
    t = torch.finfo(DT[dtype])
    return ref.abs() * (t.eps / 2) + ref.abs() * U + t.smallest_normal * t.eps / 2


def make_ids(T, E, k, seed, dup=False):
    r = np.random.RandomState(seed)
    ids = r.randint(0, E, (T, k)) if dup else np.argsort(r.rand(T, E), axis=1)[:, :k]
    return torch.from_numpy(np.ascontiguousarray(ids).astype(np.int32))


def sort_ref(ids, e0, el):
    flat = ids.reshape(-1).numpy().astype(np.int64) - e0
    ours = (flat >= 0) & (flat < el)
    slots = np.flatnonzero(ours)
    slots = slots[np.argsort(flat[slots], kind="stable")]
    counts = np.bincount(flat[ours], minlength=el)
    r2s = np.full(flat.size, -1, np.int32)
    r2s[:slots.size] = slots
    s2r = np.full(flat.size, -1, np.int32)
    s2r[slots] = np.arange(slots.size)
    return counts.astype(np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), r2s, s2r


def run_sort(d, ids, ws=None):
    n = ids.numel()
    out = [torch.full((m,), -7, dtype=torch.int32, device="cuda") for m in (d.num_local, d.num_local + 1, n, n)]
    B.moe_sort_tokens(d, ids.cuda(), *out, B.alloc_sort_workspace(d) if ws is None else ws)
    return out


@pytest.mark.parametrize("T,E,e0,el,k,dup", [
    (1, 1, 0, 1, 1, False), (1, 8, 3, 2, 8, False), (77, 8, 0, 8, 2, False), (300, 32, 5, 20, 4, True),
    (1024, 256, 0, 32, 8, False), (1025, 200, 0, 200, 8, True), (2500, 1024, 100, 900, 16, True),
    (9000, 64, 10, 33, 8, False), (40000, 256, 0, 256, 1, False)])
def test_sort(T, E, e0, el, k, dup):
    ids = make_ids(T, E, k, T + k, dup)
    d = B.make_dispatch_desc(T, 8, E, k, local_begin=e0, num_local=el)
    for got, want in zip(run_sort(d, ids), sort_ref(ids, e0, el)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,E,e0,el,k", [
    (6144, 70, 3, 63, 1), (6145, 70, 3, 63, 1), (6145, 70, 3, 64, 1), (2048, 300, 9, 256, 1), (2049, 300, 9, 256, 1),
    (2048, 300, 9, 257, 1), (8192, 16, 0, 16, 8), (32768, 300, 0, 127, 2), (32769, 300, 0, 128, 2),
    (65536, 512, 0, 511, 1), (65537, 512, 0, 511, 1), (65536, 512, 0, 512, 1), (30000, 1024, 0, 1024, 3),
    (200000, 300, 100, 100, 4), (1 << 20, 8, 7, 1, 1)])
def test_sort_at_the_boundaries_of_its_kernels(T, E, e0, el, k):
    g = torch.Generator().manual_seed(T + el)
    p = torch.rand(E, generator=g) ** 4  # uneven: some experts have most of the slots, some none
    p[torch.randperm(E, generator=g)[:E // 4]] = 0
    ids = torch.multinomial(p, T * k, replacement=True, generator=g).to(torch.int32).view(T, k)
    d = B.make_dispatch_desc(T, 8, E, k, local_begin=e0, num_local=el)
    for got, want in zip(run_sort(d, ids), sort_ref(ids, e0, el)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_ids_outside_every_expert():
    ids = torch.tensor([[0, -1], [2147483647, 3], [-2147483648, 1], [7, 8]], dtype=torch.int32)
    d = B.make_dispatch_desc(4, 8, 8, 2, local_begin=1, num_local=7)
    for got, want in zip(run_sort(d, ids), sort_ref(ids, 1, 7)):
        assert np.array_equal(got.cpu().numpy(), want)


class Case:
    """Inputs on the CPU in float64 (values of the dtype), maps, and strided, offset device copies whose padding
    and rows that no slot owns hold NaN."""

    def __init__(self, T, H, E, e0, el, k, dtype, max_rows=0, pad=0, shift=0, seed=0, dup=False):
        self.T, self.H, self.k, self.E, self.dtype = T, H, k, E, dtype
        self.ids = make_ids(T, E, k, seed, dup)
        self.cap = max_rows or T * k
        self.counts, self.offsets, _, s2r = sort_ref(self.ids, e0, el)
        self.s2r = torch.from_numpy(s2r)
        self.has = (self.s2r >= 0) & (self.s2r < self.cap)
        self.slot = torch.nonzero(self.has)[:, 0]
        self.row = self.s2r[self.slot].long()
        self.tok = self.slot // k
        g = torch.Generator().manual_seed(seed + 1)
        self.w = torch.softmax(torch.randn(T, k, generator=g), 1)
        self.x = torch.randn(T, H, generator=g).to(DT[dtype]).double()
        self.ys = torch.full((self.cap, H), float("nan"), dtype=torch.float64)
        self.ys[self.row] = torch.randn(self.row.numel(), H, generator=g).to(DT[dtype]).double()
        self.pad, self.shift = pad, shift
        self.desc = B.make_dispatch_desc(T, H, E, k, local_begin=e0, num_local=el, dtype=dtype, max_rows=max_rows,
                                         token_stride=H + pad if pad else 0, row_stride=H + 2 * pad if pad else 0)

    def dev(self, v, rows_stride, fill=float("nan")):
        """v on the GPU, its rows rows_stride apart, `shift` elements into its buffer."""
        n = v.shape[0]
        buf = torch.full((self.shift + n * rows_stride,), fill, dtype=DT[self.dtype], device="cuda")
        t = buf[self.shift:].view(n, rows_stride)[:, :self.H]
        t.copy_(v.to(DT[self.dtype]))
        return t, buf

    def tokens(self, v):
        return self.dev(v, self.H + self.pad)

    def rows(self, v):
        return self.dev(v, self.H + 2 * self.pad)

    def sentinel(self, n, stride):
        return self.dev(torch.full((n, self.H), 77.0), stride, fill=77.0)

    def untouched(self, buf, n, stride, rows=None):
        """The padding of every row, what lies before the first, and rows not in `rows` still hold 77."""
        b = buf.float().cpu()
        assert (b[:self.shift] == 77).all()
        b = b[self.shift:].view(n, stride)
        assert (b[:, self.H:] == 77).all()
        if rows is not None:
            rest = torch.ones(n, dtype=torch.bool)
            rest[rows] = False
            assert (b[rest] == 77).all()


SHAPES = [  # T, H, E, e0, el, k, max_rows, pad, shift, dup
    (1, 1, 1, 0, 1, 1, 0, 0, 0, False),
    (1, 7168, 256, 0, 256, 8, 0, 0, 0, False),
    (3, 7, 8, 2, 3, 2, 0, 0, 0, False),       # tokens without a local expert
    (65, 8, 16, 0, 16, 16, 0, 0, 0, False),   # every slot of 16 has a row
    (40, 1111, 64, 8, 16, 8, 0, 5, 1, False),  # odd rows, padded, off the 16-byte grid
    (300, 256, 8, 0, 8, 2, 0, 0, 0, True),    # a token names an expert twice
    (129, 2050, 32, 0, 32, 4, 400, 0, 3, False),  # 516 rows, of which 400 fit
    (50, 4100, 16, 3, 1, 3, 0, 4, 0, True),
    (70000, 9, 4, 0, 4, 1, 0, 0, 0, False),   # more tokens than one grid row of workgroups
]


def each(f):
    f = pytest.mark.parametrize("shape", SHAPES, ids=[f"T{s[0]}H{s[1]}k{s[5]}" for s in SHAPES])(f)
    return pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])(f)


def case_of(shape, dtype):
    T, H, E, e0, el, k, cap, pad, shift, dup = shape
    return Case(T, H, E, e0, el, k, dtype, cap, pad, shift, seed=T + H, dup=dup)


@each
def test_dispatch(shape, dtype):
    c = case_of(shape, dtype)
    xs, buf = c.sentinel(c.cap, c.H + 2 * c.pad)
    B.moe_dispatch(c.desc, c.tokens(c.x)[0], c.s2r.cuda(), xs)
    assert torch.equal(xs.double().cpu()[c.row], c.x[c.tok])
    c.untouched(buf, c.cap, c.H + 2 * c.pad, c.row)


@pytest.mark.parametrize("nbytes,shift,T", [(1, 0, 37), (15, 1, 37), (224, 0, 37), (3584, 0, 37), (8193, 3, 37),
                                            (1, 0, 1100), (1030, 0, 1100), (2047, 1, 1025), (5000, 0, 1100),
                                            (16384, 0, 1025), (20005, 5, 1030)])
def test_dispatch_bytes(nbytes, shift, T):
    E, k = 16, 4
    ids = make_ids(T, E, k, 5)
    s2r = torch.from_numpy(sort_ref(ids, 4, 9)[3])
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, 256, (T, nbytes), generator=g, dtype=torch.uint8)
    buf = torch.full((shift + T * k * nbytes,), 77, dtype=torch.uint8, device="cuda")
    xs = buf[shift:].view(T * k, nbytes)
    d = B.make_dispatch_desc(T, nbytes, E, k, local_begin=4, num_local=9, dtype="u8")
    B.moe_dispatch(d, x.cuda(), s2r.cuda(), xs)
    want = torch.full((T * k, nbytes), 77, dtype=torch.uint8)
    slot = torch.nonzero(s2r >= 0)[:, 0]
    want[s2r[slot].long()] = x[slot // k]
    assert torch.equal(xs.cpu(), want)


@each
def test_dispatch_backward_and_combine(shape, dtype):
    c = case_of(shape, dtype)
    ys = c.rows(c.ys)[0]
    for w in (None, c.w):
        y, buf = c.sentinel(c.T, c.H + c.pad)
        if w is None:
            B.moe_dispatch_backward(c.desc, ys, c.s2r.cuda(), y)
        else:
            B.moe_combine(c.desc, ys, c.s2r.cuda(), w.cuda(), y)
        v = c.ys[c.row] * (1.0 if w is None else w.double().reshape(-1)[c.slot][:, None])
        ref = torch.zeros(c.T, c.H, dtype=torch.float64).index_add_(0, c.tok, v)
        mag = torch.zeros(c.T, c.H, dtype=torch.float64).index_add_(0, c.tok, v.abs())
        err = (y.double().cpu() - ref).abs()
        assert (err <= half_step(dtype, ref) + (c.k + 1) * U * mag).all(), err.max()
        empty = torch.ones(c.T, dtype=torch.bool)
        empty[c.tok] = False
        assert (y.cpu()[empty] == 0).all()
        c.untouched(buf, c.T, c.H + c.pad)


@each
def test_combine_backward(shape, dtype):
    c = case_of(shape, dtype)
    dys, buf = c.sentinel(c.cap, c.H + 2 * c.pad)
    dw = torch.full((c.T, c.k), 77.0, device="cuda")
    dl = torch.full((c.T, c.E), 77.0, device="cuda")
    B.moe_combine_backward(c.desc, c.tokens(c.x)[0], c.rows(c.ys)[0], c.s2r.cuda(), c.w.cuda(), dys, dw,
                           topk_ids=c.ids.cuda(), dlogits=dl)
    wd = c.w.double()
    ref = c.x[c.tok] * wd.reshape(-1)[c.slot][:, None]
    assert ((dys.double().cpu()[c.row] - ref).abs() <= half_step(dtype, ref)).all()
    c.untouched(buf, c.cap, c.H + 2 * c.pad, c.row)
    prod = c.x[c.tok] * c.ys[c.row]
    rdw = torch.zeros(c.T * c.k, dtype=torch.float64)
    rdw[c.slot] = prod.sum(1)
    # a lane sums at most H / 64 terms, rounded up to whole 16-byte chunks, plus one; then 6 + 8 additions
    tol = torch.zeros_like(rdw)
    tol[c.slot] = (c.H / 64 + 9 + 14) * U * prod.abs().sum(1)
    rdw, tol = rdw.reshape(c.T, c.k), tol.reshape(c.T, c.k)
    assert ((dw.double().cpu() - rdw).abs() <= tol).all()
    assert (dw.cpu().reshape(-1)[~c.has] == 0).all()
    s = (wd * rdw).sum(1, keepdim=True)
    g = wd * (rdw - s)
    gtol = wd * (tol + (wd * tol).sum(1, keepdim=True) + (c.k + 3) * U * (rdw.abs() + (wd * rdw.abs()).sum(1, keepdim=True)))
    rdl = torch.zeros(c.T, c.E, dtype=torch.float64).scatter_add_(1, c.ids.long(), g)
    gabs = torch.zeros(c.T, c.E, dtype=torch.float64).scatter_add_(1, c.ids.long(), gtol + c.k * U * g.abs())
    assert ((dl.double().cpu() - rdl).abs() <= gabs).all()
    # without dlogits: the same dys and dw
    dys2, dw2 = torch.zeros_like(dys), torch.zeros_like(dw)
    d2 = B.make_dispatch_desc(c.T, c.H, c.E, c.k, local_begin=c.desc.local_begin, num_local=c.desc.num_local, dtype=dtype,
                              max_rows=c.desc.max_rows, token_stride=c.desc.token_stride)
    ys_dense = c.rows(c.ys)[0].contiguous()
    B.moe_combine_backward(d2, c.tokens(c.x)[0], ys_dense, c.s2r.cuda(), c.w.cuda(), dys2, dw2)
    assert torch.equal(dw2, dw) and torch.equal(dys2.cpu()[c.row], dys.cpu()[c.row])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [
    (2047, 512, 32, 0, 32, 8, 0, 0, 0, False), (2048, 512, 32, 0, 32, 8, 0, 0, 0, False),
    (2051, 1025, 16, 3, 9, 4, 0, 3, 1, True), (2300, 1023, 8, 0, 8, 4, 5000, 0, 0, False),
    (3001, 130, 64, 5, 40, 16, 0, 2, 1, False), (70001, 40, 6, 1, 4, 2, 0, 0, 0, False)],
    ids=lambda s: f"T{s[0]}H{s[1]}k{s[5]}")
def test_many_tokens_with_short_rows(shape, dtype):
    """Several tokens share a workgroup; odd numbers of them leave its last groups without one."""
    test_dispatch(shape, dtype)
    test_dispatch_backward_and_combine(shape, dtype)
    test_combine_backward(shape, dtype)


def test_non_finite_rows_reach_only_their_token():
    """A row of NaN or infinities changes its own token only, also with a weight of 0 on another slot."""
    c = Case(20, 100, 8, 0, 8, 2, "bf16", seed=3)
    c.ys[c.row[4]] = float("inf")
    c.ys[c.row[7]] = float("nan")
    c.w[c.tok[10], c.slot[10] % c.k] = 0.0
    y = torch.zeros(20, 100, dtype=torch.bfloat16, device="cuda")
    B.moe_combine(c.desc, c.rows(c.ys)[0], c.s2r.cuda(), c.w.cuda(), y)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[c.tok[[4, 7]]] = True
    assert torch.equal(torch.isfinite(y.float()).all(1).cpu(), ~bad)


@pytest.mark.parametrize("T,H,k", [(37, 520, 4), (2100, 40, 8), (2049, 300, 16)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_weights_of_slots_without_a_row_are_not_used(T, H, k, bad):
    """Slots of experts elsewhere, or past the rows, may have weights that are not finite: dys, dw, y and the gradients
    of the other logits are bit for bit what they are with a weight of 0 there."""
    c = Case(T, H, 24, 5, 9, k, "bf16", max_rows=T * k // 4, seed=T)
    assert (c.offsets[-1] > c.cap) and not c.has.all()
    ids, s2r = c.ids.cuda(), c.s2r.cuda()
    x, ys = c.tokens(c.x)[0], c.rows(c.ys)[0]

    def run(fill):
        w = torch.where(c.has.reshape(T, k), c.w, torch.full((), fill)).cuda()
        y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        dys, dw, dl = torch.zeros_like(ys), torch.zeros(T, k, device="cuda"), torch.zeros(T, c.E, device="cuda")
        B.moe_combine(c.desc, ys, s2r, w, y)
        B.moe_combine_backward(c.desc, x, ys, s2r, w, dys, dw, topk_ids=ids, dlogits=dl)
        return y, dys, dw, dl

    (y, dys, dw, dl), (y0, dys0, dw0, dl0) = run(bad), run(0.0)
    assert torch.equal(y, y0) and torch.equal(dys, dys0) and torch.equal(dw, dw0)
    # a slot's own logit is weighted with its own weight; every other one is not touched by it
    own = torch.zeros(T, c.E, dtype=torch.bool)
    own[c.tok.new_tensor(np.repeat(np.arange(T), k))[~c.has], c.ids.reshape(-1)[~c.has].long()] = True
    assert torch.equal(dl.cpu()[~own], dl0.cpu()[~own])


def test_gradient_of_the_router_against_differences():
    """dlogits, dx and dw against central differences of the float64 formula of loss = <g, combine(dispatch(x))>
    through the softmax over the chosen logits."""
    T, H, E, k = 12, 33, 10, 3
    g = torch.Generator().manual_seed(8)
    logits = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    s2r = torch.from_numpy(sort_ref(ids, 2, 6)[3])
    up = torch.randn(T, H, generator=g).double()
    ys = torch.randn(T * k, H, generator=g).double()

    def loss(lg):
        w = torch.softmax(lg.gather(1, ids.long()), 1)
        r = s2r.reshape(T, k)
        v = torch.where((r >= 0)[..., None], ys[r.clamp(min=0).long()] * w[..., None], torch.zeros(()).double())
        return (v.sum(1) * up).sum(1)  # per token: tokens do not meet

    h = 1e-5
    want = torch.zeros(T, E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(1, E, dtype=torch.float64)
        step[0, e] = h
        want[:, e] = (loss(logits + step) - loss(logits - step)) / (2 * h)
    d = B.make_dispatch_desc(T, H, E, k, local_begin=2, num_local=6, dtype="f32")
    w = torch.softmax(logits.gather(1, ids.long()), 1).float().cuda()
    dys = torch.zeros(T * k, H, device="cuda")
    dw, dl = torch.zeros(T, k, device="cuda"), torch.zeros(T, E, device="cuda")
    B.moe_combine_backward(d, up.float().cuda(), ys.float().cuda(), s2r.cuda(), w, dys, dw, topk_ids=ids.cuda(), dlogits=dl)
    # differences: rounding 2^-53 |loss| / h plus h^2; kernel: about H 2^-24 of sums of a few tens
    assert (dl.double().cpu() - want).abs().max() < 1e-4
    # dw by differences is exact (the loss is linear in w): the rows' dot products
    r = s2r.reshape(T, k)
    rdw = torch.where(r >= 0, (ys[r.clamp(min=0).long()] * up[:, None]).sum(-1), torch.zeros(()).double())
    assert (dw.double().cpu() - rdw).abs().max() < 1e-4


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31 (a row stride of 2^30 elements)."""
    T, H, E, k = 2, 40, 2, 2
    ids = torch.tensor([[0, 1], [1, 0]], dtype=torch.int32)
    s2r = torch.from_numpy(sort_ref(ids, 0, 2)[3])
    stride = 1 << 30
    buf = torch.zeros(3 * stride + H, dtype=torch.bfloat16, device="cuda")
    rows = buf.as_strided((4, H), (stride, 1))
    d = B.make_dispatch_desc(T, H, E, k, dtype="bf16", row_stride=stride)
    x = torch.randn(T, H).to(torch.bfloat16)
    B.moe_dispatch(d, x.cuda(), s2r.cuda(), rows)
    slots = torch.arange(4)
    assert torch.equal(rows.cpu()[s2r.long()], x[slots // k])
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    B.moe_dispatch_backward(d, rows, s2r.cuda(), y)
    assert torch.equal(y.cpu(), x * 2)
    dys = torch.zeros_like(buf).as_strided((4, H), (stride, 1))
    dw = torch.zeros(T, k, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    B.moe_combine_backward(d, x.cuda(), rows, s2r.cuda(), w, dys, dw)
    assert torch.equal(dys.cpu()[s2r.long()], x[slots // k] / 2)
    ref = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
    assert ((dw.double().cpu() - ref).abs() <= 24 * U * ref).all()


def test_graph_replays_and_streams():
    """sort -> dispatch -> combine -> both gradients captured once, replayed on new inputs with eager calls
    between the replays, equal bit for bit to the eager results."""
    T, H, E, k, el = 333, 520, 32, 4, 20
    d = B.make_dispatch_desc(T, H, E, k, local_begin=6, num_local=el, dtype="bf16")
    ws, ws2 = B.alloc_sort_workspace(d), B.alloc_sort_workspace(d)

    def state(seed):
        g = torch.Generator().manual_seed(seed)
        return [make_ids(T, E, k, seed).cuda(), torch.softmax(torch.randn(T, k, generator=g), 1).cuda(),
                torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()]

    def outputs():
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return [z(n, dt=torch.int32) for n in (el, el + 1, T * k, T * k)] + [z(T * k, H), z(T, H), z(T, H), z(T * k, H),
                z(T, k, dt=torch.float32), z(T, E, dt=torch.float32)]

    def step(i, o, w_s, stream=None):
        ids, w, x = i
        B.moe_sort_tokens(d, ids, *o[:4], w_s, stream=stream)
        B.moe_dispatch(d, x, o[3], o[4], stream=stream)
        B.moe_combine(d, o[4], o[3], w, o[5], stream=stream)
        B.moe_dispatch_backward(d, o[4], o[3], o[6], stream=stream)
        B.moe_combine_backward(d, x, o[4], o[3], w, o[7], o[8], topk_ids=ids, dlogits=o[9], stream=stream)

    def eager(seed, stream=None):
        o = outputs()
        torch.cuda.synchronize()
        step(state(seed), o, ws2, stream)
        torch.cuda.synchronize()
        return o

    static, out = state(1), outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(static, out, ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, out, ws)
    for seed in (2, 3, 4):
        for a, b in zip(static, state(seed)):
            a.copy_(b)
        for v in out:
            v.zero_()
        eager(seed + 50)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager(seed, stream=s)):
            assert torch.equal(a, b)


def test_binding_refuses_what_does_not_fit():
    T, H, k = 8, 64, 2
    d = B.make_dispatch_desc(T, H, 4, k, dtype="bf16", max_rows=10)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    xs = torch.zeros(10, H, dtype=torch.bfloat16, device="cuda")
    m = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    B.moe_dispatch(d, x, m, xs)
    B.moe_dispatch(d, x, m, torch.zeros(16, H, dtype=torch.bfloat16, device="cuda"))  # more rows are fine
    wide = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device="cuda")
    for bad in [(x.float(), m, xs), (x[:4], m, xs), (x, m[:8], xs), (x, m.long(), xs), (x, m, xs[:9]),
                (wide[:, :H], m, xs), (x.t().contiguous().t(), m, xs), (x, m, xs[:1].expand(10, H)), (x, m.cpu(), xs)]:
        with pytest.raises(B.MoeError):
            B.moe_dispatch(d, *bad)
    w = torch.zeros(T, k, device="cuda")
    with pytest.raises(B.MoeError):
        B.moe_combine(d, xs, m, w.half(), x)
    with pytest.raises(B.MoeError):
        B.moe_combine_backward(d, x, xs, m, w, xs.clone(), w[:, :1], topk_ids=None)
    with pytest.raises(B.MoeError):
        B.moe_combine_backward(d, x, xs, m, w, xs.clone(), w.clone(), dlogits=torch.zeros(T, 4, device="cuda"))
