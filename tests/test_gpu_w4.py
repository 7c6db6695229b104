"""4-bit weights with group scales: quantisation, the values back, and the product with 16-bit rows, against float64 on
the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {t: torch.finfo(DT[t]).eps / 2 for t in DT}  # a rounding, relative to the value
U = 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


# ---- quantisation ----

def quantize_ref(v, group, scale, zeros):
    """codes, scales and zero points of float32 values [M, K]; scales as float64 of the stored type"""
    M, K = v.shape
    b = v.double().reshape(M, K // group, group)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros((), dtype=torch.float64), b)
    lo, hi = b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15 if zeros else torch.maximum(-lo, hi) / 7).float().to(DT[scale]).double()
    bad = bad | ~torch.isfinite(s)
    some = (s > 0) & ~bad
    d = torch.where(some, s, 1.0)
    # float64 quotients of float32 numbers are never rounded to or over a border that they are not on
    z = torch.round(-lo / d).clamp(0, 15) if zeros else torch.full_like(s, 8.0)
    z = torch.where(some, z, 0.0 if zeros else 8.0)
    q = (torch.round(b / d[..., None]) + z[..., None]).clamp(0, 15)
    q = torch.where(some[..., None], q, z[..., None])
    return q.reshape(M, K).to(torch.uint8), torch.where(bad, float("nan"), s), z.to(torch.uint8)


def nibbles(q):
    return q[:, 0::2] | q[:, 1::2] << 4


def special(K, group, dtype):
    """Rows of borders: halves of steps, all-zero groups, one-sided ones, the smallest and largest values, infinities, NaN."""
    t = torch.finfo(DT[dtype])
    n = torch.arange(K, dtype=torch.float64)
    rows = []
    for step in (1.0, 0.125, 2.0 ** -7, 1.25):
        rows.append(((n % 31) - 15) / 2 * step * torch.where(n % group == 0, 0, 1) + torch.where(n % group == 0, 7 * step, 0.0))
        rows.append((n % 16) * step)
        rows.append(-((n % 31) / 2) * step)
    rows += [torch.zeros(K), -torch.zeros(K), torch.full((K,), 3.0), torch.full((K,), -5.0)]
    tiny = t.smallest_normal * t.eps
    rows += [(n % 8) * tiny, -(n % 3) * tiny * 5, (n % 16 - 8) * t.smallest_normal, torch.where(n % 3 == 0, t.max, -t.max / 7)]
    for x in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, K, dtype=torch.float64)
        r[K // 2] = x
        rows.append(r)
    return torch.stack([r.double() for r in rows]).to(DT[dtype])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,group,pad,shift", [(1, 32, 32, 0, 0), (3, 96, 32, 5, 1), (23, 2080, 32, 0, 0),
                                                 (77, 192, 64, 3, 3), (41, 1152, 128, 0, 1), (29, 384, 384, 1, 0),
                                                 (24, 2048, 256, 0, 0), (25, 8192, 8192, 7, 0), (700, 4096, 128, 0, 0),
                                                 (0, 64, 64, 0, 0)])
def test_quantize_and_back(M, K, group, pad, shift, dtype, scale, zeros):
    g = torch.Generator().manual_seed(M + K)
    v = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(DT[dtype])
    sp = special(K, group, dtype)
    if M > len(sp):
        v[:len(sp)] = sp
    q, s, z = quantize_ref(v.float(), group, scale, zeros)
    buf = torch.full((shift + M * (K + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    src = buf[shift:].view(M, K + pad)[:, :K]
    src.copy_(v)
    codes = torch.full((M * (K // 2) + 64,), 77, dtype=torch.uint8, device="cuda")
    n = M * (K // group)
    scales = torch.full((n + 16,), 77.0, dtype=DT[scale], device="cuda")
    zp = torch.full((n + 16,), 77, dtype=torch.uint8, device="cuda") if zeros else None
    d = B.make_int4_desc(M, K, group, dtype, scale, zeros, K + pad)
    B.moe_quantize_int4(d, src, codes, scales, zp)
    got = scales[:n].cpu().double().reshape(s.shape)
    assert torch.equal(torch.nan_to_num(got, nan=1e300), torch.nan_to_num(s, nan=1e300))
    if zeros:
        assert torch.equal(zp[:n].cpu().reshape(z.shape), z) and (zp[n:] == 77).all()
    assert torch.equal(codes[:M * (K // 2)].cpu().reshape(M, K // 2), nibbles(q))
    assert (codes[M * (K // 2):] == 77).all() and (scales[n:] == 77).all()
    # (q - z) s: a product of a whole number below 256 and a scale, rounded to float32 and then to the type
    want = ((q.reshape(M, K // group, group).double() - z.double()[..., None]).float() * s.float()[..., None]).reshape(M, K)
    for out in ("f32", "bf16", "f16"):
        back = torch.full((M, K + pad), 77.0, dtype=DT[out], device="cuda")
        B.moe_dequantize_int4(d, codes, scales, zp, back[:, :K], dtype=out)
        assert torch.equal(torch.nan_to_num(back[:, :K].cpu().float(), nan=1e30),
                           torch.nan_to_num(want.to(DT[out]).float(), nan=1e30))
        assert (back[:, K:] == 77).all()


def test_values_of_any_zero_byte():
    M, K = 256, 32
    q = torch.arange(M * K, dtype=torch.int64).reshape(M, K).mul(7).remainder(16).to(torch.uint8)
    z = torch.arange(M).to(torch.uint8).reshape(M, 1)
    s = torch.full((M, 1), 0.5)
    out = torch.empty(M, K, device="cuda")
    B.moe_dequantize_int4(B.make_int4_desc(M, K, 32, "f32", "f32", True), nibbles(q).cuda(), s.cuda(), z.cuda(), out)
    assert torch.equal(out.cpu(), (q.float() - z.float()) * 0.5)


# ---- the product ----

def weights(E, N, K, group, form, scale, zeros, g, whole):
    """Codes and scales, and the values they stand for in float64.  whole: scales are powers of two."""
    q = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8)
    b = (q[..., 0::2] | q[..., 1::2] << 4).contiguous()
    shape = (E, N, K // group)
    z = None
    if form == "mxfp4":
        s = torch.randint(125, 130, shape, generator=g, dtype=torch.uint8)
        w = torch.from_numpy(E2M1)[q.long()] * torch.exp2(s.double() - 127).repeat_interleave(group, -1)
        return b, s, z, w
    if whole:
        s = torch.exp2(torch.randint(-2, 3, shape, generator=g).float()).to(DT[scale])
    else:
        s = (0.02 * torch.exp(0.5 * torch.randn(shape, generator=g))).to(DT[scale])
    w = q.double()
    if zeros:
        z = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
        w = w - z.double().repeat_interleave(group, -1)
    else:
        w = w - 8
    return b, s, z, w * s.double().repeat_interleave(group, -1)


def act_ref(y, act, clamp, alpha, bias):
    if act is None:
        return y
    gate, up = y.chunk(2, -1)
    if act == "swigluoai":
        return torch.clamp(gate, max=clamp) * torch.sigmoid(alpha * torch.clamp(gate, max=clamp)) * (torch.clamp(up, -clamp, clamp) + bias)
    return gate * torch.sigmoid(gate) * up


def offsets_of(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32)


FORMS = [("int4", 32, False), ("int4", 32, True), ("int4", 64, True), ("int4", 64, False), ("int4", 128, True),
         ("int4", 128, False), ("int4", 256, True), ("int4", 384, False), ("mxfp4", 32, False)]
SIZES = [  # rows of each expert, N, K in groups
    ([1], 1, 1), ([1], 16, 4), ([3], 17, 5), ([0, 1, 0], 40, 3), ([16], 33, 7), ([17, 1, 0, 5], 70, 9), ([32, 33], 31, 6),
    ([64], 48, 12), ([65, 2], 100, 4), ([130], 20, 17), ([0, 0], 9, 2), ([300, 7, 80], 130, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,group,zeros", FORMS)
@pytest.mark.parametrize("sizes,N,kg", SIZES)
def test_whole_numbers_are_exact(sizes, N, kg, form, group, zeros, dtype):
    """Small whole rows and power-of-two scales: every partial sum is a multiple of 2^-4 below 2^20, which float32 holds, so
    the float32 results are the float64 ones."""
    K, E, R = kg * group, len(sizes), sum(sizes) + 3
    g = torch.Generator().manual_seed(N + K + R)
    scale = ["bf16", "f16", "f32"][(N + kg) % 3]
    b, s, z, w = weights(E, N, K, group, form, scale, zeros, g, True)
    apad, cpad = (0, 0) if N % 2 else (5, 3)
    abuf = torch.full((1 + R * (K + apad),), float("nan"), dtype=DT[dtype], device="cuda")
    a = abuf[1:].view(R, K + apad)[:, :K]
    x = torch.randint(-2, 3, (R, K), generator=g).double()
    a.copy_(x)
    a[sum(sizes):] = float("nan")  # rows of no expert
    d = B.make_w4_gemm_desc(R, N, K, E, form, group, "ue8m0" if form == "mxfp4" else scale, zeros, dtype, "f32",
                            a_stride=K + apad, out_stride=N + cpad)
    c = torch.full((R, N + cpad), 77.0, device="cuda")
    B.moe_w4_gemm(d, a, b.cuda(), s.cuda(), None if z is None else z.cuda(), offsets_of(sizes).cuda(), c[:, :N])
    want = torch.full((R, N), 77.0, dtype=torch.float64)
    r0 = 0
    for e, n in enumerate(sizes):
        want[r0:r0 + n] = x[r0:r0 + n] @ w[e].t()
        r0 += n
    assert torch.equal(c[:, :N].cpu().double(), want)
    assert (c[:, N:] == 77).all()


LARGE = [  # rows of each expert, N, K in blocks of 128: enough weight rows for long runs of few rows, and for tiles of many
    ([1], 98500, 3), ([3, 0, 8, 16], 24700, 5), ([1, 1], 49300, 17), ([17, 64, 0, 33, 1, 49, 20, 16], 4100, 5),
    ([200, 1, 66], 1000, 17), ([40, 0, 0, 500], 8300, 3), ([12] * 5, 1700, 18)]


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,group,zeros", FORMS)
@pytest.mark.parametrize("sizes,N,blocks", LARGE)
def test_large_shapes(sizes, N, blocks, form, group, zeros, dtype, act):
    """Shapes with many weight rows, some of whose columns are checked; whole numbers again, exact before the activation.  Groups of 32 and 64
    end inside a block of 128."""
    K = blocks * 128 + (group if group < 128 else 0)
    if group > 128:
        K = -(-K // group) * group
    E, R = len(sizes), sum(sizes)
    N = N if act is None else (N + 1) // 2
    n2 = N if act is None else 2 * N
    g = torch.Generator(device="cuda").manual_seed(N + K)
    scale = ["bf16", "f16", "f32"][(len(sizes) + blocks) % 3]
    b = torch.randint(0, 256, (E, n2, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    shape, z = (E, n2, K // group), None
    if form == "mxfp4":
        scale = "ue8m0"
        s = torch.randint(125, 130, shape, generator=g, dtype=torch.uint8, device="cuda")
    else:
        s = torch.exp2(torch.randint(-2, 3, shape, generator=g, device="cuda").float()).to(DT[scale])
        if zeros:
            z = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8, device="cuda")
    x = torch.randint(-2, 3, (R, K), generator=g, device="cuda").to(DT[dtype])
    c = torch.full((R + 1, N), 77.0, device="cuda")
    d = B.make_w4_gemm_desc(R, N, K, E, form, group, scale, zeros, dtype, "f32", act)
    B.moe_w4_gemm(d, x, b, s, z, offsets_of(sizes).cuda(), c[:R])
    cols = torch.unique(torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 70), torch.arange(N - 40, N)]))
    at = (cols if act is None else torch.cat([cols, N + cols])).cuda()
    got = c[:R, cols.cuda()].cpu().double()
    r0 = 0
    for e, n in enumerate(sizes):
        q = b[e, at].cpu()
        q = torch.stack([q & 15, q >> 4], -1).reshape(len(at), K)
        sc = s[e, at].cpu()
        if form == "mxfp4":
            w = torch.from_numpy(E2M1)[q.long()] * torch.exp2(sc.double() - 127).repeat_interleave(group, -1)
        else:
            w = (q.double() - (8 if z is None else z[e, at].cpu().double().repeat_interleave(group, -1))) * \
                sc.double().repeat_interleave(group, -1)
        y = x[r0:r0 + n].cpu().double() @ w.t()
        if act is None:
            assert torch.equal(got[r0:r0 + n], y), e
        else:
            # the sums are exact; the activation takes an exponential, an addition, a division and a product, a few roundings each;
            # where it underflows float32 it is 0
            want = act_ref(y, act, 0, 0, 0)
            assert ((got[r0:r0 + n] - want).abs() <= want.abs() * 2.0 ** -20 + 1e-30 * y.chunk(2, -1)[1].abs()).all(), e
        r0 += n
    assert (c[R] == 77).all()


def sum_bound(x, w, s, z, form, group):
    """How far the float32 sums may be off: the codes' products and the zero point's are summed apart, |x| (q + z) together at most, each
    sum of a group takes `group` additions, then come a product and an addition for each group, and the waves'."""
    K = x.shape[-1]
    sd = s.double() if form == "int4" else torch.exp2(s.double() - 127)
    ax = x.abs()
    if form == "int4":
        zz = torch.full(s.shape, 8.0, dtype=torch.float64) if z is None else z.double()
        inner = ax @ ((15 + zz) * sd).repeat_interleave(group, -1).t()
    else:
        inner = ax @ w.abs().t()
    return inner * (group + 4) * U + (ax @ w.abs().t()) * (K // group + 20) * U


@pytest.mark.parametrize("act", [None, "swiglu", "swigluoai"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,group,zeros,scale", [("int4", 32, True, "f32"), ("int4", 64, False, "f16"),
                                                    ("int4", 128, True, "bf16"), ("mxfp4", 32, False, "ue8m0")])
@pytest.mark.parametrize("sizes,N,K", [([1], 37, 1408), ([5, 0, 20, 1], 100, 2048), ([50, 3], 33, 640)])
def test_product(sizes, N, K, form, group, zeros, scale, dtype, out, act):
    E, R = len(sizes), sum(sizes)
    g = torch.Generator().manual_seed(N + K)
    b, s, z, w = weights(E, N * (1 if act is None else 2), K, group, form, scale, zeros, g, False)
    if form == "mxfp4":
        s = s - 7
        w = w / 128
    x = torch.randn(R, K, generator=g).to(DT[dtype])
    clamp, alpha, bias = 3.0, 1.702, 1.0
    d = B.make_w4_gemm_desc(R, N, K, E, form, group, scale, zeros, dtype, out, act, clamp, alpha, bias)
    c = torch.full((R, N), 77.0, dtype=DT[out], device="cuda")
    B.moe_w4_gemm(d, x.cuda(), b.cuda(), s.cuda(), None if z is None else z.cuda(), offsets_of(sizes).cuda(), c)
    r0 = 0
    for e, n in enumerate(sizes):
        xe = x[r0:r0 + n].double()
        y = xe @ w[e].t()
        err = sum_bound(xe, w[e], s[e], None if z is None else z[e], form, group)
        want = act_ref(y, act, clamp, alpha, bias)
        if act is not None:
            # |d act / d gate| <= 1.2 max(1, alpha) |up|, |d act / d up| <= |gate|; and the function's own few roundings
            gate, up = y.chunk(2, -1)
            eg, eu = err.chunk(2, -1)
            if act == "swigluoai":
                up = up.clamp(-clamp, clamp) + bias
            err = 2.1 * (up.abs() + eu) * eg + (gate.abs() + eg) * eu + want.abs() * 2.0 ** -20
        tol = err + want.abs() * HALF[out] * 1.01 + (2.0 ** -25 if out == "f16" else 0)
        off = (c[r0:r0 + n].cpu().double() - want).abs() - tol
        assert (off <= 0).all(), (e, off.max())
        r0 += n


def test_infinities_and_nan():
    """An infinite or NaN activation reaches its own row alone, as the sums by the definition have it; so does a NaN scale
    its column."""
    K, N, R = 256, 20, 5
    g = torch.Generator().manual_seed(3)
    for dtype in ("bf16", "f16"):
        for form, group in (("int4", 32), ("int4", 128), ("mxfp4", 32)):
            b, s, z, w = weights(1, N, K, group, form, "f32", form == "int4", g, True)
            x = torch.randint(-2, 3, (R, K), generator=g).to(DT[dtype])
            x[1, 70], x[2, 3], x[3, 9], x[3, 200] = float("inf"), float("nan"), float("inf"), -float("inf")
            d = B.make_w4_gemm_desc(R, N, K, 1, form, group, "ue8m0" if form == "mxfp4" else "f32", z is not None, dtype, "f32")
            c = torch.empty(R, N, device="cuda")
            zd = None if z is None else z.cuda()
            B.moe_w4_gemm(d, x.cuda(), b.cuda(), s.cuda(), zd, None, c)
            want = (x.double()[:, None, :] * w[0][None]).sum(-1)
            assert torch.equal(torch.nan_to_num(c.cpu().double(), nan=1e300, posinf=1e301, neginf=-1e301),
                               torch.nan_to_num(want, nan=1e300, posinf=1e301, neginf=-1e301))
            s[0, 4, 1] = 255 if form == "mxfp4" else float("nan")
            x = torch.ones(R, K, dtype=DT[dtype])
            B.moe_w4_gemm(d, x.cuda(), b.cuda(), s.cuda(), zd, None, c)
            bad = torch.isnan(c).cpu()
            assert bad[:, 4].all() and bad.sum() == R


def test_any_zero_byte():
    """Zero points up to 255, as bytes may be."""
    K, N, R, group = 128, 256, 3, 32
    g = torch.Generator().manual_seed(6)
    q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 256, (N, K // group), generator=g, dtype=torch.uint8)
    z[:, 0] = torch.arange(256).to(torch.uint8)
    s = torch.ones(N, K // group)
    x = torch.randint(-2, 3, (R, K), generator=g)
    want = x.double() @ (q.double() - z.double().repeat_interleave(group, 1)).t()
    for dtype in ("bf16", "f16"):
        c = torch.empty(R, N, device="cuda")
        B.moe_w4_gemm(B.make_w4_gemm_desc(R, N, K, 1, "int4", group, "f32", True, dtype, "f32"), x.to(DT[dtype]).cuda(),
                      nibbles(q).cuda(), s.cuda(), z.cuda(), None, c)
        assert torch.equal(c.cpu().double(), want)


def test_rows_past_the_tensor_and_cut_offsets():
    """Offsets of a sort that found more rows than the tensors hold: the rows that are there are computed."""
    K, N, E, R = 128, 24, 4, 30
    g = torch.Generator().manual_seed(9)
    b, s, z, w = weights(E, N, K, 64, "int4", "bf16", True, g, True)
    x = torch.randint(-2, 3, (R, K), generator=g)
    off = torch.tensor([0, 10, 25, 60, 2 ** 31 - 1], dtype=torch.int32)
    c = torch.full((R + 2, N), 77.0, device="cuda")
    d = B.make_w4_gemm_desc(R, N, K, E, "int4", 64, "bf16", True, "bf16", "f32")
    B.moe_w4_gemm(d, x.bfloat16().cuda(), b.cuda(), s.cuda(), z.cuda(), off.cuda(), c[:R])
    want = torch.cat([x[:10].double() @ w[0].t(), x[10:25].double() @ w[1].t(), x[25:].double() @ w[2].t()])
    assert torch.equal(c[:R].cpu().double(), want) and (c[R:] == 77).all()


def test_far_weights():
    """Weight rows past 2^31 bytes of codes, and rows of A far apart."""
    E, N, K = 3, 4096, 1 << 19
    b = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.ones(E, N, 1, dtype=torch.float32, device="cuda")
    b[2, N - 1, -1] = 0x93  # codes 3 and 9 of the last two
    x = torch.zeros(2, K, dtype=torch.bfloat16)
    x[:, -2], x[:, -1] = 2, 5
    big = torch.empty(3 * (1 << 30), dtype=torch.bfloat16, device="cuda")
    a = big.as_strided((2, K), ((1 << 31) + 64, 1))
    a.copy_(x)
    c = torch.zeros(2, N, device="cuda")
    d = B.make_w4_gemm_desc(2, N, K, E, "int4", K, "f32", False, "bf16", "f32", a_stride=(1 << 31) + 64)
    B.moe_w4_gemm(d, a, b, s, None, torch.tensor([0, 0, 1, 2], dtype=torch.int32).cuda(), c)
    want = torch.full((2, N), -56.0)
    want[1, N - 1] = 2 * -5 + 5 * 1
    assert torch.equal(c.cpu(), want)


def test_an_expert_layer():
    """As a decoding step uses them: weights quantised, tokens routed and sorted, sent through gate, up and down
    projections, brought back with their weights, and the router's loss and gradient beside that of the weights; captured
    once and replayed with other work between."""
    T, H, I, E, k, group = 50, 256, 128, 8, 3, 64
    g = torch.Generator().manual_seed(12)
    logits = (torch.randn(T, E, generator=g) + torch.randn(E, generator=g))
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    w = {}
    for name, (n, kk) in {"up": (2 * I, H), "down": (H, I)}.items():
        v = (torch.randn(E * n, kk, generator=g) / kk ** 0.5).bfloat16().cuda()
        codes = torch.empty(E, n, kk // 2, dtype=torch.uint8, device="cuda")
        sc = torch.empty(E, n, kk // group, dtype=torch.bfloat16, device="cuda")
        zp = torch.empty(E, n, kk // group, dtype=torch.uint8, device="cuda")
        d = B.make_int4_desc(E * n, kk, group, "bf16", "bf16", True)
        B.moe_quantize_int4(d, v, codes, sc, zp)
        vals = torch.empty(E * n, kk, device="cuda")
        B.moe_dequantize_int4(d, codes, sc, zp, vals, dtype="f32")
        w[name] = (codes, sc, zp, vals.reshape(E, n, kk).cpu().double())
    top, ids = torch.topk(logits, k)
    weight = torch.softmax(top, 1)
    dd = B.make_dispatch_desc(T, H, E, k)
    up = B.make_w4_gemm_desc(T * k, I, H, E, "int4", group, "bf16", True, "bf16", "bf16", "swiglu")
    down = B.make_w4_gemm_desc(T * k, H, I, E, "int4", group, "bf16", True, "bf16", "bf16")
    bd = B.make_balance_desc(T, E, k)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    maps = [i32(E), i32(E + 1), i32(T * k), i32(T * k)]
    o = {"xs": torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"),
         "h": torch.zeros(T * k, I, dtype=torch.bfloat16, device="cuda"),
         "ys": torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"),
         "y": torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), "counts": i32(1, E), "tokens": i32(1),
         "psum": torch.zeros(1, E, device="cuda"), "balance": torch.zeros(1, device="cuda"),
         "dys": torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"), "dw": torch.zeros(T, k, device="cuda"),
         "dl": torch.zeros(T, E, device="cuda")}
    dy = torch.randn(T, H, generator=g).bfloat16().cuda()
    ids32, wdev, ldev, one = ids.to(torch.int32).cuda(), weight.cuda(), logits.cuda(), torch.ones(1, device="cuda")
    sws, bws = B.alloc_sort_workspace(dd), B.alloc_balance_workspace(bd)

    def step():
        B.moe_sort_tokens(dd, ids32, *maps, sws)
        B.moe_dispatch(dd, x, maps[3], o["xs"])
        B.moe_w4_gemm(up, o["xs"], *w["up"][:3], maps[1], o["h"])
        B.moe_w4_gemm(down, o["h"], *w["down"][:3], maps[1], o["ys"])
        B.moe_combine(dd, o["ys"], maps[3], wdev, o["y"])
        B.moe_balance_loss(bd, ldev, ids32, o["counts"], o["tokens"], o["psum"], o["balance"], bws)
        B.moe_combine_backward(dd, dy, o["ys"], maps[3], wdev, o["dys"], o["dw"], topk_ids=ids32, dlogits=o["dl"])
        B.moe_balance_loss_backward(bd, ldev, o["counts"], o["tokens"], one, o["dl"], add=o["dl"])

    step()
    torch.cuda.synchronize()
    first = {n: v.clone() for n, v in o.items()}
    assert torch.equal(o["counts"][0], maps[0])
    # in float64: rounded to bf16 where the operators' results are
    xd, y = x.cpu().double(), torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    dl = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        rows, rb = [], []
        for j in range(k):
            e = int(ids[t, j])
            u = w["up"][3][e] @ xd[t]
            h = (u[:I] * torch.sigmoid(u[:I]) * u[I:])
            dwn = w["down"][3][e]
            rows.append(dwn @ h)
            # h and the result are rounded to bf16 (half a step), sums in float32: 2^-12 of the terms' size covers them
            eu = (w["up"][3][e].abs() @ xd[t].abs()) * 2.0 ** -12
            eh = h.abs() * 2.0 ** -8 + 2.1 * u[I:].abs() * eu[:I] + u[:I].abs() * eu[I:] + 2.1 * eu[:I] * eu[I:]
            rb.append(dwn.abs() @ eh + (dwn.abs() @ h.abs()) * 2.0 ** -12 + rows[-1].abs() * 2.0 ** -8)
        rows, rb, wt = torch.stack(rows), torch.stack(rb), weight[t].double()
        y[t] = (wt[:, None] * rows).sum(0)
        bound[t] = (wt[:, None] * rb).sum(0) + y[t].abs() * 2.0 ** -8
    assert ((o["y"].cpu().double() - y).abs() <= bound).all()
    # the router's gradient: of the weights' softmax, from the rows that the combine read, and of the balance loss
    ys = o["ys"].cpu().double()
    s2r = maps[3].cpu().reshape(T, k).long()
    dw = (ys[s2r] * dy.cpu().double()[:, None]).sum(-1)
    wt = weight.double()
    gl = wt * (dw - (wt * dw).sum(1, keepdim=True))
    dl.scatter_add_(1, ids, gl)
    p = torch.softmax(logits.double(), 1)
    c = torch.bincount(ids.reshape(-1), minlength=E).double()
    dl += E / (k * T * T) * p * (c - (p @ c)[:, None])
    size = (ys[s2r].abs() * dy.cpu().double().abs()[:, None]).sum(-1).max() + 1  # of the dot products' terms
    assert (o["dl"].cpu().double() - dl).abs().max() <= 64 * 2.0 ** -24 * size
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for v in list(o.values()) + [sws, bws]:
            v.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[n], first[n]) for n in o)


def test_the_layers_mxfp4_weights():
    """What moe_quantize_mxfp4 makes for moe_layer (row-major scales) goes into the product as it is."""
    N, K, R = 50, 256, 4
    g = torch.Generator().manual_seed(2)
    v = torch.randn(N, K, generator=g).bfloat16().cuda()
    md = B.make_mxfp4_desc(N, K, "bf16", "rows")
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(md, v, codes, sf)
    vals = torch.empty(N, K, device="cuda")
    B.moe_dequantize_mxfp4(md, codes, sf, vals, dtype="f32")
    x = torch.randn(R, K, generator=g).bfloat16()
    c = torch.empty(R, N, device="cuda")
    B.moe_w4_gemm(B.make_w4_gemm_desc(R, N, K, 1, "mxfp4", 32, "ue8m0", False, "bf16", "f32"), x.cuda(), codes, sf, None, None, c)
    w = vals.cpu().double()
    tol = (x.double().abs() @ w.abs().t()) * 64 * U
    assert ((c.cpu().double() - x.double() @ w.t()).abs() <= tol).all()


def test_streams_and_runs_give_the_same_bits():
    E, N, K, R = 4, 200, 1024, 40
    g = torch.Generator().manual_seed(1)
    b, s, z, w = (None if t is None else t.cuda() for t in weights(E, N, K, 128, "int4", "bf16", True, g, False))
    x, off = torch.randn(R, K, generator=g).bfloat16().cuda(), offsets_of([3, 20, 0, 17]).cuda()
    d = B.make_w4_gemm_desc(R, N, K, E, "int4", 128, "bf16", True, "bf16", "f32")
    outs = [torch.zeros(R, N, device="cuda") for _ in range(3)]
    B.moe_w4_gemm(d, x, b, s, z, off, outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, c in zip(streams, outs[1:]):
            B.moe_w4_gemm(d, x, b, s, z, off, c, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_refusals():
    E, N, K, R = 2, 24, 256, 8
    g = torch.Generator().manual_seed(1)
    b, s, z, _ = (t.cuda() for t in weights(E, N, K, 128, "int4", "bf16", True, g, False))
    x, off, c = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda"), offsets_of([4, 4]).cuda(), torch.zeros(R, N, device="cuda")
    d = B.make_w4_gemm_desc(R, N, K, E, "int4", 128, "bf16", True, "bf16", "f32")
    B.moe_w4_gemm(d, x, b, s, z, off, c)
    for args in ((x.half(), b, s, z, off, c), (x[:, :128], b, s, z, off, c), (x[:7], b, s, z, off, c), (x, b[:1], s, z, off, c),
                 (x, b.int(), s, z, off, c), (x, b, s.half(), z, off, c), (x, b, s[:1], z, off, c), (x, b, s, None, off, c),
                 (x, b, s, z[:1], off, c), (x, b, s, z.int(), off, c), (x, b, s, z, off[:2], c), (x, b, s, z, off.long(), c),
                 (x, b, s, z, None, c), (x, b, s, z, off, c.half()), (x, b, s, z, off, c[:, :20]), (x, b.cpu(), s, z, off, c),
                 (x, b.transpose(1, 2), s, z, off, c)):
        with pytest.raises(B.MoeError):
            B.moe_w4_gemm(d, *args)
    v, sc, zp = torch.zeros(4, 128, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.uint8, device="cuda")
    codes = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    qd = B.make_int4_desc(4, 128, 128, "f32", "f32", True)
    B.moe_quantize_int4(qd, v, codes, sc, zp)
    for args in ((v.half(), codes, sc, zp), (v[:3], codes, sc, zp), (v, codes[:3], sc, zp), (v, codes, sc[:3], zp),
                 (v, codes, sc.half(), zp), (v, codes, sc, zp[:3]), (v, codes, sc, None), (v, codes, sc, sc)):
        with pytest.raises(B.MoeError):
            B.moe_quantize_int4(qd, *args)
        with pytest.raises(B.MoeError):
            B.moe_dequantize_int4(qd, *args[1:], args[0])
