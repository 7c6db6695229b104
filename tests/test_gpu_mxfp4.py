"""MXFP4 quantisation, the values back, and the grouped product, against float64 on the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402
from moe_expert_layer_amd import synth  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


# ---- the format in numpy ----

def quantize_ref(v):
    """codes [M, K] and bytes [M, K/32] of float64 values: the nearest of the eight magnitudes, ties to the even code."""
    M, K = v.shape
    b = v.reshape(M, K // 32, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    ok = np.where(bad | (top == 0), 1.0, top)
    m, e = np.frexp(ok / 6.0)                       # ok / 6 is rounded; settle the exponent exactly
    e = np.where(m == 0.5, e - 1, e)                # 2^(e-1) itself
    e = np.where(6.0 * np.ldexp(1.0, e - 1) >= ok, e - 1, e)
    e = np.where(6.0 * np.ldexp(1.0, e) < ok, e + 1, e)
    e = np.clip(np.where(top == 0, 0, e), -127, 127)
    a = np.abs(np.where(bad[..., None], 0.0, b)) / np.ldexp(1.0, e)[..., None]
    d = np.abs(a[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    code = np.where(near.sum(-1) == 2, np.where(near[..., ::2].any(-1), near[..., ::2].argmax(-1) * 2, 0), near.argmax(-1))
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(M, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values_ref(code, byte):
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def nibbles(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def pack_ref(byte):
    M, G = byte.shape
    J, AM = (G + 3) // 4, (M + 3) // 4 * 4
    p = np.zeros((AM, 4 * J), np.uint8)
    p[:M, :G] = byte
    return np.ascontiguousarray(p.reshape(AM, J, 4).transpose(1, 0, 2)).view(np.int32).reshape(J, AM)


def scales_dev(byte, layout):
    return torch.from_numpy(pack_ref(byte) if layout == "packed" else byte).cuda()


# ---- quantisation ----

def special_rows(K, dtype):
    """A row per kind of block: every midpoint with a 6 beside it, powers of two, zeros, the smallest and largest
    values, infinities and NaN in one block among ordinary ones."""
    t = torch.finfo(DT[dtype])
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = []
    for scale in (1.0, 2.0 ** -9, 2.0 ** 9):
        r = np.zeros(K)
        r[0], r[1] = 6 * scale, -6 * scale
        for i, m in enumerate(mids):
            r[2 + 2 * i], r[3 + 2 * i] = m * scale, -m * scale
        rows.append(r)
    for top in (6.0, 4.0, 1.5, 1.0, 3.0):  # amax on a power of two and on the border 6 * 2^e
        r = np.zeros(K)
        r[5] = top
        r[9] = -top * (1 + t.eps)          # one step above the border
        rows.append(r)
        rows.append(np.where(np.arange(K) == 5, top, 0.0))
    rows.append(np.zeros(K))
    rows.append(-np.zeros(K))
    tiny = t.smallest_normal * t.eps
    rows.append(np.where(np.arange(K) % 3 == 0, tiny, -t.smallest_normal))
    rows.append(np.where(np.arange(K) % 3 == 0, t.max, -t.max / 7))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-3, 3, K)
        r[K // 2] = bad
        rows.append(r)
    return torch.from_numpy(np.stack(rows)).to(DT[dtype])


@pytest.mark.parametrize("layout", ["rows", "packed"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,pad,shift", [(1, 32, 0, 0), (3, 96, 0, 0), (29, 544, 7, 1), (129, 7168, 0, 0),
                                           (33, 160, 0, 3), (2500, 7168, 0, 0), (0, 64, 0, 0)])
def test_quantize_and_back(M, K, pad, shift, dtype, layout):
    g = torch.Generator().manual_seed(M + K)
    v = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(DT[dtype])
    sp = special_rows(K, dtype)
    if M >= len(sp):
        v[:len(sp)] = sp
    code, byte = quantize_ref(v.double().numpy())
    buf = torch.full((shift + M * (K + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    src = buf[shift:].view(M, K + pad)[:, :K]
    src.copy_(v)
    want_sf = pack_ref(byte) if layout == "packed" else byte
    codes = torch.full((M * (K // 2) + 64,), 77, dtype=torch.uint8, device="cuda")
    sf = torch.full((want_sf.size + 16,), 77, dtype=torch.int32 if layout == "packed" else torch.uint8, device="cuda")
    d = B.make_mxfp4_desc(M, K, dtype, layout, K + pad)
    B.moe_quantize_mxfp4(d, src, codes, sf)
    assert np.array_equal(codes.cpu().numpy()[:M * (K // 2)].reshape(M, K // 2), nibbles(code))
    assert np.array_equal(sf.cpu().numpy()[:want_sf.size].reshape(want_sf.shape), want_sf)
    assert (codes[M * (K // 2):] == 77).all() and (sf[want_sf.size:] == 77).all()
    want = torch.from_numpy(values_ref(code, byte)).float()
    for out in ("f32", "bf16", "f16"):
        back = torch.full((M, K + pad), 77.0, dtype=DT[out], device="cuda")
        B.moe_dequantize_mxfp4(d, codes, sf, back[:, :K], dtype=out)
        assert torch.equal(torch.nan_to_num(back[:, :K].cpu().float(), nan=1e30),
                           torch.nan_to_num(want.to(DT[out]).float(), nan=1e30))
        assert (back[:, K:] == 77).all()


def test_dequantize_every_scale_byte():
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    out = torch.zeros(256, 32, device="cuda")
    B.moe_dequantize_mxfp4(B.make_mxfp4_desc(256, 32, "f32"), torch.from_numpy(nibbles(code)).cuda(),
                           torch.from_numpy(byte).cuda(), out)
    want = torch.from_numpy(values_ref(code, byte).astype(np.float32))
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_packed_scales_are_what_pack_scales_writes():
    M, K = 37, 800
    v = torch.randn(M, K).to(torch.bfloat16).cuda()
    c = [torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = torch.zeros(M, K // 32, dtype=torch.uint8, device="cuda")
    packed = torch.full(((K // 32 + 3) // 4 * 40,), -1, dtype=torch.int32, device="cuda")
    again = packed.clone()
    B.moe_quantize_mxfp4(B.make_mxfp4_desc(M, K), v, c[0], rows)
    B.moe_quantize_mxfp4(B.make_mxfp4_desc(M, K, scale_layout="packed"), v, c[1], packed)
    B.moe_pack_scales(M, K // 32, rows, again)
    assert torch.equal(c[0], c[1]) and torch.equal(packed, again)


def test_quantized_weights_run_the_layer():
    """bfloat16 weights -> moe_quantize_mxfp4 -> moe_layer, against the oracle on the same bytes."""
    from oracle import moe_oracle as O
    from tests import gpu_util as G
    w = synth.shrink(synth.workload("mxfp4_large"), tokens=70, hidden=512, inter=256, num_experts=16, num_local=12,
                     local_begin=2, topk=4)
    inp = synth.generate(w)
    g = torch.Generator().manual_seed(5)
    for name, n, k in (("w1", 2 * w.inter, w.hidden), ("w2", w.hidden, w.inter)):
        v = (0.05 * torch.randn(w.num_local * n, k, generator=g)).to(torch.bfloat16).cuda()
        codes = torch.zeros(w.num_local * n, k // 2, dtype=torch.uint8, device="cuda")
        sf = torch.zeros(w.num_local * n, k // 32, dtype=torch.uint8, device="cuda")
        B.moe_quantize_mxfp4(B.make_mxfp4_desc(w.num_local * n, k), v, codes, sf)
        assert inp[name].size == codes.numel() and inp[name + "_sf"].size == sf.numel()
        inp[name] = codes.cpu().numpy().reshape(inp[name].shape)
        inp[name + "_sf"] = sf.cpu().numpy().reshape(inp[name + "_sf"].shape)
    got = G.run_layer(w, G.upload(inp))
    ref = O.layer(w, inp)
    assert G.rel_fro(G.bf16_to_f64(got["y_bf16"]), G.bf16_to_f64(ref["y_bf16"])) <= 2e-3


@pytest.mark.parametrize("layout", ["rows", "packed"])
def test_quantize_offsets_past_32_bits(layout):
    """Values of more than 2^32 elements (rows 2^16 + 1 elements apart) and codes of more than 2^31 bytes."""
    M, K, pad = 65600, 1 << 16, 1
    row = torch.randn(3, K, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    code, byte = quantize_ref(row.double().numpy())
    src = torch.zeros(M, K + pad, dtype=torch.bfloat16, device="cuda")[:, :K]
    at = [0, 65000, M - 1]
    src[at] = row.cuda()
    codes = torch.full((M, K // 2), 77, dtype=torch.uint8, device="cuda")
    sf = (torch.full((K // 128, M), 77, dtype=torch.int32, device="cuda") if layout == "packed"
          else torch.full((M, K // 32), 77, dtype=torch.uint8, device="cuda"))
    d = B.make_mxfp4_desc(M, K, "bf16", layout, K + pad)
    B.moe_quantize_mxfp4(d, src, codes, sf)
    got = sf[:, at].t().contiguous().view(torch.uint8) if layout == "packed" else sf[at]
    assert np.array_equal(codes[at].cpu().numpy(), nibbles(code)) and np.array_equal(got.cpu().numpy(), byte)
    zero = [1, 40000, M - 2]
    assert (codes[zero] == 0).all()
    src.fill_(77.0)
    B.moe_dequantize_mxfp4(d, codes, sf, src)
    assert torch.equal(src[at].cpu().double(), torch.from_numpy(values_ref(code, byte))) and (src[zero] == 0).all()


# ---- product ----

class Product:
    def __init__(self, sizes, N, K, rows=0, lo=126, hi=128, seed=0, la="packed", lb="packed", out="f32", pad=0, shift=0,
                 variant=-1):
        r = np.random.RandomState(seed)
        self.G, self.N, self.K = len(sizes), N, K
        self.off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.rows = rows or max(1, int(self.off[-1]))
        self.ac, self.bc = (r.randint(0, 16, (m, K)).astype(np.uint8) for m in (self.rows, self.G * N))
        self.ab, self.bb = (r.randint(lo, hi + 1, (m, K // 32)).astype(np.uint8) for m in (self.rows, self.G * N))
        self.la, self.lb, self.out, self.pad, self.shift = la, lb, out, pad, shift
        self.desc = B.make_mxfp4_gemm_desc(self.rows, N, K, self.G, out, la, lb, variant=variant,
                                           out_stride=N + pad if pad else 0)

    def args(self):
        return (torch.from_numpy(nibbles(self.ac)).cuda(), scales_dev(self.ab, self.la),
                torch.from_numpy(nibbles(self.bc)).cuda(), scales_dev(self.bb, self.lb),
                torch.from_numpy(self.off).cuda())

    def run(self, args=None, stream=None):
        ld = self.N + self.pad
        buf = torch.full((self.shift + self.rows * ld,), 77.0, dtype=DT[self.out], device="cuda")
        c = buf[self.shift:].view(self.rows, ld)[:, :self.N]
        B.moe_mxfp4_gemm(self.desc, *(args or self.args()), c, stream=stream)
        b = buf.float().cpu()
        assert (b[:self.shift] == 77).all()
        b = b[self.shift:].view(self.rows, ld)
        assert (b[:, self.N:] == 77).all() and (b[int(self.off[-1]):] == 77).all()
        return c.cpu()[:int(self.off[-1])]

    def ref(self, absolute=False):
        f = np.abs if absolute else (lambda v: v)
        a, b = f(values_ref(self.ac, self.ab)), f(values_ref(self.bc, self.bb)).reshape(self.G, self.N, self.K)
        parts = [a[self.off[e]:self.off[e + 1]] @ b[e].T for e in range(self.G)]
        return torch.from_numpy(np.concatenate(parts))


PRODUCTS = [  # sizes, N, K
    ([1], 1, 32), ([1], 4099, 7168), ([5], 15, 96), ([16], 17, 160), ([0, 3, 0], 33, 416), ([2, 0, 31, 1], 64, 512),
    ([33, 7], 130, 544), ([40, 100], 257, 1056), ([130, 0, 260, 3], 200, 2048), ([600], 520, 288), ([257, 255], 256, 4096)]
IDS = [f"G{len(s)}R{sum(s)}N{n}K{k}" for s, n, k in PRODUCTS]


@pytest.mark.parametrize("variant", [-1, 0, 1, 2])
@pytest.mark.parametrize("sizes,N,K", PRODUCTS, ids=IDS)
def test_product_exact(sizes, N, K, variant):
    """Scales in {1/2, 1, 2}: every product is a multiple of 2^-4 and every sum below 2^20, so float32 sums in any
    order are exact, and so must the results be.  Rows behind the last group stay as they were."""
    p = Product(sizes, N, K, rows=sum(sizes) + 5, seed=K + N, pad=3, shift=1, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [1, 2])
def test_product_more_tiles_than_workgroups(variant):
    p = Product([4000, 0, 700], 4100, 288, rows=4701, seed=5, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [-1, 0])
@pytest.mark.parametrize("sizes,N,K", [([9000], 2, 32), ([700, 0, 65, 3], 22, 64), ([130, 1000], 33, 512),
                                       ([1, 300, 5], 70, 544), ([1000, 600, 64], 40, 1056), ([5, 1], 5000, 96)])
def test_product_rows_spread_over_workgroups(sizes, N, K, variant):
    """Few columns, or K of one stretch: a group's rows go to several workgroups, or single waves."""
    p = Product(sizes, N, K, rows=sum(sizes) + 3, seed=K + N, pad=1, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes,N,K", PRODUCTS[1:9:2] + [([512, 256], 512, 1024)], ids=IDS[1:9:2] + ["whole"])
def test_product_rounding(sizes, N, K, out, variant):
    """Scales over 2^-7 .. 2^8: K / 64 matrix instructions each round the running sum (at most 2^-23 of the sum of
    magnitudes, whichever way they round), up to 16 partial sums are added, then one rounding to the type."""
    p = Product(sizes, N, K, lo=116, hi=127, seed=N, out=out, variant=variant)
    ref, mag = p.ref(), p.ref(absolute=True)
    t = torch.finfo(DT[out])
    tol = (K / 64 + 17) * 2.0 ** -23 * mag + ref.abs() * t.eps / 2 * (1 + 2.0 ** -10) + t.smallest_normal * t.eps / 2
    assert ((p.run().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("la", ["rows", "packed"])
@pytest.mark.parametrize("lb", ["rows", "packed"])
@pytest.mark.parametrize("sizes,N,K", [([3, 9], 50, 640), ([300, 10], 300, 1152)], ids=["few", "many"])
def test_product_scale_layouts(sizes, N, K, la, lb, variant):
    p = Product(sizes, N, K, la=la, lb=lb, seed=2, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("rows", [7, 600])
def test_product_nan_scales(rows, variant):
    """Scale byte 255 makes its row, or its column of its group, NaN, and nothing else."""
    p = Product([rows, rows], 70, 256, seed=4, variant=variant)
    p.ab[rows // 2, 3] = 255
    p.bb[70 + 11, 0] = 255
    got, ref = p.run(), p.ref()
    want = torch.zeros(2 * rows, 70, dtype=torch.bool)
    want[rows // 2] = True
    want[rows:, 11] = True
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got.double()[~want], ref[~want])


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("rows", [7, 600])
def test_product_garbage_past_k(rows, variant):
    """The padding of the last packed scale word is not part of the sum, whatever it holds."""
    p = Product([rows], 40, 288, seed=9, variant=variant)
    a, asf, b, bsf, off = p.args()
    for s in (asf, bsf):  # bytes 1 to 3 of the last word lie past K
        s[-1] |= torch.tensor(-256, dtype=torch.int32, device="cuda")  # 0xffffff00
    assert torch.equal(p.run((a, asf, b, bsf, off)).double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("rows", [20, 700])
def test_product_offsets_are_cut_to_the_rows(rows, variant):
    """Offsets outside [0, rows] or descending do not lead outside the tensors."""
    p3 = Product([rows, 0, 0], 48, 256, seed=1, variant=variant)
    a, asf, b, bsf, _ = p3.args()
    for off in ([-5, rows // 2, 3, 2 * rows], [0, 1 << 30, 5, -7], [rows, rows + 1, rows + 2, rows + 3]):
        c = torch.full((rows, 48), 77.0, device="cuda")
        B.moe_mxfp4_gemm(p3.desc, a, asf, b, bsf, torch.tensor(off, dtype=torch.int32, device="cuda"), c)
        torch.cuda.synchronize()
    av, bv = values_ref(p3.ac, p3.ab), values_ref(p3.bc, p3.bb).reshape(3, 48, 256)
    off = torch.tensor([0, rows, rows, rows], dtype=torch.int32, device="cuda")
    c = torch.full((rows, 48), 77.0, device="cuda")
    B.moe_mxfp4_gemm(p3.desc, a, asf, b, bsf, off, c)
    assert torch.equal(c.cpu().double(), torch.from_numpy(av @ bv[0].T))


def guarded(rows, ld, n, guard=300):
    """c [rows, n] of float32, its rows ld apart, with more than a tile's rows before and behind it, all 77; and what
    the rows around c and the padding of its own hold after a call."""
    buf = torch.full((rows + 2 * guard, ld), 77.0, device="cuda")

    def rest():
        b = buf.cpu()
        return torch.cat([b[:guard].reshape(-1), b[guard + rows:].reshape(-1), b[:, n:].reshape(-1)])

    return buf[guard:guard + rows, :n], rest


@pytest.mark.parametrize("variant", [-1, 0, 1, 2])
@pytest.mark.parametrize("K", [256, 1056])
@pytest.mark.parametrize("rows,off", [
    (250, [0, 130, 130, 200, 500, 520]),     # a group across the last row, one behind it
    (20, [0, 3, 19, 20, 21, 4000]),          # small groups, the last row's group ends with it
    (600, [0, 0, 1, 601, 601, 2 ** 31 - 1]),
    (300, [290, 295, 299, 300, 310, 310]),   # rows before the first group
    (300, [-400, -7, 5, 290, 300, 301]), (40, [40, 50, 60, 70, 80, 90]), (40, [-9, -8, -7, -6, 0, 0])])
def test_product_ascending_offsets_are_cut(rows, off, K, variant):
    """Ascending offsets reach past the tensors' rows (a sort that found more rows than there is room for) or start
    elsewhere: every row inside is its group's product, the others and everything around c stay as they were."""
    G, N = len(off) - 1, 48
    p = Product([rows] + [0] * (G - 1), N, K, seed=rows, variant=variant)
    a, asf, b, bsf, _ = p.args()
    desc = B.make_mxfp4_gemm_desc(rows, N, K, G, "f32", variant=variant, out_stride=N + 3)
    c, rest = guarded(rows, N + 3, N)
    B.moe_mxfp4_gemm(desc, a, asf, b, bsf, torch.tensor(off, dtype=torch.int32, device="cuda"), c)
    av, bv = values_ref(p.ac, p.ab), values_ref(p.bc, p.bb).reshape(G, N, K)
    want = np.full((rows, N), 77.0)
    for e in range(G):
        lo, hi = (min(max(o, 0), rows) for o in off[e:e + 2])
        want[lo:hi] = av[lo:hi] @ bv[e].T
    assert torch.equal(c.cpu().double(), torch.from_numpy(want))
    assert (rest() == 77).all()


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("rows", [20, 300, 700])
def test_product_descending_offsets_stay_inside_the_tensors(rows, variant):
    """Groups that overlap or end before they start: the results are anyone's, but nothing around c is written."""
    p = Product([rows, 0, 0], 48, 256, seed=1, variant=variant)
    a, asf, b, bsf, _ = p.args()
    desc = B.make_mxfp4_gemm_desc(rows, 48, 256, 3, "f32", variant=variant, out_stride=50)
    for off in ([-5, rows // 2, 3, 2 * rows], [0, 1 << 30, 5, -7], [rows, 0, rows, 0], [5, 0, rows + 9, 2]):
        c, rest = guarded(rows, 50, 48)
        B.moe_mxfp4_gemm(desc, a, asf, b, bsf, torch.tensor(off, dtype=torch.int32, device="cuda"), c)
        assert (rest() == 77).all()


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("rows", [3, 300])
def test_plain_product_without_offsets(rows, variant):
    p = Product([rows], 100, 512, seed=6, variant=variant)
    a, asf, b, bsf, _ = p.args()
    assert torch.equal(p.run((a, asf, b, bsf, None)).double(), p.ref())


def random_product(rows, N, K, G, sizes, seed):
    """Codes, scales over 2^-11 .. 2^0 and offsets, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda lo, hi, *n: torch.randint(lo, hi, n, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    words = lambda m: byte(116, 128, (K + 127) // 128, (m + 3) // 4 * 4, 4).view(torch.int32)  # noqa: E731
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
    return byte(0, 256, rows, K // 2), words(rows), byte(0, 256, G, N, K // 2), words(G * N), off


def product_of(args, rows, N, K, G, variant):
    c = torch.full((rows, N), 77.0, device="cuda")
    B.moe_mxfp4_gemm(B.make_mxfp4_gemm_desc(rows, N, K, G, "f32", variant=variant), *args, c)
    return c


@pytest.mark.parametrize("rows,G,N,K", [(1, 32, 4096, 7168), (8, 64, 4096, 7168), (4, 256, 512, 4096)])
def test_choice_of_kernel_with_fewer_rows_than_groups(rows, G, N, K):
    """Only the groups that have rows are read: the choice is the rows kernel's, by which the sum along K is split
    over waves.  Float32 results tell it from the tiles, which sum in one run."""
    sizes = np.bincount(np.random.RandomState(rows).permutation(G)[:rows], minlength=G)
    args = random_product(rows, N, K, G, sizes, 1)
    auto, by_rows, by_tiles = (product_of(args, rows, N, K, G, v) for v in (-1, 0, 2))
    assert torch.equal(auto, by_rows) and not torch.equal(auto, by_tiles)


def test_choice_of_kernel_with_many_groups():
    """From 682 groups on the LDS of a CU holds one workgroup of the 128 x 128 tiles instead of two, and the choice is
    the rows kernel's (told by its float32 results)."""
    rows, G, N, K = 2880, 720, 512, 4096
    args = random_product(rows, N, K, G, np.full(G, 4), 2)
    auto, by_rows, by_tiles = (product_of(args, rows, N, K, G, v) for v in (-1, 0, 2))
    assert torch.equal(auto, by_rows) and not torch.equal(auto, by_tiles)


@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("G", [681, 682, 1024])
def test_product_more_tiles_than_workgroups_of_many_groups(G, variant):
    r = np.random.RandomState(G)
    p = Product(list(r.randint(0, 7, G)), 130, 288, rows=6 * G, seed=G, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
def test_product_many_groups(variant):
    """1024 groups, most of them empty: the tile plan's largest size."""
    r = np.random.RandomState(3)
    sizes = np.where(r.rand(1024) < 0.8, 0, r.randint(1, 12, 1024))
    sizes[700] = 300
    p = Product(list(sizes), 20, 160, seed=8, variant=variant)
    assert torch.equal(p.run().double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
def test_products_on_two_streams_at_once(variant):
    ps = [Product([200, 0, 313], 300, 2048, seed=s, variant=variant) for s in (1, 2)]
    args = [p.args() for p in ps]
    out = [torch.zeros(p.rows, p.N, device="cuda") for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, a, c, s in zip(ps, args, out, streams):
            B.moe_mxfp4_gemm(p.desc, *a, c, stream=s)
    torch.cuda.synchronize()
    for p, c in zip(ps, out):
        assert torch.equal(c.cpu().double(), p.ref())


@pytest.mark.parametrize("variant", [0, 1, 2])
def test_product_scales_on_a_4_byte_boundary(variant):
    p = Product([90], 64, 256, seed=3, la="rows", lb="rows", variant=variant)
    a, asf, b, bsf, off = p.args()
    shifted = []
    for s in (asf, bsf):
        buf = torch.zeros(s.numel() + 4, dtype=torch.uint8, device="cuda")
        buf[4:] = s.reshape(-1)
        shifted.append(buf[4:])
    assert torch.equal(p.run((a, shifted[0], b, shifted[1], off)).double(), p.ref())


def test_product_offsets_past_32_bits():
    """Weights of more than 2^32 code bytes and results past 2^31 elements from the start."""
    G, N, K = 3, 1 << 17, 1 << 15  # 2^31 bytes of codes a group
    b = torch.zeros(G * N, K // 2, dtype=torch.uint8, device="cuda")
    b_sf = torch.full((K // 128, G * N), 0x7f7f7f7f, dtype=torch.int32, device="cuda")
    at = 2 * N + 100001
    b[at] = 0x22  # ones
    a = torch.full((4, K // 2), 0x44, dtype=torch.uint8, device="cuda")  # twos
    a_sf = torch.full((K // 128, 4), 0x7f7f7f7f, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 1, 2, 4], dtype=torch.int32, device="cuda")
    ld = 1 << 30
    c = torch.zeros(3 * ld + N, dtype=torch.float16, device="cuda").as_strided((4, N), (ld, 1))
    B.moe_mxfp4_gemm(B.make_mxfp4_gemm_desc(4, N, K, G, "f16", out_stride=ld), a, a_sf, b, b_sf, off, c)
    want = torch.zeros(4, N)
    want[2:, 100001] = float("inf")  # 2 K = 2^16 rounds to infinity in float16
    assert torch.equal(c.cpu().float(), want)


def test_product_graph_and_stream():
    small, large = Product([3, 0, 5], 200, 768, seed=1), Product([300, 0, 200], 264, 768, seed=2)
    for p in (small, large):
        args = p.args()
        c = torch.zeros(p.rows, p.N, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            B.moe_mxfp4_gemm(p.desc, *args, c)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.moe_mxfp4_gemm(p.desc, *args, c)
        other = Product([len(p.off)] * p.G, p.N, p.K, rows=p.rows, seed=7)
        for i in range(3):
            q = Product(list(np.diff(p.off)[::-1]) if i else list(np.diff(p.off)), p.N, p.K, seed=20 + i)
            for a, b in zip(args, q.args()):
                a.copy_(b)
            c.zero_()
            other.run()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.cpu().double(), q.ref())
            torch.cuda.synchronize()
            assert torch.equal(q.run(stream=s), c.cpu())


def test_binding_refuses_what_does_not_fit():
    p = Product([4, 5], 48, 256)
    a, asf, b, bsf, off = p.args()
    c = torch.zeros(9, 48, device="cuda")
    for bad in [(a[:8], asf, b, bsf, off, c), (a, asf[:1], b, bsf, off, c), (a, asf.view(torch.uint8), b, bsf, off, c),
                (a, asf, b[:90], bsf, off, c), (a, asf, b, bsf, off[:2], c), (a, asf, b, bsf, off.long(), c),
                (a, asf, b, bsf, off, c.half()), (a, asf, b, bsf, off, c[:8]), (a, asf, b, bsf, None, c),
                (a, asf, b, bsf, off.cpu(), c)]:
        with pytest.raises(B.MoeError):
            B.moe_mxfp4_gemm(p.desc, *bad)


# ---- together ----

def test_experts_from_their_parts():
    """Route -> sort -> 4-bit tokens in expert order -> gate/up product -> SwiGLU -> 4-bit -> down product ->
    weighted back into token order; every step against float64 on what the step before gave."""
    T, H, I, E, e0, el, k = 150, 512, 256, 16, 3, 10, 4
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g).cuda()

    def quant(v, layout="packed"):
        M, K = v.shape
        codes = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
        sf = (torch.zeros((K // 32 + 3) // 4, (M + 3) // 4 * 4, dtype=torch.int32, device="cuda") if layout == "packed"
              else torch.zeros(M, K // 32, dtype=torch.uint8, device="cuda"))
        B.moe_quantize_mxfp4(B.make_mxfp4_desc(M, K, scale_layout=layout), v, codes, sf)
        code, byte = quantize_ref(v.double().cpu().numpy())
        return codes, sf, values_ref(code, byte)

    w1, w1_sf, w1v = quant((0.05 * torch.randn(el * 2 * I, H, generator=g)).to(torch.bfloat16).cuda())
    w2, w2_sf, w2v = quant((0.05 * torch.randn(el * H, I, generator=g)).to(torch.bfloat16).cuda())
    w1v, w2v = w1v.reshape(el, 2 * I, H), w2v.reshape(el, H, I)

    top = torch.topk(logits, k, dim=1)
    ids, w = top.indices.to(torch.int32), torch.softmax(top.values, 1)
    cap = T * k
    d = B.make_dispatch_desc(T, H, E, k, local_begin=e0, num_local=el, max_rows=cap)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, off, r2s, s2r = i32(el), i32(el + 1), i32(cap), i32(cap)
    B.moe_sort_tokens(d, ids, counts, off, r2s, s2r, B.alloc_sort_workspace(d))
    # the sort agrees with the layer's own routing
    ld = B.make_desc(T, H, I, E, k, e0, el)
    o = [torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"), i32(el), i32(el + 1),
         i32(cap), i32(cap)]
    B.moe_route_permute(ld, logits, *o, B.alloc_workspace(ld))
    for a, b in zip((ids, counts, off, r2s, s2r), [o[0]] + o[2:]):
        assert torch.equal(a, b)
    # tokens quantised once, their codes and scales gathered as bytes; the same as quantising gathered rows
    xc, xsf, xv = quant(x, "rows")
    ac = torch.zeros(cap, H // 2, dtype=torch.uint8, device="cuda")
    asf = torch.zeros(cap, H // 32, dtype=torch.uint8, device="cuda")
    for src, dst in ((xc, ac), (xsf, asf)):
        B.moe_dispatch(B.make_dispatch_desc(T, src.shape[1], E, k, local_begin=e0, num_local=el, dtype="u8"), src, s2r, dst)
    xs = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    B.moe_dispatch(d, x, s2r, xs)
    R = int(off[-1])
    ac2, asf2, _ = quant(xs, "rows")
    assert torch.equal(ac2[:R], ac[:R]) and torch.equal(asf2[:R], asf[:R])
    rows = r2s.cpu().numpy()[:R] // k
    o_ = off.cpu().numpy()

    def product(a, a_sf, la, b, b_sf, n, kk, av, bv):
        c = torch.zeros(cap, n, dtype=torch.bfloat16, device="cuda")
        B.moe_mxfp4_gemm(B.make_mxfp4_gemm_desc(cap, n, kk, el, "bf16", la, "packed"), a, a_sf, b, b_sf, off, c)
        ref = np.concatenate([av[o_[e]:o_[e + 1]] @ bv[e].T for e in range(el)])
        mag = np.concatenate([np.abs(av[o_[e]:o_[e + 1]]) @ np.abs(bv[e]).T for e in range(el)])
        tol = np.abs(ref) * 2.0 ** -8 + (kk / 64 + 17) * 2.0 ** -23 * mag
        assert (np.abs(c.double().cpu().numpy()[:R] - ref) <= tol).all()
        return c

    gu = product(ac, asf, "rows", w1, w1_sf, 2 * I, H, xv[rows], w1v)
    h = (torch.nn.functional.silu(gu[:, :I].float()) * gu[:, I:].float()).to(torch.bfloat16)
    hc, hsf, hv = quant(h)
    ys = product(hc, hsf, "packed", w2, w2_sf, H, I, hv[:R], w2v)
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    B.moe_combine(d, ys, s2r, w, y)
    wr = w.double().cpu().reshape(-1).numpy()[r2s.cpu().numpy()[:R]]
    v = ys.double().cpu().numpy()[:R] * wr[:, None]
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(ref, rows, v)
    np.add.at(mag, rows, np.abs(v))
    assert (np.abs(y.double().cpu().numpy() - ref) <= np.abs(ref) * 2.0 ** -8 + (k + 2) * 2.0 ** -24 * mag + 1e-40).all()


def test_rows_past_the_capacity_are_dropped_in_every_step():
    """sort -> dispatch -> quantise -> product -> combine with tensors of fewer rows than the sort finds: the slots whose
    rows are there give what float64 gives for them, the others nothing, and nothing past the rows is written."""
    T, H, N, E, e0, el, k, cap = 120, 256, 96, 12, 2, 8, 4, 200
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    top = torch.topk(torch.randn(T, E, generator=g).cuda(), k, dim=1)
    ids, w = top.indices.to(torch.int32), torch.softmax(top.values, 1)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, off, r2s, s2r = i32(el), i32(el + 1), i32(T * k), i32(T * k)
    d = B.make_dispatch_desc(T, H, E, k, local_begin=e0, num_local=el, max_rows=cap)
    B.moe_sort_tokens(d, ids, counts, off, r2s, s2r, B.alloc_sort_workspace(d))
    o = off.cpu().numpy()
    cut = np.minimum(o, cap)
    straddled = int(np.searchsorted(o, cap, side="left")) - 1
    assert o[-1] > cap + 50 and o[straddled] < cap < o[straddled + 1] and straddled < el - 1
    xs = torch.full((cap + 300, H), 77.0, dtype=torch.bfloat16, device="cuda")
    B.moe_dispatch(d, x, s2r, xs[:cap])
    tok = r2s.cpu().numpy()[:cap] // k
    assert torch.equal(xs.cpu()[:cap], x.cpu()[tok]) and (xs[cap:] == 77).all()
    a = torch.zeros(cap, H // 2, dtype=torch.uint8, device="cuda")
    asf = torch.zeros(H // 128, cap, dtype=torch.int32, device="cuda")
    B.moe_quantize_mxfp4(B.make_mxfp4_desc(cap, H, scale_layout="packed"), xs[:cap], a, asf)
    av = values_ref(*quantize_ref(x.double().cpu().numpy()[tok]))
    bc, bb = np.random.RandomState(1).randint(0, 16, (el * N, H)).astype(np.uint8), np.full((el * N, H // 32), 122, np.uint8)
    bv = values_ref(bc, bb).reshape(el, N, H)
    ys, rest = guarded(cap, N, N)
    B.moe_mxfp4_gemm(B.make_mxfp4_gemm_desc(cap, N, H, el, "f32"), a, asf, torch.from_numpy(nibbles(bc)).cuda(),
                     scales_dev(bb, "packed"), off, ys)
    assert (rest() == 77).all()
    ref, mag = (np.concatenate([f(av[cut[e]:cut[e + 1]]) @ f(bv[e]).T for e in range(el)]) for f in (np.array, np.abs))
    # H / 64 matrix instructions round the running sum, up to 16 partial sums are added
    assert (np.abs(ys.double().cpu().numpy() - ref) <= (H / 64 + 17) * 2.0 ** -23 * mag).all()
    y = torch.full((T, N), 77.0, device="cuda")
    dn = B.make_dispatch_desc(T, N, E, k, local_begin=e0, num_local=el, dtype="f32", max_rows=cap)
    B.moe_combine(dn, ys, s2r, w, y)
    v = ys.double().cpu().numpy() * w.double().cpu().reshape(-1).numpy()[r2s.cpu().numpy()[:cap]][:, None]
    want, size = np.zeros((T, N)), np.zeros((T, N))
    np.add.at(want, tok, v)
    np.add.at(size, tok, np.abs(v))
    assert (np.abs(y.double().cpu().numpy() - want) <= (k + 2) * 2.0 ** -24 * size).all()
    assert (y.cpu()[torch.from_numpy(~np.isin(np.arange(T), tok))] == 0).all()
