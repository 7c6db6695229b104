"""The 4-bit product at real weights' numbers of groups.  Scales and zero points are brought in units of 32 or 64 groups, four at a
time where their number is a multiple of four and one by one where it is not: here both ways, over several units, in each of the
product's kernels (few rows by few weight rows or by many, and tiles of rows: above 64 rows an expert on average, or above 16 with
a workgroup for each CU), against exact sums of whole numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)

GROUPS = [  # form, group, zero points, groups of a row
    ("int4", 32, True, 64), ("int4", 32, False, 128), ("int4", 32, True, 224), ("int4", 32, True, 68), ("int4", 32, True, 131),
    ("int4", 64, True, 64), ("int4", 64, False, 128), ("int4", 64, True, 132), ("int4", 64, True, 113),
    ("int4", 128, True, 32), ("int4", 128, True, 56), ("int4", 128, False, 64), ("int4", 128, True, 128), ("int4", 128, True, 121),
    ("int4", 256, True, 64), ("int4", 256, True, 37), ("int4", 384, False, 36), ("int4", 512, True, 32),
    ("mxfp4", 32, False, 64), ("mxfp4", 32, False, 128), ("mxfp4", 32, False, 224), ("mxfp4", 32, False, 135)]
SIZES = {  # rows of each expert, weight rows of each expert (of both halves, with an activation)
    "few rows, 16 weight rows a workgroup": ([1, 0, 13], 100),
    "few rows, 32 weight rows a workgroup": ([3, 17, 1, 8], 2700),
    "few rows, many weight rows": ([1, 0, 16, 4, 2, 7], 22000),
    "tens of rows, many workgroups": ([20, 0, 33, 64, 17, 16, 5, 30], 4100),
    "many rows": ([130, 0, 71, 99], 300)}


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,group,zeros,ng", GROUPS)
@pytest.mark.parametrize("where", SIZES)
def test_groups_of_several_units(where, form, group, zeros, ng, dtype, act):
    """Rows of -2 to 2, weights up to 15 (6) and scales of 2^-2 to 2^2: every sum is a multiple of 2^-3 (2^-2) up to 48 K (120 K), which
    float32 holds for K up to 16384, so the results are the float64 ones; with an activation they enter it exactly, and its few
    roundings (an exponential, an addition, a division, two products) stay below 2^-20."""
    sizes, n2 = SIZES[where]
    K, E, R = ng * group, len(sizes), sum(sizes)
    N = n2 if act is None else n2 // 2
    assert K <= 16384
    g = torch.Generator(device="cuda").manual_seed(ng + K + N)
    b = torch.randint(0, 256, (E, n2, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scale, z = ["bf16", "f16", "f32"][ng % 3], None
    if form == "mxfp4":
        scale = "ue8m0"
        s = torch.randint(125, 130, (E, n2, ng), generator=g, dtype=torch.uint8, device="cuda")
    else:
        s = torch.exp2(torch.randint(-2, 3, (E, n2, ng), generator=g, device="cuda").float()).to(DT[scale])
        if zeros:
            z = torch.randint(0, 16, (E, n2, ng), generator=g, dtype=torch.uint8, device="cuda")
    x = torch.randint(-2, 3, (R, K), generator=g, device="cuda").to(DT[dtype])
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    c = torch.full((R + 1, N), 77.0, device="cuda")
    d = B.make_w4_gemm_desc(R, N, K, E, form, group, scale, zeros, dtype, "f32", act)
    B.moe_w4_gemm(d, x, b, s, z, offsets, c[:R])
    cols = torch.unique(torch.cat([torch.arange(20), torch.arange(N // 2, N // 2 + 20), torch.arange(N - 20, N)]))
    at = (cols if act is None else torch.cat([cols, N + cols])).cuda()
    got = c[:R, cols.cuda()].cpu().double()
    r0 = 0
    for e, n in enumerate(sizes):
        q = b[e, at].cpu()
        q = torch.stack([q & 15, q >> 4], -1).reshape(len(at), K)
        sc = s[e, at].cpu().double()
        if form == "mxfp4":
            w = E2M1[q.long()] * torch.exp2(sc - 127).repeat_interleave(group, -1)
        else:
            w = (q.double() - (8 if z is None else z[e, at].cpu().double().repeat_interleave(group, -1))) * sc.repeat_interleave(group, -1)
        y = x[r0:r0 + n].cpu().double() @ w.t()
        if act is None:
            assert torch.equal(got[r0:r0 + n], y), e
        else:
            gate, up = y.chunk(2, -1)
            want = gate * torch.sigmoid(gate) * up
            # where the sigmoid underflows float32 the result is 0
            assert ((got[r0:r0 + n] - want).abs() <= want.abs() * 2.0 ** -20 + 1e-30 * up.abs()).all(), e
        r0 += n
    assert (c[R] == 77).all()


@pytest.mark.parametrize("where", SIZES)
def test_subnormal_rows(where):
    """Rows of float16 numbers below its normal ones, multiples of 2^-24, are not taken as 0."""
    sizes, N = SIZES[where]
    K, group, E, R = 512, 128, len(sizes), sum(sizes)
    g = torch.Generator().manual_seed(N)
    q = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8)
    s = torch.ones(E, N, K // group)
    x = torch.randint(-1000, 1001, (R, K), generator=g).double() * 2.0 ** -24
    c = torch.empty(R, N, device="cuda")
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32).cuda()
    B.moe_w4_gemm(B.make_w4_gemm_desc(R, N, K, E, "int4", group, "f32", False, "f16", "f32"), x.half().cuda(),
                  (q[..., 0::2] | q[..., 1::2] << 4).contiguous().cuda(), s.cuda(), None, offsets, c)
    r0 = 0
    for e, n in enumerate(sizes):  # sums up to 1000 * 15 * 512 steps, below 2^23
        assert torch.equal(c[r0:r0 + n].cpu().double(), x[r0:r0 + n] @ (q[e].double() - 8).t())
        r0 += n
