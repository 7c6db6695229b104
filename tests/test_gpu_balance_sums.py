"""The balance loss's sums over tokens, bit for bit where they are exact and within the roundings of their real order elsewhere, and
its workspace."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_expert_layer_amd import binding as B  # noqa: E402
from test_gpu_balance import DT, U, call_forward, dev, make_case, probabilities, spans  # noqa: E402


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,S,padded", [(1, 1, False), (33, 1, False), (700, 5, True), (1024, 1, False), (1025, 1, False),
                                        (4097, 1, True), (8193, 7, True), (20000, 1, False), (70001, 3, False)])
@pytest.mark.parametrize("E", [1, 2, 8, 16, 32, 64, 128, 256, 512, 1024])
def test_equal_logits_are_exact(E, T, S, padded, score):
    """Logits of 0 and a power of two of experts: every probability is 1 / E, the sums N / E and the loss of a sequence whose ids all count
    is 1, all exactly.  One token more or less in any piece shows."""
    k = min(E, 3)
    case = make_case(T, S, padded, T + E)
    r = np.random.RandomState(T)
    ids = r.randint(0, E, (T, k)).astype(np.int32)
    d = B.make_balance_desc(T, E, k, S, "bf16", score)
    out = call_forward(d, torch.zeros(T, E, dtype=torch.bfloat16, device="cuda"), dev(ids), case, False)
    n = np.array([len(t) for t in spans(case)])
    assert np.array_equal(out["tokens"].cpu().numpy(), n)
    assert np.array_equal(out["psum"].cpu().numpy().astype(np.float64), np.repeat(n[:, None] / E, E, 1))
    assert np.array_equal(out["balance"].cpu().numpy(), (n > 0).astype(np.float32))
    assert np.array_equal(out["counts"].cpu().numpy(), [np.bincount(ids[t].reshape(-1), minlength=E) for t in spans(case)])


def terms(T, E, longest):
    """How many additions stand between a token's probability and the sum of its sequence: those of a lane (its share of a chunk, or of the
    sequence where that is not cut), over the groups of a wave, over eight waves, and the rounding of the float64 sum."""
    lanes = 4 if E <= 16 else 8 if E <= 32 else 16 if E <= 512 else 64
    at_a_time = 8 * 64 // lanes
    piece = longest if T <= 1024 else min(longest, min(max(-(-T // 256), 32), 8192))
    return -(-piece // at_a_time) + 4 + 7 + 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,S,padded", [(1000, 31, 6, 4, True), (1024, 32, 8, 1, False), (1025, 33, 8, 6, True), (5000, 127, 8, 3, True),
                                            (20000, 256, 8, 1, False), (9000, 12, 2, 1, True), (2100, 1024, 8, 5, False)])
def test_sums_within_their_roundings(T, E, k, S, padded, dtype, score):
    g = torch.Generator().manual_seed(T + E)
    case = make_case(T, S, padded, T)
    logits = (3 * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)).to(DT[dtype])
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    softmax = score == "softmax"
    out = call_forward(B.make_balance_desc(T, E, k, S, dtype, score), logits.cuda(), ids.cuda(), case, softmax)
    longest = max(len(t) for t in spans(case)) if case["mask"] is None else T
    steps = terms(T, E, longest)
    for s, t in enumerate(spans(case)):
        p, lse, rel = probabilities(logits[t].double().numpy(), score)
        P, n = p.sum(0), max(len(t), 1)
        tol = (p * rel).sum(0) + P * steps * U + 1e-37
        assert (np.abs(out["psum"][s].cpu().double().numpy() - P) <= tol).all()
        c = np.bincount(ids[t].reshape(-1), minlength=E)
        f = E / (k * n ** 2)
        want = f * (c * P).sum()
        assert abs(float(out["balance"][s]) - want) <= f * (c * tol).sum() + want * 2 * U
        if softmax:
            # a logarithm of a sum that is off as its terms are, by their shares, a few roundings, and its square
            lerr = (p * rel).sum(1) + np.abs(lse) * 3 * U
            want = (lse ** 2).sum() / n
            assert abs(float(out["z"][s]) - want) <= (2 * np.abs(lse) * lerr).sum() / n + want * (steps + 2) * U


@pytest.mark.parametrize("T", [1, 1024, 1025, 8191, 8192, 8193, 10000, 16385, 70001])
def test_nothing_past_the_workspace(T):
    E, k, S = 20, 2, 3
    d = B.make_balance_desc(T, E, k, S)
    need = B.moe_balance_workspace_size(d)
    ws = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    case = make_case(T, S, False, T)
    x = torch.zeros(T, E, device="cuda")
    ids = torch.randint(0, E, (T, k), dtype=torch.int32).cuda()
    out = call_forward(d, x, ids, case, True, ws[:need])
    assert (ws[need:] == 0xa5).all()
    assert out["tokens"].cpu().tolist() == [len(t) for t in spans(case)]
