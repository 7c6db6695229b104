"""The layer at the sizes where its grouping changes kernels: one workgroup without atomics up to 6144 slots with at
most 63 local experts, one with them up to 2048 slots with at most 256, two launches while the padded chunk counts
are at most 32768 (512 chunks of 1024 slots with up to 63 local experts, 64 chunks with 256 to 511), else three.
Each kernel also writes the GEMMs' tile plan, which moe_layer reads and the three-call path derives by itself."""
import numpy as np
import pytest

from moe_expert_layer_amd import synth
from oracle import moe_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import gpu_util as G

CASES = [  # tokens, experts, first local, local, topk
    (1536, 70, 3, 63, 4), (1537, 70, 3, 63, 4),      # 6144 slots in one workgroup, 6148 in two launches
    (768, 70, 3, 64, 8),                             # 6144 slots, one local expert too many for the first
    (256, 300, 9, 256, 8), (257, 300, 9, 256, 8),    # 2048 slots in one workgroup, 2056 in two launches
    (256, 300, 9, 257, 8),                           # one local expert too many
    (4096, 256, 0, 32, 8),                           # a prefill chunk: two launches
    (8192, 320, 0, 300, 8), (8193, 320, 0, 300, 8),  # 64 chunks of 300 experts in two launches, 65 in three
    (32768, 70, 3, 63, 16), (32769, 70, 3, 63, 16),  # 512 chunks in two launches, 513 in three
    (100, 600, 20, 512, 8), (1000, 1024, 0, 1024, 4),  # more local experts than two launches take
]


@pytest.mark.parametrize("T,E,e0,EL,k", CASES)
def test_layer_at_the_boundaries_of_the_grouping(T, E, e0, EL, k):
    G.say(f"[grouping] T={T} E={E} e0={e0} EL={EL} k={k}")
    w = synth.shrink(synth.workload("prefill_zipf"), tokens=T, hidden=128, inter=128, num_experts=E, local_begin=e0,
                     num_local=EL, topk=k, seed=T + EL)
    inp = synth.generate(w)
    ids, tw = O.route(inp["logits"], k)
    ref = dict(zip(("counts", "offsets", "row_to_slot", "slot_to_row"), O.permute(ids, e0, EL)), topk_ids=ids, topk_w=tw)
    assert ref["counts"].max() > 4 * max(1, np.median(ref["counts"]))  # uneven: a wrong plan would show
    dev = G.upload(inp)
    for variant in (-1, 0, 1, 2):
        fused, split = G.run_layer(w, dev, variant), G.run_split(w, dev, variant)
        G.check_routing(fused, ref)
        G.check_routing(split, ref)
        assert np.array_equal(fused["y_bf16"], split["y_bf16"])
    if T <= 2000:
        want = O.layer(w, inp)["y_bf16"]
        assert G.rel_fro(G.bf16_to_f64(fused["y_bf16"]), G.bf16_to_f64(want)) <= 2e-3
