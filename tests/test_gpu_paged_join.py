"""Units that the division cuts, joined by the kernel itself or by the join
kernel, with head slices, cut by themselves and on the line."""
import numpy as np
import pytest
import torch

from tests.paged_util import Batch, attend, check, decode, status

pytestmark = pytest.mark.gpu

SHORT = [1 + i % 5 for i in range(35)]
# name: case, whether the decode kernel joins inside.  It does where no unit can be
# cut in more than four: tables of at most 640 rows (the longest unit is 11 long with
# what it costs besides its steps, a part at least 4), or 99 and more head units.
CASES = {
    "own_cut": (Batch(kv=[600, 1, 300, 77, 590], hk=1, g=6, page=16), True),
    "own_cut_slices": (Batch(kv=[600, 333], hk=1, g=17, page=16), True),
    "own_cut_slices_d64": (Batch(kv=[600] * 2, hk=2, g=33, D=64, page=16), True),
    "line": (Batch(kv=[600] + SHORT, hk=8, g=2, D=64, page=16), True),
    "line_slices": (Batch(kv=SHORT[:20] + [600] + SHORT[20:], hk=4, g=17, D=64, page=16), True),
    "many_heads": (Batch(kv=[2100, 50], hk=100, g=1, D=64, page=64), True),
    "many_slices": (Batch(kv=[2000], hk=50, g=17, D=64, page=64), True),
    "behind_slices": (Batch(kv=[1500] * 2, hk=2, g=17, page=32), False),
}


def division(s, ctas):
    """Part boundaries inside a unit's steps, and whether units are cut by themselves,
    from the records that the division leaves in the workspace (paged_common.cuh,
    PlanRec: twelve ints, the fourth the place inside the unit, the seventh the length
    of the part, the eighth what units cost besides their steps, 0 for cuts by
    themselves)."""
    rec = s["ws"][256:256 + 48 * ctas].view(torch.int32).view(ctas, 12).cpu().numpy()
    rec = rec[rec[:, 6] > 0]
    return int(np.sum(rec[:, 3] > rec[:, 7])), bool(np.all(rec[:, 7] == 0))


def captured(s, path):
    """What a captured call's graph says of itself, kernel names included."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        decode(s)
    graph.debug_dump(str(path))
    return path.read_text()


@pytest.mark.parametrize("name", CASES)
def test_cut_units_are_joined(cuda_device, tmp_path, name):
    case, inside = CASES[name]
    s = case.make()
    decode(s)
    torch.cuda.synchronize()
    text = captured(s, tmp_path / "call.dot")
    assert "paged_decode_kernel" in text
    assert ("paged_join_kernel" in text) == (not inside)
    cuts, own = division(s, 2 * torch.cuda.get_device_properties(0).multi_processor_count)
    assert cuts >= 2 and (own or not name.startswith("own")) and (not own or not name.startswith("line"))
    check(case, s)
    assert status(s)[0] == 0
    first = s["out"].clone()
    for _ in range(5):  # the counters of the join are as the next call wants them
        s["out"].fill_(7.0)
        decode(s)
        assert torch.equal(s["out"], first)
    one = dict(s)
    one["out"] = torch.full_like(s["out"], 7.0)
    one["lse"] = torch.full_like(s["lse"], 7.0)
    attend(one)
    check(case, one)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_chunks_repeat_themselves(cuda_device, dtype):
    case = Batch(kv=[3000, 700, 3], q=[40, 200, 3], hk=2, g=4, page=64, dtype=dtype, nan=False)
    s = case.make()
    attend(s)
    first, lse = s["out"].clone(), s["lse"].clone()
    for _ in range(10):
        s["out"].fill_(7.0)
        attend(s)
        assert torch.equal(s["out"], first) and torch.equal(s["lse"], lse)
