"""Calls that repeat themselves bit for bit, on batches whose CTAs run through many
short units: what one unit leaves in shared memory is not the next one's before it is
done with."""
import pytest
import torch

from tests.paged_util import Batch, attend, check, decode, status

pytestmark = pytest.mark.gpu

MIXED = [36, 118, 19, 4004, 50, 25, 7186, 17, 2500, 19, 64, 25, 36, 3000, 50, 1]
CASES = {
    "short_between_long": Batch(kv=(MIXED * 4)[:56], hk=8, g=4, nan=False),
    "short_between_long_d64": Batch(kv=(MIXED * 4)[:56], hk=8, g=4, D=64, nan=False),
    "all_short": Batch(kv=[1 + (i * 13) % 64 for i in range(700)], hk=8, g=2, nan=False),
    "all_short_d64": Batch(kv=[1 + (i * 13) % 64 for i in range(700)], hk=8, g=2, D=64, nan=False),
    "slices": Batch(kv=[1 + (i * 13) % 64 for i in range(200)], hk=4, g=40, nan=False),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
@pytest.mark.parametrize("name", CASES)
def test_repeats(cuda_device, op, name, dtype):
    case = Batch(**{**CASES[name].__dict__, "dtype": dtype})
    s = case.make()
    run = decode if op == "decode" else attend
    run(s)
    first, lse = s["out"].clone(), s["lse"].clone()
    some = range(0, len(case.kv), max(1, len(case.kv) // 24))
    check(case, s, only=set(some))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(150):
        s["out"].fill_(7.0)
        run(s)
        wrong += (s["out"] != first).any() | (s["lse"] != lse).any()
    assert int(wrong) == 0
    assert status(s)[0] == 0


DIRT = {
    "g5": Batch(kv=[900, 40, 333], q=[130, 3, 60], hk=2, g=5, nan=False),
    "g3_d64": Batch(kv=[1500, 77], q=[300, 20], hk=2, g=3, D=64, nan=False),
    "cap": Batch(kv=[900, 40, 333], q=[130, 3, 60], hk=2, g=8, cap=30.0, std=1.5, nan=False),
    "cap_g5_window": Batch(kv=[900, 40, 333], q=[130, 3, 60], hk=2, g=5, cap=30.0, std=1.5, window=50, prefix=[9, 0, 70],
                           page=8, nan=False),
    "cap_d64_slopes": Batch(kv=[700, 54], q=[90, 54], hk=1, g=7, D=64, cap=20.0, std=1.5, slopes=True, nan=False),
    "whole": Batch(kv=[1162, 300], q=[200, 33], hk=2, g=7, D=64, causal=False, nan=False),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
@pytest.mark.parametrize("name", DIRT)
def test_results_do_not_go_by_what_was_there(cuda_device, op, name, dtype):
    """Rows and keys that are not there hold what the last kernel left in shared
    memory: here, calls over much larger or smaller numbers."""
    case = Batch(**{**DIRT[name].__dict__, "dtype": dtype})
    if op == "decode":
        case = Batch(**{**case.__dict__, "kv": [n + i for n in case.kv for i in range(8)], "q": None,
                        "prefix": [n for n in case.prefix for _ in range(8)] if case.prefix else None})
    s = case.make()
    run = decode if op == "decode" else attend
    run(s)
    check(case, s, only={0, 1})
    first, lse = s["out"].clone(), s["lse"].clone()
    for std in (100.0, 1e-3, 10.0):
        dirt = Batch(kv=[640] * 40, q=None if op == "decode" else [256] * 40, hk=4, g=4, D=case.D, std=std, dtype=dtype,
                     nan=False, page=128, causal=False).make()
        for _ in range(3):
            run(dirt)
            s["out"].fill_(7.0)
            run(s)
            assert torch.equal(s["out"], first) and torch.equal(s["lse"], lse), std
