"""Pages that no query sees may be gone: a serving loop that frees the pages
behind a sliding window leaves anything in their table entries."""
import pytest
import torch

from tests.paged_util import Batch, attend, check, decode, status

pytestmark = pytest.mark.gpu


def free_unseen(case: Batch, s, mark):
    """Table entries of pages that no query of their sequence sees <- mark; how many."""
    n = 0
    for b, kv in enumerate(case.kv):
        see = case.seen(b)
        for p in range(-(-kv // case.page)):
            if not see[p * case.page:(p + 1) * case.page].any():
                s["table"][b, p] = mark
                n += 1
    return n


DECODE = {
    "page8": Batch(kv=[300, 41, 1000, 1], page=8, window=37),
    "page16": Batch(kv=[1500, 500, 77], page=16, window=40),
    "prefix_gap": Batch(kv=[1500, 300, 90], page=8, window=20, prefix=[3, 70, 9]),
    "page256": Batch(kv=[1500, 700], page=256, window=30, prefix=[0, 5]),
    "g17_d64": Batch(kv=[700], page=8, window=21, hk=1, g=17, D=64, prefix=[9]),
    "whole": Batch(kv=[400], page=8, window=33, causal=False),
}
ATTEND = {
    "page8": Batch(kv=[900, 300], q=[40, 9], page=8, window=37),
    "page16": Batch(kv=[700, 600, 50], q=[150, 1, 50], page=16, window=40),
    "prefix_gap": Batch(kv=[900, 400], q=[130, 20], page=8, window=20, prefix=[3, 140]),
    "page256": Batch(kv=[1500, 700], q=[60, 5], page=256, window=30, prefix=[0, 5]),
    "d64_options": Batch(kv=[900], q=[100], page=8, window=50, prefix=[7], D=64, cap=20.0, slopes=True, hk=1, g=5),
    "whole": Batch(kv=[400], q=[60], page=8, window=33, causal=False),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mark", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("op,name", [("decode", n) for n in DECODE] + [("attend", n) for n in ATTEND])
def test_freed_pages_are_no_error(cuda_device, op, name, mark, dtype):
    case = Batch(**{**(DECODE if op == "decode" else ATTEND)[name].__dict__, "dtype": dtype})
    s = case.make()
    table = s["table"].clone()
    assert free_unseen(case, s, mark) > 0
    (decode if op == "decode" else attend)(s)
    assert status(s)[0] == 0
    s["table"].copy_(table)  # the oracle reads the rows of those pages too: NaN
    check(case, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
@pytest.mark.parametrize("where", ["prefix", "window"])
def test_bad_pages_that_are_seen_are_still_reported(cuda_device, op, where, dtype):
    """The first and the last page with a seen key, each on its own."""
    case = Batch(kv=[60, 500], q=[1, 1] if op == "decode" else [5, 30], page=8, window=30, prefix=[0, 9], dtype=dtype,
                 nan=False)
    s = case.make()
    free_unseen(case, s, -1)
    s["table"][1, 1 if where == "prefix" else (500 - case.q_lens()[1] - 30 + 1) // 8] = -1
    (decode if op == "decode" else attend)(s)
    assert status(s) == (7, 1)
    check(case, s, only=(0,))
