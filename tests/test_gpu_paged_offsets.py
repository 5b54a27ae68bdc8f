"""Bad token offsets and lengths: every one is reported, the sequences whose own
offsets are good keep their results, and nothing else is written."""
import numpy as np
import pytest
import torch

import kv_cache_compression_fkv_b200 as fkv
from tests.paged_util import DT, Batch, attend, check, status

pytestmark = pytest.mark.gpu

# offsets for sequences of 10, 20 and 30 new tokens; the good sequences
OFFSETS = [([0, 70, 30, 60], (2,)), ([0, -4, 30, 60], (2,)), ([0, 10, 30, 1000], (0, 1)), ([0, 10, 9, 5], (0,)),
           ([0, 10, 30, 29], (0, 1)), ([0, 10, 2 ** 31 - 1, -2 ** 31], (0,))]
KV, Q, FIRST = [40, 50, 60], [10, 20, 30], [0, 10, 30, 60]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu,good", OFFSETS)
def test_attend(cuda_device, cu, good, dtype):
    case = Batch(kv=KV, q=Q, dtype=dtype)
    s = case.make()
    s["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
    attend(s)
    torch.cuda.synchronize()
    assert status(s)[0] == 7
    check(case, s, only=good)
    for b in set(range(3)) - set(good):
        assert torch.all(s["out"][FIRST[b]:FIRST[b + 1]] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu,good", OFFSETS)
def test_append(cuda_device, cu, good, dtype):
    case = Batch(kv=KV, q=Q, dtype=dtype, nan=False)
    s = case.make()
    want_k, want_v = s["k_cache"].clone(), s["v_cache"].clone()
    rows = torch.randn((60, case.hq + 4, 128), device="cuda").to(DT[dtype])
    q, k, v = rows.split([case.hq, 2, 2], dim=1)
    q_out = torch.full((60, case.hq, 128), 7.0, dtype=DT[dtype], device="cuda")
    want_q = q_out.clone()
    s["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
    fkv.paged_append(s["cache"], s["kv_len"], k, v, s["ws"], cu_q=s["cu_q"], q=q, q_out=q_out)
    torch.cuda.synchronize()
    for b in good:
        for i in range(Q[b]):
            t, p = FIRST[b] + i, KV[b] - Q[b] + i
            page = int(s["table"][b, p // case.page])
            want_k[page, :, p % case.page] = k[t]
            want_v[page, :, p % case.page] = v[t]
            want_q[t] = q[t]
    assert torch.equal(s["k_cache"], want_k) and torch.equal(s["v_cache"], want_v) and torch.equal(q_out, want_q)
    assert status(s)[0] == 7


@pytest.mark.parametrize("cu", [[0, 60, 50], [0, 60, 61], [0, 60, -1]])
def test_append_reports_a_sequence_that_no_token_falls_to(cuda_device, cu):
    case = Batch(kv=[70, 20], q=[60, 0], nan=False)
    s = case.make()
    k = torch.randn((60, 2, 128), device="cuda").to(torch.bfloat16)
    s["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
    fkv.paged_append(s["cache"], s["kv_len"], k, k, s["ws"], cu_q=s["cu_q"])
    torch.cuda.synchronize()
    assert status(s) == (7, 1)


@pytest.mark.parametrize("kv", [-1, 10 ** 9])
@pytest.mark.parametrize("seqs,tokens", [(3, 2), (200, 1), (200, 199)])
def test_append_reports_the_length_of_a_sequence_without_tokens(cuda_device, kv, seqs, tokens):
    """As the attention over the same batch does; more sequences than tokens."""
    case = Batch(kv=[9] * seqs, q=[1] * tokens + [0] * (seqs - tokens), hk=1, g=1, D=64, page=8, nan=False)
    s = case.make()
    s["kv_len"][seqs - 1] = kv
    k = torch.randn((tokens, 1, 64), device="cuda").to(torch.bfloat16)
    fkv.paged_append(s["cache"], s["kv_len"], k, k, s["ws"], cu_q=s["cu_q"])
    torch.cuda.synchronize()
    assert status(s) == (7, seqs - 1)
    s["ws"].zero_()
    attend(s)
    torch.cuda.synchronize()
    assert status(s) == (7, seqs - 1)


def test_append_many_sequences_with_one_bad(cuda_device):
    """The search among more than 32 sequences lands on a bad one: the tokens of
    the others still find theirs."""
    n = 300
    case = Batch(kv=[5] * n, q=[2] * n, hk=1, g=1, D=64, page=8, nan=False)
    for at, value in ((150, 2 * n), (150, -1), (64, 500), (299, 3), (1, 599)):
        s = case.make()
        want_k = s["k_cache"].clone()
        k = torch.randn((2 * n, 1, 64), device="cuda").to(torch.bfloat16)
        s["cu_q"][at] = value
        cu = s["cu_q"].tolist()
        fkv.paged_append(s["cache"], s["kv_len"], k, k, s["ws"], cu_q=s["cu_q"])
        torch.cuda.synchronize()
        assert status(s)[0] == 7
        # rows of sequences whose both offsets are as they were, and whose tokens no
        # other good sequence claims
        claims = np.zeros(2 * n, int)
        for b in range(n):
            if 0 <= cu[b] <= cu[b + 1] <= 2 * n:
                claims[cu[b]:cu[b + 1]] += 1
        for b in range(n):
            if at in (b, b + 1):
                continue
            for i in range(2):
                if claims[2 * b + i] == 1:
                    p = 3 + i
                    want_k[int(s["table"][b, 0]), :, p] = k[2 * b + i]
        same = (s["k_cache"] == want_k).flatten(2).all(-1).all(-1)
        touched = [int(s["table"][b, 0]) for b in range(n)
                   if at not in (b, b + 1) and claims[2 * b] == 1 and claims[2 * b + 1] == 1]
        assert bool(same[touched].all())
