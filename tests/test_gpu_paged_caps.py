"""Capped scores over the whole range of caps: c tanh(z / c) keeps the relative
accuracy of z where c is far above it."""
import math

import numpy as np
import pytest
import torch

import kv_cache_compression_fkv_b200 as fkv
from oracle.fkv_paged import U32
from tests.paged_util import DT, Batch, attend, check, decode, f64, status

pytestmark = pytest.mark.gpu

CAPS = [1e-12, 0.05, 5.0, 50.0, 1e3, 1e6, 1e12]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
@pytest.mark.parametrize("cap", CAPS)
def test_caps(cuda_device, op, cap, dtype):
    for D in (64, 128):
        case = Batch(kv=[300, 41], q=[1, 1] if op == "decode" else [70, 3], cap=cap, std=2.0, D=D, dtype=dtype,
                     prefix=[3, 0], window=200)
        s = case.make()
        (decode if op == "decode" else attend)(s)
        torch.cuda.synchronize()
        check(case, s)
        assert status(s)[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
@pytest.mark.parametrize("cap", CAPS)
def test_score_of_one_key(cuda_device, op, cap, dtype):
    """With one key the log-sum-exp is its score.  Queries of a wide range of
    sizes, so that z / c is far below, around and far above 1 where it can be."""
    n, D = 96, 64
    g = torch.Generator().manual_seed(5)
    size = torch.logspace(-4, 3, n).view(n, 1, 1)
    q = (torch.randn((n, 16, D), generator=g) * size).to(DT[dtype])
    k = torch.randn((n, 1, 8, D), generator=g).to(DT[dtype])
    qd, kd = q.cuda(), k.cuda()
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    cache = fkv.PagedCache(kd, kd, table, num_q_heads=16, softcap=cap)
    ws, out = cache.workspace(), torch.empty_like(qd)
    lse = torch.empty((n, 16), device="cuda")
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    if op == "decode":
        fkv.paged_decode(cache, one, qd, out, ws, lse=lse)
    else:
        fkv.paged_attend(cache, one, None, qd, out, ws, lse=lse)
    raw = np.einsum("nhd,nd->nh", f64(q), f64(k)[:, 0, 0]) / math.sqrt(D)
    z = cap * np.tanh(raw / cap)
    # the products and sums of q.k and its scaling; the tanh and its factors,
    # relative to the smaller of c and |raw| (oracle/fkv_paged.py); in and out of
    # base 2 and the logarithm of a sum that is 1 within 2^-21
    tol = (D + 4) * U32 * np.einsum("nhd,nd->nh", np.abs(f64(q)), np.abs(f64(k)[:, 0, 0])) / math.sqrt(D)
    tol = np.minimum(tol, 2 * cap) + 32 * U32 * np.minimum(cap, np.abs(raw)) + 8 * U32 * np.abs(z) + 2.0 ** -21
    err = np.abs(f64(lse) - z)
    assert np.all(err <= tol), (float(np.max(err - tol)), float(np.max(err / tol)))
    assert torch.equal(out, kd[:, :, 0].expand(n, 16, D))
    assert fkv.read_status(ws)[0] == 0
