"""Per-head norm and rotation, and the append to a paged cache, against the
float64 oracle; then the operators together as a serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import fkv_workloads as wl
import kv_cache_compression_fkv_b200 as fkv
from oracle import fkv_oracle
from oracle import fkv_paged as orc
from tests.paged_util import DT, HALF, Batch, attend, check, decode, f64, status

pytestmark = pytest.mark.gpu

# fp32 error of a normed and rotated value, relative to |y_a| + |y_b| of its
# pair: the sum of squares of at most 128 terms in a tree of depth <= 12 and
# the mean (13 roundings, halved by the root), root, quotient and two products
# (4), the cosine (an angle off by 2^-24 turns: 2 pi 2^-24, and 2 roundings of the
# function), two products and a sum (3): below 24 roundings.
ROUNDINGS = 24


def close(got, ref, mag, dtype):
    assert np.all(np.abs(got - ref) <= HALF[dtype] * np.abs(ref) + 1.01 * ROUNDINGS * orc.U32 * mag)


def omega_of(n, seed=0):
    return torch.tensor(10000.0 ** (-np.arange(n) / max(n, 1)), dtype=torch.float32)


ROWS = [
    # tokens, hq, hk, D, dtype, style, axis_pairs, far
    (1, 1, 1, 128, "bf16", "interleaved", (64,), 100),
    (7, 12, 12, 128, "bf16", "interleaved", (22, 21, 21), 5000),
    (33, 8, 2, 128, "bf16", "half", (64,), 1 << 20),
    (5, 3, 1, 64, "bf16", "half", (16,), 1 << 30),
    (5, 40, 40, 64, "bf16", "interleaved", (1, 0, 2), 77),
    (4, 5, 3, 128, "bf16", "half", (3, 5), 99),
    (9, 4, 2, 128, "fp32", "half", (32,), 1 << 20),
    (9, 4, 2, 128, "fp32", "interleaved", (33,), 1 << 30),
    (130, 3, 1, 64, "fp32", "interleaved", (11, 7), 4000),
    (3, 2, 2, 64, "fp32", "half", (32,), 4000),
    (3, 2, 2, 64, "bf16", "half", (0,), 4000),
]


@pytest.mark.parametrize("tokens,hq,hk,D,dtype,style,axis_pairs,far", ROWS)
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope(cuda_device, tokens, hq, hk, D, dtype, style, axis_pairs, far, norm):
    g = torch.Generator().manual_seed(tokens * hq + D)
    dt, n = DT[dtype], sum(axis_pairs)
    x = {"q": (torch.randn((tokens, hq, D), generator=g) * 3).to(dt),
         "k": (torch.randn((tokens, hk, D), generator=g) * 0.01).to(dt)}
    x["k"][0] = 0
    w = {"q": torch.randn(D, generator=g), "k": None}
    pos = torch.randint(-5, far, (len(axis_pairs), tokens), generator=g, dtype=torch.int32)
    om = omega_of(n)
    rope = fkv.make_rope(om.cuda() if n else None, axis_pairs=axis_pairs, style=style, norm=norm, eps=1e-5,
                         q_weight=w["q"].cuda())
    d = {i: v.cuda() for i, v in x.items()}
    out = {i: torch.full_like(v, float("nan")) for i, v in d.items()}
    fkv.qk_norm_rope(rope, d["q"], d["k"], pos.cuda(), out["q"], out["k"])
    for i in "qk":
        ref, mag = orc.norm_rope(f64(x[i]), weight=None if w[i] is None else f64(w[i]), eps=1e-5, norm=norm,
                                 omega=om.numpy(), positions=pos.numpy(), axis_pairs=axis_pairs, style=style)
        close(f64(out[i]), ref, mag, dtype)
    # one of the two alone, in place, head-major and out of a packed projection: the same bits
    again = d["q"].clone()
    fkv.qk_norm_rope(rope, again, None, pos.cuda(), again, None)
    assert torch.equal(again, out["q"])
    packed = torch.cat([d["k"], d["q"], d["k"]], dim=1)
    heads = torch.full((hq, tokens, D), float("nan"), dtype=dt, device="cuda")
    k2 = torch.empty_like(d["k"])
    fkv.qk_norm_rope(rope, packed[:, hk:hk + hq], packed[:, :hk], pos.cuda(), heads.transpose(0, 1), k2)
    assert torch.equal(heads.transpose(0, 1), out["q"]) and torch.equal(k2, out["k"])


def test_qk_norm_rope_long_rows(cuda_device):
    """Offsets past 32 bits: head 1 of the last token lies 2^33 elements out."""
    tokens, stride = 3, 1 << 32
    big = torch.empty((stride * 2 + 4096,), dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((tokens, 2, 64), (stride, 64, 1))
    q.copy_(torch.randn((tokens, 2, 64), device="cuda"))
    rope = fkv.make_rope(omega_of(32).cuda())
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda").view(1, -1)
    dense, out = q.clone(), torch.empty((tokens, 2, 64), dtype=torch.bfloat16, device="cuda")
    fkv.qk_norm_rope(rope, dense, None, pos, out, None)
    fkv.qk_norm_rope(rope, q, None, pos, q, None)
    assert torch.equal(q, out)


def _append(case: Batch, s, rope, k, v, q=None, q_out=None, positions=None, cu=True):
    fkv.paged_append(s["cache"], s["kv_len"], k, v, s["ws"], cu_q=s["cu_q"] if cu else None, rope=rope,
                     positions=positions, q=q, q_out=q_out)


def _places(case: Batch, s):
    """(page, row) of every new token, in token order; None where it has none."""
    table, got = s["table"].cpu().numpy(), []
    for b, n in enumerate(case.q_lens()):
        for i in range(n):
            p = case.kv[b] - n + i
            got.append((int(table[b, p // case.page]), p % case.page, p, b) if p >= 0 else None)
    return got


APPEND = {
    "one_each": Batch(kv=[1, 16, 17, 200], q=[1, 1, 1, 1]),
    "prompts": Batch(kv=[40, 0, 33, 129], q=[40, 0, 10, 128], hk=3, g=2, pad=5),
    "d64_page8_rows_outside": Batch(kv=[40, 9, 33], q=[40, 9, 1], D=64, page=8, rows_outside=True, pad=1),
    "fp32": Batch(kv=[40, 9, 33], q=[40, 9, 1], dtype="fp32", page=256, pad=2),
    "many": Batch(kv=[5 + i % 7 for i in range(1100)], q=[i % 3 for i in range(1100)], hk=1, g=1, D=64, page=8),
    "negative": Batch(kv=[3, 40], q=[7, 2]),
}


@pytest.mark.parametrize("name", APPEND)
@pytest.mark.parametrize("style", ["interleaved", "half", None])
def test_append(cuda_device, name, style):
    case = APPEND[name]
    case = Batch(**{**case.__dict__, "nan": False})
    s = case.make()
    dt, D = DT[case.dtype], case.D
    g = torch.Generator().manual_seed(11)
    t = s["q"].shape[0]
    rows = (torch.randn((t, case.hq + 2 * case.hk, D), generator=g) * 2).to(dt).cuda()
    q, k, v = rows.split([case.hq, case.hk, case.hk], dim=1)
    before = {n: s[n].clone() for n in ("k_cache", "v_cache")}
    om = omega_of(24)
    kw = torch.randn(D, generator=g)
    rope = None if style is None else fkv.make_rope(om.cuda(), style=style, k_weight=kw.cuda())
    q_out = torch.full((t, case.hq, D), 7.0, dtype=dt, device="cuda")
    _append(case, s, rope, k, v, q, q_out)
    torch.cuda.synchronize()
    assert status(s)[0] == (7 if name == "negative" else 0)
    places = _places(case, s)
    pos = np.array([[p[2] if p else 0 for p in places]])
    n = len(places)
    got_k, got_v = f64(s["k_cache"]), f64(s["v_cache"])
    rope_kw = dict(norm=style is not None, omega=om.numpy() if style else (), positions=pos, axis_pairs=(24,),
                   style=style or "half")
    ref_k, mag = orc.norm_rope(f64(k)[:n], weight=f64(kw) if style else None, **rope_kw)
    want_k, want_v = f64(before["k_cache"]), f64(before["v_cache"])
    for i, p in enumerate(places):
        if p is None:
            continue
        close(got_k[p[0], :, p[1]], ref_k[i], mag[i], case.dtype)
        want_k[p[0], :, p[1]] = got_k[p[0], :, p[1]]
        want_v[p[0], :, p[1]] = f64(v)[i]
    assert np.array_equal(got_k, want_k) and np.array_equal(got_v, want_v)  # every other row is as it was
    neg = np.array([p is None for p in places])
    if name == "negative":
        pos[0, neg] = np.arange(neg.sum()) - neg.sum()
        rope_kw["positions"] = pos
    ref_q, mag = orc.norm_rope(f64(q)[:n], **rope_kw)
    close(f64(q_out)[:n], ref_q, mag, case.dtype)
    assert np.all(f64(q_out)[n:] == 7.0)
    # without queries, and with given positions: the keys of those positions
    if style:
        s2 = case.make()
        far = torch.zeros((1, t), dtype=torch.int32)
        far[0, :n] = torch.from_numpy(pos[0].astype(np.int32)) + 100000
        _append(case, s2, rope, k, v, positions=far.cuda())
        rope_kw["positions"] = far[:, :n].numpy()
        ref_k, mag = orc.norm_rope(f64(k)[:n], weight=f64(kw), **rope_kw)
        for i, p in enumerate(places):
            if p is not None:
                close(f64(s2["k_cache"][p[0], :, p[1]]), ref_k[i], mag[i], case.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_turns_queries_in_place(cuda_device, dtype):
    case = Batch(kv=[40, 50, 60], q=[10, 20, 30], dtype=dtype, nan=False)
    a, b = case.make(), case.make()
    rows = torch.randn((60, case.hq + 2 * case.hk, 128), device="cuda").to(DT[dtype])
    q, k, v = rows.split([case.hq, case.hk, case.hk], dim=1)
    rope = fkv.make_rope(omega_of(64).cuda(), style="half")
    out = torch.empty((60, case.hq, 128), dtype=DT[dtype], device="cuda")
    _append(case, a, rope, k, v, q, out)
    _append(case, b, rope, k, v, q, q)
    assert torch.equal(q, out) and torch.equal(a["k_cache"], b["k_cache"])


def test_append_one_token_per_sequence_without_offsets(cuda_device):
    case = Batch(kv=[1, 16, 17, 200], q=[1, 1, 1, 1], nan=False)
    a, b = case.make(), case.make()
    k = torch.randn((4, 2, 128), device="cuda").to(torch.bfloat16)
    rope = fkv.make_rope(omega_of(64).cuda())
    _append(case, a, rope, k, k)
    _append(case, b, rope, k, k, cu=False)
    assert torch.equal(a["k_cache"], b["k_cache"]) and torch.equal(a["v_cache"], b["v_cache"])


def test_append_reports_bad_pages_and_lengths(cuda_device):
    case = Batch(kv=[40, 50, 60], q=[10, 20, 30], nan=False)
    k = torch.randn((60, 2, 128), device="cuda").to(torch.bfloat16)
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        s, ok = case.make(), case.make()
        for x in (s, ok):
            if x is s:
                x["table"][1, 2] = bad  # positions 32..47
            _append(case, x, None, k, k)
        assert status(s) == (7, 1) and status(ok)[0] == 0
        page = int(ok["table"][1, 2])
        fresh = case.make()
        ok["k_cache"][page] = fresh["k_cache"][page]
        assert torch.equal(s["k_cache"], ok["k_cache"])
    for n in (-5, 10 ** 9):
        s = case.make()
        s["kv_len"][2] = n
        _append(case, s, None, k, k)
        assert status(s) == (7, 2)
    for at, value in ((1, 70), (2, 5), (3, 1000), (1, -4)):
        s = case.make()
        s["cu_q"][at] = value
        _append(case, s, None, k, k)
        torch.cuda.synchronize()
        assert status(s)[0] in (0, 7)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_loop(cuda_device, dtype):
    """Prompts, then single tokens, of three sequences: append and read back at
    every step, against attention over all rows kept densely on the side."""
    hk, g, D, page, steps = 2, 4, 128, 16, 20
    prompts = [70, 1, 33]
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(3)
    pages = 3 * 8
    k_cache = torch.full((pages, hk, page, D), float("nan"), dtype=dt, device="cuda")
    v_cache = torch.full_like(k_cache, float("nan"))
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(3, 8).cuda()
    cache = fkv.PagedCache(k_cache, v_cache, table, num_q_heads=hk * g, window=50, softcap=30.0)
    ws = cache.workspace()
    om = omega_of(64)
    rope = fkv.make_rope(om.cuda(), style="half")
    prefix = torch.tensor([4, 4, 4], dtype=torch.int32, device="cuda")
    dense_k, dense_v = [[], [], []], [[], [], []]
    kv = [0, 0, 0]
    for step in range(steps):
        q_lens = prompts if step == 0 else [1, 1, 1]
        t = sum(q_lens)
        rows = torch.randn((t, hk * (g + 2), D), generator=gen).to(dt).cuda()
        q, k, v = rows.split([hk * g, hk, hk], dim=1)
        start = list(kv)
        kv = [a + b for a, b in zip(kv, q_lens)]
        kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda")
        qr = torch.empty((t, hk * g, D), dtype=dt, device="cuda")
        out = torch.empty_like(qr)
        fkv.paged_append(cache, kv_len, k, v, ws, cu_q=cu, rope=rope, q=q, q_out=qr)
        if step == 0:
            fkv.paged_attend(cache, kv_len, cu, qr, out, ws, prefix_len=prefix)
        else:
            fkv.paged_decode(cache, kv_len, qr, out, ws, prefix_len=prefix)
        at = 0
        for b in range(3):
            pos = np.arange(start[b], kv[b])[None]
            # the stored key: rounded once from the oracle's, or one step beside it
            ref, mag = orc.norm_rope(f64(k[at:at + q_lens[b]]), omega=om.numpy(), positions=pos, axis_pairs=(64,),
                                     style="half")
            p = np.arange(start[b], kv[b])
            tb = table[b].cpu().numpy()
            got = f64(k_cache)[tb[p // page], :, p % page]
            close(got, ref, mag, dtype)
            dense_k[b].extend(got)
            dense_v[b].extend(f64(v[at:at + q_lens[b]]))
            kk, vv = np.stack(dense_k[b], 1), np.stack(dense_v[b], 1)
            for i in range(q_lens[b]):
                for h in (0, 3, 7):
                    r, _, mean_abs, dz, n = orc.attend_row(f64(qr[at + i, h]), kk[h // g], vv[h // g], start[b] + i,
                                                           scale=1 / math.sqrt(D), cap=30.0, window=50, prefix=4)
                    w = 2 * dz + (1e-4 + HALF["bf16"] if dtype == "bf16" else 2.0 ** -21) + (n + 64) * orc.U32
                    err = np.abs(f64(out[at + i, h]) - r)
                    assert np.all(err <= HALF[dtype] * np.abs(r) + 1.01 * w * mean_abs), (step, b, i, h)
            at += q_lens[b]
    assert fkv.read_status(ws)[0] == 0


def test_compressed_cache_read_as_pages(cuda_device):
    """The chunk step's dense compressed cache is a paged cache whose pages lie
    behind one another: paged attention over it, without order, is the compressed
    attention over the same rows."""
    w = wl.scaled(wl.get("480p"), name="as_pages", H=4, T=128, F=6, Fc=1, n_static=4, static_frames=(0, 2, 5),
                  k_dynamic=3, score_stride=4, seed=9)
    x = {k: v.cuda() for k, v in wl.generate(w).items()}
    p = fkv.params_for(w, comp_rows=4 * 128)  # the three kept frames and room for the chunk
    o = fkv.allocate(p)
    fkv.step(p, x, o)
    assert o["kept_cnt"].tolist() == [[3, 3, 3, 3]]
    comp = {n: o[n + "_comp"][0] for n in "kv"}  # [H][4 * 128][D]
    page = 64
    as_pages = {n: c.view(4, 8, page, 128).transpose(0, 1) for n, c in comp.items()}
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    cache = fkv.PagedCache(as_pages["k"], as_pages["v"], table, num_q_heads=4, causal=False)
    ws = cache.workspace()
    kv_len = torch.tensor([512], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 128], dtype=torch.int32, device="cuda")
    rows = {n: x[n + "_cur"][0].transpose(0, 1) for n in "qkv"}  # [128][4][D]
    fkv.paged_append(cache, kv_len, rows["k"], rows["v"], ws, cu_q=cu)
    for n in "kv":
        assert torch.equal(comp[n][:, 384:], x[n + "_cur"][0])
    out = torch.empty((4, 128, 128), dtype=torch.bfloat16, device="cuda")
    fkv.paged_attend(cache, kv_len, cu, rows["q"], out.transpose(0, 1), ws)
    assert fkv.read_status(ws)[0] == 0
    for h in range(4):
        keys, values = f64(comp["k"][h]), f64(comp["v"][h])
        ref = fkv_oracle.attention(f64(x["q_cur"][0, h]), keys, values, w.scale)
        for got in (out[h], o["out"][0, h]):
            assert np.max(np.abs(f64(got) - ref)) <= 2e-2 and np.mean(np.abs(f64(got) - ref)) <= 2e-3


def test_norm_rope_feeds_the_chunk_step(cuda_device):
    """A token-major projection normed, rotated and laid out head-major in one
    call is what the chunk step reads."""
    w = wl.scaled(wl.get("480p"), name="feeds", H=4, T=128, F=3, Fc=1, n_static=4, static_frames=(0, 2),
                  k_dynamic=2, score_stride=4, seed=10)
    x = {k: v.cuda() for k, v in wl.generate(w).items()}
    p = fkv.params_for(w)
    o = fkv.allocate(p)
    g = torch.Generator().manual_seed(2)
    rows = (torch.randn((128, 12, 128), generator=g)).to(torch.bfloat16)
    om, pos = omega_of(64), torch.stack([torch.full((128,), 3), torch.arange(128) // 16, torch.arange(128) % 16])
    rope = fkv.make_rope(om.cuda(), axis_pairs=(22, 21, 21))
    d = rows.cuda()
    fkv.qk_norm_rope(rope, d[:, :4], d[:, 4:8], pos.to(torch.int32).cuda(), x["q_cur"][0].transpose(0, 1),
                     x["k_cur"][0].transpose(0, 1))
    fkv.step(p, x, o)
    assert fkv.read_status(o["ws"])[0] == 0
    for h in range(4):
        turned = []
        for first, name in ((0, "q_cur"), (4, "k_cur")):
            ref, mag = orc.norm_rope(f64(rows[:, first + h:first + h + 1]), omega=om.numpy(), positions=pos.numpy(),
                                     axis_pairs=(22, 21, 21))
            close(f64(x[name][0, h]), ref[:, 0], mag[:, 0], "bf16")
            turned.append(f64(x[name][0, h]))
        n = int(o["kept_cnt"][0, h]) * w.T
        keys = np.concatenate([f64(o["k_comp"][0, h, :n]), turned[1]])
        vals = np.concatenate([f64(o["v_comp"][0, h, :n]), f64(x["v_cur"][0, h])])
        ref = fkv_oracle.attention(turned[0], keys, vals, w.scale)
        assert np.max(np.abs(f64(o["out"][0, h]) - ref)) <= 2e-2
