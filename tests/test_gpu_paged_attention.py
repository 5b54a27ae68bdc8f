"""Attention over the paged cache, single tokens and ragged chunks, against the
float64 oracle.  Every place that no query sees holds NaN."""
import pytest
import torch

import kv_cache_compression_fkv_b200 as fkv
from tests.paged_util import Batch, attend, check, decode, status

pytestmark = pytest.mark.gpu

DECODE = {
    "one_key": Batch(kv=[1]),
    "empty_between": Batch(kv=[0, 5, 0, 33, 0]),
    "page_ends": Batch(kv=[15, 16, 17, 31, 32, 63, 64, 65, 128], page=16),
    "page8": Batch(kv=[7, 8, 9, 100], page=8),
    "page256": Batch(kv=[255, 256, 257, 700], page=256),
    "page1024": Batch(kv=[1023, 1025], page=1024, hk=1),
    "d64": Batch(kv=[1, 77, 300], D=64, page=32),
    "mha": Batch(kv=[50, 201], hk=5, g=1),
    "g3": Batch(kv=[50, 201], hk=2, g=3),
    "g16": Batch(kv=[129, 3], hk=1, g=16),
    "g17": Batch(kv=[129, 40], hk=2, g=17),
    "g33_d64": Batch(kv=[70], hk=1, g=33, D=64),
    "split": Batch(kv=[5003], hk=1, g=4, page=64),
    "split_many": Batch(kv=[3001, 17, 2500], hk=3, g=2),
    # short tables: the kernel joins cut units itself (up to 8 parts)
    "cut_inside": Batch(kv=[900, 1, 850, 77, 1500, 1501], hk=1, g=6, page=32),
    "cut_inside_d64": Batch(kv=[1500] * 3, hk=3, g=17, D=64),
    "window": Batch(kv=[1, 40, 41, 500, 1500], window=40),
    "window1": Batch(kv=[1, 40, 500], window=1),
    "window_prefix": Batch(kv=[1, 40, 500, 1500, 20], window=40, prefix=[3, 0, 70, 64, 99]),
    "prefix_all": Batch(kv=[40, 300], window=1, prefix=[40, 1000]),
    "cap": Batch(kv=[40, 300], cap=5.0, std=2.0),
    "slopes": Batch(kv=[40, 300, 1200], slopes=True),
    "everything": Batch(kv=[2000, 33, 0, 700], hk=2, g=5, window=300, prefix=[20, 1, 4, 600], cap=20.0,
                        slopes=True, rows_outside=True, page=32),
    "rows_outside": Batch(kv=[33, 600], rows_outside=True),
    "peaked": Batch(kv=[900], std=6.0),
    "fp32": Batch(kv=[0, 1, 33, 500, 2000], dtype="fp32"),
    "fp32_d64_everything": Batch(kv=[2000, 33, 0, 700], hk=2, g=5, D=64, window=300, prefix=[20, 1, 4, 600],
                                 cap=20.0, slopes=True, rows_outside=True, page=8, dtype="fp32"),
    "fp32_mha": Batch(kv=[700, 3, 64], hk=4, g=1, dtype="fp32"),
    "fp32_g20": Batch(kv=[70], hk=1, g=20, dtype="fp32"),
}


# more sequences than one warp, one CTA and one round of a CTA divide
for _n, _dtype in ((33, "bf16"), (33, "fp32"), (170, "bf16"), (900, "bf16"), (300, "fp32")):
    DECODE[f"sequences_{_n}_{_dtype}"] = Batch(kv=[(i * 37) % 90 for i in range(_n)], hk=1, g=2, D=64, page=8,
                                               dtype=_dtype)
DECODE["window_beyond_all"] = Batch(kv=[1, 200], window=2 ** 31 - 1)


@pytest.mark.parametrize("name", DECODE)
def test_decode(cuda_device, name):
    case = DECODE[name]
    s = case.make()
    decode(s)
    torch.cuda.synchronize()
    check(case, s)
    assert status(s)[0] == 0


ATTEND = {
    "one": Batch(kv=[1], q=[1]),
    "square": Batch(kv=[200], q=[200]),
    "ragged": Batch(kv=[0, 5, 90, 300, 33], q=[0, 5, 40, 7, 33], pad=3),
    "behind_cache": Batch(kv=[700, 900], q=[130, 64]),
    "whole": Batch(kv=[300, 150], q=[70, 150], causal=False),
    "short_kv": Batch(kv=[3, 0], q=[10, 4]),       # rows at negative positions see nothing
    "short_kv_prefix": Batch(kv=[3], q=[10], prefix=[2]),
    "blocks": Batch(kv=[127, 128, 129, 256, 257], q=[127, 128, 129, 128, 1], hk=1, g=1),
    "g1": Batch(kv=[260], q=[260], hk=3, g=1),
    "g3": Batch(kv=[260], q=[100], hk=2, g=3),
    "g5_page8": Batch(kv=[100, 50], q=[60, 50], hk=1, g=5, page=8),
    "g128": Batch(kv=[40], q=[3], hk=1, g=128),
    "g130": Batch(kv=[40], q=[2], hk=1, g=130, D=64),
    "page256": Batch(kv=[600], q=[100], page=256),
    "d64": Batch(kv=[300, 77], q=[200, 77], D=64),
    "window": Batch(kv=[600, 100], q=[300, 100], window=70),
    "window1": Batch(kv=[300], q=[150], window=1),
    "window_prefix": Batch(kv=[900, 100], q=[150, 90], window=50, prefix=[140, 20]),
    "prefix": Batch(kv=[300, 64], q=[300, 64], prefix=[100, 64]),
    "whole_window": Batch(kv=[500], q=[200], causal=False, window=60),
    "cap": Batch(kv=[300], q=[140], cap=5.0, std=2.0),
    "slopes": Batch(kv=[300, 800], q=[140, 20], slopes=True),
    "everything": Batch(kv=[700, 33, 0, 400], q=[150, 33, 0, 61], hk=2, g=4, window=120, prefix=[20, 1, 0, 300],
                        cap=20.0, slopes=True, rows_outside=True, page=32, pad=5),
    "split": Batch(kv=[4000], q=[9], hk=1, g=2, page=64),
    "peaked": Batch(kv=[400], q=[100], std=6.0),
    "fp32": Batch(kv=[0, 5, 90, 300, 33], q=[0, 5, 40, 7, 33], pad=3, dtype="fp32"),
    "fp32_everything": Batch(kv=[500, 33, 0, 400], q=[90, 33, 0, 61], hk=2, g=4, D=64, window=120,
                             prefix=[20, 1, 0, 300], cap=20.0, slopes=True, rows_outside=True, page=8, pad=5,
                             dtype="fp32"),
    "fp32_g20_whole": Batch(kv=[70], q=[9], hk=1, g=20, dtype="fp32", causal=False),
}


for _n, _dtype in ((33, "bf16"), (33, "fp32"), (400, "bf16")):
    ATTEND[f"sequences_{_n}_{_dtype}"] = Batch(kv=[(i * 37) % 90 for i in range(_n)],
                                               q=[min((i * 37) % 90, (i * 5) % 7) for i in range(_n)], hk=1, g=2,
                                               D=64, page=8, dtype=_dtype, pad=2)
ATTEND["window_beyond_all"] = Batch(kv=[3, 200], q=[9, 50], window=2 ** 31 - 1)
# more units than CTAs of any of the kernels: cut on the line, most in two
_LINE = [(i * 397) % 1100 for i in range(20)]
for _dtype in ("bf16", "fp32"):
    ATTEND[f"line_{_dtype}"] = Batch(kv=_LINE, q=[min(n, (i * 7) % 12) for i, n in enumerate(_LINE)], hk=24, g=1,
                                     dtype=_dtype)
    DECODE[f"line_{_dtype}"] = Batch(kv=_LINE, hk=24, g=1, dtype=_dtype)
ATTEND["many_tiles"] = Batch(kv=[700, 600], q=[700, 600], hk=1, g=16)  # 88 and 75 query tiles


@pytest.mark.parametrize("name", ATTEND)
def test_attend(cuda_device, name):
    case = ATTEND[name]
    s = case.make()
    attend(s)
    torch.cuda.synchronize()
    check(case, s)
    assert status(s)[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_of_single_tokens_is_decode(cuda_device, dtype):
    case = Batch(kv=[300, 1, 77, 1025], window=100, prefix=[5, 0, 0, 9], dtype=dtype)
    s = case.make()
    attend(s)
    check(case, s)
    s["out"].fill_(7.0)
    fkv.paged_attend(s["cache"], s["kv_len"], None, s["q"], s["out"], s["ws"], prefix_len=s["prefix"],
                     lse=s["lse"])
    check(case, s)
    s["out"].fill_(7.0)
    decode(s)
    check(case, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
def test_strided_rows(cuda_device, dtype, op):
    """q out of a packed projection, out head by head."""
    case = Batch(kv=[90, 33], q=[1, 1] if op == "decode" else [20, 33], hk=2, g=3, dtype=dtype)
    s = case.make()
    t = s["q"].shape[0]
    packed = torch.full((t, case.hq + 4, case.D), float("nan"), dtype=s["q"].dtype, device="cuda")
    packed[:, 2:2 + case.hq] = s["q"]
    s["q"] = packed[:, 2:2 + case.hq]
    s["out"] = torch.full((case.hq, t, case.D), 7.0, dtype=s["q"].dtype, device="cuda").transpose(0, 1)
    (decode if op == "decode" else attend)(s)
    check(case, s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["decode", "attend"])
def test_bad_pages_and_lengths_are_reported(cuda_device, dtype, op):
    """Out-of-range page ids read as zeros, lengths are clamped to the table;
    both are reported with their sequence, and other sequences are unharmed."""
    case = Batch(kv=[90, 70, 33], q=[1, 1, 1] if op == "decode" else [20, 9, 33], dtype=dtype, nan=False)
    run = decode if op == "decode" else attend
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        s = case.make()
        want = s["table"].clone()
        s["table"][1, 2] = bad  # rows 32..47 of sequence 1
        run(s)
        assert status(s) == (7, 1)
        zero = int(want[1, 2])
        s["table"].copy_(want)
        s["k_cache"][zero] = 0
        s["v_cache"][zero] = 0
        check(case, s)
    for n in (-5, 10 ** 9):
        s = case.make()
        s["table"].clamp_(min=0)
        s["kv_len"][1] = n
        run(s)
        assert status(s) == (7, 1)
        # against the oracle, not bit for bit: where the work is cut, and with it
        # the order of the fp32 sums, goes by all lengths of the batch
        check(case, s, only=(0, 2))


def test_bad_token_offsets_are_reported(cuda_device):
    case = Batch(kv=[40, 50, 60], q=[10, 20, 30])
    for at, value in ((1, 70), (2, 5), (3, 1000), (1, -4)):
        s = case.make()
        s["cu_q"][at] = value
        attend(s)
        torch.cuda.synchronize()
        assert status(s)[0] == 7


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_graph_replay_follows_the_lengths(cuda_device, dtype):
    """One captured call, replayed with other lengths, offsets and pages, and a
    second graph on the same workspace in between."""
    cases = [Batch(kv=[300, 20, 700], q=[100, 20, 10], seed=1, dtype=dtype),
             Batch(kv=[40, 900, 0], q=[3, 126, 1], seed=2, dtype=dtype),
             Batch(kv=[128, 128, 800], q=[1, 1, 128], seed=3, dtype=dtype)]
    made = [c.make() for c in cases]
    pages = max(m["k_cache"].shape[0] for m in made)
    width = max(m["table"].shape[1] for m in made)
    s = dict(made[0])
    for n in ("k_cache", "v_cache"):
        s[n] = torch.zeros((pages,) + made[0][n].shape[1:], dtype=made[0][n].dtype, device="cuda")
    s["table"] = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    s["cache"] = fkv.PagedCache(s["k_cache"], s["v_cache"], s["table"], num_q_heads=cases[0].hq)
    graphs = []
    for run in (attend, lambda d: fkv.paged_decode(s["cache"], s["kv_len"], s["q"][:3], d["single"], s["ws"])):
        s["single"] = torch.empty((3, cases[0].hq, 128), dtype=s["q"].dtype, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run(s)
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(s)
        graphs.append(g)
    assert status(s)[0] == 7  # the warm-up ran over a table without pages
    s["ws"].zero_()
    for c, m in zip(cases, made):
        for n in ("k_cache", "v_cache"):
            s[n][:m[n].shape[0]].copy_(m[n])
        s["table"].fill_(-1)
        s["table"][:, :m["table"].shape[1]] = m["table"]
        for n in ("kv_len", "cu_q", "q"):
            s[n].copy_(m[n])
        for _ in range(2):
            s["out"].fill_(7.0)
            graphs[0].replay()
            graphs[1].replay()
            check(c, s)
            one = dict(s, out=s["single"], q=s["q"][:3], lse=s["lse"])
            ref = dict(s, out=torch.empty_like(s["single"]), q=s["q"][:3], lse=None)
            fkv.paged_decode(s["cache"], s["kv_len"], ref["q"], ref["out"], s["ws"])
            assert torch.equal(one["out"], ref["out"])
    assert status(s)[0] == 0


def test_calls_on_two_streams_with_their_own_workspaces(cuda_device):
    cases = [Batch(kv=[2000, 100], q=[100, 40], seed=5), Batch(kv=[1500, 300], q=[64, 90], seed=6)]
    made = [c.make() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, st in zip(made, streams):
            attend(m, stream=st)
    torch.cuda.synchronize()
    for c, m in zip(cases, made):
        check(c, m)


def test_results_do_not_depend_on_timing(cuda_device):
    case = Batch(kv=[5000, 700, 3], hk=2, g=4, page=64)
    s = case.make()
    decode(s)
    first = s["out"].clone()
    for _ in range(10):
        s["out"].fill_(7.0)
        decode(s)
        assert torch.equal(s["out"], first)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_keys_and_values_in_one_buffer(cuda_device, dtype):
    """[pages][heads][rows][2][D]: rows of the cache 2 D apart."""
    case = Batch(kv=[90, 33], q=[20, 33], dtype=dtype)
    s = case.make()
    both = torch.stack([s["k_cache"], s["v_cache"]], dim=3)
    k, v = both[..., 0, :], both[..., 1, :]
    s["cache"] = fkv.PagedCache(k, v, s["table"], num_q_heads=case.hq)
    attend(s)
    check(case, s)
    assert status(s)[0] == 0


def test_pages_shared_by_sequences(cuda_device):
    """A common prefix in the same pages."""
    case = Batch(kv=[70, 80, 64], q=[6, 16, 1], nan=False)
    s = case.make()
    s["table"][1, :4] = s["table"][0, :4]
    s["table"][2, :4] = s["table"][0, :4]
    attend(s)
    check(case, s)


def test_no_tokens_or_sequences(cuda_device):
    for dtype in ("bf16", "fp32"):
        case = Batch(kv=[40], q=[0], dtype=dtype)
        s = case.make()
        attend(s)
        empty = torch.empty((0, 2), dtype=torch.int32, device="cuda")
        c = fkv.PagedCache(s["k_cache"], s["v_cache"], empty, num_q_heads=4)
        none = torch.empty((0, 4, 128), dtype=s["q"].dtype, device="cuda")
        fkv.paged_decode(c, empty.view(-1), none, none.clone(), s["ws"])
        assert status(s)[0] == 0


def test_offsets_past_32_bits(cuda_device):
    """Pages whose element offsets pass 2^32 (a 9 GB cache, both dtypes of one buffer)."""
    pages, hk, page, D = 140000, 2, 128, 128
    k = torch.empty((pages, hk, page, D), dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 32
    ids = [pages - 1, 3, pages - 70000, pages - 2]
    for i in ids:
        k[i] = torch.randn((hk, page, D), device="cuda")
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    small = k[ids].clone()
    n = torch.tensor([4 * page - 5], dtype=torch.int32, device="cuda")
    outs = []
    for cache, t in ((k, table), (small, torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4))):
        c = fkv.PagedCache(cache, cache, t, num_q_heads=4)
        ws = c.workspace()
        g = torch.Generator(device="cuda").manual_seed(1)
        q = torch.randn((130, 4, D), generator=g, device="cuda").to(torch.bfloat16)
        one, many = torch.empty_like(q[:1]), torch.empty_like(q)
        fkv.paged_decode(c, n, q[:1], one, ws)
        fkv.paged_attend(c, n, torch.tensor([0, 130], dtype=torch.int32, device="cuda"), q, many, ws)
        new = torch.randn((1, hk, D), generator=g, device="cuda").to(torch.bfloat16)
        fkv.paged_append(c, n, new, new, ws)
        assert torch.equal(cache[t[0, 3].long(), :, page - 6], new[0])
        outs.append((one, many))
        assert fkv.read_status(ws)[0] == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
