"""Paged-cache entry points without a GPU: struct layouts, refusals before
anything is launched, and the division of the work compiled for the host."""
import ctypes
import os
import subprocess

import pytest
import torch

import kv_cache_compression_fkv_b200 as fkv
from kv_cache_compression_fkv_b200 import _lib, build, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: the checks come first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_struct_layouts_match_the_header(tmp_path, lib):
    structs = {"fkv_paged_t": _lib.Paged, "fkv_rows_t": _lib.Rows, "fkv_rope_t": _lib.Rope}
    body, want = "", []
    for name, cls in structs.items():
        for f in cls._fields_:
            body += f'printf("%zu ", offsetof({name}, {f[0]}));'
            want.append(getattr(cls, f[0]).offset)
        body += f'printf("%zu ", sizeof({name}));'
        want.append(ctypes.sizeof(cls))
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fkv.h"\nint main(void){' + body + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    assert got == want


def _paged(**kw):
    c = _lib.Paged()
    base = dict(dtype=0, flags=1, head_dim=128, num_q_heads=8, num_kv_heads=2, page_size=16, num_pages=10,
                num_seqs=3, max_pages=4, window=0, scale=0.1, softcap=0.0, page_stride=2 * 16 * 128,
                head_stride=16 * 128, row_stride=128, table_stride=4, k_cache=FAKE, v_cache=FAKE,
                page_table=FAKE, kv_len=FAKE, cu_q=FAKE)
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _rows(ptr=FAKE, ts=8 * 128, hs=128):
    return ctypes.byref(_lib.Rows(ptr, ts, hs))


BAD = [
    ({"dtype": 2}, 1), ({"flags": 2}, 1), ({"head_dim": 96}, 3), ({"head_dim": 0}, 2),
    ({"num_q_heads": 7}, 2), ({"num_q_heads": 0}, 2), ({"num_kv_heads": 0}, 2), ({"num_q_heads": 65536}, 2),
    ({"page_size": 12}, 3), ({"page_size": 4}, 3), ({"page_size": 2048}, 3), ({"page_size": 0}, 2),
    ({"num_pages": -1}, 2), ({"num_seqs": -1}, 2), ({"num_seqs": 4097}, 2), ({"max_pages": -1}, 2),
    ({"max_pages": 1 << 27, "table_stride": 1 << 27}, 2), ({"window": -1}, 2),
    ({"scale": 0.0}, 1), ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1),
    ({"scale": 1e-13}, 1), ({"scale": -1.0}, 1), ({"softcap": 1e-13}, 1), ({"softcap": 1e13}, 1),
    ({"softcap": -1.0}, 1), ({"softcap": float("nan")}, 1), ({"softcap": float("inf")}, 1),
    ({"page_stride": 64}, 2), ({"row_stride": 0}, 2), ({"head_stride": -128}, 2), ({"row_stride": 132}, 1),
    ({"row_stride": 1 << 41}, 2), ({"table_stride": 3}, 2),
    ({"k_cache": None}, 1), ({"v_cache": FAKE + 8}, 1), ({"kv_len": None}, 1), ({"kv_len": FAKE + 2}, 1),
    ({"page_table": None}, 1), ({"prefix_len": FAKE + 1}, 1), ({"alibi_slopes": FAKE + 2}, 1),
]


@pytest.mark.parametrize("change,status", BAD)
def test_bad_caches_are_refused(lib, change, status):
    c, r = _paged(**change), _rows()
    assert lib.fkv_paged_decode(c, r, r, None, FAKE, None) == status
    assert lib.fkv_paged_attend(c, 5, r, r, None, FAKE, None) == status
    assert lib.fkv_paged_append(c, None, 5, None, r, r, None, FAKE, None) == status


def test_bad_rows_and_workspaces_are_refused(lib):
    c = _paged()
    ok = _rows()
    for bad, status in ((_rows(ptr=None), 1), (_rows(ptr=FAKE + 8), 1), (_rows(ts=1028), 1), (_rows(ts=-1024), 2),
                        (_rows(hs=1 << 41), 2)):
        assert lib.fkv_paged_decode(c, bad, ok, None, FAKE, None) == status
        assert lib.fkv_paged_attend(c, 5, bad, ok, None, FAKE, None) == status
        assert lib.fkv_paged_append(c, None, 5, None, bad, ok, None, FAKE, None) == status
        assert lib.fkv_paged_append(c, None, 5, None, ok, bad, None, FAKE, None) == status
        assert lib.fkv_paged_append(c, None, 5, bad, ok, ok, ok, FAKE, None) == status
    # outputs whose rows overlap
    for bad in (_rows(ts=0), _rows(hs=0), _rows(ts=128), _rows(ts=64), _rows(hs=64), _rows(ts=512, hs=256)):
        assert lib.fkv_paged_decode(c, ok, bad, None, FAKE, None) == 2
        assert lib.fkv_paged_attend(c, 5, ok, bad, None, FAKE, None) == 2
        assert lib.fkv_paged_append(c, None, 5, ok, ok, ok, bad, FAKE, None) == 2
    for ws in (None, FAKE + 16):
        assert lib.fkv_paged_decode(c, ok, ok, None, ws, None) == 6
        assert lib.fkv_paged_attend(c, 5, ok, ok, None, ws, None) == 6
        assert lib.fkv_paged_append(c, None, 5, None, ok, ok, None, ws, None) == 6
    assert lib.fkv_paged_decode(None, ok, ok, None, FAKE, None) == 1
    assert lib.fkv_paged_decode(c, None, ok, None, FAKE, None) == 1
    assert lib.fkv_paged_decode(c, ok, ok, FAKE + 2, FAKE, None) == 1
    for n in (-1, (1 << 30) + 1):
        assert lib.fkv_paged_attend(c, n, ok, ok, None, FAKE, None) == 2
        assert lib.fkv_paged_append(c, None, n, None, ok, ok, None, FAKE, None) == 2
        assert lib.fkv_qk_norm_rope(_rope(), 0, 128, n, 8, 8, ok, ok, ok, ok, None) == 2
    assert lib.fkv_paged_attend(_paged(cu_q=None), 5, ok, ok, None, FAKE, None) == 2  # 3 sequences
    assert lib.fkv_paged_append(_paged(cu_q=None), None, 5, None, ok, ok, None, FAKE, None) == 2
    assert lib.fkv_paged_append(c, None, 5, ok, ok, ok, None, FAKE, None) == 1  # q without q_out
    assert lib.fkv_paged_workspace_size(None) == 1


def test_nothing_to_do_is_no_error(lib):
    r = _rows()
    assert lib.fkv_paged_attend(_paged(), 0, None, None, None, FAKE, None) == 0
    assert lib.fkv_paged_decode(_paged(num_seqs=0, kv_len=None, page_table=None), None, None, None, FAKE, None) == 0
    assert lib.fkv_paged_append(_paged(), None, 0, None, None, None, None, FAKE, None) == 0
    rope = ctypes.byref(_lib.Rope(n_axes=1))
    assert lib.fkv_qk_norm_rope(rope, 0, 128, 0, 4, 4, None, None, None, None, None) == 0
    assert lib.fkv_qk_norm_rope(rope, 0, 128, 7, 0, 0, r, r, r, r, None) == 0


def _rope(**kw):
    r = _lib.Rope(style=0, norm=1, n_axes=1, eps=1e-6, omega=FAKE, positions=FAKE, axis_stride=5)
    pairs = kw.pop("axis_pairs", (32, 0, 0))
    for i, n in enumerate(pairs):
        r.axis_pairs[i] = n
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.byref(r)


@pytest.mark.parametrize("change,status", [
    ({"style": 2}, 1), ({"n_axes": 0}, 2), ({"n_axes": 4}, 2), ({"axis_pairs": (65, 0, 0)}, 2),
    ({"axis_pairs": (-1, 0, 0)}, 2), ({"style": 1, "axis_pairs": (12, 0, 0)}, 3), ({"eps": -1.0}, 1),
    ({"eps": float("nan")}, 1), ({"omega": None}, 1), ({"n_axes": 2, "axis_stride": 4}, 2),
    ({"q_weight": FAKE + 2}, 1), ({"k_weight": FAKE + 1}, 1), ({"omega": FAKE + 2}, 1), ({"positions": FAKE + 2}, 1),
    ({"n_axes": 3, "axis_pairs": (30, 30, 5), "axis_stride": 5}, 2)])
def test_bad_ropes_are_refused(lib, change, status):
    r, rows = _rope(**change), _rows()
    assert lib.fkv_qk_norm_rope(r, 0, 128, 5, 8, 8, rows, rows, rows, rows, None) == status
    assert lib.fkv_paged_append(_paged(), r, 5, None, rows, rows, None, FAKE, None) == status


def test_bad_norm_rope_calls_are_refused(lib):
    r, rows = _rope(), _rows()
    call = lib.fkv_qk_norm_rope
    assert call(None, 0, 128, 5, 8, 8, rows, rows, rows, rows, None) == 1
    assert call(r, 5, 128, 5, 8, 8, rows, rows, rows, rows, None) == 1
    assert call(r, 0, 80, 5, 8, 8, rows, rows, rows, rows, None) == 3
    assert call(r, 0, 128, -5, 8, 8, rows, rows, rows, rows, None) == 2
    assert call(r, 0, 128, 5, -8, 8, rows, rows, rows, rows, None) == 2
    assert call(r, 0, 128, 5, 8, 1 << 17, rows, rows, rows, rows, None) == 2
    assert call(r, 0, 128, 5, 8, 8, rows, None, rows, rows, None) == 1
    assert call(r, 0, 128, 5, 8, 8, rows, rows, rows, None, None) == 1
    assert call(_rope(positions=None), 0, 128, 5, 8, 8, rows, rows, rows, rows, None) == 1


def test_python_checks():
    z = torch.zeros
    with pytest.raises(ValueError):
        fkv.make_rope(z(4), axis_pairs=(3,))
    with pytest.raises(ValueError):
        fkv.make_rope(z(4))  # not on a GPU
    with pytest.raises(KeyError):
        fkv.make_rope(None, style="other")
    with pytest.raises(ValueError):
        fkv.qk_norm_rope(fkv.make_rope(), z(2, 2, 128), None, None, z(2, 2, 128), None)
    with pytest.raises(ValueError):
        fkv.qk_norm_rope(fkv.make_rope(), None, None, None, None, None)
    k = z((4, 2, 16, 128), dtype=torch.bfloat16)
    t = z((2, 3), dtype=torch.int32)
    for args in ((k, k, t), (k.half(), k.half(), t), (k, k[:2], t), (k, k.float(), t), (k.transpose(2, 3),) * 2 + (t,)):
        with pytest.raises(ValueError):
            fkv.PagedCache(*args, num_q_heads=4)
    meta = k.to("meta")
    with pytest.raises(ValueError):
        fkv.PagedCache(meta, meta, t, num_q_heads=4)
    packed = paged._rows(z((3, 2, 64), dtype=torch.bfloat16), "x", (3, 2, 64), torch.bfloat16, -1)
    assert _lib.Rows.from_buffer_copy(packed).token_stride == 128
    for bad in (z((3, 2, 64)), z((3, 64, 2), dtype=torch.bfloat16).transpose(1, 2), z((3, 1, 64), dtype=torch.bfloat16),
                z((3, 2, 64), dtype=torch.bfloat16, device="meta")):
        with pytest.raises(ValueError):
            paged._rows(bad, "x", (3, 2, 64), torch.bfloat16, -1 if bad.device.type == "cpu" else 0)


HARNESS = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "paged_plan.h"
using namespace fkv;
static int rnd(int n) { return rand() % n; }
int main() {
  // every key that a row sees lies in exactly one block of its tile's span;
  // every block of the span but a forced one is seen by some row; every
  // (token, head) is in exactly one row
  for (int it = 0; it < 4000; ++it) {
    TileRule g = {};
    g.G = 1 + rnd(40);
    g.Hkv = 1 + rnd(3);
    g.R = (it & 1) ? 16 : 128;
    g.tk_shift = (it & 2) ? 6 : 7;
    const int TK = 1 << g.tk_shift;
    g.mt = (g.G + g.R - 1) / g.R;
    g.tq = g.mt == 1 ? g.R / g.G : 1;
    g.causal = rnd(3) > 0;
    g.window = rnd(3) ? 0 : 1 + rnd(300);
    Seq s;
    s.q0 = 0;
    s.q_len = 1 + rnd(60);
    s.kv = rnd(900);
    s.pre = rnd(3) ? 0 : rnd(900);
    if (s.pre > s.kv) s.pre = s.kv;
    const int nq = query_tiles(g, s);
    std::vector<int> owner(s.q_len * g.G * g.Hkv, 0);
    for (int qt = 0; qt < nq; ++qt) {
      const Span t = tile_span(g, s, qt);
      std::vector<int> visits(64, 0), seen(64, 0);
      for (int j = 0; j < t.n; ++j) {
        const int blk = block_at(t, j);
        if (blk < 0 || blk >= 64) return 1;
        visits[blk]++;
      }
      for (int hm = 0; hm < g.Hkv * g.mt; ++hm)
        for (int r = 0; r < g.R; ++r) {
          int token, head;
          if (!row_place(g, s, qt, hm, r, &token, &head)) continue;
          if (token < 0 || token >= s.q_len || head < 0 || head >= g.G * g.Hkv) return 2;
          owner[token * g.G * g.Hkv + head]++;
          const RowSpan v = row_span(g, s, s.kv - s.q_len + token);
          for (int j = 0; j < s.kv; ++j) {
            const bool see = j < s.pre || (j >= v.lo && j <= v.hi);
            const int p = s.kv - s.q_len + token;
            const bool want = ((!g.causal || j <= p) && (!g.window || j > p - g.window)) || j < s.pre;
            if (see != want) return 3;
            if (!see) continue;
            if (visits[j / TK] != 1) return 4;
            if (!(j < s.pre || (j >= t.lo && j <= t.hi))) return 5;
            seen[j / TK] = 1;
          }
        }
      for (int blk = 0; blk < 64; ++blk) {
        if (visits[blk] > 1) return 6;
        if (visits[blk] && !seen[blk] && t.n > 1) return 7;
      }
    }
    for (int o : owner)
      if (o != 1) return 8;
  }
  // units cut by themselves: all parts fit the grid, none is empty, none but the
  // last of a unit is shorter, and the division without integers is exact
  for (int it = 0; it < 200000; ++it) {
    const int units = rnd(200), slots = rnd(600), least = 1 + rnd(4), most = rnd(2) ? 0 : 1 + rnd(8);
    const int longest = it & 1 ? 1 + rnd(40) : 1 + rnd(1 << 21);
    const int P = own_part(units, slots, longest, least, most);
    if ((units == 0 || units > slots) != (P == 0)) return 9;
    if (P == 0) continue;
    if (P > longest || (P < least && P != longest)) return 10;
    const int k = parts_of(longest, P);
    if (k != (longest + P - 1) / P || (k - 1) * P >= longest || int64_t(k) * P < longest) return 11;
    if (int64_t(k) * units > slots || (most && k > most && P > least)) return 12;
  }
  if (own_part(1, 1, kDivMax / 2, 1, 0) != 0) return 13;
  for (int it = 0; it < 1000000; ++it) {
    const int k = 1 + (it & 1 ? rnd(700) : rnd(kDivMax)), n = it % 3 ? rnd(kDivMax) : rnd(kDivMax / k) * k;
    if (div_down(n, k) != n / k) return 14;
  }
  puts("ok");
  return 0;
}
"""


def test_division_covers_every_visible_key_once(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "plan"
    csrc = os.path.join(ROOT, "kv_cache_compression_fkv_b200", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.returncode
