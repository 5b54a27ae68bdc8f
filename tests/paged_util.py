"""Inputs and checks shared by the paged-cache tests: ragged batches whose
unread places hold NaN, the float64 oracle over them, and tolerances."""
import dataclasses
import math
from typing import List, Optional

import numpy as np
import torch

import kv_cache_compression_fkv_b200 as fkv
from oracle import fkv_paged as orc

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # largest rounding error, relative


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


@dataclasses.dataclass
class Batch:
    """kv: cached lengths with the new tokens; q: new tokens (decode: all 1)."""

    kv: List[int]
    q: Optional[List[int]] = None
    hk: int = 2
    g: int = 2
    D: int = 128
    page: int = 16
    dtype: str = "bf16"
    causal: bool = True
    window: int = 0
    prefix: Optional[List[int]] = None
    cap: float = 0.0
    slopes: bool = False
    rows_outside: bool = False  # cache kept as [pages][rows][heads][D]
    pad: int = 0                # padded rows behind the last sequence
    seed: int = 0
    std: float = 1.0
    nan: bool = True            # NaN wherever no query of the sequence sees

    @property
    def hq(self):
        return self.hk * self.g

    def q_lens(self):
        return [1] * len(self.kv) if self.q is None else self.q

    def seen(self, b):
        """Keys of sequence b that some query sees."""
        kv, q = self.kv[b], self.q_lens()[b]
        see = np.zeros(kv, bool)
        for i in range(q):
            see |= orc.visible(kv, kv - q + i, causal=self.causal, window=self.window,
                               prefix=self.prefix[b] if self.prefix else 0)
        return see

    def make(self, device="cuda"):
        g = torch.Generator().manual_seed(self.seed + 1000)
        dt, page = DT[self.dtype], self.page
        need = [-(-n // page) for n in self.kv]
        width, pages = max(need + [1]) + 1, sum(need) + 3
        ids = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(self.kv), width), -7, dtype=torch.int32)
        shape = (pages, self.hk, page, self.D)
        k = torch.full(shape, float("nan") if self.nan else 0.0)
        v = k.clone()
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
            see = self.seen(b)
            for p in range(n):
                for r in range(min(page, self.kv[b] - p * page)):
                    if see[p * page + r] or not self.nan:
                        k[int(table[b, p]), :, r] = torch.randn(self.hk, self.D, generator=g) * self.std
                        v[int(table[b, p]), :, r] = torch.randn(self.hk, self.D, generator=g)
        tokens = sum(self.q_lens()) + self.pad
        q = (torch.randn((tokens, self.hq, self.D), generator=g) * self.std).to(dt)
        k, v = k.to(dt), v.to(dt)
        s = {"q": q.to(device), "table": table.to(device),
             "kv_len": torch.tensor(self.kv, dtype=torch.int32, device=device),
             "cu_q": torch.tensor([0] + list(np.cumsum(self.q_lens())), dtype=torch.int32, device=device),
             "slopes": (2.0 ** -torch.linspace(0.5, 8, self.hq)).to(device) if self.slopes else None,
             "prefix": torch.tensor(self.prefix, dtype=torch.int32, device=device) if self.prefix else None}
        for name, c in (("k", k), ("v", v)):
            if self.rows_outside:
                s[name + "_cache"] = c.transpose(1, 2).contiguous().to(device).transpose(1, 2)
            else:
                s[name + "_cache"] = c.to(device)
        s["out"] = torch.full((tokens, self.hq, self.D), 7.0, dtype=dt, device=device)
        s["lse"] = torch.full((tokens, self.hq), 7.0, device=device)
        s["cache"] = fkv.PagedCache(s["k_cache"], s["v_cache"], s["table"], num_q_heads=self.hq,
                                    softcap=self.cap, window=self.window, causal=self.causal,
                                    alibi_slopes=s["slopes"])
        s["ws"] = s["cache"].workspace()
        return s


def check(case: Batch, s, only=None):
    """Every row of out and lse (of the sequences `only`, where given) against
    the oracle; padded rows untouched."""
    out, lse = f64(s["out"]), f64(s["lse"])
    k_cache, v_cache, q = f64(s["k_cache"]), f64(s["v_cache"]), f64(s["q"])
    table = s["table"].cpu().numpy()
    slopes = f64(s["slopes"]) if case.slopes else np.zeros(case.hq)
    t = 0
    for b, n_q in enumerate(case.q_lens()):
        kv = case.kv[b]
        if only is not None and b not in only:
            t += n_q
            continue
        k = orc.cache_rows(k_cache, table[b], kv)
        v = orc.cache_rows(v_cache, table[b], kv)
        for i in range(n_q):
            for h in range(case.hq):
                ref, z, mean_abs, dz, n = orc.attend_row(
                    q[t, h], k[h // case.g], v[h // case.g], kv - n_q + i, scale=1 / math.sqrt(case.D),
                    cap=case.cap, slope=slopes[h], causal=case.causal, window=case.window,
                    prefix=case.prefix[b] if case.prefix else 0)
                # weights: a score error dz moves a weight by 2 dz (itself and
                # the sum); its exponential is within 1e-4 in the bf16 kernels
                # (polynomial 8.6e-5, hardware 2^-22) and 2^-21 in fp32; in
                # bf16 each weight is rounded once; the n products are added
                # in fp32.  The result is rounded once.
                w = 2 * dz + (1e-4 + HALF["bf16"] if case.dtype == "bf16" else 2.0 ** -21) + (n + 64) * orc.U32
                tol = HALF[case.dtype] * np.abs(ref) + 1.01 * w * mean_abs
                err = np.abs(out[t, h] - ref)
                assert np.all(err <= tol), (b, i, h, float(np.max(err - tol)), float(np.max(err)))
                if n == 0:
                    assert lse[t, h] == -np.inf, (b, i, h)
                else:
                    tz = w + 4 * orc.U32 * abs(z)
                    assert abs(lse[t, h] - z) <= tz, (b, i, h, lse[t, h], z, tz)
            t += 1
    assert np.all(out[t:] == 7.0) and np.all(lse[t:] == 7.0)


def status(s):
    return fkv.read_status(s["ws"])


def decode(s, **kw):
    fkv.paged_decode(s["cache"], s["kv_len"], s["q"], s["out"], s["ws"], prefix_len=s["prefix"],
                     lse=s["lse"], **kw)


def attend(s, **kw):
    fkv.paged_attend(s["cache"], s["kv_len"], s["cu_q"], s["q"], s["out"], s["ws"],
                     prefix_len=s["prefix"], lse=s["lse"], **kw)
