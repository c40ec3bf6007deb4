"""The 8-bit cache's operators from their definitions, in 64 bits on the CPU,
for the tests: quantising, reading back, attention, and seeded problems."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()   # value of every code


def quantise_row(x: torch.Tensor):
    """(codes uint8 [..., D], scale bytes uint8 [...]) of the rows of x."""
    x = x.double()
    amax = x.abs().amax(-1)
    finite = torch.isfinite(x).all(-1)
    safe = torch.where(finite, amax, torch.ones_like(amax))
    # smallest e >= -127 with amax <= 448 * 2^e
    e = torch.full_like(safe, -127.0)
    for cand in range(127, -128, -1):
        e = torch.where(safe <= 448.0 * 2.0 ** cand, float(cand), e)
    e = torch.where(safe == 0, 0.0, e)
    y = torch.where(finite[..., None], x, torch.zeros_like(x)) * torch.exp2(-e)[..., None]
    # nearest of the 253 finite values; ties to the even code
    vals, codes = torch.sort(E4M3[:127])          # non-negative finite values, ascending, codes 0..126
    mag = y.abs()
    hi = torch.searchsorted(vals, mag.reshape(-1)).clamp(0, 126).reshape(mag.shape)
    lo = (hi - 1).clamp_min(0)
    dh, dl = (vals[hi] - mag).abs(), (vals[lo] - mag).abs()
    pick = torch.where((dl < dh) | ((dl == dh) & (codes[lo] % 2 == 0)), lo, hi)
    code = codes[pick].to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 7)
    scale = torch.where(finite, e + 127, 255.0).to(torch.uint8)
    code = torch.where(finite[..., None], code, torch.zeros_like(code))
    return code, scale


def scale_of(b: torch.Tensor) -> torch.Tensor:
    return torch.where(b == 255, math.nan, torch.exp2(b.double() - 127))


@dataclass
class Q8Problem:
    q_lens: list
    kv_lens: list
    hq: int
    hkv: int
    d: int
    p: int
    dtype: torch.dtype
    causal: bool
    scale: float
    table: torch.Tensor      # [S, width] int32
    q: torch.Tensor          # [T, Hq, D]
    k_codes: torch.Tensor    # uint8 [pages, P, Hkv, D]
    v_codes: torch.Tensor
    k_scales: torch.Tensor   # uint8 [pages, Hkv, P]
    v_scales: torch.Tensor

    @property
    def cu(self):
        return np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)

    def rows(self, s, codes, scales, n):
        """The n first cached rows of sequence s: [n, Hkv, D] float64."""
        pos = torch.arange(n)
        page = self.table[s].long()[pos // self.p]
        bad = (page < 0) | (page >= codes.shape[0])
        page = torch.where(bad, torch.zeros_like(page), page)
        val = E4M3[codes[page, pos % self.p].long()] * scale_of(scales[page, :, pos % self.p])[..., None]
        val[bad] = 0.0
        return val

    def v_scale(self, s, n, h):
        """V scales of the n first cached rows of sequence s, head h (NaN and unreadable ones as 1)."""
        pos = torch.arange(n)
        page = self.table[s].long()[pos // self.p]
        bad = (page < 0) | (page >= self.v_codes.shape[0])
        e = scale_of(self.v_scales[torch.where(bad, 0, page), h, pos % self.p])
        return torch.where(bad | torch.isnan(e), 1.0, e)


def make(q_lens, kv_lens, *, hq, hkv, d, p, dtype=torch.bfloat16, causal=True, seed=0, spare=3, extra_width=1,
         poison=True, scale=None, gain=1.0):
    """A seeded problem; unused pages and slots past kv_len hold NaN codes and
    NaN scales when `poison`."""
    gen = torch.Generator().manual_seed(seed)
    used = [(n + p - 1) // p for n in kv_lens]
    pages = sum(used) + spare
    perm = torch.randperm(pages, generator=gen)
    table = torch.full((len(q_lens), max([1] + used) + extra_width), 0, dtype=torch.int32)
    k_codes = torch.full((pages, p, hkv, d), 0x7F if poison else 0, dtype=torch.uint8)
    v_codes = k_codes.clone()
    k_scales = torch.full((pages, hkv, p), 255 if poison else 127, dtype=torch.uint8)
    v_scales = k_scales.clone()
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = perm[at:at + n].to(torch.int32)
        at += n
        if kv_lens[s] == 0:
            continue
        pos = torch.arange(kv_lens[s])
        page = table[s].long()[pos // p]
        for codes, scales in ((k_codes, k_scales), (v_codes, v_scales)):
            x = torch.randn(kv_lens[s], hkv, d, generator=gen) * gain
            x *= torch.exp(0.7 * torch.randn(kv_lens[s], hkv, 1, generator=gen))    # rows differ in size
            c, e = quantise_row(x)
            codes[page, pos % p] = c
            scales[page, :, pos % p] = e
    q = torch.randn(sum(q_lens), hq, d, generator=gen).to(dtype)
    return Q8Problem(list(q_lens), list(kv_lens), hq, hkv, d, p, dtype, causal,
                     float(scale if scale is not None else 1.0 / math.sqrt(d)), table, q, k_codes, v_codes, k_scales,
                     v_scales)


def attend(pr: Q8Problem):
    """(out, lse, tol_out, tol_lse) in float64, the tolerances element by element.

    Tolerance, with u = eps / 2 of the output type, A = sum_j softmax_j |v_j|
    and ds the largest error of a row's scores:
      ds  = scale * max_j sum_d |q_d k_jd| * D * 2^-24   fp32 accumulation of D products, worst order
          + scale * max|q| * 2^-21 * max_j sum_d |k_jd|  q held as a sum of 8-bit parts
      weights carry exp(ds) and, in bf16, one rounding to bf16 (2^-8), the normaliser
      the same: |out - ref| <= u |out| + A * (2 ds + w), w = 2 * 2^-8 for bf16
      and 2 * 2^-17 for fp32 (weights held to 17 bits or better there),
      plus 2^-16 A (2^-18 for fp32: a row's fp32 sums and exponentials);
      and 2^-29 * C * sum_j |code_jd| over the visible keys, C = max_j softmax_j 2^ev_j the row's
      largest weight times V scale: weights are held relative to C 2^-8 .. C (four e4m3 parts, each
      16 times finer than the one before: the last one's smallest step 2^-9 leaves 2^-10 / 16^3 / 256
      = 2^-30 of the largest) or, in fp16, to at least 2^4 for C, with a smallest half step of 2^-25;
      |lse - ref| <= ds + 2^-20 (1 + |lse|).
    """
    t = sum(pr.q_lens)
    out = torch.zeros(t, pr.hq, pr.d, dtype=torch.float64)
    lse = torch.full((t, pr.hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    g = pr.hq // pr.hkv
    half = torch.finfo(pr.dtype).eps / 2
    w = 2.0 ** -7 + 2.0 ** -16 if pr.dtype == torch.bfloat16 else 2.0 ** -16 + 2.0 ** -18
    at = 0
    for s, (a, b) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        if a and b:
            k, v = pr.rows(s, pr.k_codes, pr.k_scales, b), pr.rows(s, pr.v_codes, pr.v_scales, b)
            q = pr.q[at:at + a].double()
            # a token with a NaN row in K or V is NaN for whoever sees it
            bad = torch.isnan(k).any(-1) | torch.isnan(v).any(-1)            # [b, Hkv]
            for h in range(pr.hq):
                kh, vh = k[:, h // g].nan_to_num(0.0), v[:, h // g].nan_to_num(0.0)
                x = (q[:, h] @ kh.T) * pr.scale
                seen = torch.ones(a, b, dtype=torch.bool)
                if pr.causal:
                    seen = torch.arange(b) <= torch.arange(a)[:, None] + (b - a)
                x = x.masked_fill(~seen, -math.inf)
                some = seen.any(-1)
                m = torch.where(some, x.amax(-1), 0.0)
                e = torch.exp(x - m[:, None])
                total = e.sum(-1)
                pw = e / torch.where(some, total, 1.0)[:, None]
                o, l = pw @ vh, torch.where(some, m + torch.log(total), -math.inf)
                nan = (seen & bad[:, h // g]).any(-1)
                ds = pr.scale * ((q[:, h].abs() @ kh.abs().T).masked_fill(~seen, 0).amax(-1) * pr.d * 2.0 ** -24 +
                                 q[:, h].abs().amax(-1) * 2.0 ** -21 * kh.abs().sum(-1).amax())
                out[at:at + a, h] = torch.where(nan[:, None], math.nan, o)
                lse[at:at + a, h] = torch.where(nan, math.nan, l)
                vs = pr.v_scale(s, b, h // g)
                floor = 2.0 ** -29 * (pw * vs).amax(-1)[:, None] * (seen.double() @ (vh.abs() / vs[:, None]))
                tol_o[at:at + a, h] = half * o.abs() + (pw @ vh.abs()) * (2 * ds[:, None] + w) + floor
                tol_l[at:at + a, h] = torch.where(some, ds + 2.0 ** -20 * (1 + l.abs()), 0.0)
        at += a
    return out, lse, tol_o, tol_l


def check(out, lse, ref, what=""):
    o, l, tol_o, tol_l = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    for name, got, want, tol in (("out", out, o, tol_o), ("lse", lse, l, tol_l)):
        nan = torch.isnan(want)
        assert torch.equal(nan, torch.isnan(got)), f"{what}: NaN of {name} in other places"
        inf = torch.isinf(want)
        assert torch.equal(got[inf], want[inf]) and torch.isfinite(got[~inf & ~nan]).all(), f"{what}: {name} infinite"
        fine = ~nan & ~inf
        err = (got - want).abs()[fine]
        over = err > tol[fine] + 1e-30
        assert not over.any(), (f"{what}: {name} off by {err.max():.3e}, {int(over.sum())} of {over.numel()} over "
                                f"the tolerance, worst ratio {(err / (tol[fine] + 1e-30)).max():.2f}")
