"""Tight bounds of the error of attention over the 8-bit cache, and a model of
the e4m3 parts that the row-group kernel makes of q and of the weights.

u = 2^-24, the largest relative error of an fp32 rounding.  Sums of a row's
largest terms, of what a row sees only:

  scores    x_j = scale q.k_j, S_j = scale sum_d |q_d k_jd|, nz_j nonzero products
    accumulation in fp32, 16 products or more at a time, each time off by one ulp (2 u) of
    the terms' magnitudes at most; adding zeros is exact:  min(D / 16 + 2, nz_j) 2 u S_j
    q in parts: bf16 values down to 2^-12 of the row's largest are exact, smaller ones off by
    2^-21 of the largest; fp32: u of the value and 2^-37 of the largest
    factors, their product, the constant log2 e and the joining of the parts: 5 u |x_j|
    -> ds, the largest of the row
  weights   relative error of exp2's argument (log2 units) with Y = max_j |log2 p_j 2^ev_j| relative
    to the row's maximum, X = max_j |x_j| log2 e, E = max_j |ev_j|:
    three sums behind each other, each off by u of its result, with results up to X + E + 8 + Y,
    and two in the factor of the block: 5 u ln2 (X + E + Y + 16); exp2 itself 2^-22 in
    the weight, the factor and the normaliser
  parts     n of them are off by 2^-(5 n - 1) at most: the first by half a step of 4 bits, 2^-4, and each
    further one takes 4 bits and the sign of a rest that is half a step at most.  Of a weight: four
    (bf16) 2^-19, six (fp32) 2^-29, below u; fp16 in the chunk kernel 2^-11
  floor     a weight's smallest step is 2^-10 / 16^(parts - 1) / 2^8 of C = max_j p_j 2^ev_j, the largest
    weight times V scale (rows of zeros, which add nothing, do not count); in the chunk kernel
    2^-25 / 2^4 of C' = max_j p_j 2^et_j, et_j the largest V scale of the key's 128 (64 at
    head_dim 256) but at most 2^15 ev_j, rows of zeros with 2^-24 of their weight.  Times sum_j |code_j|.
  values    fp32 sums over the keys: kv / 16 + 16 additions of one ulp (2 u)
  out       |out - ref| <= u_out |ref| + A (2 ds + parts + the weights' terms + the sums') + floor
            with A = sum_j p_j |v_j|;  |lse - ref| <= ds + 2^-21 + 4 u |lse| (+ kv / 64 u: its sum)
            + in the chunk kernel, whose exp2's argument is the weight's distance from the row's units, rounded once:
            u ln2 times its largest size: 11 (2^5 at the unit, 2^6 above it) and how far a tile's
            scale is from the unit, 24 above it with rows of zeros, up to 64 below by the spread of the scales
"""
from __future__ import annotations

import math

import torch

import q8_reference as R

U = 2.0 ** -24
LOG2E = math.log2(math.e)


def rows_limit(pr):
    """Longest q_len that the row-group kernel takes."""
    return max(1, 16 // (pr.hq // pr.hkv)) if pr.dtype == torch.bfloat16 else 1 << 30


def codes_of(pr, s, codes, n):
    pos = torch.arange(n)
    page = pr.table[s].long()[pos // pr.p]
    bad = (page < 0) | (page >= codes.shape[0])
    c = R.E4M3[codes[torch.where(bad, 0, page), pos % pr.p].long()]
    c[bad] = 0
    return c


def attend(pr):
    """(out, lse, tol_out, tol_lse) in float64."""
    out, lse, _, _ = R.attend(pr)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    half = torch.finfo(pr.dtype).eps / 2
    g = pr.hq // pr.hkv
    bn = 64 if pr.d == 256 else 128
    at = 0
    for s, (a, b) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        if a and b:
            few = a <= rows_limit(pr)
            parts = U if pr.dtype == torch.float32 else 2.0 ** -19 if few else 2.0 ** -11
            step = 2.0 ** -38 if pr.dtype == torch.float32 else 2.0 ** -30 if few else 2.0 ** -29
            k, v = pr.rows(s, pr.k_codes, pr.k_scales, b), pr.rows(s, pr.v_codes, pr.v_scales, b)
            vcodes = codes_of(pr, s, pr.v_codes, b)
            q = pr.q[at:at + a].double()
            seen = torch.ones(a, b, dtype=torch.bool)
            if pr.causal:
                seen = torch.arange(b) <= torch.arange(a)[:, None] + (b - a)
            some = seen.any(-1)
            for h in range(pr.hq):
                kh, vh, qh = k[:, h // g].nan_to_num(0.0), v[:, h // g].nan_to_num(0.0), q[:, h].nan_to_num(0.0, 0.0, 0.0)
                x = pr.scale * (qh @ kh.T)
                big = qh.abs().amax(-1, keepdim=True)
                sums = pr.scale * (qh.abs() @ kh.abs().T)
                nz = (qh != 0).double() @ (kh != 0).double().T
                if pr.dtype == torch.bfloat16:
                    lost = 2.0 ** -21 * big * (((qh != 0) & (qh.abs() < 2.0 ** -12 * big)).double() @ kh.abs().T)
                else:
                    lost = U * sums / pr.scale + 2.0 ** -37 * big * ((qh != 0).double() @ kh.abs().T)
                ds = (nz.clamp(max=pr.d / 16 + 2) * 2 * U * sums + pr.scale * lost + 5 * U * x.abs())
                ds = ds.masked_fill(~seen, 0).amax(-1)
                ev = torch.log2(pr.v_scale(s, b, h // g))
                codes = vcodes[:, h // g].abs().sum(-1)
                counts = seen & (codes > 0)
                xm = x.masked_fill(~seen, -math.inf)
                m = torch.where(some, xm.amax(-1), 0.0)
                e = torch.exp(xm - m[:, None])
                total = torch.where(some, e.sum(-1), 1.0)
                p = e / total[:, None]
                # exponents (log2) of weight times V scale, relative to the largest weight
                y = ((xm - m[:, None]) * LOG2E + ev).masked_fill(~counts, -math.inf)
                top = y.amax(-1)
                top = torch.where(top == -math.inf, 0.0, top)
                reach = (x.masked_fill(~seen, 0).abs().amax(-1) * LOG2E + ev.masked_fill(codes == 0, 0).abs().max() + top.abs())
                ew = 5 * U * math.log(2) * (reach + 24) + 3 * 2.0 ** -22
                if few:
                    c = torch.exp2(top) / total
                else:
                    live = torch.where(codes > 0, ev, torch.tensor(-math.inf, dtype=ev.dtype))
                    tiles = torch.nn.functional.pad(live, (0, -b % bn), value=-math.inf).view(-1, bn).amax(-1)
                    et = torch.minimum(tiles.repeat_interleave(bn)[:b], ev + 15)
                    z = torch.where(codes > 0, et, tiles.repeat_interleave(bn)[:b] - 24)
                    c = torch.exp2(((xm - m[:, None]) * LOG2E + z).masked_fill(~seen, -math.inf).amax(-1)) / total
                floor = step * c * (seen.double() @ codes)
                big_a = p @ vh.abs()
                rel = 2 * ds + parts + ew + (b / 16 + 16) * 2 * U
                tol_o[at:at + a, h] = half * out[at:at + a, h].nan_to_num(0.0).abs() + big_a * rel[:, None] + floor[:, None] + 1e-37
                l = lse[at:at + a, h].nan_to_num(0.0, 0.0, 0.0).abs()
                far = 0.0
                if not few:
                    real = ev[codes > 0]
                    far = 11 + (24 if (codes == 0).any() else 0) + (min(64, (real.max() - real.min()).item()) if len(real) else 0)
                tol_l[at:at + a, h] = torch.where(some, ds + 2.0 ** -21 + 4 * U * l + (b / 64 + math.log(2) * far) * U, 0.0)
        at += a
    return out, lse, tol_o, tol_l


# ----------------------------------------------------- the parts, on the CPU
def as_parts(x: torch.Tensor, n: int, top: float = 448.0) -> torch.Tensor:
    """x (|x| <= top), as a sum of n e4m3 parts, each 16 times finer than the one before."""
    x = x.double()
    total, rest = torch.zeros_like(x), x.clone()
    for i in range(n):
        part = rest.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
        total += part * 16.0 ** -i
        rest = (rest - part) * 16.0
    return total


def model(pr, nq: int, np_: int, zeros_count=False):
    """(out, lse) of a problem with q in nq parts and the weights of each 128 keys in np_ parts,
    relative to the largest weight times V scale of a row that is not zeros (of any row with
    `zeros_count`); all else in 64 bits."""
    t = sum(pr.q_lens)
    out = torch.zeros(t, pr.hq, pr.d, dtype=torch.float64)
    lse = torch.full((t, pr.hq), -math.inf, dtype=torch.float64)
    g = pr.hq // pr.hkv
    at = 0
    for s, (a, b) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        if a and b:
            k, v = pr.rows(s, pr.k_codes, pr.k_scales, b), pr.rows(s, pr.v_codes, pr.v_scales, b)
            codes = codes_of(pr, s, pr.v_codes, b)
            for h in range(pr.hq):
                q = pr.q[at:at + a, h].double()
                unit = torch.exp2(torch.ceil(torch.log2(q.abs().amax(-1, keepdim=True) / 448)))
                q = as_parts(q / unit, nq) * unit
                ev = torch.log2(pr.v_scale(s, b, h // g))
                live = (codes[:, h // g].abs().sum(-1) > 0) | zeros_count
                seen = torch.arange(b) <= torch.arange(a)[:, None] + (b - a if pr.causal else b)
                x = (pr.scale * (q @ k[:, h // g].T)).masked_fill(~seen, -math.inf)
                m = x.amax(-1, keepdim=True)
                e = torch.exp(x - m)
                o = torch.zeros(a, pr.d, dtype=torch.float64)
                for j in range(0, b, 128):
                    y = (x[:, j:j + 128] - m) * LOG2E + ev[j:j + 128]
                    y = y.masked_fill(~live[j:j + 128], -math.inf)
                    yb = y.amax(-1, keepdim=True)
                    yb = torch.where(yb == -math.inf, 0.0, yb)
                    w = as_parts(torch.exp2(y - yb + 8), np_) * torch.exp2(yb - 8)
                    o += w @ codes[j:j + 128, h // g]
                some = seen.any(-1)
                total = torch.where(some, e.nan_to_num(0.0).sum(-1), 1.0)
                out[at:at + a, h] = torch.where(some[:, None], o / total[:, None], 0.0)
                lse[at:at + a, h] = torch.where(some, m[:, 0] + torch.log(total), -math.inf)
        at += a
    return out, lse


# ------------------------------------- problems whose errors all have one sign
def score_problem(rows=200):
    """fp32 queries that meet one key in one value: lse is that one product.  Its error: the parts
    of q (u), the joining of their products (1.1 u), the product with the factors (u), the constants
    log2 e and ln 2 and the product with the latter (2 u together): at most 5.1 u of lse, where four
    parts of q lose up to 32 u (five are off by u, as the fp32 value is)."""
    pr = R.make([rows], [1], hq=1, hkv=1, d=64, p=8, dtype=torch.float32, causal=False, seed=1)
    one = torch.zeros(1, 1, 64)
    one[..., 0] = 1.0
    c, e = R.quantise_row(one)
    page = pr.table[0, 0].long()
    pr.k_codes[page, 0], pr.k_scales[page, :, 0] = c[0], e[0]
    pr.q[:] = 0
    pr.q[:, 0, 0] = 1 + torch.rand(rows, generator=torch.Generator().manual_seed(2))
    return pr, 5.1 * U


def weight_problem(dtype, rows):
    """53 keys have score 0 and values -v, which cost no rounding, and 75 have scores close to
    log2(53 / 75) in every row and values v: out is close to zero and holds the error of one weight,
    the same for all of those keys.

    Tolerance: the output's rounding, and of sum p |v| over the second kind: the parts of the weight
    (fp32 u, bf16 in the row-group kernel 2^-19, in the chunk kernel 2^-11); of all: exp2 (2^-22 in the
    weight and in the sum), its argument (three sums of at most 8: 17 u), the score (two products, 7 u),
    the sum of the weights (11 u), joining, factor and normalising (6 u): 50 u.  Returns the problem, out, the tolerance
    and the weights of the second kind."""
    gen = torch.Generator().manual_seed(4)
    scale = math.log(75 / 53)
    pr = R.make([rows], [128], hq=1, hkv=1, d=64, p=16, dtype=dtype, causal=False, seed=1, scale=scale)
    k, v = torch.zeros(128, 1, 64), torch.zeros(128, 1, 64)
    k[53:, :, :2] = -1.0
    v[:53] = -256.0                                 # every row's scale is 2^0
    v[53:] = 256.0
    for x, codes, scales in ((k, pr.k_codes, pr.k_scales), (v, pr.v_codes, pr.v_scales)):
        c, e = R.quantise_row(x)
        page, slot = pr.table[0].long()[torch.arange(128) // 16], torch.arange(128) % 16
        codes[page, slot], scales[page, :, slot] = c, e
    pr.q[:] = 0
    pr.q[:, 0, 0] = 1.0
    pr.q[:, 0, 1] = (2.0 ** -8 * (0.1 + torch.rand(rows, generator=gen))).to(dtype) * (torch.arange(rows) % 2 * 2 - 1)
    out = R.attend(pr)[0]
    w = torch.exp(-pr.q[:, 0, :2].double().sum(-1) * scale)
    parts = U if dtype == torch.float32 else 2.0 ** -19 if rows <= rows_limit(pr) else 2.0 ** -11
    tol = torch.finfo(dtype).eps / 2 * out.abs() + 256 * (75 * w / (53 + 75 * w) * parts + 50 * U)[:, None, None]
    return pr, out, tol, w


def zero_sink(dtype, size, q_len=4, kv_len=200, hq=2, hkv=1, d=64, lift=8.0, causal=True, n=1):
    """Problems whose first key has a V row of zeros and scores about `lift` (natural units) above
    the others', the other values being about `size`."""
    gen = torch.Generator().manual_seed(9)
    pr = R.make([q_len] * n, [kv_len] * n, hq=hq, hkv=hkv, d=d, p=16, dtype=dtype, causal=causal, seed=9)
    for s in range(n):
        k = torch.randn(kv_len, hkv, d, generator=gen) * 0.3
        v = torch.randn(kv_len, hkv, d, generator=gen) * size
        k[:, :, 0] = 0
        k[0, :, 0] = 8.0
        v[0] = 0
        pos = torch.arange(kv_len)
        page, slot = pr.table[s].long()[pos // 16], pos % 16
        for x, codes, scales in ((k, pr.k_codes, pr.k_scales), (v, pr.v_codes, pr.v_scales)):
            c, e = R.quantise_row(x)
            codes[page, slot], scales[page, :, slot] = c, e
    pr.q[..., 0] = lift / (8.0 * pr.scale)
    return pr
