"""The 8-bit cache's kernels where their bookkeeping or arithmetic can go wrong:
rings, masks that leave a block's rows empty, units of the accumulators, rows
of zeros, the top of the format's range."""
from dataclasses import replace

import pytest
import torch

import q8_reference as R
from test_q8_gpu import BF16, Dev, lib  # noqa: F401 (lib: builds the library)

pytestmark = pytest.mark.gpu


def places(pr, s, pos):
    """Page and slot of positions `pos` (a tensor) of sequence s."""
    return pr.table[s].long()[pos // pr.p], pos % pr.p


@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunk_scales_change_from_block_to_block(d):
    """V scales that differ by 2^6 from key to key, the other way round in the next
    block: a factor taken from another block would show at once.  Repeats bit for bit."""
    pr = R.make([300, 150, 280], [3000, 2500, 280], hq=4, hkv=4, d=d, p=16, seed=3)
    for s, b in enumerate(pr.kv_lens):
        pos = torch.arange(b)
        page, slot = places(pr, s, pos)
        up = ((pos + pos // 128) % 2 * 6).to(torch.uint8)[:, None]
        pr.v_scales[page, :, slot] += up
    dv = Dev(pr).attend()
    dv.checked(what=f"head_dim {d}")
    first = dv.out.clone(), dv.lse.clone()
    for _ in range(20):
        dv.out.fill_(77.0)
        dv.attend()
        assert torch.equal(dv.out, first[0]) and torch.equal(dv.lse, first[1])


def low_scores(pr, by):
    """Shifts every score of the problem down by about `by` (natural units): the first value of
    each K row becomes the largest power of two it can hold, q's first one its opposite."""
    for codes in (pr.k_codes,):
        codes[..., 0] = 0x70                       # 2^7 of the row's scale
    for s, b in enumerate(pr.kv_lens):
        if b:
            page, slot = places(pr, s, torch.arange(b))
            pr.k_scales[page, :, slot] = 121       # 2^-6: k_0 = 2
    pr.q[..., 0] = -by / (2 * pr.scale)


@pytest.mark.parametrize("by", [90.0, 100.0, 300.0, 5000.0])
@pytest.mark.parametrize("dtype,hq,q_len", [(BF16, 8, 3), (BF16, 16, 8), (BF16, 8, 16), (torch.float32, 8, 3), (torch.float32, 16, 40)])
def test_rows_without_a_key_in_a_block_and_low_scores(dtype, hq, q_len, by):
    """The causal mask hides a sequence's last block from all but its last tokens, and all scores
    are far below zero.  Many sequences, so that one CTA runs over both blocks of a group."""
    n = 120
    pr = R.make([q_len] * n, [128 + 1 + i % max(1, q_len - 1) for i in range(n)], hq=hq, hkv=8, d=64, p=16,
                dtype=dtype, seed=5)
    low_scores(pr, by)
    Dev(pr).attend().checked(what=f"scores around -{by}")


def set_rows(pr, s, k, v):
    """Sequence s holds the rows k, v [kv_len, Hkv, D], quantised."""
    page, slot = places(pr, s, torch.arange(pr.kv_lens[s]))
    for x, codes, scales in ((k, pr.k_codes, pr.k_scales), (v, pr.v_codes, pr.v_scales)):
        c, e = R.quantise_row(x)
        codes[page, slot] = c
        scales[page, :, slot] = e


@pytest.mark.parametrize("fade", [0.0, 0.35])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_beside_one_whose_maximum_climbs(d, fade):
    """One row's scores climb by 10 every 64 keys, which rescales its warp's sums each time.  The
    other rows have flat scores, of maxima from 90 to 180, or scores that climb slowly on values
    that shrink by 2^fade every 64 keys: their outputs count every key.  The sequence many times
    over, so that one CTA runs over most of it."""
    steps, gen = 60, torch.Generator().manual_seed(7)
    n = 64 * steps
    pr = R.make([64], [n], hq=1, hkv=1, d=d, p=16, causal=False, scale=0.7)
    t = 14 * (torch.arange(n) // 64)
    k = torch.zeros(n, 1, d)
    for i, cap in enumerate((448, 448, 16)):           # exact codes: multiples of 32, then small integers
        part = (t - t % 32 if i < 2 else t).clamp(max=cap)
        k[:, 0, i] = part
        t = t - part
    k[:, 0, 3] = t
    k[:, 0, 5] = 128.0
    k[:, 0, 6] = fade * torch.log(torch.tensor(2.0)) / 0.7 * (torch.arange(n) // 64) * 32
    v = torch.rand(n, 1, d, generator=gen) + 0.5
    v *= torch.exp2(-fade * (torch.arange(n) // 64))[:, None, None]
    set_rows(pr, 0, k, v)
    pr.q[:] = 0
    pr.q[:, 0, 5] = 1 + torch.arange(64) / 64
    pr.q[:, 0, 6] = 1 / 32
    for r in (5, 37):                                  # one row of each warp
        pr.q[r] = 0
        pr.q[r, 0, :4] = 1
    ref, times = R.attend(pr), 150
    pr = replace(pr, q_lens=pr.q_lens * times, kv_lens=pr.kv_lens * times, table=pr.table.repeat(times, 1),
                 q=pr.q.repeat(times, 1, 1))
    Dev(pr).attend().checked([x.repeat(times, *[1] * (x.dim() - 1)) for x in ref], what=f"head_dim {d}")


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_largest_finite_rows_stay_finite(d, dtype):
    """Values up to the types' largest: the codes that would stand for 2^128 are those below."""
    pr = R.make([40], [40], hq=2, hkv=2, d=d, p=16, dtype=dtype, seed=1)
    gen = torch.Generator().manual_seed(8)
    rows = []
    for i in range(2):
        x = (torch.rand(40, 2, d, generator=gen) * 2 - 1) * torch.finfo(dtype).max
        x[0] = torch.finfo(dtype).max
        x[1] = -torch.finfo(dtype).max
        x[2, :, ::2] = 248.0 * 2.0 ** 120                      # half way between 240 and 256
        x[3] = torch.linspace(200.0, 255.0, d) * 2.0 ** 120
        x[4] = 448.0 * 2.0 ** 119                              # the largest of the scale below
        rows.append(x.to(dtype))
    assert all(torch.isfinite(x).all() for x in rows)
    dv = Dev(pr)
    dv.rb.rpa_q8_write(rows[0].cuda(), rows[1].cuda(), *dv.cache, dev_flags=dv.flags)
    back = [torch.empty_like(r, device="cuda") for r in rows]
    dv.rb.rpa_q8_read(*back, *dv.cache, dev_flags=dv.flags)
    assert int(dv.flags.item()) == 0
    page, slot = places(pr, 0, torch.arange(40))
    for x, got, codes, scales in zip(rows, back, (dv.kc, dv.vc), (dv.ks, dv.vs)):
        c, e = R.quantise_row(x)
        top = (e == 247)[..., None] & ((c & 0x7F) == 0x78)
        assert top.any() and (e == 246).any()
        c = torch.where(top, c - 1, c)
        assert torch.equal(codes.view(torch.uint8).cpu()[page, slot], c)
        assert torch.equal(scales.view(torch.uint8).cpu()[page, :, slot], e)
        got = got.double().cpu()
        assert torch.equal(got, R.E4M3[c.long()] * R.scale_of(e)[..., None]) and torch.isfinite(got).all()
        err = (got - x.double()).abs()
        assert (err <= torch.maximum(x.double().abs() * 2.0 ** -4, R.scale_of(e)[..., None] * 2.0 ** -10)).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,causal", [(10, 2, False), (6, 2, True), (14, 2, True), (10, 2, True)])
def test_rows_of_a_tile_without_a_query_do_not_matter(hq, hkv, causal, d):
    """A G that does not divide 128 leaves rows of a tile without a query: what a call before left there
    (in every SM, at G = 1, where a tile has none) changes no bit."""
    pr = R.make([171, 172, 180, 103], [946, 262, 194, 1489], hq=hq, hkv=hkv, d=d, p=32, causal=causal, seed=6,
                scale=0.19 / d ** 0.5)
    pr.q[:] = pr.q.abs()
    pr.k_codes &= 0x7F                              # all scores positive, some far above others
    before = Dev(R.make([300] * 80, [300] * 80, hq=2, hkv=2, d=d, p=32, causal=False, seed=7))
    before.q.fill_(0.0)
    before.attend()
    dv = Dev(pr).attend()
    first = dv.out.clone(), dv.lse.clone()
    for fill in (torch.nan, 1e30, 1.0, torch.inf):
        before.q.fill_(fill)
        before.attend()
        dv.out.fill_(77.0)
        dv.attend()
        assert torch.equal(dv.out, first[0]) and torch.equal(dv.lse, first[1]), f"after queries of {fill}"
