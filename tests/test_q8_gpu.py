"""The 8-bit cache on the GPU against the 64-bit reference: write and read bit
for bit, attention within derived tolerances, and a run of the three together
as a serving loop makes it."""
import math

import numpy as np
import pytest
import torch

import q8_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ragged_paged_attention_03_b200 import build
    build.build()


def f8(t):
    return t.cuda().view(torch.float8_e4m3fn)


def e8(t):
    return t.cuda().view(torch.float8_e8m0fnu)


class Dev:
    """Device copies of a problem's arrays, with room for `more_seqs` unused
    sequences and `more_rows` unused rows."""

    def __init__(self, pr, more_seqs=0, more_rows=0):
        from ragged_paged_attention_03_b200 import binding as rb
        self.rb, self.pr = rb, pr
        s = len(pr.q_lens) + more_seqs
        self.table = torch.full((s, pr.table.shape[1]), -7, dtype=torch.int32)
        self.table[:len(pr.q_lens)] = pr.table
        self.table = self.table.cuda()
        self.cu = torch.full((s + 1,), -3, dtype=torch.int32)
        self.cu[:len(pr.cu)] = torch.from_numpy(pr.cu)
        self.cu = self.cu.cuda()
        self.kv = torch.full((s,), -5, dtype=torch.int32)
        self.kv[:len(pr.kv_lens)] = torch.tensor(pr.kv_lens, dtype=torch.int32)
        self.kv = self.kv.cuda()
        self.n = torch.tensor([len(pr.q_lens)], dtype=torch.int32).cuda()
        self.kc, self.vc = f8(pr.k_codes.clone()), f8(pr.v_codes.clone())
        self.ks, self.vs = e8(pr.k_scales.clone()), e8(pr.v_scales.clone())
        t = pr.q.shape[0] + more_rows
        self.q = torch.full((t, pr.hq, pr.d), math.nan, dtype=pr.dtype, device="cuda")
        self.q[:pr.q.shape[0]] = pr.q.cuda()
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full_like(self.q, 77.0)
        self.lse = torch.full((t, pr.hq), 77.0, dtype=F32, device="cuda")
        self.max_q = max([1] + pr.q_lens)
        dims = rb.make_dims(self.q, self.kc, self.table)
        size = rb.rpa_q8_workspace_size(dims, s, self.max_q)
        # poisoned, with a guard behind it that must keep its bytes
        # (bytes of a large positive integer: no word of it may be taken for a result)
        self.ws_all = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        self.ws = self.ws_all[:size]

    @property
    def cache(self):
        return self.kc, self.vc, self.ks, self.vs, self.table, self.cu, self.kv, self.n

    def attend(self, **kw):
        a = dict(max_q_len=self.max_q, scale=self.pr.scale, causal=self.pr.causal, out=self.out, workspace=self.ws,
                 lse=self.lse, dev_flags=self.flags)
        a.update(kw)
        self.rb.rpa_q8_attend(self.q, *self.cache, **a)
        return self

    def checked(self, ref=None, what="", flags=0):
        torch.cuda.synchronize()
        assert int(self.flags.item()) == flags
        t = self.pr.q.shape[0]
        R.check(self.out[:t], self.lse[:t], ref if ref is not None else R.attend(self.pr), what)
        assert (self.out[t:] == 77).all() and (self.lse[t:] == 77).all(), "rows behind the batch were written"
        assert (self.ws_all[self.ws.numel():] == 0x5A).all(), "written past the workspace"


# --------------------------------------------------------------- write / read
IO = [  # q_lens, kv_lens, hkv, d, p
    ([1], [1], 1, 64, 8),
    ([1, 1, 1], [37, 16, 1], 8, 128, 16),
    ([5, 0, 33, 1], [5, 7, 40, 300], 3, 64, 8),
    ([100, 1, 0, 17, 64], [130, 250, 0, 17, 64], 4, 256, 64),
    ([300, 7], [700, 7], 2, 128, 256),
    ([1] * 70, list(range(1, 71)), 1, 256, 32),
]


def io_problem(case, seed, dtype, poison):
    q_lens, kv_lens, hkv, d, p = case
    return R.make(q_lens, kv_lens, hq=hkv, hkv=hkv, d=d, p=p, dtype=dtype, seed=seed, poison=poison)


def new_rows(pr, seed, dtype, odd=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(sum(pr.q_lens), pr.hkv, pr.d, generator=gen)
    x *= torch.exp(4 * torch.randn(x.shape[0], pr.hkv, 1, generator=gen))
    if odd and x.shape[0] > 8:
        x[1, 0] = 0
        x[2, 0] = 1e-41            # subnormal
        x[3, 0] = 3e38
        x[4, 0, 5] = math.inf
        x[5, 0, pr.d - 1] = math.nan
        x[6, 0] = torch.linspace(-448, 448, pr.d)          # ties among them
        x[7, 0] = 1.0                                      # amax far from the scale's border
        x[8, 0] = -448.0 * 2.0 ** -20                      # on the border
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(IO)))
def test_write_is_exact(case, dtype):
    pr = io_problem(IO[case], case, dtype, True)
    dv = Dev(pr, more_seqs=2, more_rows=3)
    rows = [new_rows(pr, 100 + i, dtype) for i in range(2)]
    wide = [torch.full((r.shape[0] + 3, *r.shape[1:]), 5.0, dtype=dtype) for r in rows]
    want = []
    for r, w, codes, scales in zip(rows, wide, (pr.k_codes, pr.v_codes), (pr.k_scales, pr.v_scales)):
        w[:r.shape[0]] = r
        codes, scales = codes.clone(), scales.clone()
        c, e = R.quantise_row(r)
        at = 0
        for s, (a, b) in enumerate(zip(pr.q_lens, pr.kv_lens)):
            pos = torch.arange(b - a, b)
            page = pr.table[s].long()[pos // pr.p]
            codes[page, pos % pr.p] = c[at:at + a]
            scales[page, :, pos % pr.p] = e[at:at + a]
            at += a
        want.append((codes, scales))
    dv.rb.rpa_q8_write(wide[0].cuda(), wide[1].cuda(), *dv.cache, dev_flags=dv.flags)
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == 0
    for got, (codes, scales) in zip(((dv.kc, dv.ks), (dv.vc, dv.vs)), want):
        assert torch.equal(got[1].view(torch.uint8).cpu(), scales)
        assert torch.equal(got[0].view(torch.uint8).cpu(), codes)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(IO)))
def test_read_is_exact(case, dtype):
    pr = io_problem(IO[case], case, dtype, True)
    dv = Dev(pr, more_seqs=2, more_rows=3)
    t = sum(pr.q_lens)
    outs = [torch.full((t + 3, pr.hkv, pr.d), 77.0, dtype=dtype, device="cuda") for _ in range(2)]
    dv.rb.rpa_q8_read(*outs, *dv.cache, dev_flags=dv.flags)
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == 0
    for got, codes, scales in zip(outs, (pr.k_codes, pr.v_codes), (pr.k_scales, pr.v_scales)):
        want = torch.cat([pr.rows(s, codes, scales, b)[b - a:] for s, (a, b) in
                          enumerate(zip(pr.q_lens, pr.kv_lens))])
        assert torch.equal(got[:t].cpu(), want.to(dtype))
        assert (got[t:] == 77).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_read_of_extreme_scales(dtype):
    """Every scale byte, NaN and the subnormal end among them, every code."""
    pr = R.make([256], [256], hq=1, hkv=1, d=256, p=16, dtype=dtype, poison=False, spare=0, extra_width=0)
    codes = torch.arange(256, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x11
    page = pr.table[0].long()
    pr.k_codes[page] = codes.expand(16, 16, 1, 256).clone()
    pr.k_scales[page] = torch.arange(256, dtype=torch.uint8).view(16, 1, 16)
    dv = Dev(pr)
    outs = [torch.empty(256, 1, 256, dtype=dtype, device="cuda") for _ in range(2)]
    dv.rb.rpa_q8_read(*outs, *dv.cache)
    want = pr.rows(0, pr.k_codes, pr.k_scales, 256).to(dtype)
    nan = torch.isnan(want)
    assert nan[255].all() and not nan[:255].any()
    got = outs[0].cpu()
    assert torch.equal(nan, torch.isnan(got)) and torch.equal(got[~nan], want[~nan])


def test_write_skips_bad_pages_and_reports():
    pr = io_problem(IO[2], 1, BF16, True)
    pr.table[2, 1] = pr.k_codes.shape[0]       # positions 8..15 of sequence 2
    pr.table[3, 37] = -1                       # position 299 of sequence 3: its one new token
    dv = Dev(pr)
    rows = new_rows(pr, 5, BF16).cuda()
    before = dv.kc.view(torch.uint8).clone()
    dv.rb.rpa_q8_write(rows, rows, *dv.cache, dev_flags=dv.flags)
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == dv.rb.RPA_DEV_BAD_PAGE
    changed = (dv.kc.view(torch.uint8) != before).flatten(2).any(-1).sum().item()
    # 5 + 33 new tokens of sequences 0 and 2, less the one of 2's on the bad page (7..39 new: 8..15 bad)
    assert changed == 5 + 33 - 8
    moved = dv.kc.view(torch.uint8) != before
    assert torch.equal(dv.kc.view(torch.uint8)[moved], dv.vc.view(torch.uint8)[moved])
    out = torch.full((39, 3, 64), 77.0, dtype=BF16, device="cuda")
    dv.rb.rpa_q8_read(out, out.clone(), *dv.cache, dev_flags=dv.flags)
    assert (out[5 + 1:5 + 9] == 0).all() and (out[38] == 0).all()


# ------------------------------------------------------------------ attention
G = dict(  # name: q_lens, kv_lens, hq, hkv, d, p, causal
    one_key=([1], [1], 1, 1, 64, 8, True),
    one=([1], [100], 4, 1, 64, 16, True),
    decode=([1] * 9, [1, 15, 16, 17, 127, 128, 129, 300, 2049], 8, 2, 128, 16, True),
    decode_g1=([1] * 5, [5, 64, 65, 700, 1], 3, 3, 128, 8, True),
    decode_g16=([1] * 4, [33, 1000, 2, 257], 32, 2, 64, 32, True),
    decode_g7=([1] * 4, [33, 1000, 2, 257], 14, 2, 128, 128, True),
    decode_d256=([1] * 6, [900, 3, 129, 64, 511, 1], 8, 2, 256, 64, True),
    decode_d256_g16=([1] * 3, [900, 3, 129], 16, 1, 256, 256, True),
    decode_long=([1, 1], [9000, 20000], 4, 1, 128, 16, True),
    few=([2, 3, 4, 1, 0, 5], [2, 100, 515, 64, 50, 1029], 8, 2, 128, 16, True),
    few_cross=([2, 3, 4, 1, 0, 5], [0, 100, 3, 64, 50, 1029], 8, 2, 64, 16, False),
    longer_than_kv=([9, 40, 3], [4, 0, 1], 4, 2, 128, 8, True),
    chunk=([50, 17, 1, 128, 129], [50, 80, 37, 128, 700], 8, 2, 128, 16, True),
    chunk_d64=([65, 300, 2], [65, 811, 1000], 6, 3, 64, 8, True),
    chunk_d256=([70, 140, 1], [500, 140, 333], 4, 2, 256, 64, True),
    chunk_mha=([200, 31], [333, 31], 3, 3, 128, 256, True),
    chunk_g16=([20, 33], [333, 64], 16, 1, 128, 32, True),
    chunk_g5=([40, 9], [333, 64], 10, 2, 64, 16, True),
    cross=([1, 40, 333, 20], [600, 0, 77, 1], 4, 4, 64, 32, False),
    cross_gqa=([100, 257], [1000, 129], 8, 2, 128, 16, False),
    cross_d256=([100, 57], [300, 129], 4, 2, 256, 16, False),
    fresh=([513, 256], [513, 256], 4, 1, 128, 16, True),
    many_short=([17 + i % 30 for i in range(100)], [17 + i % 30 + (i % 7) * 20 for i in range(100)], 16, 16, 64, 16, True),
    many_short_gqa=([9 + i % 70 for i in range(60)], [9 + i % 70 for i in range(60)], 32, 8, 128, 16, True),
    long_ctx=([20], [6000], 4, 1, 128, 16, True),
)


def problem(name, dtype=BF16, **kw):
    q, kv, hq, hkv, d, p, causal = G[name]
    return R.make(q, kv, hq=hq, hkv=hkv, d=d, p=p, causal=causal, dtype=dtype,
                  **{"seed": sorted(G).index(name), **kw})


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", sorted(G))
def test_attend(name, dtype):
    Dev(problem(name, dtype), more_seqs=3, more_rows=5).attend().checked(what=name)


@pytest.mark.parametrize("name", ["decode", "chunk", "chunk_d256", "cross", "few"])
def test_attend_without_lse_or_flags(name):
    pr = problem(name)
    dv = Dev(pr).attend(lse=None, dev_flags=None)
    assert (dv.lse == 77).all()
    dv.attend().checked(what=name)


@pytest.mark.parametrize("name", ["decode", "chunk", "fresh", "cross_gqa"])
def test_attend_loose_max_q(name):
    """max_q_len is a bound, not the longest: another choice of kernels."""
    dv = Dev(problem(name))
    dims = dv.rb.make_dims(dv.q, dv.kc, dv.table)
    ws = torch.full((dv.rb.rpa_q8_workspace_size(dims, dv.kv.numel(), 5000),), 0x5A, dtype=torch.uint8, device="cuda")
    dv.attend(max_q_len=5000, workspace=ws).checked(what=name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["decode", "chunk", "chunk_d256", "few_cross"])
def test_attend_nan_rows_stay_behind_the_mask(name, dtype):
    """A NaN row of K or V reaches the query rows that see it and no other."""
    pr = problem(name, dtype)
    for s, (a, b) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        for pos, scales in ((b - 1, pr.k_scales), (b - 3, pr.v_scales)):
            if pos > 0 and a > 1:
                scales[pr.table[s, pos // pr.p].long(), 0, pos % pr.p] = 255
    ref = R.attend(pr)
    assert torch.isnan(ref[0]).any() and not torch.isnan(ref[0]).all() or name == "decode"
    Dev(pr).attend().checked(ref, what=name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["decode", "chunk"])
def test_attend_nan_query_stays_in_its_head(name, dtype):
    pr = problem(name, dtype)
    t = sum(pr.q_lens) - 1
    pr.q[t, 1, 3] = math.nan
    pr.q[0, 0, 0] = math.inf
    out, lse, tol_o, tol_l = R.attend(pr)
    dv = Dev(pr).attend()
    for r, h in ((t, 1), (0, 0)):
        assert torch.isnan(dv.out[r, h]).all()
        dv.out[r, h], dv.lse[r, h] = 0, 0
        out[r, h], lse[r, h] = 0, 0
    dv.checked((out, lse, tol_o, tol_l), what=name)


@pytest.mark.parametrize("gain,scale", [(1e-12, 1e11), (1e10, 1e-11), (30.0, None), (1e-3, None)])
@pytest.mark.parametrize("name", ["decode", "chunk"])
def test_attend_large_and_small_values(name, gain, scale):
    """Keys far from 1 (their scales far from 2^0) and sharp or flat softmaxes."""
    Dev(problem(name, gain=gain, scale=scale)).attend().checked(what=name)


@pytest.mark.parametrize("name", ["decode", "chunk", "few"])
def test_attend_one_loud_token(name):
    """One key far above the others, and one value row 2^12 times the others' size."""
    pr = problem(name)
    for s, b in enumerate(pr.kv_lens):
        if b > 4:
            pr.v_scales[pr.table[s, 0].long(), :, 1] += 12
            pr.k_scales[pr.table[s, (b // 2) // pr.p].long(), 0, (b // 2) % pr.p] += 4
    Dev(pr).attend().checked(what=name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["decode", "decode_d256", "few", "chunk", "chunk_d64", "fresh", "cross_gqa"])
def test_attend_scales_far_apart(name, dtype):
    """Rows of one sequence that differ in size by up to 2^60, rows of zeros
    (scale 2^0) among far smaller ones, and a huge last token, which a causal
    mask hides from all rows but the last."""
    pr = problem(name, dtype, gain=1e-6)
    gen = torch.Generator().manual_seed(5)
    for s, b in enumerate(pr.kv_lens):
        if b == 0:
            continue
        pos = torch.arange(b)
        page, slot = pr.table[s].long()[pos // pr.p], pos % pr.p
        dk = torch.randint(-40, 20, (b, pr.hkv), generator=gen)
        dv = torch.randint(-30, 31, (b, pr.hkv), generator=gen)
        if b > 40:
            dv[-1] += 40
            dv[b // 2:b // 2 + 8] = -60
        for scales, d in ((pr.k_scales, dk), (pr.v_scales, dv)):
            scales[page, :, slot] = (scales[page, :, slot].int() + d).to(torch.uint8)
        zero = torch.randperm(b, generator=gen)[:b // 8]
        for codes, scales in ((pr.k_codes, pr.k_scales), (pr.v_codes, pr.v_scales)):
            codes[page[zero], slot[zero]] = 0
            scales[page[zero], :, slot[zero]] = 127
    Dev(pr).attend().checked(what=name)


@pytest.mark.parametrize("name", ["decode", "chunk", "chunk_d64", "chunk_d256", "few"])
def test_attend_bad_pages_read_as_zeros(name):
    pr = problem(name)
    bad = 0
    for s, b in enumerate(pr.kv_lens):
        if b > 3 * pr.p:
            pr.table[s, 1] = -1 if s % 2 else pr.k_codes.shape[0]
            bad += 1
    assert bad
    dv = Dev(pr)
    dv.attend().checked(flags=dv.rb.RPA_DEV_BAD_PAGE, what=name)


BAD = {
    "decreasing": lambda d: d.cu.__setitem__(2, int(d.cu[1]) - 1),
    "not from 0": lambda d: d.cu.__setitem__(0, 1),
    "past T": lambda d: d.cu.__setitem__(len(d.pr.q_lens), d.q.shape[0] + 1),
    "negative kv": lambda d: d.kv.__setitem__(1, -1),
    "kv past the table": lambda d: d.kv.__setitem__(1, d.table.shape[1] * d.pr.p + 1),
    "too many": lambda d: d.n.fill_(d.kv.numel() + 1),
    "negative count": lambda d: d.n.fill_(-1),
}


@pytest.mark.parametrize("how", sorted(BAD))
@pytest.mark.parametrize("name", ["decode", "chunk"])
def test_bad_lengths_write_nothing(name, how):
    pr = problem(name)
    dv = Dev(pr)
    BAD[how](dv)
    dv.attend()
    assert int(dv.flags.item()) == 4
    assert (dv.out == 77).all() and (dv.lse == 77).all()
    rows = torch.ones(sum(pr.q_lens), pr.hkv, pr.d, dtype=BF16, device="cuda")
    before = [t.view(torch.uint8).clone() for t in (dv.kc, dv.vc, dv.ks, dv.vs)]
    got = torch.full_like(rows, 77.0)
    for call, a in ((dv.rb.rpa_q8_write, rows), (dv.rb.rpa_q8_read, got)):
        dv.flags.zero_()
        call(a, a.clone() if call is dv.rb.rpa_q8_write else got, *dv.cache, dev_flags=dv.flags)
        assert int(dv.flags.item()) == 4
    assert (got == 77).all()
    for b, t in zip(before, (dv.kc, dv.vc, dv.ks, dv.vs)):
        assert torch.equal(b, t.view(torch.uint8))


def test_q_len_above_the_bound_writes_nothing():
    dv = Dev(problem("chunk"))
    dv.attend(max_q_len=16)
    assert int(dv.flags.item()) == 4 and (dv.out == 77).all()


def test_write_needs_kv_not_below_q():
    dv = Dev(problem("longer_than_kv"))
    rows = torch.ones(52, 2, 128, dtype=BF16, device="cuda")
    dv.rb.rpa_q8_write(rows, rows, *dv.cache, dev_flags=dv.flags)
    assert int(dv.flags.item()) == 4


def test_no_sequences():
    dv = Dev(problem("decode"))
    dv.n.zero_()
    dv.attend()
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == 0 and (dv.out == 77).all()


@pytest.mark.parametrize("name", ["decode", "decode_long", "chunk", "long_ctx", "few"])
def test_repeats_bit_for_bit(name):
    """The same call twice, and beside another one on another stream with a workspace of its own."""
    dv, other = Dev(problem(name)), Dev(problem(name, seed=99))
    dv.attend()
    first = (dv.out.clone(), dv.lse.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        other.attend(stream=side)
        dv.attend()
    torch.cuda.synchronize()
    assert torch.equal(dv.out, first[0]) and torch.equal(dv.lse, first[1])
    other.checked(what=name)


@pytest.mark.parametrize("names", [("decode", "decode"), ("chunk", "chunk"), ("few", "few")])
def test_captured_and_replayed(names):
    """One graph of write, attend and read, replayed over batches of other
    lengths; what it does is what the calls do outside a graph."""
    name = names[0]
    q, kv, hq, hkv, d, p, causal = G[name]
    pr = R.make(q, kv, hq=hq, hkv=hkv, d=d, p=p, causal=causal, seed=1, poison=True)
    dv = Dev(pr, more_seqs=1, more_rows=8)
    t = dv.q.shape[0]
    k_new = torch.zeros(t, hkv, d, dtype=BF16, device="cuda")
    v_new = torch.zeros_like(k_new)
    k_out, v_out = torch.zeros_like(k_new), torch.zeros_like(k_new)

    def step():
        dv.rb.rpa_q8_write(k_new, v_new, *dv.cache, dev_flags=dv.flags)
        dv.attend()
        dv.rb.rpa_q8_read(k_out, v_out, *dv.cache, dev_flags=dv.flags)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.RandomState(7)
    for trial in range(4):
        # other lengths within the capacities: some sequences shorter, some gone
        q2 = [int(rng.randint(0, a + 1)) for a in q]
        kv2 = [int(rng.randint(a, b + 1)) for a, b in zip(q2, kv)]
        if trial == 3:
            q2, kv2 = q2[:-1], kv2[:-1]
        pr2 = R.make(q2, kv2, hq=hq, hkv=hkv, d=d, p=p, causal=causal, seed=50 + trial, spare=0, extra_width=0)
        pages, width = pr2.k_codes.shape[0], pr2.table.shape[1]
        for big, small in ((dv.kc, pr2.k_codes), (dv.vc, pr2.v_codes), (dv.ks, pr2.k_scales), (dv.vs, pr2.v_scales)):
            big.view(torch.uint8)[:pages] = small.cuda()
        rows = [new_rows(pr2, 60 + trial + i, BF16, odd=False) for i in range(2)]
        n, tt = len(q2), sum(q2)
        dv.table[:n, :width] = pr2.table.cuda()
        dv.cu[:n + 1] = torch.from_numpy(pr2.cu).cuda()
        dv.kv[:n] = torch.tensor(kv2, dtype=torch.int32)
        dv.n.fill_(n)
        dv.q[:tt] = pr2.q.cuda()
        k_new[:tt], v_new[:tt] = rows[0].cuda(), rows[1].cuda()
        for x in (dv.out, dv.lse, k_out, v_out):
            x.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert int(dv.flags.item()) == 0
        # the reference's cache with the new rows written
        at = 0
        for s, (a, b) in enumerate(zip(q2, kv2)):
            pos = torch.arange(b - a, b)
            page = pr2.table[s].long()[pos // p]
            for r, codes, scales in zip(rows, (pr2.k_codes, pr2.v_codes), (pr2.k_scales, pr2.v_scales)):
                c, e = R.quantise_row(r[at:at + a])
                codes[page, pos % p] = c
                scales[page, :, pos % p] = e
            at += a
        R.check(dv.out[:tt], dv.lse[:tt], R.attend(pr2), f"{name} replay {trial}")
        want = torch.cat([pr2.rows(s, pr2.k_codes, pr2.k_scales, b)[b - a:] for s, (a, b) in
                          enumerate(zip(q2, kv2))])
        assert torch.equal(k_out[:tt].cpu(), want.to(BF16))
        assert (dv.out[tt:] == 77).all() and (k_out[tt:] == 77).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hq,hkv,p", [(128, 8, 2, 16), (64, 4, 4, 8), (256, 4, 1, 64)])
def test_serving_loop(d, hq, hkv, p, dtype):
    """A prompt, then single tokens, each step write -> attend, as a model
    calls them; at the end everything is read back and attended to afresh."""
    from ragged_paged_attention_03_b200 import binding as rb
    gen = torch.Generator().manual_seed(11)
    prompt, steps = [37, 130, 5], 6
    total = [a + steps for a in prompt]
    width = (max(total) + p - 1) // p
    pages = 3 * width
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(3, width)
    pr = R.Q8Problem([], [], hq, hkv, d, p, dtype, True, 1 / math.sqrt(d), table, None,
                     torch.full((pages, p, hkv, d), 0x7F, dtype=torch.uint8),
                     torch.full((pages, p, hkv, d), 0x7F, dtype=torch.uint8),
                     torch.full((pages, hkv, p), 255, dtype=torch.uint8),
                     torch.full((pages, hkv, p), 255, dtype=torch.uint8))
    kc, vc, ks, vs = f8(pr.k_codes), f8(pr.v_codes), e8(pr.k_scales), e8(pr.v_scales)
    kc, vc, ks, vs = kc.clone(), vc.clone(), ks.clone(), vs.clone()
    pt = table.cuda()
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = [0, 0, 0]
    for step in range(steps + 1):
        q_lens = prompt if step == 0 else [1, 1, 1]
        kv = [a + b for a, b in zip(kv, q_lens)]
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        t = int(cu[-1])
        q, k, v = (torch.randn(t, h, d, generator=gen).to(dtype) for h in (hq, hkv, hkv))
        cud, kvd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu.tolist(), kv))
        out = torch.empty(t, hq, d, dtype=dtype, device="cuda")
        lse = torch.empty(t, hq, device="cuda")
        dims = rb.make_dims(out, kc, pt)
        ws = torch.empty(rb.rpa_q8_workspace_size(dims, 3, max(q_lens)), dtype=torch.uint8, device="cuda")
        rb.rpa_q8_write(k.cuda(), v.cuda(), kc, vc, ks, vs, pt, cud, kvd, n, dev_flags=flags)
        rb.rpa_q8_attend(q.cuda(), kc, vc, ks, vs, pt, cud, kvd, n, max(q_lens), pr.scale, True, out, ws, lse=lse,
                         dev_flags=flags)
        pr.q_lens, pr.kv_lens, pr.q = list(q_lens), list(kv), q
        for s in range(3):
            pos = torch.arange(kv[s] - q_lens[s], kv[s])
            page = table[s].long()[pos // p]
            for x, codes, scales in ((k, pr.k_codes, pr.k_scales), (v, pr.v_codes, pr.v_scales)):
                c, e = R.quantise_row(x[cu[s]:cu[s + 1]])
                codes[page, pos % p] = c
                scales[page, :, pos % p] = e
        R.check(out, lse, R.attend(pr), f"step {step}")
    assert int(flags.item()) == 0
    cud = torch.tensor(np.concatenate([[0], np.cumsum(kv)]).tolist(), dtype=torch.int32, device="cuda")
    back = [torch.empty(sum(kv), hkv, d, dtype=dtype, device="cuda") for _ in range(2)]
    rb.rpa_q8_read(*back, kc, vc, ks, vs, pt, cud, kvd, n, dev_flags=flags)
    want = torch.cat([pr.rows(s, pr.v_codes, pr.v_scales, kv[s]) for s in range(3)])
    assert torch.equal(back[1].cpu(), want.to(dtype))


def test_other_stream_and_other_device_are_refused_or_served():
    dv = Dev(problem("decode"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dv.attend()
    side.synchronize()
    dv.checked()
    with pytest.raises(ValueError):
        dv.rb.rpa_q8_attend(dv.q, dv.kc, dv.vc, dv.ks, dv.vs, dv.table.cpu(), dv.cu, dv.kv, dv.n, 1, 1.0, True,
                            dv.out, dv.ws)
    with pytest.raises(ValueError):
        dv.rb.rpa_q8_attend(dv.q.transpose(0, 1).contiguous().transpose(0, 1), *dv.cache, 1, 1.0, True,
                            dv.out, dv.ws)
    with pytest.raises(TypeError):
        dv.rb.rpa_q8_attend(dv.q.half(), *dv.cache, 1, 1.0, True, dv.out.half(), dv.ws)
    with pytest.raises(dv.rb.RpaError):
        dv.attend(workspace=dv.ws[:dv.ws.numel() - 256])


RANDOM = 60


@pytest.mark.parametrize("seed", range(RANDOM))
def test_random(seed):
    rng = np.random.RandomState(1000 + seed)
    d, p = int(rng.choice([64, 128, 256])), int(rng.choice([8, 16, 32, 64, 128, 256]))
    hkv, g = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 4, 6, 8, 16]))
    causal = bool(rng.rand() < 0.7)
    n = int(rng.randint(1, 7))
    top = int(rng.choice([1, 3, 40, 300]))
    q = [int(rng.randint(0, top + 1)) for _ in range(n)]
    kv = [int(math.exp(rng.uniform(0, math.log(2500)))) + (a if rng.rand() < 0.8 else 0) - 1 for a in q]
    if sum(q) == 0:
        q[0] = 1
    pr = R.make(q, kv, hq=hkv * g, hkv=hkv, d=d, p=p, causal=causal, seed=seed,
                dtype=BF16 if rng.rand() < 0.7 else F32)
    Dev(pr, more_seqs=int(rng.randint(0, 3)), more_rows=int(rng.randint(0, 9))).attend().checked(what=f"seed {seed}")
