"""The 8-bit cache at sizes where indexing can go wrong: more sequences than a
block has threads, offsets past 32 bits in the pool and in the token arrays,
calls at once on two streams."""
import numpy as np
import pytest
import torch

import q8_reference as R
from test_q8_gpu import BF16, F32, Dev, e8, f8, lib, new_rows  # noqa: F401 (lib: builds the library)

pytestmark = pytest.mark.gpu


def many(n, dtype, seed, d=64, hq=4, hkv=2, p=8):
    rng = np.random.RandomState(seed)
    q = rng.choice([0, 1, 1, 1, 2, 5, 40], size=n).tolist()
    kv = [int(a + rng.randint(0, 60)) for a in q]
    return R.make(q, kv, hq=hq, hkv=hkv, d=d, p=p, dtype=dtype, seed=seed)


# 224, 256, 512 threads validate and scan the lengths; 512 fit in shared memory
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,more", [(225, 3), (257, 3), (513, 3), (1100, 3), (30, 900), (512, 0), (509, 3), (510, 3)])
def test_many_sequences(n, more, dtype):
    pr = many(n, dtype, n)
    dv = Dev(pr, more_seqs=more, more_rows=2)
    dv.attend().checked(what=f"{n} sequences")
    t = sum(pr.q_lens)
    rows = [new_rows(pr, 7 + i, dtype, odd=False) for i in range(2)]
    pad = torch.full((2, pr.hkv, pr.d), 5.0, dtype=dtype)
    dv.rb.rpa_q8_write(*[torch.cat([r, pad]).cuda() for r in rows], *dv.cache, dev_flags=dv.flags)
    back = [torch.full((t + 2, pr.hkv, pr.d), 77.0, dtype=dtype, device="cuda") for _ in range(2)]
    dv.rb.rpa_q8_read(*back, *dv.cache, dev_flags=dv.flags)
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == 0
    for got, r in zip(back, rows):
        c, e = R.quantise_row(r)
        want = c.view(torch.float8_e4m3fn).double() * R.scale_of(e)[..., None]
        assert torch.equal(got[:t].cpu(), want.to(dtype))
        assert (got[t:] == 77).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 4], [50, 700, 70]), ([200, 1, 33], [450, 64, 40])])
def test_pool_past_32_bits(q_lens, kv_lens):
    """The pages of a small pool, moved to the end of one of 4.6e9 codes: the same bits."""
    pr = R.make(q_lens, kv_lens, hq=16, hkv=8, d=128, p=32, dtype=BF16, seed=3)
    dv = Dev(pr).attend()
    dv.checked()
    small = pr.k_codes.shape[0]
    pages = 140_000
    big = [torch.empty((pages, 32, 8, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.full((pages, 8, 32), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2)]
    where = pages - 1 - torch.arange(small, device="cuda")
    for dst, src in zip(big + sc, (dv.kc, dv.vc, dv.ks, dv.vs)):
        dst[where] = src.view(torch.uint8)
    cache = (f8(big[0]), f8(big[1]), e8(sc[0]), e8(sc[1]), (pages - 1 - dv.table).contiguous(), dv.cu, dv.kv, dv.n)
    out, lse = torch.full_like(dv.out, 77.0), torch.full_like(dv.lse, 77.0)
    dv.rb.rpa_q8_attend(dv.q, *cache, max_q_len=dv.max_q, scale=pr.scale, causal=True, out=out, workspace=dv.ws, lse=lse,
                        dev_flags=dv.flags)
    assert torch.equal(out, dv.out) and torch.equal(lse, dv.lse)
    rows = [new_rows(pr, 5 + i, BF16).cuda() for i in range(2)]
    back = [torch.empty_like(r) for r in rows * 2]
    for i, c in enumerate((dv.cache, cache)):
        dv.rb.rpa_q8_write(*rows, *c, dev_flags=dv.flags)
        dv.rb.rpa_q8_read(*back[2 * i:2 * i + 2], *c, dev_flags=dv.flags)
    torch.cuda.synchronize()
    assert int(dv.flags.item()) == 0
    for a, b in zip(back[:2], back[2:]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for dst, src in zip(cache[:4], dv.cache[:4]):
        assert torch.equal(dst.view(torch.uint8)[where], src.view(torch.uint8))


def test_rows_past_32_bits_written_and_read():
    """2.25e9 values each of K and V: a block of rows again and again."""
    from ragged_paged_attention_03_b200 import binding as rb
    hkv, d, p, block, times = 8, 256, 256, 4096, 268
    t = block * times
    x = torch.randn((block, hkv, d), generator=torch.Generator().manual_seed(0)).to(BF16)
    rows = x.cuda().repeat(times, 1, 1)
    pages = t // p
    codes = [torch.empty((pages, p, hkv, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.empty((pages, hkv, p), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    cache = (*codes, *scales, table, i32([0, t]), i32([t]), i32([1]))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    rb.rpa_q8_write(rows, rows, *cache, dev_flags=flags)
    back = [torch.full_like(rows, 77.0) for _ in range(2)]
    rb.rpa_q8_read(*back, *cache, dev_flags=flags)
    torch.cuda.synchronize()
    assert int(flags.item()) == 0
    c, e = R.quantise_row(x)
    want = (c.view(torch.float8_e4m3fn).double() * R.scale_of(e)[..., None]).to(BF16).cuda()
    for b in back:
        assert (b.view(times, block, hkv, d) == want).all()


@pytest.mark.parametrize("q_len,kv_len", [(2000, 40), (2, 300)])
def test_queries_past_32_bits(q_len, kv_len):
    """2.2e9 query values: one sequence again and again, attended alike."""
    from ragged_paged_attention_03_b200 import binding as rb
    pr = R.make([q_len], [kv_len], hq=32, hkv=8, d=128, p=16, dtype=BF16, causal=False, seed=1)
    want = R.attend(pr)
    times = 540_000 // q_len
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")
    table = pr.table[:1].cuda().repeat(times, 1)
    q = pr.q.cuda().repeat(times, 1, 1)
    cu = i32(np.arange(times + 1) * q_len)
    cache = (f8(pr.k_codes), f8(pr.v_codes), e8(pr.k_scales), e8(pr.v_scales), table, cu, i32([kv_len] * times), i32([times]))
    out, lse = torch.full_like(q, 77.0), torch.full((q.shape[0], 32), 77.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((rb.rpa_q8_workspace_size(rb.make_dims(q, cache[0], table), times, q_len),), 0x5A, dtype=torch.uint8,
                    device="cuda")
    rb.rpa_q8_attend(q, *cache, max_q_len=q_len, scale=pr.scale, causal=False, out=out, workspace=ws, lse=lse,
                     dev_flags=flags)
    torch.cuda.synchronize()
    assert int(flags.item()) == 0
    for s in (0, 1, times // 2, times - 2, times - 1):
        at = slice(s * q_len, (s + 1) * q_len)
        R.check(out[at], lse[at], want, f"sequence {s}")
    # every other row is within twice the tolerance of the first one's
    tol = torch.stack([w.reshape(q_len, -1).amax(1) for w in want[2:3]]).cuda()[0]
    gap = (out.view(times, q_len, -1).float() - out[:q_len].reshape(1, q_len, -1).float()).abs().amax(-1)
    assert (gap <= 2 * tol).all()


@pytest.mark.parametrize("kinds", [("decode", "chunk"), ("chunk", "chunk")])
def test_two_streams_at_once(kinds):
    """Each call with its own workspace: the same bits as one after the other."""
    shapes = {"decode": ([1] * 40, [900 + 31 * i for i in range(40)]), "chunk": ([130, 1, 260, 17], [1200, 300, 260, 900])}
    dvs = [Dev(R.make(*shapes[k], hq=16, hkv=4, d=128, p=16, dtype=BF16, seed=i)) for i, k in enumerate(kinds)]
    alone = []
    for dv in dvs:
        dv.attend()
        torch.cuda.synchronize()
        alone.append((dv.out.clone(), dv.lse.clone()))
    streams = [torch.cuda.Stream() for _ in dvs]
    for _ in range(20):
        for dv in dvs:
            dv.out.fill_(77.0)
        torch.cuda.synchronize()
        for dv, s in zip(dvs, streams):
            with torch.cuda.stream(s):
                dv.attend()
        torch.cuda.synchronize()
        for dv, (out, lse) in zip(dvs, alone):
            assert torch.equal(dv.out, out) and torch.equal(dv.lse, lse) and int(dv.flags.item()) == 0
