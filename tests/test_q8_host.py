"""The 8-bit cache without a GPU: the C ABI's refusals (all before any device
work), the binding's checks, and pins of the tests' reference."""
import ctypes
import math

import pytest
import torch

import q8_reference as R
from ragged_paged_attention_03_b200 import build as B


@pytest.fixture(scope="module")
def rb():
    B.build()
    from ragged_paged_attention_03_b200 import binding
    return binding


GOOD = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, num_pages=1000, max_pages_per_seq=64,
            total_q_tokens=8, dtype=1)
FAKE = 1 << 20      # a well-aligned non-null pointer: no accepted call is made with it


def dims(rb, **kw):
    return rb.rpa_dims(**{**GOOD, **kw})


def io(rb, name, kw=(), k=FAKE, v=FAKE, cache=(FAKE,) * 4, pt=FAKE, cu=FAKE, kv=FAKE, n=FAKE, max_seqs=4, d="good"):
    c = rb.rpa_q8_cache(*cache) if cache is not None else None
    dd = dims(rb, **dict(kw)) if d == "good" else None
    return getattr(rb.library(), name)(k, v, ctypes.byref(c) if c else None, pt, cu, kv, n, max_seqs,
                                       ctypes.byref(dd) if dd else None, None, None)


def attend(rb, kw=(), q=FAKE, cache=(FAKE,) * 4, pt=FAKE, cu=FAKE, kv=FAKE, n=FAKE, max_seqs=4, max_q=1, scale=0.1,
           out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, d="good"):
    c = rb.rpa_q8_cache(*cache) if cache is not None else None
    dd = dims(rb, **dict(kw)) if d == "good" else None
    return rb.library().rpa_q8_attend(q, ctypes.byref(c) if c else None, pt, cu, kv, n, max_seqs, max_q, scale, 1,
                                      out, lse, ctypes.byref(dd) if dd else None, ws, ws_bytes, None, None)


BAD_DIMS = [(dict(head_dim=96), 2), (dict(page_size=12), 2), (dict(page_size=4), 2), (dict(page_size=512), 2),
            (dict(num_kv_heads=5), 2), (dict(num_q_heads=64, num_kv_heads=2), 2), (dict(dtype=7), 1),
            (dict(num_pages=0), 1), (dict(max_pages_per_seq=0), 1), (dict(total_q_tokens=-1), 1)]


@pytest.mark.parametrize("kw,code", BAD_DIMS)
def test_bad_dims(rb, kw, code):
    for name in ("rpa_q8_write", "rpa_q8_read"):
        assert io(rb, name, kw) == code
    assert attend(rb, kw) == code
    n = ctypes.c_int64(7)
    assert rb.library().rpa_q8_workspace_size(ctypes.byref(dims(rb, **kw)), 4, 1, ctypes.byref(n)) == code
    assert n.value == 0


@pytest.mark.parametrize("hole", ["k", "v", "cache", "pt", "cu", "kv", "n", "d"])
def test_write_read_null_pointers(rb, hole):
    for name in ("rpa_q8_write", "rpa_q8_read"):
        assert io(rb, name, **{hole: None}) == 1


@pytest.mark.parametrize("hole", ["q", "cache", "pt", "cu", "kv", "n", "out", "ws", "d"])
def test_attend_null_pointers(rb, hole):
    assert attend(rb, **{hole: None}) == 1


@pytest.mark.parametrize("i", range(4))
def test_null_cache_parts(rb, i):
    cache = [FAKE] * 4
    cache[i] = None
    assert io(rb, "rpa_q8_write", cache=cache) == 1
    assert io(rb, "rpa_q8_read", cache=cache) == 1
    assert attend(rb, cache=cache) == 1


def test_misaligned(rb):
    for name in ("rpa_q8_write", "rpa_q8_read"):
        assert io(rb, name, k=FAKE + 8) == 1
        assert io(rb, name, v=FAKE + 16) == 1
        assert io(rb, name, cache=(FAKE, FAKE + 4, FAKE, FAKE)) == 1
    assert attend(rb, q=FAKE + 2) == 1
    assert attend(rb, out=FAKE + 8) == 1
    assert attend(rb, out=FAKE + 16) == 1
    assert attend(rb, cache=(FAKE + 1, FAKE, FAKE, FAKE)) == 1
    assert attend(rb, ws=FAKE + 128) == 8


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, math.nan])
def test_attend_bad_scale(rb, scale):
    assert attend(rb, scale=scale) == 1


def test_negative_counts(rb):
    assert io(rb, "rpa_q8_write", max_seqs=-1) == 1
    assert attend(rb, max_seqs=-1) == 1
    assert attend(rb, max_q=-1) == 1
    n = ctypes.c_int64(0)
    lib = rb.library()
    assert lib.rpa_q8_workspace_size(ctypes.byref(dims(rb)), -1, 1, ctypes.byref(n)) == 1
    assert lib.rpa_q8_workspace_size(ctypes.byref(dims(rb)), 1, -1, ctypes.byref(n)) == 1
    assert lib.rpa_q8_workspace_size(ctypes.byref(dims(rb)), 1, 1, None) == 1


def test_no_work_is_no_op(rb):
    # nothing is looked at, not even the pointers
    for name in ("rpa_q8_write", "rpa_q8_read"):
        assert io(rb, name, max_seqs=0, k=None, cache=None) == 0
        assert io(rb, name, dict(total_q_tokens=0), v=None) == 0
    assert attend(rb, max_seqs=0, q=None, ws=None) == 0
    assert attend(rb, dict(total_q_tokens=0), out=None) == 0
    assert attend(rb, max_q=0, cache=None) == 0


@pytest.mark.parametrize("kw", [{}, dict(dtype=0), dict(head_dim=256), dict(num_q_heads=8), dict(num_q_heads=128)])
@pytest.mark.parametrize("max_seqs,max_q", [(1, 1), (128, 1), (4, 512), (300, 7)])
def test_workspace_is_checked(rb, kw, max_seqs, max_q):
    kw = {**kw, "total_q_tokens": max_seqs * max_q}
    need = rb.rpa_q8_workspace_size(dims(rb, **kw), max_seqs, max_q)
    assert need > 0 and need % 256 == 0
    assert attend(rb, kw, max_seqs=max_seqs, max_q=max_q, ws_bytes=need - 1) == 8


def tensors(device="cpu", t=3, hkv=2, d=64, p=8, pages=5, s=2):
    return dict(k_codes=torch.zeros(pages, p, hkv, d, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                v_codes=torch.zeros(pages, p, hkv, d, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                k_scales=torch.zeros(pages, hkv, p, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu),
                v_scales=torch.zeros(pages, hkv, p, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu),
                page_table=torch.zeros(s, 4, dtype=torch.int32, device=device),
                kv_lens=torch.zeros(s, dtype=torch.int32, device=device),
                num_seqs=torch.zeros(1, dtype=torch.int32, device=device))


@pytest.mark.parametrize("change,error", [
    (dict(k_codes=torch.zeros(5, 8, 2, 64, dtype=torch.uint8)), TypeError),
    (dict(v_codes=torch.zeros(5, 8, 2, 32).to(torch.float8_e4m3fn)), TypeError),
    (dict(k_scales=torch.zeros(5, 2, 8, dtype=torch.uint8)), TypeError),
    (dict(v_scales=torch.zeros(5, 8, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu)), TypeError),
    (dict(page_table=torch.zeros(1, 4, dtype=torch.int32)), ValueError),
    (dict(k_new=torch.zeros(3, 2, 128, dtype=torch.bfloat16)), ValueError),
    (dict(), ValueError),          # everything is right but on the CPU
])
def test_binding_refuses(rb, change, error):
    a = tensors()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    a.update(k_new=k, v_new=k.clone(), cu_q_lens=torch.zeros(3, dtype=torch.int32))
    a.update(change)
    with pytest.raises(error):
        rb.rpa_q8_write(**a)


# ------------------------------------------------------------- the reference
def test_reference_values_by_hand():
    # amax 448 -> scale 1; 2^e steps up just above it, down at 224
    rows = torch.zeros(7, 64)
    rows[0, 0] = 448.0
    rows[1, 0] = 448.001
    rows[2, 0] = 224.0
    rows[3, :4] = torch.tensor([400.0, 17.0, 2.0 ** -10, 3 * 2.0 ** -10])   # ties: to 384, 16, 0 and 2^-8
    rows[5, 3] = math.inf
    rows[6, 9] = math.nan
    codes, scale = R.quantise_row(rows)
    assert scale.tolist() == [127, 128, 126, 127, 127, 255, 255]
    val = R.E4M3[codes.long()] * R.scale_of(scale)[..., None]
    assert val[0, 0] == 448 and val[1, 0] == 448 and val[2, 0] == 224
    assert val[3, :4].tolist() == [384.0, 16.0, 0.0, 2.0 ** -8]
    assert (codes[4:] == 0).all()


@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-3, 1.0, 300.0, 1e20, 3e38])
def test_reference_error_bound(size):
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(1)).clamp(-4, 4) / 4 * size
    codes, scale = R.quantise_row(x)
    s = R.scale_of(scale)[..., None]
    err = (R.E4M3[codes.long()] * s - x.double()).abs()
    assert (err <= torch.maximum(x.double().abs() * 2.0 ** -4, s * 2.0 ** -10)).all()
    amax = x.double().abs().amax(-1, keepdim=True)
    assert (amax <= 448 * s).all() and ((amax > 224 * s) | (scale[..., None] == 0)).all()


def test_reference_matches_torch_rounding():
    y = torch.linspace(-448, 448, 40001)
    y = torch.cat([y, y * 2.0 ** -12])
    rows = torch.zeros(len(y), 64)
    rows[:, 0] = 448.0
    rows[:, 1] = y
    codes, scale = R.quantise_row(rows)
    assert (scale == 127).all()
    assert torch.equal(codes[:, 1], y.to(torch.float8_e4m3fn).view(torch.uint8))


def test_reference_attention_one_key_and_empty():
    pr = R.make([2, 1, 3], [1, 0, 2], hq=4, hkv=2, d=64, p=8, causal=True, seed=3)
    out, lse, _, _ = R.attend(pr)
    v = pr.rows(0, pr.v_codes, pr.v_scales, 1)
    k = pr.rows(0, pr.k_codes, pr.k_scales, 1)
    # kv_len 1 < q_len 2: the first row sees nothing, the second the one key
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.allclose(out[1], v[0].repeat_interleave(2, 0), rtol=0, atol=1e-12)
    assert torch.allclose(lse[1], (pr.q[1].double() * k[0].repeat_interleave(2, 0)).sum(-1) * pr.scale, atol=1e-12)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
