"""Cases of the operators on the 8-bit K/V cache: quantising new K/V rows into
their pages (``rpa_q8_write``), reading cached rows back (``rpa_q8_read``) and
attention over the quantised pages (``rpa_q8_attend``).

The cache holds e4m3 codes ``[num_pages, P, Hkv, D]`` and one power-of-two
scale per (token, KV head), e8m0 ``[num_pages, Hkv, P]``.  For a row x of D
values the scale is 2^e with the smallest e >= -127 such that
max|x| <= 448 * 2^e (e = 0 for a row of zeros), and the codes are x * 2^-e
rounded to nearest-even.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


def listed():
    return [
        # one decode step's new tokens of 128 sequences: the smallest write of a serving loop
        _io("write_decode_128", "write", BF16, 8, 128, 16, 128, 1, 1, 1024, 8192),
        # the prompt tokens of a prefill batch, written whole
        _io("write_prefill_8x2048", "write", BF16, 8, 128, 16, 8, 2048, 2048, 0, 0),
        # fp32 model, ragged chunks on small pages (pages end inside every chunk)
        _io("write_ragged_f32", "write", F32, 4, 64, 8, 37, 1, 700, 0, 3000),
        # contexts brought back for inspection or for a transfer to another cache
        _io("read_context", "read", BF16, 8, 128, 16, 4, 1536, 8704, 0, 0),
        # the last rows of ragged sequences, fp32, head_dim 256 on large pages
        _io("read_ragged_f32_d256", "read", F32, 4, 256, 64, 23, 1, 600, 0, 2000),
        # one user, one token, a short context: latency
        _at("attend_one", BF16, 4, 1, 64, 16, 1, 1, 1, 99, 99, True),
        # a decode step of 128 users
        _at("attend_decode_128", BF16, 32, 8, 128, 16, 128, 1, 1, 1023, 8191, True),
        # a few users with very long contexts, head_dim 256
        _at("attend_decode_long_d256", BF16, 16, 4, 256, 64, 8, 1, 1, 131071, 131071, True),
        # chunked prefill: 512 new tokens each after a cached context
        _at("attend_chunk_4x512", BF16, 32, 8, 128, 16, 4, 512, 512, 1024, 8192, True),
        # fresh prefill, every key new (already written)
        _at("attend_prefill_8x2048", BF16, 32, 8, 128, 16, 8, 2048, 2048, 0, 0, True),
        # cross attention: ragged decoder chunks over an encoder's states, some of them empty
        _at("attend_cross", BF16, 16, 16, 64, 32, 24, 1, 448, 0, 1500, False),
        # fp32 model: single tokens and short ragged chunks
        _at("attend_mixed_f32", F32, 8, 2, 128, 16, 24, 1, 60, 30, 2000, True),
    ]


def _io(name, op, dtype, hkv, d, page, seqs, q_lo, q_hi, ctx_lo, ctx_hi):
    return {"name": name, "op": op, "dtype": dtype, "hq": hkv, "hkv": hkv, "d": d, "page": page, "seqs": seqs,
            "q_lo": q_lo, "q_hi": q_hi, "kv_lo": ctx_lo, "kv_hi": ctx_hi, "self": True, "causal": True}


def _at(name, dtype, hq, hkv, d, page, seqs, q_lo, q_hi, kv_lo, kv_hi, causal):
    # causal: kv_lo / kv_hi bound the cached context before the new tokens;
    # otherwise the length of the states attended to, whatever q_len is
    return {"name": name, "op": "attend", "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "page": page, "seqs": seqs,
            "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "self": causal, "causal": causal}


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "attend"])
        dtype = rng.choice([BF16, BF16, BF16, F32])
        d = rng.choice([64, 128, 256])
        page = rng.choice([8, 16, 16, 32, 64, 128, 256])
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        seqs = _spread(rng, 1, 160)
        if op != "attend":
            q_hi = _spread(rng, 1, 8192)
            ctx = _spread(rng, 0, 4096)
            c = _io("", op, dtype, hkv, d, page, seqs, rng.choice([1, q_hi]), q_hi, rng.choice([0, ctx]), ctx)
        else:
            hq = hkv * rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
            kind = rng.choice(["decode", "decode", "chunk", "cross"])
            q_hi = _spread(rng, 1, 4) if kind == "decode" else _spread(rng, 2, 2048)
            kv_hi = _spread(rng, 16, 131072) if kind == "decode" else _spread(rng, 1, 16384)
            c = _at("", dtype, hq, hkv, d, page, seqs, rng.choice([1, q_hi]), q_hi,
                    rng.choice([0 if kind != "decode" else 1, kv_hi // 4, kv_hi]), kv_hi, kind != "cross")
            most = kv_hi + (q_hi if kind != "cross" else 0)
            if seqs * most * q_hi * hq > 1 << 30:       # the plain form's scores, padded
                continue
        w = work(c)
        if not 0 < w["bytes"] <= 2e9 or w["flops"] > 2.7e11:
            continue
        del c["name"]
        return c


def _lengths(case):
    """(q_lens, kv_lens): the case's alone, the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    q = [_spread(rng, case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    kv = [_spread(rng, case["kv_lo"], case["kv_hi"]) for _ in range(case["seqs"])]
    if case["self"]:
        kv = [a + b for a, b in zip(q, kv)]
    return q, kv


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def work(case):
    q, kv = _lengths(case)
    es = 2 if case["dtype"] == BF16 else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] != "attend":
        return {"bytes": sum(q) * hkv * 2 * (d * es + d + 1), "flops": 0}
    pairs = keys = 0
    for a, b in zip(q, kv):
        if a == 0:
            continue
        keys += b
        if case["causal"]:
            c = b - a
            pairs += a * c + a * (a + 1) // 2
        else:
            pairs += a * b
    return {"bytes": sum(q) * hq * (2 * d * es + 4) + keys * hkv * 2 * (d + 1), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """e4m3 codes and e8m0 scales of the rows of x (its last axis), in 32 bits."""
    x = x.float()
    amax = x.abs().amax(-1)
    mant, expo = torch.frexp(amax)                      # amax = mant * 2^expo, mant in [0.5, 1)
    e = (expo - 9 + (mant > 0.875)).clamp_min(-127)     # 448 = 0.875 * 2^9
    e = torch.where(amax == 0, 0, e)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    finite = torch.isfinite(amax)
    codes = torch.where(finite[..., None], codes.view(torch.uint8), 0).view(torch.float8_e4m3fn)
    scale = torch.where(finite, e + 127, 255).to(torch.uint8).view(torch.float8_e8m0fnu)
    return codes, scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    q_lens, kv_lens = _lengths(case)
    hq, hkv, d, p = case["hq"], case["hkv"], case["d"], case["page"]
    used = [(n + p - 1) // p for n in kv_lens]
    width = max(1, max(used))
    pages = sum(used) + max(1, sum(used) // 4)          # a quarter of the pool is free or another batch's
    perm = torch.randperm(pages, generator=cpu)
    table = torch.zeros(len(used), width, dtype=torch.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = perm[at:at + n]
        at += n
    cu = torch.zeros(len(q_lens) + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(q_lens).cumsum(0)
    total = int(cu[-1])
    seq_of = torch.repeat_interleave(torch.arange(len(q_lens)), torch.tensor(q_lens))
    i_of = torch.arange(total) - cu[seq_of]
    gain = torch.exp(0.5 * torch.randn(1, hkv, d, generator=gen, device=dev))   # channels differ in size

    def rows(n):
        return torch.randn(n, hkv, d, generator=gen, device=dev).mul_(gain)

    def pool():
        codes = torch.empty(pages, p, hkv, d, dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(pages, hkv, p, dtype=torch.float8_e8m0fnu, device=dev)
        step = max(1, (1 << 27) // (p * hkv * d))
        for a in range(0, pages, step):
            n = min(step, pages - a)
            c, e = _quantise(rows(n * p).view(n, p, hkv, d))
            codes[a:a + n] = c
            scale[a:a + n] = e.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e8m0fnu)
        return codes, scale

    st = dict(case=case, table=table.to(dev), cu=cu.to(torch.int32).to(dev),
              kv=torch.tensor(kv_lens, dtype=torch.int32, device=dev),
              n=torch.tensor([len(q_lens)], dtype=torch.int32, device=dev),
              seq_of=seq_of.to(dev), i_of=i_of.to(dev), q_max=max(q_lens))
    tdt = _dtype(case)
    if case["op"] == "write":
        st["k"], st["v"] = rows(total).to(tdt), rows(total).to(tdt)
        st["kc"] = torch.zeros(pages, p, hkv, d, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        st["ke"] = torch.full((pages, hkv, p), 127, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
        st["vc"], st["ve"] = st["kc"].clone(), st["ke"].clone()
        return st
    st["kc"], st["ke"] = pool()
    st["vc"], st["ve"] = pool()
    if case["op"] == "read":
        st["k"] = torch.empty(total, hkv, d, dtype=tdt, device=dev)
        st["v"] = torch.empty_like(st["k"])
        return st
    # query rows of unit variance against keys whose channels have gains: scores of a few units
    st["q"] = torch.randn(total, hq, d, generator=gen, device=dev).to(tdt)
    st["scale"] = 1.0 / math.sqrt(d)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(total, hq, dtype=torch.float32, device=dev)
    return st


# -------------------------------------------------------------------- runs
def run(st):
    op = st["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "attend": _own_attend}[op](st)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](st)


def _own_write(st):
    from ragged_paged_attention_03_b200 import binding
    binding.rpa_q8_write(st["k"], st["v"], st["kc"], st["vc"], st["ke"], st["ve"], st["table"], st["cu"], st["kv"],
                         st["n"])
    return st["kc"], st["vc"], st["ke"], st["ve"]


def _own_read(st):
    from ragged_paged_attention_03_b200 import binding
    binding.rpa_q8_read(st["k"], st["v"], st["kc"], st["vc"], st["ke"], st["ve"], st["table"], st["cu"], st["kv"],
                        st["n"])
    return st["k"], st["v"]


def _own_attend(st):
    from ragged_paged_attention_03_b200 import binding
    if "ws" not in st:      # kept by the program from its first call on
        dims = binding.make_dims(st["q"], st["kc"], st["table"])
        size = binding.rpa_q8_workspace_size(dims, st["table"].shape[0], st["q_max"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=st["q"].device)
    binding.rpa_q8_attend(st["q"], st["kc"], st["vc"], st["ke"], st["ve"], st["table"], st["cu"], st["kv"], st["n"],
                          st["q_max"], st["scale"], st["case"]["causal"], st["out"], st["ws"], lse=st["lse"])
    return st["out"], st["lse"]


def _slots(st):
    """Page and slot of every new token."""
    p = st["case"]["page"]
    q_len = st["cu"][1:] - st["cu"][:-1]
    pos = (st["kv"] - q_len)[st["seq_of"]] + st["i_of"]
    return st["table"][st["seq_of"], pos // p].long(), pos % p


def _plain_write(st):
    page, slot = _slots(st)
    for x, codes, scale in ((st["k"], st["kc"], st["ke"]), (st["v"], st["vc"], st["ve"])):
        c, e = _quantise(x)
        codes.view(torch.uint8)[page, slot] = c.view(torch.uint8)
        scale.view(torch.uint8)[page, :, slot] = e.view(torch.uint8)
    return st["kc"], st["vc"], st["ke"], st["ve"]


def _plain_read(st):
    page, slot = _slots(st)
    for x, codes, scale in ((st["k"], st["kc"], st["ke"]), (st["v"], st["vc"], st["ve"])):
        c = codes.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
        e = scale.view(torch.uint8)[page, :, slot].view(torch.float8_e8m0fnu).float()
        x.copy_(c * e[..., None])
    return st["k"], st["v"]


def _pages_of(st, codes, scale):
    """[S, width * P, Hkv, D] in fp32: every page of every sequence's row of the table."""
    table = st["table"].long()
    c = codes.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    e = scale.view(torch.uint8)[table].view(torch.float8_e8m0fnu).float().transpose(2, 3)
    return c.mul_(e[..., None]).flatten(1, 2)


def _plain_attend(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    n_seq = st["table"].shape[0]
    q = torch.zeros(n_seq, st["q_max"], hkv, g, d, dtype=torch.float32, device=st["q"].device)
    q[st["seq_of"], st["i_of"]] = st["q"].float().view(-1, hkv, g, d)
    k = _pages_of(st, st["kc"], st["ke"])
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3), k.permute(0, 2, 3, 1)) * st["scale"]
    del k
    x = x.unflatten(2, (g, st["q_max"]))                            # [S, Hkv, G, q, k]
    pos = torch.arange(x.shape[-1], device=x.device)
    seen = (pos < st["kv"][:, None])[:, None, :]                    # [S, 1, k]
    if case["causal"]:
        q_len = st["cu"][1:] - st["cu"][:-1]
        last = (st["kv"] - q_len)[:, None] + torch.arange(st["q_max"], device=x.device)
        seen = seen & (pos <= last[..., None])                      # [S, q, k]
    seen = seen[:, None, None]
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    v = _pages_of(st, st["vc"], st["ve"])
    v.masked_fill_((pos >= st["kv"][:, None])[..., None, None], 0.0)
    o = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (g, st["q_max"]))
    o.div_(torch.where(total == 0, 1.0, total))
    lse = (m + torch.log(total))[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4), lse.permute(0, 3, 1, 2)      # [S, q, Hkv, G, ...]
    st["out"].copy_(o[st["seq_of"], st["i_of"]].reshape(-1, hq, d))
    st["lse"].copy_(lse[st["seq_of"], st["i_of"]].reshape(-1, hq))
    return st["out"], st["lse"]


# ------------------------------------------------------- the definition in 64 bits
def _nearest_e4m3(y):
    """y rounded to the nearest e4m3 value, ties to even, as float64."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    q_lens, kv_lens = _lengths(case)
    p, d, hkv = case["page"], case["d"], case["hkv"]
    if case["op"] == "write":
        sides = []
        for x in (st["k"], st["v"]):
            x = x.double()
            amax = x.abs().amax(-1)
            e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0))
            e = e + (amax > 448.0 * torch.exp2(e)).double()     # where log2's own rounding fell short,
            e = e - (amax <= 224.0 * torch.exp2(e)).double()    # or went too far
            e = torch.where(amax == 0, 0.0, e.clamp_min(-127.0))
            codes = torch.zeros(st["kc"].shape, dtype=torch.float64, device=x.device)
            scale = torch.ones(st["ke"].shape, dtype=torch.float64, device=x.device)
            at = 0
            for s, (a, b) in enumerate(zip(q_lens, kv_lens)):
                pos = torch.arange(b - a, b, device=x.device)
                page = st["table"][s].long()[pos // p]
                codes[page, pos % p] = _nearest_e4m3(x[at:at + a] / torch.exp2(e[at:at + a])[..., None])
                scale[page, :, pos % p] = torch.exp2(e[at:at + a])
                at += a
            sides.append((codes, scale))
        return sides[0][0], sides[1][0], sides[0][1], sides[1][1]

    def row(s, n, codes, scale):
        """Cached rows [0, n) of sequence s: [n, Hkv, D]."""
        used = st["table"][s, :(n + p - 1) // p].long()
        c = codes.view(torch.uint8)[used].view(torch.float8_e4m3fn).double()
        e = scale.view(torch.uint8)[used].view(torch.float8_e8m0fnu).double()
        return (c * e.transpose(1, 2).unsqueeze(-1)).reshape(-1, hkv, d)[:n]

    if case["op"] == "read":
        return tuple(torch.cat([row(s, b, c, e)[b - a:] for s, (a, b) in enumerate(zip(q_lens, kv_lens))])
                     for c, e in ((st["kc"], st["ke"]), (st["vc"], st["ve"])))
    hq = case["hq"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((out.shape[0], hq), -math.inf, dtype=torch.float64, device=out.device)
    at = 0
    for s, (a, b) in enumerate(zip(q_lens, kv_lens)):
        if a and b:
            k, v = row(s, b, st["kc"], st["ke"]), row(s, b, st["vc"], st["ve"])
            q = st["q"][at:at + a].double()
            for h in range(hq):
                x = (q[:, h] @ k[:, h * hkv // hq].T) * st["scale"]
                if case["causal"]:
                    i = torch.arange(a, device=x.device)[:, None] + (b - a)
                    x.masked_fill_(torch.arange(b, device=x.device) > i, -math.inf)
                lse[at:at + a, h] = torch.logsumexp(x, -1)
                out[at:at + a, h] = torch.softmax(x, -1) @ v[:, h * hkv // hq]
        at += a
    return out, lse
