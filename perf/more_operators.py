"""Cases that time the paged token cache's 4-bit pages and its prompts: storing tokens in 4 bits
and reading them back, attention of one new token per sequence over 4-bit pages, and attention
of several new tokens per sequence (prompts, drafts to verify, frames of a stream) over pages of
every type.

`listed()` names the cases, `prepare()` makes one's inputs on the GPU, `run()` is one pass
(the plain torch form, or the library's calls when `own` is set), `work()` counts what a
pass has to move and compute, `exact()` computes a pass in 64 bits.

A sequence's token i (its logical index) lies on page `table[seq, i // page]` at slot `i % page`.
Pages of 16 or 8 bits are [n_pages][page][kv][d]. A 4-bit page is [kv][page / 16] records, each
of 16 tokens of one head: 16 * d / 2 bytes of codes, then [16][d / 16] bytes of scales.
* A value is (c - 8) * s * 2^exp[head], c its code, 0 .. 15, s the scale of its 16 neighbours.
* A scale's byte b is the fp16 number with the bits b << 7: five bits of exponent, three of fraction.
* Codes lie [d / 32][16 tokens][16 bytes]; two bytes hold four values: the 16-bit number
  c0 | c1 << 4 | c2 << 8 | c3 << 12, turned left by one bit.
"""
import math

import torch

own = False

SCALE_MAX = 3840.0                       # the largest scale, byte 215
NOT_A_NUMBER = 255                       # the scale of 16 values with a NaN among them


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a few tokens of several sessions pass through the cache, so that what is computed on them now
        # has the rounding that later tokens will see: nothing but latency
        dict(name="store 16 tokens of 8 sequences", op="store", n_seqs=8, lo=16, hi=16, heads=4, kv_heads=4, d=64,
             page=16, dtype="int4"),
        # long prompts of several sequences do the same
        dict(name="store 8 prompts", op="store", n_seqs=8, lo=511, hi=16384, heads=40, kv_heads=8, d=128, page=64,
             dtype="int4"),
        # one short history goes back to 16 bits
        dict(name="read one short history", op="read", n_seqs=1, lo=300, hi=300, heads=4, kv_heads=4, d=64, page=16,
             dtype="int4"),
        # eight sessions' histories do, for a dense attention over them; every head has its own keys
        dict(name="read 8 histories", op="read", n_seqs=8, lo=2072, hi=11432, heads=40, kv_heads=40, d=128, page=64,
             dtype="int4"),
        # a token of one short conversation on a tiny model
        dict(name="attend one short sequence, 4 bits", op="attend", n_seqs=1, lo=300, hi=300, heads=4, kv_heads=4,
             d=64, page=16, dtype="int4", mass=False),
        # a large serving batch, long histories
        dict(name="attend 32 sequences, 4 bits", op="attend", n_seqs=32, lo=4001, hi=32768, heads=40, kv_heads=8,
             d=128, page=64, dtype="int4", mass=False),
        # one very long sequence: the only parallelism is along its length
        dict(name="attend one long sequence, 4 bits", op="attend", n_seqs=1, lo=131071, hi=131071, heads=40,
             kv_heads=8, d=128, page=64, dtype="int4", mass=False),
        # every length from one token up in small pages, with the weights that eviction goes by
        dict(name="attend 64 ragged sequences, 4 bits", op="attend", n_seqs=64, lo=1, hi=16384, heads=32, kv_heads=8,
             d=64, page=16, dtype="int4", mass=True),
        # four drafted tokens of each of 16 sequences are verified at once
        dict(name="verify 4 tokens of 16 sequences, 4 bits", op="prompt", n_seqs=16, new_lo=4, new_hi=4, lo=1000,
             hi=8192, heads=32, kv_heads=8, d=128, page=64, dtype="int4", causal=True),
        # the next stretch of long prompts, odd lengths, over what is already in the cache
        dict(name="prompts of 131 .. 1021 over 16384, 4 bits", op="prompt", n_seqs=4, new_lo=131, new_hi=1021,
             lo=2003, hi=16384, heads=40, kv_heads=8, d=128, page=64, dtype="int4", causal=True),
        # a whole long prompt, nothing before it
        dict(name="one prompt of 8192", op="prompt", n_seqs=1, new_lo=8192, new_hi=8192, lo=8192, hi=8192, heads=32,
             kv_heads=8, d=128, page=64, dtype="bf16", causal=True),
        # one 832x480 frame of two streams sees itself and six before it, every head with its own keys
        dict(name="a frame of 2 streams, e4m3", op="prompt", n_seqs=2, new_lo=1560, new_hi=1560, lo=10920, hi=10920,
             heads=40, kv_heads=40, d=128, page=64, dtype="e4m3", causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend", "prompt", "prompt", "prompt"])
    kv, group = rng.choice([1, 2, 4, 5, 8, 8, 16]), rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(op=op, heads=kv * group, kv_heads=kv, d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 48, 64, 128]),
             dtype="int4" if op != "prompt" else rng.choice(["int4", "int4", "bf16", "e4m3"]))
    row = kv * c["d"]                       # values of one token's keys
    if op == "prompt":
        c["n_seqs"] = n = _log(rng, 1, 16)
        work_cap = 150_000_000_000 // (n * kv * group * c["d"])            # pairs of tokens of a sequence
        c["new_hi"] = _log(rng, 1, min(8192 // n, math.isqrt(work_cap)))
        c["new_lo"] = _log(rng, 1, c["new_hi"])
        most = min(32768, work_cap // c["new_hi"], 64_000_000 // (n * row))
        c["hi"] = _log(rng, c["new_hi"], max(most, c["new_hi"]))
        c["lo"] = max(c["new_hi"], _log(rng, 1, c["hi"]))
        c["causal"] = rng.random() < 0.7
        return c
    c["n_seqs"] = _log(rng, 1, 64)
    values = dict(store=40_000_000, read=200_000_000, attend=220_000_000)[op]
    most = min(65536, values // (c["n_seqs"] * row), 40_000_000 // (c["n_seqs"] * kv * group))
    c["hi"] = _log(rng, 1, max(most, 64))
    c["lo"] = _log(rng, 1, c["hi"])
    if op == "attend":
        c["mass"] = rng.random() < 0.4
    return c


def _lengths(n, lo, hi):
    """n lengths spread over [lo, hi] on a logarithmic scale, the longest first."""
    u = [math.modf(i * 0.6180339887498949)[0] for i in range(n)]
    return [hi] + [min(hi, max(lo, int(round(lo * (hi / lo) ** x)))) for x in u[1:]]


def _counts(case):
    """New tokens of each sequence."""
    if case["op"] != "prompt":
        return _lengths(case["n_seqs"], case["lo"], case["hi"])
    # the longest prompts go to the shortest histories
    return _lengths(case["n_seqs"], case["new_lo"], case["new_hi"])[::-1]


# ------------------------------------------------------------------ inputs
def _record_views(pool, case):
    """Codes [n_pages][kv][page / 16][d / 32][16][16] and scales [n_pages][kv][page / 16][16][d / 16] of 4-bit pages."""
    kv, d, page = case["kv_heads"], case["d"], case["page"]
    rec = pool.view(-1, kv, page // 16, 9 * d)
    return rec[..., : 8 * d].unflatten(-1, (d // 32, 16, 16)), rec[..., 8 * d:].unflatten(-1, (16, d // 16))


def _pack(c):
    """Codes [..., 4 * n] as 2 * n bytes."""
    x = c.to(torch.int32).unflatten(-1, (-1, 4))
    x = x[..., 0] | x[..., 1] << 4 | x[..., 2] << 8 | x[..., 3] << 12
    x = (x << 1 | x >> 15) & 0xFFFF
    return torch.stack((x & 0xFF, x >> 8), -1).flatten(-2).to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)
    c, n = dict(case), case["n_seqs"]
    op, heads, kv, d, page, dtype = c["op"], c["heads"], c["kv_heads"], c["d"], c["page"], c["dtype"]
    lens = _lengths(n, c["lo"], c["hi"])
    pages_of = [-(-x // page) for x in lens]
    width = max(pages_of)
    n_pages = sum(pages_of) + 3
    # pages of the pool in no order, as they come out of a free list
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32)
    spread = torch.arange(width)[None, :] < torch.tensor(pages_of)[:, None]
    table[spread] = ids[: sum(pages_of)].cpu()
    table = table.to(dev)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def bits(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.uint8)

    exps = torch.randint(-3, 3, (2, kv), generator=g, device=dev, dtype=torch.int32)
    pool = []
    for i in range(2):
        if dtype == "int4":
            # normal values at scales of about 2^-3 .. 2^-1, times 2^exp; two keys' channels in a block of 16 are larger
            x = torch.empty((n_pages, page * kv * 9 * d // 16), dtype=torch.uint8, device=dev)
            codes, scales = _record_views(x, c)
            for p0 in range(0, n_pages, 256):
                part = codes[p0: p0 + 256]
                normal = randn(*part.shape[:-1], 32)
                if i == 0:
                    normal[..., ::16] *= 3.0
                part.copy_(_pack((normal * 2.2).round().clamp(-8, 7) + 8))
                scales[p0: p0 + 256] = bits(12 * 8, 14 * 8, scales[p0: p0 + 256].shape)
        else:
            x = torch.empty((n_pages, page, kv, d), dtype=torch.bfloat16, device=dev)
            x.normal_(generator=g)
            if dtype == "e4m3":
                x = (x * 16).to(torch.float8_e4m3fn)
        pool.append(x)
    if dtype == "e4m3":                      # values of about unit size come out
        exps -= 4
    cap = width * page
    s = dict(case=c, n=n, lens=lens, cap=cap, k_pages=pool[0], v_pages=pool[1], exps=exps, table=table,
             seq_len=torch.tensor(lens, dtype=torch.int32, device=dev), scale=1.0 / math.sqrt(d))
    s["seq_pos"] = s["seq_len"].clone()
    s["token_pos"] = torch.arange(cap, dtype=torch.int32, device=dev).repeat(n, 1)
    # weights gathered so far: a few tokens hold most of them
    s["mass"] = torch.exp(2.0 * randn(n, cap))
    s["counts"] = _counts(c)
    s["counts_dev"] = torch.tensor(s["counts"], device=dev)
    rows = sum(s["counts"])
    if op == "store":
        # keys have a few large channels, values do not
        loud = torch.exp(randn(kv, d))
        s["k"] = (randn(rows, kv, d) * loud).to(torch.bfloat16)
        s["v"] = randn(rows, kv, d).to(torch.bfloat16)
    if op in ("attend", "prompt"):
        s["q"] = (1.5 * randn(n if op == "attend" else rows, heads, d)).to(torch.bfloat16)
    if own:
        import chunked_kv_cache_gb300 as sr
        s["cache"] = sr.PagedCache(
            heads, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=n, max_pages=width,
            page_dtype="int4" if dtype == "int4" else pool[0].dtype, device=dev,
            buffers=dict(k_pages=s["k_pages"], v_pages=s["v_pages"], block_table=table, seq_len=s["seq_len"],
                         seq_pos=s["seq_pos"], token_pos=s["token_pos"], token_mass=s["mass"], kv_exp=exps))
    return s


# ------------------------------------------------------------------ the plain form
def _two_to(e):
    """2^e in 64 bits, exactly."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _places(s, seq, idx):
    """Pages and slots of tokens idx of sequences seq (both of one shape)."""
    page = s["case"]["page"]
    return s["table"][seq, idx // page].long().clamp(min=0), idx % page


def _gather(s, name, exp, pg, slot):
    """Tokens' rows [..., kv, d] in 32 bits."""
    pages = s[name]
    if pages.dtype == torch.bfloat16:
        return pages[pg, slot].float()
    if pages.dtype == torch.float8_e4m3fn:
        x = pages.view(torch.uint8)[pg, slot].view(torch.float8_e4m3fn).float()
        return x * _two_to(exp).float()[:, None]
    codes, scales = _record_views(pages, s["case"])
    x = codes[pg, :, slot // 16, :, slot % 16].flatten(-2)                 # [..., kv, d / 2]
    x = x[..., 0::2].int() | x[..., 1::2].int() << 8                       # four values each
    x = x >> 1 | (x & 1) << 15
    x = torch.stack((x & 15, x >> 4 & 15, x >> 8 & 15, x >> 12), -1).flatten(-2)
    b = scales[pg, :, slot // 16, slot % 16]                               # [..., kv, d / 16]
    scale = (b.to(torch.int16) << 7).view(torch.float16).float() * _two_to(exp).float()[:, None]
    return ((x - 8).float().unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2)


def _quantise(x, exp):
    """Rows [n][kv][d] as codes and scales' bytes."""
    y = (x.double() * _two_to(-exp)[None, :, None]).unflatten(-1, (-1, 16))
    nan = y.isnan().any(-1)
    y = torch.where(nan[..., None], 0.0, y)
    want = (y.abs().amax(-1) / 7.0).clamp(max=SCALE_MAX)
    # to four significant bits, or to multiples of 2^-17: halves up
    step = _two_to((want.clamp(min=2.0 ** -14).view(torch.int64) >> 52) - 1023 - 3)
    scale = torch.floor(want / step + 0.5) * step
    b = (scale.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)
    t = (y / scale.clamp(min=2.0 ** -60)[..., None]).nan_to_num(nan=0.0)
    t = torch.where(scale[..., None] > 0, t, 0.0)
    code = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-8, 7) + 8   # halves away from zero
    return code.flatten(-2), torch.where(nan, NOT_A_NUMBER, b)


def _plain_store(s):
    n, dev, c = s["n"], s["k"].device, s["case"]
    s["seq_len"].zero_()
    s["seq_pos"].zero_()
    rows = s["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device=dev), s["counts_dev"], output_size=rows)
    first = torch.cumsum(s["counts_dev"], 0) - s["counts_dev"]
    i = torch.arange(rows, device=dev) - first[seq]
    idx = s["seq_len"][seq].long() + i
    pg, slot = _places(s, seq, idx)
    for j, name in enumerate("kv"):
        code, b = _quantise(s[name], s["exps"][j])
        codes, scales = _record_views(s[name + "_pages"], c)
        codes[pg, :, slot // 16, :, slot % 16] = _pack(code).unflatten(-1, (-1, 16))
        scales[pg, :, slot // 16, slot % 16] = b
    s["token_pos"][seq, idx] = (s["seq_pos"][seq].long() + i).to(torch.int32)
    s["mass"][seq, idx] = 0.0
    s["seq_len"] += s["counts_dev"].to(torch.int32)
    s["seq_pos"] += s["counts_dev"].to(torch.int32)


def _plain_read(s):
    """Every sequence's last tokens, back to back."""
    n, dev = s["n"], s["table"].device
    rows = sum(s["counts"])
    seq = torch.repeat_interleave(torch.arange(n, device=dev), s["counts_dev"], output_size=rows)
    first = torch.cumsum(s["counts_dev"], 0) - s["counts_dev"]
    idx = (s["seq_len"] - s["counts_dev"])[seq].long() + torch.arange(rows, device=dev) - first[seq]
    pg, slot = _places(s, seq, idx)
    return dict(k=_gather(s, "k_pages", s["exps"][0], pg, slot).to(torch.bfloat16),
                v=_gather(s, "v_pages", s["exps"][1], pg, slot).to(torch.bfloat16))


def _plain_attend(s):
    c, n, dev = s["case"], s["n"], s["q"].device
    kv, d = c["kv_heads"], c["d"]
    idx = torch.arange(s["cap"], device=dev)
    live = idx[None, :] < s["seq_len"][:, None]
    pg, slot = _places(s, torch.arange(n, device=dev)[:, None], idx[None, :].expand(n, -1))
    k = _gather(s, "k_pages", s["exps"][0], pg, slot)                      # [n][L][kv][d]
    q = s["q"].float().view(n, kv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                # [n][kv][group][L]
    del k
    x = torch.where(live[:, None, None, :], x, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp(min=1e-30)
    v = _gather(s, "v_pages", s["exps"][1], pg, slot)
    v = torch.where(live[:, :, None, None], v, 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(n, -1, d).to(torch.bfloat16)
    out = dict(o=o, lse=(top + torch.log(total)).reshape(n, -1))
    if c["mass"]:
        s["mass"] += p.sum((1, 2))
        out["mass"] = s["mass"]
    return out


def _plain_prompt(s):
    c, dev = s["case"], s["q"].device
    kv, d, heads = c["kv_heads"], c["d"], c["heads"]
    o = torch.empty_like(s["q"])
    lse = torch.empty((o.shape[0], heads), dtype=torch.float32, device=dev)
    r = 0
    for i, (length, count) in enumerate(zip(s["lens"], s["counts"])):
        idx = torch.arange(length, device=dev)
        pg, slot = _places(s, torch.full_like(idx, i), idx)
        k = _gather(s, "k_pages", s["exps"][0], pg, slot).permute(1, 2, 0)           # [kv][d][L]
        v = _gather(s, "v_pages", s["exps"][1], pg, slot).transpose(0, 1)            # [kv][L][d]
        step = max(1, 500_000_000 // (heads * length))
        for a in range(0, count, step):
            b = min(count, a + step)
            q = s["q"][r + a: r + b].float().view(b - a, kv, -1, d).permute(1, 2, 0, 3)   # [kv][group][rows][d]
            x = torch.matmul(q.flatten(1, 2), k).unflatten(1, (-1, b - a)) * s["scale"]
            if c["causal"]:
                at = length - count + torch.arange(a, b, device=dev)
                x = torch.where(idx[None, :] <= at[:, None], x, float("-inf"))
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - top)
            total = e.sum(-1, keepdim=True)
            y = torch.matmul((e / total).flatten(1, 2), v).unflatten(1, (-1, b - a))
            o[r + a: r + b] = y.permute(2, 0, 1, 3).reshape(b - a, heads, d).to(torch.bfloat16)
            lse[r + a: r + b] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(b - a, heads)
        r += count
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        cache = s["cache"]
        if op == "attend":
            o, lse = cache.attention(s["q"], lse=True, mass_decay=1.0 if c["mass"] else None)
            return dict(o=o, lse=lse, mass=s["mass"]) if c["mass"] else dict(o=o, lse=lse)
        if op == "prompt":
            o, lse = cache.prompt_attention(s["q"], s["counts"], lse=True, causal=c["causal"])
            return dict(o=o, lse=lse)
        if op == "store":
            cache.reset()
            cache.append(s["k"], s["v"], counts=s["counts"])
        k, v = cache.read(s["counts"])
        return dict(k=k, v=v)
    if op == "attend":
        return _plain_attend(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "store":
        _plain_store(s)
    return _plain_read(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, n = case, case["n_seqs"]
    kv, d, heads, op = c["kv_heads"], c["d"], c["heads"], c["op"]
    row = 2 * kv * d * {"bf16": 2, "e4m3": 1, "int4": 9 / 16}[c["dtype"]]  # a token's keys and values in the pages
    new = 2 * kv * d * 2                     # the same in 16 bits
    lens, counts = _lengths(n, c["lo"], c["hi"]), _counts(c)
    tokens, rows = sum(lens), sum(counts)
    pages = sum(-(-x // c["page"]) for x in lens) * 4
    if op == "store":                        # in, the pages written and read, out again
        return {"bytes": int(rows * (2 * new + 2 * row + 8)), "flops": 0}
    if op == "read":
        return {"bytes": int(rows * (new + row) + pages), "flops": 0}
    if op == "attend":
        rows, flops = n, 4 * tokens * heads * d
    else:
        seen = sum(m * x - (m * (m - 1) // 2 if c["causal"] else 0) for m, x in zip(counts, lens))
        flops = 4 * seen * heads * d
    nbytes = tokens * row + rows * heads * (2 * d * 2 + 4) + pages
    if op == "attend" and c["mass"]:
        nbytes += tokens * 8
        flops += tokens * heads
    return {"bytes": int(nbytes), "flops": int(flops)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _power(e):
    """Powers of two from a table: pow() on the GPU is off by a last bit here and there."""
    table = torch.tensor([2.0 ** k for k in range(-80, 81)], dtype=torch.float64, device=e.device)
    return table[e.long() + 80]


def _exact_tokens(s, i, j):
    """Sequence i's keys (j 0) or values (1): [length][kv][d]."""
    c = s["case"]
    kv, d, page = c["kv_heads"], c["d"], c["page"]
    length = s["lens"][i]
    npg = -(-length // page)
    x = s["k_pages" if j == 0 else "v_pages"].view(torch.uint8)[s["table"][i, :npg].long()]
    if c["dtype"] == "bf16":
        return x.view(torch.bfloat16).reshape(npg * page, kv, d)[:length].double()
    head = _power(s["exps"][j])[None, :, None]
    if c["dtype"] == "e4m3":
        return x.view(torch.float8_e4m3fn).reshape(npg * page, kv, d)[:length].double() * head
    rec = x.view(npg, kv, page // 16, 9 * d)
    words = rec[..., : 8 * d].contiguous().view(torch.int16).long() % 65536          # units of four values
    nibbles = [(words * 32768 % 65536 + words // 2) // 16 ** k % 16 - 8 for k in range(4)]
    n = torch.stack(nibbles, -1).view(npg, kv, page // 16, d // 32, 16, 32)
    n = n.permute(0, 2, 4, 1, 3, 5).reshape(npg * page, kv, d)
    b = rec[..., 8 * d:].reshape(npg, kv, page // 16, 16, d // 16).permute(0, 2, 3, 1, 4).reshape(npg * page, kv, d // 16)
    b = b.double()
    e, m = torch.floor(b / 8), b % 8
    s16 = torch.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * _power(e - 15))
    return (n.double() * s16.repeat_interleave(16, -1) * head)[:length]


def _exact_stored(x, exp):
    """What rows x [n][kv][d] become: blocks of 16 with a scale of four significant bits."""
    y = (x.double() / _power(exp)[None, :, None]).reshape(*x.shape[:2], -1, 16)
    unit = y.abs().max(-1, keepdim=True).values / 7
    mant, e = torch.frexp(unit)                                            # unit = mant * 2^e, mant in [1/2, 1)
    e = e.clamp(min=-13)
    mant = unit * _power(-e)
    scale = torch.floor(mant * 16 + 0.5) / 16 * _power(e)
    scale = scale.clamp(max=15 * 2.0 ** 8)
    k = torch.where(scale > 0, y / torch.where(scale > 0, scale, 1.0), 0.0)
    k = torch.where(k < 0, -torch.floor(0.5 - k), torch.floor(k + 0.5)).clamp(-8, 7)
    return (k * scale).reshape(x.shape) * _power(exp)[None, :, None]


def exact(case, seed):
    op = case["op"]
    if op == "attend" and work(case)["flops"] > 4e10:
        return None
    s = prepare(case, seed)
    if op == "store":
        return dict(k=_exact_stored(s["k"], s["exps"][0]), v=_exact_stored(s["v"], s["exps"][1]))
    kv, d = case["kv_heads"], case["d"]
    if op == "read":
        both = [torch.cat([_exact_tokens(s, i, j)[-m:] for i, m in enumerate(s["counts"])]) for j in range(2)]
        return dict(k=both[0], v=both[1])
    os, lses, r = [], [], 0
    for i, length in enumerate(s["lens"]):
        k, v = (_exact_tokens(s, i, j).transpose(0, 1) for j in range(2))  # [kv][L][d]
        count = s["counts"][i] if op == "prompt" else 1
        step = max(1, 60_000_000 // (length * case["heads"]))
        for a in range(0, count, step):
            b = min(a + step, count)
            q = s["q"][r + a: r + b].double().view(b - a, kv, -1, d)
            w = torch.einsum("rhgd,hld->hgrl", q, k) / math.sqrt(d)
            if op == "prompt" and case["causal"]:
                last = length - count + torch.arange(a, b, device=w.device)
                w.masked_fill_(torch.arange(length, device=w.device) > last[:, None], float("-inf"))
            lse = torch.logsumexp(w, -1)
            p = torch.exp(w - lse[..., None])
            os.append(torch.einsum("hgrl,hld->rhgd", p, v).reshape(b - a, -1, d))
            lses.append(lse.permute(2, 0, 1).reshape(b - a, -1))
            if op == "attend" and case["mass"]:
                if i == 0:
                    mass = s["mass"].double()
                mass[i, :length] += p.sum((0, 1, 2))
        r += count
    out = dict(o=torch.cat(os), lse=torch.cat(lses))
    if op == "attend" and case["mass"]:
        out["mass"] = mass
    return out
