"""Cases that time the paged token cache: appending tokens to pages, attention of one
new token per sequence over them, and eviction by accumulated attention weight.

`listed()` names the cases, `prepare()` makes one's inputs on the GPU, `run()` is one pass
(the plain torch form, or the library's calls when `own` is set), `work()` counts what a
pass has to move and compute, `exact()` computes a pass in 64 bits.

A sequence's token i (its logical index) is row `table[seq, i // page] * page + i % page`
of the page pool [n_pages * page][n_kv][d]. Pages hold bf16, or e4m3 with one power-of-two
scale per key/value head: value = e4m3 * 2^exp[head].
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one short conversation on a tiny model: nothing but latency
        dict(name="attend one short sequence", op="attend", n_seqs=1, lo=300, hi=300, heads=4, kv_heads=4, d=64,
             page=16, dtype="bf16", mass=False),
        # eight sessions at unequal fill levels (conditioning tokens alone, up to a full history), every head
        # with its own keys
        dict(name="attend 8 sessions, 40 key heads", op="attend", n_seqs=8, lo=2072, hi=11432, heads=40, kv_heads=40,
             d=128, page=64, dtype="bf16", mass=False),
        # one very long sequence: the only parallelism is along its length
        dict(name="attend one long sequence", op="attend", n_seqs=1, lo=131071, hi=131071, heads=40, kv_heads=8,
             d=128, page=64, dtype="bf16", mass=False),
        # a serving batch of every length from one token up, in small pages
        dict(name="attend 64 ragged sequences", op="attend", n_seqs=64, lo=1, hi=16384, heads=32, kv_heads=8, d=128,
             page=16, dtype="bf16", mass=False),
        # a large batch on 8-bit pages
        dict(name="attend 32 sequences, e4m3", op="attend", n_seqs=32, lo=4001, hi=32768, heads=40, kv_heads=8,
             d=128, page=64, dtype="e4m3", mass=False),
        # the same read as a serving batch with eviction makes: weights accumulated per token
        dict(name="attend 16 sequences with mass", op="attend", n_seqs=16, lo=1000, hi=8192, heads=40, kv_heads=8,
             d=128, page=64, dtype="bf16", mass=True),
        # one short prompt enters the cache
        dict(name="append one short prompt", op="append", n_seqs=1, lo=64, hi=64, heads=4, kv_heads=4, d=64, page=16,
             dtype="bf16"),
        # long prompts of several sequences enter together
        dict(name="append 8 prompts", op="append", n_seqs=8, lo=511, hi=16384, heads=40, kv_heads=8, d=128, page=64,
             dtype="bf16"),
        # the same, rounded to 8-bit pages
        dict(name="append 8 prompts, e4m3", op="append", n_seqs=8, lo=511, hi=16384, heads=40, kv_heads=8, d=128,
             page=64, dtype="e4m3"),
        # token by token at a fixed budget: one token in, one out, eight sequences
        dict(name="evict one of 1025, 8 sequences", op="evict", n_seqs=8, budget=1024, block=1, sink=4, recent=256,
             heads=32, kv_heads=8, d=128, page=16, dtype="bf16"),
        # a block of tokens in, as many out, long budgets
        dict(name="evict 512 of 16896, 16 sequences", op="evict", n_seqs=16, budget=16384, block=512, sink=64,
             recent=2048, heads=40, kv_heads=8, d=128, page=64, dtype="bf16"),
        # a whole serving step at a fixed budget: append, attend with weights, evict
        dict(name="serve step, 32 sequences", op="step", n_seqs=32, budget=4096, block=1, sink=4, recent=512,
             heads=32, kv_heads=8, d=128, page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "evict", "step"])
    kv, group = rng.choice([1, 2, 4, 5, 8, 8, 16]), rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(op=op, heads=kv * group, kv_heads=kv, d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 48, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "e4m3"]))
    row = kv * c["d"]                       # values of one token's keys
    if op in ("attend", "append"):
        c["n_seqs"] = _log(rng, 1, 64)
        most = min(65536, (450_000_000 if op == "attend" else 220_000_000) // (c["n_seqs"] * row * 2),
                   40_000_000 // (c["n_seqs"] * kv * group))
        most = max(most, 64)
        c["hi"] = _log(rng, 1, most)
        c["lo"] = _log(rng, 1, c["hi"])
        if op == "attend":
            c["mass"] = rng.random() < 0.4
    else:
        c["n_seqs"] = _log(rng, 1, 32)
        c["budget"] = _log(rng, 64, min(16384, max(256, 200_000_000 // (c["n_seqs"] * row * 2))))
        c["block"] = 1 if op == "step" else _log(rng, 1, max(1, min(512, c["budget"] // 8)))
        c["recent"] = rng.randint(c["block"], c["budget"] // 2)
        c["sink"] = rng.randint(0, c["budget"] // 8)
    return c


def _lengths(n, lo, hi):
    """n lengths spread over [lo, hi] on a logarithmic scale, the longest first."""
    u = [math.modf(i * 0.6180339887498949)[0] for i in range(n)]
    return [hi] + [min(hi, max(lo, int(round(lo * (hi / lo) ** x)))) for x in u[1:]]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)
    c, n = dict(case), case["n_seqs"]
    op, heads, kv, d, page = c["op"], c["heads"], c["kv_heads"], c["d"], c["page"]
    if op in ("attend", "append"):
        lens = _lengths(n, c["lo"], c["hi"])
        caps = lens
    else:
        lens = [c["budget"]] * n
        caps = [c["budget"] + c["block"]] * n
    pages_of = [-(-x // page) for x in caps]
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

    # stale values everywhere: what earlier sequences left in the pages
    e4m3 = c["dtype"] == "e4m3"
    exps = torch.randint(-3, 3, (2, kv), generator=g, device=dev, dtype=torch.int32)
    pool = []
    for i in range(2):
        x = torch.empty((n_pages, page, kv, d), dtype=torch.bfloat16, device=dev)
        x.normal_(generator=g)
        if e4m3:
            x = (x * 16).to(torch.float8_e4m3fn)
        pool.append(x)
    if e4m3:                                 # values of about unit size come out
        exps -= 4
    cap = width * page
    s = dict(case=c, n=n, lens=lens, cap=cap, k_pages=pool[0], v_pages=pool[1], exps=exps, table=table,
             seq_len=torch.tensor(lens, dtype=torch.int32, device=dev),
             scale=1.0 / math.sqrt(d))
    if op in ("attend", "append"):
        s["seq_pos"] = s["seq_len"].clone()
        s["token_pos"] = torch.arange(cap, dtype=torch.int32, device=dev).repeat(n, 1)
    else:
        # positions with gaps where tokens were evicted before; the sinks and the recent tokens are whole
        old = c["budget"] - c["recent"]
        gaps = torch.randint(1, 5, (n, old), generator=g, device=dev)
        gaps[:, : c["sink"]] = 1
        pos = torch.cumsum(gaps, 1) - 1
        start = pos[:, -1:] + 1
        rec = start + torch.arange(c["recent"] + cap - c["budget"], device=dev)
        s["token_pos"] = torch.cat([pos, rec], 1).to(torch.int32)
        s["seq_pos"] = (start[:, 0] + c["recent"]).to(torch.int32)
    # weights gathered so far: a few tokens hold most of them
    s["mass"] = torch.exp(2.0 * randn(n, cap))
    if op == "append":
        rows = sum(lens)
    else:
        rows = n * c.get("block", 1)
    s["k"] = (randn(rows, kv, d) if op != "attend" else randn(1, kv, d)).to(torch.bfloat16)
    s["v"] = (randn(rows, kv, d) if op != "attend" else randn(1, kv, d)).to(torch.bfloat16)
    s["counts"] = lens if op == "append" else [c.get("block", 1)] * n
    s["counts_dev"] = torch.tensor(s["counts"], device=dev)
    s["q"] = (1.5 * randn(n, heads, d)).to(torch.bfloat16)
    if own:
        import chunked_kv_cache_gb300 as sr
        s["cache"] = sr.PagedCache(
            heads, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=n, max_pages=width,
            page_dtype=pool[0].dtype, device=dev,
            buffers=dict(k_pages=s["k_pages"], v_pages=s["v_pages"], block_table=table, seq_len=s["seq_len"],
                         seq_pos=s["seq_pos"], token_pos=s["token_pos"], token_mass=s["mass"], kv_exp=exps))
    return s


# ------------------------------------------------------------------ the plain form
def _rows(s, seq, idx):
    """Pool rows of tokens idx of sequences seq."""
    page = s["case"]["page"]
    return s["table"][seq, idx // page].long().clamp(min=0) * page + idx % page


def _gather(s, pages, exp, rows):
    kv, d = s["case"]["kv_heads"], s["case"]["d"]
    if pages.dtype == torch.bfloat16:
        return pages.view(-1, kv, d)[rows].float()
    x = pages.view(torch.uint8).view(-1, kv, d)[rows].view(torch.float8_e4m3fn).float()
    return x * torch.exp2(exp.float())[:, None]


def _store(s, pages, exp, rows, x):
    kv, d = s["case"]["kv_heads"], s["case"]["d"]
    if pages.dtype == torch.bfloat16:
        pages.view(-1, kv, d)[rows] = x
        return
    y = (x.float() * torch.exp2(-exp.float())[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    pages.view(torch.uint8).view(-1, kv, d)[rows] = y.view(torch.uint8)


def _plain_append(s):
    n, dev = s["n"], s["k"].device
    rows = s["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device=dev), s["counts_dev"], output_size=rows)
    first = torch.cumsum(s["counts_dev"], 0) - s["counts_dev"]
    i = torch.arange(rows, device=dev) - first[seq]
    idx = s["seq_len"][seq].long() + i
    at = _rows(s, seq, idx)
    _store(s, s["k_pages"], s["exps"][0], at, s["k"])
    _store(s, s["v_pages"], s["exps"][1], at, s["v"])
    s["token_pos"][seq, idx] = (s["seq_pos"][seq].long() + i).to(torch.int32)
    s["mass"][seq, idx] = 0.0
    s["seq_len"] += s["counts_dev"].to(torch.int32)
    s["seq_pos"] += s["counts_dev"].to(torch.int32)


def _plain_attend(s, mass):
    c, n, dev = s["case"], s["n"], s["q"].device
    kv, d = c["kv_heads"], c["d"]
    most = s["cap"]
    idx = torch.arange(most, device=dev)
    live = idx[None, :] < s["seq_len"][:, None]
    rows = _rows(s, torch.arange(n, device=dev)[:, None], idx[None, :])
    k = _gather(s, s["k_pages"], s["exps"][0], rows)                       # [n][L][kv][d]
    q = s["q"].float().view(n, kv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                # [n][kv][group][L]
    del k
    x = torch.where(live[:, None, None, :], x, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp(min=1e-30)
    v = _gather(s, s["v_pages"], s["exps"][1], rows)
    v = torch.where(live[:, :, None, None], v, 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(n, -1, d).to(torch.bfloat16)
    lse = (top + torch.log(total)).reshape(n, -1)
    if mass:
        s["mass"] += p.sum((1, 2))
    return o, lse


def _plain_evict(s):
    c, n, dev = s["case"], s["n"], s["q"].device
    budget, most, cap = c["budget"], c["block"], s["cap"]
    idx = torch.arange(cap, device=dev)[None, :]
    live = idx < s["seq_len"][:, None]
    whole = (s["token_pos"] < c["sink"]) | (s["token_pos"] >= s["seq_pos"][:, None] - c["recent"])
    key = torch.where(whole, float("inf"), s["mass"])
    key = torch.where(live, key, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    keep = torch.zeros((n, cap), dtype=torch.bool, device=dev)
    keep.scatter_(1, order[:, :budget], True)
    keep &= live
    # the j-th evicted token among the first `budget` gives its place to the j-th kept one behind them
    hole = torch.sort((~(live & ~keep))[:, :budget].to(torch.int8), dim=1, stable=True).indices[:, :most]
    back = torch.sort((~keep)[:, budget:].to(torch.int8), dim=1, stable=True).indices[:, :most] + budget
    moves = keep[:, budget:].sum(1, keepdim=True)
    real = torch.arange(back.shape[1], device=dev)[None, :] < moves
    hole = torch.where(real, hole[:, : back.shape[1]], back)              # no move: a token onto itself
    b = torch.arange(n, device=dev)[:, None]
    src, dst = _rows(s, b, back), _rows(s, b, hole)
    kv, d = c["kv_heads"], c["d"]
    for pages in (s["k_pages"], s["v_pages"]):
        x = pages.view(torch.uint8).view(-1, kv * d * pages.element_size())
        x[dst] = x[src]
    s["token_pos"].scatter_(1, hole, s["token_pos"].gather(1, back))
    s["mass"].scatter_(1, hole, s["mass"].gather(1, back))
    s["seq_len"].clamp_(max=budget)


# ------------------------------------------------------------------ one pass
def _cache_state(s):
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], token_pos=s["token_pos"], mass=s["mass"],
                seq_len=s["seq_len"], seq_pos=s["seq_pos"])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        cache = s["cache"]
        if op == "attend":
            o, lse = cache.attention(s["q"], lse=True, mass_decay=1.0 if c["mass"] else None)
            return dict(o=o, lse=lse, mass=s["mass"]) if c["mass"] else dict(o=o, lse=lse)
        if op == "append":
            cache.reset()
            cache.append(s["k"], s["v"], counts=s["counts"])
            return _cache_state(s)
        cache.append(s["k"], s["v"], counts=s["counts"])
        out = {}
        if op == "step":
            out["o"], out["lse"] = cache.attention(s["q"], lse=True, mass_decay=1.0)
        cache.evict(c["budget"], n_sink=c["sink"], n_recent=c["recent"])
        return dict(out, **_cache_state(s))
    if op == "attend":
        o, lse = _plain_attend(s, c["mass"])
        return dict(o=o, lse=lse, mass=s["mass"]) if c["mass"] else dict(o=o, lse=lse)
    if op == "append":
        s["seq_len"].zero_()
        s["seq_pos"].zero_()
        _plain_append(s)
        return _cache_state(s)
    _plain_append(s)
    out = {}
    if op == "step":
        out["o"], out["lse"] = _plain_attend(s, True)
    _plain_evict(s)
    return dict(out, **_cache_state(s))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, n = case, case["n_seqs"]
    kv, d, heads = c["kv_heads"], c["d"], c["heads"]
    size = 2 if c["dtype"] == "bf16" else 1
    row = 2 * kv * d * size                  # a token's keys and values in the pages
    new = 2 * kv * d * 2                     # a new token's, as they come in
    op = c["op"]
    if op in ("attend", "append"):
        lens = _lengths(n, c["lo"], c["hi"])
    else:
        lens = [c["budget"] + c["block"]] * n
    tokens = sum(lens)
    nbytes = flops = 0
    if op in ("attend", "step"):
        nbytes += tokens * row + n * heads * (2 * d * 2 + 4) + sum(-(-x // c["page"]) for x in lens) * 4
        flops += 4 * tokens * heads * d
        if op == "step" or c["mass"]:
            nbytes += tokens * 8
            flops += tokens * heads
    if op in ("append", "evict", "step"):
        rows = tokens if op == "append" else n * c["block"]
        nbytes += rows * (new + row + 8)
    if op in ("evict", "step"):
        nbytes += tokens * 8 + n * c["block"] * (2 * row + 16)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_attend(s, i, length):
    """One sequence: outputs, log-sum-exp and the weights of its tokens summed over heads."""
    c = s["case"]
    kv, d, page = c["kv_heads"], c["d"], c["page"]
    npg = -(-length // page)
    at = s["table"][i, :npg].long()
    both = []
    for j, pages in enumerate((s["k_pages"], s["v_pages"])):
        x = pages.view(torch.uint8)[at].view(pages.dtype).reshape(npg * page, kv, d)[:length]
        x = x.to(torch.float64)
        if c["dtype"] == "e4m3":
            x = x * (2.0 ** s["exps"][j].double())[None, :, None]
        both.append(x.transpose(0, 1))                                     # [kv][L][d]
    q = s["q"][i].double().view(kv, -1, d)
    w = torch.einsum("hgd,hld->hgl", q, both[0]) / math.sqrt(d)
    lse = torch.logsumexp(w, -1)
    p = torch.exp(w - lse[..., None])
    o = torch.einsum("hgl,hld->hgd", p, both[1])
    return o.reshape(-1, d), lse.reshape(-1), p.sum((0, 1))


def _exact_append(s, starts):
    c = s["case"]
    kv, d, page = c["kv_heads"], c["d"], c["page"]
    r = 0
    for i, count in enumerate(s["counts"]):
        t = torch.arange(starts[i], starts[i] + count, device=s["k"].device)
        at, slot = s["table"][i].long()[t // page], t % page
        for j, (pages, x) in enumerate(((s["k_pages"], s["k"]), (s["v_pages"], s["v"]))):
            y = x[r: r + count].double()
            if c["dtype"] == "e4m3":
                y = torch.ldexp(y, -s["exps"][j][None, :, None]).clamp(-448, 448)
            pages.view(torch.uint8)[at, slot] = y.to(pages.dtype).view(torch.uint8)
        s["token_pos"][i, t] = (s["seq_pos"][i] + t - starts[i]).to(torch.int32)
        s["mass"][i, t] = 0
        s["seq_len"][i] = starts[i] + count
        s["seq_pos"][i] += count
        r += count


def _exact_evict(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    for i in range(s["n"]):
        length, nxt = int(s["seq_len"][i]), int(s["seq_pos"][i])
        if length <= budget:
            continue
        pos, m = s["token_pos"][i].tolist(), s["mass"][i].tolist()
        free = [t for t in range(length) if c["sink"] <= pos[t] < nxt - c["recent"]]
        free.sort(key=lambda t: (m[t], -t))
        gone = set(free[: length - budget])
        holes = sorted(t for t in gone if t < budget)
        back = [t for t in range(budget, length) if t not in gone]
        tab = s["table"][i].tolist()
        for h, b in zip(holes, back):
            for pages in (s["k_pages"], s["v_pages"]):
                x = pages.view(torch.uint8)
                x[tab[h // page], h % page] = x[tab[b // page], b % page]
            s["token_pos"][i, h] = pos[b]
            s["mass"][i, h] = m[b]
        s["seq_len"][i] = budget


def exact(case, seed):
    if case["op"] in ("attend", "step") and work(case)["flops"] > 4e10:
        return None
    if case["op"] == "evict" and case["n_seqs"] * case["block"] > 20000:
        return None
    s = prepare(case, seed)
    s["mass"] = s["mass"].double()
    op = case["op"]
    out = {}
    if op == "append":
        s["seq_pos"].zero_()
        _exact_append(s, [0] * s["n"])
    elif op in ("evict", "step"):
        _exact_append(s, s["lens"])
    if op in ("attend", "step"):
        o, lse = [], []
        for i, length in enumerate(s["seq_len"].tolist()):
            a, b, w = _exact_attend(s, i, length)
            o.append(a)
            lse.append(b)
            if op == "step" or case["mass"]:
                s["mass"][i, :length] += w
        out["o"], out["lse"] = torch.stack(o), torch.stack(lse)
        if op == "attend":
            if case["mass"]:
                out["mass"] = s["mass"]
            return out
    if op in ("evict", "step"):
        _exact_evict(s)
    for name in ("k_pages", "v_pages", "token_pos", "mass", "seq_len", "seq_pos"):
        out[name] = s[name]
    return out
