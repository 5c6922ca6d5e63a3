"""Pages' assignment (host_transfer_amd.kv_pages) and the 8-bit paged K/V cache (host_transfer_amd.kv8)
as cases to measure.

Three operators: `assign` (page tables, slots and positions of a step's tokens, from the requests'
lengths), `append` (norm + rotation of new keys and queries, and the new keys and values into a cache of
e4m3 codes with a power-of-two scale for each block of tokens and head) and `attend` (a chunk of new
tokens, or single tokens, over such a cache).  Where `own` is false, `run` computes them in elementary
torch operations in 32 bits (assign in whole numbers).
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the next token of the 20 sequences of the OPT-13B K/V shape: the smallest step
        dict(name="assign_kv_opt13b", op="assign", seqs=20, page=16, kv=2047, add=1, reject=0, ended=0, started=0),
        # a step of 250 requests that verify drafted tokens: some were rejected, some requests ended
        dict(name="assign_drafts", op="assign", seqs=250, page=16, kv=8192, add=5, reject=4, ended=5, started=0),
        # a step that admits 40 prompts beside 24 running requests
        dict(name="assign_prompts", op="assign", seqs=64, page=32, kv=30000, add=4096, reject=0, ended=2, started=40),
        # one new token of one sequence, in the middle of a block: the smallest call of a decode step
        dict(name="append8_one_token", op="append", dtype="bf16", hq=32, hkv=8, d=128, page=16, block=16, seqs=1,
             q=1, kv=37, spread=0, rope=128, inter=False, norm=True, pad=0),
        # one decode token of the 20 sequences of the OPT-13B K/V shape (no rotation there)
        dict(name="append8_kv_opt13b", op="append", dtype="f16", hq=0, hkv=40, d=128, page=16, block=16, seqs=20,
             q=1, kv=2048, spread=6, rope=0, inter=False, norm=False, pad=0),
        # a batch of prompts, padded behind the last: norms and rotation of queries and keys for every head
        dict(name="append8_prompts", op="append", dtype="bf16", hq=32, hkv=8, d=128, page=64, block=16, seqs=6,
             q=4001, kv=4001, spread=60, rope=128, inter=False, norm=True, pad=23),
        # a short conversation, one token: latency
        dict(name="attend8_short", op="attend", dtype="bf16", hq=16, hkv=2, d=64, page=16, block=16, seqs=1, q=1,
             kv=37, spread=0, window=0, causal=True, empty=False),
        # one decode token of the OPT-13B K/V shape: 20 sequences of 1,920 + 128 tokens
        dict(name="attend8_kv_opt13b", op="attend", dtype="f16", hq=40, hkv=40, d=128, page=16, block=16, seqs=20,
             q=1, kv=2048, spread=6, window=0, causal=True, empty=False),
        # one decode token over long contexts, queries in groups
        dict(name="attend8_long", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=64, block=32, seqs=4, q=1,
             kv=131072, spread=50, window=0, causal=True, empty=False),
        # five drafted tokens of each request are verified
        dict(name="attend8_drafts", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=16, block=16, seqs=24, q=5,
             kv=8192, spread=80, window=0, causal=True, empty=True),
        # chunks of prompts that are prefilled piece by piece, ragged
        dict(name="attend8_chunk", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=16, block=16, seqs=6, q=511,
             kv=9001, spread=70, window=0, causal=True, empty=True),
        # one whole prompt
        dict(name="attend8_prompt", op="attend", dtype="f16", hq=32, hkv=8, d=128, page=64, block=64, seqs=1,
             q=12000, kv=12000, spread=0, window=0, causal=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "attend", "attend"])
    if op == "assign":
        seqs = _log(rng, 1, 3000)
        started = rng.choice([0, 0, 0, rng.randrange(0, seqs + 1)])
        add = _log(rng, 1, max(2, 160_000 // max(1, started))) if started else rng.choice([1, 1, 2, 5, 9])
        return dict(op=op, seqs=seqs, page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]),
                    kv=_log(rng, 20, min(131072, 12_000_000 // seqs)), add=min(add, 8000),
                    reject=rng.choice([0, 0, 1, 4, 30]), ended=rng.choice([0, 0, min(seqs, _log(rng, 1, 40))]),
                    started=started)
    d = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 5, 8, 8, 40])
    if hkv * d > 8192:
        hkv = 8
    group = rng.choice([1, 2, 3, 4, 8])
    if hkv * group > 64:
        group = 1
    block = rng.choice([1, 8, 16, 16, 16, 24, 32, 64])
    page = block * rng.choice([1, 1, 2, 3, 4]) if block > 1 else rng.choice([1, 4])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), d=d, hkv=hkv, page=page, block=block,
             spread=rng.randrange(0, 100))
    width = hkv * d
    if op == "append":
        q = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 9, 4000)])
        c["seqs"] = _log(rng, 1, 256 if q <= 8 else 8)
        c["q"] = max(1, min(q, 16_000_000 // width // max(1, group // 2) // c["seqs"]))
        c["kv"] = c["q"] + rng.choice([0, _log(rng, 1, max(2, min(4000, 60_000_000 // width // c["seqs"])))])
        c.update(hq=rng.choice([0, hkv * group]), rope=rng.choice([0, d, d, 32]), inter=rng.random() < 0.5,
                 norm=rng.random() < 0.5, pad=rng.choice([0, 0, 1, 30]))
        return c
    c["hq"] = hkv * group
    if rng.random() < 0.55:
        c["q"], c["seqs"] = rng.choice([1, 1, 1, 2, 4, 5]), _log(rng, 1, 64)
    else:
        c["q"], c["seqs"] = _log(rng, 6, 4096), _log(rng, 1, 8)
    room = 250_000_000 // width // c["seqs"]
    work_ = int(3e8 // (c["q"] * c["seqs"] * c["hq"] * d / 1000))
    c["kv"] = _log(rng, 1, max(2, min(131072, room, work_)))
    c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    c["causal"] = bool(c["window"]) or rng.random() < 0.85
    c["empty"] = rng.random() < 0.3
    return c


def _lens(c):
    """Lengths of the sequences: new tokens and all tokens (the new ones are the last)."""
    s = c["seqs"]
    qs, ks = [], []
    for i in range(s):
        cut = c["spread"] * i / (100.0 * max(1, s - 1))
        k = max(1, c["kv"] - int(c["kv"] * cut))
        q = c["q"] if c["q"] <= 8 else max(1, c["q"] - int(c["q"] * cut))
        qs.append(min(q, k))
        ks.append(k)
    if c.get("empty"):  # a slot of the batch that no sequence uses, in the middle
        qs.insert(s // 2, 0)
        ks.insert(s // 2, 0)
    return qs, ks


def _requests(c):
    """Tokens held, kept and new of each request of an assign case."""
    had, keep, add = [], [], []
    for i in range(c["seqs"]):
        h = 1 + (i * 7919 + 13) * 104729 % c["kv"]
        a, k = (c["add"] if c["add"] <= 16 else 1), h
        if c["reject"]:
            k = max(0, h - i % (c["reject"] + 1))
        if i < c["ended"]:
            k = a = 0
        elif i >= c["seqs"] - c["started"]:
            h = k = 0
            a = max(1, c["add"] - i * 31 % (c["add"] // 2 + 1))
        had.append(h)
        keep.append(k)
        add.append(a)
    return had, keep, add


def _pages(n, p):
    return -(-n // p)


def work(c):
    if c["op"] == "assign":
        had, keep, add = _requests(c)
        moved = sum(abs(_pages(k + a, c["page"]) - _pages(h, c["page"])) for h, k, a in zip(had, keep, add))
        return dict(bytes=24 * c["seqs"] + 16 * sum(add) + 8 * moved, flops=0)
    d, hkv, hq = c["d"], c["hkv"], c["hq"]
    qs, ks = _lens(c)
    nq = sum(qs)
    if c["op"] == "append":
        blocks = sum(_pages(k, c["block"]) - (k - q) // c["block"] for q, k in zip(qs, ks) if q)
        table = nq * (4 * c["rope"] + 8) if c["rope"] else 0
        ops = nq * (hq + hkv) * (3 * c["rope"] + (4 * d if c["norm"] else 0)) + 6 * nq * hkv * d
        return dict(bytes=nq * d * (4 * hq + 6 * hkv) + table + 2 * blocks * hkv, flops=ops)
    w, pairs, keys = c["window"], 0, 0
    for q, k in zip(qs, ks):
        if not c["causal"]:
            pairs += q * k
        elif w:
            pairs += sum(min(w, p + 1) for p in range(k - q, k))
        else:
            pairs += q * k - q * (q - 1) // 2
        keys += min(k, q + w - 1) if w and q else (k if q else 0)
    exps = 2 * hkv * sum(_pages(k, c["block"]) for k in ks)
    return dict(bytes=2 * nq * hq * d * 2 + 4 * nq * hq + keys * hkv * d * 2 + exps +
                4 * sum(_pages(k, c["page"]) for k in ks), flops=4 * pairs * hq * d)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dt, scale=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if scale is not None:
        x *= scale
    return x.to(dt)


def _power(e):
    """2^(e - 127) of whole numbers e in [1, 254], exactly."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _exponent(amax):
    """The least e in [1, 254] with amax <= 448 * 2^(e - 127)."""
    m, x = torch.frexp(amax)
    return torch.where(amax == 0, 1, (x + 118 + (m > 0.875)).clamp(1, 254)).to(torch.uint8)


def _scales(g, h, d):
    """Channel scales of a K/V row: log-uniform in [0.1, 4] (as the K/V workload's)."""
    u = torch.rand((h, d), generator=g, device="cuda")
    return torch.exp(math.log(0.1) + u * math.log(40.0))


def _pool(g, c, n_pages):
    """Codes (pages, page, heads, d) and exponents (pages, blocks, heads) of K/V rows, filled in
    pieces (the 32-bit form is not held whole)."""
    p, b, h, d = c["page"], c["block"], c["hkv"], c["d"]
    codes = torch.empty((n_pages, p, h, d), dtype=E4M3, device="cuda")
    exps = torch.empty((n_pages, p // b, h), dtype=torch.uint8, device="cuda")
    s = _scales(g, h, d)
    step = max(1, 50_000_000 // (p * h * d))
    for i in range(0, n_pages, step):
        x = _normal(g, codes[i:i + step].shape, DT[c["dtype"]], s).float().unflatten(1, (p // b, b))
        e = _exponent(x.abs().amax((2, 4)))
        exps[i:i + step] = e
        codes[i:i + step] = (x / _power(e)[:, :, None, :, None]).to(E4M3).flatten(1, 2)
    return codes, exps


def _rope_table(n_pos, r):
    """Row p: r/2 cosines, then r/2 sines, of p * 10000^(-2i/r) (angles in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_assign(c, g):
    had, keep, add = _requests(c)
    p = c["page"]
    held = [_pages(h, p) for h in had]
    width = max(max(_pages(k + a, p) for k, a in zip(keep, add)), max(held)) + 2
    acquired = sum(max(0, _pages(k + a, p) - h) for k, a, h in zip(keep, add, held))
    n_pages = sum(held) + acquired + 7
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    own_pages = i32(held)
    col = torch.arange(width, device="cuda")
    first = own_pages.cumsum(0) - own_pages
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    n_rows = sum(add) + 3  # a batch padded by some rows
    e32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    free = e32(n_pages)
    free[:n_pages - sum(held)] = order[sum(held):]
    return dict(table=torch.where(col < own_pages[:, None], order[at], -1).int(), free=free,
                free_count=i32([n_pages - sum(held)]), had=i32(had), keep=i32(keep), add=i32(add), n_pages=n_pages,
                q_start=e32(c["seqs"] + 1), kv_len=e32(c["seqs"]), length=e32(c["seqs"]), left=e32(1),
                unserved=e32(1), slots=torch.zeros(n_rows, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(n_rows, dtype=torch.int64, device="cuda"))


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "assign":
        st = _prepare_assign(c, g)
        st["c"] = c
        if own:
            from host_transfer_amd import kv_pages
            st["pool"] = kv_pages.Pool(st["table"], st["free"], st["n_pages"], c["page"])
            st["ws"] = torch.empty(max(16, kv_pages.assign_workspace(c["seqs"], st["slots"].numel())),
                                   dtype=torch.uint8, device="cuda")
        return st
    dt, d, hkv, hq, p = DT[c["dtype"]], c["d"], c["hkv"], c["hq"], c["page"]
    qs, ks = _lens(c)
    need = [_pages(k, p) for k in ks]
    n_pages = sum(need) + 2
    st = {"c": c, "qs": qs, "ks": ks}
    st["k"], st["ke"] = _pool(g, c, n_pages)
    st["v"], st["ve"] = _pool(g, c, n_pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(ks), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    starts = [0]
    for q in qs:
        starts.append(starts[-1] + q)
    st["starts"], st["table"] = starts, table
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(ks, dtype=torch.int32, device="cuda")
    nq = starts[-1] + c.get("pad", 0)
    # the rows of one fused projection: queries, keys and values of a token side by side
    qkv = _normal(g, (nq, hq + 2 * hkv, d), dt)
    st["q"] = qkv[:, :hq] if hq else None
    if c["op"] == "append":
        st["nk"], st["nv"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_out"] = torch.zeros((nq, hq, d), dtype=dt, device="cuda") if hq else None
        # the sequence and the position of every row (a row behind the last: sequence -1)
        st["seq"] = torch.repeat_interleave(torch.arange(len(qs), device="cuda"),
                                            torch.tensor(qs, device="cuda"), output_size=starts[-1])
        last = st["kv_len"].long() - st["q_start"][1:].long()
        pos = torch.full((nq,), -1, dtype=torch.int64, device="cuda")
        pos[:starts[-1]] = torch.arange(starts[-1], device="cuda") + last[st["seq"]]
        st["pos"] = pos
        st["rope"] = _rope_table(max(2048, c["kv"]), c["rope"]) if c["rope"] else None
        st["qn"] = st["kn"] = None
        if c["norm"]:
            st["qn"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if hq else None
            st["kn"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
    else:
        st["scale"] = 1.0 / math.sqrt(d)
        st["out"] = torch.zeros((nq, hq, d), dtype=dt, device="cuda")
        st["lse"] = torch.zeros((nq, hq), dtype=torch.float32, device="cuda")
    if own:
        from host_transfer_amd import kv, kv8
        st["cache"] = kv8.Cache(st["k"], st["v"], st["ke"], st["ve"])
        st["batch"] = kv.Batch(st["q_start"], st["kv_len"], table, max_q=max(qs), max_kv=max(ks))
        if c["op"] == "attend":
            n = kv8.attend_workspace(st["cache"], st["batch"], nq, hq)
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- the operators

def run(st):
    c = st["c"]
    if c["op"] == "assign":
        if own:
            from host_transfer_amd import kv_pages
            kv_pages.assign(st["pool"], st["had"], st["add"], st["free_count"], st["q_start"], st["kv_len"],
                            st["length"], st["left"], st["slots"], st["positions"], keep=st["keep"],
                            unserved=st["unserved"], workspace=st["ws"])
        else:
            _assign(st)
        return {k: st[k] for k in ("table", "free", "left", "q_start", "kv_len", "length", "slots", "positions",
                                   "unserved")}
    if c["op"] == "append":
        if own:
            from host_transfer_amd import kv8
            kv8.append(st["cache"], st["batch"], st["nk"], st["nv"], q=st["q"], q_out=st["q_out"],
                       positions=st["pos"] if c["rope"] else None, rope=st["rope"],
                       flags=kv8.ROPE_INTERLEAVED if c["inter"] and c["rope"] else 0, q_norm=st["qn"],
                       k_norm=st["kn"], eps=1e-6)
        else:
            _append(st)
        # codes as the e4m3 numbers they are, exponents as whole numbers: a value is code * 2^(e - 127)
        out = {"k": st["k"], "v": st["v"], "k_exp": st["ke"], "v_exp": st["ve"]}
        if c["hq"]:
            out["q"] = st["q_out"]
        return out
    if own:
        from host_transfer_amd import kv8
        kv8.attend(st["cache"], st["batch"], st["q"], st["out"], st["scale"], window=c["window"],
                   flags=kv8.CAUSAL if c["causal"] else 0, lse=st["lse"], workspace=st["ws"])
    else:
        _attend(st)
    return {"out": st["out"], "lse": st["lse"]}


def _assign(st):
    """Every request and page at once, by prefix sums."""
    p, table, free = st["c"]["page"], st["table"], st["free"]
    n, width = table.shape
    had, keep, add = (st[k].long() for k in ("had", "keep", "add"))
    want = keep + add
    held, wanted = (had + p - 1) // p, (want + p - 1) // p
    ends = add.cumsum(0)
    fits = (ends <= st["slots"].numel()) & (wanted <= width)
    need = torch.where(fits, (wanted - held).clamp(min=0), 0)
    col = torch.arange(width, device="cuda")
    gives = (col >= wanted[:, None]) & (col < held[:, None]) & (table >= 0) & (table < st["n_pages"])
    gives &= fits[:, None]
    order = gives.flatten().cumsum(0).view(n, width) - 1 + st["free_count"]
    avail = order[-1, -1] + 1
    # pages given back go on the stack; a place behind it takes the writes of all others
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(gives, order, free.numel()).flatten(), table.flatten())
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= avail))
    taken = torch.where(served & (need > 0), upto, 0).amax()
    at = avail - 1 - ((upto - need - held)[:, None] + col)
    fresh = (col >= held[:, None]) & (col < wanted[:, None]) & served[:, None]
    table.copy_(torch.where(fresh, stack[at.clamp(0, free.numel())], table))
    free.copy_(stack[:-1])
    st["left"].copy_((avail - taken).view(1))
    st["q_start"][1:] = ends.clamp(max=st["slots"].numel())
    st["kv_len"].copy_(torch.where(served, want, 0))
    st["length"].copy_(torch.where(served, want, had))
    st["unserved"].copy_((~served).sum().view(1))
    r = torch.arange(st["slots"].numel(), device="cuda")
    s = torch.searchsorted(ends, r, right=True)
    there = s < n
    s = s.clamp(max=n - 1)
    there &= served[s]
    pos = torch.where(there, keep[s] + r - (ends - add)[s], 0)
    page = table[s, (pos // p).clamp(max=width - 1)].long()
    st["positions"].copy_(torch.where(there, pos, -1))
    st["slots"].copy_(torch.where(there & (page >= 0) & (page < st["n_pages"]), page * p + pos % p, -1))


def _norm_rotate(st, x, w):
    """x (n, heads, d) in 32 bits: each head's norm, then the rotation of its first channels."""
    c = st["c"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    r = c["rope"]
    if r:
        cs = st["rope"][st["pos"][:x.shape[0]]][:, None, :]
        co, si = cs[..., :r // 2], cs[..., r // 2:]
        if c["inter"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat([a * co - b * si, b * co + a * si], -1)
        y = torch.cat([z, y[..., r:]], -1)
    return y


def _append(st):
    c = st["c"]
    n, p, b, h, d = st["starts"][-1], c["page"], c["block"], c["hkv"], c["d"]
    pos = st["pos"][:n]
    slot = st["table"][st["seq"], pos // p].long() * p + pos % p
    block, inside = slot // b, slot % b
    # the first new token of each block, b where it has none
    begin = torch.full((st["ke"].numel() // h,), b, device="cuda").scatter_reduce(0, block, inside, "amin")
    # the blocks that gain tokens, in the tokens' order (their number follows from the lengths)
    first = inside == begin[block]
    count = sum(_pages(k, b) - (k - q) // b for q, k in zip(st["qs"], st["ks"]) if q)
    touched = block.new_empty(count + 1).scatter_(0, torch.where(first, first.cumsum(0) - 1, count), block)[:count]
    for codes, exps, x in ((st["k"], st["ke"], _norm_rotate(st, st["nk"][:n], st["kn"])),
                           (st["v"], st["ve"], st["nv"][:n].float())):
        top = torch.zeros((begin.numel(), h), device="cuda")
        top.scatter_reduce_(0, block[:, None].expand(n, h), x.abs().amax(-1), "amax")
        was = exps.view(-1, h)[touched]
        now = _exponent(top[touched])
        now = torch.where((begin[touched] == 0)[:, None], now, torch.maximum(now, was))
        raw = codes.view(torch.uint8).view(-1, b, h, d)
        # tokens in front of the first new one, at the new scale (a division by one leaves them as they are)
        old = raw[touched].view(E4M3).float() * (_power(was) / _power(now))[:, None, :, None]
        old = old.to(E4M3).view(torch.uint8)
        before = torch.arange(b, device="cuda") < begin[touched][:, None]
        raw[touched] = torch.where(before[:, :, None, None], old, raw[touched])
        exps.view(-1, h)[touched] = now
        e = exps.view(-1, h)[block]
        raw.view(-1, h, d)[slot] = (x / _power(e)[:, :, None]).to(E4M3).view(torch.uint8)
    if c["hq"]:
        st["q_out"][:n] = _norm_rotate(st, st["q"][:n], st["qn"]).to(st["q_out"].dtype)


def _keys(st, i, k, lo=0):
    """The key and value rows lo..k-1 of sequence i, in 32 bits: (tokens, heads, d) each."""
    p, b = st["c"]["page"], st["c"]["block"]
    ids = st["table"][i, lo // p:_pages(k, p)].long()
    off = lo - lo // p * p
    out = []
    for codes, exps in ((st["k"], st["ke"]), (st["v"], st["ve"])):
        x = codes.view(torch.uint8)[ids].view(E4M3).float().unflatten(1, (p // b, b))
        x = x * _power(exps[ids])[:, :, None, :, None]
        out.append(x.flatten(0, 2)[off:off + k - lo])
    return out


def _softmax_rows(s, v):
    """Rows of scores (..., m, n) over values (..., n, d): outputs and logs of the sums."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(s - top)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, torch.ones_like(z), z)
    return o, (torch.log(z) + top)[..., 0]


def _attend(st):
    c = st["c"]
    g, d, w = c["hq"] // c["hkv"], c["d"], c["window"]
    for i, (q, k) in enumerate(zip(st["qs"], st["ks"])):
        if not q:
            continue
        lo = max(0, k - q - w + 1) if w else 0
        ks, vs = _keys(st, i, k, lo)
        kt = ks.permute(1, 2, 0).contiguous()
        vt = vs.transpose(0, 1).contiguous()
        step = max(1, min(q, 800_000_000 // ((k - lo) * c["hq"])))
        for r in range(0, q, step):
            m = min(step, q - r)
            pos = torch.arange(k - q + r, k - q + r + m, device="cuda")[:, None, None]
            at = torch.arange(lo, k, device="cuda")
            part = slice(st["starts"][i] + r, st["starts"][i] + r + m)
            x = st["q"][part].float().view(m, c["hkv"], g * d).transpose(0, 1).reshape(c["hkv"], m * g, d)
            s = (torch.matmul(x, kt) * st["scale"]).view(c["hkv"], m, g, k - lo)
            if c["causal"]:
                hide = at > pos
                if w:
                    hide = hide | (at <= pos - w)
                s = s.masked_fill(hide, -math.inf)
            o, lse = _softmax_rows(s.view(c["hkv"], m * g, k - lo), vt)
            o = o.view(c["hkv"], m, g * d).transpose(0, 1).reshape(m, c["hq"], d)
            st["out"][part] = o.to(st["out"].dtype)
            st["lse"][part] = lse.view(c["hkv"], m, g).transpose(0, 1).reshape(m, c["hq"])


# ---------------------------------------------------------------- from the definition, 64 bits

def exact(c, seed):
    global own
    if c["op"] == "assign":
        return None  # whole numbers: they have to be equal
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    return _exact_append(c, st) if c["op"] == "append" else _exact_attend(c, st)


def _grid(x):
    """The e4m3 number next to x (64 bits, |x| <= 464), ties to the even one."""
    step = torch.exp2(torch.frexp(x.abs())[1].clamp(min=-5).double() - 4)
    return torch.round(x / step) * step


def _exact_append(c, st):
    p, b, h, d, r = c["page"], c["block"], c["hkv"], c["d"], c["rope"]
    n = st["starts"][-1]
    if sum(_pages(q, b) + 1 for q in st["qs"]) > 6000:
        return None

    def turn(x, w):
        y = x[:n].double()
        if w is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        if r:
            t = st["rope"][st["pos"][:n]].double()
            y = y.clone()
            for i in range(r // 2):
                lo, hi = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
                co, si = t[:, None, i], t[:, None, r // 2 + i]
                ya, yb = y[..., lo].clone(), y[..., hi].clone()
                y[..., lo], y[..., hi] = ya * co - yb * si, yb * co + ya * si
        return y
    out = {"k_exp": None, "v_exp": None}
    table = st["table"].tolist()
    for name, new in (("k", turn(st["nk"], st["kn"])), ("v", st["nv"][:n].double())):
        val = st[name].double()
        exps = st[name + "e"].double() - 127
        for s, (q, k) in enumerate(zip(st["qs"], st["ks"])):
            j = k - q
            while j < k:  # block by block
                base, end = j // b * b, min(k, j // b * b + b)
                page, place = table[s][base // p], base % p
                x = new[st["starts"][s] + j - (k - q):st["starts"][s] + end - (k - q)]
                big = x.abs().amax((0, 2))
                e = torch.ceil(torch.log2(big / 448)).clamp(min=-126)
                e = torch.where(big > 448 * torch.exp2(e), e + 1, torch.where(big <= 224 * torch.exp2(e), e - 1, e))
                old = exps[page, place // b]
                if j > base:
                    e = torch.maximum(e, old)
                    shift = torch.exp2(old - e)[None, :, None]
                    val[page, place:place + j - base] = _grid(val[page, place:place + j - base] * shift)
                val[page, place + j - base:place + end - base] = _grid(x * torch.exp2(-e)[None, :, None])
                j = end
        out[name] = val
    if c["hq"]:
        q = st["q_out"].double()
        q[:n] = turn(st["q"], st["qn"])
        out["q"] = q
    return out


def _exact_attend(c, st):
    p, b, g, d = c["page"], c["block"], c["hq"] // c["hkv"], c["d"]
    out, lse = st["out"].double(), st["lse"].double()
    for i in range(len(st["qs"])):
        q, k = st["qs"][i], st["ks"][i]
        if q == 0:
            continue
        tok = torch.arange(k, device="cuda")
        row = st["table"][i].long()[tok // p] * p + tok % p
        for h in range(c["hkv"]):
            kk, vv = (x.view(-1, c["hkv"], d).view(torch.uint8)[row, h].view(E4M3).double() *
                      torch.exp2(e.view(-1, c["hkv"])[row // b, h].double() - 127)[:, None]
                      for x, e in ((st["k"], st["ke"]), (st["v"], st["ve"])))
            step = max(1, 200_000_000 // (k * g))
            for lo in range(0, q, step):
                hi = min(q, lo + step)
                at = slice(st["starts"][i] + lo, st["starts"][i] + hi)
                x = st["q"][at, h * g:(h + 1) * g].double().reshape(-1, d)
                s = (x @ kk.t().contiguous()) * st["scale"]
                if c["causal"]:
                    far = (torch.arange(k - q + lo, k - q + hi, device="cuda").repeat_interleave(g)[:, None]
                           - tok[None])
                    s[far < 0] = -math.inf
                    if c["window"]:
                        s[far >= c["window"]] = -math.inf
                z = torch.logsumexp(s, 1)
                o = torch.exp(s - z[:, None]) @ vv
                out[at, h * g:(h + 1) * g] = o.view(hi - lo, g, d)
                lse[at, h * g:(h + 1) * g] = z.view(hi - lo, g)
    return {"out": out, "lse": lse}
