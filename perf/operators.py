"""The paged K/V operators (host_transfer_amd.kv) as cases to measure.

Four operators: `append` (norm + rotation of new queries and keys, and their placement in a
paged cache), `bounds` (per-page key bounds), `attend` (a chunk of new tokens, or single tokens,
over a paged cache) and `sparse` (pages selected for each query by their bounds, then attention
over the selected pages).  Where `own` is false, `run` computes them in elementary torch
operations in 32 bits (page scores, whose order decides which pages are read, in 64).
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _kv():
    from host_transfer_amd import kv
    return kv


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step
        dict(name="append_one_token", op="append", dtype="bf16", hq=32, hkv=8, d=128, n=1, page=16,
             rope=128, inter=False, norm=True, skip=0),
        # one decode token of the 20 sequences of the OPT-13B K/V shape (no rotation there)
        dict(name="append_kv_opt13b", op="append", dtype="f16", hq=0, hkv=40, d=128, n=20, page=16,
             rope=0, inter=False, norm=False, skip=0),
        # a prompt batch, padded: norms and rotation of queries and keys for every head
        dict(name="append_prompt", op="append", dtype="bf16", hq=32, hkv=8, d=128, n=16000, page=64,
             rope=128, inter=False, norm=True, skip=7),
        # the pages that one decode token of 64 sequences touches
        dict(name="bounds_decode", op="bounds", dtype="bf16", hkv=8, d=128, page=16, seqs=64, q=1,
             kv=700, spread=90),
        # every page of four prompts
        dict(name="bounds_prompt", op="bounds", dtype="f16", hkv=8, d=128, page=32, seqs=4, q=16384,
             kv=16384, spread=40),
        # a short conversation, one token: latency
        dict(name="attend_short", op="attend", dtype="bf16", hq=16, hkv=2, d=64, page=16, seqs=1, q=1,
             kv=37, spread=0, window=0, causal=True, empty=False),
        # one decode token of the OPT-13B K/V shape: 20 sequences of 1,920 + 128 tokens
        dict(name="attend_kv_opt13b", op="attend", dtype="f16", hq=40, hkv=40, d=128, page=16, seqs=20,
             q=1, kv=2048, spread=6, window=0, causal=True, empty=False),
        # one decode token over long contexts, queries in groups
        dict(name="attend_long", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=64, seqs=4, q=1,
             kv=131072, spread=50, window=0, causal=True, empty=False),
        # chunks of prompts that are prefilled piece by piece, ragged
        dict(name="attend_chunk", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=6,
             q=511, kv=9001, spread=70, window=0, causal=True, empty=True),
        # one whole prompt
        dict(name="attend_prompt", op="attend", dtype="bf16", hq=32, hkv=8, d=128, page=64, seqs=1,
             q=16384, kv=16384, spread=0, window=0, causal=True, empty=False),
        # one decode token over long contexts, 128 pages of 16 tokens each
        dict(name="sparse_decode", op="sparse", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=8, q=1,
             kv=65536, spread=50, first=1, last=4, select=128),
        # a chunk whose queries each select their own pages
        dict(name="sparse_chunk", op="sparse", dtype="f16", hq=32, hkv=8, d=128, page=32, seqs=2, q=200,
             kv=20011, spread=60, first=1, last=2, select=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "bounds", "attend", "attend", "sparse"])
    d = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 5, 8, 8, 40])
    if hkv * d > 8192:
        hkv = 8
    group = rng.choice([1, 2, 3, 4, 8])
    if hkv * group > 64:
        group = 1
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), d=d, hkv=hkv,
             page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]))
    width = hkv * d
    if op == "append":
        c.update(hq=rng.choice([0, hkv * group]), n=_log(rng, 1, 16000 * 1024 // width // max(1, group // 2) + 1),
                 rope=rng.choice([0, d, d, 32]), inter=rng.random() < 0.5, norm=rng.random() < 0.5,
                 skip=rng.choice([0, 0, 3, 10]))
        return c
    if op == "bounds":
        c["page"] = max(c["page"], 8)
        c["seqs"] = _log(rng, 1, 64)
        room = 60_000_000 // width // c["seqs"]
        c["kv"] = _log(rng, 1, max(2, min(65536, room)))
        c["q"] = min(c["kv"], _log(rng, 1, 16384))
        c["spread"] = rng.randrange(0, 100)
        return c
    c["hq"] = hkv * group
    c["spread"] = rng.randrange(0, 100)
    if op == "attend":
        if rng.random() < 0.5:
            c["q"], c["seqs"] = rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 64)
        else:
            c["q"], c["seqs"] = _log(rng, 5, 4096), _log(rng, 1, 8)
        room = 250_000_000 // width // c["seqs"]
        work = int(4e8 // (c["q"] * c["seqs"] * c["hq"] * d / 1000))
        c["kv"] = _log(rng, 1, max(2, min(131072, room, work)))
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        c["causal"] = bool(c["window"]) or rng.random() < 0.85
        c["empty"] = rng.random() < 0.3
        return c
    c["page"] = max(c["page"], 8)
    c["q"] = rng.choice([1, 1, 1, _log(rng, 2, 200)])
    c["seqs"] = _log(rng, 1, 32) if c["q"] == 1 else _log(rng, 1, 3)
    room = 120_000_000 // width // c["seqs"]
    if c["q"] > 1:
        room = min(room, 24000)
    c["kv"] = _log(rng, 2, max(4, min(100_000, room)))
    c["select"] = _log(rng, 4, max(5, min(160, 4096 // c["page"])))
    c["first"] = rng.choice([0, 1])
    c["last"] = rng.choice([1, 2])
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


def _visible(c, causal=True, window=0):
    """(query, key) pairs that are attended."""
    n = 0
    for q, k in zip(*_lens(c)):
        if not causal:
            n += q * k
        elif window:
            n += sum(min(window, p + 1) for p in range(k - q, k))
        else:
            n += q * k - q * (q - 1) // 2
    return n


def work(c):
    d, hkv, hq = c["d"], c["hkv"], c.get("hq", 0)
    if c["op"] == "append":
        row = 2 * (hq + 2 * hkv) * d
        n = c["n"]
        rot = n * (hq + hkv) * (3 * c["rope"] + (4 * d if c["norm"] else 0))
        return dict(bytes=n * (2 * row + 4 * c["rope"] + (16 if c["rope"] else 8)), flops=rot)
    qs, ks = _lens(c)
    if c["op"] == "bounds":
        p = c["page"]
        toks = pages = 0
        for q, k in zip(qs, ks):
            lo = (k - q) // p
            toks += k - lo * p
            pages += -(-k // p) - lo
        return dict(bytes=toks * hkv * d * 2 + pages * (hkv * d * 4 + 4), flops=2 * toks * hkv * d)
    nq = sum(qs)
    io = 2 * nq * hq * d * 2 + 4 * nq * hq
    if c["op"] == "attend":
        w, pairs = c["window"], _visible(c, c["causal"], c["window"])
        keys = sum(min(k, q + w - 1) if w and q else (k if q else 0) for q, k in zip(qs, ks))
        return dict(bytes=io + keys * hkv * d * 4 + 4 * sum(-(-k // c["page"]) for k in ks),
                    flops=4 * pairs * hq * d)
    p, scored, read, keys = c["page"], 0, 0, 0
    for q, k in zip(qs, ks):
        n_pages = -(-k // p)
        some = 0
        for pos in range(k - q, k):
            have = pos // p + 1
            keys += min(pos + 1, c["select"] * p)
            if have > c["select"]:
                some += have - min(have, c["first"] + c["last"])
        scored += some
        # the bounds are read once; of the keys, what one query selects is read at the least
        read += (n_pages * hkv * d * 4 if some else 0) + min(k, c["select"] * p) * hkv * d * 4
    return dict(bytes=io + read + 4 * nq * hkv * c["select"], flops=hq * d * (4 * scored + 4 * keys))


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


def _scales(g, h, d):
    """Channel scales of a K/V row: log-uniform in [0.1, 4] (as the K/V workload's)."""
    u = torch.rand((h, d), generator=g, device="cuda")
    return torch.exp(math.log(0.1) + u * math.log(40.0))


def _pool(g, c, n_pages):
    """A page pool of K/V rows, filled in pieces (its 32-bit form is not held whole)."""
    shape = (n_pages, c["page"], c["hkv"], c["d"])
    pool = torch.empty(shape, dtype=DT[c["dtype"]], device="cuda")
    s = _scales(g, c["hkv"], c["d"])
    step = max(1, 50_000_000 // (c["page"] * c["hkv"] * c["d"]))
    for i in range(0, n_pages, step):
        x = pool[i:i + step]
        x.copy_(_normal(g, x.shape, x.dtype, s))
    return pool


def _rope_table(n_pos, r):
    """Row p: r/2 cosines, then r/2 sines, of p * 10000^(-2i/r) (angles in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(c, seed):
    g = _gen(seed)
    dt, d, hkv, p = DT[c["dtype"]], c["d"], c["hkv"], c["page"]
    hq = c.get("hq", 0)
    st = {"c": c}
    if c["op"] == "append":
        n = c["n"]
        n_pages = -(-n // p) + 3
        # the rows of one fused projection: queries, keys and values of a token side by side
        qkv = _normal(g, (n, hq + 2 * hkv, d), dt)
        st["q"] = qkv[:, :hq] if hq else None
        st["k"], st["v"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["kp"], st["vp"] = _pool(g, c, n_pages), _pool(g, c, n_pages)
        st["q_out"] = torch.zeros((n, hq, d), dtype=dt, device="cuda") if hq else None
        order = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        slots = order[t // p] * p + t % p
        if c["skip"]:  # rows that pad the batch have no place
            slots = torch.where(t % c["skip"] == c["skip"] - 1, torch.full_like(slots, -1), slots)
        st["slots"] = slots
        st["pos"] = st["rope"] = None
        if c["rope"]:
            n_pos = max(2048, n)
            st["rope"] = _rope_table(n_pos, c["rope"])
            st["pos"] = (t + int(torch.randint(0, n_pos, (1,), generator=g, device="cuda"))) % n_pos
        st["qn"] = st["kn"] = None
        if c["norm"]:
            st["qn"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if hq else None
            st["kn"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        if own:
            st["cache"] = _kv().Cache(st["kp"], st["vp"])
        return st
    qs, ks = _lens(c)
    need = [-(-k // p) for k in ks]
    n_pages = sum(need) + 2
    st["kp"] = _pool(g, c, n_pages)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(ks), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    starts = [0]
    for q in qs:
        starts.append(starts[-1] + q)
    st["starts"], st["qs"], st["ks"] = starts, qs, ks
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(ks, dtype=torch.int32, device="cuda")
    st["table"] = table
    nq = starts[-1]
    st["scale"] = 1.0 / math.sqrt(d)
    if c["op"] != "bounds":
        st["vp"] = _pool(g, c, n_pages)
        st["q"] = _normal(g, (nq, hq + 2 * hkv, d), dt)[:, :hq]  # the queries of a fused projection
        st["out"] = torch.zeros((nq, hq, d), dtype=dt, device="cuda")
        st["lse"] = torch.zeros((nq, hq), dtype=torch.float32, device="cuda")
    else:
        st["vp"] = st["kp"]
    if c["op"] == "bounds":
        st["bounds"] = torch.zeros((n_pages, hkv, 2, d), dtype=dt, device="cuda")
    if c["op"] == "sparse":
        st["bounds"] = torch.stack([st["kp"].amin(1), st["kp"].amax(1)], 2).contiguous()
        for i, k in enumerate(ks):  # the last page of a sequence is bounded over the tokens it has
            if k % p:
                last = st["kp"][table[i, k // p].long(), :k % p]
                st["bounds"][table[i, k // p].long()] = torch.stack([last.amin(0), last.amax(0)], 1)
        st["sel"] = torch.full((nq, hkv, c["select"]), -1, dtype=torch.int32, device="cuda")
    if own:
        kv = _kv()
        st["cache"] = kv.Cache(st["kp"], st["vp"])
        st["batch"] = kv.Batch(st["q_start"], st["kv_len"], table, max_q=max(qs), max_kv=max(ks))
        nbytes = 0
        if c["op"] == "attend":
            nbytes = kv.attend_workspace(st["cache"], st["batch"], nq, hq)
        elif c["op"] == "sparse":
            nbytes = max(kv.select_workspace(st["cache"], st["batch"], nq, c["select"]),
                         kv.attend_selected_workspace(st["cache"], st["batch"], nq, hq, c["select"]))
        st["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- the operators

def run(st):
    c = st["c"]
    if own:
        kv = _kv()
        if c["op"] == "append":
            kv.append(st["cache"], st["k"], st["v"], st["slots"], q=st["q"], q_out=st["q_out"],
                      positions=st["pos"], rope=st["rope"],
                      flags=kv.ROPE_INTERLEAVED if c["inter"] and c["rope"] else 0,
                      q_norm=st["qn"], k_norm=st["kn"], eps=1e-6)
            return _append_out(st)
        if c["op"] == "bounds":
            kv.page_bounds(st["cache"], st["batch"], st["bounds"])
            return st["bounds"]
        if c["op"] == "attend":
            kv.attend(st["cache"], st["batch"], st["q"], st["out"], st["scale"], window=c["window"],
                      flags=kv.CAUSAL if c["causal"] else 0, lse=st["lse"], workspace=st["ws"])
            return {"out": st["out"], "lse": st["lse"]}
        kv.select(st["cache"], st["batch"], st["bounds"], st["q"], st["sel"], n_first=c["first"],
                  n_last=c["last"], workspace=st["ws"])
        kv.attend_selected(st["cache"], st["batch"], st["q"], st["sel"], st["out"], st["scale"],
                           lse=st["lse"], workspace=st["ws"])
        return {"sel": st["sel"], "out": st["out"], "lse": st["lse"]}
    return {"append": _append, "bounds": _bounds, "attend": _attend, "sparse": _sparse}[c["op"]](st)


def _append_out(st):
    out = {"k": st["kp"], "v": st["vp"]}
    if st["q"] is not None:
        out["q"] = st["q_out"]
    return out


def _norm_rotate(st, x, w):
    """x (n, heads, d) in 32 bits: each head's norm, then the rotation of its first channels."""
    c = st["c"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    r = c["rope"]
    if r:
        cs = st["rope"][st["pos"]][:, None, :]
        co, si = cs[..., :r // 2], cs[..., r // 2:]
        if c["inter"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat([a * co - b * si, b * co + a * si], -1)
        y = torch.cat([z, y[..., r:]], -1)
    return y.to(x.dtype)


def _append(st):
    c = st["c"]
    have = (st["slots"] >= 0).nonzero()[:, 0]
    rows = st["slots"][have]
    st["kp"].view(-1, c["hkv"], c["d"])[rows] = _norm_rotate(st, st["k"], st["kn"])[have]
    st["vp"].view(-1, c["hkv"], c["d"])[rows] = st["v"][have]
    if st["q"] is not None:
        y = _norm_rotate(st, st["q"], st["qn"])
        st["q_out"].copy_(torch.where((st["slots"] >= 0)[:, None, None], y, torch.zeros_like(y)))
    return _append_out(st)


def _bounds(st):
    c = st["c"]
    p = c["page"]
    for i, (q, k) in enumerate(zip(st["qs"], st["ks"])):
        lo, hi = (k - q) // p, -(-k // p)
        ids = st["table"][i, lo:hi].long()
        x = st["kp"][ids].float()
        there = (torch.arange(lo * p, hi * p, device="cuda") < k).view(hi - lo, p, 1, 1)
        low = torch.where(there, x, math.inf).amin(1)
        high = torch.where(there, x, -math.inf).amax(1)
        st["bounds"][ids] = torch.stack([low, high], 2).to(st["bounds"].dtype)
    return st["bounds"]


def _keys(st, i, k, lo=0):
    """The key and value rows lo..k-1 of sequence i, in 32 bits: (tokens, heads, d) each."""
    p = st["c"]["page"]
    ids = st["table"][i, lo // p:-(-k // p)].long()
    off = lo - lo // p * p
    return [x[ids].flatten(0, 1)[off:off + k - lo].float() for x in (st["kp"], st["vp"])]


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
        rows = slice(st["starts"][i], st["starts"][i] + q)
        kt = ks.permute(1, 2, 0).contiguous()
        vt = vs.transpose(0, 1).contiguous()
        step = max(1, min(q, 800_000_000 // ((k - lo) * c["hq"])))
        for r in range(0, q, step):
            m = min(step, q - r)
            pos = torch.arange(k - q + r, k - q + r + m, device="cuda")[:, None, None]
            at = torch.arange(lo, k, device="cuda")
            part = slice(rows.start + r, rows.start + r + m)
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
    return {"out": st["out"], "lse": st["lse"]}


def _sparse(st):
    c = st["c"]
    hkv, d, p, n_sel = c["hkv"], c["d"], c["page"], c["select"]
    g = c["hq"] // hkv
    for i, (q, k) in enumerate(zip(st["qs"], st["ks"])):
        n_pages = -(-k // p)
        ids = st["table"][i, :n_pages].long()
        bd = st["bounds"][ids].double().permute(1, 2, 3, 0)  # head, low/high, d, page
        step = max(1, min(q, 100_000_000 // (n_pages * g * hkv),
                          300_000_000 // (hkv * n_sel * p * d)))
        for r in range(0, q, step):
            m = min(step, q - r)
            part = slice(st["starts"][i] + r, st["starts"][i] + r + m)
            pos = torch.arange(k - q + r, k - q + r + m, device="cuda")
            x = st["q"][part].view(m, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, m * g, d)
            x64 = x.double()
            # the largest value that a key within the page's bounds can have against a query
            s = torch.matmul(x64.clamp(min=0), bd[:, 1].contiguous())
            s = s + torch.matmul(x64.clamp(max=0), bd[:, 0].contiguous())
            s = s.view(hkv, m, g, n_pages).amax(2).transpose(0, 1)
            last = (pos // p)[:, None, None]
            pg = torch.arange(n_pages, device="cuda")[None, None]
            s = torch.where((pg < c["first"]) | (pg > last - c["last"]), torch.full_like(s, math.inf), s)
            s = torch.where(pg > last, torch.full_like(s, -math.inf), s)
            top = torch.sort(s, dim=-1, descending=True, stable=True)[1][..., :n_sel]
            top = torch.where(top > last, torch.full_like(top, n_pages), top).sort(-1)[0]
            top = torch.where(top >= n_pages, torch.full_like(top, -1), top)
            sel = torch.full((m, hkv, n_sel), -1, dtype=torch.int64, device="cuda")
            sel[..., :top.shape[-1]] = top
            st["sel"][part] = sel.int()
            at = sel[..., None] * p + torch.arange(p, device="cuda")
            hide = ((sel[..., None] < 0) | (at > pos[:, None, None, None])).flatten(2)
            phys = ids[sel.clamp(min=0)]
            head = torch.arange(hkv, device="cuda")[None, :, None]
            kk = st["kp"].permute(0, 2, 1, 3)[phys, head].flatten(2, 3).float()
            vv = st["vp"].permute(0, 2, 1, 3)[phys, head].flatten(2, 3).float()
            xs = st["q"][part].view(m, hkv, g, d).float()
            sc = torch.matmul(xs, kk.transpose(-1, -2).contiguous()) * st["scale"]
            o, lse = _softmax_rows(sc.masked_fill(hide[:, :, None], -math.inf), vv)
            st["out"][part] = o.reshape(m, c["hq"], d).to(st["out"].dtype)
            st["lse"][part] = lse.reshape(m, c["hq"])
    return {"sel": st["sel"], "out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------- from the definition, 64 bits

def exact(c, seed):
    global own
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    return {"append": _exact_append, "bounds": _exact_bounds, "attend": _exact_attend,
            "sparse": _exact_sparse}[c["op"]](c, st)


def _exact_append(c, st):
    n, r, d = c["n"], c["rope"], c["d"]
    keep = st["slots"] >= 0

    def turn(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        if not r:
            return y
        t = st["rope"][st["pos"]].double()
        y = y.clone()
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r // 2)
            co, si = t[:, None, i], t[:, None, r // 2 + i]
            ya, yb = y[..., a].clone(), y[..., b].clone()
            y[..., a], y[..., b] = ya * co - yb * si, yb * co + ya * si
        return y
    k, v = st["kp"].double().flatten(0, 1), st["vp"].double().flatten(0, 1)
    k.index_copy_(0, st["slots"][keep], turn(st["k"], st["kn"])[keep])
    v.index_copy_(0, st["slots"][keep], st["v"].double()[keep])
    out = {"k": k.view(st["kp"].shape), "v": v.view(st["vp"].shape)}
    if st["q"] is not None:
        out["q"] = turn(st["q"], st["qn"]) * keep[:, None, None]
    return out


def _exact_bounds(c, st):
    p = c["page"]
    out = st["bounds"].double()
    big = torch.finfo(torch.float64).max
    for i, (q, k) in enumerate(zip(st["qs"], st["ks"])):
        first, last = (k - q) // p, (k - 1) // p
        pages = st["table"][i, first:last + 1].long()
        x = st["kp"][pages].double()
        low, high = x.clone(), x
        tail = k - last * p
        low[-1, tail:], high = big, x.clone()
        high[-1, tail:] = -big
        out[pages, :, 0], out[pages, :, 1] = low.min(1).values, high.max(1).values
    return out


def _exact_attend(c, st):
    p, g, d = c["page"], c["hq"] // c["hkv"], c["d"]
    out, lse = st["out"].double(), st["lse"].double()
    for i in range(len(st["qs"])):
        q, k = st["qs"][i], st["ks"][i]
        if q == 0:
            continue
        tok = torch.arange(k, device="cuda")
        row = st["table"][i].long()[tok // p] * p + tok % p
        for h in range(c["hkv"]):
            kk = st["kp"].view(-1, c["hkv"], d)[row, h].double()
            vv = st["vp"].view(-1, c["hkv"], d)[row, h].double()
            step = max(1, 200_000_000 // (k * g))
            for a in range(0, q, step):
                b = min(q, a + step)
                at = slice(st["starts"][i] + a, st["starts"][i] + b)
                x = st["q"][at, h * g:(h + 1) * g].double().reshape(-1, d)
                s = (x @ kk.t().contiguous()) * st["scale"]
                if c["causal"]:
                    far = (torch.arange(k - q + a, k - q + b, device="cuda").repeat_interleave(g)[:, None]
                           - tok[None])
                    s[far < 0] = -math.inf
                    if c["window"]:
                        s[far >= c["window"]] = -math.inf
                z = torch.logsumexp(s, 1)
                o = torch.exp(s - z[:, None]) @ vv
                out[at, h * g:(h + 1) * g] = o.view(b - a, g, d)
                lse[at, h * g:(h + 1) * g] = z.view(b - a, g)
    return {"out": out, "lse": lse}


def _exact_sparse(c, st):
    p, hkv, d, n_sel = c["page"], c["hkv"], c["d"], c["select"]
    g = c["hq"] // hkv
    if sum(st["qs"]) * hkv > 6000:
        return None
    sel = torch.full_like(st["sel"], -1)
    out, lse = st["out"].double(), st["lse"].double()
    for i in range(len(st["qs"])):
        q, k = st["qs"][i], st["ks"][i]
        ids = st["table"][i].long()
        bd = st["bounds"][ids[:-(-k // p)]].double()
        for j in range(q):
            row, pos = st["starts"][i] + j, k - q + j
            own_page = pos // p
            x = st["q"][row].double().view(hkv, g, d)
            forced = sorted({a for a in range(own_page + 1)
                             if a < c["first"] or a > own_page - c["last"]})
            free = max(0, min(n_sel, own_page + 1) - len(forced))
            lo, hi = c["first"], own_page - c["last"] + 1
            for h in range(hkv):
                pick = torch.tensor(forced, device="cuda")
                if free:
                    b = bd[lo:hi, h]
                    val = torch.maximum(x[h][:, None] * b[:, 0], x[h][:, None] * b[:, 1]).sum(-1).amax(0)
                    best = torch.sort(val, descending=True, stable=True).indices[:free] + lo
                    pick = torch.cat([pick, best]).sort().values
                sel[row, h, :len(pick)] = pick.int()
                tok = (pick[:, None] * p + torch.arange(p, device="cuda")).flatten()
                tok = tok[tok <= pos]
                at = ids[tok // p] * p + tok % p
                kk = st["kp"].view(-1, hkv, d)[at, h].double()
                vv = st["vp"].view(-1, hkv, d)[at, h].double()
                s = (x[h] @ kk.t().contiguous()) * st["scale"]
                z = torch.logsumexp(s, 1)
                out[row, h * g:(h + 1) * g] = torch.exp(s - z[:, None]) @ vv
                lse[row, h * g:(h + 1) * g] = z
    return {"sel": sel, "out": out, "lse": lse}
