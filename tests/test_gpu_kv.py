"""The paged K/V operators on the GPU against plain 64-bit computations
(tests/kv_case.py): placement with norm and rotation, page bounds, attention
over the cache, page selection and attention over the selected pages, at the
sizes, strides and masks where they can go wrong."""
import math

import pytest
import torch

from host_transfer_amd import kv
from tests import kv_case as K

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
PAD = -4.25  # what rows and pages that a call must leave alone hold


def log(msg):
    print("[kv] " + msg, flush=True)


def ws(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")


def gpu_batch(c, max_q=None, max_kv=None):
    return kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda(),
                    c.max_q if max_q is None else max_q, c.max_kv if max_kv is None else max_kv)


def run_attend(c, scale, causal=True, window=0, sel=None, max_q=None, max_kv=None):
    k, v = c.pools()
    cache, batch = kv.Cache(k, v), gpu_batch(c, max_q, max_kv)
    hq = c.h * c.group
    q = c.wide_q.cuda()[:, :hq]
    out = torch.full((c.n, hq + 1, c.d), PAD, dtype=c.dtype, device="cuda")
    lse = torch.full((c.n, hq), PAD, device="cuda")
    if sel is None:
        w = ws(kv.attend_workspace(cache, batch, c.n, hq))
        kv.attend(cache, batch, q, out[:, :hq], scale, window=window,
                  flags=kv.CAUSAL if causal else 0, lse=lse, workspace=w)
    else:
        w = ws(kv.attend_selected_workspace(cache, batch, c.n, hq, sel.shape[2]))
        kv.attend_selected(cache, batch, q, sel.cuda(), out[:, :hq], scale, lse=lse, workspace=w)
    torch.cuda.synchronize()
    assert (out[:, hq] == PAD).all(), "wrote past the heads of out"
    return out[:, :hq], lse


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,rope,inter,norm", [
    (8, 0, False, False), (16, 16, False, True), (64, 64, False, True), (64, 32, True, True),
    (80, 80, False, False), (80, 48, True, True), (96, 96, False, True), (128, 128, False, True),
    (128, 128, True, False), (128, 32, False, True), (136, 0, False, True), (192, 192, False, True),
    (256, 256, False, True), (256, 128, True, True)])
def test_append(dtype, d, rope, inter, norm):
    for n, hq, h, page, head_major in ((1, 3, 1, 16, False), (37, 4, 2, 24, True), (70, 0, 5, 1, False)):
        g = torch.Generator().manual_seed(n + d)
        n_pages = -(-n // page) + 2
        log(f"append {dtype} d={d} rope={rope} inter={inter} norm={norm} n={n} hq={hq} page={page}")
        qkv = torch.randn((n, hq + 2 * h, d), generator=g).to(dtype)
        slots = torch.randperm(n_pages * page, generator=g)[:n]
        pos = torch.randint(0, 50, (n,), generator=g)
        if n > 5:  # tokens that are not placed: padding, past the pool, past the table
            slots[1], slots[2], slots[3] = -1, n_pages * page, 1 << 40
            if rope:
                pos[4], pos[5] = 50, -1
        placed = (slots >= 0) & (slots < n_pages * page)
        if rope:
            placed &= (pos >= 0) & (pos < 50)
        table = K.rope_table(50, rope) if rope else None
        qn = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None
        kn = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None
        pools = [torch.full((n_pages, page, h, d), PAD, dtype=dtype, device="cuda") for _ in "kv"]
        if head_major:
            pools = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in pools]
        gpu = qkv.cuda()
        q_out = torch.full((n, hq, d), PAD, dtype=dtype, device="cuda") if hq else None
        dev = lambda t: None if t is None else t.cuda()
        kv.append(kv.Cache(*pools), gpu[:, hq:hq + h], gpu[:, hq + h:], slots.cuda(),
                  q=gpu[:, :hq] if hq else None, q_out=q_out, positions=dev(pos) if rope else None,
                  rope=dev(table), flags=kv.ROPE_INTERLEAVED if inter else 0, q_norm=dev(qn),
                  k_norm=dev(kn), eps=1e-5)
        torch.cuda.synchronize()
        safe = pos.clamp(0, 49)
        want = [K.norm_rotate(qkv[:, a:b].double(), safe, table, inter, w, 1e-5)
                for a, b, w in ((0, hq, qn), (hq, hq + h, kn))]
        u = K.half_step(dtype)
        # fp32: the sum of d squares, the root, three products, the rotation's two products and sum
        rel = u + (d + 16) * K.U32
        tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
        rows_k, rows_v = (x.cpu().reshape(-1, h, d) for x in pools)
        # the rotation's output is bounded by the pair's length, not by itself
        length = lambda x: x.abs().amax(-1, keepdim=True) * (2 if rope else 0) * 16 * K.U32
        err = (rows_k[slots[placed]].double() - want[1][placed]).abs()
        assert (err <= rel * want[1][placed].abs() + length(want[1][placed]) + tiny).all()
        assert torch.equal(rows_v[slots[placed]], qkv[placed, hq + h:])
        left = torch.ones(n_pages * page, dtype=torch.bool)
        left[slots[placed]] = False
        assert (rows_k[left] == PAD).all() and (rows_v[left] == PAD).all(), "touched other rows"
        if not norm and not rope:
            assert torch.equal(rows_k[slots[placed]], qkv[placed, hq:hq + h])
        if hq:
            got = q_out.cpu()
            assert (got[~placed] == 0).all()
            err = (got[placed].double() - want[0][placed]).abs()
            assert (err <= rel * want[0][placed].abs() + length(want[0][placed]) + tiny).all()


def test_append_in_place_and_broadcast():
    """q_out = q; one key row for all tokens (stride 0); a strided page pool (K and V side by side)."""
    n, hq, h, d, page = 19, 6, 3, 64, 8
    g = torch.Generator().manual_seed(1)
    q = torch.randn((n, hq, d), generator=g).to(BF16)
    k = torch.randn((1, h, d), generator=g).to(BF16)
    pool = torch.full((4, 2, page, h, d), PAD, dtype=BF16, device="cuda")
    table = K.rope_table(32, d)
    pos = torch.arange(n)
    slots = torch.arange(n) + 3
    gq, gk = q.cuda(), k.cuda().expand(n, h, d)
    log("append in place")
    kv.append(kv.Cache(pool[:, 0], pool[:, 1]), gk, gk, slots.cuda(), q=gq, q_out=gq,
              positions=pos.cuda(), rope=table.cuda())
    torch.cuda.synchronize()
    want = K.norm_rotate(q.double(), pos, table, False, None, 0)
    lim = K.half_step(BF16) * want.abs() + 32 * K.U32 * want.abs().amax(-1, keepdim=True)
    assert ((gq.cpu().double() - want).abs() <= lim).all()
    wk = K.norm_rotate(k.double().expand(n, h, d), pos, table, False, None, 0)
    rows = pool[:, 0].cpu().reshape(-1, h, d)
    lim = K.half_step(BF16) * wk.abs() + 32 * K.U32 * wk.abs().amax(-1, keepdim=True)
    assert ((rows[slots].double() - wk).abs() <= lim).all()
    assert (rows[:3] == PAD).all() and (rows[n + 3:] == PAD).all()
    assert torch.equal(pool[:, 1].cpu().reshape(-1, h, d)[slots], k.expand(n, h, d))


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,page", [(8, 1, 1), (64, 3, 16), (80, 2, 24), (128, 8, 64), (256, 1, 7)])
def test_page_bounds(dtype, d, h, page):
    lens = [(1, 1), (0, 40), (5, 5), (3, page * 2 + 1), (40, 129), (1, page * 3), (2, 0), (1, 2 * page)]
    c = K.Case(lens, dtype=dtype, h=h, group=1, d=d, page=page, fill=math.nan)
    c.k[int(c.table[7, 1]), min(1, page - 1), 0, 2] = math.nan
    c.k[int(c.table[5, 2]), 0, 0, 1] = math.inf
    c.table[0, 0] = c.n_pages  # a page that is not there
    log(f"bounds {dtype} d={d} h={h} page={page}")
    k, v = c.pools()
    bounds = torch.full((c.n_pages, h, 2, d), PAD, dtype=dtype, device="cuda")
    kv.page_bounds(kv.Cache(k, v), gpu_batch(c), bounds)
    torch.cuda.synchronize()
    got = bounds.cpu()
    want = K.page_bounds(c)
    for i in range(c.n_pages):
        if i in want:
            for side in (0, 1):
                a, b = got[i, :, side], want[i][side]
                assert ((a == b) | (torch.isnan(a) & torch.isnan(b))).all(), (i, side)
        else:
            assert (got[i] == PAD).all(), "touched another page"


# ---------------------------------------------------------------- attention

LENS = [(1, 1), (3, 3), (0, 0), (17, 64), (1, 65), (2, 200), (0, 31), (130, 300), (66, 66)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,group,page", [(8, 1, 1, 16), (40, 2, 3, 8), (64, 2, 4, 16), (80, 1, 2, 24),
                                            (96, 2, 1, 1), (128, 2, 8, 16), (128, 1, 5, 64),
                                            (136, 1, 2, 16), (192, 2, 2, 32), (256, 1, 20, 16)])
def test_attend(dtype, d, h, group, page):
    c = K.Case(LENS, dtype=dtype, h=h, group=group, d=d, page=page, fill=math.nan, tail_rows=3,
               head_major=page == 16)
    scale = 1 / math.sqrt(d)
    for causal, window in ((True, 0), (True, 1), (True, 50), (False, 0)):
        log(f"attend {dtype} d={d} h={h} group={group} page={page} causal={causal} window={window}")
        out, lse = run_attend(c, scale, causal, window)
        K.check_attention(c, out, lse, K.attention(c, scale, causal=causal, window=window),
                          f"causal={causal} window={window}")
        assert (out[c.n - 3:] == PAD).all() and (lse[c.n - 3:] == PAD).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,group,page", [(64, 2, 1, 16), (80, 1, 4, 24), (96, 2, 2, 16),
                                            (128, 2, 4, 16), (128, 1, 16, 1), (192, 1, 17, 64),
                                            (256, 1, 3, 32)])
def test_attend_single_tokens(dtype, d, h, group, page):
    """One new token a sequence, from one key to several splits of the keys."""
    lens = [(1, n) for n in (1, 2, 15, 16, 17, 31, 64, 65, 127, 257, 1000, 2049)] + [(0, 0), (1, 700)]
    c = K.Case(lens, dtype=dtype, h=h, group=group, d=d, page=page, fill=math.nan, tail_rows=1)
    scale = 0.7 / math.sqrt(d)
    for causal, window, max_kv in ((True, 0, None), (True, 33, None), (False, 0, None),
                                   (True, 0, 20000)):
        if max_kv:
            c.table = torch.cat([c.table, torch.full((len(lens), 20000 // page + 1), 1 << 30,
                                                     dtype=torch.int32)], 1)
        log(f"single tokens {dtype} d={d} group={group} page={page} window={window} max_kv={max_kv}")
        out, lse = run_attend(c, scale, causal, window, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, scale, causal=causal, window=window))
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()


@pytest.mark.parametrize("q", [1, 2, 5, 40, 200])
def test_attend_bad_pages_and_lengths(q):
    """Pages that are not there (ids of every wrong kind), lengths past the bounds given, rows
    at positions before the first token."""
    lens = [(q, 400), (q, 170), (q, q - 1 if q < 3 else q // 2), (q, 250)]
    c = K.Case(lens, d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    for s, p, bad in ((0, 0, -1), (0, 7, c.n_pages), (0, 24, 1 << 30), (1, 3, -(1 << 31)),
                      (3, 15, -5), (3, 14, -5), (3, 13, c.n_pages + 7)):
        c.table[s, p] = bad
    log(f"bad pages q={q}")
    out, lse = run_attend(c, 0.125)
    K.check_attention(c, out, lse, K.attention(c, 0.125), f"q={q}")
    # a sequence whose pages are all missing
    c.table[0] = -1
    out, lse = run_attend(c, 0.125)
    K.check_attention(c, out, lse, K.attention(c, 0.125), f"q={q}: no page")
    # tokens past max_kv are not read, new tokens past max_q are left as they were
    c = K.Case([(q, 400), (q, 170)], d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    out, lse = run_attend(c, 0.125, causal=False, max_kv=300)
    full = c.lens
    ref_c = K.Case([(q, 400), (q, 170)], d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    ref_c.table[0, 19:] = -1
    ref_c.table[0, 18] = c.table[0, 18]
    cut = ref_c.keys
    ref_c.keys = lambda s, upto=None: cut(s, 300)
    K.check_attention(c, out, lse, K.attention(ref_c, 0.125, causal=False), f"q={q}: max_kv")
    assert full == c.lens
    if q > 1:
        out, lse = run_attend(c, 0.125, max_q=q - 1)
        assert (out[q - 1] == PAD).all() and (out[2 * q - 1] == PAD).all()
        want = K.attention(c, 0.125)
        want[4][[q - 1, 2 * q - 1]] = False
        K.check_attention(c, out, lse, want, f"q={q}: max_q")


@pytest.mark.parametrize("q", [1, 3, 40, 150])
def test_attend_values_out_of_range(q):
    """NaN and infinite keys and values: a row that sees one carries it, another does not."""
    lens = [(q, 190), (q, 333)]
    for kind, val in (("v", math.nan), ("v", math.inf), ("v", -math.inf), ("k", math.nan)):
        c = K.Case(lens, dtype=BF16, d=64, h=2, group=2, page=16, seed=3)
        for s, (_, n) in enumerate(lens):
            for j, ch in ((n - 1, 5), (n - 1 - q // 2, 6), (n - q // 2 - 40, 7)):
                j = max(0, j)
                x = c.k if kind == "k" else c.v
                if kind == "k" and j < n - 1 - q // 2:
                    continue  # a NaN score for every row
                x[int(c.table[s, j // 16]), j % 16, 1, ch] = val
        log(f"out of range {kind}={val} q={q}")
        for window in (0, 20):
            out, lse = run_attend(c, 0.125, window=window)
            K.check_attention(c, out, lse, K.attention(c, 0.125, window=window), f"{kind}={val}")


def test_attend_large_scores():
    """Scores far apart (a softmax of one key), and all equal."""
    for dtype in (F16, BF16):
        for scale in (0.0, 30.0, -5.0):
            c = K.Case([(1, 300), (33, 140), (70, 500)], dtype=dtype, d=64, h=1, group=2, page=16)
            log(f"large scores {dtype} {scale}")
            out, lse = run_attend(c, scale)
            K.check_attention(c, out, lse, K.attention(c, scale), f"scale={scale}")
    # rising scores: every tile has a new maximum
    c = K.Case([(1, 700), (64, 700)], dtype=F16, d=64, h=1, group=1, page=16)
    c.q[:] = 1.0
    for s in range(2):
        for j in range(700):
            c.k[int(c.table[s, j // 16]), j % 16] = (j - 350) / 16.0
    log("rising scores")
    out, lse = run_attend(c, 0.25)
    K.check_attention(c, out, lse, K.attention(c, 0.25), "rising")


def n_splits(c, max_kv=None):
    """Into how many parts a call splits each row's keys: its workspace has head_dim + 2 floats of each."""
    k, v = c.pools()
    hq = c.h * c.group
    need = kv.attend_workspace(kv.Cache(k, v), gpu_batch(c, max_kv=max_kv), c.n, hq)
    return need // (c.n * hq * (c.d + 2) * 4)


@pytest.mark.parametrize("q_len,h,group", [(1, 1, 2), (1, 4, 3), (3, 2, 4), (2, 8, 1), (40, 1, 2), (70, 4, 1)])
def test_attend_values_out_of_range_in_any_split(q_len, h, group):
    """NaN and infinite values whose weight rounds to zero in 32 bits (scores 200 below the largest),
    in the largest score's split, in others and in masked places: the same result wherever the keys are
    split, and the formula's.  Few rows and chunks; without a split, few of them and many."""
    n, d, page = 1500, 16, 16
    for max_kv in (None, 9000, 90000):
        c = K.Case([(q_len, n), (q_len, 700)], dtype=BF16, d=d, h=h, group=group, page=page, seed=q_len)
        if max_kv:
            c.table = torch.cat([c.table, torch.full((2, max_kv // page + 1), -1, dtype=torch.int32)], 1)
        c.q[..., 0], c.k[..., 0] = 1.0, 0.0
        at = lambda s, j: (int(c.table[s, j // page]), j % page)
        for s, j in ((0, 777), (1, 3)):  # the largest scores: a value of 200 above the others
            c.k[at(s, j)][:, 0] = 200.0
        odd = {5: math.nan, 70: math.inf, 760: -math.inf, 780: math.inf, 1100: math.nan, n - 1: -math.inf,
               n - 2: math.nan, n - 30: math.inf, 698: math.inf}
        for i, (j, val) in enumerate(odd.items()):  # a channel each, and one that meets both infinities
            for s in range(2):
                if j < c.lens[s][1]:
                    c.v[at(s, j)][:, i + 1] = val
                    if val == math.inf or j == 760:
                        c.v[at(s, j)][:, 12] = val
        splits = n_splits(c, max_kv)
        log(f"out of range in {splits} splits, q={q_len} h={h} group={group}")
        assert max_kv is None or splits > (8 if max_kv == 90000 else 1)
        for causal, window in ((False, 0), (True, 0), (True, 500)):
            out, lse = run_attend(c, 1.0, causal, window, max_kv=max_kv)
            K.check_attention(c, out, lse, K.attention(c, 1.0, causal=causal, window=window),
                              f"{splits} splits, causal={causal} window={window}")
        if max_kv is None and q_len <= 3:
            sel = torch.arange(94, dtype=torch.int32).expand(c.n, h, 94).contiguous()
            out, lse = run_attend(c, 1.0, sel=sel)
            K.check_attention(c, out, lse, K.attention(c, 1.0, sel=sel), "lists")
    # no score above -inf: zeros, whatever the values
    c.q[..., 0], c.k[..., 0] = 1.0, -math.inf
    out, lse = run_attend(c, 1.0, False, max_kv=max_kv)
    assert (out == 0).all() and (lse == -math.inf).all()


def wider_table(c, max_kv):
    """The case's page table with room for max_kv tokens; the pages past its own are not there."""
    room = -(-max_kv // c.page)
    if c.table.shape[1] < room:
        more = torch.full((c.table.shape[0], room - c.table.shape[1]), -1, dtype=torch.int32)
        c.table = torch.cat([c.table, more], 1)


@pytest.mark.parametrize("dtype,d,h,group,page", [
    (BF16, 64, 2, 2, 16), (F16, 128, 1, 4, 24), (BF16, 128, 2, 1, 64), (F16, 96, 1, 2, 16),
    (BF16, 192, 1, 2, 16), (F16, 256, 1, 2, 32), (BF16, 40, 1, 4, 8)])
def test_attend_chunks_in_splits(dtype, d, h, group, page):
    """Chunks whose keys are split over workgroups, into few parts and into many: causal,
    windowed and open masks, sequences that have no keys in most of the splits, a split whose pages are
    all missing, rows behind the last sequence left as they were."""
    c = K.Case([(50, 1500), (0, 0), (33, 700), (24, 1100), (1, 64), (60, 60)], dtype=dtype, d=d, h=h,
               group=group, page=page, fill=math.nan, tail_rows=2, seed=d + group)
    c.table[3, 512 // page:-(-768 // page)] = -1
    c.table[0, 1200 // page] = c.n_pages
    wider_table(c, 40000)
    scale = 1 / math.sqrt(d)
    for causal, window in ((True, 0), (True, 1000), (False, 0)):
        ref = K.attention(c, scale, causal=causal, window=window)
        for max_kv, least in ((1500, 2), (4200, 3), (9000, 9), (40000, 40)):
            splits = n_splits(c, max_kv)
            log(f"chunks in {splits} splits {dtype} d={d} h={h} group={group} {causal} {window}")
            assert splits >= least
            out, lse = run_attend(c, scale, causal, window, max_kv=max_kv)
            K.check_attention(c, out, lse, ref, f"{splits} splits, causal={causal} window={window}")
            assert (out[c.n - 2:] == PAD).all() and (lse[c.n - 2:] == PAD).all()


@pytest.mark.parametrize("dtype,d,h,group,page", [
    (BF16, 64, 4, 2, 16), (F16, 128, 8, 1, 16), (BF16, 128, 4, 4, 24), (F16, 40, 4, 3, 8),
    (BF16, 192, 4, 2, 16), (F16, 256, 8, 2, 32), (BF16, 96, 12, 1, 1), (F16, 8, 4, 16, 64)])
def test_attend_few_rows_of_four_heads(dtype, d, h, group, page):
    """Caches whose heads are a multiple of four, one to four new tokens of a sequence: every mask,
    pages that are not there, rows before the first token, with and without splits of the keys."""
    most = min(4, 16 // group)
    lens = [(min(q, most), n) for q, n in ((1, 1), (4, 3), (0, 0), (2, 64), (1, 65), (3, 200), (0, 31),
                                           (4, 129), (1, 310), (2, 33))]
    c = K.Case(lens, dtype=dtype, d=d, h=h, group=group, page=page, fill=math.nan, tail_rows=2, seed=d)
    for s, j, bad in ((5, 40, -1), (5, 150, c.n_pages), (8, 300, 1 << 30), (7, 0, -(1 << 31))):
        c.table[s, j // page] = bad
    wider_table(c, 30000)
    scale = 1 / math.sqrt(d)
    for causal, window in ((True, 0), (True, 1), (True, 50), (False, 0)):
        ref = K.attention(c, scale, causal=causal, window=window)
        for max_kv in (60, 310, 5000, 30000) if (causal, window) == (True, 0) else (310, 30000):
            if max_kv == 60:  # tokens past it are not read
                small = K.Case([(q, min(n, 60)) for q, n in lens], dtype=dtype, d=d, h=h, group=group,
                               page=page, seed=d)
                small.k, small.v, small.q, small.table = c.k, c.v, c.q, c.table
                small.n, small.n_pages, small.wide_q, small.lens = c.n, c.n_pages, c.wide_q, lens
                keys = small.keys
                small.keys = lambda s, upto=None: keys(s, 60)
                want = K.attention(small, scale)
            else:
                want = ref
            log(f"four heads {dtype} d={d} h={h} group={group} {causal} {window} max_kv={max_kv}: "
                f"{n_splits(c, max_kv)} splits")
            out, lse = run_attend(c, scale, causal, window, max_kv=max_kv)
            K.check_attention(c, out, lse, want, f"causal={causal} window={window} max_kv={max_kv}")
            assert (out[c.n - 2:] == PAD).all() and (lse[c.n - 2:] == PAD).all()


@pytest.mark.parametrize("n_seqs", [2, 64, 65, 200])
def test_chunks_of_many_sequences(n_seqs):
    """Chunks in any order of lengths, equal ones and empty ones among them; row tiles of up to three
    to a sequence."""
    g = torch.Generator().manual_seed(n_seqs)
    kv_len = torch.randint(0, 130, (n_seqs,), generator=g)
    kv_len[:2] = torch.tensor([520, 520])
    if n_seqs > 2:
        kv_len[-1], kv_len[5] = 400, 0
    lens = [(min(int(x), int(torch.randint(0, 60, (), generator=g))), int(x)) for x in kv_len]
    lens[0], lens[1] = (260, 520), (17, 520)
    c = K.Case(lens, dtype=BF16, d=32, h=1, group=1, page=16, tail_rows=2)
    for window in (0, 50):
        log(f"chunks of {n_seqs} sequences, window {window}")
        out, lse = run_attend(c, 0.2, window=window)
        K.check_attention(c, out, lse, K.attention(c, 0.2, window=window), f"{n_seqs} sequences")
        assert (out[-2:] == PAD).all() and (lse[-2:] == PAD).all()


@pytest.mark.parametrize("dtype,d,page", [(BF16, 128, 16), (F16, 64, 64), (BF16, 80, 24), (F16, 256, 16)])
def test_chunk_first_keys_of_a_long_context(dtype, d, page):
    """The first 64 keys of a chunk's context have most of the weight, and their place in LDS is the
    first that later keys take.  200 sequences that share their pages and have the same queries, two
    workgroups or more to each CU: the same bits for every sequence and every call, and the
    formula's values."""
    q_len, n, copies = 70, 1300, 200
    c = K.Case([(q_len, n)], dtype=dtype, h=2, group=2, d=d, page=page, seed=d)
    for j in range(64):  # (their scores are twice as far apart as the others')
        c.k[int(c.table[0, j // page]), j % page] *= 2
    log(f"first keys {dtype} d={d} page={page}")
    k, v = c.pools()
    cache, hq = kv.Cache(k, v), 4
    start = torch.arange(copies + 1, dtype=torch.int32, device="cuda") * q_len
    batch = kv.Batch(start, c.kv_len.cuda().expand(copies).contiguous(),
                     c.table.cuda().expand(copies, -1).contiguous(), q_len, n)
    q = c.wide_q.cuda()[:, :hq].repeat(copies, 1, 1)
    w = ws(kv.attend_workspace(cache, batch, q.shape[0], hq))
    for rep in range(3):
        out = torch.full_like(q, PAD)
        lse = torch.full(q.shape[:2], PAD, device="cuda")
        kv.attend(cache, batch, q, out, 1 / math.sqrt(d), lse=lse, workspace=w)
        torch.cuda.synchronize()
        o, z = out.view(copies, q_len, hq, d), lse.view(copies, q_len, hq)
        if rep == 0:
            first = o[0].clone(), z[0].clone()
            K.check_attention(c, *first, K.attention(c, 1 / math.sqrt(d)), "first keys")
        assert (o == first[0]).all() and (z == first[1]).all(), rep


@pytest.mark.parametrize("q_len", [1, 40])
def test_attend_all_scores_minus_infinity(q_len):
    """A row that sees scores of -inf only is one that sees nothing; with one finite score that key
    has all the weight."""
    for finite in (None, 3):
        c = K.Case([(q_len, 60), (q_len, 900)], dtype=BF16, d=64, h=1, group=2, page=16)
        c.q[:, :, 0] = 1.0
        c.k[:, :, :, 0] = -math.inf
        if finite is not None:
            for s in range(2):
                c.k[int(c.table[s, 0]), finite, 0, 0] = 1.0
        log(f"scores of -inf, {q_len} rows, finite at {finite}")
        out, lse = run_attend(c, 0.125, causal=False)
        if finite is None:
            assert (out == 0).all() and (lse == -math.inf).all()
        else:
            for s in range(2):  # a weight of 1 times a value of the dtype: exact
                rows = slice(int(c.q_start[s]), int(c.q_start[s + 1]))
                v = c.v[int(c.table[s, 0]), finite, 0].cuda()
                assert torch.equal(out[rows], v.expand_as(out[rows]))
                assert torch.isfinite(lse[rows]).all()


@pytest.mark.parametrize("q_len", [1, 2, 40])
def test_attend_many_small_weights(q_len):
    """One large score and so many small ones that their sum counts, each below half of fp16's
    smallest step next to it: weights of e^-17.5 = 2^-25.2, 30,000 of them are 7.5e-4 of the sum."""
    n = 30000
    c = K.Case([(q_len, n)], dtype=F16, d=16, h=1, group=1, page=64)
    c.q[:] = 0.0
    c.q[:, 0, 0] = 1.0
    c.k[:], c.v[:] = 0.0, 1.0
    c.k[:, :, 0, 0] = -17.5
    for j in (0, n // 2):  # the large score first, or after many small ones
        first = c.k.clone()
        c.k[int(c.table[0, j // 64]), j % 64] = 0.0
        c.v[int(c.table[0, j // 64]), j % 64] = 0.0
        log(f"many small weights, {q_len} rows, large score at {j}")
        out, lse = run_attend(c, 1.0, causal=False)
        want = (n - 1) * math.exp(-17.5) / (1 + (n - 1) * math.exp(-17.5))
        # a weight off by half a step of fp16 and, of the exponent's 18 * log2(e), 2^-24 of it
        # eight times; the sums of equal terms by less than n of these; the output once
        tol = want * (2 ** -11 + 2 ** -11 + 8 * 26 * 2.0 ** -24 + n * 2.0 ** -24)
        assert (out.double() - want).abs().max() <= tol, (float(out.max()), want)
        c.k, c.v[:] = first, 1.0


@pytest.mark.parametrize("q_len", [1, 40])
def test_attend_fp16_huge_scores(q_len):
    """Scores up to 2^35: differences of scores are then far above 1 or exactly 0, so the row's
    result is the mean of the values of its largest score's keys."""
    for top in (600.0, 4000.0, 60000.0):
        c = K.Case([(q_len, 700)], dtype=F16, d=128, h=1, group=2, page=16)
        c.q[:] = 1.0
        c.q[:, 1] = top
        best = [5, 300, 301, 698]  # by an eighth above all others
        at = lambda j: (int(c.table[0, j // 16]), j % 16)
        c.k[:] = top * 7 / 8
        for j in best:
            c.k[at(j)] = top
        log(f"huge scores {top}, {q_len} rows")
        out, lse = run_attend(c, 0.7, causal=False)
        v = torch.stack([c.v[at(j)] for j in best]).double()[:, 0]
        # four equal weights y, of any size between two powers of two: the sum takes 4 y, the values
        # are multiplied by y rounded to fp16, y (1 + d) with |d| <= 2^-11, so the quotient
        # is the mean times 1 + d; it is rounded again, by 2^-11; sums of four and the quotient in fp32
        tol = 2 * 2 ** -11 * v.mean(0).abs() + 16 * 2.0 ** -24 * v.abs().mean(0) + 2.0 ** -25
        for h in range(2):
            assert ((out[:, h].cpu().double() - v.mean(0)).abs() <= tol).all(), (top, h)
            want = 0.7 * 128 * float(c.k.max()) * (1.0, top)[h] + math.log(4)
            assert ((lse[:, h].cpu().double() - want).abs() <= (128 + 16) * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("q_len,h", [(1, 1), (2, 4), (40, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attend_values_at_the_ends_of_the_type(dtype, q_len, h):
    """A mean of values is none above them: where all are fp16's largest, or in bf16 of a size whose
    sum over the keys 32 bits hold, the output is that and not an infinity; in splits too, and over
    lists."""
    n, page = 100, 16
    big = torch.finfo(F16).max if dtype == F16 else 2.0 ** 120
    u = K.half_step(dtype)
    for max_kv in (None, 9000):
        c = K.Case([(q_len, n), (q_len, 63)], dtype=dtype, d=16, h=h, group=2, page=page, seed=q_len)
        if max_kv:
            wider_table(c, max_kv)
        c.v[:] = big
        c.v[..., 3], c.v[..., 4] = -big, 0.0
        for kind in ("random", "rounded up", "rising"):
            if kind != "random":
                c.q[:], c.k[:] = 1.0, 0.0
            if kind == "rounded up":  # all weights but one just above half a step: they gain nearly all of it
                x = -math.log(2) + math.log1p(1.05 * u)
                c.k[..., 0] = torch.tensor(x, dtype=dtype)
                c.k[..., 1] = x - c.k[0, 0, 0, 0].double()
            for s, (_, kv_n) in enumerate(c.lens):
                for j in range(kv_n):
                    if kind == "rounded up" and j == 0:
                        c.k[int(c.table[s, 0]), 0] = 0.0
                    if kind == "rising" and j >= 64:  # 2^7.8 times the first keys' weights
                        c.k[int(c.table[s, j // page]), j % page, :, 0] = 7.8 * math.log(2)
            log(f"ends of the type {dtype} q={q_len} h={h} max_kv={max_kv} {kind}")
            sel = torch.arange(7, dtype=torch.int32).expand(c.n, h, 7).contiguous()
            for out, lse in (run_attend(c, 1.0, causal=False, max_kv=max_kv), run_attend(c, 1.0, sel=sel)):
                o = out.cpu().double()
                # the weights' rounding, the output's, and 100 terms in 32 bits
                tol = (2 * u + 2 * (n + 8) * K.U32) * big
                off = float((o - c.v[0, 0, 0].double()).abs().nan_to_num(math.inf).max())
                assert off <= tol and bool(torch.isfinite(lse).all()), (kind, off)


def test_attend_scale_zero():
    """All seen keys weigh the same; a query or key that is no number still makes its rows NaN."""
    for q_len in (1, 40):
        c = K.Case([(q_len, 90), (q_len, 70)], dtype=BF16, d=64, h=1, group=2, page=16)
        c.q[0, 1, 3] = math.nan
        c.q[q_len, 0, 60] = math.inf
        log(f"scale 0, {q_len} rows")
        out, lse = run_attend(c, 0.0)
        K.check_attention(c, out, lse, K.attention(c, 0.0), f"scale 0, {q_len} rows")


def test_max_q_far_above_the_rows():
    """max_q only has to be at least the new tokens of a sequence: a bound far above them is none of
    the launch's size."""
    c = K.Case([(1, 100), (30, 333), (2, 9)], dtype=BF16, d=64, h=2, group=3, page=16)
    hq, n_select = c.h * c.group, 5
    sel = K.select(c, K.all_bounds(c), 1, 1, n_select)
    for max_q in (33, 1 << 20, (1 << 31) - 1):
        log(f"max_q {max_q}")
        out, lse = run_attend(c, 0.125, max_q=max_q)
        K.check_attention(c, out, lse, K.attention(c, 0.125), f"max_q {max_q}")
        k, v = c.pools()
        cache, batch = kv.Cache(k, v), gpu_batch(c, max_q=max_q)
        got = torch.full((c.n, c.h, n_select), -7, dtype=torch.int32, device="cuda")
        bounds = K.all_bounds(c).cuda()
        kv.select(cache, batch, bounds, c.wide_q.cuda()[:, :hq], got, n_first=1, n_last=1,
                  workspace=ws(kv.select_workspace(cache, batch, c.n, n_select)))
        kv.page_bounds(cache, batch, bounds)
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), sel.int()), f"max_q {max_q}"


# ---------------------------------------------------------------- selection

SEL_LENS = [(1, 1), (1, 500), (0, 0), (7, 333), (1, 16), (3, 17), (1, 999), (2, 1), (40, 260)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,group,page,first,last,n_select", [
    (64, 2, 1, 16, 0, 1, 4), (128, 2, 4, 16, 1, 2, 8), (80, 1, 3, 8, 1, 1, 2), (256, 1, 8, 16, 2, 3, 21),
    (8, 2, 2, 32, 0, 1, 1), (96, 3, 2, 1, 4, 4, 50), (128, 1, 16, 24, 1, 1, 64)])
def test_select_and_attend(dtype, d, h, group, page, first, last, n_select):
    c = K.Case(SEL_LENS, dtype=dtype, d=d, h=h, group=group, page=page, fill=math.nan, tail_rows=2)
    bounds = K.all_bounds(c)
    log(f"select {dtype} d={d} h={h} group={group} page={page} {first}/{last}/{n_select}")
    k, v = c.pools()
    cache, batch = kv.Cache(k, v), gpu_batch(c)
    sel = torch.full((c.n, h, n_select), -7, dtype=torch.int32, device="cuda")
    q = c.wide_q.cuda()[:, :h * group]
    kv.select(cache, batch, bounds.cuda(), q, sel, n_first=first, n_last=last,
              workspace=ws(kv.select_workspace(cache, batch, c.n, n_select)))
    torch.cuda.synchronize()
    want = K.select(c, bounds, first, last, n_select)
    assert torch.equal(sel.cpu(), want)
    scale = 1 / math.sqrt(d)
    out, lse = run_attend(c, scale, sel=want)
    K.check_attention(c, out, lse, K.attention(c, scale, sel=want), "selected")
    assert (out[c.n - 2:] == PAD).all() and (lse[c.n - 2:] == PAD).all()


def test_select_ties_and_odd_scores():
    """Equal scores take the lower page; NaN bounds rank first, pages without bounds last, signed
    zeros tie."""
    page, n_pages = 4, 300
    c = K.Case([(1, page * n_pages)], dtype=F16, d=16, h=1, group=2, page=page, extra=0)
    bounds = torch.zeros(c.n_pages, 1, 2, 16, dtype=F16)
    ids = c.table[0, :n_pages].long()
    c.q[:] = 1.0
    bounds[ids[100:200], 0, 1] = 2.0
    bounds[ids[50:60]] = -0.0
    bounds[ids[250], 0, :, 3] = math.nan
    bounds[ids[251], 0, 1, 3] = math.inf
    bounds[ids[252], 0, :, 3] = -math.inf
    c.table[0, 120] = -1
    c.table[0, 130] = 1 << 20
    k, v = c.pools()
    for n_select in (4, 30, 103, 104, 120, 170, 297, 298, 299, 300):
        sel = torch.full((1, 1, n_select), -7, dtype=torch.int32, device="cuda")
        cache, batch = kv.Cache(k, v), gpu_batch(c)
        log(f"ties {n_select}")
        kv.select(cache, batch, bounds.cuda(), c.wide_q.cuda()[:, :2], sel, n_first=1, n_last=1,
                  workspace=ws(kv.select_workspace(cache, batch, 1, n_select)))
        assert torch.equal(sel.cpu(), K.select(c, bounds, 1, 1, n_select)), n_select


@pytest.mark.parametrize("n_pages,n_select", [(1000, 40), (1500, 700), (4100, 128), (13000, 500)])
def test_select_many_pages(n_pages, n_select):
    """Long lists: pages whose scores differ, pages in large groups of equal bounds (more open
    ones than are ranked one by one), and scores that differ by less than 32 bits hold."""
    for kind in ("random", "groups", "close"):
        page, d = 1, 32
        c = K.Case([(1, n_pages)], dtype=BF16, d=d, h=2, group=2, page=page, extra=0, seed=n_pages)
        g = torch.Generator().manual_seed(n_pages)
        a, b = torch.randn((2, n_pages, 2, d), generator=g)
        if kind == "groups":  # every 400 pages share their bounds
            a, b = (x[torch.arange(n_pages) % -(-n_pages // 400)] for x in (a, b))
        if kind == "close":  # one large channel hides the others from 32-bit sums
            a = a * 2.0 ** -14
            b = b * 2.0 ** -14
            a[..., 0] = b[..., 0] = 300.0
            c.q[..., 0] = 200.0
        bounds = torch.zeros((c.n_pages, 2, 2, d), dtype=BF16)
        ids = c.table[0, :n_pages].long()
        bounds[ids, :, 0], bounds[ids, :, 1] = torch.minimum(a, b).to(BF16), torch.maximum(a, b).to(BF16)
        c.table[0, 5] = -1
        k, v = c.pools()
        cache, batch = kv.Cache(k, v), gpu_batch(c)
        sel = torch.full((1, 2, n_select), -7, dtype=torch.int32, device="cuda")
        log(f"many pages {n_pages} {n_select} {kind}")
        kv.select(cache, batch, bounds.cuda(), c.wide_q.cuda()[:, :4], sel, n_first=2, n_last=3,
                  workspace=ws(kv.select_workspace(cache, batch, 1, n_select)))
        assert torch.equal(sel.cpu(), K.select(c, bounds, 2, 3, n_select)), kind


@pytest.mark.parametrize("group", [17, 40])
def test_select_large_groups(group):
    """More query heads a key head than one product holds."""
    c = K.Case([(1, 700), (2, 301)], dtype=F16, d=64, h=1, group=group, page=8)
    bounds = K.all_bounds(c)
    k, v = c.pools()
    cache, batch = kv.Cache(k, v), gpu_batch(c)
    sel = torch.full((c.n, 1, 12), -7, dtype=torch.int32, device="cuda")
    log(f"large group {group}")
    kv.select(cache, batch, bounds.cuda(), c.wide_q.cuda()[:, :group], sel, n_first=1, n_last=2,
              workspace=ws(kv.select_workspace(cache, batch, c.n, 12)))
    want = K.select(c, bounds, 1, 2, 12)
    assert torch.equal(sel.cpu(), want)
    out, lse = run_attend(c, 0.1, sel=want)
    K.check_attention(c, out, lse, K.attention(c, 0.1, sel=want), "large group")


def test_attend_selected_lists():
    """Lists with repeats, pages past the sequence, gaps and nothing at all."""
    c = K.Case([(1, 100), (3, 260), (1, 90)], d=64, h=2, group=3, page=16, fill=math.nan)
    sel = torch.full((c.n, 2, 6), -1, dtype=torch.int32)
    lists = [[0, 2, 2, 6, -1, -1], [1, 40, 3, 1 << 30, -1, 2], [-1] * 6, [0, 1, 2, 3, 4, 16],
             [5, 5, 5, 5, 5, 5]]
    for r in range(c.n):
        sel[r, 0] = torch.tensor(lists[r])
        sel[r, 1] = torch.tensor(lists[(r + 2) % 5])
    # what the rule leaves of each list: in range and above the entry before it
    pages = c.table.shape[1] - 1
    kept = sel.clone()
    for r in range(c.n):
        for h in range(2):
            for e in range(6):
                x = int(sel[r, h, e])
                if not 0 <= x < -(-c.max_kv // 16) or (e and x <= int(sel[r, h, e - 1])):
                    kept[r, h, e] = -1
    assert pages >= 17
    log("lists")
    out, lse = run_attend(c, 0.125, sel=sel)
    K.check_attention(c, out, lse, K.attention(c, 0.125, sel=kept), "lists")


def test_attend_selected_page_named_twice():
    """A list that names a page again behind a smaller entry counts its keys twice."""
    c = K.Case([(1, 128)], dtype=F16, d=32, h=1, group=2, page=16)
    sel = torch.tensor([[[5, -1, 5, 2, 7, 6]]], dtype=torch.int32)  # kept: 5, 5, 7
    log("page named twice")
    out, lse = run_attend(c, 0.2, sel=sel)
    tok = torch.cat([torch.arange(p * 16, p * 16 + 16) for p in (5, 5, 7)])
    rows = c.table[0].long()[tok // 16] * 16 + tok % 16
    k64, v64 = (x.double().view(-1, 1, 32)[rows, 0] for x in (c.k, c.v))
    s = (k64 @ c.q[0].double().t() * 0.2).t()
    z = torch.logsumexp(s, 1)
    want = torch.exp(s - z[:, None]) @ v64
    # as K.attention: scores, weights, sums of 48 terms, the output
    delta = float((c.q[0].double().abs() @ k64.abs().t()).max()) * 0.2 * 40 * K.U32 + 8 * K.U32
    u = K.half_step(F16)
    tol = u * want.abs() + (u + 2 * delta + 56 * K.U32) * (torch.exp(s - z[:, None]) @ v64.abs()) + 2.0 ** -25
    assert ((out[0].cpu().double() - want).abs() <= tol).all()
    assert ((lse[0].cpu().double() - z).abs() <= delta + 60 * K.U32 * (1 + z.abs())).all()


def test_batch_in_two_calls():
    """The sequences up to s and from s on, over the same rows: each call leaves the other's rows as
    they were, and together they give what one call gives."""
    c = K.Case([(40, 200), (30, 90), (1, 700), (1, 33), (0, 5), (1, 260)], dtype=BF16, h=4, group=2, d=64,
               page=16, fill=math.nan, tail_rows=2)
    k, v = c.pools()
    cache, q = kv.Cache(k, v), c.wide_q.cuda()[:, :8]
    start, kv_len, table = c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda()
    ref = K.attention(c, 0.125)
    sel_ref = K.select(c, K.all_bounds(c), 1, 1, 4)
    out, lse = torch.full_like(c.q, PAD).cuda(), torch.full((c.n, 8), PAD, device="cuda")
    sel = torch.full((c.n, 4, 4), -7, dtype=torch.int32, device="cuda")
    log("two calls")
    for a, b, max_q, max_kv in ((2, 6, 1, 700), (0, 2, 40, 200)):
        part = kv.Batch(start[a:b + 1], kv_len[a:b], table[a:b], max_q, max_kv)
        kv.attend(cache, part, q, out, 0.125, lse=lse,
                  workspace=ws(kv.attend_workspace(cache, part, c.n, 8)))
        kv.select(cache, part, K.all_bounds(c).cuda(), q, sel,
                  workspace=ws(kv.select_workspace(cache, part, c.n, 4)))
        torch.cuda.synchronize()
        if a:
            assert (out[:70] == PAD).all() and (lse[:70] == PAD).all() and (sel[:70] == -7).all()
    K.check_attention(c, out, lse, ref, "two calls")
    assert torch.equal(sel.cpu(), sel_ref)
    assert (out[-2:] == PAD).all() and (lse[-2:] == PAD).all()


def test_select_rows_some_at_a_time():
    """A prompt's rows in pieces, each with the kv_len that its last row has: the whole call's lists,
    from a smaller workspace."""
    c = K.Case([(90, 700)], dtype=BF16, h=2, group=2, d=64, page=8, tail_rows=0)
    bounds = K.all_bounds(c).cuda()
    cache, q, table = kv.Cache(*c.pools()), c.wide_q.cuda()[:, :4], c.table.cuda()
    sel = torch.full((90, 2, 6), -7, dtype=torch.int32, device="cuda")
    log("rows some at a time")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    whole = kv.select_workspace(cache, gpu_batch(c), 90, 6)
    for a, b in ((0, 40), (40, 41), (41, 90)):
        part = kv.Batch(i32(0, b - a), i32(700 - 90 + b), table, b - a, 700)
        need = kv.select_workspace(cache, part, b - a, 6)
        assert need < whole
        kv.select(cache, part, bounds, q[a:b], sel[a:b], workspace=ws(need))
    torch.cuda.synchronize()
    assert torch.equal(sel.cpu(), K.select(c, bounds.cpu(), 1, 1, 6))


@pytest.mark.parametrize("q_len,h", [(1, 1), (2, 4), (40, 1), (70, 4)])
def test_attend_infinite_scores(q_len, h):
    """A score of +inf makes its row NaN, its log of the sum too, whatever split it lies in; a score of
    -inf is a weight of zero, and rows that do not see the key are as without it."""
    n, page = 600, 16
    for max_kv in (None, 5000, 60000):
        c = K.Case([(q_len, n), (q_len, 333)], dtype=BF16, d=64, h=h, group=2, page=page, seed=7)
        plain = K.Case([(q_len, n), (q_len, 333)], dtype=BF16, d=64, h=h, group=2, page=page, seed=7)
        for x in (c, plain):
            if max_kv:
                wider_table(x, max_kv)
        c.q[..., 0] = torch.where(torch.arange(2 * h) % 2 == 0, 1.0, -1.0).to(BF16)
        plain.q[..., 0] = c.q[..., 0]
        j = 333 - 1 - q_len // 2  # of the second sequence: seen by its later rows
        at = (int(c.table[1, j // page]), j % page)
        c.k[at][:, 0] = math.inf
        log(f"infinite scores q={q_len} h={h} max_kv={max_kv}")
        out, lse = run_attend(c, 0.125, max_kv=max_kv)
        want = list(K.attention(plain, 0.125))
        # where the score is -inf the key counts as one that is not there
        gone = K.Case([(q_len, n), (q_len, 333)], dtype=BF16, d=64, h=h, group=2, page=page, seed=7)
        gone.q, gone.table, keys = c.q, c.table, gone.keys

        def without(s, upto=None):
            pos, rows = keys(s, upto)
            return (pos[pos != j], rows[pos != j]) if s == 1 else (pos, rows)
        gone.keys = without
        left = K.attention(gone, 0.125)
        for r, s, pos in c.rows():
            if s == 1 and pos >= j:
                for t in range(4):
                    want[t][r, 1::2] = left[t][r, 1::2]
                want[0][r, 0::2], want[1][r, 0::2] = math.nan, math.nan
        K.check_attention(c, out, lse, want, f"infinite scores, max_kv={max_kv}")


# ---------------------------------------------------------------- together

def test_decode_loop_with_the_compressed_store():
    """Prompt and decode steps as a user runs them: rows appended to the paged cache, the new rows
    compressed on write, pages fetched back from the compressed store into a second pool, and
    attention over both pools giving the same bits; pages selected and attended; the decode step
    captured in a graph and replayed with new lengths."""
    from host_transfer_amd import ibp
    h, group, d, page, n_pages, steps = 4, 2, 64, 16, 24, 5
    hq, width = h * group, h * d
    prompt = [37, 64, 5]
    g = torch.Generator().manual_seed(9)
    pools = [torch.zeros((n_pages, page, h, d), dtype=F16, device="cuda") for _ in "kv"]
    cache = kv.Cache(*pools)
    table = torch.full((3, 8), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g)
    for s in range(3):
        table[s] = order[s * 8:(s + 1) * 8]
    rope = K.rope_table(128, d)
    kn, qn = (1 + 0.2 * torch.randn(2, d, generator=g)).to(F16)
    d_table, d_rope, d_kn, d_qn = table.cuda(), rope.cuda(), kn.cuda(), qn.cuda()
    # IBP metadata over a sample of rows of that shape
    sample = torch.randn((256, width), generator=g).to(F16).cuda()
    B, C, rows_n = 2 * width, 256, n_pages * page
    mask, bitval = (torch.zeros(B // 4, dtype=torch.int32, device="cuda") for _ in range(2))
    counts = torch.zeros(8 * B, dtype=torch.int32, device="cuda")
    ibp.build_metadata(sample, B, None, 256, B, 0.99, mask, bitval, counts)
    store = ibp.HostBuffer(rows_n * B)
    part = torch.zeros((rows_n * (B // C) + 31) // 32, dtype=torch.int32, device="cuda")

    def slots_of(s, pos):
        return int(table[s, pos // page]) * page + pos % page

    def feed(lens, new):
        """Appends `new[s]` tokens of each sequence (all but the last `new` are there)."""
        n = sum(new)
        qkv = torch.randn((n, hq + 2 * h, d), generator=g).to(F16).cuda()
        pos = [kv_n - q + i for kv_n, q in zip(lens, new) for i in range(q)]
        seq = [s for s, q in enumerate(new) for _ in range(q)]
        slots = torch.tensor([slots_of(s, p) for s, p in zip(seq, pos)])
        q_out = torch.empty((n, hq, d), dtype=F16, device="cuda")
        kv.append(cache, qkv[:, hq:hq + h], qkv[:, hq + h:], slots.cuda(), q=qkv[:, :hq], q_out=q_out,
                  positions=torch.tensor(pos).cuda(), rope=d_rope, q_norm=d_qn, k_norm=d_kn)
        return q_out, slots

    def batch_of(lens, new, max_q, max_kv):
        start = torch.tensor([0] + new).cumsum(0).int().cuda()
        return kv.Batch(start, torch.tensor(lens, dtype=torch.int32).cuda(), d_table, max_q, max_kv)

    def attend(cache_, b, q):
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        kv.attend(cache_, b, q, out, 0.125, lse=lse,
                  workspace=ws(kv.attend_workspace(cache_, b, q.shape[0], hq)))
        return out, lse

    bounds = torch.zeros((n_pages, h, 2, d), dtype=F16, device="cuda")
    lens, new = list(prompt), list(prompt)
    for step in range(steps):
        log(f"decode loop step {step}: {lens}")
        q, slots = feed(lens, new)
        b = batch_of(lens, new, max(new), 128)
        kv.page_bounds(cache, b, bounds)
        out, lse = attend(cache, b, q)
        # the new rows of K (pool 0) into the compressed store, each a segment of one row
        kp = pools[0].view(rows_n, width)
        for lo in range(0, len(slots), 200):
            part_slots = slots[lo:lo + 200].tolist()
            ibp.compress_segments(kp, B, part_slots, part_slots, [1] * len(part_slots), rows_n, B, C,
                                  mask.repeat(len(part_slots)), bitval.repeat(len(part_slots)), store,
                                  B, part, None)
        # all pages back from the store into another pool, in another order of pages
        perm = torch.randperm(n_pages, generator=g)
        ids = (perm[:, None] * page + torch.arange(page)).reshape(-1).cuda()
        k2 = torch.zeros_like(pools[0])
        ibp.gather_decompress(store, rows_n * B, B, None, part, rows_n, ids, rows_n, B, C, mask,
                              bitval, k2)
        v2 = pools[1][perm.cuda()].contiguous()
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(n_pages)
        b2 = kv.Batch(b._keep[0], b._keep[1], inv[table.long()].int().cuda(), max(new), 128)
        out2, lse2 = attend(kv.Cache(k2, v2), b2, q)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        # the same from the formulas
        c = K.Case([(a, l) for a, l in zip(new, lens)], dtype=F16, h=h, group=group, d=d, page=page)
        c.k, c.v, c.table, c.n_pages = pools[0].cpu(), pools[1].cpu(), table, n_pages
        c.q, c.n = q.cpu(), q.shape[0]
        K.check_attention(c, out, lse, K.attention(c, 0.125), f"step {step}")
        assert torch.equal(bounds.cpu()[table[0, (lens[0] - 1) // page]],
                           K.all_bounds(c)[table[0, (lens[0] - 1) // page]])
        sel = torch.empty((c.n, h, 3), dtype=torch.int32, device="cuda")
        kv.select(cache, b, bounds, q, sel, n_first=1, n_last=1,
                  workspace=ws(kv.select_workspace(cache, b, c.n, 3)))
        want = K.select(c, K.all_bounds(c), 1, 1, 3)
        assert torch.equal(sel.cpu(), want)
        o3, l3 = torch.empty_like(q), torch.empty_like(lse)
        kv.attend_selected(cache, b, q, sel, o3, 0.125, lse=l3,
                           workspace=ws(kv.attend_selected_workspace(cache, b, c.n, hq, 3)))
        K.check_attention(c, o3, l3, K.attention(c, 0.125, sel=want), f"selected, step {step}")
        lens, new = [x + 1 for x in lens], [1, 1, 1]
    store.free()


def test_graph_replay_and_streams():
    """A decode step (append, bounds, attend, select, attend_selected) captured once and replayed
    with other inputs in the same buffers, eager work between; and attention on two streams at
    the same time.  The same bits as eager calls every time."""
    c = K.Case([(1, 900), (1, 300), (1, 1)], dtype=BF16, d=128, h=2, group=4, page=16)
    k, v = c.pools()
    cache = kv.Cache(k, v)
    hq, n = 8, 3
    batch = gpu_batch(c, max_kv=928)
    q = c.wide_q.cuda()[:, :hq].contiguous()
    rows = torch.randn((n, 2, 2, 128), device="cuda").to(BF16)
    slots = torch.tensor([5, 60, 100], device="cuda")
    bounds = K.all_bounds(c).cuda()
    w1 = ws(kv.attend_workspace(cache, batch, n, hq))
    w2 = ws(max(kv.select_workspace(cache, batch, n, 10),
                kv.attend_selected_workspace(cache, batch, n, hq, 10)))

    def step(out, lse, sel, out2):
        kv.append(cache, rows[:, 0], rows[:, 1], slots)
        kv.page_bounds(cache, batch, bounds)
        kv.attend(cache, batch, q, out, 0.1, lse=lse, workspace=w1)
        kv.select(cache, batch, bounds, q, sel, n_first=1, n_last=2, workspace=w2)
        kv.attend_selected(cache, batch, q, sel, out2, 0.1, workspace=w2)

    def buffers():
        return (torch.zeros((n, hq, 128), dtype=BF16, device="cuda"), torch.zeros((n, hq), device="cuda"),
                torch.zeros((n, 2, 10), dtype=torch.int32, device="cuda"),
                torch.zeros((n, hq, 128), dtype=BF16, device="cuda"))
    got, want = buffers(), buffers()
    step(*got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    log("capture")
    with torch.cuda.graph(graph):
        step(*got)
    for rep in range(4):
        q.copy_(torch.randn_like(q))
        rows.copy_(torch.randn_like(rows))
        batch._keep[1].copy_(torch.tensor([900 - 100 * rep, 300 - 77 * rep, 1 + rep]))
        step(*want)
        torch.cuda.synchronize()
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
        c.k, c.v, c.q = k.cpu(), v.cpu(), q.cpu()
        c.lens = [(1, x) for x in batch._keep[1].tolist()]
        K.check_attention(c, got[0], got[1], K.attention(c, 0.1), f"replay {rep}")
    # two streams, each with its workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want[0]) for _ in range(8)]
    works = [ws(w1.numel()) for _ in streams]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        kv.attend(cache, batch, q, o, 0.1, workspace=works[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want[0])


def test_graph_of_a_prompt_chunk():
    """Chunks over the cache (many rows, keys split over workgroups) and their selection captured
    in two graphs that share a workspace, replayed in turn with other lengths and inputs."""
    c = K.Case([(40, 700), (70, 300)], dtype=F16, d=64, h=2, group=2, page=16, fill=math.nan)
    k, v = c.pools()
    cache, batch = kv.Cache(k, v), gpu_batch(c, max_kv=704)
    q = c.wide_q.cuda()[:, :4].contiguous()
    bounds = K.all_bounds(c).cuda()
    w = ws(max(kv.attend_workspace(cache, batch, c.n, 4), kv.select_workspace(cache, batch, c.n, 6),
               kv.attend_selected_workspace(cache, batch, c.n, 4, 6)))

    def dense(out, lse):
        kv.attend(cache, batch, q, out, 0.125, lse=lse, workspace=w)

    def sparse(out, lse, sel):
        kv.select(cache, batch, bounds, q, sel, n_first=1, n_last=1, workspace=w)
        kv.attend_selected(cache, batch, q, sel, out, 0.125, lse=lse, workspace=w)

    def buffers():
        return [torch.zeros_like(q), torch.zeros((c.n, 4), device="cuda"), torch.zeros_like(q),
                torch.zeros((c.n, 4), device="cuda"),
                torch.zeros((c.n, 2, 6), dtype=torch.int32, device="cuda")]
    got, want = buffers(), buffers()
    dense(*got[:2])
    sparse(*got[2:])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    log("capture chunk")
    with torch.cuda.graph(graphs[0]):
        dense(*got[:2])
    with torch.cuda.graph(graphs[1]):
        sparse(*got[2:])
    for rep in range(3):
        q.copy_(torch.randn_like(q))
        batch._keep[1].copy_(torch.tensor([700 - 100 * rep, 300 - 115 * rep]))
        dense(*want[:2])
        sparse(*want[2:])
        torch.cuda.synchronize()
        for t in got:
            t.fill_(5)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
        c.q = q.cpu()
        c.lens = [(40, 700 - 100 * rep), (70, 300 - 115 * rep)]
        K.check_attention(c, got[0], got[1], K.attention(c, 0.125), f"chunk replay {rep}")


def test_graph_and_streams_of_chunks_in_splits():
    """Chunks whose keys are split over workgroups: captured and replayed with other lengths and inputs,
    eager calls between, and on two streams at once, each with its workspace."""
    c = K.Case([(40, 1800), (33, 1300)], dtype=BF16, d=128, h=2, group=2, page=16)
    wider_table(c, 6000)
    k, v = c.pools()
    cache, batch = kv.Cache(k, v), gpu_batch(c, max_kv=6000)
    q = c.wide_q.cuda()[:, :4].contiguous()
    need = kv.attend_workspace(cache, batch, c.n, 4)
    assert need > c.n * 4 * 8 * 130 * 4
    works = [ws(need) for _ in range(3)]

    def call(out, lse, work, **kw):
        kv.attend(cache, batch, q, out, 0.09, lse=lse, workspace=work, **kw)
    got, want = ([torch.zeros_like(q), torch.zeros((c.n, 4), device="cuda")] for _ in range(2))
    call(*got, works[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    log("capture split chunks")
    with torch.cuda.graph(graph):
        call(*got, works[0])
    for rep in range(3):
        q.copy_(torch.randn_like(q))
        batch._keep[1].copy_(torch.tensor([1800 - 500 * rep, 1300 - 600 * rep]))
        call(*want, works[1])
        torch.cuda.synchronize()
        for t in got:
            t.fill_(5)
        for w in works[:1]:
            w.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), rep
        c.q, c.lens = q.cpu(), [(40, 1800 - 500 * rep), (33, 1300 - 600 * rep)]
        K.check_attention(c, *got, K.attention(c, 0.09), f"replay {rep}")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(q), torch.zeros((c.n, 4), device="cuda")] for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        call(*o, works[1 + i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


@pytest.mark.parametrize("q_len", [1, 50])
def test_pages_beyond_32_bit_offsets(q_len):
    """A pool of more than 2^32 elements, its pages used at both ends: every call."""
    page, h, d = 64, 8, 128
    n_pages = (1 << 32) // (page * h * d) + 40
    pools = [torch.empty((n_pages, page, h, d), dtype=BF16, device="cuda") for _ in "kv"]
    c = K.Case([(q_len, 900), (q_len, 333)], dtype=BF16, d=d, h=h, group=2, page=page)
    where = torch.arange(c.n_pages)
    where = torch.where(where % 2 == 0, n_pages - 1 - where, where)  # page of the small pool -> here
    log(f"far pages q={q_len}")
    for big, small in zip(pools, (c.k, c.v)):
        big[where.cuda()] = small.cuda()
    far = torch.where(c.table >= 0, where[c.table.clamp(min=0).long()].int(), c.table)
    cache = kv.Cache(*pools)
    batch = kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), far.cuda(), q_len, 900)
    # the last new token of each sequence again, through append
    slots = torch.tensor([int(far[s, (n - 1) // page]) * page + (n - 1) % page
                          for s, (_, n) in enumerate(c.lens)])
    assert int(slots.max()) * h * d > 1 << 32
    kk, vv = (torch.stack([x[int(c.table[s, (n - 1) // page]), (n - 1) % page]
                           for s, (_, n) in enumerate(c.lens)]) for x in (c.k, c.v))
    for big in pools:
        big.view(-1, h, d)[slots.cuda()] = 9.0
    kv.append(cache, kk.cuda(), vv.cuda(), slots.cuda())
    bounds = torch.zeros((n_pages, h, 2, d), dtype=BF16, device="cuda")
    kv.page_bounds(cache, kv.Batch(torch.tensor([0, 900, 1233], dtype=torch.int32).cuda(),
                                   c.kv_len.cuda(), far.cuda(), 900, 900), bounds)
    small_bounds = K.all_bounds(c)
    assert torch.equal(bounds[where.cuda()].cpu()[c.table[0, :15].long()],
                       small_bounds[c.table[0, :15].long()])
    q = c.wide_q.cuda()[:, :2 * h]
    out = torch.zeros((c.n, 2 * h, d), dtype=BF16, device="cuda")
    lse = torch.zeros((c.n, 2 * h), device="cuda")
    kv.attend(cache, batch, q, out, 0.1, lse=lse,
              workspace=ws(kv.attend_workspace(cache, batch, c.n, 2 * h)))
    K.check_attention(c, out, lse, K.attention(c, 0.1), "far pages")
    sel = torch.zeros((c.n, h, 4), dtype=torch.int32, device="cuda")
    kv.select(cache, batch, bounds, q, sel, n_first=0, n_last=1,
              workspace=ws(kv.select_workspace(cache, batch, c.n, 4)))
    want = K.select(c, small_bounds, 0, 1, 4)
    assert torch.equal(sel.cpu(), want)
    kv.attend_selected(cache, batch, q, sel, out, 0.1, lse=lse,
                       workspace=ws(kv.attend_selected_workspace(cache, batch, c.n, 2 * h, 4)))
    K.check_attention(c, out, lse, K.attention(c, 0.1, sel=want), "far pages, selected")


def test_empty_calls():
    """No tokens, no rows, no sequences, a cache whose sequences are all empty."""
    c = K.Case([(0, 0), (0, 40)], d=64, tail_rows=3)
    k, v = c.pools()
    cache = kv.Cache(k, v)
    empty = torch.zeros((0, 2, 64), dtype=BF16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    none = kv.Batch(i32(0), i32(), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 0, 0)
    log("empty calls")
    kv.append(cache, empty, empty, torch.zeros(0, dtype=torch.int64, device="cuda"))
    bounds = torch.full((c.n_pages, 2, 2, 64), PAD, dtype=BF16, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=BF16, device="cuda")
    out = torch.full_like(q, PAD)
    sel = torch.full((3, 2, 5), -7, dtype=torch.int32, device="cuda")
    for batch in (none, gpu_batch(c), kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda(), 2, 48)):
        for n in (0, 3):
            kv.page_bounds(cache, batch, bounds)
            kv.attend(cache, batch, q[:n], out[:n], 1.0,
                      workspace=ws(kv.attend_workspace(cache, batch, n, 4)))
            kv.select(cache, batch, bounds, q[:n], sel[:n], n_first=0, n_last=1,
                      workspace=ws(kv.select_workspace(cache, batch, n, 5)))
            kv.attend_selected(cache, batch, q[:n], sel[:n], out[:n], 1.0,
                               workspace=ws(kv.attend_selected_workspace(cache, batch, n, 4, 5)))
    torch.cuda.synchronize()
    assert (out == PAD).all() and (sel == -7).all() and (bounds == PAD).all()
