"""The serving calls together, as a user runs them: pages assigned, keys and values appended, attention,
over the cache in 8 bits and the one in 16, step after step of one captured graph; the 8-bit rows
through the compressed store."""
import random

import pytest
import torch

from host_transfer_amd import ibp, kv, kv8, kv_pages
from tests import kv8_case as K8
from tests import kv_case as K
from tests import kv_pages_case as P

pytestmark = pytest.mark.gpu

PAD = -4.25


def log(msg):
    print("[kv serving] " + msg, flush=True)


def ws(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype,d,page,block,group", [(torch.bfloat16, 64, 16, 8, 2), (torch.float16, 128, 8, 8, 4)])
def test_requests_come_and_go(dtype, d, page, block, group):
    """Requests start with a prompt, verify drafted tokens of which some are rejected, end, and give their
    pages to others; the pool is too small for all at times.  One graph, no length on the host: after each
    replay the tables, the caches and both attentions are as the plain computations have them."""
    h, n, n_rows, max_pages, n_pages, max_q = 4, 6, 48, 10, 160 // page, 24
    hq, rng, g = h * group, random.Random(d), torch.Generator().manual_seed(d)
    st = P.State([0] * n, page, n_pages, max_pages, extra=0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free = st.table.cuda(), st.free.cuda()
    had, keep, add, kv_len = (i32([0] * n) for _ in range(4))
    count, q_start, unserved = i32([st.free_count]), i32([0] * (n + 1)), i32([0])
    slots, positions = (torch.zeros(n_rows, dtype=torch.int64, device="cuda") for _ in "sp")
    pool = kv_pages.Pool(table, free, n_pages, page)
    pools16 = [torch.zeros((n_pages, page, h, d), dtype=dtype, device="cuda") for _ in "kv"]
    codes = [torch.zeros((n_pages, page, h, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
    exps = [torch.zeros((n_pages, page // block, h), dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache16, cache8 = kv.Cache(*pools16), kv8.Cache(*(x.view(K8.E4M3) for x in codes), *exps)
    batch = kv.Batch(q_start, kv_len, table, max_q, max_pages * page)
    qkv = torch.zeros((n_rows, hq + 2 * h, d), dtype=dtype, device="cuda")
    rope = K.rope_table(max_pages * page, d)
    g_rope = rope.cuda()
    kn, qn = (1 + 0.2 * torch.randn(2, d, generator=g)).to(dtype)
    g_kn, g_qn = kn.cuda(), qn.cuda()
    q16, q8, out16, out8 = (torch.zeros((n_rows, hq, d), dtype=dtype, device="cuda") for _ in range(4))
    lse16, lse8 = (torch.zeros((n_rows, hq), device="cuda") for _ in range(2))
    w_pages = ws(kv_pages.assign_workspace(n, n_rows))
    w16 = ws(kv.attend_workspace(cache16, batch, n_rows, hq))
    w8 = ws(kv8.attend_workspace(cache8, batch, n_rows, hq))

    def step():
        kv_pages.assign(pool, had, add, count, q_start, kv_len, had, count, slots, positions, keep=keep,
                        unserved=unserved, workspace=w_pages)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        kv.append(cache16, k, v, slots, q=q, q_out=q16, positions=positions, rope=g_rope, q_norm=g_qn, k_norm=g_kn)
        kv.attend(cache16, batch, q16, out16, 0.125, lse=lse16, workspace=w16)
        kv8.append(cache8, batch, k, v, q=q, q_out=q8, positions=positions, rope=g_rope, q_norm=g_qn, k_norm=g_kn)
        kv8.attend(cache8, batch, q8, out8, 0.125, lse=lse8, workspace=w8)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()  # nothing is wanted yet
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    short = ended = rejected = 0
    for turn in range(25):
        k, a = [], []
        for s in range(n):
            if st.had[s] == 0:
                k.append(0)
                a.append(rng.choice([0, rng.randrange(1, max_q + 1)]))
            elif rng.random() < 0.08 or st.had[s] > max_pages * page - 10:
                k.append(0)
                a.append(0)
                ended += 1
            else:
                k.append(max(1, st.had[s] - rng.randrange(0, 4)))
                a.append(rng.randrange(1, 6))
                rejected += st.had[s] - k[-1]
        while sum(a) > n_rows:
            a[a.index(max(a))] //= 2
        want = P.step(st, k, a, n_rows)
        rows = torch.randn((n_rows, hq + 2 * h, d), generator=g) * torch.exp(torch.randn((n_rows, 1, 1), generator=g))
        rows = rows.to(dtype)
        keep.copy_(i32(k))
        add.copy_(i32(a))
        qkv.copy_(rows)
        for t in (out16, out8, q16, q8):
            t.fill_(PAD)
        before = [x.cpu() for x in codes], [x.cpu() for x in exps]
        graph.replay()
        torch.cuda.synchronize()
        got = dict(table=table, free=free, left=count, q_start=q_start, kv_len=kv_len, length=had, slots=slots,
                   positions=positions, unserved=unserved)
        for name, x in got.items():
            assert torch.equal(x.cpu(), want[name]), (turn, name)
        st.table, st.free, st.had = want["table"], want["free"], want["length"].tolist()
        st.free_count = int(want["left"])
        short += int(want["unserved"]) > 0

        c = K8.Case8([(x, int(y)) for x, y in zip(a, want["kv_len"])], dtype=dtype, h=h, group=group, d=d, page=page,
                     block=block)
        c.table, c.n_pages, c.n = want["table"], n_pages, n_rows
        c.max_rows, c.most_kv = max_q, max_pages * page
        c.k8, c.v8 = (x.view(K8.E4M3) for x in before[0])
        c.ke, c.ve = before[1]
        pos = want["positions"].clamp(min=0)
        placed = want["slots"] >= 0
        new_k = K.norm_rotate(rows[:, hq:hq + h].double(), pos, rope, False, kn, 1e-6)
        ref = K8.append(c, new_k, rows[:, hq + h:].double(), placed)
        now = [x.cpu().view(K8.E4M3) for x in codes] + [x.cpu() for x in exps]
        for i, name in enumerate("kv"):
            val, e, written, exact = ref[name]
            same = now[i].double() == val
            assert same[~written].all() and torch.equal(now[2 + i], e), (turn, name)
            off = (now[i].double() - exact).abs()[written]
            lim = K8.grid_step(exact[written]) / 2
            if name == "k":  # the norm's and the rotation's 32 bits
                lim = lim + (d + 48) * K.U32 * 2 * exact[written].abs().amax(-1, keepdim=True)
            assert (off <= lim).all(), (turn, name)
        c.k8, c.v8, c.ke, c.ve = now
        c.renew()
        c.q = q8.cpu()
        K.check_attention(c, out8, lse8, K.attention(c, 0.125), f"8 bits, turn {turn}")
        c.k, c.v, c.q = pools16[0].cpu(), pools16[1].cpu(), q16.cpu()
        assert torch.equal(c.v.view(-1, h, d)[want["slots"][placed]], rows[placed, hq + h:])
        K.check_attention(c, out16, lse16, K.attention(c, 0.125), f"16 bits, turn {turn}")
        # the output's rounding, and 32 bits: the sum of d squares, the root, the products, the rotation's pairs
        new_q = K.norm_rotate(rows[:, :hq].double(), pos, rope, False, qn, 1e-6)[placed]
        lim = (K.half_step(dtype) + (d + 16) * K.U32) * new_q.abs() + 32 * K.U32 * new_q.abs().amax(-1, keepdim=True)
        lim = lim + torch.finfo(dtype).smallest_normal * K.half_step(dtype)
        for q in (q8, q16):
            assert ((q.cpu()[placed].double() - new_q).abs() <= lim).all()
        assert (out8.cpu()[sum(a):] == PAD).all() and (q8.cpu()[sum(a):] == PAD).all()
        for s, y in enumerate(want["kv_len"].tolist()):
            if y == 0 and a[s]:  # not served: nothing attended
                r = int(c.q_start[s])
                assert (out8[r:r + a[s]] == 0).all() and (out16[r:r + a[s]] == 0).all() and (q8[r:r + a[s]] == 0).all()
    log(f"{dtype}: {short} steps short of pages, {ended} requests ended, {rejected} tokens rejected")
    assert short and ended and rejected


def test_rows_of_codes_through_the_compressed_store():
    """A pool's rows of codes compressed (a tensor per token), fetched into another pool in another order
    of pages: attention over both gives the same bits."""
    h, d, page, block = 4, 64, 16, 16
    c = K8.Case8([(1, 200), (3, 77), (30, 130)], dtype=torch.bfloat16, h=h, group=2, d=d, page=page, block=block)
    c.k8.view(torch.uint8)[..., :8] &= 0x87  # channels whose values are small
    c.renew()
    k8, v8, ke, ve = c.pools8()
    B, C, rows_n = h * d, 256, c.n_pages * page
    mask, bitval = (torch.zeros(B // 4, dtype=torch.int32, device="cuda") for _ in range(2))
    counts = torch.zeros(8 * B, dtype=torch.int32, device="cuda")
    store = ibp.HostBuffer(rows_n * B)
    part = torch.zeros((rows_n + 31) // 32, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(rows_n, dtype=torch.int32, device="cuda")
    perm = torch.randperm(c.n_pages)
    ids = (perm[:, None] * page + torch.arange(page)).reshape(-1).cuda()
    other = []
    for x in (k8, v8):
        flat = x.view(torch.uint8)
        ibp.build_metadata(flat, B, None, rows_n, B, 0.99, mask, bitval, counts)
        ibp.compress(flat, B, rows_n, 0, rows_n, B, C, mask, bitval, store, B, part, lengths)
        back = torch.zeros_like(flat)
        ibp.gather_decompress(store, rows_n * B, B, None, part, rows_n, ids, rows_n, B, C, mask, bitval, back)
        torch.cuda.synchronize()
        assert torch.equal(back, flat[perm.cuda()])
        other.append(back.view(K8.E4M3))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(c.n_pages)
    moved = torch.where(c.table >= 0, inv[c.table.clamp(min=0).long()].int(), c.table)
    q = c.wide_q.cuda()[:, :8]
    results = []
    for pools, table in (((k8, v8, ke, ve), c.table), ((*other, ke[perm.cuda()], ve[perm.cuda()]), moved)):
        cache, batch = kv8.Cache(*pools), kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), table.cuda(), 30, 200)
        out, lse = torch.zeros_like(q.contiguous()), torch.zeros((c.n, 8), device="cuda")
        kv8.attend(cache, batch, q, out, 0.125, lse=lse, workspace=ws(kv8.attend_workspace(cache, batch, c.n, 8)))
        results.append((out, lse))
    torch.cuda.synchronize()
    log("rows of codes through the compressed store")
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    K.check_attention(c, *results[0], K.attention(c, 0.125), "from the store")
    store.free()
