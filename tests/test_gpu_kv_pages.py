"""The pages' assignment on the GPU against a plain loop over requests and pages
(tests/kv_pages_case.py): everything it writes, whole, equal."""
import random

import pytest
import torch

from host_transfer_amd import kv_pages
from tests import kv_pages_case as P

pytestmark = pytest.mark.gpu

PAD = -99


def log(msg):
    print("[kv pages] " + msg, flush=True)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(st, keep, add, n_rows, in_place=False, positions=True):
    """One call on a copy of st; what it wrote, on the CPU."""
    n = len(st.had)
    table, free = st.table.cuda(), st.free.cuda()
    had, count = i32(st.had), i32([st.free_count])
    o = dict(q_start=i32([PAD] * (n + 1)), kv_len=i32([PAD] * n), length=had if in_place else i32([PAD] * n),
             left=count if in_place else i32([PAD]), unserved=i32([PAD]),
             slots=torch.full((n_rows,), PAD, dtype=torch.int64, device="cuda"),
             positions=torch.full((n_rows,), PAD, dtype=torch.int64, device="cuda") if positions else None)
    pool = kv_pages.Pool(table, free, st.n_pages, st.page)
    ws = torch.empty(max(16, kv_pages.assign_workspace(n, n_rows)), dtype=torch.uint8, device="cuda")
    kv_pages.assign(pool, had, i32(add), count, o["q_start"], o["kv_len"], o["length"], o["left"], o["slots"],
                    o["positions"], keep=None if keep is None else i32(keep), unserved=o["unserved"], workspace=ws)
    torch.cuda.synchronize()
    o.update(table=table, free=free)
    return {k: v.cpu() for k, v in o.items() if v is not None}


def check(got, want):
    for k, v in got.items():
        assert torch.equal(v, want[k]), (k, v, want[k])


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 300, 1023, 1024, 1025, 2500, 5000])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_step(n, page):
    """Requests of every kind in one step: running, with rejected drafts, ended, new, idle."""
    rng = random.Random(n * 31 + page)
    for trial, long in ((0, False), (1, True), (2, False), (3, False)):
        had, keep, add = [], [], []
        for s in range(n):
            h = rng.choice([0, 1, page, page + 1, rng.randrange(0, 40 if not long else 900)])
            kind = rng.randrange(6)
            k, a = {0: (h, 1), 1: (max(0, h - rng.randrange(0, 5)), rng.randrange(0, 6)), 2: (0, 0), 3: (h, 0),
                    4: (h, rng.randrange(0, 30)), 5: (h // 2, rng.randrange(0, 3))}[kind]
            had.append(h)
            keep.append(k)
            add.append(a)
        if long:
            add[n // 2] = 3 * page + 777
        need = sum(max(0, -(-(k + a) // page) - -(-h // page)) for h, k, a in zip(had, keep, add))
        # plenty, exactly the pages that are needed if none is given back, too few, none
        n_free = (need + 3, need, need // 2, 0)[trial]
        st = P.State(had, page, n_free, max_pages=max(-(-(max(had) + max(add)) // page), 1) + 1, seed=trial)
        n_rows = sum(add) + (0, 5, 0, 1)[trial]
        log(f"n={n} page={page} trial={trial} rows={n_rows} free={n_free} need={need}")
        check(run(st, keep, add, n_rows, in_place=trial % 2 == 1), P.step(st, keep, add, n_rows))
        if trial == 0:  # all kept
            check(run(st, None, add, n_rows, positions=False), P.step(st, None, add, n_rows))


def test_what_is_not_served():
    """Too few rows, more pages than a row has, tokens past the limit, lengths below zero, a stack whose count is wrong."""
    page = 16
    had, keep, add = [40, 5, 0, 100, 30, 16, -7, 9], [40, 5, 0, 90, -3, 99, 4, 9], [3, 80, 2, 5, 4, -6, 8, 1]
    for n_rows in (0, 1, 3, 82, 83, 85, 200):
        for max_pages in (7, 5):
            for free in (0, 1, 30):
                st = P.State([max(h, 0) if max_pages == 7 else min(max(h, 0), 80) for h in had], page, free, max_pages)
                st.had = had if max_pages == 7 else [min(h, 80) for h in had]
                log(f"rows={n_rows} max_pages={max_pages} free={free}")
                check(run(st, keep, add, n_rows), P.step(st, keep, add, n_rows))
    st = P.State([20, 20, 20], page, 6, 4)
    for add in ([1 << 30, 1, 1], [(1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1], [1, -(1 << 31), 1 << 30]):
        log(f"add={add}")
        check(run(st, None, add, 50), P.step(st, None, add, 50))
    for count in (-5, 1 << 30, -(1 << 31)):
        st = P.State([20, 20, 20], page, 6, 4)
        st.free[:] = torch.arange(st.n_pages, dtype=torch.int32)
        st.free_count = count
        log(f"count={count}")
        check(run(st, [20, 20, 0], [20, 1, 0], 50), P.step(st, [20, 20, 0], [20, 1, 0], 50))


def test_entries_that_are_no_page():
    """They are not given back, and a token that would lie there has no slot."""
    page = 8
    had = [100, 57, 1000, 3, 90, 700]
    poison = [(0, 12), (0, 0), (1, 7), (2, 1), (2, 50), (2, 124), (2, 60), (2, 61), (3, 0), (5, 87)]
    st = P.State(had, page, 3, max_pages=130, poison=poison)
    for keep, add in (([100, 57, 0, 3, 90, 700], [2, 3, 0, 2, 1, 9]), ([0, 0, 5, 0, 0, 0], [0, 0, 4, 1, 0, 1]),
                      ([90, 1, 300, 1, 17, 8], [20, 3, 1, 30, 0, 0])):
        n_rows = sum(add) + 2
        log(f"keep={keep}")
        check(run(st, keep, add, n_rows), P.step(st, keep, add, n_rows))
    st.free[1] = st.n_pages  # ids on the stack are not trusted either
    st.free[2] = -1
    check(run(st, None, [40, 1, 1, 6, 30, 2], 80), P.step(st, None, [40, 1, 1, 6, 30, 2], 80))


def test_nothing_to_do():
    st = P.State([], 16, 4, 3)
    got, want = run(st, [], [], 7), P.step(st, [], [], 7)
    check(got, want)
    st = P.State([5, 0], 16, 4, 3)
    check(run(st, [5, 0], [0, 0], 0), P.step(st, [5, 0], [0, 0], 0))


@pytest.mark.parametrize("n,rows", [(40, 600), (1500, 9000)])
def test_many_steps_in_place_captured(n, rows):
    """Sixty steps of one captured graph: after each, everything as the plain loop has it, no page is
    held twice and none is lost."""
    page, max_pages, n_pages = 4, 40, n * 6
    rng = random.Random(n)
    st = P.State([0] * n, page, n_pages, max_pages, extra=0)
    table, free = st.table.cuda(), st.free.cuda()
    had, keep, add, count = (i32([0] * n) for _ in range(4))
    count = i32([st.free_count])
    q_start, kv_len, unserved = i32([0] * (n + 1)), i32([0] * n), i32([0])
    slots, positions = (torch.zeros(rows, dtype=torch.int64, device="cuda") for _ in "sp")
    pool = kv_pages.Pool(table, free, st.n_pages, page)
    ws = torch.empty(max(16, kv_pages.assign_workspace(n, rows)), dtype=torch.uint8, device="cuda")

    def call():
        kv_pages.assign(pool, had, add, count, q_start, kv_len, had, count, slots, positions, keep=keep,
                        unserved=unserved, workspace=ws)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()  # nothing is wanted yet
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    short = 0
    for turn in range(60):
        k = [0 if rng.random() < 0.05 else max(0, h - rng.choice([0, 0, 0, 1, 3])) for h in st.had]
        a = [rng.choice([0, 1, 1, 1, 4, 12]) for _ in range(n)]
        want = P.step(st, k, a, rows)
        keep.copy_(i32(k))
        add.copy_(i32(a))
        graph.replay()
        torch.cuda.synchronize()
        got = dict(table=table, free=free, left=count, q_start=q_start, kv_len=kv_len, length=had, slots=slots,
                   positions=positions, unserved=unserved)
        check({x: y.cpu() for x, y in got.items()}, want)
        st.table, st.free, st.had = want["table"], want["free"], want["length"].tolist()
        st.free_count = int(want["left"])
        short += int(want["unserved"]) > 0
        ids = st.free[:st.free_count].tolist()
        for s, h in enumerate(st.had):
            ids += st.table[s, :-(-h // page)].tolist()
        assert sorted(ids) == list(range(st.n_pages)), f"turn {turn}: a page is lost or held twice"
    log(f"n={n}: {short} of 60 steps were short of pages or rows")
    assert 0 < short < 60
