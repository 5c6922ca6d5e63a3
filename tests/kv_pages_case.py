"""Plain computation of a step of the pages' assignment, a request and a page at a time: what the
tests of host_transfer_amd.kv_pages compare with (written from include/ibp_kv_pages.h)."""
import torch


class State:
    """Requests that hold random pages of a pool, on the CPU."""

    def __init__(self, had, page, n_free, max_pages, seed=0, extra=5, poison=()):
        """poison: (request, entry) of the table that are no page."""
        g = torch.Generator().manual_seed(seed)
        held = [-(-h // page) for h in had]
        self.page, self.max_pages = page, max_pages
        self.n_pages = sum(held) + n_free + extra  # `extra` pages belong to somebody else
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((len(had), max_pages), -77, dtype=torch.int32)
        at = 0
        for s, n in enumerate(held):
            self.table[s, :n] = order[at:at + n]
            at += n
        for k, (s, j) in enumerate(poison):
            self.table[s, j] = (-1, self.n_pages, -(1 << 31), (1 << 31) - 1)[k % 4]
        self.free = torch.full((self.n_pages,), -88, dtype=torch.int32)
        self.free[:n_free] = order[at:at + n_free]
        self.free_count = n_free
        self.had = list(had)


def step(st, keep, add, n_rows):
    """Advances a copy of st's table, stack and lengths: a dict of everything the call writes."""
    p, n_pages = st.page, st.n_pages
    table, free = st.table.clone(), st.free.clone()
    count = min(max(st.free_count, 0), n_pages)
    out = dict(q_start=[0], kv_len=[], length=[])
    plan, end = [], 0
    for s, had in enumerate(st.had):
        h = max(had, 0)
        k = h if keep is None else min(max(keep[s], 0), h)
        a = max(add[s], 0)
        end += a
        want = k + a
        held, wanted = min(-(-h // p), st.max_pages), -(-want // p)
        fits = end <= n_rows and wanted <= st.max_pages and want <= 1 << 30 and h <= 1 << 30
        plan.append((h, k, a, held, wanted, want, fits))
        out["q_start"].append(min(end, n_rows))
        if fits:
            for j in range(wanted, held):
                if 0 <= int(table[s, j]) < n_pages:
                    if count < n_pages:
                        free[count] = table[s, j]
                        count += 1
    left, asked, served = count, 0, []
    for s, (h, k, a, held, wanted, want, fits) in enumerate(plan):
        need = max(0, wanted - held) if fits else 0
        asked += need
        ok = fits and (need == 0 or asked <= count)
        if ok:
            for j in range(held, wanted):
                left -= 1
                table[s, j] = free[left]
        served.append(ok)
        out["kv_len"].append(want if ok else 0)
        out["length"].append(want if ok else h)
    slots, positions = [-1] * n_rows, [-1] * n_rows
    row = 0
    for s, (h, k, a, held, wanted, want, fits) in enumerate(plan):
        for i in range(a):
            if row < n_rows and served[s]:
                pos = k + i
                page = int(table[s, pos // p])
                positions[row] = pos
                slots[row] = page * p + pos % p if 0 <= page < n_pages else -1
            row += 1
            if row >= n_rows:
                break
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(table=table, free=free, left=i32([left]), unserved=i32([served.count(False)]),
                slots=torch.tensor(slots, dtype=torch.int64), positions=torch.tensor(positions, dtype=torch.int64),
                **{k: i32(v) for k, v in out.items()})
