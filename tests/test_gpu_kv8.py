"""The 8-bit paged K/V cache on the GPU against plain 64-bit computations (tests/kv8_case.py):
placement with norm, rotation and block exponents, and attention over the cache, at the sizes,
strides and masks where they can go wrong."""
import math

import pytest
import torch

from host_transfer_amd import kv, kv8
from tests import kv8_case as K8
from tests import kv_case as K

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
PAD = -4.25  # what rows and pages that a call must leave alone hold


def log(msg):
    print("[kv8] " + msg, flush=True)


def ws(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")


def gpu_batch(c, max_q=None, max_kv=None):
    return kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda(),
                    c.max_q if max_q is None else max_q, c.max_kv if max_kv is None else max_kv)


# ---------------------------------------------------------------- append

def run_append(c, qkv, hq, *, rope=None, pos=None, inter=False, qn=None, kn=None, max_q=None, max_kv=None,
               in_place=False, head_major=None):
    """One call; (codes k, codes v, exponents k, v, q_out), on the CPU."""
    k8, v8, ke, ve = c.pools8(head_major)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    gpu = qkv.cuda()
    q = gpu[:, :hq] if hq else None
    q_out = q if in_place else torch.full((c.n, hq, c.d), PAD, dtype=c.dtype, device="cuda") if hq else None
    kv8.append(kv8.Cache(k8, v8, ke, ve), gpu_batch(c, max_q, max_kv), gpu[:, hq:hq + c.h], gpu[:, hq + c.h:], q=q,
               q_out=q_out, positions=dev(pos), rope=dev(rope), flags=kv8.ROPE_INTERLEAVED if inter else 0,
               q_norm=dev(qn), k_norm=dev(kn), eps=1e-5)
    torch.cuda.synchronize()
    return [x.view(torch.uint8).cpu().view(K8.E4M3) for x in (k8, v8)] + [ke.cpu(), ve.cpu(), dev(q_out)]


def placed_rows(c, pos=None, n_pos=None):
    """Which rows are placed, and which belong to a sequence (of its first max_rows)."""
    placed, held = torch.zeros(c.n, dtype=torch.bool), torch.zeros(c.n, dtype=torch.bool)
    for r, s, at in c.rows():
        if r - int(c.q_start[s]) >= c.max_rows:
            continue
        held[r] = True
        page = int(c.table[s, at // c.page]) if 0 <= at < min(c.lens[s][1], c.most_kv) else -1
        placed[r] = 0 <= page < c.n_pages and (pos is None or 0 <= int(pos[r]) < n_pos)
    return placed, held


def check_cache(c, got, ref, rel):
    """rel: how far (relative to the row's largest value) 32 bits may be from the value that is
    rounded; 0: the codes have to be equal."""
    for i, name in enumerate("kv"):
        val, exps, written, exact = ref[name]
        codes, e = got[i].double(), got[2 + i]
        slack = rel if name == "k" else 0.0  # values are copied
        assert torch.equal(e, exps), f"{name}: exponents"
        same = (codes == val) | (torch.isnan(codes) & torch.isnan(val))
        if not slack:
            assert same.all(), f"{name}: codes"
            continue
        assert same[~written].all(), f"{name}: codes of other tokens"
        fine = torch.isfinite(exact)
        assert (torch.isnan(codes) == torch.isnan(val)).all()
        top = exact.abs().nan_to_num(0).amax(-1, keepdim=True).expand_as(exact)
        off = (codes - exact).abs()[fine]
        lim = (K8.grid_step(exact) / 2 + slack * (exact.abs() + top))[fine]
        assert (off <= lim).all(), f"{name}: off by {float((off / lim).max()):.3f} of the limit"


def check_q(c, got, want, placed, held, norm, rope):
    u, tiny = K.half_step(c.dtype), torch.finfo(c.dtype).smallest_normal * torch.finfo(c.dtype).eps / 2
    got = got.cpu()
    assert (got[held & ~placed] == 0).all()
    assert (got[~held] == PAD).all(), "touched rows of no sequence"
    err = (got[placed].double() - want[placed]).abs()
    lim = (u + (c.d + 16) * K.U32) * want[placed].abs() + tiny
    if rope:  # the rotation's output is bounded by the pair's length, not by itself
        lim = lim + want[placed].abs().amax(-1, keepdim=True) * 32 * K.U32
    assert (err <= lim).all()


LENS = [(1, 1), (3, 3), (0, 9), (1, 37), (5, 40), (40, 40), (70, 131), (0, 0), (2, 18), (1, 33), (17, 49)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,rope,inter,norm,block,page", [
    (16, 0, False, False, 16, 16), (64, 64, False, True, 16, 32), (64, 32, True, True, 8, 8), (80, 48, True, True, 24, 48),
    (96, 96, False, True, 16, 16), (128, 128, False, True, 16, 64), (128, 128, True, False, 1, 4),
    (128, 0, False, False, 64, 64), (144, 0, False, True, 5, 10), (192, 192, False, True, 32, 32),
    (256, 256, False, True, 16, 16), (256, 128, True, True, 100, 100)])
def test_append(dtype, d, rope, inter, norm, block, page):
    for hq, h, head_major, tail in ((6, 2, False, 4), (0, 5, True, 0)):
        c = K8.Case8(LENS, block=block, dtype=dtype, h=h, group=1, d=d, page=page, tail_rows=tail, seed=d + block)
        c.max_rows, c.most_kv = 1 << 30, 1 << 30
        g = torch.Generator().manual_seed(d)
        log(f"append {dtype} d={d} rope={rope} inter={inter} norm={norm} block={block} page={page} hq={hq} h={h}")
        scale = torch.exp(2 * torch.randn((c.n, 1, 1), generator=g))
        qkv = (torch.randn((c.n, hq + 2 * h, d), generator=g) * scale).to(dtype)
        pos = torch.randint(0, 50, (c.n,), generator=g) if rope else None
        table = K.rope_table(50, rope) if rope else None
        if rope:
            pos[3], pos[30], pos[100] = 50, -1, 1 << 40
        c.table[5, 1] = c.n_pages  # a page that is not there
        qn = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None
        kn = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None
        placed, held = placed_rows(c, pos, 50)
        assert int(placed.sum()) > 100
        got = run_append(c, qkv, hq, rope=table, pos=pos, inter=inter, qn=qn, kn=kn, head_major=head_major)
        safe = None if pos is None else pos.clamp(0, 49)
        x = qkv.double()
        new_k = K.norm_rotate(x[:, hq:hq + h], safe, table, inter, kn, 1e-5)
        # fp32: the sum of d squares, the root, three products, the rotation's two products and sum
        rel = (d + 48) * K.U32 if rope or norm else 0.0
        check_cache(c, got, K8.append(c, new_k, x[:, hq + h:], placed), rel)
        if hq:
            check_q(c, got[4], K.norm_rotate(x[:, :hq], safe, table, inter, qn, 1e-5), placed, held, norm, rope)


def test_append_lengths_and_limits():
    """New tokens in front of position 0, past max_kv, past max_q; a block whose page is not there."""
    for max_q, max_kv in ((None, None), (9, None), (None, 40), (3, 33)):
        lens = [(20, 12), (60, 90), (1, 41), (5, 3), (33, 33), (4, 44)]
        c = K8.Case8(lens, block=8, dtype=BF16, h=3, group=1, d=64, page=16, tail_rows=2)
        c.max_rows, c.most_kv = max_q or 1 << 30, max_kv or 1 << 30
        c.table[1, 4], c.table[4, 0] = -1, 1 << 30
        g = torch.Generator().manual_seed(5)
        qkv = torch.randn((c.n, 8, 64), generator=g).to(BF16)
        log(f"append max_q={max_q} max_kv={max_kv}")
        placed, held = placed_rows(c)
        got = run_append(c, qkv, 2, max_q=max_q, max_kv=max_kv)
        x = qkv.double()
        check_cache(c, got, K8.append(c, x[:, 2:5], x[:, 5:], placed), 0.0)
        check_q(c, got[4], x[:, :2], placed, held, False, False)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_odd_values(dtype):
    """Infinities, NaN, zeros, the type's ends, ties of the rounding, in fresh and in extended blocks."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    lens = [(16, 16), (3, 19), (16, 48), (1, 30), (8, 8)]
    c = K8.Case8(lens, block=16, dtype=dtype, h=2, group=1, d=32, page=16)
    c.max_rows = c.most_kv = 1 << 30
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((c.n, 4, 32), generator=g).to(dtype)
    qkv[0, :, 0], qkv[1, :, 1], qkv[2, :, 2], qkv[3, :, 3] = math.inf, -math.inf, math.nan, -0.0
    qkv[16:19] = 0  # an extended block gains zeros
    qkv[19:35, 0], qkv[19:35, 1] = 0, big  # fresh blocks of zeros, of the largest values
    qkv[19:35, 2], qkv[19:35, 3] = tiny * 2 ** -3, math.inf
    qkv[35] = 60000.0  # raises the exponent of an extended block far
    # ties: halves between neighbouring codes, around 448 * 2^n and in the subnormal part
    ladder = [448, 440, 456, 432, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17, 19, 21, 1.0625, 1.1875, 2.0 ** -6, 0.0]
    for i in range(8):
        qkv[36 + i] = 0.25
        qkv[36 + i, :, :14] = (torch.tensor(ladder) * (-1) ** i).to(dtype)
    c.k8.view(torch.uint8)[int(c.table[1, 1]), 0] = 0x7F  # a NaN in front of new tokens stays one
    c.renew()
    placed, _ = placed_rows(c)
    log(f"append odd values {dtype}")
    got = run_append(c, qkv, 0)
    x = qkv.double()
    check_cache(c, got, K8.append(c, x[:, :2], x[:, 2:], placed), 0.0)
    assert int(got[2].min()) >= 1


@pytest.mark.parametrize("q_len,block", [(1, 16), (2, 16), (5, 8)])
def test_append_step_by_step(q_len, block):
    """A sequence that grows some tokens at a time, with values that now and then are larger: after each
    call everything as computed from the call before."""
    c = K8.Case8([(q_len, q_len)], block=block, dtype=BF16, h=2, group=1, d=64, page=2 * block, extra=8)
    c.max_rows = c.most_kv = 1 << 30
    c.table = torch.tensor([[3, 0, 5, 1, 4, 2, 6, 7]], dtype=torch.int32)
    g = torch.Generator().manual_seed(9)
    for step in range(45 // q_len):
        c.lens = [(q_len, (step + 1) * q_len)]
        c.kv_len = torch.tensor([c.lens[0][1]], dtype=torch.int32)
        qkv = (torch.randn((q_len, 6, 64), generator=g) * 2.0 ** int(torch.randint(-4, 5, (1,), generator=g))).to(BF16)
        placed, held = placed_rows(c)
        got = run_append(c, qkv, 2, in_place=True)
        x = qkv.double()
        check_cache(c, got, K8.append(c, x[:, 2:4], x[:, 4:], placed), 0.0)
        assert torch.equal(got[4].cpu(), qkv[:, :2])
        c.k8, c.v8, c.ke, c.ve = got[:4]
    log(f"step by step q={q_len} block={block}: exponents {c.ke.flatten().tolist()[:8]}")


def test_append_long_prompt_beside_single_tokens():
    """More possible blocks than rows: units are counted by rows."""
    lens = [(1, 5 + 3 * i) for i in range(40)] + [(300, 411)] + [(1, 17)] * 9 + [(0, 5), (2, 2)]
    for block, page in ((16, 16), (3, 6), (64, 64)):
        c = K8.Case8(lens, block=block, dtype=BF16, h=2, group=1, d=128, page=page, tail_rows=3)
        c.max_rows = c.most_kv = 1 << 30
        c.table[40, 7] = -5
        g = torch.Generator().manual_seed(block)
        qkv = torch.randn((c.n, 7, 128), generator=g).to(BF16)
        placed, held = placed_rows(c)
        log(f"long prompt beside single tokens, block={block}")
        got = run_append(c, qkv, 3)
        x = qkv.double()
        check_cache(c, got, K8.append(c, x[:, 3:5], x[:, 5:], placed), 0.0)
        check_q(c, got[4], x[:, :3], placed, held, False, False)


@pytest.mark.parametrize("dtype,d,h,q_len,block,page", [
    (BF16, 64, 8, 1, 16, 16), (F16, 64, 20, 4, 8, 16), (BF16, 128, 8, 1, 16, 32), (F16, 128, 11, 3, 16, 16),
    (BF16, 256, 4, 2, 32, 32), (F16, 80, 9, 2, 1, 4), (BF16, 128, 40, 4, 16, 16)])
def test_append_few_tokens_of_many_sequences(dtype, d, h, q_len, block, page):
    """Enough sequences of few new tokens that a wave holds several heads of a token: extended, fresh and
    crossed blocks, exponents that rise and not, heads that are no multiple of a wave's."""
    g = torch.Generator().manual_seed(d + h)
    n = 300
    lens = []
    for s in range(n):
        q = int(torch.randint(0, q_len + 1, (1,), generator=g))
        lens.append((q, q + int(torch.randint(0, 40, (1,), generator=g))))
    lens[7] = (q_len, q_len)
    c = K8.Case8(lens, block=block, dtype=dtype, h=h, group=1, d=d, page=page, tail_rows=2, seed=h)
    c.max_rows = c.most_kv = 1 << 30
    c.table[11, 0] = -1
    log(f"few tokens of many sequences {dtype} d={d} h={h} q={q_len} block={block}")
    for rope, norm in ((0, False), (d if d % 32 == 0 else 48, True)):
        scale = torch.exp2(torch.randint(-2, 3, (c.n, h + 3, 1), generator=g).float())
        qkv = torch.randn((c.n, 3 + 2 * h, d), generator=g)
        qkv[:, 3:3 + h] *= scale[:, 3:]
        qkv[:, 3 + h:] *= scale[:, 3:]
        qkv = qkv.to(dtype)
        pos = torch.randint(0, 50, (c.n,), generator=g) if rope else None
        table = K.rope_table(50, rope) if rope else None
        if rope:
            pos[5], pos[60] = -1, 50
        kn = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None
        placed, held = placed_rows(c, pos, 50)
        got = run_append(c, qkv, 3, rope=table, pos=pos, qn=kn, kn=kn)
        safe = None if pos is None else pos.clamp(0, 49)
        x = qkv.double()
        new_k = K.norm_rotate(x[:, 3:3 + h], safe, table, False, kn, 1e-5)
        check_cache(c, got, K8.append(c, new_k, x[:, 3 + h:], placed), (d + 48) * K.U32 if rope else 0.0)
        check_q(c, got[4], K.norm_rotate(x[:, :3], safe, table, False, kn, 1e-5), placed, held, norm, rope)


# ---------------------------------------------------------------- attention

def run_attend(c, scale, causal=True, window=0, max_q=None, max_kv=None):
    cache, batch = kv8.Cache(*c.pools8()), gpu_batch(c, max_q, max_kv)
    hq = c.h * c.group
    q = c.wide_q.cuda()[:, :hq]
    out = torch.full((c.n, hq + 1, c.d), PAD, dtype=c.dtype, device="cuda")
    lse = torch.full((c.n, hq), PAD, device="cuda")
    w = ws(kv8.attend_workspace(cache, batch, c.n, hq))
    kv8.attend(cache, batch, q, out[:, :hq], scale, window=window, flags=kv8.CAUSAL if causal else 0, lse=lse,
               workspace=w)
    torch.cuda.synchronize()
    assert (out[:, hq] == PAD).all(), "wrote past the heads of out"
    return out[:, :hq], lse


def n_splits(c, max_kv=None):
    """Into how many parts a call splits each row's keys: its workspace has head_dim + 2 floats of each."""
    hq = c.h * c.group
    need = kv8.attend_workspace(kv8.Cache(*c.pools8()), gpu_batch(c, max_kv=max_kv), c.n, hq)
    return need // (c.n * hq * (c.d + 2) * 4)


def wider_table(c, max_kv):
    """The case's page table with room for max_kv tokens; the pages past its own are not there."""
    room = -(-max_kv // c.page)
    if c.table.shape[1] < room:
        more = torch.full((c.table.shape[0], room - c.table.shape[1]), -1, dtype=torch.int32)
        c.table = torch.cat([c.table, more], 1)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_len", [1, 20])
def test_values_are_exact(dtype, q_len):
    """Every code with exponents over the type's range: a row that sees one key gives its value itself."""
    d, h = 256, 4
    exps = list(range(103, 136)) if dtype is F16 else list(range(1, 247, 3)) + [0, 246]
    c = K8.Case8([(q_len, 1)] * len(exps), dtype=dtype, h=h, group=1, d=d, page=16, block=4, extra=3)
    bits = torch.arange(256, dtype=torch.int64)
    for i, e in enumerate(exps):
        for hh in range(h):
            c.v8.view(torch.uint8)[int(c.table[i, 0]), 0, hh] = ((bits * (2 * hh + 1)) % 256).to(torch.uint8)
            c.ve[int(c.table[i, 0]), 0, hh] = e
    c.renew()
    log(f"exact values {dtype} q={q_len}")
    out, _ = run_attend(c, 0.1, causal=False)
    # (bf16: a weight of 2^-32 times a value below 2^-94 is below fp32's normal numbers)
    most, least = (65504.0, 2.0 ** -20) if dtype is F16 else (3.4e38, 2.0 ** -94)
    for i in range(len(exps)):
        want = c.v[int(c.table[i, 0]), 0].clamp(-most, most)
        for r in range(q_len):
            got = out[i * q_len + r].cpu().double()
            same = (got == want) | (torch.isnan(got) & torch.isnan(want))
            small = want.abs() < least
            assert same[~small].all(), (exps[i], got[~same & ~small][:5], want[~same & ~small][:5])
            step = 2.0 ** -24 if dtype is F16 else least
            assert ((got - want).abs()[small] <= step).all()


ATTEND_LENS = [(1, 1), (3, 3), (0, 0), (17, 64), (1, 65), (2, 200), (0, 31), (130, 300), (66, 66)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,group,page,block", [
    (16, 1, 1, 16, 16), (48, 2, 3, 8, 8), (64, 2, 4, 16, 16), (80, 1, 2, 24, 8), (96, 2, 1, 1, 1), (128, 2, 8, 16, 16),
    (128, 1, 5, 64, 32), (144, 1, 2, 16, 4), (192, 2, 2, 32, 32), (256, 1, 20, 16, 16)])
def test_attend(dtype, d, h, group, page, block):
    c = K8.Case8(ATTEND_LENS, dtype=dtype, h=h, group=group, d=d, page=page, block=block, strange=True,
                 fill=math.nan, tail_rows=3, head_major=page == 16)
    scale = 1 / math.sqrt(d)
    for causal, window in ((True, 0), (True, 1), (True, 50), (False, 0)):
        log(f"attend {dtype} d={d} h={h} group={group} page={page} block={block} causal={causal} window={window}")
        out, lse = run_attend(c, scale, causal, window)
        K.check_attention(c, out, lse, K.attention(c, scale, causal=causal, window=window),
                          f"causal={causal} window={window}")
        assert (out[c.n - 3:] == PAD).all() and (lse[c.n - 3:] == PAD).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,h,group,page,block", [
    (64, 2, 1, 16, 16), (80, 1, 4, 24, 24), (96, 4, 2, 16, 8), (128, 2, 4, 16, 16), (128, 1, 16, 1, 1),
    (128, 4, 8, 64, 16), (192, 1, 17, 64, 64), (256, 1, 3, 32, 16), (256, 4, 2, 16, 16)])
def test_attend_single_tokens(dtype, d, h, group, page, block):
    """One new token a sequence, from one key to several splits of the keys."""
    lens = [(1, n) for n in (1, 2, 15, 16, 17, 31, 64, 65, 127, 257, 1000, 2049)] + [(0, 0), (1, 700)]
    c = K8.Case8(lens, dtype=dtype, h=h, group=group, d=d, page=page, block=block, strange=True, fill=math.nan,
                 tail_rows=1)
    scale = 0.7 / math.sqrt(d)
    for causal, window, max_kv in ((True, 0, None), (True, 33, None), (False, 0, None), (True, 0, 20000)):
        if max_kv:
            wider_table(c, max_kv)
        log(f"single tokens {dtype} d={d} group={group} page={page} window={window} max_kv={max_kv}")
        out, lse = run_attend(c, scale, causal, window, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, scale, causal=causal, window=window),
                          f"window={window} max_kv={max_kv}")
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q_len,d,h,group,page", [
    (2, 128, 2, 8, 16), (3, 64, 4, 8, 16), (5, 128, 8, 4, 16), (4, 96, 1, 8, 24), (9, 192, 4, 3, 16), (6, 256, 1, 5, 64),
    (17, 128, 4, 1, 16), (32, 64, 1, 1, 16), (33, 128, 2, 1, 16), (11, 128, 4, 3, 32), (5, 128, 4, 8, 16),
    (8, 64, 4, 8, 16), (64, 96, 1, 1, 16), (65, 80, 4, 1, 16), (9, 128, 1, 7, 8)])
def test_attend_drafted_tokens(dtype, q_len, d, h, group, page):
    """Some new tokens of each sequence, around the sizes at which another way of running them begins;
    unsplit and in splits."""
    lens = [(q_len, n) for n in (q_len, q_len + 1, 64, 65, 200, 700, 1300)] + [(0, 9), (1, 500), (max(1, q_len - 1), 90)]
    c = K8.Case8(lens, dtype=dtype, h=h, group=group, d=d, page=page, block=page // 2, strange=True, fill=math.nan,
                 tail_rows=2)
    c.table[4, 3 % c.table.shape[1]] = -1
    wider_table(c, 20000)
    scale = 1 / math.sqrt(d)
    for causal, window, max_kv in ((True, 0, None), (True, 70, None), (False, 0, None), (True, 0, 20000)):
        log(f"drafts {dtype} q={q_len} d={d} h={h} group={group} causal={causal} window={window} max_kv={max_kv}")
        out, lse = run_attend(c, scale, causal, window, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, scale, causal=causal, window=window),
                          f"causal={causal} window={window} max_kv={max_kv}")
        assert (out[c.n - 2:] == PAD).all() and (lse[c.n - 2:] == PAD).all()


@pytest.mark.parametrize("q", [1, 2, 5, 40, 200])
def test_attend_bad_pages_and_lengths(q):
    """Pages that are not there (ids of every wrong kind), lengths past the bounds given, rows
    at positions before the first token."""
    lens = [(q, 400), (q, 170), (q, q - 1 if q < 3 else q // 2), (q, 250)]
    c = K8.Case8(lens, d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    for s, p, bad in ((0, 0, -1), (0, 7, c.n_pages), (0, 24, 1 << 30), (1, 3, -(1 << 31)),
                      (3, 15, -5), (3, 14, -5), (3, 13, c.n_pages + 7)):
        c.table[s, p] = bad
    log(f"bad pages q={q}")
    out, lse = run_attend(c, 0.125)
    K.check_attention(c, out, lse, K.attention(c, 0.125), f"q={q}")
    c.table[0] = -1  # a sequence whose pages are all missing
    out, lse = run_attend(c, 0.125)
    K.check_attention(c, out, lse, K.attention(c, 0.125), f"q={q}: no page")
    # tokens past max_kv are not read, new tokens past max_q are left as they were
    c = K8.Case8([(q, 400), (q, 170)], d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    out, lse = run_attend(c, 0.125, causal=False, max_kv=300)
    ref = K8.Case8([(q, 400), (q, 170)], d=64, h=2, group=2, page=16, fill=math.nan, seed=q)
    cut = ref.keys
    ref.keys = lambda s, upto=None: cut(s, 300)
    K.check_attention(c, out, lse, K.attention(ref, 0.125, causal=False), f"q={q}: max_kv")
    if q > 1:
        out, lse = run_attend(c, 0.125, max_q=q - 1)
        assert (out[q - 1] == PAD).all() and (out[2 * q - 1] == PAD).all()
        want = K.attention(c, 0.125)
        want[4][[q - 1, 2 * q - 1]] = False
        K.check_attention(c, out, lse, want, f"q={q}: max_q")


@pytest.mark.parametrize("q_len,h,group", [(1, 1, 2), (1, 4, 3), (3, 2, 4), (5, 4, 4), (2, 8, 1), (40, 1, 2), (70, 4, 1)])
def test_attend_nan_in_any_split(q_len, h, group):
    """NaN values whose weight rounds to zero in 32 bits, in the largest score's split, in others and in
    masked places; a NaN key: the rows that see them, and no others, carry them, wherever the keys are split."""
    n, d, page = 1500, 16, 16
    for max_kv in (None, 9000, 90000):
        c = K8.Case8([(q_len, n), (q_len, 700)], dtype=BF16, d=d, h=h, group=group, page=page, seed=q_len)
        if max_kv:
            wider_table(c, max_kv)
        c.q[..., 0] = 1.0
        at = lambda s, j: (int(c.table[s, j // page]), j % page)  # noqa: E731
        k8, v8 = c.k8.view(torch.uint8), c.v8.view(torch.uint8)
        k8[..., 0] = 0
        for s, j in ((0, 777), (1, 3)):  # the largest scores: a code of 448 in a channel of its own
            k8[at(s, j)][:, 0] = 0x7E
        for i, j in enumerate((5, 70, 760, 780, 1100, n - 1, n - 2, n - 30, 698)):
            for s in range(2):
                if j < c.lens[s][1]:
                    v8[at(s, j)][:, i + 1] = 0x7F if i % 2 else 0xFF
        c.renew()
        splits = n_splits(c, max_kv)
        log(f"NaN in {splits} splits, q={q_len} h={h} group={group}")
        assert max_kv is None or splits > (8 if max_kv == 90000 else 1)
        for causal, window in ((False, 0), (True, 0), (True, 500)):
            out, lse = run_attend(c, 8.0, causal, window, max_kv=max_kv)
            K.check_attention(c, out, lse, K.attention(c, 8.0, causal=causal, window=window),
                              f"{splits} splits, causal={causal} window={window}")
        k8[at(0, n - 1)][:, 2] = 0x7F
        c.renew()
        out, lse = run_attend(c, 1.0, True, 0, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, 1.0), f"{splits} splits, a NaN key")


@pytest.mark.parametrize("dtype,d,h,group,page", [
    (BF16, 64, 2, 2, 16), (F16, 128, 1, 4, 24), (BF16, 128, 2, 1, 64), (F16, 96, 1, 2, 16),
    (BF16, 192, 1, 2, 16), (F16, 256, 1, 2, 32), (BF16, 48, 1, 4, 8)])
def test_attend_chunks_in_splits(dtype, d, h, group, page):
    """Chunks whose keys are split over workgroups, into few parts and into many: causal,
    windowed and open masks, sequences that have no keys in most of the splits, a split whose pages are
    all missing, rows behind the last sequence left as they were."""
    c = K8.Case8([(50, 1500), (0, 0), (33, 700), (24, 1100), (1, 64), (60, 60)], dtype=dtype, d=d, h=h,
                 group=group, page=page, block=page // 2, strange=True, fill=math.nan, tail_rows=2, seed=d + group)
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


@pytest.mark.parametrize("q_len,h", [(1, 1), (2, 4), (40, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attend_ends_of_the_range(dtype, q_len, h):
    """Values and keys at the upper and lower end of the rows' type, all equal and mixed; scales of both signs and zero."""
    for e, code in ((135, 0x78), (135, 0x70), (1, 0x7E), (112, 0x01)) if dtype is F16 else \
            ((246, 0x7E), (245, 0x70), (12, 0x7E), (140, 0x01)):
        c = K8.Case8([(q_len, 300), (q_len, 77)], dtype=dtype, d=64, h=h, group=2, page=16)
        c.v8.view(torch.uint8)[:] = code
        c.ve[:] = e
        c.ke[:] = 100  # scores near zero: equal weights
        c.renew()
        c.v.clamp_(-65504 * 2 if dtype is F16 else -3.4e38, 65504 * 2 if dtype is F16 else 3.4e38)
        log(f"ends {dtype} q={q_len} h={h} e={e} code={code}")
        out, lse = run_attend(c, 0.01)
        ref = list(K.attention(c, 0.01))
        if dtype is F16:
            # a mean within the type's range; each value is read as the half of itself, which fp16's
            # least step, 2^-24, rounds by up to 2^-25: up to 2^-24 of the value, and of a mean of them
            ref[0], ref[2] = ref[0].clamp(-65504, 65504), ref[2] + 2.0 ** -24
        K.check_attention(c, out, lse, ref, f"e={e}")
    if dtype is F16:  # past twice the type's range: infinities, of the rows that see them
        c = K8.Case8([(q_len, 300), (q_len, 77)], dtype=dtype, d=64, h=h, group=2, page=16)
        for s, (_, n) in enumerate(c.lens):
            for j, code in ((0, 0x38), (n - 1, 0xB8), (n - 1 - q_len // 2, 0x38), (3, 0xB0)):
                at = int(c.table[s, j // 16]), j % 16
                c.ve[at[0]] = 144
                c.v8.view(torch.uint8)[at[0]] &= 0x80  # (the block's others are zeros)
                c.v8.view(torch.uint8)[at][..., j % 60] = code
        c.renew()
        c.v[c.v.abs() > 131000] *= math.inf  # 2^17; 2^16 is read as it is
        log(f"past the range {dtype} q={q_len} h={h}")
        for window in (0, 60):
            out, lse = run_attend(c, 0.1, window=window)
            K.check_attention(c, out, lse, K.attention(c, 0.1, window=window), "past the range")
    for scale in (0.0, -0.3, 5.0):
        c = K8.Case8([(q_len, 300), (q_len, 77)], dtype=dtype, d=64, h=h, group=2, page=16, strange=True)
        log(f"scale {scale}")
        out, lse = run_attend(c, scale)
        K.check_attention(c, out, lse, K.attention(c, scale), f"scale={scale}")


@pytest.mark.parametrize("n_seqs,h,q_len", [(3, 4, 1), (64, 4, 2), (65, 1, 1), (200, 4, 1), (300, 1, 3), (1024, 1, 1),
                                            (1030, 1, 1)])
def test_attend_keys_shared_out(n_seqs, h, q_len):
    """Sequences of very different lengths, some without rows or keys, whose keys are shared out over
    workgroups: up to 64 sequences, more, and more than are shared out."""
    rng = torch.Generator().manual_seed(n_seqs)
    lens = []
    for s in range(n_seqs):
        r = int(torch.randint(0, 10, (1,), generator=rng))
        kv = int(torch.randint(1, 120, (1,), generator=rng))
        lens.append({0: (0, kv), 1: (min(q_len, 1), 0), 2: (q_len, q_len)}.get(r, (q_len, q_len + kv)))
    lens[n_seqs // 2], lens[0] = (q_len, 1500), (1, 700)
    c = K8.Case8(lens, dtype=BF16, h=h, group=2, d=16, page=16, strange=True, fill=math.nan, tail_rows=1, seed=n_seqs)
    for causal, window, max_kv in ((True, 0, None), (True, 200, None), (False, 0, 30000)):
        if max_kv:
            wider_table(c, max_kv)
        log(f"keys shared out: {n_seqs} sequences, h={h} q={q_len} causal={causal} window={window}")
        out, lse = run_attend(c, 0.25, causal, window, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, 0.25, causal=causal, window=window), f"window={window}")
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()


@pytest.mark.parametrize("dtype,n_seqs,h,group,d,most", [
    (BF16, 1, 1, 4, 128, 60), (F16, 3, 2, 3, 64, 130), (BF16, 5, 8, 8, 128, 8), (F16, 20, 2, 2, 80, 100),
    (BF16, 34, 1, 2, 64, 70), (F16, 70, 2, 1, 128, 140), (BF16, 9, 4, 2, 256, 70), (BF16, 100, 2, 12, 16, 3)])
def test_chunk_keys_shared_out(monkeypatch, dtype, n_seqs, h, group, d, most):
    """Chunks of very different lengths against contexts of very different lengths, one or more tiles of rows,
    most without rows in some cases, whose keys are shared out over workgroups; a workspace of all ones."""
    monkeypatch.setitem(globals(), "ws", lambda n: torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda"))
    rng = torch.Generator().manual_seed(n_seqs)
    lens = [(int(torch.randint(0, 1 + (most if s % 3 == 0 else 3), (1,), generator=rng)),
             int(torch.randint(0, 300, (1,), generator=rng))) for s in range(n_seqs)]
    lens = [(q, q + kv if s % 7 else kv) for s, (q, kv) in enumerate(lens)]  # (some with fewer keys than rows)
    lens[n_seqs // 2] = (most, 3000)
    c = K8.Case8(lens, dtype=dtype, h=h, group=group, d=d, page=16, strange=True, fill=math.nan, tail_rows=1,
                 seed=n_seqs)
    for causal, window, max_kv in ((True, 0, None), (True, 1100, None), (False, 0, 9000)):
        if max_kv:
            wider_table(c, max_kv)
        log(f"chunks shared out: {n_seqs} sequences, h={h} group={group} d={d} causal={causal} window={window}")
        out, lse = run_attend(c, 0.125, causal, window, max_kv=max_kv)
        K.check_attention(c, out, lse, K.attention(c, 0.125, causal=causal, window=window), f"window={window}")
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()


@pytest.mark.parametrize("q_len", [1, 40])
def test_windows_where_the_longest_context_has_the_largest_length(q_len):
    """So many sequences of up to 2^30 tokens that their keys are not shared out: no workspace, with a window either."""
    c = K8.Case8([(q_len, q_len + 40 + 5 * (s % 50)) for s in range(128)], dtype=BF16, h=1, group=1, d=16, page=1024,
                 block=16, seed=q_len)
    wide = torch.full((128, (1 << 30) // 1024), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table.cuda()
    batch = kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), wide, c.max_q, 1 << 30)
    cache, q = kv8.Cache(*c.pools8()), c.wide_q.cuda()[:, :1]
    assert kv8.attend_workspace(cache, batch, c.n, 1) == 0
    for window in (0, 1024, 30):
        out = torch.full((c.n, 1, c.d), PAD, dtype=BF16, device="cuda")
        lse = torch.full((c.n, 1), PAD, device="cuda")
        log(f"largest length q={q_len} window={window}")
        kv8.attend(cache, batch, q, out, 0.25, lse=lse, window=window)
        torch.cuda.synchronize()
        K.check_attention(c, out, lse, K.attention(c, 0.25, window=window), f"window={window}")


@pytest.mark.parametrize("q_len", [1, 2, 40])
def test_attend_many_small_weights(q_len):
    """Thousands of weights far below the largest one: their sum counts, in fp16 too."""
    n = 6000
    for dtype in (F16, BF16):
        c = K8.Case8([(q_len, n)], dtype=dtype, d=64, h=1, group=2, page=16)
        c.q[:], c.q[..., 0] = 0.0, 1.0
        c.k8.view(torch.uint8)[:] = 0
        c.ke[:] = 127
        c.k8.view(torch.uint8)[int(c.table[0, 3]), 5, 0, 0] = torch.tensor(16.0).to(K8.E4M3).view(torch.uint8)
        c.renew()
        log(f"small weights {dtype} q={q_len}")
        out, lse = run_attend(c, 1.0)
        K.check_attention(c, out, lse, K.attention(c, 1.0), str(dtype))


@pytest.mark.parametrize("n_seqs", [2, 64, 65])
def test_chunks_of_many_sequences(n_seqs):
    """Chunks against longer contexts, up to 64 sequences (the longest first) and more."""
    lens = [(3 + 7 * (s % 5), 60 + 13 * (s * 37 % 50)) for s in range(n_seqs)]
    lens[0] = (40, 300)
    c = K8.Case8(lens, dtype=BF16, h=1, group=2, d=64, page=16, fill=math.nan, seed=n_seqs)
    log(f"chunks of {n_seqs} sequences")
    out, lse = run_attend(c, 0.125)
    K.check_attention(c, out, lse, K.attention(c, 0.125), f"{n_seqs}")


@pytest.mark.parametrize("q_len", [1, 5, 50])
def test_pages_beyond_32_bit_offsets(q_len):
    """A pool of more than 2^32 bytes, its pages used at both ends: append, then attention."""
    page, h, d = 64, 8, 128
    n_pages = (1 << 32) // (page * h * d) + 40
    big = [torch.empty((n_pages, page, h, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
    exps = [torch.zeros((n_pages, 4, h), dtype=torch.uint8, device="cuda") for _ in "kv"]
    c = K8.Case8([(q_len, 900), (q_len, 333)], dtype=BF16, d=d, h=h, group=2, page=page, block=16)
    c.max_rows = c.most_kv = 1 << 30
    where = torch.arange(c.n_pages)
    where = torch.where(where % 2 == 0, n_pages - 1 - where, where)  # page of the small pool -> here
    log(f"far pages q={q_len}")
    for b, e, codes, ex in zip(big, exps, (c.k8, c.v8), (c.ke, c.ve)):
        b[where.cuda()] = codes.view(torch.uint8).cuda()
        e[where.cuda()] = ex.cuda()
    far = torch.where(c.table >= 0, where[c.table.clamp(min=0).long()].int(), c.table)
    cache = kv8.Cache(*(x.view(K8.E4M3) for x in big), *exps)
    batch = kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), far.cuda(), q_len, 900)
    assert int(far.max()) * page * h * d > 1 << 32
    rows = torch.randn((c.n, 2 * h, d), generator=torch.Generator().manual_seed(1)).to(BF16)
    gpu = rows.cuda()
    kv8.append(cache, batch, gpu[:, :h], gpu[:, h:])
    placed, _ = placed_rows(c)
    x = rows.double()
    ref = K8.append(c, x[:, :h], x[:, h:], placed)
    got = [b[where.cuda()].cpu().view(K8.E4M3) for b in big] + [e[where.cuda()].cpu() for e in exps]
    check_cache(c, got, ref, 0.0)
    c.k8, c.v8, c.ke, c.ve = got
    c.renew()
    q = c.wide_q.cuda()[:, :2 * h]
    out = torch.zeros((c.n, 2 * h, d), dtype=BF16, device="cuda")
    lse = torch.zeros((c.n, 2 * h), device="cuda")
    kv8.attend(cache, batch, q, out, 0.1, lse=lse, workspace=ws(kv8.attend_workspace(cache, batch, c.n, 2 * h)))
    K.check_attention(c, out, lse, K.attention(c, 0.1), "far pages")


def test_graph_replay_and_streams():
    """Append and attention of single tokens, of drafted ones and of chunks in splits captured, replayed
    with other inputs in the same buffers, eager work between; then attention on two streams at once, each
    with its workspace.  The same bits as eager calls every time."""
    for q_len, group, max_kv in ((1, 4, 928), (5, 4, 928), (40, 2, 6000)):
        c = K8.Case8([(q_len, 900), (q_len, 300), (q_len, 50)], dtype=BF16, d=128, h=2, group=group, page=16)
        wider_table(c, max_kv)
        pools = c.pools8()
        cache, batch, hq = kv8.Cache(*pools), gpu_batch(c, max_kv=max_kv), 2 * group
        start = [p.clone() for p in pools]
        q = c.wide_q.cuda()[:, :hq].contiguous()
        rows = torch.randn((c.n, 4, 128), device="cuda").to(BF16)
        need = kv8.attend_workspace(cache, batch, c.n, hq)
        works = [ws(need) for _ in range(3)]

        def reset():
            for p, s in zip(pools, start):
                p.view(torch.uint8).copy_(s.view(torch.uint8))

        def step(out, lse, work):
            kv8.append(cache, batch, rows[:, :2], rows[:, 2:])
            kv8.attend(cache, batch, q, out, 0.1, lse=lse, workspace=work)
        got, want = ([torch.zeros_like(q), torch.zeros((c.n, hq), device="cuda")] for _ in range(2))
        step(*got, works[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        log(f"capture q={q_len}")
        with torch.cuda.graph(graph):
            step(*got, works[0])
        for rep in range(4):
            q.copy_(torch.randn_like(q))
            rows.copy_(torch.randn_like(rows) * 3 ** rep)
            batch._keep[1].copy_(torch.tensor([900 - 100 * rep, 300 - 77 * rep, 50 - rep]))
            reset()
            step(*want, works[1])
            torch.cuda.synchronize()
            after = [p.view(torch.uint8).clone() for p in pools]
            reset()
            for t in got:
                t.fill_(3)
            works[0].fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), rep
            assert all(torch.equal(p.view(torch.uint8), a) for p, a in zip(pools, after)), rep
            c.k8, c.v8, c.ke, c.ve = [p.view(torch.uint8).cpu() for p in pools]
            c.k8, c.v8 = c.k8.view(K8.E4M3), c.v8.view(K8.E4M3)
            c.renew()
            c.q, c.lens = q.cpu(), [(q_len, x) for x in batch._keep[1].tolist()]
            K.check_attention(c, *got, K.attention(c, 0.1), f"replay {rep}")
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [[torch.zeros_like(q), torch.zeros((c.n, hq), device="cuda")] for _ in range(6)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            kv8.attend(cache, batch, q, o[0], 0.1, lse=o[1], workspace=works[1 + i % 2], stream=streams[i % 2])
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_empty_calls():
    """No rows, no sequences, a cache whose sequences are all empty."""
    c = K8.Case8([(0, 0), (0, 40)], d=64, tail_rows=3)
    pools = c.pools8()
    before = [p.view(torch.uint8).clone() for p in pools]
    cache = kv8.Cache(*pools)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    none = kv.Batch(i32(0), i32(), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 0, 0)
    log("empty calls")
    q = torch.zeros((3, 4, 64), dtype=BF16, device="cuda")
    out = torch.full_like(q, PAD)
    for batch in (none, gpu_batch(c), kv.Batch(c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda(), 2, 48)):
        for n in (0, 3):
            kv8.append(cache, batch, q[:n, :2], q[:n, 2:], q=q[:n], q_out=out[:n])
            kv8.attend(cache, batch, q[:n], out[:n], 1.0, workspace=ws(kv8.attend_workspace(cache, batch, n, 4)))
    torch.cuda.synchronize()
    assert (out == PAD).all()
    assert all(torch.equal(p.view(torch.uint8), b) for p, b in zip(pools, before))
