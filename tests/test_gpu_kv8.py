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
