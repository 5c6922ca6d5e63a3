"""The 8-bit paged K/V cache on the GPU at the ends of what its header allows: values next to the rows'
type's range, scores of any size, batches with far more rows than tokens, more workgroups than one dimension
of a launch takes."""
import math

import pytest
import torch

from host_transfer_amd import kv, kv8
from tests import kv8_case as K8
from tests import kv_case as K
from tests.test_gpu_kv8 import PAD, gpu_batch, log, run_attend, wider_table, ws

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
MOST = torch.finfo(BF16).max


@pytest.mark.parametrize("q_len,h,n", [(1, 1, 300), (2, 4, 300), (1, 4, 3000), (40, 2, 300), (40, 2, 3000)])
def test_bf16_values_next_to_the_range(q_len, h, n):
    """Appended bf16 values past 1.9375 * 2^127 are next to the code of 2^128, which is no bf16 number: they are
    read as what they stand for, and their mean is the type's largest number at most."""
    c = K8.Case8([(q_len, n), (q_len, 77)], dtype=BF16, d=64, h=h, group=2, page=16)
    c.ke[:] = 100  # scores near zero: equal weights
    rows = torch.full((c.n, 2 * h, 64), MOST, dtype=BF16)
    rows[:, :, 1::4] = -MOST
    rows[:, :, 2] = 1.0
    pools = c.pools8()
    cache, batch = kv8.Cache(*pools), gpu_batch(c)
    gpu = rows.cuda()
    kv8.append(cache, batch, gpu[:, :h], gpu[:, h:])
    c.v8, c.ve = pools[1].view(torch.uint8).cpu().view(K8.E4M3), pools[3].cpu()
    c.renew()
    new = c.v[int(c.table[0, (n - 1) // 16]), (n - 1) % 16]
    assert (new[:, 0] == 2.0 ** 128).all() and (new[:, 1] == -2.0 ** 128).all()
    assert torch.equal(c.v8.float()[int(c.table[0, (n - 1) // 16]), (n - 1) % 16, :, 0], torch.full((h,), 256.0))
    for code, e in ((None, 0), (0x78, 247), (0x7E, 247), (0xFE, 247), (0x77, 247), (0x7F, 247)):
        if code is not None:
            c.v8.view(torch.uint8)[:], c.ve[:] = code, e
            c.renew()
        log(f"bf16 ends q={q_len} h={h} n={n} code={code}")
        ref = list(K.attention(c, 0.01))
        ref[0] = ref[0].clamp(-MOST, MOST)
        K.check_attention(c, *run_attend(c, 0.01), ref, f"code={code}")


@pytest.mark.parametrize("q_len,h,n", [(1, 1, 300), (2, 4, 300), (1, 4, 3000), (40, 2, 300), (40, 2, 3000)])
def test_bf16_values_past_the_range(q_len, h, n):
    """Values from twice the type's largest number on: infinities of the rows that see them."""
    c = K8.Case8([(q_len, n), (q_len, 77)], dtype=BF16, d=64, h=h, group=2, page=16, block=1)
    for s, j, code, e in ((0, 5, 0x78, 248), (0, n - 2, 0x7E, 254), (1, 3, 0xFE, 255), (1, 9, 0xF0, 248)):
        at = int(c.table[s, j // 16]), j % 16
        c.v8.view(torch.uint8)[at] = 0
        c.v8.view(torch.uint8)[at][:, (7 * j) % 64] = code
        c.ve[at] = e
    c.renew()
    c.v[c.v.abs() > 1.99 * 2.0 ** 128] *= math.inf  # 0xF0 with 248 is -2^128, read as it is
    for window in (0, 60):
        log(f"bf16 past the range q={q_len} h={h} n={n} window={window}")
        K.check_attention(c, *run_attend(c, 0.1, window=window), K.attention(c, 0.1, window=window), f"window={window}")


@pytest.mark.parametrize("q_len,h,n", [(1, 1, 300), (2, 4, 300), (40, 2, 300)])
@pytest.mark.parametrize("e,code,q", [(247, 0x78, 2.0 ** -124), (247, 0x7E, 2.0 ** -124), (246, 0x7E, 2.0 ** -124),
                                      (1, 0x7E, 2.0 ** 120), (1, 0x40, 2.0 ** 126), (2, 0x7E, 2.0 ** 119),
                                      (3, 0x7E, 2.0 ** 118)])
def test_bf16_keys_at_the_ends(q_len, h, n, e, code, q):
    """Keys next to the upper end of bf16 and of the least exponents, where small and large queries meet them."""
    c = K8.Case8([(q_len, n), (q_len, 77)], dtype=BF16, d=64, h=h, group=2, page=16, block=1)
    c.q[:] = 0
    c.q[..., 0], c.q[..., 1] = q, 1.0
    c.k8.view(torch.uint8)[:], c.ke[:] = 0, 127
    for s, j in ((0, 5), (0, 70), (0, 200), (1, 2), (1, 30)):
        at = int(c.table[s, j // 16]), j % 16
        c.k8.view(torch.uint8)[at][:, 0] = code + (0x80 if j == 70 else 0)
        c.ke[at] = e
    c.k8.view(torch.uint8)[int(c.table[0, 1]), 0][:, 1] = 0x48  # 4, of a block of exponent 127
    c.renew()
    scale = 0.25 * 64 / abs(float(c.k[int(c.table[0, 0]), 5, 0, 0]) * q)  # scores of 16, -16, 16
    log(f"bf16 keys at the ends q={q_len} h={h} e={e} code={code}")
    K.check_attention(c, *run_attend(c, scale), K.attention(c, scale), f"e={e}")


H = 2.0 ** 24  # scores (in the exponent of 2) are whole numbers from here on


@pytest.mark.parametrize("q_len,h,n", [(1, 1, 300), (2, 4, 300), (1, 4, 3000), (1, 1, 9000), (3, 8, 9000), (40, 2, 300),
                                       (40, 2, 3000), (40, 1, 20000)])
@pytest.mark.parametrize("high", [1.0, 2.0 ** 17, 2.0 ** 20 - 31, 2.0 ** 20, 2.0 ** 22, H - 40, H - 31, H - 16, H - 1, H, H + 1,
                                  H + 40, 2.0 ** 30, 2.0 ** 60])
def test_large_values_under_equal_scores(q_len, h, n, high):
    """Keys that share the largest score, of any size, with values near the type's largest: a mean, wherever the scores
    lie; other keys' scores are far below, in front of and behind them.

    A row's output is the mean of the values whose score is its largest (the others' weights are 0). Weights of
    equal scores are equal; each is rounded to bf16 for the product and not in their sum (u), the sums carry
    (n + 8) U32, the output is rounded once (u); the tolerance is twice their sum, as second-order terms are no
    more than that.  lse: the score carries the rounding of scale * log2(e) (2 U32), of the product, of the base, of ln 2
    and of two products with it: 8 U32 of its magnitude, and the sum's (n + 8) U32."""
    c = K8.Case8([(q_len, n), (q_len, 130)], dtype=BF16, d=16, h=h, group=2, page=16)
    scale = high / math.log2(math.e)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    g = torch.Generator().manual_seed(n)
    # levels of the keys' scores, -scale, 0 or scale: eight by eight at random; -scale but for eight of 0
    levels = [torch.randint(-1, 2, (n // 8 + 1,), generator=g).repeat_interleave(8)[:n], torch.full((130,), -1)]
    levels[1][40:48] = 0
    if high < 100:
        levels = [torch.ones_like(x) for x in levels]
    k8 = c.k8.view(torch.uint8).view(-1, h, 16)
    k8[:] = 0
    for s, level in enumerate(levels):
        j = torch.arange(len(level))
        k8[c.table[s].long()[j // 16] * 16 + j % 16, :, 0] = torch.tensor([0xB8, 0, 0x38], dtype=torch.uint8)[level + 1][:, None]
    c.ke[:] = 127
    c.v8.view(torch.uint8)[:] = torch.where(torch.rand(c.v8.shape, generator=g) < 0.9, 0x7E, 0x70).to(torch.uint8)
    c.ve[:] = 246
    c.renew()
    u, U = torch.finfo(BF16).eps / 2, K.U32
    for window in (0, 33):
        log(f"equal scores q={q_len} h={h} n={n} high={high} window={window}")
        out, lse = run_attend(c, scale, window=window)
        out, lse = out.cpu().double(), lse.cpu().double()
        for r, s, pos in c.rows():
            lv = levels[s]
            lo = max(pos - window + 1, 0) if window else 0
            top = lv[lo:pos + 1].max()
            j = lo + (lv[lo:pos + 1] == top).nonzero().flatten()
            ids = c.table[s].long()[j // 16]
            want = c.v[ids, j % 16].mean(0)  # (h, d)
            want = want.repeat_interleave(2, 0)
            tol = 2 * (2 * u + (n + 8) * U)
            assert ((out[r] - want).abs() <= tol * want).all(), (r, window, float((out[r] / want - 1).abs().max()))
            want_lse = scale * float(top) + math.log(len(j))
            assert ((lse[r] - want_lse).abs() <= 8 * U * abs(scale * float(top)) + (n + 8) * U + 8 * U * abs(want_lse)).all()


def test_few_new_tokens_in_a_batch_of_many_rows():
    """A chunk in a batch whose rows are mostly of no sequence (a buffer of the largest step's size)."""
    c = K8.Case8([(2, 2000)], dtype=BF16, d=16, h=1, group=32, page=16, tail_rows=139_998)
    wider_table(c, 40_000)
    log("few new tokens in a batch of many rows")
    cache, batch = kv8.Cache(*c.pools8()), gpu_batch(c, max_kv=40_000)
    q = c.wide_q.cuda()[:, :32]
    out = torch.full((c.n, 32, 16), PAD, dtype=BF16, device="cuda")
    lse = torch.full((c.n, 32), PAD, device="cuda")
    kv8.attend(cache, batch, q, out, 0.25, lse=lse, workspace=ws(kv8.attend_workspace(cache, batch, c.n, 32)))
    torch.cuda.synchronize()
    K.check_attention(c, out, lse, K.attention(c, 0.25))
    assert (out[2:] == PAD).all() and (lse[2:] == PAD).all()


def test_append_more_blocks_than_a_launch_dimension():
    """2^26 (block, K or V, head)s: a wave each, four to a workgroup, so more workgroups than 2^24 - 1."""
    n, h, d, page = 1 << 19, 64, 16, 64
    n_pages = n // page
    k8, v8 = (torch.full((n_pages, page, h, d), 0x55, dtype=torch.uint8, device="cuda") for _ in "kv")
    ke, ve = (torch.zeros((n_pages, page, h), dtype=torch.uint8, device="cuda") for _ in "kv")
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().cuda()[None]
    batch = kv.Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                     torch.tensor([n], dtype=torch.int32, device="cuda"), table, n, n)
    # one row for all tokens
    one = torch.randn((1, 2 * h, d), generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    rows = one.expand(n, 2 * h, d)
    log("append of 2^26 blocks")
    kv8.append(kv8.Cache(k8.view(K8.E4M3), v8.view(K8.E4M3), ke, ve), batch, rows[:, :h], rows[:, h:])
    torch.cuda.synchronize()
    for codes, exps, x in ((k8, ke, one[0, :h]), (v8, ve, one[0, h:])):
        x = x.double().cpu()
        e = torch.tensor([K8.exponent(float(m)) for m in x.abs().amax(-1)], dtype=torch.uint8)
        want = K8.codes_of(K8.grid(x * torch.exp2(127 - e.double())[:, None])).view(torch.uint8).cuda()
        assert (exps == e.cuda()).all() and (codes == want).all()
