"""Attention over the 8-bit paged cache whose keys are split into many parts: every way of joining them, with more
parts than its lanes hold at a time. Into how many parts an item (a sequence, or a tile of 128 of its rows) is
split is read from the workspace: (first place, parts) of each item."""
import math

import pytest
import torch

from host_transfer_amd import kv8
from tests import kv8_case as K8
from tests import kv_case as K
from tests.test_gpu_kv8 import PAD, gpu_batch, log

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def run(c, scale, causal=True, window=0):
    """(out, lse, parts of each item that has rows)."""
    cache, batch, hq = kv8.Cache(*c.pools8()), gpu_batch(c), c.h * c.group
    q = c.wide_q.cuda()[:, :hq]
    out = torch.full((c.n, hq, c.d), PAD, dtype=c.dtype, device="cuda")
    lse = torch.full((c.n, hq), PAD, device="cuda")
    work = torch.full((kv8.attend_workspace(cache, batch, c.n, hq),), 0xFF, dtype=torch.uint8, device="cuda")
    kv8.attend(cache, batch, q, out, scale, window=window, flags=kv8.CAUSAL if causal else 0, lse=lse, workspace=work)
    torch.cuda.synchronize()
    few = c.max_q * c.group <= 32
    tiles = 1 if few else -(-c.max_q * c.group // 128)
    parts = work[:16 * 1024].view(torch.int32)[:2 * tiles * len(c.lens)].view(tiles, -1, 2)[..., 1].cpu()
    have = torch.tensor([[q_len * c.group > 128 * (tiles - 1 - t) for q_len, _ in c.lens] for t in range(tiles)])
    return out, lse, parts[have]


def odd_values(c, s, at):
    """NaN values of sequence s at these positions, in a channel of their own."""
    v8 = c.v8.view(torch.uint8)
    for i, j in enumerate(at):
        v8[int(c.table[s, j // c.page]), j % c.page, :, i + 1] = 0x7F if i % 2 else 0xFF


@pytest.mark.parametrize("dtype,q_len,h,group,d,lens,least", [
    # a wave a row, 64 parts at a time: 3 x 8 heads x 32 rows; one long sequence of 40 heads, 13 rows each
    (BF16, 8, 8, 4, 64, [9000, 300, 70], 65), (F16, 4, 8, 8, 128, [9000, 300, 70], 65),
    (F16, 13, 40, 1, 16, [9000], 65), (BF16, 16, 8, 2, 256, [6000, 100, 50], 65),
    # a workgroup a row, for few rows of many parts: up to 1024 of them
    (BF16, 1, 1, 2, 64, [40000], 129), (F16, 1, 4, 1, 128, [33000], 129), (BF16, 3, 1, 1, 256, [40000], 65),
    # four rows to as many lanes as one takes: 8,192 rows and heads; 4, 8 and 16 parts at a time
    (BF16, 5, 8, 4, 64, [5000] + [120 + 17 * i for i in range(51)], 9),
    (F16, 4, 8, 8, 128, [8000] + [90 + 13 * i for i in range(31)], 9),
    (BF16, 8, 8, 4, 256, [6000] + [60 + 9 * i for i in range(31)], 17)])
def test_few_rows_in_many_parts(dtype, q_len, h, group, d, lens, least):
    c = K8.Case8([(q_len, n) for n in lens], dtype=dtype, h=h, group=group, d=d, page=16, block=16, strange=d < 256,
                 fill=math.nan, tail_rows=1, seed=d + h)
    odd_values(c, 0, [0, 3, lens[0] // 2, lens[0] - 1, lens[0] - 700])
    c.renew()
    for causal, window in ((True, 0), (False, 0), (True, lens[0] - 900)):
        out, lse, parts = run(c, 1 / math.sqrt(d), causal, window)
        log(f"few rows {dtype} q={q_len} h={h} group={group} d={d} causal={causal} window={window}: "
            f"{parts.tolist()[:8]} parts")
        assert int(parts.max()) >= (least if not window else 2) and int(parts.min()) >= 1
        K.check_attention(c, out, lse, K.attention(c, 1 / math.sqrt(d), causal=causal, window=window),
                          f"causal={causal} window={window}")
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()


@pytest.mark.parametrize("dtype,q_len,h,group,d,lens,least", [
    # tiles of 128 rows, four rows to as many lanes as one takes: 4, 8 and 16 parts at a time
    (BF16, 70, 1, 2, 64, [20000, 900], 9), (F16, 70, 1, 2, 128, [20000, 2000], 9), (BF16, 70, 1, 2, 128, [20000], 17),
    (BF16, 50, 1, 3, 256, [20000], 17), (F16, 140, 2, 1, 192, [14000, 100], 17),
    # one tile a sequence: a wave a row, a workgroup a row, four rows to some lanes
    (BF16, 40, 2, 2, 64, [20000, 77, 700, 700], 17), (F16, 40, 1, 1, 128, [24000], 33), (BF16, 33, 1, 1, 256, [24000], 33),
    (BF16, 8, 4, 8, 128, [12000] + [100 + 9 * i for i in range(31)], 9)])
def test_chunks_in_many_parts(dtype, q_len, h, group, d, lens, least):
    c = K8.Case8([(q_len, n) for n in lens], dtype=dtype, h=h, group=group, d=d, page=16, block=8, strange=d < 256,
                 fill=math.nan, tail_rows=1, seed=d + h)
    odd_values(c, 0, [0, 3, lens[0] // 2, lens[0] - 1, lens[0] - 700])
    c.renew()
    for causal, window in ((True, 0), (False, 0), (True, lens[0] - 900)):
        out, lse, parts = run(c, 1 / math.sqrt(d), causal, window)
        log(f"chunks {dtype} q={q_len} h={h} group={group} d={d} causal={causal} window={window}: "
            f"{parts.tolist()[:8]} parts")
        assert int(parts.max()) >= (least if not window else 2) and int(parts.min()) >= 1
        K.check_attention(c, out, lse, K.attention(c, 1 / math.sqrt(d), causal=causal, window=window),
                          f"causal={causal} window={window}")
        assert (out[c.n - 1:] == PAD).all() and (lse[c.n - 1:] == PAD).all()
