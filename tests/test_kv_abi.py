"""The paged K/V part of the C ABI on the CPU: exports, and the refusal of bad
arguments with the documented status and a message, before any HIP call."""
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a fake, suitably aligned address: validation never dereferences it


@pytest.fixture(scope="module")
def kv():
    from host_transfer_amd import kv as mod
    return mod


def test_every_declared_function_is_exported(kv):
    text = open(os.path.join(ROOT, "include", "ibp_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*int\s+(ibp_kv_\w+)\s*\(", text, flags=re.M))
    assert len(names) == 8, names
    from host_transfer_amd import ibp
    out = subprocess.run(["nm", "-D", "--defined-only", ibp.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\bT (ibp_\w+)$", out, flags=re.M))
    assert names == set(kv.EXPORTED)


def test_headers_are_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "ibp_kv.h"\nint main(void) { ibp_kv_batch b; b.n_rows = 0; '
                   'return (int)b.n_rows; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "t.o")],
                   check=True)


def refused(code, fn, *a, **kw):
    from host_transfer_amd import ibp
    with pytest.raises(ibp.IbpError) as e:
        fn(*a, **kw)
    assert e.value.code == code, (e.value.code, ibp.last_error())
    assert ibp.last_error()


def cache(kv, **kw):
    a = dict(k=P, v=3 * P, n_pages=10, page_tokens=16, n_heads=2, head_dim=64, dtype=kv.BF16)
    a.update(kw)
    return kv.Cache.from_pointers(**a)


def batch(kv, **kw):
    a = dict(q_start=P, kv_len=P, page_table=P, table_stride=8, n_seqs=3, max_q=4, max_kv=128)
    a.update(kw)
    return kv.Batch.from_pointers(**a)


BAD_CACHES = [("ERR_NULL", dict(k=0)), ("ERR_NULL", dict(v=None)), ("ERR_SIZE", dict(n_pages=0)),
              ("ERR_SIZE", dict(n_pages=1 << 31)), ("ERR_SIZE", dict(page_tokens=0)),
              ("ERR_SIZE", dict(page_tokens=65537)), ("ERR_SIZE", dict(n_heads=0)),
              ("ERR_SIZE", dict(n_heads=65536)), ("ERR_SIZE", dict(head_dim=0)),
              ("ERR_SIZE", dict(head_dim=60)), ("ERR_SIZE", dict(head_dim=264)),
              ("ERR_SIZE", dict(dtype=2)), ("ERR_ALIGN", dict(k=P + 8)), ("ERR_ALIGN", dict(v=P + 2)),
              ("ERR_ALIGN", dict(token_stride=130)), ("ERR_SIZE", dict(token_stride=64)),
              ("ERR_SIZE", dict(page_stride=1024)), ("ERR_SIZE", dict(head_stride=56)),
              ("ERR_SIZE", dict(page_stride=1 << 62)),
              ("ERR_SIZE", dict(token_stride=64, head_stride=1 << 33, page_stride=1 << 40))]


def test_cache_refusals(kv):
    from host_transfer_amd import ibp
    rows = kv.Rows(P, 128, 64, 2)
    for name, kw in BAD_CACHES:
        code = getattr(ibp, name)
        c = cache(kv, **kw)
        refused(code, kv.append, c, rows, rows, P, n_tokens=3, stream=0)
        refused(code, kv.page_bounds, c, batch(kv), P, stream=0)
        refused(code, kv.attend, c, batch(kv), rows, kv.Rows(2 * P, 128, 64, 2), 1.0, n_rows=3, stream=0)


def test_append_refusals(kv):
    from host_transfer_amd import ibp
    c = cache(kv)
    good = kv.Rows(P, 128, 64, 2)
    q = kv.Rows(P, 256, 64, 4)

    def call(code, k=good, v=good, slots=P, **kw):
        refused(code, kv.append, c, k, v, slots, **{**dict(n_tokens=3, stream=0), **kw})
    call(ibp.ERR_NULL, slots=None)
    call(ibp.ERR_NULL, k=kv.Rows(0, 128, 64, 2))
    call(ibp.ERR_SIZE, k=kv.Rows(P, 128, 64, 3))
    call(ibp.ERR_SIZE, v=kv.Rows(P, 128, 64, 1))
    call(ibp.ERR_SIZE, v=kv.Rows(P, 128, 64, 0))
    call(ibp.ERR_ALIGN, k=kv.Rows(P + 8, 128, 64, 2))
    call(ibp.ERR_ALIGN, k=kv.Rows(P, 132, 64, 2))
    call(ibp.ERR_ALIGN, slots=P + 4)
    call(ibp.ERR_NULL, q=q)
    call(ibp.ERR_NULL, q_out=q)
    call(ibp.ERR_SIZE, q=q, q_out=kv.Rows(2 * P, 128, 64, 2))
    call(ibp.ERR_SIZE, q=q, q_out=kv.Rows(2 * P, 248, 64, 4))       # rows of q_out overlap
    call(ibp.ERR_SIZE, q=q, q_out=kv.Rows(P, 512, 64, 4))           # in place with other strides
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=24, n_positions=9)
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=80, n_positions=9)
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=0, n_positions=9)
    call(ibp.ERR_NULL, rope=P, rope_dim=64, n_positions=9)
    call(ibp.ERR_ALIGN, rope=P + 4, positions=P, rope_dim=64, n_positions=9)
    call(ibp.ERR_ALIGN, k_norm=P + 2)
    for eps in (-1e-6, float("nan"), float("inf")):
        call(ibp.ERR_SIZE, k_norm=P, eps=eps)
    call(ibp.ERR_FLAGS, flags=2)
    call(ibp.ERR_SIZE, n_tokens=1 << 31)
    refused(ibp.ERR_SIZE, kv.append, cache(kv, v=P), good, good, P, n_tokens=3, stream=0)  # one pool
    with pytest.raises(ValueError):
        kv.append(c, good, good, P, stream=0)


def test_batch_and_attend_refusals(kv):
    from host_transfer_amd import ibp
    c = cache(kv)
    q, o = kv.Rows(P, 256, 64, 4), kv.Rows(2 * P, 256, 64, 4)

    def call(code, b=None, q=q, out=o, scale=1.0, n_rows=3, **kw):
        refused(code, kv.attend, c, b or batch(kv), q, out, scale, n_rows=n_rows, stream=0, **kw)
    for code, kw in ((ibp.ERR_NULL, dict(q_start=0)), (ibp.ERR_NULL, dict(kv_len=0)),
                     (ibp.ERR_NULL, dict(page_table=0)), (ibp.ERR_ALIGN, dict(q_start=P + 2)),
                     (ibp.ERR_ALIGN, dict(page_table=P + 1)), (ibp.ERR_SIZE, dict(table_stride=7)),
                     (ibp.ERR_SIZE, dict(table_stride=1 << 41))):
        call(code, b=batch(kv, **kw))
        refused(code, kv.page_bounds, c, batch(kv, **kw), P, stream=0)
    for kw in (dict(max_q=-1), dict(max_kv=1 << 31), dict(n_seqs=1 << 31)):
        with pytest.raises(ValueError):
            batch(kv, **kw)
    call(ibp.ERR_NULL, q=kv.Rows(0, 256, 64, 4))
    call(ibp.ERR_NULL, out=kv.Rows(0, 256, 64, 4))
    call(ibp.ERR_SIZE, q=kv.Rows(P, 256, 64, 3))                    # 3 query heads, 2 key heads
    call(ibp.ERR_SIZE, out=kv.Rows(2 * P, 256, 64, 2))
    call(ibp.ERR_SIZE, out=kv.Rows(2 * P, 0, 64, 4))                # rows of out overlap
    call(ibp.ERR_SIZE, out=kv.Rows(P, 256, 64, 4))                  # out = q
    call(ibp.ERR_ALIGN, out=kv.Rows(2 * P + 8, 256, 64, 4))
    call(ibp.ERR_ALIGN, lse=P + 2)
    call(ibp.ERR_SIZE, n_rows=1 << 31)
    call(ibp.ERR_SIZE, n_rows=1 << 22)                              # x 4 heads
    # more workgroups than a launch takes: the largest batch of the longest sequences
    big = batch(kv, n_seqs=1 << 25, table_stride=8)
    if torch.cuda.device_count() > 0:
        call(ibp.ERR_SIZE, b=big)
    for s in (float("nan"), float("inf")):
        call(ibp.ERR_SIZE, scale=s)
    call(ibp.ERR_FLAGS, flags=2)
    call(ibp.ERR_FLAGS, flags=0, window=5)
    refused(ibp.ERR_NULL, kv.page_bounds, c, batch(kv), 0, stream=0)
    refused(ibp.ERR_ALIGN, kv.page_bounds, c, batch(kv), P + 2, stream=0)
    with pytest.raises(ValueError):
        kv.attend(c, batch(kv), q, o, 1.0, stream=0)


def test_scale_past_the_exponents(kv):
    from host_transfer_amd import ibp
    q, o = kv.Rows(P, 256, 64, 4), kv.Rows(2 * P, 256, 64, 4)
    for s in (2.0 ** 127, -3e38):
        refused(ibp.ERR_SIZE, kv.attend, cache(kv), batch(kv), q, o, s, n_rows=3, stream=0)
        refused(ibp.ERR_SIZE, kv.attend_selected, cache(kv), batch(kv), q, P, o, s, n_select=4, n_rows=3,
                stream=0)


def test_select_refusals(kv):
    from host_transfer_amd import ibp
    c = cache(kv)
    q, o = kv.Rows(P, 256, 64, 4), kv.Rows(2 * P, 256, 64, 4)

    def call(code, b=None, bounds=P, q=q, sel=P, n_first=1, n_last=1, n_select=4, n_rows=3,
             n_bounds=10):
        refused(code, kv.select, c, b or batch(kv), bounds, q, sel, n_first=n_first, n_last=n_last,
                n_select=n_select, n_bounds=n_bounds, n_rows=n_rows, stream=0)
    call(ibp.ERR_SIZE, n_last=0)
    call(ibp.ERR_SIZE, n_first=4)
    call(ibp.ERR_SIZE, n_first=2, n_last=3)
    call(ibp.ERR_SIZE, n_first=5)
    call(ibp.ERR_SIZE, n_select=0)
    call(ibp.ERR_SIZE, n_select=4097)
    call(ibp.ERR_NULL, bounds=0)
    call(ibp.ERR_NULL, sel=0)
    call(ibp.ERR_ALIGN, bounds=P + 8)
    call(ibp.ERR_ALIGN, sel=P + 2)
    call(ibp.ERR_SIZE, n_bounds=1 << 31)
    call(ibp.ERR_SIZE, q=kv.Rows(P, 256, 64, 5))
    call(ibp.ERR_NULL)                                              # no workspace: 8 pages, 4 selected
    n = kv.select_workspace(c, batch(kv), 3, 4)
    assert n > 0 and kv.select_workspace(c, batch(kv), 3, 8) == 0
    refused(ibp.ERR_SIZE, kv.select_workspace, c, batch(kv), 3, 0)
    f = kv.attend_selected
    refused(ibp.ERR_SIZE, f, c, batch(kv), q, P, o, 1.0, n_select=0, n_rows=3, stream=0)
    refused(ibp.ERR_NULL, f, c, batch(kv), q, 0, o, 1.0, n_select=4, n_rows=3, stream=0)
    refused(ibp.ERR_ALIGN, f, c, batch(kv), q, P + 2, o, 1.0, n_select=4, n_rows=3, stream=0)


def test_cache_and_batch_on_another_device(kv):
    """Tensors' owners remember their device: a call with another one current is refused."""
    rows, out = kv.Rows(P, 128, 64, 2), kv.Rows(2 * P, 128, 64, 2)
    for on in ("cache", "batch"):
        c, b = cache(kv), batch(kv)
        (c if on == "cache" else b).device = 99
        calls = [lambda: kv.page_bounds(c, b, P, stream=0),
                 lambda: kv.attend(c, b, rows, out, 1.0, n_rows=3, stream=0),
                 lambda: kv.select(c, b, P, rows, P, n_select=4, n_bounds=9, n_rows=3, stream=0),
                 lambda: kv.attend_selected(c, b, rows, P, out, 1.0, n_select=4, n_rows=3, stream=0)]
        if on == "cache":
            calls.append(lambda: kv.append(c, rows, rows, P, n_tokens=3, stream=0))
        for call in calls:
            with pytest.raises(ValueError, match=f"{on}: on device 99"):
                call()


def test_workspace_is_checked(kv):
    """A workspace that is too small or misaligned is refused (through the C call: the binding
    takes tensors only)."""
    import ctypes
    from host_transfer_amd import ibp
    c, b = cache(kv), batch(kv)
    need = kv.select_workspace(c, b, 3, 4)
    q = kv.Rows(P, 256, 64, 4)._c
    f = ibp._lib.ibp_kv_select
    for ptr, size, code in ((P, need - 1, ibp.ERR_SIZE), (P + 8, need, ibp.ERR_ALIGN),
                            (None, need, ibp.ERR_NULL)):
        assert f(c._c, b._c(c, 3), P, 10, q, 1, 1, 4, P, ptr, size, None) == code
    assert f(None, b._c(c, 3), P, 10, q, 1, 1, 4, P, P, need, None) == ibp.ERR_NULL
    assert f(c._c, None, P, 10, q, 1, 1, 4, P, P, need, None) == ibp.ERR_NULL
    assert f(c._c, b._c(c, 3), P, 10, None, 1, 1, 4, P, P, need, None) == ibp.ERR_NULL
    assert ibp._lib.ibp_kv_select_workspace(c._c, b._c(c, 3), 4, None) == ibp.ERR_NULL
    assert ibp._lib.ibp_kv_attend_workspace(c._c, b._c(c, 3), 4, None) == ibp.ERR_NULL
    assert ibp._lib.ibp_kv_attend_selected_workspace(c._c, b._c(c, 3), 4, 4, None) == ibp.ERR_NULL
    assert isinstance(need, int) and isinstance(f, ctypes._CFuncPtr)


def test_tensors_are_checked(kv):
    """What the binding refuses by itself: tensors of another dtype, shape or device."""
    x = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for k, v in ((x, x), (x.float(), x.float()), (x, x[:3]), (x[0], x[0])):
        with pytest.raises(ValueError):
            kv.Cache(k, v)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kv.Batch(i, i[:3], torch.zeros(3, 2, dtype=torch.int32), 1, 16)
    c = cache(kv)
    with pytest.raises(ValueError):
        kv.append(c, torch.zeros(3, 2, 32, dtype=torch.bfloat16), torch.zeros(3, 2, 64), P, stream=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_beside_a_cache_of_pointers_are_checked(kv, dtype):
    """A cache given by addresses has a dtype all the same: rows, bounds and weights that are tensors
    of another one, or in host memory, are refused like those beside a cache of tensors."""
    c, b = cache(kv), batch(kv)
    r, q, o = kv.Rows(P, 128, 64, 2), kv.Rows(P, 256, 64, 4), kv.Rows(2 * P, 256, 64, 4)
    x, y = torch.zeros(3, 2, 64, dtype=dtype), torch.zeros(3, 4, 64, dtype=dtype)
    bounds, w = torch.zeros(10, 2, 2, 64, dtype=dtype), torch.zeros(64, dtype=dtype)
    calls = dict(k=lambda: kv.append(c, x, r, P, n_tokens=3, stream=0),
                 v=lambda: kv.append(c, r, x, P, n_tokens=3, stream=0),
                 q=lambda: kv.append(c, r, r, P, q=y, q_out=o, n_tokens=3, stream=0),
                 q_out=lambda: kv.append(c, r, r, P, q=q, q_out=y, n_tokens=3, stream=0),
                 k_norm=lambda: kv.append(c, r, r, P, k_norm=w, n_tokens=3, stream=0),
                 q_norm=lambda: kv.append(c, r, r, P, q=q, q_out=o, q_norm=w, n_tokens=3, stream=0),
                 bounds=lambda: kv.page_bounds(c, b, bounds, stream=0))
    for call, name in ((lambda: kv.attend(c, b, y, o, 1.0, n_rows=3, stream=0), "q"),
                       (lambda: kv.attend(c, b, q, y, 1.0, n_rows=3, stream=0), "out"),
                       (lambda: kv.select(c, b, P, y, P, n_select=8, n_bounds=9, stream=0), "q"),
                       (lambda: kv.select(c, b, bounds, q, P, n_select=8, n_rows=3, stream=0), "bounds"),
                       (lambda: kv.attend_selected(c, b, y, P, o, 1.0, n_select=8, stream=0), "q"),
                       *((f, n) for n, f in calls.items())):
        with pytest.raises(ValueError, match=f"^{name}: "):
            call()


def test_pointers_need_their_sizes(kv):
    """A rotation table or bounds given by address without their length: refused, not taken as empty
    (no token would be placed)."""
    c, r, q = cache(kv), kv.Rows(P, 128, 64, 2), kv.Rows(P, 256, 64, 4)
    for kw in (dict(rope_dim=64), dict(n_positions=9), {}):
        with pytest.raises(ValueError, match="n_positions and rope_dim"):
            kv.append(c, r, r, P, positions=P, rope=P, n_tokens=3, stream=0, **kw)
    with pytest.raises(ValueError, match="n_bounds"):
        kv.select(c, batch(kv), P, q, P, n_select=8, n_rows=3, stream=0)


def test_out_in_part_over_q(kv):
    """out (or append's q_out) that starts inside q's rows is refused; slices of one buffer that lie
    side by side are not."""
    from host_transfer_amd import ibp
    c, r = cache(kv), kv.Rows(P, 128, 64, 2)
    ts = 1024  # elements, of a row of 16 slices of 64
    bad = [64, -64, 128, 192, ts, -ts, ts + 64, 2 * ts - 64, 2 * ts + 192, 8, -8, 56, ts - 200, -2 * ts + 200]
    good = [256, -256, 512, ts - 256, ts + 256, 3 * ts, 3 * ts + 64, -3 * ts - 192, 9 * ts]
    # three tokens of four heads, and, the heads outermost, four tokens of three heads
    for token_stride, head_stride, heads, tokens in ((ts, 64, 4, 3), (64, ts, 3, 4)):
        q = kv.Rows(P, token_stride, head_stride, heads)
        for d in bad + good:
            o = kv.Rows(P + 2 * d, token_stride, head_stride, heads)
            # what does not overlap is refused for eps and scale, so that nothing is enqueued
            calls = [lambda: kv.append(c, r, r, P, q=q, q_out=o, n_tokens=tokens, eps=-1.0, stream=0)]
            if heads == 4:  # (three are no multiple of the cache's two)
                calls.append(lambda: kv.attend(c, batch(kv), q, o, float("nan"), n_rows=tokens, stream=0))
            for call in calls:
                with pytest.raises(ibp.IbpError) as e:
                    call()
                assert e.value.code == ibp.ERR_SIZE
                assert ("overlap" in ibp.last_error()) == (d in bad), (d, heads, ibp.last_error())


def test_valid_calls_without_a_device_report_a_hip_error(kv):
    """Valid calls that enqueue nothing (no tokens, no rows)."""
    from host_transfer_amd import ibp
    c = cache(kv)
    b = batch(kv, n_seqs=0)
    r, o, q = kv.Rows(P, 128, 64, 2), kv.Rows(2 * P, 256, 64, 4), kv.Rows(P, 256, 64, 4)
    calls = [lambda: kv.append(c, r, r, None, n_tokens=0, stream=0),
             lambda: kv.page_bounds(c, b, P, stream=0),
             lambda: kv.attend(c, b, q, o, 1.0, n_rows=0, stream=0),
             lambda: kv.select(c, b, P, q, None, n_select=8, n_bounds=4, n_rows=0, stream=0),
             lambda: kv.attend_selected(c, b, q, None, o, 1.0, n_select=8, n_rows=0, stream=0)]
    for call in calls:
        if torch.cuda.device_count() > 0:
            call()
            continue
        refused(ibp.ERR_HIP, call)
        assert "HIP error" in ibp.last_error()
