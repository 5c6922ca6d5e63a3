"""The 8-bit paged cache's part of the C ABI on the CPU: exports, and the refusal of bad arguments
with the documented status and a message, before any HIP call."""
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a fake, suitably aligned address: validation never dereferences it
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def kv8():
    from host_transfer_amd import kv8 as mod
    return mod


def test_every_declared_function_is_exported(kv8):
    text = open(os.path.join(ROOT, "include", "ibp_kv8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*int\s+(ibp_kv8_\w+)\s*\(", text, flags=re.M))
    assert names == set(kv8.EXPORTED) == {"ibp_kv8_append", "ibp_kv8_attend", "ibp_kv8_attend_workspace"}
    from host_transfer_amd import ibp
    out = subprocess.run(["nm", "-D", "--defined-only", ibp.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\bT (ibp_\w+)$", out, flags=re.M))


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "ibp_kv8.h"\nint main(void) { ibp_kv8_cache c; c.n_pages = 0; '
                   'return (int)c.n_pages; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "t.o")],
                   check=True)


def refused(code, fn, *a, **kw):
    from host_transfer_amd import ibp
    with pytest.raises(ibp.IbpError) as e:
        fn(*a, **kw)
    assert e.value.code == code, (e.value.code, ibp.last_error())
    assert ibp.last_error()


def cache(kv8, **kw):
    a = dict(k=P, v=3 * P, k_exp=5 * P, v_exp=6 * P, n_pages=10, page_tokens=16, block_tokens=8, n_heads=2, head_dim=64)
    a.update(kw)
    return kv8.Cache.from_pointers(**a)


def batch(kv8, **kw):
    a = dict(q_start=P, kv_len=P, page_table=P, table_stride=8, n_seqs=3, max_q=4, max_kv=128)
    a.update(kw)
    return kv8.Batch.from_pointers(**a)


def append(kv8, c=None, b=None, k=None, v=None, **kw):
    kw = {**dict(n_rows=3, dtype=BF16, stream=0), **kw}
    k, v = (kv8.Rows(P, 128, 64, 2) if x is None else x for x in (k, v))
    kv8.append(c or cache(kv8), b or batch(kv8), k, v, **kw)


def attend(kv8, c=None, b=None, q=None, out=None, scale=1.0, **kw):
    kw = {**dict(n_rows=3, dtype=BF16, stream=0), **kw}
    q = kv8.Rows(P, 256, 64, 4) if q is None else q
    out = kv8.Rows(2 * P, 256, 64, 4) if out is None else out
    kv8.attend(c or cache(kv8), b or batch(kv8), q, out, scale, **kw)


BAD_CACHES = [("ERR_NULL", dict(k=0)), ("ERR_NULL", dict(v=None)), ("ERR_NULL", dict(k_exp=0)),
              ("ERR_NULL", dict(v_exp=0)), ("ERR_SIZE", dict(n_pages=0)),
              ("ERR_SIZE", dict(n_pages=1 << 31)), ("ERR_SIZE", dict(page_tokens=0)),
              ("ERR_SIZE", dict(page_tokens=65537, block_tokens=1)), ("ERR_SIZE", dict(block_tokens=0)),
              ("ERR_SIZE", dict(block_tokens=3)), ("ERR_SIZE", dict(block_tokens=32)), ("ERR_SIZE", dict(n_heads=0)),
              ("ERR_SIZE", dict(n_heads=65536)), ("ERR_SIZE", dict(head_dim=0)),
              ("ERR_SIZE", dict(head_dim=72)), ("ERR_SIZE", dict(head_dim=272)),
              ("ERR_ALIGN", dict(k=P + 8)), ("ERR_ALIGN", dict(v=P + 2)),
              ("ERR_ALIGN", dict(token_stride=136)), ("ERR_SIZE", dict(token_stride=64)),
              ("ERR_SIZE", dict(page_stride=1024)), ("ERR_SIZE", dict(head_stride=48)),
              ("ERR_SIZE", dict(page_stride=1 << 62)),
              ("ERR_SIZE", dict(token_stride=64, head_stride=1 << 33, page_stride=1 << 40))]


def test_cache_refusals(kv8):
    from host_transfer_amd import ibp
    for name, kw in BAD_CACHES:
        code = getattr(ibp, name)
        refused(code, append, kv8, cache(kv8, **kw))
        refused(code, attend, kv8, cache(kv8, **kw))
    for kw in (dict(v=P), dict(v_exp=5 * P)):
        refused(ibp.ERR_SIZE, append, kv8, cache(kv8, **kw))  # one memory for both


def test_append_refusals(kv8):
    from host_transfer_amd import ibp
    q = kv8.Rows(P, 256, 64, 4)

    def call(code, **kw):
        refused(code, append, kv8, **kw)
    call(ibp.ERR_NULL, k=kv8.Rows(0, 128, 64, 2))
    call(ibp.ERR_SIZE, k=kv8.Rows(P, 128, 64, 3))
    call(ibp.ERR_SIZE, v=kv8.Rows(P, 128, 64, 1))
    call(ibp.ERR_SIZE, v=kv8.Rows(P, 128, 64, 0))
    call(ibp.ERR_ALIGN, k=kv8.Rows(P + 8, 128, 64, 2))
    call(ibp.ERR_ALIGN, k=kv8.Rows(P, 132, 64, 2))
    call(ibp.ERR_NULL, q=q)
    call(ibp.ERR_NULL, q_out=q)
    call(ibp.ERR_SIZE, q=q, q_out=kv8.Rows(2 * P, 128, 64, 2))
    call(ibp.ERR_SIZE, q=q, q_out=kv8.Rows(2 * P, 248, 64, 4))       # rows of q_out overlap
    call(ibp.ERR_SIZE, q=q, q_out=kv8.Rows(P, 512, 64, 4))           # in place with other strides
    call(ibp.ERR_SIZE, q=q, q_out=kv8.Rows(P + 128, 256, 64, 4))     # in part over q
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=24, n_positions=9)
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=80, n_positions=9)
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=0, n_positions=9)
    call(ibp.ERR_SIZE, rope=P, positions=P, rope_dim=64, n_positions=1 << 49)
    call(ibp.ERR_NULL, rope=P, rope_dim=64, n_positions=9)
    call(ibp.ERR_ALIGN, rope=P + 4, positions=P, rope_dim=64, n_positions=9)
    call(ibp.ERR_ALIGN, rope=P, positions=P + 4, rope_dim=64, n_positions=9)
    call(ibp.ERR_ALIGN, k_norm=P + 2)
    for eps in (-1e-6, float("nan"), float("inf")):
        call(ibp.ERR_SIZE, k_norm=P, eps=eps)
    call(ibp.ERR_FLAGS, flags=2)
    call(ibp.ERR_SIZE, n_rows=1 << 31)
    for kw in (dict(dtype=None), dict(dtype=torch.float32), dict(n_rows=None), dict(rope=P), dict(rope=P, rope_dim=64)):
        with pytest.raises(ValueError):
            append(kv8, **kw)


def test_batch_and_attend_refusals(kv8):
    from host_transfer_amd import ibp

    def call(code, **kw):
        refused(code, attend, kv8, **kw)
    for code, kw in ((ibp.ERR_NULL, dict(q_start=0)), (ibp.ERR_NULL, dict(kv_len=0)),
                     (ibp.ERR_NULL, dict(page_table=0)), (ibp.ERR_ALIGN, dict(q_start=P + 2)),
                     (ibp.ERR_ALIGN, dict(page_table=P + 1)), (ibp.ERR_SIZE, dict(table_stride=7)),
                     (ibp.ERR_SIZE, dict(table_stride=1 << 41)), (ibp.ERR_SIZE, dict(max_kv=(1 << 30) + 1))):
        call(code, b=batch(kv8, **kw))
        refused(code, append, kv8, b=batch(kv8, **kw))
    call(ibp.ERR_NULL, q=kv8.Rows(0, 256, 64, 4))
    call(ibp.ERR_NULL, out=kv8.Rows(0, 256, 64, 4))
    call(ibp.ERR_SIZE, q=kv8.Rows(P, 256, 64, 3))                    # 3 query heads, 2 key heads
    call(ibp.ERR_SIZE, out=kv8.Rows(2 * P, 256, 64, 2))
    call(ibp.ERR_SIZE, out=kv8.Rows(2 * P, 0, 64, 4))                # rows of out overlap
    call(ibp.ERR_SIZE, out=kv8.Rows(P, 256, 64, 4))                  # out = q
    call(ibp.ERR_SIZE, out=kv8.Rows(P + 128, 256, 64, 4))            # in part over q
    call(ibp.ERR_ALIGN, out=kv8.Rows(2 * P + 8, 256, 64, 4))
    call(ibp.ERR_ALIGN, lse=P + 2)
    call(ibp.ERR_SIZE, n_rows=1 << 31)
    call(ibp.ERR_SIZE, n_rows=1 << 22)                              # x 4 heads
    for s in (float("nan"), float("inf"), 2.0 ** 126, -3e38):
        call(ibp.ERR_SIZE, scale=s)
    call(ibp.ERR_FLAGS, flags=2)
    call(ibp.ERR_FLAGS, flags=0, window=5)
    for kw in (dict(dtype=None), dict(dtype=torch.float64), dict(n_rows=None)):
        with pytest.raises(ValueError):
            attend(kv8, **kw)
    f, c, b, q = ibp._lib.ibp_kv8_attend, cache(kv8), batch(kv8), kv8.Rows(P, 256, 64, 4)._c
    o = kv8.Rows(2 * P, 256, 64, 4)._c
    for bad in (2, 1 << 31):  # a dtype that is none
        assert f(c._c, b._c(c, 3), bad, q, o, 1.0, 0, 1, None, None, 0, None) == ibp.ERR_SIZE
    for args in ((None, b._c(c, 3), 1, q, o), (c._c, None, 1, q, o), (c._c, b._c(c, 3), 1, None, o),
                 (c._c, b._c(c, 3), 1, q, None)):
        assert f(*args, 1.0, 0, 1, None, None, 0, None) == ibp.ERR_NULL
    assert ibp._lib.ibp_kv8_attend_workspace(c._c, b._c(c, 3), 4, None) == ibp.ERR_NULL


def test_another_device(kv8):
    for on in ("cache", "batch"):
        c, b = cache(kv8), batch(kv8)
        (c if on == "cache" else b).device = 99
        for call in (lambda: append(kv8, c, b), lambda: attend(kv8, c, b)):
            with pytest.raises(ValueError, match=f"{on}: on device 99"):
                call()


def test_tensors_are_checked(kv8):
    """What the binding refuses by itself: tensors of another dtype, shape, order or device."""
    x = torch.zeros(4, 16, 2, 64, dtype=torch.float8_e4m3fn)
    e = torch.zeros(4, 2, 2, dtype=torch.uint8)
    for k, v, ke, ve in ((x, x, e, e), (x.view(torch.uint8), x, e, e), (x, x[:3], e, e), (x[0], x[0], e, e)):
        with pytest.raises(ValueError):  # (host tensors, all of them)
            kv8.Cache(k, v, ke, ve)
    y, q = torch.zeros(3, 2, 64, dtype=BF16), torch.zeros(3, 4, 64, dtype=BF16)
    r = kv8.Rows(P, 128, 64, 2)
    for name, call in (("k", lambda: append(kv8, k=y)), ("v", lambda: append(kv8, v=y)),
                       ("k", lambda: append(kv8, k=y.half())), ("q_out", lambda: append(kv8, q=r, q_out=q)),
                       ("k_norm", lambda: append(kv8, k_norm=torch.zeros(64, dtype=BF16))),
                       ("positions", lambda: append(kv8, positions=torch.zeros(3, dtype=torch.int64))),
                       ("q", lambda: attend(kv8, q=q)), ("out", lambda: attend(kv8, out=q)),
                       ("lse", lambda: attend(kv8, lse=torch.zeros(3, 4)))):
        with pytest.raises(ValueError, match=f"^{name}: "):
            call()


def test_valid_calls_without_a_device_report_a_hip_error(kv8):
    """Valid calls that enqueue nothing (no rows, no sequences)."""
    from host_transfer_amd import ibp
    for call in (lambda: append(kv8, b=batch(kv8, n_seqs=0), n_rows=0), lambda: attend(kv8, b=batch(kv8, n_seqs=0), n_rows=0)):
        if torch.cuda.device_count() > 0:
            call()
            continue
        refused(ibp.ERR_HIP, call)
        assert "HIP error" in ibp.last_error()
