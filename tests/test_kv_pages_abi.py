"""The pages' assignment's part of the C ABI on the CPU: exports, and the refusal of bad arguments
with the documented status and a message, before any HIP call."""
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # fake, suitably aligned addresses, P apart: validation never dereferences them


@pytest.fixture(scope="module")
def kv_pages():
    from host_transfer_amd import kv_pages as mod
    return mod


def test_every_declared_function_is_exported(kv_pages):
    text = open(os.path.join(ROOT, "include", "ibp_kv_pages.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*int\s+(ibp_kv_\w+)\s*\(", text, flags=re.M))
    assert names == set(kv_pages.EXPORTED) == {"ibp_kv_assign", "ibp_kv_assign_workspace"}
    from host_transfer_amd import ibp
    out = subprocess.run(["nm", "-D", "--defined-only", ibp.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\bT (ibp_\w+)$", out, flags=re.M))


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "ibp_kv_pages.h"\nint main(void) { ibp_kv_step s; s.n_rows = 0; '
                   'return (int)s.n_rows; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "t.o")],
                   check=True)


def pool(kv_pages, **kw):
    a = dict(page_table=P, free_pages=2 * P, n_pages=100, page_tokens=16, max_pages=8)
    a.update(kw)
    return kv_pages.Pool.from_pointers(**a)


NAMES = ("had", "add", "free_count", "q_start", "kv_len", "length", "free_count_out", "slots")


def call(kv_pages, p=None, **kw):
    a = {n: (3 + i) * P for i, n in enumerate(NAMES)}
    a.update(positions=12 * P, keep=13 * P, unserved=14 * P, n_seqs=5, n_rows=9, stream=0)
    a.update(kw)
    kv_pages.assign(p or pool(kv_pages), *(a.pop(n) for n in NAMES), **a)


def refused(code, fn, *a, **kw):
    from host_transfer_amd import ibp
    with pytest.raises(ibp.IbpError) as e:
        fn(*a, **kw)
    assert e.value.code == code, (e.value.code, ibp.last_error())
    assert ibp.last_error()


def test_refusals(kv_pages):
    from host_transfer_amd import ibp
    for name in NAMES:
        refused(ibp.ERR_NULL, call, kv_pages, **{name: 0})
        refused(ibp.ERR_ALIGN, call, kv_pages, **{name: 30 * P + 2})
    for name in ("positions", "keep", "unserved"):
        refused(ibp.ERR_ALIGN, call, kv_pages, **{name: 30 * P + 2})
    refused(ibp.ERR_ALIGN, call, kv_pages, slots=30 * P + 4)
    for code, kw in ((ibp.ERR_NULL, dict(page_table=0)), (ibp.ERR_NULL, dict(free_pages=0)),
                     (ibp.ERR_ALIGN, dict(page_table=P + 2)), (ibp.ERR_ALIGN, dict(free_pages=2 * P + 1)),
                     (ibp.ERR_SIZE, dict(n_pages=0)), (ibp.ERR_SIZE, dict(n_pages=1 << 31)),
                     (ibp.ERR_SIZE, dict(page_tokens=0)), (ibp.ERR_SIZE, dict(page_tokens=65537)),
                     (ibp.ERR_SIZE, dict(max_pages=1 << 31)), (ibp.ERR_SIZE, dict(table_stride=7)),
                     (ibp.ERR_SIZE, dict(table_stride=(1 << 31) + 1))):
        refused(code, call, kv_pages, pool(kv_pages, **kw))
    refused(ibp.ERR_SIZE, call, kv_pages, n_seqs=(1 << 20) + 1)
    refused(ibp.ERR_SIZE, call, kv_pages, n_rows=1 << 31)
    for kw in (dict(n_seqs=-1), dict(n_rows=-1), dict(n_seqs=1 << 32), dict(n_seqs=None), dict(n_rows=None)):
        with pytest.raises(ValueError):
            call(kv_pages, **kw)
    with pytest.raises(ValueError):
        pool(kv_pages, n_pages=-1)


def test_overlaps(kv_pages):
    """Arrays that overlap are refused, but for length = had and free_count in place."""
    from host_transfer_amd import ibp
    at = {n: (3 + i) * P for i, n in enumerate(NAMES)}
    for name, where in (("q_start", at["had"] + 16), ("kv_len", at["add"]), ("length", at["had"] + 4),
                        ("length", at["add"]), ("slots", at["q_start"] + 16), ("positions", at["slots"] + 64),
                        ("positions", at["slots"] - 64), ("unserved", at["free_count"]), ("kv_len", P + 4 * 39),
                        ("slots", 2 * P + 392), ("free_count_out", at["q_start"] + 20), ("keep", at["kv_len"] + 16),
                        ("length", 13 * P), ("free_count_out", at["had"])):
        refused(ibp.ERR_SIZE, call, kv_pages, **{name: where})
        assert "overlap" in ibp.last_error(), (name, where)
    # side by side; refused for the missing workspace, so that nothing is enqueued
    for kw in (dict(length=at["had"]), dict(free_count_out=at["free_count"]), dict(kv_len=at["q_start"] + 24),
               dict(kv_len=P + 4 * 40), dict(positions=at["slots"] + 8 * 5000)):
        refused(ibp.ERR_NULL, call, kv_pages, n_rows=5000, **kw)
        assert "workspace" in ibp.last_error()


def test_workspace(kv_pages):
    from host_transfer_amd import ibp
    assert kv_pages.assign_workspace(20, 100) == 0
    need = kv_pages.assign_workspace(20, 100_000)
    assert need > 0 and kv_pages.assign_workspace(5000, 1) > need
    refused(ibp.ERR_SIZE, kv_pages.assign_workspace, (1 << 20) + 1, 1)
    refused(ibp.ERR_SIZE, kv_pages.assign_workspace, 1, 1 << 31)
    assert ibp._lib.ibp_kv_assign_workspace(1, 1, None) == ibp.ERR_NULL
    f = ibp._lib.ibp_kv_assign
    step = kv_pages._CStep(3 * P, None, 4 * P, 5 * P, 100_000, 20)
    out = kv_pages._CAssigned(6 * P, 7 * P, 8 * P, 9 * P, None, 10 * P, None)
    for ptr, size, code in ((40 * P, need - 1, ibp.ERR_SIZE), (40 * P + 8, need, ibp.ERR_ALIGN),
                            (None, need, ibp.ERR_NULL)):
        assert f(pool(kv_pages)._c, step, out, ptr, size, None) == code
    for a in ((None, step, out), (pool(kv_pages)._c, None, out), (pool(kv_pages)._c, step, None)):
        assert f(*a, None, 0, None) == ibp.ERR_NULL


def test_tensors_are_checked(kv_pages):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        kv_pages.Pool(torch.zeros(3, 2, dtype=torch.int32), i, 4, 16)
    for name in NAMES + ("positions", "keep", "unserved"):
        with pytest.raises(ValueError, match=f"^{name}: "):
            call(kv_pages, **{name: torch.zeros(9, dtype=torch.float32)})
    p = pool(kv_pages)
    p.device = 99
    with pytest.raises(ValueError, match="pool: on device 99"):
        call(kv_pages, p)


def test_valid_call_without_a_device_reports_a_hip_error(kv_pages):
    if torch.cuda.device_count() > 0:
        pytest.skip("for a machine without a GPU")
    from host_transfer_amd import ibp
    refused(ibp.ERR_HIP, call, kv_pages)
    assert "HIP error" in ibp.last_error()
