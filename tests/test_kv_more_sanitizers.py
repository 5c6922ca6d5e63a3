"""Address and undefined-behaviour sanitizers on the argument checks of the pages' assignment and the
8-bit cache's calls (api_kv_pages.hip, api_kv8.hip; host side only), driven by
tests/helpers/kv_more_sanitize_main.c.  Skipped where a GPU is visible: valid calls are for a machine
without one."""
import os

import pytest

from tests.test_sanitizers import ENV, HIPCC, ROOT, _run


def test_host_code_under_asan_ubsan(tmp_path):
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("the no-device calls need a machine without a GPU")
    csrc = os.path.join(ROOT, "host_transfer_amd", "csrc")
    build = os.path.join(ROOT, "host_transfer_amd", "_build")
    apis = ("api", "api_kv8", "api_kv_pages")
    names = sorted(f[:-4] for f in os.listdir(csrc) if f.endswith(".hip") and f[:-4] not in apis)
    objs = [os.path.join(build, f + ".hip.o") for f in names]
    if not all(os.path.exists(o) for o in objs):
        from host_transfer_amd.csrc import build as hb
        hb.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer"]
    for f in apis:
        objs.append(str(tmp_path / (f + "_san.o")))
        _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang",
              "-target-feature", "-Xclang", "-packed-fp32-ops"] + san +
             ["-I", os.path.join(ROOT, "include"), "-I", csrc, "-c", os.path.join(csrc, f + ".hip"), "-o",
              objs[-1]])
    objs.append(str(tmp_path / "main.o"))
    _run([HIPCC, "-x", "c", "-O1", "-g"] + san + ["-I", os.path.join(ROOT, "include"), "-c",
         os.path.join(ROOT, "tests", "helpers", "kv_more_sanitize_main.c"), "-o", objs[-1]])
    exe = str(tmp_path / "kv_san")
    _run([HIPCC, "--offload-arch=gfx950"] + san[:4] + ["-o", exe] + objs)
    r = _run([exe], env=ENV, timeout=120)
    assert "kv sanitizer run ok" in r.stdout and "status" not in r.stdout, r.stdout[-2000:]
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
