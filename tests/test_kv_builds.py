"""The cache's traced and debug builds (preprocessed only: neither needs a
GPU)."""
import os
import re
import subprocess

import pytest

from speculative_decoding_verification_63_gb300 import _build


def preprocessed(**kw):
    flags = [f for f in _build.compile_flags(**kw) if f.startswith(("-I", "-D", "-std"))]
    src = os.path.join(_build.CSRC, "kvcache.cu")
    return subprocess.run([_build.nvcc(), "-E", "-x", "cu", *flags, src], capture_output=True,
                          text=True, check=True).stdout


@pytest.fixture(scope="module")
def release():
    return preprocessed()


def test_nvtx_build_opens_a_range_per_cache_call(release):
    out = preprocessed(nvtx=True)
    for name in ("sv_kv_write", "sv_kv_read", "sv_kv_attention"):
        assert re.search(r"sv_status\s+" + name + r"\s*\([^{]*\{\s*const\s+SvKvRange\s+sv_range_"
                         r"\s*\(\s*\"" + name + r"\"\s*\)", out), name
    assert "nvtxRangePushA" in out and "SvKvRange" not in release


@pytest.mark.parametrize("what,pattern", [
    ("bulk copies of keys and values, both kernels",
     r"::sv::sv_check\([^;]*bulk_args_ok\(dst, item\.src, item\.bytes\)[^;]*"),
    ("the page table's index, attention", r"::sv::sv_check\([^;]*a_pos >> a\.c\.page_shift"),
    ("the page table's index, write", r"::sv::sv_check\([^;]*slot < a\.c\.slots"),
    ("the page table's index, read", r"::sv::sv_check\([^;]*pos >> a\.c\.page_shift\) < a\.c\.slots"),
    ("a page's rows", r"::sv::sv_check\([^;]*row0 \+ count <= P"),
    ("parts of a cut unit", r"::sv::sv_check\([^;]*last < min\(grid, kKaMaxCtas\)"),
    ("partials", r"::sv::sv_check\([^;]*c < min\(static_cast<int>\(gridDim\.x\), kTcMaxCtas\)"),
])
def test_checks_build_guards_the_caches_accesses(release, what, pattern):
    debug = preprocessed(checks=True)
    found = re.findall(pattern, debug)
    assert len(found) >= (2 if what.startswith("bulk") else 1), what
    assert "::sv::sv_check(" not in release
