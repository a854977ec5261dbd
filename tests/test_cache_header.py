"""The paged cache's part of the boundary: include/sel/cache.h declares these names and no others, both builds of the
library export them, the binding has their signatures, and the header compiles as C99 with warnings as errors."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sel", "cache.h")
NAMES = ["sel_cache_attention", "sel_cache_attention_workspace_size", "sel_cache_gather", "sel_cache_set_wait_limit",
         "sel_cache_write"]

PROGRAM = r"""
#include <stdio.h>
#include "sel/cache.h"

int main(void)
{
    static char x[256] __attribute__((aligned(256)));
    int at[4] __attribute__((aligned(16))) = {0, 0, 0, 0};
    sel_cache c = {0};
    c.data = x, c.dtype = SEL_BF16, c.pages = 1, c.page_size = 4, c.d = 16, c.page_stride = 64, c.row_stride = 16;
    /* answered before any CUDA call: nothing to do, then one bad argument each */
    if (sel_cache_write(x, SEL_F32, 0, 16, at, SEL_I32, &c, NULL, NULL) != SEL_OK) return 1;
    if (sel_cache_write(x, SEL_E4M3, 1, 16, at, SEL_I32, &c, NULL, NULL) != SEL_EINVAL) return 2;
    if (sel_cache_gather(&c, at, 1, 1, 1, at, SEL_I32, 0, 1, 1, x, NULL, NULL) != SEL_OK) return 3;
    if (sel_cache_gather(&c, at, 1, 1, 1, at, SEL_I32, 1, -1, 1, x, NULL, NULL) != SEL_EINVAL) return 4;
    if (sel_cache_attention(x, 0, 1, 16, 16, &c, at, 1, 1, 1, NULL, NULL, 0, 0, 0, 16, 1.0f, x, NULL, NULL, 0, NULL,
                            NULL) != SEL_OK) return 5;
    if (sel_cache_attention(x, 1, 0, 16, 16, &c, at, 1, 1, 1, NULL, NULL, 0, 0, 0, 16, 1.0f, x, NULL, NULL, 0, NULL,
                            NULL) != SEL_EINVAL) return 6;
    c.d = SEL_CACHE_ATTN_MAX_D + 8, c.row_stride = c.d, c.page_stride = 4 * c.d;
    if (sel_cache_attention(x, 1, 1, c.d, c.d, &c, at, 1, 1, 1, NULL, NULL, 0, 0, 0, 16, 1.0f, x, NULL, NULL, 0, NULL,
                            NULL) != SEL_EUNSUPPORTED) return 7;
    if (sel_cache_attention_workspace_size(0, 1, 16, 16, 1, 1, 4, 0, 0) != 0) return 8;
    if (sel_cache_set_wait_limit(-1) != SEL_OK) return 9;
    return SEL_CACHE_GROUP == 128 ? 0 : 10;
}
"""


def test_the_header_declares_these_names():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(sel_[a-z_]+)\s*\(", text))) == NAMES


def test_both_builds_export_them_and_the_binding_has_them():
    from gather_radix_select_gb300 import _native, build
    for path, debug in ((build.SO, False), (build.DEBUG_SO, True)):
        if not os.path.exists(path):
            build.build(debug=debug)
        lib = ctypes.CDLL(path)
        for name in NAMES:
            assert hasattr(lib, name), name
            assert name in _native.SIGNATURES, name


def test_the_header_is_c99_and_answers_without_a_gpu(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    from gather_radix_select_gb300 import build
    if not os.path.exists(build.SO):
        build.build()
    src, exe = tmp_path / "use_cache.c", tmp_path / "use_cache"
    src.write_text(PROGRAM)
    subprocess.check_call([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                           "-o", str(exe), build.SO, "-Wl,-rpath," + os.path.dirname(build.SO)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
