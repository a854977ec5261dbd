"""The serving part of the boundary: include/sel/cache_serving.h declares these names and no others, both builds of the
library export them, the binding has their signatures, and the header compiles as C99 with warnings as errors."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sel", "cache_serving.h")
NAMES = ["sel_cache_append", "sel_cache_attention_shared", "sel_cache_attention_shared_workspace_size",
         "sel_cache_attention_window", "sel_cache_attention_window_workspace_size"]

PROGRAM = r"""
#include "sel/cache_serving.h"

int main(void)
{
    static char x[256] __attribute__((aligned(256)));
    static float angles[64] __attribute__((aligned(256)));
    int at[4] __attribute__((aligned(16))) = {0, 0, 0, 0};
    sel_cache c = {0};
    sel_rotation r = {0};
    c.data = x, c.dtype = SEL_BF16, c.pages = 1, c.page_size = 4, c.d = 16, c.page_stride = 64, c.row_stride = 16;
    r.table = angles, r.positions = 4, r.stride = 16, r.first = 0, r.rot = 16;
    /* answered before any CUDA call: nothing to do, then one bad argument each */
    if (sel_cache_append(x, SEL_BF16, 0, 16, &c, at, 1, 1, 1, at, SEL_I32, &r, NULL, 0, 0, 0, 0, NULL, NULL, NULL) !=
        SEL_OK) return 1;
    r.rot = 32;
    if (sel_cache_append(x, SEL_BF16, 1, 16, &c, at, 1, 1, 1, at, SEL_I32, &r, NULL, 0, 0, 0, 0, NULL, NULL, NULL) !=
        SEL_EINVAL) return 2;
    if (sel_cache_attention_window(x, 0, 1, 16, 16, &c, at, 1, 1, 1, NULL, 2, 1, 16, 1.0f, x, NULL, NULL, 0, NULL,
                                   NULL) != SEL_OK) return 3;
    if (sel_cache_attention_window(x, 1, 1, 16, 16, &c, at, 1, 1, 1, NULL, 0, 1, 16, 1.0f, x, NULL, NULL, 0, NULL,
                                   NULL) != SEL_EINVAL) return 4;
    if (sel_cache_attention_shared(x, 0, 1, 16, 16, &c, at, 1, 1, 1, NULL, 2, 16, 1.0f, x, NULL, NULL, 0, NULL,
                                   NULL) != SEL_OK) return 5;
    if (sel_cache_attention_shared(x, 1, 1, 16, 16, &c, at, 1, 1, 1, NULL, -1, 16, 1.0f, x, NULL, NULL, 0, NULL,
                                   NULL) != SEL_EINVAL) return 6;
    if (sel_cache_attention_window_workspace_size(0, 1, 16, 16, 1, 1, 4, 2, 0) != 0) return 7;
    return sel_cache_attention_shared_workspace_size(0, 1, 16, 16, 1, 1, 4, 2) == 0 ? 0 : 8;
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
    src, exe = tmp_path / "use_cache_serving.c", tmp_path / "use_cache_serving"
    src.write_text(PROGRAM)
    subprocess.check_call([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                           "-o", str(exe), build.SO, "-Wl,-rpath," + os.path.dirname(build.SO)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
