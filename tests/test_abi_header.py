"""include/dsel.h compiles alone, as C99 and C11 and C++, with no warning; the cache's fields lie where they did.  CPU only."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

import draft_selection_amd as ds

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

LAYOUT = [str(x) for x in (C.sizeof(ds.CacheArgs), ds.CacheArgs.k_scale.offset, ds.CacheArgs.v_scale.offset)]
SOURCE = r"""
#include "dsel.h"
#include <stdio.h>
int main(void) {
    dsel_cache c = {0};
    uint8_t byte = 0;
    float scale = 1.0f;
    c.k_scale = &scale;
    c.v_block = &byte;
    printf("%d %d %d\n", (int)sizeof(c), (int)((char *)&c.k_scale - (char *)&c), (int)((char *)&c.v_scale - (char *)&c));
    return c.v_scale == 0;
}
"""


@pytest.mark.parametrize("lang,std", [("c", "c99"), ("c", "c11"), ("c", "gnu99"), ("c++", "c++11"), ("c++", "c++17")])
def test_the_header_compiles(tmp_path, lang, std):
    cc = shutil.which("gcc" if lang == "c" else "g++")
    if cc is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "a.out")
    warn = [] if lang == "c" else ["-Wno-missing-field-initializers"]
    r = subprocess.run([cc, "-x", lang, f"-std={std}", "-pedantic-errors", "-Wall", "-Wextra", "-Werror", *warn,
                        "-I", os.path.join(ROOT, "include"), "-o", exe, "-"], input=SOURCE, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe], capture_output=True, text=True).stdout.split() == LAYOUT
