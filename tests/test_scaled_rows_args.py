"""kvx_cache's place for row scales under both of its names, and what the operators make of it, without a GPU."""
import os
import subprocess

import pytest
import torch

from conftest import ROOT
from paged_kv_cache_kvx_gb300 import kvx
from test_cache_args import EINVAL, OK, append, cache
from test_shared_args import read, shared, size

PROGRAM = r"""
#include <stddef.h>
#include <stdio.h>
#include "kvx.h"
int main(void) {
    kvx_cache by_place = {(uint8_t *)0, 0, (const uint64_t *)0, 1, 2, 0, 1, 64, KVX_BF16, 16, 0, 128, 1, 1};
    kvx_cache set = by_place;
%s
    set.reserved = 0;
    set.scale_offset = 48;
    printf("%%d %%d %%d %%d %%u %%u %%d\n", (int)sizeof(kvx_cache), (int)offsetof(kvx_cache, scale_offset),
           (int)offsetof(kvx_cache, reserved), (int)offsetof(kvx_cache, token_stride), set.reserved, (unsigned)by_place.token_stride,
           (int)by_place.v_scale);
    return 0;
}
"""
NAMED = "    kvx_cache named = {.pool = 0, .page_tokens = 16, .reserved = 0, .token_stride = 128}, other = {.scale_offset = 16};\n" \
        "    set.B += named.reserved + other.scale_offset;\n"


@pytest.mark.parametrize("cc", ["gcc -std=c99", "gcc -std=c11", "gcc -std=c17", "g++ -std=c++11", "g++ -std=c++17", "g++ -std=c++20"])
def test_programs_that_name_the_field_either_way(cc, tmp_path):
    src = tmp_path / ("p.c" if cc.startswith("gcc") else "p.cpp")
    src.write_text(PROGRAM % (NAMED if cc.startswith("gcc") or "++20" in cc else ""))
    res = subprocess.run([*cc.split(), "-Wall", "-Wextra", "-Wno-missing-field-initializers", "-Wno-missing-braces", "-pedantic-errors", "-Werror",
                          "-I" + os.path.join(ROOT, "include"), "-o", str(tmp_path / "p"), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    out = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout
    S = kvx.CacheStruct
    assert out.split() == [str(x) for x in (kvx.ctypes.sizeof(S), S.scale_offset.offset, S.scale_offset.offset, S.token_stride.offset,
                                            48, 128, 1)]


def test_python_names_the_field_either_way():
    for c in (kvx.CacheStruct(scale_offset=64), kvx.CacheStruct(reserved=64)):
        assert c.reserved == c.scale_offset == 64
        c.reserved = 32
        assert c.scale_offset == 32


def quantised(scale_offset):
    """A cache in host memory, whose address is not that of anything on a device: nothing here gets that far."""
    raw = torch.zeros((1 << 16) + 16, dtype=torch.uint8)
    pool = raw[-raw.data_ptr() % 16:][:1 << 16]
    return kvx.Cache(pool, torch.zeros(4, 4, dtype=torch.int64), heads=2, dim=64, dtype=torch.float8_e4m3fn, page_tokens=16,
                     scale_offset=scale_offset)


def test_the_library_sees_where_the_scales_are():
    """16 rows of 64 bytes: from byte 1024 on they are behind the rows, before that they are not."""
    for place, what in ((0, OK), (1024, OK), (1024 + 16, OK), (1024 - 16, EINVAL), (1024 + 8, EINVAL), (16, EINVAL)):
        c = quantised(place).c
        assert append(c, cs=None, rot=0) == read(c) == shared(c) == what
        assert (size(c) > 0) == (what == OK)


@pytest.mark.parametrize("dim", [16, 64, 128, 144, 256])
def test_scratch_is_what_the_header_says(dim):
    """Equal, but for rounding to 256 bytes, where a call has 128 rows and more and work for every SM; no more than that where not."""
    heads, c = 8, cache(dim=dim, token_stride=2 * dim)
    # (without a GPU the library counts one)
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1
    for n, group, groups, per, pper in ((128, 8, 1, 100, 50), (1024, 8, 1, 100, 50), (8192, 8, 3, 100, 50), (300, 7, 40, 1, 1000),
                                        (1, 1, 0, 1, 0), (3, 16, 2, 1, 1), (16, 128, 16, 100, 100)):
        got = size(c, n=n, hq=heads * group, per=per, groups=groups, pper=pper)
        if dim <= 128:
            rows = 2 * group * (n * heads + sms) + (256 * ((n * group // 256 + groups) * (heads + 2) + 2 * sms) if groups else 0)
        else:
            rows = group * (n * heads + sms) + (128 * ((n * group // 128 + groups) * (heads + 2) + 2 * sms) if groups else 0)
        said = rows * (dim + 2) * 4 + 8 * groups + 8 * n * heads
        assert got <= said + 4 * 256
        if n * group >= 128 and per * n > 100:
            assert got >= said
