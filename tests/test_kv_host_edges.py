"""Host side of the paged cache at the edges of its documentation, without a GPU: the index
arithmetic of the kernels (csrc/wq_kv.h, compiled here for the CPU) and the argument checks."""
import ctypes
import itertools
import os
import subprocess

import pytest

import gemv_wq_quantize_b200 as wq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include "wq_kv.h"
using namespace wq;
extern "C" {
// item k of an append: page, slot, tokens that are placed, call token
void append_item(int lo, int hi, int len, int M, long long k, int sh, int limit, int *o)
{
    const KvPageSpan p = kv_page_span(kv_append_span(lo, hi, len, M), k, sh);
    o[0] = p.page; o[1] = p.off; o[2] = p.count ? kv_placed(p, sh, limit) : 0; o[3] = p.token; o[4] = p.count;
}
}
"""


@pytest.fixture(scope="module")
def kv(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv")
    (d / "kv.cpp").write_text(HARNESS)
    so = d / "libkv.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "gemv_wq_quantize_b200", "csrc"), str(d / "kv.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.append_item.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("limit", [64, 50])  # a block table's row of 4 pages of 16; a shorter rope table
def test_append_places_tokens_below_the_limit_only(kv, limit):
    """Positions come from the length as it is, beyond the table too: a token is placed in its own page and
    slot if its position is below the limit, and no other place is touched."""
    o = (ctypes.c_int * 5)()
    for n, total in itertools.product((1, 2, 5, 17, 40), (0, 1, 15, 33, 49, 50, 63, 64, 65, 66, 81, 103, 10 ** 6, 2 ** 31 - 1, -5)):
        got = {}
        for k in range(8):
            kv.append_item(3, 3 + n, total, 100, k, 4, limit, o)
            page, off, count, token, _ = o
            for i in range(count):
                assert 0 <= page < 4 and 0 <= off + i < 16 and token + i not in got
                got[token + i] = page * 16 + off + i
        total = max(total, 0)
        assert got == {3 + i: total - n + i for i in range(n) if 0 <= total - n + i < limit}, (n, total)
