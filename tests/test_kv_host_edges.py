"""Host side of the paged cache at the edges of its documentation, without a GPU: the index
arithmetic of the kernels (csrc/wq_kv.h, compiled here for the CPU) and the argument checks."""
import ctypes
import itertools
import os
import random
import re
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
int few_rows(long long M, long long n, int q_heads, int kv_heads, long long idle) { return kv_few_rows(M, n, q_heads, kv_heads, idle); }
long long row_item(int q0, int b, int group, int rows, int few) { return kv_row_item(q0, b, group, rows, few); }
long long tiles(int n, int g, int r) { return kv_tiles(n, g, r); }
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
    lib.few_rows.argtypes = [ctypes.c_longlong] * 2 + [ctypes.c_int] * 2 + [ctypes.c_longlong]
    for f in (lib.row_item, lib.tiles):
        f.restype = ctypes.c_longlong
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


# ---------------------------------------------------------------- which attention kernel
IDLE = 24 * 148


@pytest.mark.parametrize("new,heads,tiled", [
    # a prompt chunk among single tokens: the chunk's rows go to the tile kernel, the others do not
    ([1] * 64 + [900], (32, 32), [900]),
    ([1] * 64 + [900], (8, 8), [900]),
    ([1] * 256 + [512], (32, 8), [512]),
    ([1] * 200 + [2000], (32, 32), [2000]),
    ([1] * 200 + [2000], (4, 4), [2000]),
    ([1] * 64 + [256], (32, 32), [256]),
    ([1] * 31 + [0] * 33 + [900], (32, 32), [900]),          # slots without tokens
    # too few rows for it
    ([1] * 64 + [100], (32, 32), []),
    ([1] * 64 + [32], (32, 8), []),
    ([40], (32, 32), []),
    ([10], (1024, 1024), []),
    # decode and draft batches
    ([1] * 256, (32, 8), []),
    ([1] * 248 + [0] * 8, (32, 32), []),
    ([6] * 64, (32, 32), []),
    ([2] * 512, (32, 32), []),
    ([1] * 4096, (64, 1), [1] * 4096),                       # (64 rows each)
    # prompts
    ([300, 200, 1], (32, 8), [300, 200]),
    ([20] * 16, (32, 32), [20] * 16),
    ([2048, 2048], (32, 8), [2048, 2048]),
])
def test_long_sequences_go_to_the_tile_kernel(kv, new, heads, tiled):
    few = kv.few_rows(sum(new), len(new), *heads, IDLE)
    group = heads[0] // heads[1]
    assert few >= 16 and [n for n in new if n * group > few] == tiled


def test_row_blocks_counted_by_rows_cover_every_long_sequence(kv):
    r = random.Random(0)
    for _ in range(300):
        group, rows, few = r.choice((1, 2, 5, 8)), r.choice((128, 256)), r.choice((16, 111, 444))
        q0 = 0
        for b in range(40):
            n = r.choice((0, 1, 3, 17, 30, 112, 300, 2000))
            first, end = kv.row_item(q0, b, group, rows, few), kv.row_item(q0 + n, b + 1, group, rows, few)
            assert first <= end
            if n * group > few:
                assert end - first >= kv.tiles(n, group, rows)
            q0 += n
    # rows near 2^31
    assert kv.row_item(2 ** 31 - 1, 4095, 1, 256, 16) == (2 ** 31 - 1) // 256 + (2 ** 31 - 1) // 17
    assert kv.row_item(2 ** 28 - 1, 4095, 8, 128, 0) == (2 ** 31 - 8) // 128 + 4095


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from gemv_wq_quantize_b200 import build
    build.build(quiet=True)
    return wq.load_library()


def _calls(lib, cache, batch):
    """The status of an append and of an attention call, nothing of which is launched if they refuse."""
    fake = ctypes.c_void_p(0x10000)
    return (lib.kv_append(fake, wq.WQ_F16, 4, 4, None, 0, 0, 0, fake, cache, batch, None),
            lib.kv_attention(fake, wq.WQ_F16, 4, 4, cache, batch, 1.0, fake, None, 0, None))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_a_table_row_ends_well_below_2_to_the_31(lib, page):
    """The kernels look up to a step of keys past the last one in 32 bits, so the last 1023 positions are
    refused."""
    cache = wq._KVCacheC(0x10000, 0x10000, 0x10000, 0x10000, 8, page, 2, 128, wq.FMT_INT)
    for pages in ((2 ** 31 - 1023) // page + 1, (2 ** 31 - 1) // page):
        batch = wq._KVBatchC(0x10000, 0x10000, 0x10000, 2, pages)
        assert _calls(lib, cache, batch) == (wq.WQ_ERR_INVALID_ARG,) * 2
    batch = wq._KVBatchC(0x10000, 0x10000, 0x10000, 2, (2 ** 31 - 1024) // page)
    assert lib.kv_attention_workspace_size(4, 4, cache, batch) > 0


@pytest.mark.parametrize("format", [wq.FMT_E2M1, 3, -1])
def test_a_cache_holds_int8_or_e4m3(format):
    with pytest.raises(ValueError, match="format"):
        wq.make_kv_cache(4, 16, 2, 128, format=format)


# ---------------------------------------------------------------- order in the kernels
@pytest.mark.parametrize("source", ["wq_kv_attn.cu", "wq_kv_tiles.cu"])
def test_tensor_memory_is_taken_between_the_wait_and_the_next_launch(source):
    """A block that held Tensor Memory while it waited for a kernel that still wanted some would lock both
    up, and so would a next kernel's block that was let in before this one had its own."""
    with open(os.path.join(ROOT, "gemv_wq_quantize_b200", "csrc", source)) as f:
        text = "\n".join(line.split("//")[0] for line in f)
    wait, take, launch = (text.index(w) for w in ("grid_dep_wait();", "tmem_alloc(", "grid_dep_launch();"))
    assert wait < take < launch


@pytest.mark.parametrize("source", ["wq_norm.cu", "wq_kv_append.cu", "wq_kv_attn.cu", "wq_kv_tiles.cu"])
def test_what_a_kernel_ahead_may_write_is_not_read_as_constant(source):
    """These kernels are resident before the ones ahead have ended; the read-only path (__ldg) is for memory
    that nobody writes meanwhile.  Only the rope table (`tab`) is."""
    with open(os.path.join(ROOT, "gemv_wq_quantize_b200", "csrc", source)) as f:
        text = f.read()
    assert all(re.match(r"(reinterpret_cast<const float\d \*>\()?tab \+", rest) for rest in text.split("__ldg(")[1:])
