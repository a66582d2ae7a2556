"""Host side of the layer operators (rmsnorm_quant_*, kv_append, kv_attention) without a GPU:
the index arithmetic of the kernels (csrc/wq_kv.h, compiled here for the CPU) over every small
case, bad pages and lengths included; the argument checks of the C entry points (nothing is
launched); the binding's checks; and the plain implementations' own pins."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest
import torch

import gemv_wq_quantize_b200 as wq
import layer_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include "wq_kv.h"
using namespace wq;
extern "C" {
void span(int lo, int hi, int len, int M, int cap, int *o) { KvSpan s = kv_span(lo, hi, len, M, cap); o[0] = s.q0; o[1] = s.n; o[2] = s.len; }
long long item_start(int q0, int b, int sh, int by) { return kv_item_start(q0, b, sh, by); }
void page_span(int q0, int n, int len, long long k, int sh, int *o)
{ KvPageSpan r = kv_page_span(KvSpan{q0, n, len}, k, sh); o[0] = r.page; o[1] = r.off; o[2] = r.count; o[3] = r.token; }
long long page_ok(int e, long long n) { return kv_page_ok(e, n); }
long long code_offset(long long p, int h, int s, int H, int sh, int pitch) { return kv_code_offset(p, h, s, H, sh, pitch); }
long long scale_index(long long p, int h, int H) { return kv_scale_index(p, h, H); }
long long tiles(int n, int g, int r) { return kv_tiles(n, g, r); }
long long units(int len, int shift) { return kv_units(len, shift); }
long long row_item(int q0, int b, int g, int r) { return kv_row_item(q0, b, g, r); }
long long share(int t, int c, int g) { return kv_share(t, c, g); }
}
"""


@pytest.fixture(scope="module")
def kv(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv")
    (d / "kv.cpp").write_text(HARNESS)
    so = d / "libkv.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "gemv_wq_quantize_b200", "csrc"), str(d / "kv.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for f in ("item_start", "page_ok", "code_offset", "scale_index", "tiles", "units", "share", "row_item"):
        getattr(lib, f).restype = ctypes.c_longlong
    for f, t in (("page_ok", [ctypes.c_int, ctypes.c_longlong]), ("share", [ctypes.c_int] * 3),
                 ("code_offset", [ctypes.c_longlong] + [ctypes.c_int] * 5), ("scale_index", [ctypes.c_longlong] + [ctypes.c_int] * 2),
                 ("page_span", [ctypes.c_int] * 3 + [ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p])):
        getattr(lib, f).argtypes = t
    return lib


def _span(kv, *a):
    o = (ctypes.c_int * 3)()
    kv.span(*a, o)
    return tuple(o)


def _page_span(kv, *a):
    o = (ctypes.c_int * 4)()
    kv.page_span(*a, o)
    return tuple(o)


def test_spans_stay_inside_the_call(kv):
    M, cap = 7, 12
    for lo, hi, ln in itertools.product((-3, 0, 2, 7, 9, 2 ** 31 - 1, -2 ** 31), repeat=3):
        q0, n, length = _span(kv, lo, hi, ln, M, cap)
        assert 0 <= q0 <= q0 + n <= M and 0 <= length <= cap
    assert _span(kv, 2, 5, 9, M, cap) == (2, 3, 9)


@pytest.mark.parametrize("by_seq", [0, 1])
@pytest.mark.parametrize("shift", [4, 5])
def test_items_cover_every_new_token_once(kv, shift, by_seq):
    """For every way a sequence's new tokens lie on its pages: the items between two starts (few
    tokens: its first pages) cover each token with a place exactly once, in its page and slot, and
    the rest are idle."""
    ps = 1 << shift
    for n in list(range(0, 3 * ps + 3)):
        for past in range(0, 2 * ps, 3 if n > 4 else 1):
            for missing in (0, 1, n):  # tokens without a place
                ln = past + n - missing
                if ln < 0 or missing > n or (missing and past):
                    continue
                for q0 in (0, 5, ps - 1, 3 * ps):
                    # sequences of few tokens walk their pages, the others' pages are items
                    first, end = kv.item_start(q0, 3, shift, by_seq), kv.item_start(q0 + n, 4, shift, by_seq)
                    got = {}
                    for k in range(end - first if n > 8 else 4):
                        page, off, count, token = _page_span(kv, q0, n, ln, k, shift)
                        for i in range(count):
                            assert 0 <= off + i < ps
                            assert token + i not in got
                            got[token + i] = (page, off + i)
                    want = {q0 + i: divmod(ln - n + i, ps) for i in range(n) if ln - n + i >= 0}
                    assert got == want, (n, past, missing, q0)


def test_an_item_before_the_sequence_is_idle(kv):
    assert _page_span(kv, 0, 40, 40, -1, 4) == (0, 0, 0, 0)


def test_item_starts_never_overlap(kv):
    r = np.random.default_rng(0)
    for shift, by_seq in itertools.product((4, 6, 8), (0, 1)):
        cu = np.concatenate([[0], np.cumsum(r.integers(0, 300, 50))])
        starts = [kv.item_start(int(q), b, shift, by_seq) for b, q in enumerate(cu)]
        assert all(b - a >= 2 for a, b, n in zip(starts, starts[1:], np.diff(cu)) if n > 8)
        assert starts == sorted(starts)


def test_row_blocks_of_sequences_never_overlap(kv):
    r = np.random.default_rng(1)
    for group, rows in ((1, 256), (5, 256), (8, 256), (3, 16)):
        cu = np.concatenate([[0], np.cumsum(r.integers(0, 700, 40))])
        for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
            first, end = kv.row_item(int(lo), b, group, rows), kv.row_item(int(hi), b + 1, group, rows)
            assert end - first >= kv.tiles(int(hi - lo), group, rows)


def test_pages_offsets_and_shares(kv):
    for e in (-2 ** 31, -1, 0, 4, 5, 2 ** 31 - 1):
        assert kv.page_ok(e, 5) == (e if 0 <= e < 5 else -1)
    # every (page, head, slot) has a place of its own, within the cache
    pages, heads, shift, pitch = 3, 2, 4, 112
    at = sorted(kv.code_offset(p, h, s, heads, shift, pitch) for p in range(pages) for h in range(heads) for s in range(16))
    assert at == [pitch * i for i in range(pages * heads * 16)]
    assert sorted(kv.scale_index(p, h, heads) for p in range(pages) for h in range(heads)) == list(range(6))
    # beyond 32 bits
    assert kv.code_offset(2 ** 31 - 1, 7, 15, 8, 8, 256) == (((2 ** 31 - 1) * 8 + 7) * 256 + 15) * 256
    for total, grid in itertools.product((0, 1, 2, 147, 148, 149, 1000, 2 ** 31 - 1), (1, 2, 147, 148, 296, 1001)):
        cuts = [kv.share(total, c, grid) for c in range(grid + 1)]
        assert cuts[0] == 0 and cuts[-1] == total and all(0 <= b - a <= total // grid + 1 for a, b in zip(cuts, cuts[1:]))
        if grid <= total:
            assert all(b > a for a, b in zip(cuts, cuts[1:]))  # no share is empty
    assert kv.tiles(0, 4, 8) == 0 and kv.tiles(3, 5, 8) == 2 and kv.units(0, 6) == 1 and kv.units(65, 6) == 2
    assert kv.units(2 ** 31 - 1, 7) == 2 ** 24 and kv.units(2 ** 31 - 1, 30) == 2


# ---------------------------------------------------------------- refusals of the C entry points
FAKE = ctypes.c_void_p(0x10000)
MIS16, MIS4 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    from gemv_wq_quantize_b200 import build
    build.build(quiet=True)
    return wq.load_library()


def _cache(**kw):
    d = dict(k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000, num_pages=8, page_size=16, kv_heads=2, head_dim=128,
             format=wq.FMT_INT)
    d.update(kw)
    return wq._KVCacheC(**d)


def _batch(**kw):
    d = dict(cu_q=0x10000, seq_len=0x10000, block_table=0x10000, n_seqs=2, max_pages=4)
    d.update(kw)
    return wq._KVBatchC(**d)


def test_norm_refusals(lib):
    INV, AL = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_ALIGNMENT
    for f in (lib.rmsnorm_quant_int8, lib.rmsnorm_quant_fp8):
        def call(X=FAKE, res=FAKE, gamma=FAKE, dt=wq.WQ_F16, eps=1e-5, M=2, K=128, h=FAKE, q=FAKE, s=FAKE):
            return f(X, res, gamma, dt, eps, M, K, h, q, s, None)
        for kw in (dict(X=None), dict(gamma=None), dict(q=None), dict(s=None), dict(res=None), dict(h=None), dict(M=0),
                   dict(K=0), dict(K=12), dict(M=2 ** 31), dict(dt=wq.WQ_F32), dict(eps=0.0), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**kw) == INV, kw
        for kw in (dict(X=MIS16), dict(res=MIS16), dict(gamma=MIS16), dict(h=MIS16), dict(q=MIS16), dict(s=MIS4)):
            assert call(**kw) == AL, kw
        assert lib.wq_last_error()


CACHE_BAD = [
    (dict(k=None), "INVALID_ARG"), (dict(v_scale=None), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(num_pages=2 ** 30), "INVALID_ARG"), (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
    (dict(page_size=512), "UNSUPPORTED"), (dict(head_dim=12), "UNSUPPORTED"), (dict(head_dim=130), "UNSUPPORTED"),
    (dict(head_dim=260), "UNSUPPORTED"), (dict(kv_heads=0), "INVALID_ARG"), (dict(kv_heads=3), "INVALID_ARG"),
    (dict(format=wq.FMT_E2M1), "INVALID_ARG"), (dict(k=0x10008), "ALIGNMENT"), (dict(k_scale=0x10002), "ALIGNMENT")]
BATCH_BAD = [
    (dict(cu_q=None), "INVALID_ARG"), (dict(n_seqs=0), "INVALID_ARG"), (dict(n_seqs=4097), "UNSUPPORTED"),
    (dict(max_pages=0), "INVALID_ARG"), (dict(max_pages=2 ** 27), "INVALID_ARG"), (dict(block_table=0x10002), "ALIGNMENT")]


@pytest.mark.parametrize("which,kw,err", [("cache", *c) for c in CACHE_BAD] + [("batch", *c) for c in BATCH_BAD])
def test_cache_and_batch_refusals(lib, which, kw, err):
    c = _cache(**kw) if which == "cache" else _cache()
    b = _batch(**kw) if which == "batch" else _batch()
    want = getattr(wq, "WQ_ERR_" + err)
    assert lib.kv_append(FAKE, wq.WQ_F16, 4, 4, None, 0, 0, 0, FAKE, c, b, None) == want
    assert lib.kv_attention(FAKE, wq.WQ_F16, 4, 4, c, b, 1.0, FAKE, None, 0, None) == want
    assert lib.kv_attention_workspace_size(4, 4, c, b) == 0


def test_append_and_attention_refusals(lib):
    INV, AL = wq.WQ_ERR_INVALID_ARG, wq.WQ_ERR_ALIGNMENT

    def append(qkv=FAKE, dt=wq.WQ_F16, M=4, hq=4, rope=FAKE, rl=64, rd=64, style=0, out=FAKE):
        return lib.kv_append(qkv, dt, M, hq, rope, rl, rd, style, out, _cache(), _batch(), None)

    for kw in (dict(qkv=None), dict(out=None), dict(M=0), dict(M=2 ** 30), dict(dt=wq.WQ_F32), dict(hq=0), dict(hq=3),
               dict(rope=None), dict(rd=0), dict(rd=3), dict(rd=130), dict(rd=-2), dict(rl=0), dict(style=2)):
        assert append(**kw) == INV, kw
    for kw in (dict(qkv=MIS16), dict(rope=MIS16), dict(out=MIS16)):
        assert append(**kw) == AL, kw

    def attend(q=FAKE, dt=wq.WQ_F16, M=4, hq=4, sm=1.0, out=FAKE, ws=None):
        return lib.kv_attention(q, dt, M, hq, _cache(), _batch(), sm, out, ws, 1 << 30 if ws else 0, None)

    for kw in (dict(q=None), dict(out=None), dict(M=0), dict(dt=wq.WQ_I8), dict(hq=5), dict(sm=float("nan")),
               dict(sm=float("inf"))):
        assert attend(**kw) == INV, kw
    for kw in (dict(q=MIS16), dict(out=MIS16), dict(ws=MIS16)):
        assert attend(**kw) == AL, kw
    assert lib.kv_append(FAKE, wq.WQ_F16, 4, 4, None, 0, 0, 0, FAKE, None, _batch(), None) == INV
    assert lib.kv_attention(FAKE, wq.WQ_F16, 4, 4, _cache(), None, 1.0, FAKE, None, 0, None) == INV
    assert lib.kv_attention_workspace_size(4, 4, _cache(), _batch()) > 0


def test_binding_refuses_cpu_tensors():
    x, g = torch.zeros(2, 128, dtype=torch.float16), torch.ones(128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        wq.rmsnorm_quant_int8(x, g, 1e-5)
    with pytest.raises(ValueError):
        wq.rmsnorm_quant_fp8(x.float(), g, 1e-5)
    c = torch.zeros(4, 2, 16, 128, dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        wq.KVCache(c, c, torch.zeros(4, 2), torch.zeros(4, 2), 128)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        wq.KVBatch(i, i[:2], torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        wq.make_kv_cache(4, 16, 2, 128, device="cpu")


# ---------------------------------------------------------------- pins of the plain implementations
def test_reference_e4m3_against_torch():
    """All 256 codes, and the rounding of values between them, as torch's own type has it."""
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_value(codes), t)
    assert np.array_equal(ref.e4m3_code(t)[t != 0], codes[t != 0])
    x = np.float32(np.random.default_rng(0).standard_normal(20000) * np.exp(np.random.default_rng(1).uniform(-9, 6, 20000)))
    mid = np.sort(np.unique(np.abs(t)))
    x = np.concatenate([x, np.float32((mid[1:] + mid[:-1]) / 2)])  # ties
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_nearest(x), want) and np.array_equal(ref.e4m3_value(ref.e4m3_code(x)), want)


def test_reference_rotation_keeps_lengths():
    r = np.random.default_rng(0)
    x, ang = np.float32(r.standard_normal((3, 20))), r.uniform(0, 6, 5)
    tab = np.float32(np.concatenate([np.cos(ang), np.sin(ang)]))
    z = x[:, :10].astype(np.float64)
    for style, pairs in (("half", [(i, i + 5) for i in range(5)]), ("pairs", [(2 * i, 2 * i + 1) for i in range(5)])):
        y = ref.rotate_bits(x, tab, style)
        assert np.array_equal(y[:, 10:], x[:, 10:])
        for u, (i, j) in enumerate(pairs):
            w = (z[:, i] + 1j * z[:, j]) * np.exp(1j * ang[u])
            assert np.allclose(y[:, i] + 1j * y[:, j], w, rtol=0, atol=8 * 2.0 ** -24 * 4)


def test_reference_attention_against_a_plain_softmax():
    r = np.random.default_rng(0)
    c = ref.Cache(r.integers(-127, 128, (3, 2, 16, 16)).astype(np.int8), r.integers(-127, 128, (3, 2, 16, 16)).astype(np.int8),
                  np.float32(r.random((3, 2)) * 0.02), np.float32(r.random((3, 2))), 16, "int8")
    q = r.standard_normal((3, 4, 16))
    out, *_ = ref.attention_64(q, c, [0, 2, 3], [20, 0], [[2, 0], [1, 1]], 0.25, 3)
    k = torch.from_numpy(np.concatenate([c.k[2] * c.ks[2, :, None, None], c.k[0] * c.ks[0, :, None, None]], 1)[:, :20]).double()
    v = torch.from_numpy(np.concatenate([c.v[2] * c.vs[2, :, None, None], c.v[0] * c.vs[0, :, None, None]], 1)[:, :20]).double()
    k, v = k.repeat_interleave(2, 0), v.repeat_interleave(2, 0)
    mask = torch.ones(2, 20, dtype=torch.bool).tril(18)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[:2]).transpose(0, 1), k, v, mask, scale=0.25)
    assert np.allclose(out[:2], want.transpose(0, 1).numpy(), atol=1e-6) and not out[2].any()
