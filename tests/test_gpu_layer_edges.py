"""Calls of the layer operators at the edges of what their documentation allows: lengths beyond
the block table, tiny, zero and huge scales and scores, in each attention kernel."""
import numpy as np
import pytest
import torch

import gemv_wq_quantize_b200 as wq
import layer_reference as ref
from test_gpu_layer_ops import MARK, U, Setup, _append, _attend, _attend_check, _bound, _lib, _many, _np  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- append: lengths beyond the block table
def _rope(positions, r):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, r, 2) / r)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


BEYOND = [
    # new, lengths (table: 4 pages of 16), rope
    ([1, 1], [65, 30], True),
    ([4, 1], [66, 30], False),                        # two of four fit
    ([8, 2], [1000, 30], True),
    ([1, 1], [2 ** 31 - 1, 30], False),
    ([40, 1], [80, 30], True),                        # a long run, part of which fits
    ([30, 40], [90, 50], False),                      # none of it does
    ([12] + [1] * 20, [2 ** 31 - 1] + [30] * 20, True),
]


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("case", BEYOND, ids=lambda c: "q%s_len%s" % (c[0][0], c[1][0]))
def test_append_beyond_the_block_table(case, out):
    """Tokens at or behind the table's capacity are left out: no slot, scale or code of an earlier token
    changes, their queries are zeros, the tokens that fit are stored, and the error word says so."""
    new, total, turned = case
    fit = [min(t, 64) for t in total]
    s = Setup(new, fit, 4, 2, 32, 16, "fp16", out, seed=sum(new))
    s.fill([max(f - n, 0) if t <= 64 else min(max(t - n, 0), 64) for n, t, f in zip(new, total, fit)])
    s.table, s.total = np.ascontiguousarray(s.table[:, :4]), total
    s.table[s.table == 1 << 30] = 0  # (tables are padded with a valid page, another sequence's perhaps)
    rope = _rope(200, 32) if turned else None
    cache, batch = s.device()
    qkv = s.qkv() * 4  # larger than what the pages hold: a stray token would raise their scales
    qkv = ref.to_t(qkv, s.dt)
    got = _append(s, qkv, rope, "half", cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3
    want = np.zeros((s.M, 4, 32))
    for b, (n, t) in enumerate(zip(new, total)):
        first, placed = int(s.cu[b]), max(0, min(n, 64 - (t - n)))
        ref.append_bits(qkv, s.host, [first, first + placed], [t - n + placed], s.table[b: b + 1], 4, 2, rope, "half", s.dt, want)
    assert np.array_equal(_np(got), want)
    assert np.array_equal(_np(cache.k_scale), s.host.ks.astype(np.float64), equal_nan=True)
    assert np.array_equal(_np(cache.v_scale), s.host.vs.astype(np.float64), equal_nan=True)
    assert np.array_equal(cache.k.cpu().numpy(), s.host.k) and np.array_equal(cache.v.cpu().numpy(), s.host.v)


# ---------------------------------------------------------------- attention: tiny and zero value scales
def _scaled(s, workspaces, vs):
    """The setup's value scales times a power of two, and its attention within the usual bound plus half a
    step of the smallest bfloat16 values."""
    used = np.isfinite(s.host.vs)
    s.host.vs[used] = (s.host.vs[used].astype(np.float64) * vs).astype(np.float32)
    cache, batch = s.device()
    q = s.q()
    want, mass, score, top, own = ref.attention_64(q, s.host, s.cu, s.total, s.table, float(np.float32(s.D ** -0.5)), s.num_pages)
    for ws in workspaces:
        g = _np(_attend(s, q, cache, batch, workspace=ws))
        lim = _bound(want, mass, score, top, max(s.total), s.dtype) + 1.01 * 2.0 ** -134
        assert np.isfinite(g[own]).all() and (np.abs(g - want)[own] <= lim[own]).all(), \
            np.max(np.abs(g - want)[own] / lim[own])


VALUE_SCALES = [0.0, 2.0 ** -97, 2.0 ** -108, 2.0 ** -118, 2.0 ** -126, 2.0 ** 100, 2.0 ** 117]


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("vs", VALUE_SCALES)
def test_attention_value_scales_of_any_size(vs, D, out):
    """Few rows.  The scales are 2^-7 .. 2^-4 (INT8) times vs; all are valid in a cache."""
    _scaled(Setup([1, 3], [700, 90], 4, 2, D, 32, "bf16", out, seed=7).fill([700, 90]), (True, None), vs)


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("vs", VALUE_SCALES)
def test_attention_many_rows_value_scales_of_any_size(vs, D, out):
    new = [130, 40]
    _scaled(Setup(new, [300, 40], *_many(new, 2, 1), D, 32, "bf16", out, seed=8).fill([300, 40]), (True,), vs)


@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("fp16", "fp8"), ("bf16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("sm,size", [(3.0, 1.0), (0.0, 1.0), (-0.2, 1.0), (0.1, 1e-30), (1e-5, 1e4)])
def test_attention_many_rows_scores_of_any_size(sm, size, D, dtype, out):
    """One weight that takes all, a zero scale (a plain mean), a negative one, tiny and large queries."""
    new = [140, 60]
    s = Setup(new, [200, 90], *_many(new, 2, 1), D, 32, dtype, out, seed=7).fill([200, 90])
    q = ref.to_t(s.q() * size, s.dt)
    cache, batch = s.device()
    _attend_check(s, q, _attend(s, q, cache, batch, sm_scale=sm), sm)


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("D,many", [(64, False), (64, True), (128, True), (256, False), (256, True)])
def test_attention_value_scales_very_far_apart(D, many, out):
    """Pages whose values are next to nothing beside the others' still count in the sum of the weights."""
    new = [130] if many else [3]
    s = Setup(new, [400], *(_many(new, 2, 1) if many else (4, 2)), D, 32, "bf16", out, seed=10).fill([400])
    r = np.random.default_rng(4)
    used = np.isfinite(s.host.vs)
    s.host.vs[used] = (2.0 ** r.uniform(-140, 3, used.sum())).astype(np.float32)
    q = s.q()
    cache, batch = s.device()
    _attend_check(s, q, _attend(s, q, cache, batch))


# ---------------------------------------------------------------- attention: huge scores
@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_attention_scores_a_step_apart(out):
    """Scores of 2^25 and more in base 2, where one step of binary32 is 4: a key one or two steps over the
    reference weighs 16 or 256 times as much, in a later step of 128 keys too."""
    s = Setup([1], [256], 1, 1, 64, 32, "bf16", out, seed=3).fill([256])
    log2e = np.float32(1.4426950408889634)
    sm = np.float32(2 ** 19 / 1.4426950408889634)
    assert np.float32(sm * log2e) == 2 ** 19  # as the kernel forms it
    at = np.arange(256)
    pages, slots = s.table[0, at // 32], at % 32
    c = np.zeros((256, 64))
    c[:, 0] = 64
    step = np.zeros(256)
    step[5], step[200], step[210] = 1, 2, 1
    c[:, 1] = step
    s.host.k[pages, 0, slots, :64] = ref.codes_of(c, 1, out)
    s.host.ks[:] = np.where(np.isfinite(s.host.ks), 1.0, s.host.ks)
    q = np.zeros((1, 1, 64))
    q[0, 0, :2] = 1, 2.0 ** -17  # the score: 2^19 (64 + step 2^-17) = 2^25 + 4 step
    cache, batch = s.device()
    got = _np(_attend(s, ref.to_t(q, s.dt), cache, batch, sm_scale=float(sm)))[0, 0]
    w = 2.0 ** (4 * step)
    v = ref.values_of(s.host.v[pages, 0, slots, :64], out) * s.host.vs[pages, 0].astype(np.float64)[:, None]
    want, mass = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    # scores and weights are exact powers of two: value scale and its parts (2^-16), the sums, the type
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + (2.0 ** -16 + 2.0 ** -18) * mass).all()


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,many", [(64, False), (128, True), (256, False), (256, True)])
def test_attention_huge_scores(D, many, dtype, out):
    """Scores of 2^20 to 2^90 in base 2, with one key far above the others, which comes late: the result
    is that key's value (every other weight is 0)."""
    new = [140] if many else [3]
    heads = _many(new, 2, 1) if many else (2, 1)
    s = Setup(new, [700], *heads, D, 16, dtype, out, seed=9).fill([700])
    r = np.random.default_rng(1)
    at = np.arange(700)
    pages, slots = s.table[0, at // 16], at % 16
    code = np.minimum(np.arange(700) // 8, 90).astype(np.float64)  # the maximum rises step by step
    code[525] = 120
    s.host.k[pages, :, slots, 0] = ref.codes_of(code, 1, out)[:, None]
    s.host.ks[:] = np.where(np.isfinite(s.host.ks), 2.0 ** 40 if dtype == "fp16" else 1.0, s.host.ks)
    q = np.zeros((s.M, s.q_heads, D))
    q[..., 0] = 2.0 ** (r.uniform(-12, 12, q.shape[:2]) if dtype == "fp16" else r.uniform(15, 80, q.shape[:2]))
    q = ref.to_t(q, s.dt)
    cache, batch = s.device()
    got = _np(_attend(s, q, cache, batch, sm_scale=0.3))
    p, i = s.table[0, 525 // 16], 525 % 16
    v = ref.values_of(s.host.v[p, :, i, :D], out) * s.host.vs[p].astype(np.float64)[:, None]
    want = np.repeat(v, s.q_heads // heads[1], 0)[None]
    # the weight's own 16 (or 8-bit parts': 16) bits, the type's rounding, the exponential and 1 / sum
    lim = (U[dtype] + 2.0 ** -11 + 2.0 ** -18) * np.abs(want) * 1.01
    assert np.isfinite(got).all() and (np.abs(got - want) <= lim).all()


@pytest.mark.parametrize("new,hq,hkv,D", [([300, 1, 90], 16, 16, 64), ([1300, 1, 90], 4, 4, 64), ([130, 1], 32, 8, 256), ([3, 1], 4, 2, 64)])
def test_offsets_behind_the_last_sequence_may_be_zero(new, hq, hkv, D):
    """Slots without tokens behind the last sequence, their offsets left at 0 (or at anything without rows): the
    same bits, in each kernel and the append."""
    total = [n + 40 for n in new] + [9, 0]
    s = Setup(new + [0, 0], total, hq, hkv, D, 32, "fp16", "int8", seed=D).fill([t - n for n, t in zip(new + [0, 0], total)])
    qkv, got = s.qkv(), []
    for tail in ([s.M, s.M], [0, 0], [5, 5], [s.M, 0]):
        cache, batch = s.device()
        batch.cu_q[-2:].copy_(torch.tensor(tail, dtype=torch.int32))
        q = _append(s, qkv, None, "half", cache, batch)
        got.append([q, _attend(s, _np(q), cache, batch), cache.k, cache.v, cache.k_scale, cache.v_scale])
    torch.cuda.synchronize()
    assert wq.device_error() == 0
    for g in got[1:]:
        assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(got[0], g))


# ---------------------------------------------------------------- attention: what few rows keep of a weight
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_few_rows_keep_small_weights(out, D):
    """One key with the value 0 outweighs 6000 others by 2^18 to 2^25, whose values are all positive: the
    result is what the small weights add up to."""
    n = 6000
    s = Setup([1], [n], 2, 1, D, 64, "bf16", out, seed=5).fill([n])
    at = np.arange(n)
    pages, slots = s.table[0, at // 64], at % 64
    r = np.random.default_rng(2)
    kc = np.zeros((n, D))
    kc[:, 0] = r.integers(-20, 20, n)
    kc[0, 0] = 120
    vc = np.abs(ref.values_of(s.host.v[pages, 0, slots, :D], out))
    vc[0] = 0
    s.host.k[pages, 0, slots, :D] = ref.codes_of(kc, 1, out)
    s.host.v[pages, 0, slots, :D] = ref.codes_of(vc, 1, out)
    s.host.ks[:] = np.where(np.isfinite(s.host.ks), 1.0, s.host.ks)
    q = np.zeros((1, 2, D))
    q[..., 0] = 0.125, 0.1171875
    cache, batch = s.device()
    got = _np(_attend(s, ref.to_t(q, s.dt), cache, batch, sm_scale=1.0))
    want, mass, score, top, _ = ref.attention_64(q, s.host, s.cu, s.total, s.table, 1.0, s.num_pages)
    # A weight times its value scale is kept to half of 2^-26 (INT8) or to 2^-16 of itself and half of
    # 2^-27 (e4m3), in units of a power of two that is at most twice the largest value scale; then
    # the scores' and the exponentials' errors, and a sum per 128 keys.
    rel = 2 * 2.0 ** -24 * score + 2.0 ** -20 + (n / 128 + 64) * 2.0 ** -24 + (2.0 ** -16 if out == "fp8" else 0)
    lim = U["bf16"] * np.abs(want) + rel * mass + (2.0 ** -26 if out == "int8" else 2.0 ** -27) * top
    assert (np.abs(got - want) <= 1.01 * lim).all(), np.max(np.abs(got - want) / lim)


# ---------------------------------------------------------------- shapes
@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("new,total,hq,hkv,D", [
    ([1, 3, 1], [300, 90, 17], 64, 1, 128),
    ([1, 1, 2], [300, 90, 17], 40, 2, 256),
    ([80, 1, 20], [300, 90, 20], 64, 1, 128),
    ([70, 1, 13], [300, 90, 20], 48, 2, 192),
])
def test_attention_of_large_groups(new, total, hq, hkv, D, out):
    """Up to 64 query heads a key head, in both kernels."""
    s = Setup(new, total, hq, hkv, D, 128, "bf16", out, seed=hq).fill(total)
    cache, batch = s.device()
    q = s.q()
    _attend_check(s, q, _attend(s, q, cache, batch))


@pytest.mark.parametrize("new", [[1, 4, 1], [200, 1, 90]])
def test_a_cache_beyond_4_gigabytes(new):
    """The same call in a small cache and in the last pages of one whose keys alone pass 2^32 bytes."""
    s = Setup(new, [300, 40, 290], 16, 8, 256, 256, "fp16", "int8", seed=6)
    s.fill([t - n for n, t in zip(new, s.total)])
    far = 2 ** 32 // (8 * 256 * 256) + 1
    if torch.cuda.mem_get_info()[0] < 3 * far * 8 * 256 * 256:
        pytest.skip("needs 13 GB")
    qkv, results = s.qkv(), []
    for offset in (0, far):
        cache, batch = s.device()
        if offset:
            big = wq.make_kv_cache(offset + s.num_pages, 256, 8, 256)
            for name in ("k", "v", "k_scale", "v_scale"):
                getattr(big, name)[offset:].copy_(getattr(cache, name))
            batch.block_table.add_(offset)
            cache = big
        q = _append(s, qkv, s.rope(256), "half", cache, batch)
        o = _attend(s, _np(q), cache, batch)
        results.append([q, o] + [getattr(cache, n)[offset:].clone() for n in ("k", "v", "k_scale", "v_scale")])
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())


# ---------------------------------------------------------------- queries that are not finite
@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("D,many", [(64, False), (256, False), (128, True), (256, True)])
def test_attention_rows_beside_one_that_is_not_finite(D, many, dtype, out):
    """An infinity or NaN spoils the row that holds it, and no other."""
    new = [130, 40] if many else [3, 1]
    s = Setup(new, [300, 90], *(_many(new, 2, 1) if many else (4, 2)), D, 32, dtype, out, seed=12).fill([300, 90])
    q = s.q()
    bad = np.zeros(q.shape[:2], bool)
    bad[1, 0] = bad[2, 1] = bad[-1, 0] = True
    x = q.copy()
    x[1, 0, 3], x[2, 1, D - 1], x[-1, 0, 0] = np.nan, np.inf, -np.inf
    cache, batch = s.device()
    got = _np(_attend(s, x, cache, batch))
    want, mass, score, top, _ = ref.attention_64(q, s.host, s.cu, s.total, s.table, float(np.float32(D ** -0.5)), s.num_pages)
    lim = _bound(want, mass, score, top, 300, dtype)
    assert (np.abs(got - want) <= lim)[~bad].all() and np.isnan(got[1, 0]).all()


# ---------------------------------------------------------------- the binding
def test_workspace_size_of_an_invalid_call_is_an_error():
    cache = wq.make_kv_cache(4, 16, 2, 64)
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    batch = wq.KVBatch(i, i[:2], torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    assert wq.kv_attention_workspace_size(4, 4, cache, batch) > 0
    for M, heads in ((0, 4), (4, 3), (4, 0), (2 ** 30, 4)):
        with pytest.raises(wq.WqError):
            wq.kv_attention_workspace_size(M, heads, cache, batch)


# ---------------------------------------------------------------- decode and a prompt chunk in one call
MIXED = [
    # new, total, q_heads, kv_heads, D
    ([1] * 40 + [300], [50] * 40 + [420], 24, 24, 64),
    ([1] * 20 + [300] + [1] * 20 + [0, 0, 30], [50] * 20 + [300] + [7] * 20 + [0, 9, 90], 24, 24, 128),
    ([300] + [1] * 90 + [257], [290] + [33] * 90 + [500], 20, 10, 96),
    ([1] * 30 + [0] * 5 + [260], [40] * 30 + [0] * 5 + [300], 24, 24, 256),
    ([260, 1] + [2] * 40, [700, 90] + [33] * 40, 20, 20, 192),
]


@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("case", MIXED, ids=lambda c: "s%d_h%d-%d_d%d" % (len(c[0]), c[2], c[3], c[4]))
def test_attention_of_decode_and_a_chunk(case, dtype, out):
    """A long run among single tokens (its rows on the tile kernel, the others beside them), and the same
    bits as often as it runs."""
    new, total, hq, hkv, D = case
    idle = (24 if D <= 128 else 16) * torch.cuda.get_device_properties(0).multi_processor_count
    assert (sum(new) - len(new)) * hq > 2 * idle and sum(new) * (hq // hkv) <= 16 * len(new)
    s = Setup(new, total, hq, hkv, D, 32, dtype, out, seed=D, tail=3).fill(total)
    cache, batch = s.device()
    q = s.q()
    got = _attend(s, q, cache, batch)
    _attend_check(s, q, got)
    for _ in range(3):
        assert torch.equal(_attend(s, q, cache, batch), got)
