"""The steps of a decoder layer between its matmuls (rmsnorm_quant_*, kv_append, kv_attention) on
the GPU, against the plain implementations of layer_reference.py.

Norm and append are compared bit for bit with the definition's roundings, and the norm also
with 64 bits; attention within a bound made of its own roundings (see _bound)."""
import numpy as np
import pytest
import torch

import gemv_wq_quantize_b200 as wq
import layer_reference as ref

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step of the type, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemv_wq_quantize_b200 import build
    build.build(quiet=True)
    wq.load_library()
    wq.device_error()
    yield
    torch.cuda.synchronize()
    assert wq.device_error() == 0


def _dev(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()


def _np(t):
    return t.detach().float().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


# ---------------------------------------------------------------- norm
def _norm_inputs(M, K, dt, seed, residual=True):
    r = np.random.default_rng(seed)
    x = ref.to_t(r.standard_normal((M, K)), dt)
    res = ref.to_t(r.standard_normal((M, K)) * np.where(r.random(K) < 0.02, 20, 1), dt) if residual else None
    return x, res, ref.to_t(1 + 0.2 * r.standard_normal(K), dt)


def _norm_run(x, res, gamma, eps, dt, out, **kw):
    f = wq.rmsnorm_quant_int8 if out == "int8" else wq.rmsnorm_quant_fp8
    q, s, h = f(_dev(x, dt), _dev(gamma, dt), eps, residual=None if res is None else _dev(res, dt), **kw)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy(), None if h is None else _np(h)


def _norm_check(x, res, gamma, eps, dt, out):
    q, s, h = _norm_run(x, res, gamma, eps, dt, out)
    bq, bs, bh = ref.norm_bits(x, res, gamma, eps, dt, out)
    if res is not None:
        assert np.array_equal(h, bh, equal_nan=True)
    assert np.array_equal(s, bs, equal_nan=True)
    assert np.array_equal(q, bq)
    return q, s


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (3, 264), (5, 3200), (2, 4104), (2, 8640), (2, 11008), (1, 16384),
                                 (2, 16392), (37, 128), (300, 1000),
                                 (300, 1032), (300, 2056), (300, 4104)])
def test_norm_bits(M, K, dtype, out):
    dt = DT[dtype]
    for residual in (True, False):
        x, res, gamma = _norm_inputs(M, K, dt, M + K, residual)
        q, s = _norm_check(x, res, gamma, 1e-5, dt, out)
        # against 64 bits.  y: rstd and two products, 3 roundings of 2^-24; scale: two more (the
        # reciprocal and the product); the quotient one more: 3 + 5 + 1 of a code, then half a step
        y = ref.norm_64(x, res, gamma, float(np.float32(1e-5)), dt)
        s64 = np.abs(y).max(1) / ref.QMAX[out]
        assert (np.abs(s - s64) <= 5.01 * 2.0 ** -24 * s64).all()
        c64 = y / s64[:, None]
        d = np.abs(ref.values_of(q, out) - c64)
        slack = 9.01 * 2.0 ** -24 * np.abs(c64)
        half = 0.5 if out == "int8" else np.maximum(2.0 ** -4 * np.abs(c64), 2.0 ** -10)
        assert (d <= half + slack).all()


@pytest.mark.parametrize("out", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_norm_special_rows(dtype, out):
    """Zero rows, tiny and huge rows, infinities and NaN, a zero gamma."""
    dt = DT[dtype]
    x, res, gamma = _norm_inputs(8, 512, dt, 3)
    x[0], res[0] = 0, 0
    x[1], res[1] = ref.to_t(np.full(512, 2.0 ** -24), dt), 0
    x[2], res[2] = 30000.0 if dtype == "fp16" else 1e37, 0
    x[3, 100] = np.inf
    x[4, 511] = np.nan
    if dtype == "fp16":
        x[5, 7], res[5, 7] = 65504, 65504  # the sum overflows the type
    else:
        x[5] = ref.to_t(np.full(512, 1e-39), dt)
    res[6] = -x[6]  # cancels to zero
    q, s = _norm_check(x, res, gamma, 1e-6, dt, out)
    assert s[0] == 0 and s[6] == 0 and not q[0].any() and not q[6].any()
    assert np.isnan(s[3]) and np.isnan(s[4]) and not q[3].any() and not q[4].any()
    gamma[:] = 0
    _norm_check(np.nan_to_num(x, nan=1.0, posinf=1.0), res, gamma, 1e-6, dt, out)


@pytest.mark.parametrize("K", [512, 16392])
def test_norm_in_place(K):
    """The new residual stream written over the old one, or over X."""
    x, res, gamma = _norm_inputs(4, K, torch.float16, 5)
    bq, bs, bh = ref.norm_bits(x, res, gamma, 1e-5, torch.float16, "int8")
    for which in (0, 1):
        X, R = _dev(x, torch.float16), _dev(res, torch.float16)
        q, s, h = wq.rmsnorm_quant_int8(X, _dev(gamma, torch.float16), 1e-5, residual=R, out_residual=(X, R)[which])
        assert h is (X, R)[which]
        assert np.array_equal(_np(h), bh) and np.array_equal(q.cpu().numpy(), bq) and np.array_equal(s.cpu().numpy(), bs)


def test_norm_feeds_the_w4a8_matmul():
    """Codes and scales equal to norm, then act_quant_int8, when the normed row is exact in 16 bits;
    and w4a8_gemm takes them as they are."""
    M, K, N = 5, 512, 256
    x, res, gamma = _norm_inputs(M, K, torch.float16, 9)
    q, s, _ = wq.rmsnorm_quant_int8(_dev(x, torch.float16), _dev(gamma, torch.float16), 1e-5, residual=_dev(res, torch.float16))
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(1)) * 0.02
    qc = wq.QuantConfig()
    Wq, ws, _ = wq.quantize_pack(W.cuda(), qc)
    C = wq.w4a8_gemm(q, s, Wq, ws, None, N, K, qc)
    w = wq.unpack(Wq, N, K, qc).cpu().double().numpy() * np.repeat(_np(ws), 128, 1)
    want = (q.cpu().double().numpy() * s.cpu().double().numpy()[:, None]) @ w.T
    # the matmul's own bound: exact group sums, a few binary32 roundings, one binary16 rounding
    mass = np.abs(q.cpu().double().numpy() * s.cpu().double().numpy()[:, None]) @ np.abs(w).T
    assert (np.abs(_np(C) - want) <= 2.0 ** -11 * np.abs(want) + 16 * 2.0 ** -24 * mass + 2.0 ** -25).all()


# ---------------------------------------------------------------- the cache
class Setup:
    """Sequences with new and past tokens, pages in random order, unused bytes full of rubbish."""

    def __init__(self, new, total, q_heads, kv_heads, D, page, dtype, out, seed=0, tail=0, spare=3):
        r = self.r = np.random.default_rng(seed)
        self.new, self.total, self.q_heads, self.kv_heads, self.D = new, total, q_heads, kv_heads, D
        self.page, self.dtype, self.out, self.dt = page, dtype, out, DT[dtype]
        self.pitch = -(-D // 16) * 16
        need = [-(-t // page) for t in total]
        self.width = max(max(need), 1) + 1
        self.num_pages = sum(need) + spare
        order = r.permutation(self.num_pages)
        # entries that are not needed hold numbers that are no pages
        self.table = np.full((len(new), self.width), 1 << 30, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at: at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.M = int(self.cu[-1]) + tail
        shape = (self.num_pages, kv_heads, page, self.pitch)
        # rubbish: -128 (INT8), NaN (e4m3), scales NaN
        kind = np.int8 if out == "int8" else np.uint8
        rubbish = -128 if out == "int8" else 0x7f
        k, v = np.full(shape, rubbish, kind), np.full(shape, rubbish, kind)
        ks, vs = (np.full((self.num_pages, kv_heads), np.nan, np.float32) for _ in range(2))
        self.host = ref.Cache(k, v, ks, vs, D, out)

    def fill(self, upto):
        """Valid codes and scales for the first upto[b] tokens of each sequence."""
        c, r = self.host, self.r
        for b, t in enumerate(upto):
            for p in range(-(-t // self.page)):
                page, n = self.table[b, p], min(self.page, t - p * self.page)
                for codes, scales in ((c.k, c.ks), (c.v, c.vs)):
                    x = r.standard_normal((self.kv_heads, n, self.D)) * (36 if self.out == "int8" else 130)
                    codes[page, :, :n, : self.D] = ref.codes_of(x, 1, self.out)
                    scales[page] = (0.5 + r.random(self.kv_heads)) * 4 / ref.QMAX[self.out]
        return self

    def device(self):
        c = self.host
        t = [torch.from_numpy(x).cuda() for x in (c.k, c.v, c.ks, c.vs)]
        cache = wq.KVCache(*t, self.D)
        batch = wq.KVBatch(*(torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
                             for x in (self.cu, np.array(self.total), self.table)))
        return cache, batch

    def qkv(self):
        x = self.r.standard_normal((self.M, self.q_heads + 2 * self.kv_heads, self.D))
        x *= np.exp(self.r.standard_normal((self.M, 1, 1)))  # tokens of different size: scales grow
        return ref.to_t(x.reshape(self.M, -1), self.dt)

    def rope(self, r):
        if not r:
            return None
        ang = np.arange(max(self.total))[:, None] * 10000.0 ** (-np.arange(0, r, 2) / r)
        return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)

    def q(self):
        return ref.to_t(self.r.standard_normal((self.M, self.q_heads, self.D)), self.dt)


MARK = 7.5  # rows that no call writes keep it


def _append(s, qkv, rope, style, cache, batch, stream=None):
    out = torch.full((s.M, s.q_heads, s.D), MARK, dtype=s.dt, device="cuda")
    wq.kv_append(_dev(qkv, s.dt), cache, batch, s.q_heads, rope=None if rope is None else torch.from_numpy(rope).cuda(),
                 rope_style=wq.ROPE_HALF if style == "half" else wq.ROPE_PAIRS, out=out, stream=stream)
    return out


def _append_check(s, qkv, rope, style):
    cache, batch = s.device()
    out = _append(s, qkv, rope, style, cache, batch)
    want = np.full((s.M, s.q_heads, s.D), MARK)
    ref.append_bits(qkv, s.host, s.cu, s.total, s.table, s.q_heads, s.kv_heads, rope, style, s.dt, want)
    assert np.array_equal(_np(out), want, equal_nan=True)
    assert np.array_equal(_np(cache.k_scale), s.host.ks.astype(np.float64), equal_nan=True)
    assert np.array_equal(_np(cache.v_scale), s.host.vs.astype(np.float64), equal_nan=True)
    assert np.array_equal(cache.k.cpu().numpy(), s.host.k)
    assert np.array_equal(cache.v.cpu().numpy(), s.host.v)
    return cache, batch


APPEND = [
    # new, total, q_heads, kv_heads, D, page, rope_dim, style
    ([1], [1], 1, 1, 16, 16, 16, "half"),
    ([1, 1, 1], [5, 17, 33], 4, 2, 128, 16, 128, "half"),
    ([1, 1, 0, 1], [16, 0, 40, 64], 8, 8, 128, 32, 64, "pairs"),       # an idle slot, a sequence without new tokens
    ([3, 5, 2], [3, 20, 100], 4, 1, 100, 32, 100, "half"),
    ([6, 1, 9], [4, 1, 300], 5, 1, 100, 16, 50, "half"),                # more new tokens than places
    ([70, 17, 130], [70, 90, 200], 4, 2, 64, 64, 32, "pairs"),
    ([260, 3], [300, 3], 2, 2, 128, 128, 128, "half"),
    ([300], [555], 2, 1, 256, 256, 256, "half"),
    ([40, 40], [61, 40], 3, 3, 20, 16, 20, "pairs"),
    ([40, 40], [61, 40], 6, 3, 80, 32, 6, "half"),
    ([33, 1, 12], [64, 2, 12], 2, 2, 192, 64, 96, "pairs"),
    ([25], [77], 2, 2, 52, 16, 0, "half"),                              # no rotation
    ([3, 1, 2, 0, 1], [33, 17, 3, 9, 1], 6, 3, 100, 16, 100, "half"),   # few tokens, over a page's end
    ([0] * 20 + [40], [5] * 20 + [55], 4, 2, 128, 16, 36, "half"),      # few on average, many at once
    ([0] * 30 + [100], [0] * 30 + [100], 2, 1, 256, 256, 256, "half"),
    ([9], [60], 2, 1, 132, 64, 132, "half"),
    ([2, 1], [40, 16], 3, 1, 36, 32, 18, "half"),
    ([1] * 40 + [150, 8, 9], [7] * 40 + [160, 30, 31], 2, 1, 64, 64, 64, "half"),  # a chunk in a decode batch
]


@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("fp16", "fp8"), ("bf16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "q%s_d%d_p%d_r%d%s" % ("-".join(map(str, c[0])), c[4], c[5], c[6], c[7]))
def test_append_bits(case, dtype, out):
    new, total, hq, hkv, D, page, r, style = case
    s = Setup(new, total, hq, hkv, D, page, dtype, out, seed=sum(total) + D, tail=2)
    s.fill([max(t - n, 0) for n, t in zip(new, total)])
    _append_check(s, s.qkv(), s.rope(r), style)


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_append_token_by_token(out):
    """A page filled one token at a time: its scale only grows, earlier codes follow, and every
    value stays within the re-codings' half steps of what was appended."""
    s = Setup([1, 1], [1, 1], 2, 1, 64, 16, "fp16", out, seed=4)
    s.table[:] = 1 << 30
    s.table[0, 0], s.table[1, 0] = 2, 0
    cache, batch = s.device()
    rope = np.concatenate([np.ones((40, 8)), np.zeros((40, 8))], 1).astype(np.float32)  # angle 0
    kept = []
    for step in range(16):
        s.total = [step + 1, step + 1]
        batch.seq_len.copy_(torch.tensor(s.total, dtype=torch.int32))
        qkv = s.qkv() * (1 + step % 5)
        qkv = ref.to_t(qkv, s.dt)
        before = _np(cache.k_scale).copy()
        _append(s, qkv, rope, "half", cache, batch)
        want = np.full((s.M, 2, 64), MARK)
        ref.append_bits(qkv, s.host, s.cu, s.total, s.table, 2, 1, rope, "half", s.dt, want)
        assert np.array_equal(cache.k.cpu().numpy(), s.host.k) and np.array_equal(cache.v.cpu().numpy(), s.host.v)
        if step:
            assert (_np(cache.k_scale)[[2, 0]] >= before[[2, 0]]).all()
        kept.append(qkv.reshape(2, 4, 64)[:, 2])
    scale = _np(cache.k_scale)
    for b, page in enumerate((2, 0)):
        got = ref.values_of(cache.k.cpu().numpy()[page, 0, :, :64], out) * scale[page, 0]
        x = np.stack([t[b] for t in kept])
        # each of at most 16 codings is off by half a step (INT8: of the scale; e4m3: 2^-4 of
        # the value, or 2^-10 of the scale)
        half = 0.5 * scale[page, 0] if out == "int8" else np.maximum(2.0 ** -4 * np.abs(x) * 1.7, 2.0 ** -10 * scale[page, 0])
        assert (np.abs(got - x) <= 16 * half * 1.001).all()


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_append_infinities_and_nan(out):
    """They do not reach the page's scale or its other tokens."""
    s = Setup([4, 2], [7, 18], 2, 1, 32, 16, "fp16", out, seed=8).fill([3, 16])
    qkv = s.qkv()
    x = qkv.reshape(s.M, 4, 32)
    x[1, 2, 5], x[1, 2, 6], x[2, 3, 0], x[3, 3, 31], x[4, 2, 3] = np.inf, np.nan, -np.inf, np.nan, -np.inf
    x[5, 3] = np.nan
    cache, _ = _append_check(s, x.reshape(s.M, -1), None, "half")
    used = s.table[0, 0], s.table[1, 0], s.table[1, 1]
    assert np.isfinite(_np(cache.k_scale)[list(used)]).all() and np.isfinite(_np(cache.v_scale)[list(used)]).all()


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_append_zeros_and_tiny_values(out):
    """A page of zeros has scale 0; later tokens give it one.  Subnormal scales."""
    s = Setup([3], [3], 1, 1, 16, 16, "bf16", out, seed=2)
    cache, batch = _append_check(s, np.zeros((3, 48)), None, "half")
    assert _np(cache.k_scale)[s.table[0, 0], 0] == 0
    s.total, s.new = [6], [3]
    _append_check(s, ref.to_t(np.random.default_rng(0).standard_normal((3, 48)) * 1e-38, torch.bfloat16), None, "half")
    s.total = [9]
    _append_check(s, s.qkv(), None, "half")


def test_append_twice_is_the_same_as_once():
    s = Setup([5, 40], [20, 90], 4, 2, 128, 32, "fp16", "int8", seed=11).fill([15, 50])
    cache, batch = s.device()
    qkv, rope = s.qkv(), s.rope(128)
    a = _append(s, qkv, rope, "half", cache, batch)
    once = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    b = _append(s, qkv, rope, "half", cache, batch)
    assert torch.equal(a, b)
    for x, y in zip(once, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


# ---------------------------------------------------------------- attention
def _bound(want, mass, score, top, keys, dtype):
    """The result's own rounding, and errors of the weighted sum: weights in binary16 (2^-11 of
    each), scores (in units of 2^-24; a weight moves by as much, numerator and denominator:
    twice), the exponentials and rescalings (2^-18), one sum per 16 keys (2^-24 each).  A weight is
    also off by an absolute amount.  Few rows: weights of at most 1 times their value scale over a
    power of two that is at most twice the largest scale are cut to multiples of 2^-28 (INT8
    digits; e4m3 parts: subnormal steps of 2^-9 / (256 * 16^3) = 2^-29), half a step is 2^-29,
    times 2: 2^-28 of the largest scale, for every code.  Many rows: binary16 of 2^11 times the
    same, half a subnormal step of 2^-25: 2^-25 / 2^11 * 2 = 2^-35."""
    rel = 2.0 ** -11 + 2 * 2.0 ** -24 * score + 2.0 ** -18 + (keys / 16 + 32) * 2.0 ** -24
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0  # binary16 subnormals
    return U[dtype] * np.abs(want) * 1.01 + rel * mass * 1.01 + 2.0 ** -28 * top + tiny


def _attend(s, q, cache, batch, workspace=True, **kw):
    ws = wq.make_workspace(wq.kv_attention_workspace_size(s.M, s.q_heads, cache, batch)) if workspace is True else workspace
    out = torch.full((s.M, s.q_heads, s.D), MARK, dtype=s.dt, device="cuda")
    return wq.kv_attention(_dev(q, s.dt), cache, batch, out=out, workspace=ws, **kw)


def _attend_check(s, q, got, sm_scale=None):
    sm = s.D ** -0.5 if sm_scale is None else sm_scale
    want, mass, score, top, own = ref.attention_64(q, s.host, s.cu, s.total, s.table, float(np.float32(sm)), s.num_pages)
    g = _np(got)
    assert (g[~own] == MARK).all()
    off = np.abs(g - want)[own]
    lim = _bound(want, mass, score, top, max(s.total), s.dtype)[own]
    assert np.isfinite(g[own]).all()
    assert (off <= lim).all(), f"worst {np.max(off / np.maximum(lim, 1e-300))} of the bound"


ATTEND = [
    # new, total, q_heads, kv_heads, D, page
    ([1], [1], 1, 1, 16, 16),
    ([1], [700], 1, 1, 128, 16),
    ([1, 1, 1, 1], [15, 16, 17, 1000], 8, 2, 128, 16),
    ([1, 0, 1, 1], [64, 40, 0, 129], 4, 4, 64, 32),           # no new tokens; an idle slot
    ([1, 1], [333, 64], 8, 1, 256, 64),
    ([1, 1, 1], [500, 2, 77], 5, 1, 100, 32),
    ([3, 6, 1], [50, 6, 300], 4, 4, 100, 32),
    ([5, 2], [3, 200], 4, 2, 80, 16),                          # rows before the first key
    ([4, 7], [260, 70], 16, 2, 192, 128),
    ([40, 9], [40, 300], 4, 2, 128, 64),
    ([130, 1, 17], [200, 500, 17], 4, 1, 64, 256),
    ([1] * 9, [1, 2, 3, 31, 32, 33, 400, 64, 65], 2, 2, 20, 32),
    ([67], [67], 3, 1, 52, 16),
    ([1, 1, 1, 1, 1], [5, 300, 64, 1000, 17], 2, 1, 256, 32),  # one row of a head above 128
    ([2, 1, 3, 1], [40, 300, 3, 129], 4, 2, 192, 16),
]


@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("fp16", "fp8"), ("bf16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "q%s_h%d-%d_d%d_p%d" % ("-".join(map(str, c[0])), c[2], c[3], c[4], c[5]))
def test_attention(case, dtype, out):
    new, total, hq, hkv, D, page = case
    s = Setup(new, total, hq, hkv, D, page, dtype, out, seed=sum(total) + D, tail=3).fill(total)
    cache, batch = s.device()
    q = s.q()
    got = _attend(s, q, cache, batch)
    _attend_check(s, q, got)
    _attend_check(s, q, _attend(s, q, cache, batch, workspace=None))
    # the same bits again, and in a workspace that an earlier call used
    ws = wq.make_workspace(wq.kv_attention_workspace_size(s.M, hq, cache, batch))
    for _ in range(2):
        assert torch.equal(_attend(s, q, cache, batch, workspace=ws), got)


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_attention_one_key_dominates(out):
    """A first key with a much larger score over many small ones, whose joint weight still counts."""
    s = Setup([1], [4000], 2, 1, 64, 64, "fp16", out, seed=5).fill([4000])
    q = s.q()
    first = s.table[0, 0]
    k = ref.values_of(s.host.k[first, 0, 0, :64], out) * s.host.ks[first, 0]
    q[0, 0] = ref.to_t(k / (k @ k) * 8 * 14, torch.float16)  # a score of 14 at the first key
    cache, batch = s.device()
    _attend_check(s, q, _attend(s, q, cache, batch))


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_attention_page_scales_far_apart(out):
    s = Setup([2, 1], [300, 90], 4, 2, 128, 16, "fp16", out, seed=6).fill([300, 90])
    r = np.random.default_rng(1)
    used = np.isfinite(s.host.ks)
    s.host.vs[used] = (10.0 ** r.uniform(-6, 1, used.sum())).astype(np.float32)
    s.host.ks[used] *= (10.0 ** r.uniform(-2, 0.3, used.sum())).astype(np.float32)
    q = s.q()
    cache, batch = s.device()
    _attend_check(s, q, _attend(s, q, cache, batch))


def test_attention_scores_of_any_size():
    """Large scores (one weight takes all), a zero scale (a plain mean), a negative one, tiny queries."""
    for sm, size in ((3.0, 1.0), (0.0, 1.0), (-0.2, 1.0), (0.1, 1e-30), (1e-5, 1e4)):
        s = Setup([1, 4], [200, 90], 4, 2, 64, 32, "bf16", "int8", seed=7).fill([200, 90])
        q = ref.to_t(s.q() * size, torch.bfloat16)
        cache, batch = s.device()
        _attend_check(s, q, _attend(s, q, cache, batch, sm_scale=sm), sm)


def _many(new, q_heads, kv_heads):
    """(q_heads, kv_heads) in the same ratio with more rows in all than the split by keys takes."""
    f = -(-3600 // (sum(new) * q_heads))
    return f * q_heads, f * kv_heads


TILES = [
    ([300], [300], 4, 2, 128, 16),                             # three blocks of 256 rows, causal
    ([200, 3, 129], [900, 200, 129], 4, 2, 128, 64),           # long past; a sequence of few rows among them
    ([256, 128, 1, 0, 57], [256, 640, 5, 90, 57], 1, 1, 128, 32),
    ([140, 60], [100, 60], 2, 1, 64, 128),                     # rows before the first key
    ([90, 45], [333, 45], 5, 1, 100, 32),
    ([70], [1500], 8, 1, 48, 256),
    ([100, 100], [100, 0], 3, 3, 112, 16),                     # all rows without keys
    ([300], [300], 4, 2, 256, 64),                             # heads above 128: blocks of 128 rows
    ([200, 3, 129], [900, 200, 129], 2, 1, 192, 16),
    ([40, 1, 0, 90], [700, 333, 90, 91], 4, 1, 132, 128),
    ([140, 60], [100, 60], 2, 1, 256, 256),
    ([100, 65], [0, 65], 3, 3, 160, 32),
]


@pytest.mark.parametrize("dtype,out", [("fp16", "int8"), ("fp16", "fp8"), ("bf16", "int8"), ("bf16", "fp8")])
@pytest.mark.parametrize("case", TILES, ids=lambda c: "q%s_h%d-%d_d%d_p%d" % ("-".join(map(str, c[0])), c[2], c[3], c[4], c[5]))
def test_attention_many_rows(case, dtype, out):
    new, total, hq, hkv, D, page = case
    hq, hkv = _many(new, hq, hkv)
    s = Setup(new, total, hq, hkv, D, page, dtype, out, seed=sum(total) + D, tail=3).fill(total)
    cache, batch = s.device()
    q = s.q()
    got = _attend(s, q, cache, batch)
    _attend_check(s, q, got)
    assert torch.equal(_attend(s, q, cache, batch), got)


@pytest.mark.parametrize("D", [128, 200])
@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_attention_many_rows_uneven(out, D):
    """Value scales and scores that rise by orders of magnitude along the keys and fall again: the running
    references move often."""
    s = Setup([150], [700], *_many([150], 2, 1), D, 16, "fp16", out, seed=31).fill([700])
    order = s.table[0, : -(-700 // 16)]
    rise = np.concatenate([np.linspace(-4, 0, 30), np.linspace(0, -5, order.size - 30)])
    s.host.vs[order, 0] = (10.0 ** rise * 0.03).astype(np.float32)
    s.host.ks[order, 0] = (s.host.ks[order, 0] * 10.0 ** np.linspace(-2, 0.8, order.size)).astype(np.float32)
    q = s.q()
    cache, batch = s.device()
    _attend_check(s, q, _attend(s, q, cache, batch))


@pytest.mark.parametrize("D", [128, 256])
def test_attention_many_rows_with_a_bad_page(D):
    s = Setup([60, 60], [300, 300], *_many([120], 2, 1), D, 16, "bf16", "fp8", seed=33).fill([300, 300])
    s.table[0, 4] = -7
    cache, batch = s.device()
    q = s.q()
    got = _attend(s, q, cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3
    _attend_check(s, q, got)


@pytest.mark.parametrize("D,new,heads", [(128, 1, 1), (256, 1, 1), (256, 1, 12), (64, 1, 2)])
def test_attention_most_sequences(D, new, heads):
    """4096 sequences, the most of a call, in each kernel for few rows."""
    r = np.random.default_rng(8)
    total = [int(x) for x in r.integers(0, 20, 4096)]
    s = Setup([new] * 4096, total, heads, 1, D, 16, "bf16", "int8", seed=D).fill(total)
    cache, batch = s.device()
    q = s.q()
    _attend_check(s, q, _attend(s, q, cache, batch))


def test_attention_many_sequences():
    """More sequences than a block has threads."""
    r = np.random.default_rng(3)
    new = list(r.integers(0, 3, 300))
    total = [int(n + r.integers(0, 60)) for n in new]
    s = Setup(new, total, 2, 1, 32, 16, "fp16", "int8", seed=9, tail=1).fill(total)
    cache, batch = s.device()
    q = s.q()
    _attend_check(s, q, _attend(s, q, cache, batch))
    _attend_check(s, q, _attend(s, q, cache, batch, workspace=None))


def test_calls_on_another_stream_and_in_a_graph():
    """Append and attention captured once; replays read the batch's arrays as they are then."""
    s = Setup([1, 1], [40, 3], 4, 2, 128, 16, "fp16", "int8", seed=12)
    s.table[:] = np.arange(s.num_pages + 3)[: s.table.size].reshape(s.table.shape) % s.num_pages
    s.total = [37, 2]
    s.fill([36, 1])
    cache, batch = s.device()
    side = torch.cuda.Stream()
    rope = s.rope(128)
    rope = np.concatenate([rope] * 3)[:60]
    rope_d = torch.from_numpy(rope).cuda()
    ws = wq.make_workspace(wq.kv_attention_workspace_size(2, 4, cache, batch))
    qkv_d = torch.zeros(2, 8 * 128, dtype=torch.float16, device="cuda")
    q_d, o_d = (torch.zeros(2, 4, 128, dtype=torch.float16, device="cuda") for _ in range(2))

    def step():
        wq.kv_append(qkv_d, cache, batch, 4, rope=rope_d, out=q_d)
        wq.kv_attention(q_d, cache, batch, out=o_d, workspace=ws)

    torch.cuda.synchronize()
    saved = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for t, x in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), saved):
        t.copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for it in range(4):
        qkv = s.qkv()
        qkv_d.copy_(_dev(qkv, torch.float16))
        s.total = [37 + it, 2 + it]
        batch.seq_len.copy_(torch.tensor(s.total, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = np.zeros((2, 4, 128))
        ref.append_bits(qkv, s.host, s.cu, s.total, s.table, 4, 2, rope, "half", s.dt, want)
        assert np.array_equal(_np(q_d), want)
        assert np.array_equal(cache.k.cpu().numpy(), s.host.k)
        _attend_check(s, want, o_d)
    # on a stream of its own, arguments and all
    out = wq.kv_attention(q_d, cache, batch, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, o_d)
    del g


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_beside_decode_in_a_graph(D):
    """Both attention kernels and a following matmul captured: every replay, back to back, gives the bits
    of the plain calls (nothing starts before what it reads is written)."""
    new, total = [300, 1, 20, 1], [420, 2000, 20, 64]
    s = Setup(new, total, 16, 2, D, 32, "fp16", "fp8", seed=D).fill([120, 1999, 0, 63])
    assert s.M * 16 > 24 * torch.cuda.get_device_properties(0).multi_processor_count
    cache, batch = s.device()
    ws = wq.make_workspace(wq.kv_attention_workspace_size(s.M, 16, cache, batch))
    qc = wq.QuantConfig()
    W, sc, _ = wq.quantize_pack(torch.randn(256, 16 * D, generator=torch.Generator().manual_seed(1)).cuda(), qc)
    qkv, rope = _dev(s.qkv(), s.dt), torch.from_numpy(s.rope(D)).cuda()
    mm = wq.make_workspace(wq.workspace_size(s.M, 256, 16 * D, qc))

    def step():
        q = wq.kv_append(qkv, cache, batch, 16, rope=rope)
        o = wq.kv_attention(q, cache, batch, workspace=ws)
        return q, o, wq.w4a16_gemm(o.view(s.M, -1), W, sc, None, 256, 16 * D, qc, workspace=mm)

    want = step()  # (appending the same tokens again leaves the same cache: their pages' scales stand)
    want = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del g


def test_bad_pages_and_lengths_are_reported():
    """A block-table entry that is no page, and a length beyond the table: error 3, the other
    sequences' results as ever, nothing written elsewhere."""
    s = Setup([1, 1, 1], [40, 40, 40], 2, 1, 64, 16, "fp16", "int8", seed=13).fill([40, 40, 40])
    good = s.table.copy()
    s.table[1, 1] = s.num_pages  # one past the end
    cache, batch = s.device()
    q = s.q()
    got = _attend(s, q, cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3
    _attend_check(s, q, got)  # the reference leaves the same tokens out
    s.table[1, 1], s.table[1, 2] = good[1, 1], -1  # the page that the append writes
    cache, batch = s.device()
    before = [x.copy() for x in (s.host.k, s.host.v)]
    qkv = s.qkv()
    _append(s, qkv, None, "half", cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3
    k = cache.k.cpu().numpy()
    assert np.array_equal(k[good[1]% s.num_pages][:2], before[0][good[1] % s.num_pages][:2])
    for b in (0, 2):
        assert not np.array_equal(k[good[b, 2]], before[0][good[b, 2]])
    # a length beyond the block table, and positions beyond the rope table
    s.table = good
    cache, batch = s.device()
    batch.seq_len.copy_(torch.tensor([40, 10 ** 6, 40], dtype=torch.int32))
    s.table[1] = 0
    batch.block_table.copy_(torch.from_numpy(s.table))
    _attend(s, q, cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3
    s.table = good
    cache, batch = s.device()
    k0 = cache.k.clone()
    _append(s, qkv, np.ones((20, 64), np.float32), "half", cache, batch)
    torch.cuda.synchronize()
    assert wq.device_error() == 3 and torch.equal(cache.k, k0)


def test_overlapping_sequences_stay_inside_the_call():
    """cu_q that decreases: not valid, but nothing outside the call is written; and where the rows
    of all sequences together would be beyond counting, the call does nothing and says so."""
    s = Setup([20, 3, 30], [40, 9, 64], 4, 2, 64, 16, "fp16", "int8", seed=5, tail=4).fill([40, 9, 64])
    s.table[s.table == 1 << 30] = 0
    for cu in ([0, 53, 2, 53], [30, 10, 0, 53], [-5, 60, -7, 1 << 30]):
        cache, batch = s.device()
        batch.cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
        _attend(s, s.q(), cache, batch)
        _append(s, s.qkv(), s.rope(64), "half", cache, batch)
    torch.cuda.synchronize()
    wq.device_error()
    n, M = 4096, 65536
    cache = wq.make_kv_cache(2, 16, 64, 16, format=wq.FMT_INT)
    cu = torch.tensor([0, M] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    batch = wq.KVBatch(cu, torch.ones(n, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, dtype=torch.int32, device="cuda"))
    q = torch.zeros(M, 64, 16, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, MARK)
    wq.kv_attention(q, cache, batch, out=out, workspace=wq.make_workspace(wq.kv_attention_workspace_size(M, 64, cache, batch)))
    torch.cuda.synchronize()
    assert wq.device_error() == 3 and (out == MARK).all()


def test_attention_of_two_streams_at_once():
    """Few and many rows, each with a workspace of its own, beside each other: the bits of one
    after the other."""
    few = Setup([1] * 6, [3000, 1, 700, 2500, 64, 900], 8, 2, 64, 32, "bf16", "fp8", seed=3).fill([3000, 1, 700, 2500, 64, 900])
    many = Setup([300, 1, 90], [900, 2000, 90], 16, 2, 64, 64, "fp16", "int8", seed=4).fill([900, 2000, 90])
    runs = []
    for s in (few, many):
        cache, batch = s.device()
        runs.append((s, _dev(s.q(), s.dt), cache, batch,
                     wq.make_workspace(wq.kv_attention_workspace_size(s.M, s.q_heads, cache, batch))))
    alone = [wq.kv_attention(q, cache, batch, workspace=ws) for _, q, cache, batch, ws in runs]
    outs = [[torch.empty_like(a) for _ in range(10)] for a in alone]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for i in range(10):
        for (s, q, cache, batch, ws), st, o in zip(runs, streams, outs):
            wq.kv_attention(q, cache, batch, out=o[i], workspace=ws, stream=st)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(a, x) for x in o)


# ---------------------------------------------------------------- together
def _rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("out", ["int8", "fp8"])
def test_layer_steps_together(out):
    """Two decode steps and a prefill of a layer's attention half as a user chains them: norm ->
    quantized QKV projection -> append -> attention -> output projection, on one stream without
    waits, every stage against the reference on the stage's own inputs."""
    E, Hq, Hkv, D = 512, 4, 2, 128
    Nqkv = (Hq + 2 * Hkv) * D
    gen = torch.Generator().manual_seed(0)
    qc = wq.QuantConfig() if out == "int8" else wq.QuantConfig(bits=8, format=wq.FMT_E4M3)
    Wqkv, sqkv, _ = wq.quantize_pack((torch.randn(Nqkv, E, generator=gen) * 0.05).cuda(), qc)
    Wo, so, _ = wq.quantize_pack((torch.randn(E, Hq * D, generator=gen) * 0.05).cuda(), qc)
    gamma = ref.to_t(1 + 0.1 * np.random.default_rng(0).standard_normal(E), torch.float16)
    steps = [([20, 33], [20, 33]), ([1, 1], [21, 34]), ([1, 1], [22, 35])]
    s = Setup(*steps[-1], Hq, Hkv, D, 16, "fp16", out, seed=21)
    cache, batch = s.device()
    rope = s.rope(D)
    rope_d = torch.from_numpy(rope).cuda()
    r = np.random.default_rng(5)
    for new, total in steps:
        s.new, s.total = new, total
        s.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s.M = int(s.cu[-1])
        batch.cu_q.copy_(torch.from_numpy(s.cu))
        batch.seq_len.copy_(torch.tensor(total, dtype=torch.int32))
        x, res = (ref.to_t(r.standard_normal((s.M, E)), torch.float16) for _ in range(2))
        ws = wq.make_workspace(max(wq.kv_attention_workspace_size(s.M, Hq, cache, batch),
                                   wq.workspace_size(s.M, Nqkv, E, qc)))
        X, R = _dev(x, torch.float16), _dev(res, torch.float16)
        if out == "int8":
            a, sc, h = wq.rmsnorm_quant_int8(X, _dev(gamma, torch.float16), 1e-5, residual=R)
            qkv = wq.w4a8_gemm(a, sc, Wqkv, sqkv, None, Nqkv, E, qc, workspace=ws)
        else:
            a, sc, h = wq.rmsnorm_quant_fp8(X, _dev(gamma, torch.float16), 1e-5, residual=R)
            qkv = wq.w8a8_fp8_gemm(a, sc, Wqkv, sqkv, Nqkv, E, qc, workspace=ws)
        q = wq.kv_append(qkv, cache, batch, Hq, rope=rope_d)
        o = wq.kv_attention(q, cache, batch, workspace=ws)
        o2 = o.view(s.M, Hq * D)
        if out == "int8":
            aq, as_ = wq.act_quant_int8(o2)
            y = wq.w4a8_gemm(aq, as_, Wo, so, None, E, Hq * D, qc, workspace=ws)
        else:
            aq, as_ = wq.act_quant_fp8(o2)
            y = wq.w8a8_fp8_gemm(aq, as_, Wo, so, E, Hq * D, qc, workspace=ws)
        torch.cuda.synchronize()
        bq, bs, bh = ref.norm_bits(x, res, gamma, 1e-5, torch.float16, out)
        assert np.array_equal(a.cpu().numpy(), bq) and np.array_equal(sc.cpu().numpy(), bs) and np.array_equal(_np(h), bh)
        want = np.zeros((s.M, Hq, D))
        ref.append_bits(_np(qkv), s.host, s.cu, total, s.table, Hq, Hkv, rope, "half", s.dt, want)
        assert np.array_equal(_np(q), want) and np.array_equal(cache.k.cpu().numpy(), s.host.k)
        assert np.array_equal(cache.v.cpu().numpy(), s.host.v)
        _attend_check(s, want, o)
        w = wq.unpack(Wo, E, Hq * D, qc).cpu().numpy()
        w = ref.values_of(w, out) * np.repeat(_np(so), 128, 1)
        back = ref.values_of(aq.cpu().numpy(), out) * as_.cpu().double().numpy()[:, None]
        assert _rel(_np(y), back @ w.T) <= 1e-3
