"""Plain implementations of the layer operators (RMS norm with an 8-bit output, append to the paged
8-bit cache, attention over it) on the CPU with numpy: straight loops over the definitions, in
64 bits where a value is compared within a tolerance and with single binary32 roundings where
the definition fixes every bit.  They share no code with the library."""
import numpy as np
import torch

QMAX = {"int8": 127.0, "fp8": 448.0}
INV = {o: np.float32(1) / np.float32(q) for o, q in QMAX.items()}  # binary32 reciprocals


def to_t(x, dt):
    """float array rounded once to a 16-bit type, as float64 values."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dt).double().numpy()


def e4m3_nearest(x):
    """Nearest e4m3 value of each x (|x| clipped to 448), ties to the even last bit."""
    x = np.clip(np.asarray(x, dtype=np.float64), -448, 448)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(x / step) * step  # rint of a multiple of the step: ties to even


def e4m3_code(x):
    """The code of e4m3_nearest(x), +0 for zero."""
    v = e4m3_nearest(x)
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6))).astype(int)
    code = np.where(a < 2.0 ** -6, np.rint(a * 512).astype(int),
                    ((e + 7) << 3) | (np.rint(a * 2.0 ** (3.0 - e)).astype(int) - 8))
    return np.where(v < 0, code | 0x80, code).astype(np.uint8)


def e4m3_value(code):
    c = np.asarray(code, dtype=np.uint8).astype(int)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c & 0x80, -v, v)


def codes_of(x, s, out):
    """Codes (int8 or uint8) of finite binary32 x for one binary32 scale s."""
    x, s = np.asarray(x, dtype=np.float32), np.float32(s)
    if s == 0:
        return np.zeros(x.shape, np.int8 if out == "int8" else np.uint8)
    with np.errstate(over="ignore"):
        q = (x / s).astype(np.float32)
    if out == "int8":
        return np.clip(np.rint(q), -127, 127).astype(np.int8)
    return e4m3_code(q)


def values_of(codes, out):
    return np.asarray(codes).astype(np.int8).astype(np.float64) if out == "int8" else e4m3_value(codes)


# ---------------------------------------------------------------- RMS norm
def norm_bits(x, res, gamma, eps, dt, out):
    """(codes, scale, h) with every rounding of the definition."""
    h = np.float32(x) if res is None else to_t(np.float32(x) + np.float32(res), dt).astype(np.float32)
    codes, scales = [], []
    for row in h:
        with np.errstate(all="ignore"):
            ms = np.sum(row.astype(np.float64) ** 2) / row.size
            rstd = np.float32(1 / np.sqrt(ms + np.float64(np.float32(eps))))
            y = (row * rstd).astype(np.float32) * np.float32(gamma)
        if not np.isfinite(y).all():
            scales.append(np.float32("nan"))
            codes.append(np.zeros(row.shape, np.int8 if out == "int8" else np.uint8))
            continue
        s = np.float32(np.abs(y).max()) * INV[out]
        scales.append(s)
        codes.append(codes_of(y, s, out))
    return np.stack(codes), np.array(scales, np.float32), h.astype(np.float64)


def norm_64(x, res, gamma, eps, dt):
    """y in 64 bits (h rounded to the type, as the definition has it)."""
    h = np.asarray(x, np.float64) if res is None else to_t(np.asarray(x) + np.asarray(res), dt)
    return h / np.sqrt((h ** 2).mean(1, keepdims=True) + eps) * gamma


# ---------------------------------------------------------------- the paged cache
class Cache:
    """Host copy of a cache: codes [pages, heads, page, pitch], scales [pages, heads]."""

    def __init__(self, k, v, ks, vs, head_dim, out):
        self.k, self.v, self.ks, self.vs = k.copy(), v.copy(), ks.copy(), vs.copy()
        self.head_dim, self.out, self.page = head_dim, out, k.shape[2]


def rotate_bits(x, tab, style):
    """x [heads, D] binary32, one position's table row: single roundings."""
    x = np.float32(x).copy()
    r = 0 if tab is None else tab.size
    for u in range(r // 2):
        i, j = (u, u + r // 2) if style == "half" else (2 * u, 2 * u + 1)
        c, s = np.float32(tab[u]), np.float32(tab[r // 2 + u])
        with np.errstate(all="ignore"):
            a, b = x[:, i].copy(), x[:, j].copy()
            x[:, i] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
            x[:, j] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return x


def append_bits(qkv, cache, cu_q, seq_len, table, q_heads, kv_heads, rope, style, dt, q_out):
    """Appends to `cache` in place; fills the rows of q_out (float64) that belong to sequences."""
    D, ps, out = cache.head_dim, cache.page, cache.out
    for b in range(len(seq_len)):
        n, ln = cu_q[b + 1] - cu_q[b], seq_len[b]
        new = {}  # page -> [(slot, token row)]
        for i in range(n):
            m, p = cu_q[b] + i, ln - n + i
            x = np.float32(qkv[m]).reshape(q_heads + 2 * kv_heads, D)
            if p < 0:
                q_out[m] = 0
                continue
            tab = None if rope is None else rope[p]
            qk = rotate_bits(x[: q_heads + kv_heads], tab, style)
            q_out[m] = to_t(qk[:q_heads], dt)
            new.setdefault(table[b][p // ps], []).append((p % ps, qk[q_heads:], x[q_heads + kv_heads:]))
        for page, rows in new.items():
            first = rows[0][0]
            for codes, scales, which in ((cache.k, cache.ks, 1), (cache.v, cache.vs, 2)):
                for h in range(kv_heads):
                    x = np.stack([r[which][h] for r in rows])
                    x = np.where(np.isnan(x), np.float32(0), x)
                    fin = np.abs(x[np.isfinite(x)])
                    need = np.float32(fin.max() if fin.size else 0) * INV[out]
                    before = scales[page, h] if first > 0 else np.float32(0)
                    now = max(before, need)
                    if first > 0 and now > before:
                        ratio = np.float32(before / now)
                        old = np.float32(values_of(codes[page, h, :first, :D], out)) * ratio
                        codes[page, h, :first, :D] = codes_of(old, 1, out)
                    scales[page, h] = now
                    big = np.float32(np.finfo(np.float32).max)
                    for (slot, _, _), v in zip(rows, x):
                        codes[page, h, slot, :D] = codes_of(np.clip(v, -big, big), now, out)


def attention_64(q, cache, cu_q, seq_len, table, sm_scale, num_pages):
    """(out, mass, score, top, own): the attention in 64 bits, and for every output the terms its
    error bound is made of: sum w |v|, the largest error of a score in units of 2^-24, and the sum of
    |codes| times the largest value scale.
    own: the rows that belong to a sequence.  Tokens whose block-table entry is no page are left
    out."""
    M, Hq, D = q.shape
    Hkv, ps = cache.k.shape[1], cache.page
    out, mass, top, score = (np.zeros((M, Hq, d)) for d in (D, D, D, 1))
    own = np.zeros(M, bool)
    for b in range(len(seq_len)):
        n, ln = cu_q[b + 1] - cu_q[b], seq_len[b]
        own[cu_q[b]: cu_q[b + 1]] = True
        if ln <= 0 or n <= 0:
            continue
        at = np.arange(ln)
        pages = np.asarray(table[b])[at // ps]
        fine = (pages >= 0) & (pages < num_pages)
        pg = np.where(fine, pages, 0)
        for h in range(Hkv):
            k = values_of(cache.k[pg, h, at % ps, :D], cache.out) * cache.ks[pg, h].astype(np.float64)[:, None]
            vc, vs = values_of(cache.v[pg, h, at % ps, :D], cache.out), cache.vs[pg, h].astype(np.float64)
            v = vc * vs[:, None]
            G = Hq // Hkv
            for i in range(n):
                see = np.flatnonzero((at <= ln - n + i) & fine)
                if not see.size:
                    continue
                qs = q[cu_q[b] + i, h * G: (h + 1) * G]
                s = qs @ k[see].T * sm_scale
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                rows = (cu_q[b] + i, slice(h * G, (h + 1) * G))
                out[rows] = w @ v[see]
                mass[rows] = w @ np.abs(v[see])
                top[rows] = np.abs(vc[see]).sum(0) * vs[see].max()
                # D products and sums; the queries' 16-bit form: 2^-25 of the largest, per term
                err = (D + 16) * (np.abs(qs) @ np.abs(k[see]).T) + np.abs(qs).max(1, keepdims=True) * np.abs(k[see]).sum(1)
                score[rows] = (err * abs(sm_scale)).max(1, keepdims=True)
    return out, mass, score, top, own
