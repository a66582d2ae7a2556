"""Measured cases of the decoder-layer operators around the quantized matmuls: the RMS norm
with the residual's addition and an 8-bit output, the rotation and append of keys and values to
a paged 8-bit cache, and attention over that cache.

    listed()              the named cases
    draw(rng)             one more case of the same ranges
    prepare(case, seed)   the inputs and handles a serving program holds before the call
    run(state)            one pass (plain torch operations, or this package's kernels when `own`)
    exact(case, seed)     the operators' definition in 64 bits
    work(case)            the bytes and operations of one pass

Definitions (row-major tensors, T a 16-bit type):
  norm       h = T(x + residual); y = h / sqrt(mean(h^2) + eps) * gamma; scale = max|y| / qmax;
             code = round(y / scale), int8 (qmax 127) or e4m3 (qmax 448), one scale per token.
  append     the keys of a fused QKV row are rotated by the position's cos / sin; each page (block
             of tokens) and head has one scale = max(scale before, max|new values| / qmax), and the
             page's earlier codes are re-coded when it grows; the rotated queries are returned.
  attention  causal softmax(q k^T * sm_scale) v over the cached codes times their page's scale.
"""
import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one token of a decode step, in front of the QKV projection: latency
        _norm("norm one token", 1, 4096, "fp16", "int8", True),
        # a decode batch of the hidden size 3200, FP8 activations
        _norm("norm 128 tokens", 128, 3200, "bf16", "fp8", True),
        # a prefill chunk in front of the W4A8 projections
        _norm("norm prefill", 8192, 4096, "bf16", "int8", True),
        # a decode step of 16 sequences, as many key heads as query heads
        _kv("append decode", "append", 16, 1, 1, 100, 2000, 32, 32, 128, 16, "fp16", "int8", 128, "half"),
        # draft verification at head size 100: a few tokens each, pages that are partly filled
        _kv("append few tokens", "append", 48, 1, 6, 0, 1000, 32, 32, 100, 32, "bf16", "int8", 100, "half"),
        # ragged prefill chunks, grouped heads, half of each head rotated in adjacent pairs
        _kv("append prefill", "append", 6, 300, 2048, 0, 3000, 32, 8, 128, 64, "bf16", "fp8", 64, "pairs"),
        # one short sequence: latency
        _kv("attention one short", "attention", 1, 1, 1, 512, 512, 32, 32, 128, 16, "fp16", "int8"),
        # a ragged decode batch with grouped heads
        _kv("attention decode", "attention", 32, 1, 1, 100, 4095, 32, 8, 128, 32, "bf16", "int8"),
        # long contexts with few rows
        _kv("attention long", "attention", 2, 1, 1, 131000, 131071, 32, 8, 128, 64, "fp16", "fp8"),
        # draft verification at head size 100
        _kv("attention few tokens", "attention", 16, 2, 6, 300, 2000, 32, 32, 100, 32, "bf16", "int8"),
        # ragged prompts without a past
        _kv("attention prompts", "attention", 5, 100, 1100, 0, 0, 32, 32, 128, 16, "fp16", "int8"),
        # prefill chunks over a long past, grouped heads
        _kv("attention chunks", "attention", 2, 2048, 2048, 4096, 6000, 32, 8, 128, 64, "bf16", "fp8"),
    ]


def _norm(name, tokens, hidden, dtype, out, residual):
    return {"name": name, "op": "norm", "tokens": tokens, "hidden": hidden, "dtype": dtype, "out": out,
            "residual": residual}


def _kv(name, op, seqs, q_min, q_max, past_min, past_max, q_heads, kv_heads, head_dim, page, dtype, out, rope_dim=0,
        rope_style="half"):
    """`seqs` sequences that hold past_min..past_max tokens each and get q_min..q_max new ones."""
    c = {"name": name, "op": op, "seqs": seqs, "q_min": q_min, "q_max": q_max, "past_min": past_min,
         "past_max": past_max, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
         "dtype": dtype, "out": out}
    return dict(c, rope_dim=rope_dim, rope_style=rope_style) if op == "append" else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype, out = rng.choice(sorted(DT)), rng.choice(sorted(QMAX))
    op = rng.choice(["norm", "append", "append", "attention", "attention", "attention"])
    if op == "norm":
        hidden = 8 * _log(rng, 16, 1376)
        tokens = min(_log(rng, 1, 8192), 8192 * 4096 // hidden)
        c = _norm("", tokens, hidden, dtype, out, rng.random() < 0.8)
    else:
        kv_heads = rng.choice([1, 2, 4, 8, 32])
        q_heads = kv_heads * rng.choice([g for g in (1, 2, 4, 5, 8) if g * kv_heads <= 40])
        head_dim = rng.choice([64, 80, 100, 128, 128, 192, 256])
        page = rng.choice([16, 32, 64, 128])
        kind = rng.choice(["decode", "few", "chunk"])
        q_lo, q_hi = {"decode": (1, 1), "few": (1, 8), "chunk": (rng.randint(9, 200), rng.randint(200, 1500))}[kind]
        past = _log(rng, 16, 3000 if kind == "chunk" else 20000)
        seqs = _log(rng, 1, 6 if kind == "chunk" else 64)
        while seqs > 1 and seqs * (past + q_hi) * kv_heads * head_dim > (1 << 28):
            seqs //= 2
        if seqs * (past + q_hi) * kv_heads * head_dim > (1 << 28):
            past = (1 << 28) // (kv_heads * head_dim) - q_hi
        while seqs > 1 and seqs * q_hi * (past + q_hi) * q_heads > (1 << 29):
            seqs //= 2
        rope_dim = rng.choice([head_dim, head_dim, head_dim // 4 * 2, 0])
        c = _kv("", op, seqs, q_lo, q_hi, rng.randint(0, past), past, q_heads, kv_heads, head_dim, page, dtype, out,
                rope_dim, rng.choice(["half", "pairs"]))
    del c["name"]
    return c


def _lengths(case):
    """The (new, total) tokens of every sequence: fixed by the case, so that its work is too."""
    r = random.Random(1000003 * case["seqs"] + 1009 * case["past_max"] + 31 * case["q_max"] + case["head_dim"])
    new = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    return new, [n + r.randint(case["past_min"], case["past_max"]) for n in new]


def _pitch(head_dim):
    """Codes of one cached token and head: rounded up to whole 16-byte words."""
    return -(-head_dim // 16) * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dt = DT[case["dtype"]]
    st = {"op": case["op"], "out": case["out"], "dt": dt}
    if case["op"] == "norm":
        M, K = case["tokens"], case["hidden"]
        # a residual stream: some channels are much larger than the rest
        gain = 1 + 19 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        st["x"] = normal(M, K).to(dt)
        st["residual"] = (normal(M, K) * gain).to(dt) if case["residual"] else None
        st["gamma"] = (1 + 0.2 * normal(K)).to(dt)
        return st
    new, total = _lengths(case)
    B, ps, Hkv, D = case["seqs"], case["page"], case["kv_heads"], case["head_dim"]
    pages_of = [-(-t // ps) for t in total]
    used, width = sum(pages_of), max(pages_of)
    num_pages = used + 3
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    M = cu[-1]
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    n_pages = torch.tensor(pages_of, device="cuda")
    first = torch.cumsum(n_pages, 0) - n_pages
    at = (first[:, None] + col[None, :]).clamp(max=num_pages - 1)
    st["block_table"] = torch.where(col[None, :] < n_pages[:, None], order[at], 0).to(torch.int32).contiguous()
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["seq_len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    shape = (num_pages, Hkv, ps, _pitch(D))
    if case["out"] == "int8":
        def codes():
            c = torch.empty(shape, device="cuda", dtype=torch.float16).normal_(0, 36, generator=g)
            return c.round_().clamp_(-127, 127).to(torch.int8)
    else:
        def codes():
            c = torch.empty(shape, device="cuda", dtype=torch.float16).normal_(0, 130, generator=g)
            return c.clamp_(-448, 448).to(torch.float8_e4m3fn)
    st["k"], st["v"] = codes(), codes()
    st["k_scale"] = (0.5 + torch.rand(num_pages, Hkv, generator=g, device="cuda")) * (4 / QMAX[case["out"]])
    st["v_scale"] = (0.5 + torch.rand(num_pages, Hkv, generator=g, device="cuda")) * (4 / QMAX[case["out"]])
    st.update(q_heads=case["q_heads"], head_dim=D, width=max(new))
    if case["op"] == "append":
        Hq, r = case["q_heads"], case["rope_dim"]
        gain = 1 + 4 * (torch.rand((Hq + 2 * Hkv) * D, generator=g, device="cuda") < 0.02)
        st["qkv"] = (normal(M, (Hq + 2 * Hkv) * D) * gain).to(dt)
        st["style"] = case["rope_style"]
        st["rope"] = _rope_table(max(total), r) if r else None
    else:
        st["q"] = normal(M, case["q_heads"], D).to(dt)
        st["sm_scale"] = 1 / math.sqrt(D)
    if own:  # what a serving program holds from step to step: the cache's handle, the scratch
        import gemv_wq_quantize_b200 as wq
        st["cache"] = wq.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"], D)
        st["batch"] = wq.KVBatch(st["cu_q"], st["seq_len"], st["block_table"])
        if case["op"] == "attention":
            st["ws"] = wq.make_workspace(wq.kv_attention_workspace_size(M, case["q_heads"], st["cache"], st["batch"]))
    return st


def _rope_table(positions, r):
    """[positions, r] binary32: cos of the r/2 angles, then sin (base 10000, angles in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[st["op"]](st)


def _run_own(st):
    import gemv_wq_quantize_b200 as wq
    if st["op"] == "norm":
        f = wq.rmsnorm_quant_int8 if st["out"] == "int8" else wq.rmsnorm_quant_fp8
        codes, scale, h = f(st["x"], st["gamma"], EPS, residual=st["residual"])
        codes = codes if st["out"] == "int8" else codes.view(torch.float8_e4m3fn)
        return [codes, scale] if h is None else [codes, scale, h]
    if st["op"] == "append":
        q = wq.kv_append(st["qkv"], st["cache"], st["batch"], st["q_heads"], rope=st["rope"],
                         rope_style=wq.ROPE_HALF if st["style"] == "half" else wq.ROPE_PAIRS)
        return [q, st["k"], st["v"], st["k_scale"], st["v_scale"]]
    return wq.kv_attention(st["q"], st["cache"], st["batch"], sm_scale=st["sm_scale"], workspace=st["ws"])


def _encode(x, out):
    """Codes of x (binary32, already divided by its scale)."""
    q = QMAX[out]
    if out == "int8":
        return x.round().clamp(-q, q).to(torch.int8)
    return x.clamp(-q, q).to(torch.float8_e4m3fn)


def _ratio(x, s):
    """x / s, and 0 where s is 0."""
    return torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)


def _plain_norm(st):
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(st["dt"])
    # the mean in 64 bits: codes next to a border between two must not depend on its last bits
    mean = h.double().square().mean(1, keepdim=True)
    rstd = (1 / (mean + EPS).sqrt()).float()
    y = h.float() * rstd * st["gamma"].float()
    scale = y.abs().amax(1) / QMAX[st["out"]]
    codes = _encode(_ratio(y, scale[:, None]), st["out"])
    return [codes, scale] if st["residual"] is None else [codes, scale, h]


def _rotate(x, table, style):
    """x [M, H, D] binary32 with its first table.shape[1] values rotated (table: a row per token)."""
    r = table.shape[1]
    c, s = table[:, None, : r // 2], table[:, None, r // 2:]
    if style == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _places(st, M):
    """Sequence and position of every token."""
    cu = st["cu_q"].long()
    m = torch.arange(M, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), m, right=True)
    return b, st["seq_len"].long()[b] - cu[b + 1] + m


def _plain_append(st):
    D, ps, Hkv = st["head_dim"], st["k"].shape[2], st["k"].shape[1]
    Hq, M = st["q_heads"], st["qkv"].shape[0]
    b, pos = _places(st, M)
    page = st["block_table"].long()[b, pos // ps]
    off = pos % ps
    x = st["qkv"].float().view(M, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    if st["rope"] is not None:
        q, k = _rotate(q, st["rope"][pos], st["style"]), _rotate(k, st["rope"][pos], st["style"])
    num_pages = st["k"].shape[0]
    held = torch.full((num_pages,), ps, device=page.device).scatter_reduce(0, page, off, "amin")
    grown = page[(off == held[page]) & (off > 0)]  # pages that held tokens before
    keep = torch.arange(ps, device=page.device)[None, None, :, None] < held[grown][:, None, None, None]
    _plain_store(k, st["k"], st["k_scale"], page, off, grown, keep, D, st["out"])
    _plain_store(v, st["v"], st["v_scale"], page, off, grown, keep, D, st["out"])
    return [q.to(st["dt"]), st["k"], st["v"], st["k_scale"], st["v_scale"]]


def _plain_store(x, codes, scale, page, off, grown, keep, D, out):
    before = torch.zeros_like(scale)
    before[grown] = scale[grown]
    need = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    now = torch.maximum(before, need / QMAX[out])
    scale[page] = now[page]
    r = _ratio(before[grown], now[grown])[:, :, None, None]
    raw = codes.view(torch.int8)  # indexed stores on the codes' bytes
    old = codes[grown] if out == "int8" else raw[grown].view(codes.dtype)
    recoded = torch.where(keep & (r < 1), _encode(old.float() * r, out).view(torch.int8), raw[grown])
    raw[grown, :, :, :D] = recoded[..., :D]
    raw[page, :, off, :D] = _encode(_ratio(x, now[page][:, :, None]), out).view(torch.int8)


def _plain_attention(st):
    q, D = st["q"], st["head_dim"]
    M, Hq = q.shape[0], q.shape[1]
    ps, Hkv = st["k"].shape[2], st["k"].shape[1]
    B, W = st["block_table"].shape
    G, Q, L = Hq // Hkv, st["width"], W * ps
    b, pos = _places(st, M)
    row = torch.arange(M, device=q.device) - st["cu_q"].long()[b]
    grid = torch.zeros(B, Q, Hkv, G, D, device=q.device)
    grid[b, row] = q.float().view(M, Hkv, G, D)
    grid = grid.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    table = st["block_table"].long()

    def values(codes, scale):
        x = codes.view(torch.int8)[table].view(codes.dtype)[..., :D].float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, D)  # [B, W, Hkv, ps, D] -> tokens in order

    last = st["seq_len"].long() - (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    last = last[:, None] + torch.arange(Q, device=q.device)  # the last key of each row
    mask = torch.arange(L, device=q.device) <= last[:, :, None]
    mask = mask[:, None, :, None, :].expand(B, 1, Q, G, L).reshape(B, 1, Q * G, L)
    s = grid @ values(st["k"], st["k_scale"]).transpose(-1, -2)
    s = (s * st["sm_scale"]).masked_fill_(~mask, float("-inf"))
    s = (s - s.amax(-1, keepdim=True)).exp_()
    o = s @ values(st["v"], st["v_scale"]) / s.sum(-1, keepdim=True)
    return o.view(B, Hkv, Q, G, D).permute(0, 2, 1, 3, 4)[b, row].reshape(M, Hq, D).to(st["dt"])


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = (h + st["residual"].double()).to(st["dt"]).double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS) * st["gamma"].double()
        s = y.abs().max(1).values / QMAX[case["out"]]
        codes = _e4m3_grid(y / s.clamp(min=1e-300)[:, None]) if case["out"] == "fp8" else None
        return [codes, s] + ([] if st["residual"] is None else [h])
    new, total = _lengths(case)
    return (_exact_append if case["op"] == "append" else _exact_attention)(case, st, new, total)


def _e4m3_grid(x):
    """The nearest e4m3 value (ties to even) of |x| <= 448: steps of 2^(e - 3), at least 2^-9."""
    x = x.clamp(-448, 448)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_append(case, st, new, total):
    Hq, Hkv, D, ps, r = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"], case["rope_dim"]
    fp8, qmax = case["out"] == "fp8", QMAX[case["out"]]
    x = st["qkv"].double().view(-1, Hq + 2 * Hkv, D)
    at = torch.cat([torch.arange(t - n, t, device=x.device) for n, t in zip(new, total)])
    if r:
        tab = st["rope"].double()[at]
        turn = torch.complex(tab[:, : r // 2], tab[:, r // 2:])[:, None]
        qk = x[:, : Hq + Hkv, :r]
        if case["rope_style"] == "half":
            z = torch.complex(qk[..., : r // 2].contiguous(), qk[..., r // 2:].contiguous()) * turn
            x[:, : Hq + Hkv, :r] = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(qk.reshape(*qk.shape[:-1], r // 2, 2).contiguous()) * turn
            x[:, : Hq + Hkv, :r] = torch.view_as_real(z).flatten(-2)
    out = [x[:, :Hq]]
    table = st["block_table"].tolist()
    codes, scales = [], []
    for name, lo in (("k", Hq), ("v", Hq + Hkv)):
        scale = st[name + "_scale"].double()
        val = st[name].double() if fp8 else None
        m = 0
        for b, (n, t) in enumerate(zip(new, total)):
            p = t - n
            while p < t:
                page, o, e = table[b][p // ps], p % ps, min(t, (p // ps + 1) * ps)
                part = x[m: m + e - p, lo: lo + Hkv].transpose(0, 1)  # [Hkv, tokens, D]
                need = part.abs().amax((1, 2)) / qmax
                s = torch.maximum(scale[page], need) if o else need
                if fp8:
                    if o:
                        old = _e4m3_grid(val[page, :, :o, :D] * (scale[page] / s)[:, None, None])
                        val[page, :, :o, :D] = torch.where((s > scale[page])[:, None, None], old, val[page, :, :o, :D])
                    val[page, :, o: o + e - p, :D] = _e4m3_grid(part / s[:, None, None])
                scale[page] = s
                m, p = m + e - p, e
        codes.append(val)
        scales.append(scale)
    return out + codes + scales


def _exact_attention(case, st, new, total):
    Hq, Hkv, D, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if sum(n * t for n, t in zip(new, total)) * Hq * D > 1 << 40:
        return None
    out, m, table = [], 0, st["block_table"].long()
    for b, (n, t) in enumerate(zip(new, total)):
        pages = table[b, : -(-t // ps)]
        k, v = ((st[c][pages] if st[c].dtype == torch.int8 else st[c].view(torch.uint8)[pages].view(st[c].dtype))
                for c in ("k", "v"))
        seen = torch.arange(t, device=pages.device)[None] <= torch.arange(t - n, t, device=pages.device)[:, None]
        heads = []
        for h in range(Hq):
            j = h // (Hq // Hkv)
            kh = (k[:, j, :, :D].double() * st["k_scale"][pages, j].double()[:, None, None]).reshape(-1, D)[:t]
            vh = (v[:, j, :, :D].double() * st["v_scale"][pages, j].double()[:, None, None]).reshape(-1, D)[:t]
            w = torch.where(seen, st["q"][m: m + n, h].double() @ kh.T * st["sm_scale"], -math.inf)
            heads.append(torch.softmax(w, 1) @ vh)
        out.append(torch.stack(heads, 1))
        m += n
    return torch.cat(out)


# ---------------------------------------------------------------- bytes and operations of one pass
def work(case):
    if case["op"] == "norm":
        M, K = case["tokens"], case["hidden"]
        return {"bytes": M * K * (7 if case["residual"] else 3) + 2 * K + 4 * M, "flops": 6 * M * K}
    new, total = _lengths(case)
    M, D, Hq, Hkv, ps = sum(new), case["head_dim"], case["q_heads"], case["kv_heads"], case["page"]
    if case["op"] == "append":
        pages = sum((t - 1) // ps - (t - n) // ps + 1 for n, t in zip(new, total))
        return {"bytes": M * D * (4 * Hq + 6 * Hkv) + 4 * M * case["rope_dim"] + 8 * pages * Hkv,
                "flops": M * (3 * case["rope_dim"] * (Hq + Hkv) + 6 * D * Hkv)}
    pages = sum(-(-t // ps) for t in total)
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
    return {"bytes": sum(total) * Hkv * D * 2 + 8 * pages * Hkv + 4 * M * Hq * D + 4 * pages,
            "flops": 4 * D * Hq * pairs}
